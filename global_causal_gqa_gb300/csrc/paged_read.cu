// paged_read.cu -- the 8-bit paged cache read back into bf16: the last tokens of every sequence
// into packed rows, or (for the tile attention kernel) all keys a call can see into pages of 128.
//
// value = y * 2^(byte - 127) (q8.cuh), exact in bf16 but at the ends of its range.  A pass over
// memory: d + 1 bytes in and 2 d out per vector.  A thread takes 8 numbers of a key and the same
// of its value: 8-byte loads, 16-byte stores, whole 128-byte lines where vectors have 128 numbers.
#include <cuda_runtime.h>

#include "internal.h"
#include "packed.cuh"
#include "q8.cuh"

namespace gqa {
namespace {

constexpr int kReadThreads = 256;
constexpr int kReadTokens = 8;       // packed rows of a block, one per warp to look up
constexpr int kPageTokens = 32;      // keys of a block that fills pages
constexpr int kSite = kDiagCache << 24;   // of the debug build's checks

struct ReadParams {
    const uint2 *k, *v;
    const uint16_t *scales;          // key's byte, value's byte
    const int32_t *cu, *kv_lens, *pages;
    PackedBounds bounds;
    int nseq, Hkv, num_pages, page_size, max_pages;
    uint4 *k_out, *v_out;
    long k_stride, v_stride;         // in 16-byte chunks
    // pages of 128 keys: [nseq, out_pages, Hkv, 128, d] and their table, the identity
    int32_t *out_table;
    int out_pages, window;
    int *status;
};

// The page of position pos of sequence i; -1 (recorded): outside the pool.
__device__ __forceinline__ int page_of(const ReadParams &p, int i, int pos) {
    if (!GQA_IN_BOUNDS(pos / p.page_size, p.max_pages, p.status, kSite | 10)) return -1;
    const int page = __ldg(p.pages + (long)i * p.max_pages + pos / p.page_size);
    if (page >= 0 && page < p.num_pages) return page;
    set_status(p.status, GQA_ERR_INVALID_ARG);
    return -1;
}

// 8 numbers of a pool, times the power of two that `byte` stands for.
__device__ __forceinline__ void read_chunk(const uint2 *pool, long at, uint32_t byte, uint4 *dst) {
    const uint2 w = __ldcs(pool + at);
    const float f = scale_of(byte);
    const uint2 a = e4m3x4_bf16(w.x, f), b = e4m3x4_bf16(w.y, f);
    *dst = make_uint4(a.x, a.y, b.x, b.y);
}

// PAGES: into pages of 128 keys; else into packed rows.  D: head dim.
template <int D, bool PAGES>
__global__ void __launch_bounds__(kReadThreads) paged_read_kernel(const ReadParams p) {
    constexpr int C = D / 8;
    constexpr int kTokens = PAGES ? kPageTokens : kReadTokens;
    griddep_wait();
    griddep_launch_dependents();
    __shared__ long s_slot[kTokens];     // vector of head 0; -1: outside the pool
    __shared__ int s_on[kTokens];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int blocks = PAGES ? p.out_pages * (128 / kTokens) : 1;   // of a sequence
    const int seq = PAGES ? blockIdx.x / blocks : 0;
    const int first = (PAGES ? blockIdx.x - seq * blocks : blockIdx.x) * kTokens;
    if (PAGES) {
        if (warp == 0) {
            const PackedSeq s = packed_seq(p.cu, p.kv_lens, seq, p.bounds, p.status);
            const int lo = p.window > 0 ? max(0, s.S - s.T - p.window + 1) : 0;
            const int key = first + lane;
            s_on[lane] = s.T > 0 && key >= lo && key < s.S;
            if (s_on[lane]) {
                const int page = page_of(p, seq, key);
                s_slot[lane] = page < 0 ? -1 : (long)page * p.Hkv * p.page_size + key % p.page_size;
            }
            if (lane == 0 && first % 128 == 0)
                p.out_table[(long)seq * p.out_pages + first / 128] = seq * p.out_pages + first / 128;
        }
    } else {
        const int row = first + warp;
        int i = 0;
        if (row < p.bounds.total) i = packed_row_seq(p.cu, p.nseq, row);
        if (lane == 0) {
            s_on[warp] = 0;
            if (row < p.bounds.total && i < p.nseq) {
                const PackedSeq s = packed_seq(p.cu, p.kv_lens, i, p.bounds, p.status);
                if (row >= s.row0 && row < s.row0 + s.T) {
                    const int pos = s.S - s.T + (row - s.row0), page = page_of(p, i, pos);
                    s_on[warp] = 1;
                    s_slot[warp] = page < 0 ? -1 : (long)page * p.Hkv * p.page_size + pos % p.page_size;
                }
            }
        }
        // every sequence is looked over, also those that no row falls to
        for (long n = (long)blockIdx.x * blockDim.x + threadIdx.x; n < p.nseq;
             n += (long)gridDim.x * blockDim.x)
            packed_seq(p.cu, p.kv_lens, static_cast<int>(n), p.bounds, p.status);
    }
    __syncthreads();
    const int per = p.Hkv * C;
#pragma unroll 4
    for (int u = threadIdx.x; u < kTokens * per; u += kReadThreads) {
        const int t = u / per, r = u - t * per, h = r / C, c = r - h * C;
        if (!s_on[t]) continue;
        uint4 *kd, *vd;
        if (PAGES) {
            const int key = first + t;
            const long at = ((((long)seq * p.out_pages + key / 128) * p.Hkv + h) * 128 + key % 128) * C + c;
            kd = p.k_out + at;
            vd = p.v_out + at;
        } else {
            kd = p.k_out ? p.k_out + (long)(first + t) * p.k_stride + r : nullptr;
            vd = p.v_out ? p.v_out + (long)(first + t) * p.v_stride + r : nullptr;
        }
        const long slot = s_slot[t] < 0 ? -1 : s_slot[t] + (long)h * p.page_size;
        if (slot < 0 || !GQA_IN_BOUNDS(slot, (long)p.num_pages * p.Hkv * p.page_size, p.status,
                                       kSite | 11)) {
            if (kd) *kd = make_uint4(0, 0, 0, 0);
            if (vd) *vd = make_uint4(0, 0, 0, 0);
            continue;
        }
        const uint32_t bytes = __ldg(p.scales + slot);
        if (kd) read_chunk(p.k, slot * C + c, bytes & 255u, kd);
        if (vd) read_chunk(p.v, slot * C + c, bytes >> 8, vd);
    }
}

ReadParams read_params(const gqa_paged_kv_q8 &c, const int32_t *cu, int nseq, int *status) {
    ReadParams p{};
    p.k = static_cast<const uint2 *>(c.k);
    p.v = static_cast<const uint2 *>(c.v);
    p.scales = static_cast<const uint16_t *>(c.scales);
    p.cu = cu;
    p.kv_lens = c.kv_lens;
    p.pages = c.page_table;
    p.nseq = nseq;
    p.Hkv = c.Hkv;
    p.num_pages = c.num_pages;
    p.page_size = c.page_size;
    p.max_pages = c.max_pages;
    p.status = status;
    return p;
}

}  // namespace

cudaError_t launch_paged_read_q8(const gqa_paged_kv_q8 &c, const int32_t *cu, int nseq, int total,
                                 void *k_out, int64_t k_stride, void *v_out, int64_t v_stride,
                                 int *status, cudaStream_t s) {
    ReadParams p = read_params(c, cu, nseq, status);
    p.bounds = {total, total, 0x7fffffff, (long)c.max_pages * c.page_size};
    p.k_out = static_cast<uint4 *>(k_out);
    p.v_out = static_cast<uint4 *>(v_out);
    p.k_stride = k_stride / 8;
    p.v_stride = v_stride / 8;
    auto kern = c.d == 64    ? paged_read_kernel<64, false>
                : c.d == 128 ? paged_read_kernel<128, false>
                : c.d == 256 ? paged_read_kernel<256, false>
                             : paged_read_kernel<512, false>;
    return launch_pdl(kern, dim3((total + kReadTokens - 1) / kReadTokens), dim3(kReadThreads), 0, s,
                      p);
}

// Pages, their table's numbers and the grid are counted in 32 bits.
bool paged_expand_counts_fit(int nseq, int max_kv, int Hkv) {
    const long pages = (long)nseq * ((max_kv + 127) / 128);
    return pages * (128 / kPageTokens) <= 0x7fffffffL && pages * Hkv <= 0x7fffffffL;
}

size_t paged_expand_q8_bytes(int nseq, int max_kv, int Hkv) {
    const size_t pages = (size_t)nseq * ((max_kv + 127) / 128);
    return 2 * pages * Hkv * 128 * 128 * 2 + ((pages * 4 + 127) & ~(size_t)127);
}

cudaError_t launch_paged_expand_q8(const gqa_paged_kv_q8 &c, const PackedAttn &a, void *ws,
                                   gqa_paged_kv *out, int *status, cudaStream_t s) {
    ReadParams p = read_params(c, a.cu, a.nseq, status);
    p.bounds = {a.total, a.max_q, a.max_kv, (long)c.max_pages * c.page_size};
    p.window = a.window;
    p.out_pages = (a.max_kv + 127) / 128;
    const size_t pages = (size_t)a.nseq * p.out_pages, bytes = pages * c.Hkv * 128 * 128 * 2;
    p.k_out = static_cast<uint4 *>(ws);
    p.v_out = reinterpret_cast<uint4 *>(static_cast<char *>(ws) + bytes);
    p.out_table = reinterpret_cast<int32_t *>(static_cast<char *>(ws) + 2 * bytes);
    *out = {p.k_out, p.v_out, p.out_table, c.kv_lens, static_cast<int32_t>(pages), c.Hkv, 128, 128,
            p.out_pages, 0};
    return launch_pdl(paged_read_kernel<128, true>,
                      dim3(static_cast<unsigned>(pages * (128 / kPageTokens))), dim3(kReadThreads),
                      0, s, p);
}

}  // namespace gqa
