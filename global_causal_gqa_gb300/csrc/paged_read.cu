// paged_read.cu -- the 8-bit paged cache read back into bf16: the last tokens of every sequence
// into packed rows, or (for the tile attention kernel) all keys a call can see into pages of 128.
//
// value = y * 2^(byte - 127) (q8.cuh), exact in bf16 but at the ends of its range.  A pass over
// memory: d + 1 bytes in and 2 d out per vector.  A warp takes a row, a thread 8 numbers of a key and
// the same of its value at a time: 8-byte loads, 16-byte stores, whole 128-byte lines where vectors
// have 128 numbers.  36469 rows of 8 heads of 128 take 37 us (6.1 TB/s), eight times as many 246 us
// (6.7 TB/s); with the stores after each load, as the compiler orders them by itself, 49 and 308;
// blocks of 512 threads 51, stores that bypass L2's order of use 48.
#include <cuda_runtime.h>

#include "internal.h"
#include "packed.cuh"
#include "q8.cuh"

namespace gqa {
namespace {

constexpr int kReadThreads = 128;
constexpr int kBatch = 4;            // units of a thread in flight
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

// 8 numbers times the power of two that `byte` stands for, as bf16.
__device__ __forceinline__ uint4 read_chunk(const uint2 &w, uint32_t byte) {
    const float f = scale_of(byte);
    const uint2 a = e4m3x4_bf16(w.x, f), b = e4m3x4_bf16(w.y, f);
    return make_uint4(a.x, a.y, b.x, b.y);
}
__device__ __forceinline__ uint2 load_once(const uint2 *p) {
    uint2 v;
    asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
    return v;
}

// The units u0, u0 + step, .. of a vector row of `per` units (heads of 8 numbers each), kBatch of
// them with all their loads before the first store (the compiler may not move a load up past one).
// slot: the vector of head 0, or -1: zeros.  kd, vd: the row's place, or nullptr; `apart`: chunks
// from a head's vector to the next one's there.
template <int D>
__device__ __forceinline__ void read_row(const ReadParams &p, long slot, int u0, int step, uint4 *kd,
                                         uint4 *vd, int apart) {
    constexpr int C = D / 8;
    const int per = p.Hkv * C;
#pragma unroll 1
    for (; u0 < per; u0 += kBatch * step) {
        uint2 kw[kBatch], vw[kBatch];
        uint32_t bytes[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int u = u0 + i * step, h = u / C;
            kw[i] = vw[i] = make_uint2(0, 0);
            bytes[i] = 0x7f7f;
            const long at = slot + (long)h * p.page_size;
            if (u >= per || slot < 0 ||
                !GQA_IN_BOUNDS(at, (long)p.num_pages * p.Hkv * p.page_size, p.status, kSite | 11))
                continue;
            bytes[i] = __ldg(p.scales + at);
            if (kd) kw[i] = load_once(p.k + at * C + u % C);
            if (vd) vw[i] = load_once(p.v + at * C + u % C);
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int u = u0 + i * step;
            if (u >= per) continue;
            const long to = (long)(u / C) * apart + u % C;
            if (kd) kd[to] = read_chunk(kw[i], bytes[i] & 255u);
            if (vd) vd[to] = read_chunk(vw[i], bytes[i] >> 8);
        }
    }
}

// Packed rows, a warp each.
template <int D>
__global__ void __launch_bounds__(kReadThreads) paged_read_kernel(const ReadParams p) {
    griddep_wait();
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31;
    // every sequence is looked over, also those that no row falls to
    for (long n = (long)blockIdx.x * blockDim.x + threadIdx.x; n < p.nseq;
         n += (long)gridDim.x * blockDim.x)
        packed_seq(p.cu, p.kv_lens, static_cast<int>(n), p.bounds, p.status);
    const int row = static_cast<int>(blockIdx.x) * (kReadThreads / 32) + (threadIdx.x >> 5);
    if (row >= p.bounds.total) return;
    const int i = packed_row_seq(p.cu, p.nseq, row);
    if (i >= p.nseq) return;
    const PackedSeq s = packed_seq(p.cu, p.kv_lens, i, p.bounds, lane == 0 ? p.status : nullptr);
    if (row < s.row0 || row >= s.row0 + s.T) return;
    const int pos = s.S - s.T + (row - s.row0), page = page_of(p, i, pos);
    read_row<D>(p, page < 0 ? -1 : (long)page * p.Hkv * p.page_size + pos % p.page_size, lane, 32,
                p.k_out ? p.k_out + row * p.k_stride : nullptr,
                p.v_out ? p.v_out + row * p.v_stride : nullptr, D / 8);
}

// All keys that a call sees into pages of 128, a warp each.
__global__ void __launch_bounds__(kReadThreads) paged_expand_kernel(const ReadParams p) {
    constexpr int C = 128 / 8;
    griddep_wait();
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31, keys = kReadThreads / 32, blocks = p.out_pages * (128 / keys);
    const int seq = blockIdx.x / blocks, key0 = (blockIdx.x - seq * blocks) * keys;
    const int key = key0 + (threadIdx.x >> 5), to = seq * p.out_pages + key / 128;
    if (threadIdx.x == 0 && key % 128 == 0) p.out_table[to] = to;
    const PackedSeq s = packed_seq(p.cu, p.kv_lens, seq, p.bounds, lane == 0 ? p.status : nullptr);
    const int lo = p.window > 0 ? max(0, s.S - s.T - p.window + 1) : 0;
    if (s.T == 0 || key < lo || key >= s.S) return;
    const int page = page_of(p, seq, key);
    const long at = (long)to * p.Hkv * 128 * C + key % 128 * C;
    read_row<128>(p, page < 0 ? -1 : (long)page * p.Hkv * p.page_size + key % p.page_size, lane, 32,
                  p.k_out + at, p.v_out + at, 128 * C);
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
    auto kern = c.d == 64    ? paged_read_kernel<64>
                : c.d == 128 ? paged_read_kernel<128>
                : c.d == 256 ? paged_read_kernel<256>
                             : paged_read_kernel<512>;
    constexpr int rows = kReadThreads / 32;
    return launch_pdl(kern, dim3((total + rows - 1) / rows), dim3(kReadThreads), 0, s, p);
}

// Pages, their table's numbers and the grid are counted in 32 bits.
bool paged_expand_counts_fit(int nseq, int max_kv, int Hkv) {
    const long pages = (long)nseq * ((max_kv + 127) / 128);
    return pages * (128 / (kReadThreads / 32)) <= 0x7fffffffL && pages * Hkv <= 0x7fffffffL;
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
    return launch_pdl(paged_expand_kernel,
                      dim3(static_cast<unsigned>(pages * (128 / (kReadThreads / 32)))),
                      dim3(kReadThreads), 0, s, p);
}

}  // namespace gqa
