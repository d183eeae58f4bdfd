// packed_append.cu -- Q/K RMSNorm, RoPE and the write into the paged cache for the new tokens
// of a packed batch.
//
// "PLaMo 3アーキテクチャ徹底解析" §3.2, §4.3, §6.1: with x one (token, head) vector of d
// values, position p and the table's (c_j, s_j) = amp (cos p w_j, sin p w_j),
//   n = gamma * x / sqrt(mean(x^2) + eps)            (without a gain: n = x)
//   y_j = n_j c_j - n_{j+d/2} s_j,   y_{j+d/2} = n_j s_j + n_{j+d/2} c_j,  j < d/2,
// in fp32 with one rounding to bf16.  q goes to q_out; the key goes to its sequence's page
// (and to k_out), v is copied to the page.
//
// The work is a pass over memory: 2 (Hq + 2 Hkv) d bf16 values per token, each read and
// written once.  A vector is held by d/16 lanes, each with the two 16-byte chunks whose
// elements pair up under RoPE, so the norm is a shuffle reduction and the rotation stays in
// the thread.  Two kernels share this.  Up to 608 tokens latency counts: a block or less per
// token, whose threads walk its vectors, q heads, k heads, v heads, straight from and to global
// memory (256 tokens of 32 + 8 + 8 heads of 128: 5.2 us).  More tokens are streamed through
// shared memory by bulk copies, with two blocks of 110 KB per SM in flight (16384 tokens of 64 +
// 8 + 8 heads: 117 us with the norms and 108 without, 5.7 and 6.2 TB/s; the first kernel, with
// four blocks per SM, took 124 and 112, and at 1024 tokens 9.7 instead of 9.1).
//
// An 8-bit cache (q8.cuh) takes the same two kernels with another store: a vector's largest
// magnitude is one more shuffle reduction over its lanes, and each lane writes 8 numbers of either
// chunk (15424 tokens of 64 + 8 + 8 heads with the norms: 108 us, 5.6 TB/s).
#include <cuda_runtime.h>
#include <type_traits>

#include "internal.h"
#include "packed.cuh"
#include "q8.cuh"

namespace gqa {
namespace {

constexpr int kAppendThreads = 256;
constexpr int kAppendTokens = 8;   // most tokens of one block: one per warp to look up
constexpr int kFewTokens = 4 * 152;   // up to here: a block or less per token

struct AppendParams {
    const uint4 *q, *k, *v;
    long q_stride, k_stride, v_stride;   // in 16-byte chunks
    const int32_t *cu, *kv_lens, *pages;
    PackedBounds bounds;
    int nseq, Hq, Hkv, table_len, num_pages, page_size, max_pages;
    const float4 *q_gamma, *k_gamma;
    const float4 *table;
    float eps;
    uint4 *q_out, *k_out, *k_pool, *v_pool;
    uint8_t *scales;                     // of an 8-bit cache
    int *status;
};

// A lane's part of a vector of D values in pairs of neighbours: x[i] = elements 8c + 2i, + 1 of
// its chunk c, y[i] those D/2 on.
struct Vec {
    float2 x[4], y[4];
    __device__ __forceinline__ Vec(const uint4 &a, const uint4 &b) {
        const uint32_t aw[4] = {a.x, a.y, a.z, a.w}, bw[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[i] = make_float2(bf16lo(aw[i]), bf16hi(aw[i]));
            y[i] = make_float2(bf16lo(bw[i]), bf16hi(bw[i]));
        }
    }
    // 1 / sqrt(mean(x^2) + eps) over the vector's lanes (every lane of the warp shuffles)
    template <int D>
    __device__ __forceinline__ float inverse_norm(float eps) const {
        float2 s2 = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < 4; ++i) s2 = ffma2v(x[i], x[i], ffma2v(y[i], y[i], s2));
        float ss = s2.x + s2.y;
#pragma unroll
        for (int o = 1; o < D / 16; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        return rsqrtf(ss * (1.0f / D) + eps);   // off by 2^-22 at most
    }
    // The lane's elements in an 8-bit page and, from the first lane, their power of two: the vector
    // begins at row `slot` of the pools' vectors (every lane of the warp shuffles; `store`: this
    // one writes).
    template <int D>
    __device__ __forceinline__ void store_q8(const AppendParams &p, bool key, long slot, int c,
                                             bool store) const {
        constexpr int L = D / 16;
        float most = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            most = amax_nan(most, amax_nan(amax_nan(x[i].x, x[i].y), amax_nan(y[i].x, y[i].y)));
#pragma unroll
        for (int o = 1; o < L; o <<= 1) most = amax_nan(most, __shfl_xor_sync(0xffffffffu, most, o));
        if (!store) return;
        const uint32_t byte = scale_byte(most);
        const float f = inverse_scale(byte);
        uint32_t w[4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float2 *z = h ? y : x;
#pragma unroll
            for (int i = 0; i < 2; ++i)
                w[2 * h + i] = to_e4m3x2(z[2 * i].x * f, z[2 * i].y * f) |
                               to_e4m3x2(z[2 * i + 1].x * f, z[2 * i + 1].y * f) << 16;
        }
        uint2 *d = reinterpret_cast<uint2 *>(key ? p.k_pool : p.v_pool) + slot * (D / 8) + c;
        // (a vector that is not finite is stored as zeros: inf and NaN times f = 0 are not)
        d[0] = byte == kScaleNan ? make_uint2(0, 0) : make_uint2(w[0], w[1]);
        d[L] = byte == kScaleNan ? make_uint2(0, 0) : make_uint2(w[2], w[3]);
        if (c == 0) p.scales[2 * slot + (key ? 0 : 1)] = static_cast<uint8_t>(byte);
    }
    // times r and the gain's elements in the same places
    __device__ __forceinline__ void scale(float r, const float4 (&ga)[2], const float4 (&gb)[2]) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            x[2 * i] = fmul2(x[2 * i], make_float2(r * ga[i].x, r * ga[i].y));
            x[2 * i + 1] = fmul2(x[2 * i + 1], make_float2(r * ga[i].z, r * ga[i].w));
            y[2 * i] = fmul2(y[2 * i], make_float2(r * gb[i].x, r * gb[i].y));
            y[2 * i + 1] = fmul2(y[2 * i + 1], make_float2(r * gb[i].z, r * gb[i].w));
        }
    }
};

// The table's cos and sin of a lane's pairs 8c + 2i, + 1, and the rotation by them.
struct Rotation {
    float2 co[4], si[4];
    __device__ __forceinline__ void set(int i, const float4 &w) {
        co[i] = make_float2(w.x, w.z);
        si[i] = make_float2(w.y, w.w);
    }
    __device__ __forceinline__ void apply(Vec &v, uint4 &a, uint4 &b) const {
        uint32_t ao[4], bo[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 ra = fsub2(fmul2(v.x[i], co[i]), fmul2(v.y[i], si[i]));
            const float2 rb = ffma2v(v.x[i], si[i], fmul2(v.y[i], co[i]));
            v.x[i] = ra;
            v.y[i] = rb;
            ao[i] = pack_bf16x2(ra.x, ra.y);
            bo[i] = pack_bf16x2(rb.x, rb.y);
        }
        a = make_uint4(ao[0], ao[1], ao[2], ao[3]);
        b = make_uint4(bo[0], bo[1], bo[2], bo[3]);
    }
};

constexpr int kSite = kDiagCache << 24;   // of the debug build's checks
// Whether a token's rows and its table row are where they may be (the debug build's check).
__device__ __forceinline__ bool token_in_bounds(const AppendParams &p, long row, int pos) {
    return GQA_IN_BOUNDS(row, p.bounds.total, p.status, kSite | 7) &&
           GQA_IN_BOUNDS(pos, p.table_len, p.status, kSite | 8);
}
__device__ __forceinline__ bool slot_in_bounds(const AppendParams &p, long slot) {
    return GQA_IN_BOUNDS(slot, (long)p.num_pages * p.Hkv * p.page_size, p.status, kSite | 9);
}

// What a token at `row` of sequence i meets: its position (-1: nothing to do for it) and its
// page (-1: outside the pool).
__device__ __forceinline__ void find_token(const AppendParams &p, int row, int i, int &pos, int &page) {
    pos = page = -1;
    if (i >= p.nseq) return;
    const PackedSeq s = packed_seq(p.cu, p.kv_lens, i, p.bounds, p.status);
    if (row < s.row0 || row >= s.row0 + s.T) return;
    pos = s.S - s.T + (row - s.row0);
    if (pos >= p.table_len) {
        set_status(p.status, GQA_ERR_RANGE);
        pos = -1;
    } else if (p.pages && GQA_IN_BOUNDS(pos / p.page_size, p.max_pages, p.status, kSite | 6)) {
        page = __ldg(p.pages + (long)i * p.max_pages + pos / p.page_size);
        if (page < 0 || page >= p.num_pages) {
            set_status(p.status, GQA_ERR_INVALID_ARG);
            page = -1;
        }
    }
}

// Looks every sequence over, a thread each from the first blocks' last ones: numbers that
// contradict one another are recorded even where no row falls to them.
__device__ __forceinline__ void check_sequences(const AppendParams &p) {
    for (long i = (long)blockIdx.x * blockDim.x + blockDim.x - 1 - threadIdx.x; i < p.nseq;
         i += (long)gridDim.x * blockDim.x)
        packed_seq(p.cu, p.kv_lens, static_cast<int>(i), p.bounds, p.status);
}

// D: head dim.  `per` threads (a multiple of the D / 16 lanes of a vector) serve one token at
// a time, the block's kAppendThreads / per groups take its `tokens` tokens in turn.  Q8: the pools
// are an 8-bit cache's.
template <int D, bool Q8>
__global__ void __launch_bounds__(kAppendThreads, 4)
    packed_rope_append_kernel(const AppendParams p, int tokens, int per) {
    constexpr int L = D / 16;    // lanes of a vector; also the distance of a pair's chunks
    constexpr int C = D / 8;     // 16-byte chunks of a vector
    griddep_wait();
    griddep_launch_dependents();   // the host launches no more blocks than are resident at once
    __shared__ int s_pos[kAppendTokens];     // position; -1: nothing to do for this token
    __shared__ int s_page[kAppendTokens];    // page; -1: outside the pool
    const int row_base = blockIdx.x * tokens;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (warp < tokens) {
        const int row = row_base + warp;
        int pos = -1, page = -1;
        if (row < p.bounds.total) {
            const int i = packed_row_seq(p.cu, p.nseq, row);
            if (lane == 0) find_token(p, row, i, pos, page);
        }
        if (lane == 0) {
            s_pos[warp] = pos;
            s_page[warp] = page;
        }
    }
    check_sequences(p);
    __syncthreads();

    const int group = threadIdx.x / per, groups = kAppendThreads / per;
    const int tid = threadIdx.x - group * per;
    const int c = tid % L, u0 = tid / L, step = per / L;
    for (int t = group; t < tokens; t += groups) {
        const int pos = s_pos[t], page = s_page[t];
        if (pos < 0) continue;   // the same for the whole group, which is whole vectors
        const long row = row_base + t;
        if (!token_in_bounds(p, row, pos)) continue;
        Rotation rot;
        const float4 *tr = p.table + (long)pos * (D / 4) + 4 * c;
#pragma unroll
        for (int i = 0; i < 4; ++i) rot.set(i, __ldg(tr + i));
        auto normalise = [&](Vec &v, const float4 *gamma, bool on) {
            const float r = v.template inverse_norm<D>(p.eps);
            if (!on) return;
            const float4 ga[2] = {__ldg(gamma + 2 * c), __ldg(gamma + 2 * c + 1)};
            const float4 gb[2] = {__ldg(gamma + 2 * (c + L)), __ldg(gamma + 2 * (c + L) + 1)};
            v.scale(r, ga, gb);
        };
        // Queries, then keys and values.  Every lane of a warp makes the same number of turns
        // (the norm shuffles), past the last vector on the last one, without storing.
        const uint4 *src = p.q + row * p.q_stride + c;
        uint4 *dst = p.q_out + row * p.Hq * C + c;
        for (int ub = 0; ub < p.Hq; ub += step) {
            const int u = min(ub + u0, p.Hq - 1);
            uint4 a = __ldg(src + (long)u * C), b = __ldg(src + (long)u * C + L);
            Vec v(a, b);
            if (p.q_gamma) normalise(v, p.q_gamma, true);
            rot.apply(v, a, b);
            if (ub + u0 < p.Hq) {
                dst[(long)u * C] = a;
                dst[(long)u * C + L] = b;
            }
        }
        const int heads = p.v_pool ? 2 * p.Hkv : p.Hkv;
        const long slot = p.page_size ? ((long)page * p.Hkv * p.page_size + pos % p.page_size) : 0;
        for (int ub = 0; ub < heads; ub += step) {
            const int u = min(ub + u0, heads - 1);
            const bool isk = u < p.Hkv;
            const int g = isk ? u : u - p.Hkv;
            const uint4 *s = (isk ? p.k + row * p.k_stride : p.v + row * p.v_stride) + (long)g * C + c;
            uint4 a = __ldg(s), b = __ldg(s + L);
            Vec v(a, b);
            if (p.k_gamma) normalise(v, p.k_gamma, isk);
            if (isk) rot.apply(v, a, b);
            if constexpr (Q8)
                v.template store_q8<D>(p, isk, slot + (long)g * p.page_size, c,
                                       ub + u0 < heads && page >= 0 &&
                                           slot_in_bounds(p, slot + (long)g * p.page_size));
            if (ub + u0 >= heads) continue;
            if (!Q8 && page >= 0 && p.k_pool && slot_in_bounds(p, slot + (long)g * p.page_size)) {
                uint4 *d = (isk ? p.k_pool : p.v_pool) + (slot + (long)g * p.page_size) * C + c;
                d[0] = a;
                d[L] = b;
            }
            if (isk && p.k_out) {
                uint4 *d = p.k_out + (row * p.Hkv + g) * C + c;
                d[0] = a;
                d[L] = b;
            }
        }
    }
}

// The same for a batch that keeps every SM busy for long: a CTA streams its run of tokens
// through shared memory.  A unit of work is a token, or one of `parts` runs of its vectors (q
// heads, k heads, v heads, `per` of them each) where a whole token would take too much of it.
// Each warp has a place of its own for the vectors and the table row and takes every 8th unit:
// bulk copies in, norm and rotation in place, bulk copies out, q and k_out as they lie, keys and
// values head by head to their page.  Runs are short where there are many, since equal runs are
// not equal times (one run per SM for the 16384 tokens: 131 us); three blocks of 74 KB per SM
// with 80 registers: 121 us.
constexpr int kStreamPlaces = 8;             // warps of a CTA, of which an SM takes two
constexpr int kPlaceBytes = 13824;
constexpr int kStreamBytes = kStreamPlaces * kPlaceBytes;
constexpr int kStreamSmem = kStreamBytes + kStreamPlaces * 8 + 128;

template <int D, bool Q8>
__global__ void __launch_bounds__(32 * kStreamPlaces, 2)
    packed_append_stream_kernel(const AppendParams p, int parts, int per, int run) {
    constexpr int L = D / 16, V = 32 / L;    // lanes of a vector, vectors of a warp
    constexpr int C = D / 8, kVec = D * 2;   // 16-byte chunks and bytes of a vector
    griddep_wait();
    if (gridDim.x <= 2 * 152) griddep_launch_dependents();
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    uint8_t *ring = smem_raw + (((raw + 127u) & ~127u) - raw);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint64_t *full = reinterpret_cast<uint64_t *>(ring + kStreamBytes) + warp;
    uint8_t *place = ring + warp * kPlaceBytes, *table = place + per * kVec;
    if (lane == 0) {
        mbar_init(full, 1);
        fence_mbar_init();
    }
    __syncwarp();
    const int nq = p.q ? p.Hq : 0, nk = nq + p.Hkv, nv = p.v_pool ? nk + p.Hkv : nk;
    const int c = lane % L;
    float4 gain[2][2][2];                    // [q, k][half][chunk's elements]
#pragma unroll
    for (int w = 0; w < 2; ++w) {
        const float4 *gamma = w ? p.k_gamma : p.q_gamma;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            gain[w][i >> 1][i & 1] = gamma ? __ldg(gamma + 2 * (c + (i >> 1) * L) + (i & 1))
                                           : make_float4(1.f, 1.f, 1.f, 1.f);
    }
    const int r0 = blockIdx.x * run, units = min(run, p.bounds.total - r0) * parts;
    uint32_t phase = 0;
    for (int base = warp; base < units; base += 32 * kStreamPlaces) {
        // 32 of the warp's units looked up, a lane each
        int pos = -1, page = -1;
        if (base + lane * kStreamPlaces < units) {
            const int row = r0 + (base + lane * kStreamPlaces) / parts;
            int lo = 0, hi = p.nseq;         // entries cu[1 .. nseq] that are <= row
            while (lo < hi) {
                const int mid = (lo + hi) >> 1;
                if (__ldg(p.cu + mid + 1) <= row) lo = mid + 1;
                else hi = mid;
            }
            find_token(p, row, lo, pos, page);
        }
        __syncwarp();
        for (uint32_t todo = __ballot_sync(0xffffffffu, pos >= 0); todo; todo &= todo - 1) {
            const int j = __ffs(todo) - 1, unit = base + j * kStreamPlaces, token = unit / parts;
            const long row = r0 + token;
            const int tpos = __shfl_sync(0xffffffffu, pos, j);
            const int tpage = __shfl_sync(0xffffffffu, page, j);
            if (!token_in_bounds(p, row, tpos)) continue;
            // vectors [v0, v1): q heads up to q1, k heads (from nq) up to k1, v heads (from nk)
            const int v0 = (unit - token * parts) * per, v1 = min(v0 + per, nv);
            const int q1 = max(v0, min(v1, nq)), k1 = max(q1, min(v1, nk));
            uint8_t *keys = place + (q1 - v0) * kVec, *values = place + (k1 - v0) * kVec;
            if (lane == 0) {
                mbar_arrive_expect_tx(full, (v1 - v0) * kVec + D * 4);
                if (q1 > v0)
                    bulk_copy_g2s(place, p.q + row * p.q_stride + v0 * C, (q1 - v0) * kVec, full);
                if (k1 > q1)
                    bulk_copy_g2s(keys, p.k + row * p.k_stride + (q1 - nq) * C, (k1 - q1) * kVec, full);
                if (v1 > k1)
                    bulk_copy_g2s(values, p.v + row * p.v_stride + (k1 - nk) * C, (v1 - k1) * kVec, full);
                bulk_copy_g2s(table, p.table + (long)tpos * (D / 4), D * 4, full);
            }
            if (!__all_sync(0xffffffffu, mbar_wait(full, phase))) {
                set_timeout(p.status, kDiagCache, 0, 0, static_cast<int>(row));
                mbar_wait(full, phase);      // never leave with copies in flight
                bulk_wait_all();
                return;
            }
            phase ^= 1;
            Rotation rot;
#pragma unroll
            for (int i = 0; i < 4; ++i) rot.set(i, reinterpret_cast<const float4 *>(table)[4 * c + i]);
            // Vectors of kind W (0: q, 1: k, 2: v of an 8-bit cache), the first of them of head
            // `head`: an 8-bit cache's go from here to their page.
            auto vectors = [&](auto W, uint8_t *at, int n, bool norm, int head) {
                constexpr int w = decltype(W)::value;
#pragma unroll 1
                for (int b = 0; b < n; b += V) {
                    const int i = b + lane / L;
                    uint4 *x = reinterpret_cast<uint4 *>(at + (size_t)min(i, n - 1) * kVec) + c;
                    uint4 a = x[0], d = x[L];
                    Vec v(a, d);
                    if constexpr (w < 2) {
                        if (norm) v.scale(v.template inverse_norm<D>(p.eps), gain[w][0], gain[w][1]);
                        rot.apply(v, a, d);
                    }
                    if constexpr (Q8 && w > 0) {
                        const long slot = ((long)tpage * p.Hkv + head + i) * p.page_size +
                                          (tpos & (p.page_size - 1));
                        v.template store_q8<D>(p, w == 1, slot, c,
                                               i < n && tpage >= 0 && slot_in_bounds(p, slot));
                    }
                    __syncwarp();            // a clamped lane may have read the last vector
                    if (w < 2 && i < n) {
                        x[0] = a;
                        x[L] = d;
                    }
                }
            };
            vectors(std::integral_constant<int, 0>{}, place, q1 - v0, p.q_gamma != nullptr, 0);
            vectors(std::integral_constant<int, 1>{}, keys, k1 - q1, p.k_gamma != nullptr, q1 - nq);
            if constexpr (Q8)
                vectors(std::integral_constant<int, 2>{}, values, v1 - k1, false, k1 - nk);
            fence_proxy_async_smem();        // before the bulk copies read it
            __syncwarp();
            if (lane == 0 && q1 > v0)
                bulk_store(p.q_out + (row * p.Hq + v0) * C, place, (q1 - v0) * kVec);
            if (lane == 1 && p.k_out && k1 > q1)
                bulk_store(p.k_out + (row * p.Hkv + q1 - nq) * C, keys, (k1 - q1) * kVec);
            if (!Q8 && p.k_pool && tpage >= 0)
                for (int i = q1 + lane; i < v1; i += 32) {
                    const int g = i < nk ? i - nq : i - nk;
                    const long slot =
                        ((long)tpage * p.Hkv + g) * p.page_size + (tpos & (p.page_size - 1));
                    if (!slot_in_bounds(p, slot)) continue;
                    bulk_store((i < nk ? p.k_pool : p.v_pool) + slot * C, place + (i - v0) * kVec, kVec);
                }
            bulk_commit_group();
            bulk_wait_read_all();            // the token has left its place
            __syncwarp();
        }
    }
    check_sequences(p);
    bulk_wait_all();
}

}  // namespace

cudaError_t launch_packed_rope_append(const void *q, int64_t q_stride, const void *k,
                                      int64_t k_stride, const void *v, int64_t v_stride,
                                      const int32_t *cu, int nseq, int total, int Hq, int Hkv,
                                      int d, const float *q_gamma, const float *k_gamma,
                                      float eps, const float *table, int table_len, void *q_out,
                                      void *k_out, const gqa_paged_kv *cache, uint8_t *scales,
                                      int *status, cudaStream_t s) {
    AppendParams p{};
    p.scales = scales;
    p.q = static_cast<const uint4 *>(q);
    p.k = static_cast<const uint4 *>(k);
    p.v = static_cast<const uint4 *>(v);
    p.q_stride = q_stride / 8;
    p.k_stride = k_stride / 8;
    p.v_stride = v_stride / 8;
    p.cu = cu;
    p.nseq = nseq;
    p.Hq = Hq;
    p.Hkv = Hkv;
    p.table_len = table_len;
    p.q_gamma = reinterpret_cast<const float4 *>(q_gamma);
    p.k_gamma = reinterpret_cast<const float4 *>(k_gamma);
    p.table = reinterpret_cast<const float4 *>(table);
    p.eps = eps;
    p.q_out = static_cast<uint4 *>(q_out);
    p.k_out = static_cast<uint4 *>(k_out);
    p.status = status;
    p.bounds = {total, total, 0x7fffffff, 0x7fffffffL};
    if (cache) {
        p.kv_lens = cache->kv_lens;
        p.pages = cache->page_table;
        p.num_pages = cache->num_pages;
        p.page_size = cache->page_size;
        p.max_pages = cache->max_pages;
        p.k_pool = static_cast<uint4 *>(cache->k);
        p.v_pool = static_cast<uint4 *>(cache->v);
        p.bounds.cap = (long)cache->max_pages * cache->page_size;
    }
    if (total > kFewTokens) {
        auto kern = scales ? (d == 64    ? packed_append_stream_kernel<64, true>
                              : d == 128 ? packed_append_stream_kernel<128, true>
                              : d == 256 ? packed_append_stream_kernel<256, true>
                                         : packed_append_stream_kernel<512, true>)
                           : (d == 64    ? packed_append_stream_kernel<64, false>
                              : d == 128 ? packed_append_stream_kernel<128, false>
                              : d == 256 ? packed_append_stream_kernel<256, false>
                                         : packed_append_stream_kernel<512, false>);
        const cudaError_t err = ensure_smem_attr(reinterpret_cast<const void *>(kern), kStreamSmem);
        if (err != cudaSuccess) return err;
        // runs of vectors that fit a place, as equal as can be
        const int vectors = (q ? Hq : 0) + (cache ? 2 : 1) * Hkv, most = (kPlaceBytes - d * 4) / (d * 2);
        const int parts = (vectors + most - 1) / most, cap = parts == 1 ? 64 : parts < 4 ? 32 / parts : 8;
        const int wave = (total + 303) / 304, run = wave < cap ? wave : cap;
        return launch_pdl(kern, dim3((total + run - 1) / run), dim3(32 * kStreamPlaces), kStreamSmem, s,
                          p, parts, (vectors + parts - 1) / parts, run);
    }
    // Threads per token: a power of two, at least a warp (whose lanes shuffle together), that
    // covers the token's lanes.
    const int lanes = (Hq + 2 * Hkv) * (d / 16);
    int per = 32;
    while (per < lanes && per < kAppendThreads) per <<= 1;
    const int tokens = kAppendThreads / per;
    auto kern = scales ? (d == 64    ? packed_rope_append_kernel<64, true>
                          : d == 128 ? packed_rope_append_kernel<128, true>
                          : d == 256 ? packed_rope_append_kernel<256, true>
                                     : packed_rope_append_kernel<512, true>)
                       : (d == 64    ? packed_rope_append_kernel<64, false>
                          : d == 128 ? packed_rope_append_kernel<128, false>
                          : d == 256 ? packed_rope_append_kernel<256, false>
                                     : packed_rope_append_kernel<512, false>);
    return launch_pdl(kern, dim3((total + tokens - 1) / tokens), dim3(kAppendThreads), 0, s, p,
                      tokens, per);
}

}  // namespace gqa
