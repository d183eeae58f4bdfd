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
// the thread.  The threads of a token walk its vectors, q heads, k heads, v heads, in memory
// order (one row of the fused projection is contiguous); a thread keeps its chunk index, so
// the table row is read once per token.  Four blocks per SM (64 registers) hide the loads'
// latency better than more of them in flight per thread (96 registers: 162 us instead of 118).
#include <cuda_runtime.h>

#include "internal.h"
#include "packed.cuh"

namespace gqa {
namespace {

constexpr int kAppendThreads = 256;
constexpr int kAppendTokens = 8;   // most tokens of one block: one per warp to look up
constexpr int kDeepTokens = 4;     // tokens of a block of a batch that fills the GPU

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
    int *status;
};

// D: head dim.  `per` threads (a multiple of the D / 16 lanes of a vector) serve one token at
// a time, the block's kAppendThreads / per groups take its `tokens` tokens in turn.
template <int D>
__global__ void __launch_bounds__(kAppendThreads, 4)
    packed_rope_append_kernel(const AppendParams p, int tokens, int per) {
    constexpr int L = D / 16;    // lanes of a vector; also the distance of a pair's chunks
    constexpr int C = D / 8;     // 16-byte chunks of a vector
    griddep_wait();
    // The next kernel's blocks may come at once where this grid is all resident; a deeper grid
    // keeps the SMs to itself (prompts of 6000 tokens, append + attention: 252 against 272 us).
    if (gridDim.x <= 4 * 152) griddep_launch_dependents();
    __shared__ int s_pos[kAppendTokens];     // position; -1: nothing to do for this token
    __shared__ int s_page[kAppendTokens];    // page; -1: outside the pool
    const int row_base = blockIdx.x * tokens;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (warp < tokens) {
        const int row = row_base + warp;
        int pos = -1, page = -1;
        if (row < p.bounds.total) {
            const int i = packed_row_seq(p.cu, p.nseq, row);
            if (i < p.nseq && lane == 0) {
                const PackedSeq s = packed_seq(p.cu, p.kv_lens, i, p.bounds, p.status);
                if (row >= s.row0 && row < s.row0 + s.T) {
                    pos = s.S - s.T + (row - s.row0);
                    if (pos >= p.table_len) {
                        set_status(p.status, GQA_ERR_RANGE);
                        pos = -1;
                    } else if (p.pages) {
                        page = __ldg(p.pages + (long)i * p.max_pages + pos / p.page_size);
                        if (page < 0 || page >= p.num_pages) {
                            set_status(p.status, GQA_ERR_INVALID_ARG);
                            page = -1;
                        }
                    }
                }
            }
        }
        if (lane == 0) {
            s_pos[warp] = pos;
            s_page[warp] = page;
        }
    }
    __syncthreads();

    const int group = threadIdx.x / per, groups = kAppendThreads / per;
    const int tid = threadIdx.x - group * per;
    const int c = tid % L, u0 = tid / L, step = per / L;
    // The vector's elements in pairs of neighbours: x[i] = 8c + 2i, + 1, y[i] those d/2 on.
    struct Vec {
        float2 x[4], y[4];
    };
    auto unpack = [](const uint4 &a, const uint4 &b) {
        Vec v;
        const uint32_t aw[4] = {a.x, a.y, a.z, a.w}, bw[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v.x[i] = make_float2(bf16lo(aw[i]), bf16hi(aw[i]));
            v.y[i] = make_float2(bf16lo(bw[i]), bf16hi(bw[i]));
        }
        return v;
    };
    // gamma / sqrt(mean(x^2) + eps) over the vector's L lanes (every lane of the warp shuffles)
    auto normalise = [&](Vec &v, const float4 *gamma, bool on) {
        float2 s2 = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < 4; ++i) s2 = ffma2v(v.x[i], v.x[i], ffma2v(v.y[i], v.y[i], s2));
        float ss = s2.x + s2.y;
#pragma unroll
        for (int o = 1; o < L; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        if (!on) return;
        const float r = 1.0f / sqrtf(ss * (1.0f / D) + p.eps);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float4 ga = __ldg(gamma + 2 * c + i), gb = __ldg(gamma + 2 * (c + L) + i);
            v.x[2 * i] = fmul2(v.x[2 * i], make_float2(r * ga.x, r * ga.y));
            v.x[2 * i + 1] = fmul2(v.x[2 * i + 1], make_float2(r * ga.z, r * ga.w));
            v.y[2 * i] = fmul2(v.y[2 * i], make_float2(r * gb.x, r * gb.y));
            v.y[2 * i + 1] = fmul2(v.y[2 * i + 1], make_float2(r * gb.z, r * gb.w));
        }
    };
    for (int t = group; t < tokens; t += groups) {
        const int pos = s_pos[t], page = s_page[t];
        if (pos < 0) continue;   // the same for the whole group, which is whole vectors
        const long row = row_base + t;
        float2 co[4], si[4];     // cos and sin of pairs 8c + 2i, + 1
        const float4 *tr = p.table + (long)pos * (D / 4) + 4 * c;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float4 w = __ldg(tr + i);
            co[i] = make_float2(w.x, w.z);
            si[i] = make_float2(w.y, w.w);
        }
        auto rotate = [&](const Vec &v, uint4 &a, uint4 &b) {
            uint32_t ao[4], bo[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 ra = fsub2(fmul2(v.x[i], co[i]), fmul2(v.y[i], si[i]));
                const float2 rb = ffma2v(v.x[i], si[i], fmul2(v.y[i], co[i]));
                ao[i] = pack_bf16x2(ra.x, ra.y);
                bo[i] = pack_bf16x2(rb.x, rb.y);
            }
            a = make_uint4(ao[0], ao[1], ao[2], ao[3]);
            b = make_uint4(bo[0], bo[1], bo[2], bo[3]);
        };
        // Queries, then keys and values.  Every lane of a warp makes the same number of turns
        // (the norm shuffles), past the last vector on the last one, without storing.
        const uint4 *src = p.q + row * p.q_stride + c;
        uint4 *dst = p.q_out + row * p.Hq * C + c;
        for (int ub = 0; ub < p.Hq; ub += step) {
            const int u = min(ub + u0, p.Hq - 1);
            uint4 a = __ldg(src + (long)u * C), b = __ldg(src + (long)u * C + L);
            Vec v = unpack(a, b);
            if (p.q_gamma) normalise(v, p.q_gamma, true);
            rotate(v, a, b);
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
            Vec v = unpack(a, b);
            if (p.k_gamma) normalise(v, p.k_gamma, isk);
            if (isk) rotate(v, a, b);
            if (ub + u0 >= heads) continue;
            if (page >= 0 && p.k_pool) {
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

}  // namespace

cudaError_t launch_packed_rope_append(const void *q, int64_t q_stride, const void *k,
                                      int64_t k_stride, const void *v, int64_t v_stride,
                                      const int32_t *cu, int nseq, int total, int Hq, int Hkv,
                                      int d, const float *q_gamma, const float *k_gamma,
                                      float eps, const float *table, int table_len, void *q_out,
                                      void *k_out, const gqa_paged_kv *cache, int *status,
                                      cudaStream_t s) {
    AppendParams p{};
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
    // Threads per token: a power of two, at least a warp (whose lanes shuffle together), that
    // covers the token's lanes; for a batch that fills the GPU half a block at most and four
    // tokens per block (64 + 8 + 8 heads of 128 are 640 lanes, 5 turns of 128: 118 us for 15424
    // tokens, 133 with 3 turns of 256, 125 with eight tokens per block; 4.8 TB/s).
    const bool deep = total > 8 * 152;
    const int lanes = (Hq + 2 * Hkv) * (d / 16);
    int per = 32;
    while (per < lanes && per < (deep ? kAppendThreads / 2 : kAppendThreads)) per <<= 1;
    int tokens = kAppendThreads / per;
    if (deep && tokens < kDeepTokens) tokens = kDeepTokens;
    auto kern = d == 64    ? packed_rope_append_kernel<64>
                : d == 128 ? packed_rope_append_kernel<128>
                : d == 256 ? packed_rope_append_kernel<256>
                           : packed_rope_append_kernel<512>;
    return launch_pdl(kern, dim3((total + tokens - 1) / tokens), dim3(kAppendThreads), 0, s, p,
                      tokens, per);
}

}  // namespace gqa
