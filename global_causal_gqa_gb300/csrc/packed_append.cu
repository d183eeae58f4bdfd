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
// the table row is read once per token and the gains once per block.
#include <cuda_runtime.h>

#include "internal.h"
#include "packed.cuh"

namespace gqa {
namespace {

constexpr int kAppendThreads = 256;
constexpr int kAppendTokens = 8;   // most tokens of one block: one per warp to look up

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
__global__ void __launch_bounds__(kAppendThreads)
    packed_rope_append_kernel(const AppendParams p, int tokens, int per) {
    constexpr int L = D / 16;    // lanes of a vector; also the distance of a pair's chunks
    constexpr int C = D / 8;     // 16-byte chunks of a vector
    griddep_wait();
    griddep_launch_dependents();
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
    const int heads = p.Hq + p.Hkv + (p.v_pool ? p.Hkv : 0);
    for (int t = group; t < tokens; t += groups) {
        const int pos = s_pos[t], page = s_page[t];
        if (pos < 0) continue;   // the same for the whole group, which is whole vectors
        const long row = row_base + t;
        float cs[16];            // (cos, sin) of pairs 8c .. 8c + 7
        const float4 *tr = p.table + (long)pos * (D / 4) + 4 * c;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float4 x = __ldg(tr + i);
            cs[4 * i] = x.x;
            cs[4 * i + 1] = x.y;
            cs[4 * i + 2] = x.z;
            cs[4 * i + 3] = x.w;
        }
        const long slot = p.page_size ? pos % p.page_size : 0;
        // every lane of a warp makes the same number of turns (the norm shuffles): heads
        // past the last are computed on the last one and not stored
        for (int ub = 0; ub < heads; ub += step) {
            const int uu = ub + u0, u = min(uu, heads - 1);
            const bool isq = u < p.Hq, isk = !isq && u < p.Hq + p.Hkv;
            const int g = isq ? u : isk ? u - p.Hq : u - p.Hq - p.Hkv;
            const uint4 *src = (isq ? p.q + row * p.q_stride
                                    : isk ? p.k + row * p.k_stride : p.v + row * p.v_stride) +
                               (long)g * C;
            uint4 a = __ldg(src + c), b = __ldg(src + c + L);
            const float4 *gam = isq ? p.q_gamma : isk ? p.k_gamma : nullptr;
            float x[8], y[8];
            const uint32_t aw[4] = {a.x, a.y, a.z, a.w}, bw[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[2 * i] = bf16lo(aw[i]);
                x[2 * i + 1] = bf16hi(aw[i]);
                y[2 * i] = bf16lo(bw[i]);
                y[2 * i + 1] = bf16hi(bw[i]);
            }
            if (p.q_gamma || p.k_gamma) {
                float ss = 0.f;
#pragma unroll
                for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], fmaf(y[i], y[i], ss));
#pragma unroll
                for (int o = 1; o < L; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
                if (gam) {
                    const float r = 1.0f / sqrtf(ss * (1.0f / D) + p.eps);
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float4 ga = __ldg(gam + 2 * c + i), gb = __ldg(gam + 2 * (c + L) + i);
                        x[4 * i] *= r * ga.x;
                        x[4 * i + 1] *= r * ga.y;
                        x[4 * i + 2] *= r * ga.z;
                        x[4 * i + 3] *= r * ga.w;
                        y[4 * i] *= r * gb.x;
                        y[4 * i + 1] *= r * gb.y;
                        y[4 * i + 2] *= r * gb.z;
                        y[4 * i + 3] *= r * gb.w;
                    }
                }
            }
            if (isq || isk) {
                uint32_t ao[4], bo[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float c0 = cs[4 * i], s0 = cs[4 * i + 1];
                    const float c1 = cs[4 * i + 2], s1 = cs[4 * i + 3];
                    const float x0 = x[2 * i], x1 = x[2 * i + 1], y0 = y[2 * i], y1 = y[2 * i + 1];
                    ao[i] = pack_bf16x2(fmaf(x0, c0, -y0 * s0), fmaf(x1, c1, -y1 * s1));
                    bo[i] = pack_bf16x2(fmaf(x0, s0, y0 * c0), fmaf(x1, s1, y1 * c1));
                }
                a = make_uint4(ao[0], ao[1], ao[2], ao[3]);
                b = make_uint4(bo[0], bo[1], bo[2], bo[3]);
            }
            if (uu >= heads) continue;   // after this turn's shuffles
            uint4 *dst = nullptr;
            if (isq) {
                dst = p.q_out + (row * p.Hq + g) * C;
            } else {
                if (page >= 0)
                    dst = (isk ? p.k_pool : p.v_pool) +
                          (((long)page * p.Hkv + g) * p.page_size + slot) * C;
                if (isk && p.k_out) {
                    uint4 *ko = p.k_out + (row * p.Hkv + g) * C;
                    ko[c] = a;
                    ko[c + L] = b;
                }
            }
            if (dst) {
                dst[c] = a;
                dst[c + L] = b;
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
    // threads per token: the power of two that covers its vectors' lanes, within a block (and
    // at least a warp, whose lanes shuffle together)
    const int lanes = (Hq + 2 * Hkv) * (d / 16);
    int per = 32;
    while (per < lanes && per < kAppendThreads) per <<= 1;
    // one token per group of threads; more per block only when the grid is deep without
    int tokens = kAppendThreads / per;
    while (tokens < kAppendTokens && (long)total > 8L * 152 * tokens) tokens <<= 1;
    if (tokens > kAppendTokens) tokens = kAppendTokens;
    auto kern = d == 64    ? packed_rope_append_kernel<64>
                : d == 128 ? packed_rope_append_kernel<128>
                : d == 256 ? packed_rope_append_kernel<256>
                           : packed_rope_append_kernel<512>;
    return launch_pdl(kern, dim3((total + tokens - 1) / tokens), dim3(kAppendThreads), 0, s, p,
                      tokens, per);
}

}  // namespace gqa
