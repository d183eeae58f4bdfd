// packed_attn.cu -- attention over packed prompts and over the paged cache.
//
// Within a sequence of S keys whose T last tokens are queries ("PLaMo 3アーキテクチャ徹底解析"
// §4.5, §5.1):  o_t = sum_j softmax_j(scale q_t . k_j) v_j  over the keys j <= S - T + t, and
// with a window W those with S - T + t - j < W.
//
// One warp per (token, query head): each lane holds 4 of the 128 dimensions, the keys pass one
// by one, and the running maximum, sum and output of the softmax are rescaled as the maximum
// grows.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math_constants.h>

#include "internal.h"
#include "packed.cuh"

namespace gqa {
namespace {

constexpr int kD = 128;

// A paged call whose sequences bring at most 32 rows (tokens times heads of a group) each.
bool few_rows(int max_q, int G) { return static_cast<long>(max_q) * G <= 32; }

struct RowParams {
    const __nv_bfloat16 *q, *k, *v;
    __nv_bfloat16 *o;
    float *lse;
    long q_stride, k_stride, v_stride, o_stride;
    const int32_t *cu, *kv_lens, *pages;
    PackedBounds bounds;
    int nseq, Hq, Hkv, G, window, num_pages, page_size, max_pages;
    float scale_log2;
    int *status;
};

__global__ void packed_attn_row_kernel(const RowParams p) {
    const int row = blockIdx.x, h = blockIdx.y * (blockDim.x >> 5) + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    const int i = packed_row_seq(p.cu, p.nseq, row);
    if (i >= p.nseq || h >= p.Hq) return;
    const PackedSeq s = packed_seq(p.cu, p.kv_lens, i, p.bounds, lane == 0 ? p.status : nullptr);
    if (row < s.row0 || row >= s.row0 + s.T) return;
    const int g = h / p.G;
    const int pos = s.S - s.T + (row - s.row0);
    const int lo = p.window > 0 ? max(0, pos - p.window + 1) : 0;
    float q[4];
    {
        const uint2 w = *reinterpret_cast<const uint2 *>(p.q + row * p.q_stride + h * kD + 4 * lane);
        q[0] = bf16lo(w.x) * p.scale_log2;
        q[1] = bf16hi(w.x) * p.scale_log2;
        q[2] = bf16lo(w.y) * p.scale_log2;
        q[3] = bf16hi(w.y) * p.scale_log2;
    }
    float m = -CUDART_INF_F, l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
    for (int j = lo; j <= pos; ++j) {
        uint2 kw = make_uint2(0, 0), vw = make_uint2(0, 0);
        if (p.pages) {
            const int page = __ldg(p.pages + (long)i * p.max_pages + j / p.page_size);
            if (page >= 0 && page < p.num_pages) {
                const long at = (((long)page * p.Hkv + g) * p.page_size + j % p.page_size) * kD + 4 * lane;
                kw = *reinterpret_cast<const uint2 *>(p.k + at);
                vw = *reinterpret_cast<const uint2 *>(p.v + at);
            } else if (lane == 0) {
                set_status(p.status, GQA_ERR_INVALID_ARG);
            }
        } else {
            kw = *reinterpret_cast<const uint2 *>(p.k + (s.row0 + j) * p.k_stride + g * kD + 4 * lane);
            vw = *reinterpret_cast<const uint2 *>(p.v + (s.row0 + j) * p.v_stride + g * kD + 4 * lane);
        }
        float x = q[0] * bf16lo(kw.x) + q[1] * bf16hi(kw.x) + q[2] * bf16lo(kw.y) + q[3] * bf16hi(kw.y);
#pragma unroll
        for (int d = 16; d; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
        const float mn = fmaxf(m, x);
        const float f = exp2f(m - mn), e = exp2f(x - mn);
        m = mn;
        l = l * f + e;
        o[0] = o[0] * f + e * bf16lo(vw.x);
        o[1] = o[1] * f + e * bf16hi(vw.x);
        o[2] = o[2] * f + e * bf16lo(vw.y);
        o[3] = o[3] * f + e * bf16hi(vw.y);
    }
    const float r = 1.0f / l;
    *reinterpret_cast<uint2 *>(p.o + row * p.o_stride + h * kD + 4 * lane) =
        make_uint2(pack_bf16x2(o[0] * r, o[1] * r), pack_bf16x2(o[2] * r, o[3] * r));
    if (p.lse && lane == 0)
        p.lse[(long)h * p.bounds.total + row] = (m + log2f(l)) * 0.69314718055994531f;
}

}  // namespace

size_t paged_workspace_bytes(int, int total, int max_q, int max_kv, int Hq, int Hkv, int) {
    if (few_rows(max_q, Hq / Hkv)) return 0;
    return packed_prefill_workspace_bytes(total, max_kv, Hq, Hkv);
}

int launch_packed_attn(const PackedAttn &a, void *ws, int *status, cudaStream_t s) {
    if (!a.cache || !few_rows(a.max_q, a.Hq / a.Hkv))
        return launch_packed_prefill(a, ws, status, s);
    RowParams p{};
    p.q = static_cast<const __nv_bfloat16 *>(a.q);
    p.k = static_cast<const __nv_bfloat16 *>(a.k);
    p.v = static_cast<const __nv_bfloat16 *>(a.v);
    p.o = static_cast<__nv_bfloat16 *>(a.o);
    p.lse = a.lse;
    p.q_stride = a.q_stride;
    p.k_stride = a.k_stride;
    p.v_stride = a.v_stride;
    p.o_stride = a.o_stride;
    p.cu = a.cu;
    p.nseq = a.nseq;
    p.Hq = a.Hq;
    p.Hkv = a.Hkv;
    p.G = a.Hq / a.Hkv;
    p.window = a.window;
    p.scale_log2 = a.scale * 1.4426950408889634f;
    p.status = status;
    p.bounds = {a.total, a.max_q, a.max_kv, 0x7fffffffL};
    if (a.cache) {
        p.kv_lens = a.cache->kv_lens;
        p.pages = a.cache->page_table;
        p.num_pages = a.cache->num_pages;
        p.page_size = a.cache->page_size;
        p.max_pages = a.cache->max_pages;
        p.bounds.cap = (long)a.cache->max_pages * a.cache->page_size;
    }
    packed_attn_row_kernel<<<dim3(a.total, (a.Hq + 3) / 4), 128, 0, s>>>(p);
    return cudaPeekAtLastError() == cudaSuccess ? GQA_OK : GQA_ERR_CUDA;
}

}  // namespace gqa
