// paged_q8_few.cuh -- up to 8 rows (tokens x heads of a KV group) over 32 keys of 8-bit pages in
// shared memory, by one warp: what the kernels of paged_q8_few.cu and paged_q8_short.cu share.
#pragma once
#include "paged_stream.cuh"
#include "q8.cuh"

namespace gqa {
namespace stream {

constexpr int kFewRows = 8;
constexpr float kGrow = 6.0f, kShift = 9.0f;        // log2 units

__device__ __forceinline__ void mma16816_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                             uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
        "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    const __half2 y = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&y);
}
// Two transposed 16 x 16 matrices of bytes, their rows at the addresses of lanes 0-15 and 16-31: of
// each, the lane's columns lane / 4 and + 8, rows 4 (lane % 4) and the three after it.
__device__ __forceinline__ void ldsm_b8_trans(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m16n16.x2.trans.shared.b8 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
// Clears the NaN among the four e4m3 in w; true if there was one.
__device__ __forceinline__ bool strip_nan(uint32_t &w) {
    const uint32_t nan = __vcmpeq4(w & 0x7f7f7f7fu, 0x7f7f7f7fu);
    w &= ~nan;
    return nan != 0;
}

// Where a lane finds its parts of a warp's 32 keys, relative to the stage.
// Rows of 128 bytes, 128-byte swizzled.  A block of 16
// keys has the keys 0-7 and 8 + (0-7 ^ 4) as the rows 0-7 and 8-15 of the score product's A
// operand.  There each four numbers of a lane are two of the product's k-steps' pairs: the
// queries' dims are taken in the same order.  V's 16 x 16 matrices, transposed, bring a lane
// four rows, which are the keys of its pairs 2tq, + 1 and 8 + 2tq, + 1 in the value product: rows
// 4i .. 4i + 3 are the score rows 2i, 2i + 1, 8 + 2i, 8 + 2i + 1.  (The ^ 4: eight rows of either
// operand lie in eight different swizzled columns.)
struct FewAt {
    uint32_t values0, k[2], v;               // values0: bytes from keys to values
    int part;                                // the first of the 32 keys within the stage
    __device__ __forceinline__ FewAt(int first, uint32_t apart) {
        const int lane = threadIdx.x & 31, mat = lane >> 3, l7 = lane & 7;
        part = first;
        values0 = apart;
        const int kk = mat & 1 ? 8 + (l7 ^ 4) : l7;
#pragma unroll
        for (int b = 0; b < 2; ++b)
            k[b] = row(16 * b + kk) + (((mat >> 1) ^ (kk & 7)) << 4);
        const int rho = lane & 15, i = 2 * (rho >> 2) + (rho & 1), vk = rho & 2 ? 8 + (i ^ 4) : i;
        v = values0 + row(16 * (lane >> 4) + vk) + ((vk & 7) << 4);
    }
    __device__ __forceinline__ uint32_t row(int key) const {
        return (part + key) * kD;
    }
    __device__ __forceinline__ uint32_t values(int key) const { return values0 + row(key); }
};

// What a pair's rows see.  pos: of this lane's rows 2 (lane % 4), + 1 (past the last row: the last).
struct FewMask {
    int S, T, window, q_first, lo, lo_all, pos[2];
    __device__ __forceinline__ FewMask(const Params &p, int S_, int T_)
        : S(S_), T(T_), window(p.window), q_first(S_ - T_) {   // keys beyond are hidden from some
        lo = window > 0 ? max(0, q_first - window + 1) : 0;
        lo_all = window > 0 ? max(0, S - window) : 0;
#pragma unroll
        for (int c = 0; c < 2; ++c)
            pos[c] = q_first + min(token_of(p, 2 * (threadIdx.x & 3) + c), T - 1);
    }
};

// The warp's rows: queries and the running result.
struct FewRows {
    uint32_t qb[8][2];
    float sl[2];                              // the factor of a score of rows 2tq, + 1, log2 units
    float o[8][4];                            // dims 16 i + gq (+ 8 for the second pair)
    // mr: m, or 0 while m is -inf.  mo: the largest score plus its value's exponent, less mr (kept
    // relative: next to a score of 2^24 an exponent is lost in fp32).
    float m[2], mr[2], mo[2], l[2];

    // This lane's part of the queries: row gq, zero past the last one, in f16 with the row's largest
    // element brought to [2^14, 2^15); what that leaves of a number below 2^-14 is a multiple of
    // 2^-24, 2^-38 of the largest at most.  A row with an infinity or NaN: NaN.
    __device__ __forceinline__ void load(const Params &p, int row0, int g, int rows) {
        const int lane = threadIdx.x & 31, gq = lane >> 2, tq = lane & 3, t = token_of(p, gq);
        const __nv_bfloat16 *qr = p.q + (long)(row0 + t) * p.q_stride +
                                  (g * p.G + (gq - t * p.G)) * kD + 4 * tq;
        float most = 0.f;
#pragma unroll
        for (int ks = 0; ks < 8; ++ks) {
            uint2 w = make_uint2(0, 0);
            if (gq < rows && GQA_IN_BOUNDS(row0 + t, p.bounds.total, p.status, kSite | 13))
                w = __ldg(reinterpret_cast<const uint2 *>(qr + 16 * ks));
            qb[ks][0] = w.x;
            qb[ks][1] = w.y;
        }
#pragma unroll
        for (int ks = 0; ks < 8; ++ks)
#pragma unroll
            for (int i = 0; i < 2; ++i)
                most = amax_nan(most, amax_nan(bf16lo(qb[ks][i]), bf16hi(qb[ks][i])));
        most = amax_nan(most, __shfl_xor_sync(0xffffffffu, most, 1));
        most = amax_nan(most, __shfl_xor_sync(0xffffffffu, most, 2));
        const uint32_t e = max(__float_as_uint(most) >> 23, 15u);
        const float up = e == 255 ? CUDART_NAN_F : __uint_as_float((268 - e) << 23);
#pragma unroll
        for (int ks = 0; ks < 8; ++ks)
#pragma unroll
            for (int i = 0; i < 2; ++i)
                qb[ks][i] = pack_f16x2(bf16lo(qb[ks][i]) * up, bf16hi(qb[ks][i]) * up);
        const float down = __uint_as_float((e - 14) << 23) * p.scale_log2;
#pragma unroll
        for (int c = 0; c < 2; ++c) sl[c] = __shfl_sync(0xffffffffu, down, 4 * (2 * tq + c));
    }

    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            m[c] = mo[c] = -CUDART_INF_F;
            mr[c] = l[c] = 0.f;
        }
    }

    // Keys kb .. kb + 31, which lie in `stage`, their scale bytes at `bytes`.
    __device__ __forceinline__ void attend(const FewAt &at, const FewMask &mask, const uint8_t *stage,
                                           const uint16_t *bytes, int kb) {
        const int gq = (threadIdx.x & 31) >> 2, tq = threadIdx.x & 3;
        const uint32_t base = smem_u32(stage);
        // ---- scores: two blocks of 16 keys x rows, two chains of four products each
        float x[2][4], xs[2][2][4];
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int e = 0; e < 4; ++e) xs[0][b][e] = xs[1][b][e] = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                uint32_t w[4];
                ldsm4(w, (base + at.k[b]) ^ (i << 5));
#pragma unroll
                for (int s = 0; s < 2; ++s)
                    mma16816_f16(xs[s][b], e4m3x2_f16x2(w[2 * s]), e4m3x2_f16x2(w[2 * s + 1]),
                                 e4m3x2_f16x2(w[2 * s] >> 16),
                                 e4m3x2_f16x2(w[2 * s + 1] >> 16), qb[2 * i + s][0],
                                 qb[2 * i + s][1]);
            }
        // x[b]: keys kb + 16b + gq (rows 2tq, + 1) and + 8 + (gq ^ 4).  (The key's and the row's
        // factors make one first: either alone may take a finite score out of fp32's range, or, as
        // 0, a hidden one to NaN.)
        float ev[2][2];   // the values' exponents
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int f = 0; f < 2; ++f) {
                const uint32_t w = bytes[16 * b + (f ? 8 + (gq ^ 4) : gq)];
                const float kf = scale_of(w & 255u);
                ev[b][f] = exponent_of(w >> 8);
#pragma unroll
                for (int c = 0; c < 2; ++c)
                    x[b][2 * f + c] = (xs[0][b][2 * f + c] + xs[1][b][2 * f + c]) * (kf * sl[c]);
            }
        const bool edge = kb + 31 > mask.q_first || kb < mask.lo_all;   // of the mask
        uint32_t hidden = 0;   // bits 4b + e
        if (edge) {
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int key = kb + 16 * b + (e >> 1 ? 8 + (gq ^ 4) : gq);
                    const int pos = mask.pos[e & 1];
                    if (key > pos || (mask.window > 0 && pos - key >= mask.window)) {
                        x[b][e] = -CUDART_INF_F;
                        hidden |= 1u << (4 * b + e);
                    }
                }
        }
        // ---- online softmax
        bool grow = false;
        float top[2];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            float t = -CUDART_INF_F, to = -CUDART_INF_F;
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int f = 0; f < 2; ++f) {
                    t = fmaxf(t, x[b][2 * f + c]);
                    to = fmaxf(to, x[b][2 * f + c] - mr[c] + ev[b][f]);
                }
            top[c] = t;
            grow |= t > m[c] + kGrow || to > mo[c] + kGrow;
        }
        if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                float mx = top[c], mxo = -CUDART_INF_F;
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
                const float mn = fmaxf(m[c], mx), mrn = mn == -CUDART_INF_F ? 0.f : mn;
#pragma unroll
                for (int b = 0; b < 2; ++b)
#pragma unroll
                    for (int f = 0; f < 2; ++f) mxo = fmaxf(mxo, x[b][2 * f + c] - mrn + ev[b][f]);
#pragma unroll
                for (int d = 4; d < 32; d <<= 1)
                    mxo = fmaxf(mxo, __shfl_xor_sync(0xffffffffu, mxo, d));
                const float was = mo[c] + (mr[c] - mrn), mno = fmaxf(was, mxo);
                const float f = m[c] == -CUDART_INF_F ? 0.f : ex2_approx(m[c] - mn);
                const float fo = mo[c] == -CUDART_INF_F ? 1.f : ex2_approx(was - mno);
                m[c] = mn;
                mr[c] = mrn;
                l[c] *= f;
                mo[c] = mno;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    o[i][c] *= fo;
                    o[i][2 + c] *= fo;
                }
            }
        }
        // P as the B operand: row gq, the score rows 2tq, + 1 and 8 + 2tq, + 1 of a block
        uint32_t pb[2][2];
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            float w[4], wv[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int c = e & 1;
                const float ro = mo[c] == -CUDART_INF_F ? 0.f : mo[c] - kShift;
                const float d = x[b][e] - mr[c];
                w[e] = ex2_approx(d);
                wv[e] = ex2_approx(d + (ev[b][e >> 1] - ro));
            }
            if (edge) {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (hidden >> (4 * b + e) & 1) wv[e] = 0.f;
            }
            l[0] += w[0] + w[2];
            l[1] += w[1] + w[3];
            pb[b][0] = transpose8x8(pack_f16x2(wv[0], wv[1]));
            pb[b][1] = transpose8x8(pack_f16x2(wv[2], wv[3]));
        }
        // ---- O += V^T P
        uint32_t seen[2] = {0xffffffffu, 0xffffffffu};   // keys that some row sees
        if (edge) {
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                seen[b] = 0;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int r = 2 * tq + (i & 1);
                    const int key = kb + 16 * b + (i & 2 ? 8 + (r ^ 4) : r);
                    if (key >= mask.lo && key < mask.S) seen[b] |= 0xffu << (8 * i);
                }
            }
        }
        bool stripped = false;
#pragma unroll
        for (int nn = 0; nn < 8; ++nn) {
            uint32_t w[4];
            ldsm_b8_trans(w, (base + at.v) ^ (nn << 4));
            if (edge) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    w[i] &= seen[i >> 1];
                    if (mask.T > 1) stripped |= strip_nan(w[i]);
                }
            }
#pragma unroll
            for (int b = 0; b < 2; ++b)
                mma16816_f16(o[nn], e4m3x2_f16x2(w[2 * b]), e4m3x2_f16x2(w[2 * b + 1]),
                             e4m3x2_f16x2(w[2 * b] >> 16), e4m3x2_f16x2(w[2 * b + 1] >> 16),
                             pb[b][0], pb[b][1]);
        }
        if (__any_sync(0xffffffffu, stripped)) {
            // the NaN that were taken out, for the rows that see them
#pragma unroll 1
            for (int kk = 0; kk < 32; ++kk) {
                const int key = kb + kk;
                if (key < mask.lo || key >= mask.S) continue;
                bool sees[2];
#pragma unroll
                for (int c = 0; c < 2; ++c)
                    sees[c] = key <= mask.pos[c] &&
                              (mask.window <= 0 || mask.pos[c] - key < mask.window);
                const uint8_t *vr = stage + at.values(kk) + gq;
#pragma unroll
                for (int i = 0; i < 8; ++i)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        if ((vr[((i ^ (kk & 7)) << 4) + 8 * e] & 0x7f) != 0x7f) continue;
#pragma unroll
                        for (int c = 0; c < 2; ++c)
                            if (sees[c]) o[i][2 * e + c] = CUDART_NAN_F;
                    }
            }
        }
    }

    // O relative to m: times 2^(mo - 9), in two steps as that may be 2^-135.
    __device__ __forceinline__ void finish() {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            if (mo[c] == -CUDART_INF_F) continue;   // O is 0, or NaN
            const float f = ex2_approx(0.5f * (mo[c] - kShift));
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                o[i][c] = o[i][c] * f * f;
                o[i][2 + c] = o[i][2 + c] * f * f;
            }
        }
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) l[c] += __shfl_xor_sync(0xffffffffu, l[c], d);
    }
};

}  // namespace stream
}  // namespace gqa
