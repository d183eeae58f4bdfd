// paged_q8_few.cu -- attention of up to 8 rows (tokens x heads of a KV group) per sequence over the
// 8-bit paged cache (d = 128): decode steps.  paged_q8.cu has the definition and takes more rows.
//
// Cut and fed as the bf16 kernel (paged_decode.cu; paged_stream.cuh), in stages of 128 keys, of
// which a warp takes 32.  S^T = Y Q^T and O^T += Z^T P^T are m16n8k16 f16 MMAs with the keys, and
// then the dims, as M and the rows as N.  The e4m3 numbers become f16 exactly, two per instruction
// in registers (mma.sync's own 8-bit form takes longer than the 16-bit one: 33 cycles against 22 in
// a chain).  A query row is brought to f16 by a power of two of its own; P = 2^(x + b - mo + 9) with
// b its value's exponent, so a value's power of two is in its weight and the numbers multiply as
// they are.  l sums the weights relative to 2^m, O relative to 2^(mo - 9), mo the largest x + b seen:
// either range alone may be far from the other's.  Both references move when something exceeds them
// by 2^6; P lies between 2^15 and 2^-24, 2^-33 of the reference.
//
// A stage takes a warp 1800 cycles, the copies of a stage 1365: with few pairs per CTA both groups
// of four warps take a pair's stages in turn (BOTH; 32 caches of 8k-64k tokens 529 -> 399 us, 6.8
// TB/s, which is HBM), else the pairs, so that one's ends pass while the other streams.  The
// tcgen05 kernel of paged_q8.cu takes 425 us: it holds a stage 2.5 us, through a score product, a
// softmax and a value product in different warps, where this one holds it 1 us.
#include "paged_stream.cuh"
#include "q8.cuh"

namespace gqa {
using namespace stream;
namespace {

// BOTH: the groups take a pair's stages in turn.
template <bool BOTH>
struct FewStream {
    static constexpr bool kQ8 = true;
    static constexpr int kUnit = 128, kStages = 5, kSegSlots = 4, kTeams = 2, kEnds = BOTH ? 1 : 2;
    static constexpr int kProducer = kTeams * kConsumers, kThreads = 32 * (kProducer + 1);
    // the barrier of a stage's load: its group's, so that a group sees every phase of its own
    __device__ static int full_of(int turn, int j) { return (BOTH ? j : turn) % kTeams; }
};

constexpr int kRows = 8, kGroups = 2, kUnit = 128, kStages = 5, kSegSlots = 4;
constexpr int kScales = kStages * kStageBytes;      // two bytes per key of a stage
constexpr int kXchg = kScales + kStages * 2 * kUnit;
constexpr int kBar = kXchg + kGroups * kConsumers * kRows * kD * 4;
constexpr int kSmemBytes = kBar + 1536 + 1024;
constexpr float kGrow = 6.0f, kShift = 9.0f;        // log2 units

struct Bars : StreamBars {
    uint64_t merge[kGroups];         // the warps of a group, or of both, meet
    float2 ml[kGroups][kConsumers][kRows];
};
static_assert(sizeof(Bars) <= 1536, "barrier block");

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

// (Out of line: never run in earnest.)
__device__ __noinline__ void expired(int *status, int barrier, int n) {
    set_timeout(status, kDiagPagedDecode, kRoleConsumer, barrier, n);
}

template <bool BOTH>
__global__ void __launch_bounds__(FewStream<BOTH>::kThreads, 1)
    paged_q8_few_kernel(const __grid_constant__ CUtensorMap tmK,
                        const __grid_constant__ CUtensorMap tmV, const Params p) {
    griddep_wait();
    griddep_launch_dependents();
    using S = FewStream<BOTH>;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_addr = smem_u32(smem_raw);
    uint8_t *smem = smem_raw + (((raw_addr + 1023u) & ~1023u) - raw_addr);
    Bars *bars = reinterpret_cast<Bars *>(smem + kBar);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        const int readers = BOTH ? kGroups * kConsumers : kConsumers;
        for (int i = 0; i < kStages; ++i) {
            for (int g = 0; g < kGroups; ++g)
                mbar_init(&bars->full[g][i], kUnit / min(p.page_size, kUnit) + kScaleCopies);
            mbar_init(&bars->empty[i], kConsumers);
        }
        for (int i = 0; i < kSegSlots; ++i) {
            mbar_init(&bars->seg_full[i], 1);
            mbar_init(&bars->seg_free[i], readers);
        }
        for (int g = 0; g < kGroups; ++g) mbar_init(&bars->merge[g], readers);
        mbar_init(&bars->clc_full, 1);
        fence_mbar_init();
    }
    scan_units<S>(p, bars);
    __syncthreads();
    if (warp == S::kProducer) {
        produce<S>(tmK, tmV, p, bars, smem, smem + kScales);
        return;
    }

    // ================= consumers =================
    const int gq = lane >> 2, tq = lane & 3;
    const uint32_t ring = smem_u32(smem);
    const int group = warp / kConsumers, cw = warp % kConsumers;
    float *xchg = reinterpret_cast<float *>(smem + kXchg) + group * kConsumers * kRows * kD;
    const int part = 32 * cw;                 // first of this warp's keys in a stage
    // Rows of 128 bytes, 128-byte swizzled; `step` bytes from 8 keys to the next.  A block of 16
    // keys has the keys 0-7 and 8 + (0-7 ^ 4) as the rows 0-7 and 8-15 of the score product's A
    // operand.  There each four numbers of a lane are two of the product's k-steps' pairs: the
    // queries' dims are taken in the same order.  V's 16 x 16 matrices, transposed, bring a lane
    // four rows, which are the keys of its pairs 2tq, + 1 and 8 + 2tq, + 1 in the value product: rows
    // 4i .. 4i + 3 are the score rows 2i, 2i + 1, 8 + 2i, 8 + 2i + 1.  (The ^ 4: eight rows of either
    // operand lie in eight different swizzled columns.)
    const uint32_t step = p.joint ? 2048 : 1024;
    const uint32_t keys0 = p.joint && p.v_first ? 1024 : 0;
    const uint32_t values0 = !p.joint ? kTileBytes : p.v_first ? 0 : 1024;
    auto row_at = [&](int key) { return (key >> 3) * step + (key & 7) * kD; };
    uint32_t k_at[2], v_at;
    {
        const int mat = lane >> 3, l7 = lane & 7, kk = mat & 1 ? 8 + (l7 ^ 4) : l7;
#pragma unroll
        for (int b = 0; b < 2; ++b)
            k_at[b] = keys0 + row_at(part + 16 * b + kk) + (((mat >> 1) ^ (kk & 7)) << 4);
        const int rho = lane & 15, i = 2 * (rho >> 2) + (rho & 1), vk = rho & 2 ? 8 + (i ^ 4) : i;
        v_at = values0 + row_at(part + 16 * (lane >> 4) + vk) + ((vk & 7) << 4);
    }
    int meets = 0;
    auto meet = [&]() {
        __syncwarp();
        uint64_t *bar = &bars->merge[BOTH ? 0 : group];
        if (lane == 0) mbar_arrive(bar);
        if (warp_wait(bar, meets++ & 1)) return true;
        expired(p.status, 2, meets);
        return false;
    };
    // Segment k and this thread's part of its queries: row gq, zero past the last one, in f16 with
    // the row's largest element brought to [2^14, 2^15); what that leaves of a number below 2^-14 is
    // a multiple of 2^-24, 2^-38 of the largest at most.
    Segment sg;
    uint32_t qb[8][2];
    float sl[2];                              // the factor of a score of rows 2tq, + 1, log2 units
    auto next_segment = [&](int k) {
        const int slot = k % kSegSlots;
        if (!warp_wait(&bars->seg_full[slot], (k / kSegSlots) & 1)) {
            expired(p.status, 0, k);
            return false;
        }
        sg = bars->seg[slot];
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->seg_free[slot]);
        const int rows = sg.stages < 0 ? 0 : sg.T * p.G;   // <= kRows (the host's rule on max_q)
        const int t = token_of(p, gq);
        const __nv_bfloat16 *qr = p.q + (long)(sg.row0 + t) * p.q_stride +
                                  (sg.g * p.G + (gq - t * p.G)) * kD + 4 * tq;
        float most = 0.f;
#pragma unroll
        for (int ks = 0; ks < 8; ++ks) {
            uint2 w = make_uint2(0, 0);
            if (gq < rows && GQA_IN_BOUNDS(sg.row0 + t, p.bounds.total, p.status, kSite | 13))
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
        // a row with an infinity or NaN: NaN
        const float up = e == 255 ? CUDART_NAN_F : __uint_as_float((268 - e) << 23);
#pragma unroll
        for (int ks = 0; ks < 8; ++ks)
#pragma unroll
            for (int i = 0; i < 2; ++i)
                qb[ks][i] = pack_f16x2(bf16lo(qb[ks][i]) * up, bf16hi(qb[ks][i]) * up);
        const float down = __uint_as_float((e - 14) << 23) * p.scale_log2;
#pragma unroll
        for (int c = 0; c < 2; ++c) sl[c] = __shfl_sync(0xffffffffu, down, 4 * (2 * tq + c));
        return true;
    };
    const int first = BOTH ? 0 : group, next = BOTH ? 1 : kGroups;
    if (!next_segment(first)) return;
    uint32_t phases = 0;   // of the group's full barriers, a bit each
    for (int k = first; sg.stages >= 0; k += next) {
        const int rows = sg.T * p.G;
        // this thread's columns of the products: rows 2tq, + 1 (positions of rows past the last
        // one: the last)
        int qpos[2];
#pragma unroll
        for (int c = 0; c < 2; ++c)
            qpos[c] = sg.S - sg.T + min(token_of(p, 2 * tq + c), sg.T - 1);
        const int q_first = sg.S - sg.T;          // keys beyond are hidden from some
        const int lo = p.window > 0 ? max(0, q_first - p.window + 1) : 0;
        const int lo_all = p.window > 0 ? max(0, sg.S - p.window) : 0;
        float o[8][4];                            // dims 16 i + gq (+ 8 for the second pair)
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
        float m[2], mr[2], mo[2], l[2];           // mr: m, or 0 while m is -inf
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            m[c] = mo[c] = -CUDART_INF_F;
            mr[c] = l[c] = 0.f;
        }
        for (int j = BOTH ? group : 0; j < sg.stages; j += BOTH ? kGroups : 1) {
            const int u = sg.u0 + j, st = u % kStages;
            if (!warp_wait(&bars->full[group][st], phases >> st & 1)) {
                expired(p.status, 1, u);
                return;
            }
            phases ^= 1u << st;
            const int kb = (sg.unit0 + j) * kUnit + part;   // this warp's 32 keys
            if (kb < sg.S && kb + 31 >= lo) {
                const uint32_t base = ring + st * kStageBytes;
                const uint16_t *bytes =
                    reinterpret_cast<const uint16_t *>(smem + kScales) + st * kUnit + part;
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
                        ldsm4(w, (base + k_at[b]) ^ (i << 5));
#pragma unroll
                        for (int s = 0; s < 2; ++s)
                            mma16816_f16(xs[s][b], e4m3x2_f16x2(w[2 * s]), e4m3x2_f16x2(w[2 * s + 1]),
                                         e4m3x2_f16x2(w[2 * s] >> 16),
                                         e4m3x2_f16x2(w[2 * s + 1] >> 16), qb[2 * i + s][0],
                                         qb[2 * i + s][1]);
                    }
                // x[b]: keys kb + 16b + gq (rows 2tq, + 1) and + 8 + (gq ^ 4)
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
                            x[b][2 * f + c] = (xs[0][b][2 * f + c] + xs[1][b][2 * f + c]) * kf;
                    }
                const bool edge = kb + 31 > q_first || kb < lo_all;   // of the mask
                uint32_t hidden = 0;   // bits 4b + e
                if (edge) {
#pragma unroll
                    for (int b = 0; b < 2; ++b)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int key = kb + 16 * b + (e >> 1 ? 8 + (gq ^ 4) : gq);
                            const int at = qpos[e & 1];
                            if (key > at || (p.window > 0 && at - key >= p.window)) {
                                x[b][e] = -CUDART_INF_F;
                                hidden |= 1u << (4 * b + e);
                            }
                        }
                }
                // ---- online softmax
                bool grow = false;
                float top[2], topo[2];
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    float t = -CUDART_INF_F, to = -CUDART_INF_F;
#pragma unroll
                    for (int b = 0; b < 2; ++b)
#pragma unroll
                        for (int f = 0; f < 2; ++f) {
                            t = fmaxf(t, x[b][2 * f + c]);
                            to = fmaxf(to, fmaf(x[b][2 * f + c], sl[c], ev[b][f]));
                        }
                    top[c] = t * sl[c];
                    topo[c] = to;
                    grow |= top[c] > m[c] + kGrow || to > mo[c] + kGrow;
                }
                if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        float mx = top[c], mxo = topo[c];
#pragma unroll
                        for (int d = 4; d < 32; d <<= 1) {
                            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
                            mxo = fmaxf(mxo, __shfl_xor_sync(0xffffffffu, mxo, d));
                        }
                        const float mn = fmaxf(m[c], mx), mno = fmaxf(mo[c], mxo);
                        const float f = m[c] == -CUDART_INF_F ? 0.f : ex2_approx(m[c] - mn);
                        const float fo = mo[c] == -CUDART_INF_F ? 1.f : ex2_approx(mo[c] - mno);
                        m[c] = mn;
                        mr[c] = mn == -CUDART_INF_F ? 0.f : mn;
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
                        w[e] = ex2_approx(fmaf(x[b][e], sl[c], -mr[c]));
                        wv[e] = ex2_approx(fmaf(x[b][e], sl[c], ev[b][e >> 1] - ro));
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
                            if (key >= lo && key < sg.S) seen[b] |= 0xffu << (8 * i);
                        }
                    }
                }
                bool stripped = false;
#pragma unroll
                for (int nn = 0; nn < 8; ++nn) {
                    uint32_t w[4];
                    ldsm_b8_trans(w, (base + v_at) ^ (nn << 4));
                    if (edge) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            w[i] &= seen[i >> 1];
                            if (sg.T > 1) stripped |= strip_nan(w[i]);
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
                        if (key < lo || key >= sg.S) continue;
                        bool sees[2];
#pragma unroll
                        for (int c = 0; c < 2; ++c)
                            sees[c] = key <= qpos[c] && (p.window <= 0 || qpos[c] - key < p.window);
                        const uint8_t *vr = smem + st * kStageBytes + values0 + row_at(part + kk) + gq;
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
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars->empty[st]);
        }
        // O relative to m: times 2^(mo - 9 - m), in two steps as that may be 2^-135
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            if (mo[c] == -CUDART_INF_F) continue;   // O is 0, or NaN
            const float f = ex2_approx(0.5f * (mo[c] - kShift - m[c]));
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                o[i][c] = o[i][c] * f * f;
                o[i][2 + c] = o[i][2 + c] * f * f;
            }
        }
        // ---- the pair's (or span's) result.  The next one's queries are on their way meanwhile.
        const int row0 = sg.row0, head0 = sg.g * p.G, out = sg.slot;
        if (!next_segment(k + next)) return;
        // The warps' shares meet in shared memory, each relative to its own maximum:
        // [warp][row][128 dims], a row's dims permuted so that the lanes (4 rows x 8 dims) meet 32
        // different banks.
        if (meets > 0 && !meet()) return;   // the last ones have been read
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            const int r = 2 * tq + c;
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) l[c] += __shfl_xor_sync(0xffffffffu, l[c], d);
            if (gq == 0) bars->ml[group][cw][r] = make_float2(m[c], l[c]);
            float *mine = xchg + (cw * kRows + r) * kD;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                mine[(16 * i + gq) ^ (tq << 3)] = o[i][c];
                mine[(16 * i + 8 + gq) ^ (tq << 3)] = o[i][2 + c];
            }
        }
        if (!meet()) return;
        // a warp adds up every fourth row (BOTH: one), 4 dims per lane
        constexpr int kShares = BOTH ? kGroups * kConsumers : kConsumers;
        const float2(*mls)[kRows] = bars->ml[BOTH ? 0 : group];
        const float *shares = xchg - (BOTH ? group * kConsumers * kRows * kD : 0);
#pragma unroll 1
        for (int r = BOTH ? warp : cw; r < rows; r += kShares) {
            float M = -CUDART_INF_F, L = 0.f;
#pragma unroll
            for (int w = 0; w < kShares; ++w) M = fmaxf(M, mls[w][r].x);
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < kShares; ++w) {
                const float2 x = mls[w][r];
                const float4 y = *reinterpret_cast<const float4 *>(
                    shares + (w * kRows + r) * kD + ((4 * lane) ^ ((r >> 1 & 3) << 3)));
                // a share none of whose keys this row sees: m = -inf, l = 0 and O = 0 (NaN scores
                // alone also leave m at -inf, with l and O NaN)
                const float f =
                    x.x == -CUDART_INF_F ? (x.y == 0.f ? 0.f : 1.f) : ex2_approx(x.x - M);
                L = fmaf(x.y, f, L);
                acc.x = fmaf(y.x, f, acc.x);
                acc.y = fmaf(y.y, f, acc.y);
                acc.z = fmaf(y.z, f, acc.z);
                acc.w = fmaf(y.w, f, acc.w);
            }
            if (out >= 0) {
                const size_t rec = (size_t)out * p.rec_rows + r;
                if (!GQA_IN_BOUNDS(rec, (long)2 * p.chunks * p.rec_rows, p.status, kSite | 14)) continue;
                reinterpret_cast<float4 *>(p.ws_o + rec * kD)[lane] = acc;
                if (lane == 0) reinterpret_cast<float2 *>(p.ws_ml)[rec] = make_float2(M, L);
            } else {
                const int t = token_of(p, r), head = head0 + r - t * p.G;
                const long row = row0 + t;
                if (!GQA_IN_BOUNDS(row, p.bounds.total, p.status, kSite | 15)) continue;
                const float inv = 1.0f / L;
                reinterpret_cast<uint2 *>(p.o + row * p.o_stride + head * kD)[lane] = make_uint2(
                    pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
                if (p.lse && lane == 0)
                    p.lse[(long)head * p.bounds.total + row] =
                        (M + __log2f(L)) * 0.69314718055994531f;
            }
        }
    }
}

template <bool BOTH>
int launch(const CUtensorMap &mk, const CUtensorMap &mv, const Params &p, long grid, cudaStream_t s) {
    auto kern = paged_q8_few_kernel<BOTH>;
    if (ensure_smem_attr(reinterpret_cast<const void *>(kern), kSmemBytes) != cudaSuccess ||
        launch_pdl(kern, dim3(static_cast<unsigned>(grid)), dim3(FewStream<BOTH>::kThreads),
                   kSmemBytes, s, mk, mv, p) != cudaSuccess)
        return GQA_ERR_CUDA;
    return GQA_OK;
}

}  // namespace

int stream::launch_q8_few(const CUtensorMap &mk, const CUtensorMap &mv, const Params &p, long grid,
                          cudaStream_t s) {
    return p.whole ? launch<false>(mk, mv, p, grid, s) : launch<true>(mk, mv, p, grid, s);
}

}  // namespace gqa
