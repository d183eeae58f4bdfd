// paged_q8.cu -- attention over the 8-bit paged cache (d = 128).
//
// For query token t of a sequence with S keys and T new tokens, at position i = S - T + t, over
// keys 2^a_j y_j and values 2^b_j z_j of e4m3 numbers y, z (q8.cuh):
//   o = sum_j softmax_j(scale 2^a_j q . y_j) 2^b_j z_j  over j <= i (and i - j < W with a window).
//
// Up to 32 rows (tokens x heads of a KV group) per sequence: the streaming kernel below, bound by
// memory, 258 bytes per key and KV head.  More: all keys that the call sees are expanded to bf16
// pages in the workspace (paged_read.cu) and the tile kernel (packed_prefill.cu) takes them from
// there.
//
// The streaming kernel is cut and fed as the bf16 one (paged_decode.cu; paged_stream.cuh), in
// stages of 128 keys.  Its products run on tcgen05 with the numbers as they lie in the pages:
//   S^T [128 keys x columns] = Y Q'^T,   O^T [128 dims x columns] += Z^T P'^T,
// e4m3 A operands straight from the stage, so that no thread ever touches a key's number (with
// mma.sync, whose 8-bit form is slower than its 16-bit one, the 64 conversions and 8 ldmatrix of
// 16 keys and 8 rows alone took more than the copies; 12 rows over 700-6000 keys 88 us).  The
// operands that are not 8-bit are sums of 8-bit columns:
//   q 2^u = h + l / 16 (e4m3, the row's largest element brought to [2^7, 2^8)): bf16's 8 bits, but
//     for elements below 2^-3, which lose at most 2^-14, 2^-21 of the largest;
//   P = c + m + f (e5m2, a weight times its value's 2^b): of P in f16 the upper byte, the upper byte
//     of what is left, and the rest rounded: off by 2^-9 + 2^-11 of P, or 2^-17.
// A thread has one key and all rows: its key's and value's powers of two are its own, the rows'
// factors are read from shared memory.  l sums the weights relative to 2^m, O the products P
// relative to 2^(mo - 12), mo the largest score plus its value's exponent: either range alone may
// be far from the other's.  Both references move, for all keys of a stage together, when something
// exceeds them by 2^3, so that P stays within e5m2's range and 2^-17 is 2^-29 of its largest.
//
// Warps: two groups of four (softmax, a quarter of a stage's keys each; the groups take the pairs
// in turn, so that one's ends pass while the other streams, or with 17 to 32 rows 16 of them
// each), the producer, two that issue the products, and one that brings the queries into operands a
// pair ahead.
#include "paged_stream.cuh"
#include "q8.cuh"

namespace gqa {
using namespace stream;
namespace {

constexpr int kProducerWarp = 8, kScoreWarp = 9, kValueWarp = 10, kQueryWarp = 11;
constexpr int kScoreTiles = 2;       // of a group, in tensor memory
// A pair's factors are read after its queries' tile is free again, and that of the pair after next
// may be, too, as scores are formed ahead.
constexpr int kFactorSlots = 8;
constexpr float kGrow = 3.0f, kShift = 12.0f, kLargest = 32768.0f;   // log2 units; 2^(3 + 12)
// Values below 2^-100 count as 2^-100 in mo, so that 2^(m - mo) stays within fp32.
constexpr float kLeast = -100.0f;

struct Q8Bars : StreamBars {
    uint64_t q_full[2], q_free[2];
    uint64_t s_full[kGroups][kScoreTiles], s_free[kGroups][kScoreTiles];
    uint64_t p_full[kGroups], pv_done[kGroups], meet[kGroups], drained[2];
    uint32_t tmem;
    int vote[kGroups][2];            // the last stage of either parity that moved the references
    int nan_any[kGroups][2];
};

// Shared memory.  R: rows of a group.
template <int R, bool SPLIT>
struct Layout {
    using S = Q8Stream<SPLIT>;
    static constexpr int kTiles = SPLIT ? 2 : 1;                  // of a pair: query and score tiles
    static constexpr int kScoreCols = 2 * R, kValueCols = R == 8 ? 32 : 3 * R;
    static constexpr int kQuery = kScoreCols * kD, kWeights = kValueCols * kD;   // bytes of a tile
    static constexpr int kQ = S::kStages * kStageBytes;
    static constexpr int kP = kQ + 2 * kTiles * kQuery;
    static constexpr int kScales = kP + kGroups * kWeights;       // two bytes per key of a stage
    static constexpr int kRowFactors = kScales + S::kStages * 2 * S::kUnit;   // float4 [group][warp][R]
    static constexpr int kChanges = kRowFactors + kGroups * kConsumers * R * 16;   // float2
    static constexpr int kMost = kChanges + kGroups * kConsumers * R * 8;          // float2
    static constexpr int kSums = kMost + kGroups * kConsumers * R * 8;   // float [group][R][warp]
    static constexpr int kQueryScales = kSums + kGroups * R * kConsumers * 4;   // float [pair][rows]
    static constexpr int kNan = kQueryScales + kFactorSlots * kTiles * R * 4;   // a bit per row and dim
    static constexpr int kBars = kNan + 2 * 2 * R * 16;
    static constexpr int kBytes = kBars + static_cast<int>(sizeof(Q8Bars)) + 1024;
    static_assert(kQ % 1024 == 0 && kP % 1024 == 0 && kQuery % 1024 == 0 && kWeights % 1024 == 0 &&
                  kBars % 16 == 0 && kBytes <= 232448, "shared memory");
    static constexpr int kOutputs = kGroups * kScoreTiles * kScoreCols;   // first column of O
    static constexpr int kOutputStride = R == 8 ? 32 : 64;
    static constexpr int kColumns = R == 8 ? 128 : 256;
    static_assert(kOutputs + kGroups * kOutputStride <= kColumns, "tensor memory");
};

// Bytes of a stage from 8 keys (or values) to the next 8.
__device__ __forceinline__ uint32_t key_step(const Params &p) { return p.joint ? 2048 : 1024; }

// (Out of line: the records of expired waits are never run in earnest.)
__device__ __noinline__ void expired(int *status, int role, int barrier, int n) {
    set_timeout(status, kDiagPagedDecode, role, barrier, n);
}

template <int N>
__device__ __forceinline__ void tmem_ld(uint32_t at, uint32_t (&r)[N]) {
    if constexpr (N == 8) tmem_ld8(at, r);
    else if constexpr (N == 16) tmem_ld16(at, r);
    else tmem_ld32(at, r);
}
template <int N>
__device__ __forceinline__ void tmem_st(uint32_t at, const uint32_t (&r)[N]) {
    if constexpr (N == 8) tmem_st8(at, r);
    else tmem_st16(at, r);
}

// a[i] of all lanes brought together by `op`, a row in each lane: with R rows R - 1 exchanges of
// halves and then whole ones.  Returns the row's number; a[0] is its value.
template <int R, class Op>
__device__ __forceinline__ int gather_rows(float (&a)[R], Op op) {
    const int lane = threadIdx.x & 31;
    int row = 0;
#pragma unroll
    for (int n = R / 2, d = 16; d > 0; n >>= 1, d >>= 1) {
        const bool up = lane & d;
        if (n > 0) {
#pragma unroll
            for (int i = 0; i < n; ++i) {
                const float keep = up ? a[i + n] : a[i], give = up ? a[i] : a[i + n];
                a[i] = op(keep, __shfl_xor_sync(0xffffffffu, give, d));
            }
            row += up ? n : 0;
        } else {
            a[0] = op(a[0], __shfl_xor_sync(0xffffffffu, a[0], d));
        }
    }
    return row;
}

// byte - 127, the exponent that a scale byte stands for; NaN for 255.
__device__ __forceinline__ float exponent_of(uint32_t byte) {
    return byte == kScaleNan ? CUDART_NAN_F : __uint_as_float(0x4b000000u | byte) - 8388735.0f;
}

// ---- the queries' warp: rows of bf16 to tiles of h and l, with the factor of their scores ------
template <int R, bool SPLIT>
__device__ __forceinline__ void bring_queries(const Params &p, Q8Bars *bars, uint8_t *smem) {
    using L = Layout<R, SPLIT>;
    const int lane = threadIdx.x & 31;
    for (int k = 0;; ++k) {
        const int slot = k & (kSegSlots - 1), b = k & 1;
        if (!warp_wait(&bars->seg_full[slot], (k / kSegSlots) & 1)) {
            expired(p.status, kRoleQueries, 0, k);
            return;
        }
        const Segment sg = bars->seg[slot];
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->seg_free[slot]);
        if (sg.stages < 0) return;
        if (k >= 2 && !warp_wait(&bars->q_free[b], ((k >> 1) - 1) & 1)) {
            expired(p.status, kRoleQueries, 1, k);
            return;
        }
        const int rows = sg.T * p.G;   // <= L::kTiles * R (the host's rule on max_q)
        float *factors = reinterpret_cast<float *>(smem + L::kQueryScales) +
                         k % kFactorSlots * L::kTiles * R;
#pragma unroll 1
        for (int r0 = 0; r0 < L::kTiles * R; r0 += 8) {
            uint2 w[8];                // four dims of eight rows
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int r = r0 + i, t = token_of(p, r);
                w[i] = make_uint2(0, 0);
                if (r < rows && GQA_IN_BOUNDS(sg.row0 + t, p.bounds.total, p.status, kSite | 8))
                    w[i] = __ldg(reinterpret_cast<const uint2 *>(
                        p.q + (long)(sg.row0 + t) * p.q_stride + (sg.g * p.G + r - t * p.G) * kD +
                        4 * lane));
            }
            uint8_t *tile = smem + L::kQ + (b * L::kTiles + r0 / R) * L::kQuery;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int n = r0 % R + i;
                const float x[4] = {bf16lo(w[i].x), bf16hi(w[i].x), bf16lo(w[i].y), bf16hi(w[i].y)};
                uint32_t most = 0;     // (magnitudes compare as their bits do, NaN above all)
#pragma unroll
                for (int e = 0; e < 4; ++e) most = max(most, __float_as_uint(x[e]) & 0x7fffffffu);
                most = __reduce_max_sync(0xffffffffu, most);
                const uint32_t ex = max(most >> 23, 8u);
                const float up = __uint_as_float((261 - ex) << 23);   // 2^(7 - exponent)
                const uint32_t h = to_e4m3x2(x[0] * up, x[1] * up) |
                                   to_e4m3x2(x[2] * up, x[3] * up) << 16;
                uint32_t l = 0;
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const uint32_t y = e4m3x2_f16x2(h >> (16 * e) & 0xffffu);
                    const float2 z = __half22float2(*reinterpret_cast<const __half2 *>(&y));
                    l |= to_e4m3x2((x[2 * e] * up - z.x) * 16.f, (x[2 * e + 1] * up - z.y) * 16.f)
                         << (16 * e);
                }
                // a row with an infinity or NaN: NaN
                uint8_t *at = tile + n * kD + ((lane >> 2 ^ (n & 7)) << 4) + 4 * (lane & 3);
                *reinterpret_cast<uint32_t *>(at) = ex == 255 ? 0x7f7f7f7fu : h;
                *reinterpret_cast<uint32_t *>(at + R * kD) = l;
                if (lane == 0) factors[r0 + i] = __uint_as_float((ex - 7) << 23) * p.scale_log2;
            }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->q_full[b]);
    }
}

// ---- the threads that issue the products, a warp each -------------------------------------------
// (One thread for both took 1500 cycles per stage, as it tests barriers and issues 46 cycles per
// product in turn: 32 caches of 8k-64k tokens 548 us.)
//
// Scores: as soon as a stage's keys, its pair's queries and a score tile of its group are there.
template <int R, bool SPLIT>
__device__ __forceinline__ void issue_scores(const Params &p, Q8Bars *bars, uint8_t *smem,
                                             uint32_t tmem) {
    using L = Layout<R, SPLIT>;
    constexpr int kStages = L::S::kStages;
    const uint32_t ring = smem_u32(smem);
    const uint64_t kd0 = sdesc_sw128(ring + (p.joint && p.v_first ? 1024 : 0), 16, key_step(p));
    const uint64_t qd0 = sdesc_sw128(ring + L::kQ, 16, 1024);
    constexpr uint32_t idesc = idesc_f8_f32(128, L::kScoreCols, 0, 0);
    int n[2] = {0, 0};                 // scores of a group's stages
    for (int k = 0, u = 0;; ++k) {
        const int slot = k & (kSegSlots - 1), b = k & 1;
        if (!mbar_wait(&bars->seg_full[slot], (k / kSegSlots) & 1)) {
            expired(p.status, kRoleProducts, 0, k);
            break;
        }
        const int stages = bars->seg[slot].stages;
        mbar_arrive(&bars->seg_free[slot]);
        if (stages < 0) break;
        bool ok = mbar_wait(&bars->q_full[b], k >> 1 & 1);
        const int g0 = SPLIT ? 0 : b;
        int m = b && !SPLIT ? n[1] : n[0];
        for (int j = 0; ok && j < stages; ++j, ++u, ++m) {
            const int st = u % kStages, tile = m % kScoreTiles;
            if (m >= kScoreTiles)
#pragma unroll
                for (int i = 0; i < L::kTiles; ++i)
                    ok = ok && mbar_wait(&bars->s_free[g0 + i][tile], (m / kScoreTiles - 1) & 1);
            ok = ok && mbar_wait(&bars->full[0][st], (u / kStages) & 1);
            if (!ok) break;
            tc_fence_after();
            const uint64_t kd = kd0 + st * (kStageBytes >> 4);
#pragma unroll
            for (int i = 0; i < L::kTiles; ++i) {
                const uint64_t qd = qd0 + (b * L::kTiles + i) * (L::kQuery >> 4);
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                    umma_f8_ss(tmem + ((g0 + i) * kScoreTiles + tile) * L::kScoreCols, kd + 2 * kk,
                               qd + 2 * kk, idesc, kk > 0);
                // (this thread's own arrival hands on what it has seen: the stage's scale bytes and
                // the queries' factors)
                mbar_arrive(&bars->s_full[g0 + i][tile]);
                umma_commit(&bars->s_full[g0 + i][tile]);
            }
        }
        if (!ok) {
            expired(p.status, kRoleProducts, 1, u);
            break;
        }
        umma_commit(&bars->q_free[b]);
        if (b && !SPLIT) n[1] = m;
        else n[0] = m;
    }
    umma_commit(&bars->drained[0]);    // nothing in flight when the tensor memory is freed
    if (!mbar_wait(&bars->drained[0], 0)) expired(p.status, kRoleProducts, 2, 0);
}

// Values: as soon as a stage's weights are there.
template <int R, bool SPLIT>
__device__ __forceinline__ void issue_values(const Params &p, Q8Bars *bars, uint8_t *smem,
                                             uint32_t tmem) {
    using L = Layout<R, SPLIT>;
    constexpr int kStages = L::S::kStages;
    const uint32_t ring = smem_u32(smem), step = key_step(p);
    const uint64_t vd0 = sdesc_sw128(ring + (!p.joint ? kTileBytes : p.v_first ? 0 : 1024), 16, step);
    const uint64_t pd0 = sdesc_sw128(ring + L::kP, 16, 1024);
    constexpr uint32_t idesc = idesc_f8_f32(128, L::kValueCols, 1, 1);
    int n[2] = {0, 0};                 // a group's products
    for (int k = 0, u = 0;; ++k) {
        const int slot = k & (kSegSlots - 1);
        if (!mbar_wait(&bars->seg_full[slot], (k / kSegSlots) & 1)) {
            expired(p.status, kRoleProducts, 3, k);
            break;
        }
        const int stages = bars->seg[slot].stages;
        mbar_arrive(&bars->seg_free[slot]);
        if (stages < 0) break;
        const int g0 = SPLIT ? 0 : k & 1;
        int m = g0 ? n[1] : n[0];
        bool ok = true;
        for (int j = 0; j < stages; ++j, ++u, ++m) {
            // (both groups': group 0 takes hidden values' NaN out for both)
#pragma unroll
            for (int i = 0; i < L::kTiles; ++i)
                ok = ok && mbar_wait(&bars->p_full[g0 + i], m & 1);
            if (!ok) break;
            tc_fence_after();
            const int st = u % kStages;
            const uint64_t vd = vd0 + st * (kStageBytes >> 4);
#pragma unroll
            for (int i = 0; i < L::kTiles; ++i) {
                const uint64_t pd = pd0 + (g0 + i) * (L::kWeights >> 4);
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                    umma_f8_ss(tmem + L::kOutputs + (g0 + i) * L::kOutputStride,
                               vd + kk * (step >> 2), pd + 2 * kk, idesc, kk > 0 || j > 0);
                umma_commit(&bars->pv_done[g0 + i]);
            }
            umma_commit(&bars->empty[st]);
        }
        if (!ok) {
            expired(p.status, kRoleProducts, 4, u);
            break;
        }
        if (g0) n[1] = m;
        else n[0] = m;
    }
    umma_commit(&bars->drained[1]);
    if (!mbar_wait(&bars->drained[1], 0)) expired(p.status, kRoleProducts, 5, 0);
}

// ---- a softmax group's warp ---------------------------------------------------------------------
template <int R, bool SPLIT>
__device__ __forceinline__ void softmax(const Params &p, Q8Bars *bars, uint8_t *smem, uint32_t tmem) {
    using L = Layout<R, SPLIT>;
    constexpr int kStages = L::S::kStages, kUnit = L::S::kUnit;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int group = warp / kConsumers, cw = warp % kConsumers, tile = SPLIT ? group : 0;
    // (of its group's barriers alone a warp sees every phase: a parity two phases back reads as
    // done, so tiles that the groups shared would be read too early)
    int scored = 0;                    // score tiles read
    const int t = 32 * cw + lane;      // the thread's key of a stage, and its dim of the outputs
    const uint32_t lanes = static_cast<uint32_t>(32 * cw) << 16;
    const uint32_t outputs = tmem + lanes + L::kOutputs + group * L::kOutputStride;
    float4 *rowf = reinterpret_cast<float4 *>(smem + L::kRowFactors) + warp * R;
    float2 *change = reinterpret_cast<float2 *>(smem + L::kChanges) + warp * R;
    float2 *most = reinterpret_cast<float2 *>(smem + L::kMost) + group * kConsumers * R;
    float *sums = reinterpret_cast<float *>(smem + L::kSums) + group * R * kConsumers;
    uint8_t *weights = smem + L::kP + group * L::kWeights;
    const int first_row = SPLIT ? R * group : 0;
    int handed = 0, meets = 0;         // weights handed over; meetings of the group's warps
    auto meet = [&]() {
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->meet[group]);
        return warp_wait(&bars->meet[group], meets++ & 1);
    };
    auto products_done = [&]() {       // of all weights handed over
        return handed == 0 || warp_wait(&bars->pv_done[group], (handed - 1) & 1);
    };
    auto fail = [&](int barrier, int n) { expired(p.status, kRoleConsumer, barrier, n); };
#pragma unroll 1
    for (int k = SPLIT ? 0 : group, turn = 0;; k += SPLIT ? 1 : kGroups, turn ^= 1) {
        const int slot = k & (kSegSlots - 1);
        if (!warp_wait(&bars->seg_full[slot], (k / kSegSlots) & 1)) return fail(0, k);
        const Segment sg = bars->seg[slot];
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->seg_free[slot]);
        if (sg.stages < 0) return;
        const int rows = max(0, min(R, sg.T * p.G - first_row));
        const int q_first = sg.S - sg.T;          // keys beyond are hidden from some
        const int lo = p.window > 0 ? max(0, q_first - p.window + 1) : 0;
        const int lo_all = p.window > 0 ? max(0, sg.S - p.window) : 0;
        // NaN among the values' numbers: a bit per row and dim of this pair, and of the last one
        uint32_t *nan = reinterpret_cast<uint32_t *>(smem + L::kNan);
        auto nan_row = [&](int which, int r) {    // r: of the pair
            return nan + ((SPLIT ? which : 2 * group + which) * L::kTiles * R + r) * 4;
        };
        float m = -CUDART_INF_F, mo = -CUDART_INF_F;   // of row `lane`
        float l[R];
#pragma unroll
        for (int r = 0; r < R; ++r) l[r] = 0.f;
#pragma unroll 1
        for (int j = 0, u = sg.u0; j < sg.stages; ++j, ++u) {
            const int st = u % kStages, si = scored % kScoreTiles;
            if (!warp_wait(&bars->s_full[group][si], (scored / kScoreTiles) & 1)) return fail(1, u);
            ++scored;
            tc_fence_after();
            float y[R];
            uint32_t bytes;
            {
                uint32_t s[2 * R];
                tmem_ld<2 * R>(tmem + lanes + (group * kScoreTiles + si) * L::kScoreCols, s);
                bytes = reinterpret_cast<const uint16_t *>(smem + L::kScales)[st * kUnit + t];
                const float kf = scale_of(bytes & 255u), kl = kf * 0.0625f;
                tmem_wait_ld();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars->s_free[group][si]);
#pragma unroll
                for (int r = 0; r < R; ++r)
                    y[r] = fmaf(__uint_as_float(s[R + r]), kl, __uint_as_float(s[r]) * kf);
            }
            const float vf = scale_of(bytes >> 8);
            const int kb = (sg.unit0 + j) * kUnit, key = kb + t;
            const bool edge = kb + kUnit - 1 > q_first || kb < lo_all;   // of the mask
            uint32_t hidden = 0;       // a bit per row
            if (edge) {
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    const int at = q_first + min(token_of(p, first_row + r), sg.T - 1);
                    if (key > at || (p.window > 0 && at - key >= p.window)) {
                        hidden |= 1u << r;
                        y[r] = -CUDART_INF_F;
                    }
                }
            }
            // ---- weights w and products P, against new references where the old ones are passed
            float w[R], pw[R];
            bool update = j == 0;
#pragma unroll 1
            while (true) {
                if (update) {
                    const float ev = fmaxf(exponent_of(bytes >> 8), kLeast);
                    const float *factors =
                        reinterpret_cast<const float *>(smem + L::kQueryScales) +
                        (k % kFactorSlots * L::kTiles + tile) * R;
                    float a[R], b[R];
#pragma unroll
                    for (int r = 0; r < R; ++r) {
                        a[r] = y[r] * factors[r];
                        b[r] = a[r] + ev;
                    }
                    auto larger = [](float c, float d) { return fmaxf(c, d); };
                    const int row = gather_rows(a, larger);
                    gather_rows(b, larger);
                    if ((lane & (32 / R - 1)) == 0) most[cw * R + row] = make_float2(a[0], b[0]);
                    if (!meet()) return fail(3, u);
                    if (lane < R) {
                        float mn = m, mno = mo;
#pragma unroll
                        for (int c = 0; c < kConsumers; ++c) {
                            const float2 x = most[c * R + lane];
                            mn = fmaxf(mn, x.x);
                            mno = fmaxf(mno, x.y);
                        }
                        change[lane] =
                            make_float2(m == -CUDART_INF_F ? 0.f : ex2_approx(m - mn),
                                        mo == -CUDART_INF_F ? 1.f : ex2_approx(mo - mno));
                        m = mn;
                        mo = mno;
                        rowf[lane] =
                            make_float4(factors[lane], -fmaxf(mn, -3.0e38f),
                                        mn == -CUDART_INF_F ? 0.f : ex2_approx(mn - mno + kShift), 0.f);
                        if (j == 0 && cw == 0) {  // the last pair's bits have been read
                            uint32_t *z = nan_row(turn ^ 1, first_row + lane);
                            z[0] = z[1] = z[2] = z[3] = 0;
                            if (lane == 0) bars->nan_any[group][turn ^ 1] = 0;
                        }
                    }
                    __syncwarp();
                    if (j > 0) {
                        if (!products_done()) return fail(4, u);
                        tc_fence_after();
#pragma unroll 1
                        for (int c = 0; c < 3; ++c) {
                            uint32_t o[R];
                            tmem_ld<R>(outputs + c * R, o);
                            tmem_wait_ld();
#pragma unroll
                            for (int r = 0; r < R; ++r)
                                o[r] = __float_as_uint(__uint_as_float(o[r]) * change[r].y);
                            tmem_st<R>(outputs + c * R, o);
                        }
                        tmem_wait_st();
                        tc_fence_before();
#pragma unroll
                        for (int r = 0; r < R; ++r) l[r] *= change[r].x;
                    }
                }
                bool over = false;
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    const float4 f = rowf[r];
                    const float x = fmaf(y[r], f.x, f.y);
                    w[r] = ex2_approx(x);
                    pw[r] = w[r] * f.z * vf;
                    over |= x > kGrow || pw[r] > kLargest;
                }
                if (update) break;
                if (__any_sync(0xffffffffu, over) && lane == 0) bars->vote[group][u & 1] = u + 1;
                if (!meet()) return fail(5, u);
                if (*const_cast<volatile int *>(&bars->vote[group][u & 1]) != u + 1) break;
                update = true;
            }
            if (edge) {
#pragma unroll
                for (int r = 0; r < R; ++r)
                    if (hidden >> r & 1) pw[r] = 0.f;   // (its value's byte may be NaN)
            }
            // ---- P, a byte per column, row and key
            if (!products_done()) return fail(4, u);    // the last ones have been read
#pragma unroll
            for (int r = 0; r < R; r += 2) {
                l[r] += w[r];
                l[r + 1] += w[r + 1];
                const __half2 x = __floats2half2_rn(pw[r], pw[r + 1]);
                const uint32_t c = *reinterpret_cast<const uint32_t *>(&x) & 0xff00ff00u;
                const __half2 x1 = __hsub2(x, *reinterpret_cast<const __half2 *>(&c));
                const uint32_t d = *reinterpret_cast<const uint32_t *>(&x1) & 0xff00ff00u;
                const __half2 x2 = __hsub2(x1, *reinterpret_cast<const __half2 *>(&d));
                const uint32_t f = to_e5m2x2(x2);
                uint8_t *at = weights + r * kD + (t ^ ((r & 7) << 4));
                uint8_t *at1 = weights + (r + 1) * kD + (t ^ ((r + 1 & 7) << 4));
                at[0] = static_cast<uint8_t>(c >> 8);
                at1[0] = static_cast<uint8_t>(c >> 24);
                at[R * kD] = static_cast<uint8_t>(d >> 8);
                at1[R * kD] = static_cast<uint8_t>(d >> 24);
                at[2 * R * kD] = static_cast<uint8_t>(f);
                at1[2 * R * kD] = static_cast<uint8_t>(f >> 8);
            }
            // ---- values that the mask hides: 0 * NaN is NaN
            if (edge && (!SPLIT || group == 0)) {
                uint8_t *vr = smem + st * kStageBytes +
                              (!p.joint ? kTileBytes + t * kD
                                        : (t >> 3) * 2048 + (p.v_first ? 0 : 1024) + (t & 7) * kD);
                if (key >= sg.S || key < lo) {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        reinterpret_cast<uint4 *>(vr)[i] = make_uint4(0, 0, 0, 0);
                } else if (key > q_first || key < lo_all) {
                    // some rows see it: its NaN are taken out, and noted for the rows that do
#pragma unroll 1
                    for (int i = 0; i < kD / 4; ++i) {
                        uint32_t *at = reinterpret_cast<uint32_t *>(vr) + i;
                        const uint32_t x = *at;
                        uint32_t bad = __vcmpeq4(x & 0x7f7f7f7fu, 0x7f7f7f7fu);
                        if (!bad) continue;
                        *at = x & ~bad;
                        const int dim = 16 * (i >> 2 ^ (t & 7)) + 4 * (i & 3);
                        for (int e = 0; e < 4; ++e) {
                            if (!(bad >> (8 * e) & 1)) continue;
                            for (int r = 0; r < min(sg.T * p.G, L::kTiles * R); ++r) {
                                const int pos = q_first + token_of(p, r);
                                if (key > pos || (p.window > 0 && pos - key >= p.window)) continue;
                                atomicOr(nan_row(turn, r) + (dim + e) / 32, 1u << ((dim + e) & 31));
                                bars->nan_any[SPLIT ? r / R : group][turn] = 1;
                            }
                        }
                    }
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars->p_full[group]);
            ++handed;
        }
        // ---- the pair's (or span's) result: this thread's dim of all rows
        {
            const int row = gather_rows(l, [](float a, float b) { return a + b; });
            if ((lane & (32 / R - 1)) == 0) sums[row * kConsumers + cw] = l[0];
            // O relative to m: times 2^(mo - 12 - m), in two steps as that may be 2^-138
            if (lane < R)
                change[lane].x =
                    mo == -CUDART_INF_F ? 1.f : ex2_approx(0.5f * (mo - kShift - m));
        }
        if (!meet()) return fail(6, k);
        if (!products_done()) return fail(4, k);
        tc_fence_after();
        float o[R];
        {
            uint32_t a[R], b[R], c[R];
            tmem_ld<R>(outputs, a);
            tmem_ld<R>(outputs + R, b);
            tmem_ld<R>(outputs + 2 * R, c);
            tmem_wait_ld();
            tc_fence_before();
#pragma unroll
            for (int r = 0; r < R; ++r)
                o[r] = __uint_as_float(a[r]) + (__uint_as_float(b[r]) + __uint_as_float(c[r]));
        }
        const bool nans = *const_cast<volatile int *>(&bars->nan_any[group][turn]) != 0;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            if (r >= rows) continue;
            float x = o[r] * change[r].x * change[r].x;
            if (nans && nan_row(turn, first_row + r)[t / 32] >> (t & 31) & 1) x = CUDART_NAN_F;
            const int n = first_row + r;
            if (sg.slot >= 0) {
                const size_t rec = (size_t)sg.slot * p.rec_rows + n;
                if (GQA_IN_BOUNDS(rec, (long)2 * p.chunks * p.rec_rows, p.status, kSite | 9))
                    p.ws_o[rec * kD + t] = x;
            } else {
                const float4 s = *reinterpret_cast<const float4 *>(sums + r * kConsumers);
                const int tok = token_of(p, n), head = sg.g * p.G + n - tok * p.G;
                const long row = sg.row0 + tok;
                if (GQA_IN_BOUNDS(row, p.bounds.total, p.status, kSite | 10))
                    p.o[row * p.o_stride + head * kD + t] =
                        __float2bfloat16_rn(x * (1.0f / ((s.x + s.y) + (s.z + s.w))));
            }
        }
        if (cw == 0 && lane < rows) {
            const float4 s = *reinterpret_cast<const float4 *>(sums + lane * kConsumers);
            const float sum = (s.x + s.y) + (s.z + s.w);
            const int n = first_row + lane;
            if (sg.slot >= 0) {
                const size_t rec = (size_t)sg.slot * p.rec_rows + n;
                if (GQA_IN_BOUNDS(rec, (long)2 * p.chunks * p.rec_rows, p.status, kSite | 11))
                    reinterpret_cast<float2 *>(p.ws_ml)[rec] = make_float2(m, sum);
            } else if (p.lse) {
                const int tok = token_of(p, n), head = sg.g * p.G + n - tok * p.G;
                const long row = sg.row0 + tok;
                if (GQA_IN_BOUNDS(row, p.bounds.total, p.status, kSite | 12))
                    p.lse[(long)head * p.bounds.total + row] =
                        (m + __log2f(sum)) * 0.69314718055994531f;
            }
        }
    }
}

// R: rows of a group.  SPLIT: both groups on each pair, R rows each.
template <int R, bool SPLIT>
__global__ void __launch_bounds__(Q8Stream<SPLIT>::kThreads, 1)
    paged_q8_kernel(const __grid_constant__ CUtensorMap tmK,
                    const __grid_constant__ CUtensorMap tmV, const Params p) {
    griddep_wait();
    griddep_launch_dependents();
    using L = Layout<R, SPLIT>;
    using S = typename L::S;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_addr = smem_u32(smem_raw);
    uint8_t *smem = smem_raw + (((raw_addr + 1023u) & ~1023u) - raw_addr);
    Q8Bars *bars = reinterpret_cast<Q8Bars *>(smem + L::kBars);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < S::kStages; ++i) {
            mbar_init(&bars->full[0][i], S::kUnit / min(p.page_size, S::kUnit) + kScaleCopies);
            mbar_init(&bars->empty[i], 1);
        }
        for (int i = 0; i < kSegSlots; ++i) {
            mbar_init(&bars->seg_full[i], 1);
            mbar_init(&bars->seg_free[i], S::kReaders * kConsumers + 3);
        }
        for (int g = 0; g < kGroups; ++g) {
            mbar_init(&bars->q_full[g], 1);
            mbar_init(&bars->q_free[g], 1);
            for (int i = 0; i < kScoreTiles; ++i) {
                mbar_init(&bars->s_full[g][i], 2);
                mbar_init(&bars->s_free[g][i], kConsumers);
            }
            mbar_init(&bars->p_full[g], kConsumers);
            mbar_init(&bars->pv_done[g], 1);
            mbar_init(&bars->meet[g], kConsumers);
            mbar_init(&bars->drained[g], 1);
            for (int i = 0; i < 2; ++i) bars->vote[g][i] = bars->nan_any[g][i] = 0;
        }
        mbar_init(&bars->clc_full, 1);
        fence_mbar_init();
    }
    // columns of P that no weight is written to, and the NaN bits
    for (int i = threadIdx.x; i < kGroups * L::kWeights / 16; i += S::kThreads)
        reinterpret_cast<uint4 *>(smem + L::kP)[i] = make_uint4(0, 0, 0, 0);
    for (int i = threadIdx.x; i < 2 * 2 * R; i += S::kThreads)
        reinterpret_cast<uint4 *>(smem + L::kNan)[i] = make_uint4(0, 0, 0, 0);
    fence_proxy_async_smem();
    if (warp == kScoreWarp) {
        tmem_alloc(&bars->tmem, L::kColumns);
        tmem_relinquish();
    }
    scan_units<S>(p, bars);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bars->tmem;
    if (warp < kGroups * kConsumers) softmax<R, SPLIT>(p, bars, smem, tmem);
    else if (warp == kProducerWarp) produce<S>(tmK, tmV, p, bars, smem, smem + L::kScales);
    else if (warp == kQueryWarp) bring_queries<R, SPLIT>(p, bars, smem);
    else if (warp == kScoreWarp && lane == 0) issue_scores<R, SPLIT>(p, bars, smem, tmem);
    else if (warp == kValueWarp && lane == 0) issue_values<R, SPLIT>(p, bars, smem, tmem);
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == kScoreWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, L::kColumns);
    }
}

constexpr int kStreamRows = 32;      // up to here the streaming kernel
int rows_of(int max_q, int Hq, int Hkv) {
    const long n = static_cast<long>(max_q) * (Hq / Hkv);
    return n > kStreamRows ? 0 : n > 16 ? 32 : 16;   // of a partial; 0: the tile kernel
}

int launch_stream(const PackedAttn &a, const gqa_paged_kv_q8 &c, int rows, void *ws, int *status,
                  cudaStream_t s) {
    Params p = params_of(a, Q8Stream<false>::kUnit, rows, ws, status);
    p.scales = static_cast<const uint8_t *>(c.scales);
    // {128 numbers, 8 keys, the two pools, groups of 8 keys, (page, KV head)}: a map takes a stride
    // from pool to pool below 2^40, and then a page's keys and values come as one copy, 8 of either
    // in turn (32 caches of 8k-64k tokens in pages of 16: 577 us with two copies, 458 with one);
    // else as two.
    const uint64_t kp = reinterpret_cast<uint64_t>(c.k), vp = reinterpret_cast<uint64_t>(c.v);
    const uint64_t apart = kp < vp ? vp - kp : kp - vp, page = c.page_size;
    p.joint = apart > 0 && apart < (1ull << 40);
    p.v_first = p.joint && vp < kp;
    const uint32_t pools = p.joint ? 2 : 1;
    const uint64_t dims[5] = {kD, 8, pools, page / 8, (uint64_t)c.num_pages * c.Hkv};
    const uint64_t strides[4] = {kD, p.joint ? apart : kD, 8 * kD, page * kD};
    const uint32_t box[5] = {kD, 8, pools, (uint32_t)page / 8, 1};
    CUtensorMap mk, mv;
    if (!make_byte_map(&mk, p.v_first ? c.v : c.k, 5, dims, strides, box) ||
        !make_byte_map(&mv, c.v, 5, dims, strides, box))
        return GQA_ERR_CUDA;
    const long pairs = (long)a.nseq * a.Hkv;
    const long grid = !p.whole ? p.chunks : pairs < kSMs ? pairs : kSMs;
    const bool eight = static_cast<long>(a.max_q) * p.G <= 8;
    auto kern = rows == 32 ? paged_q8_kernel<16, true>
                : eight    ? paged_q8_kernel<8, false>
                           : paged_q8_kernel<16, false>;
    const int bytes = rows == 32 ? Layout<16, true>::kBytes
                      : eight    ? Layout<8, false>::kBytes
                                 : Layout<16, false>::kBytes;
    if (ensure_smem_attr(reinterpret_cast<const void *>(kern), bytes) != cudaSuccess ||
        launch_pdl(kern, dim3(static_cast<unsigned>(grid)), dim3(Q8Stream<false>::kThreads), bytes, s,
                   mk, mv, p) != cudaSuccess)
        return GQA_ERR_CUDA;
    if (!p.whole && launch_combine(p, a.max_q, s) != cudaSuccess) return GQA_ERR_CUDA;
    return GQA_OK;
}

}  // namespace

bool paged_q8_counts_fit(int nseq, int total, int max_q, int max_kv, int Hq, int Hkv) {
    return rows_of(max_q, Hq, Hkv) ? paged_decode_counts_fit(nseq, max_kv, Hkv)
                                   : paged_expand_counts_fit(nseq, max_kv, Hkv) &&
                                         packed_prefill_counts_fit(nseq, total, max_kv, Hq, Hkv);
}

size_t paged_q8_workspace_bytes(int nseq, int total, int max_q, int max_kv, int Hq, int Hkv) {
    if (const int rows = rows_of(max_q, Hq, Hkv))
        return whole_pairs(max_kv) ? 0
                                   : partials_bytes(n_chunks(nseq, max_kv, Hkv, 1, 0,
                                                             Q8Stream<false>::kUnit), rows);
    return paged_expand_q8_bytes(nseq, max_kv, Hkv) +
           packed_prefill_workspace_bytes(nseq, total, max_kv, Hq, Hkv);
}

int launch_paged_q8(const PackedAttn &a, const gqa_paged_kv_q8 &c, void *ws, int *status,
                    cudaStream_t s) {
    gqa_paged_kv pages = {c.k, c.v, c.page_table, c.kv_lens, c.num_pages, c.Hkv, c.page_size, c.d,
                          c.max_pages, 0};
    PackedAttn b = a;
    b.cache = &pages;
    if (const int rows = rows_of(a.max_q, a.Hq, a.Hkv))
        return launch_stream(b, c, rows, ws, status, s);
    if (launch_paged_expand_q8(c, a, ws, &pages, status, s) != cudaSuccess) return GQA_ERR_CUDA;
    b.k = pages.k;
    b.v = pages.v;
    b.cap = (long)c.max_pages * c.page_size;
    return launch_packed_prefill(
        b, static_cast<char *>(ws) + paged_expand_q8_bytes(a.nseq, a.max_kv, a.Hkv), status, s);
}

}  // namespace gqa
