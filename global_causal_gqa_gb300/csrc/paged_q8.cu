// paged_q8.cu -- attention over the 8-bit paged cache (d = 128).
//
// For query token t of a sequence with S keys and T new tokens, at position i = S - T + t, over
// keys 2^a_j y_j and values 2^b_j z_j of e4m3 numbers y, z (q8.cuh):
//   o = sum_j softmax_j(scale 2^a_j q . y_j) 2^b_j z_j  over j <= i (and i - j < W with a window).
//
// By the rows (tokens x heads of a KV group) that a sequence may have: up to 8, paged_q8_few.cu, or
// paged_q8_short.cu for many short caches; 9 to 96, the kernel below, bound by memory at 16 rows
// (32 caches of 8k-64k tokens 435 us, 6.3 TB/s) and by its warps at 32 (557 us; blocks of 32 rows
// read the pages again, from L2 for the most part: 24 drafts of 2-6 tokens of 8 rows 77 us).  More:
// all keys that the call sees are expanded to bf16 pages in the workspace (paged_read.cu) and the
// tile kernel (packed_prefill.cu) takes them from there (24 times 72, 96 and 128 rows over 700-6000
// tokens: 184, 186 and 190 us so, 158, 169 and 220 in blocks; 16 to 96 rows 179 and 106; 8 times 96
// over 20k-60k 605 and 439).
//
// The kernel is cut and fed as the bf16 one (paged_decode.cu; paged_stream.cuh), in stages of 128
// keys.  Its products run on tcgen05 with the numbers as they lie in the pages:
//   S^T [128 keys x columns] = Y Q'^T,   O^T [128 dims x columns] += Z^T P'^T,
// e4m3 A operands straight from the stage, so that no thread ever touches a key's number (by
// mma.sync, 16 rows of these caches took 575 us: the conversions alone were more than the copies).
// The operands that are not 8-bit are sums of 8-bit columns:
//   q 2^u = h + l / 16 (e4m3, the row's largest element brought to [2^7, 2^8)): bf16's 8 bits, but
//     for elements below 2^-3, which lose at most 2^-14, 2^-21 of the largest;
//   P = c + m + f (e5m2, a weight times its value's 2^b): of P in f16 the upper byte, the upper byte
//     of what is left, and the rest rounded: off by 2^-9 + 2^-11 of P, or 2^-17.
// A thread has one key and 8 rows: its key's and value's powers of two are its own, the rows'
// factors are read from shared memory.  l sums the weights relative to 2^m, O the products P
// relative to 2^(m + mo - 12), mo the largest score plus its value's exponent, less m: either range
// alone may be far from the other's.  Both references move, for all keys of a stage together, when
// something exceeds them by 2^3, so that P stays within e5m2's range and 2^-17 is 2^-29 of its
// largest.
//
// Warps: four groups of four for the softmax (8 rows; a warp a quarter of a stage's keys), the
// producer, one that issues the score products and one the value products (one thread for both
// took 1500 cycles a stage), and one that brings the queries into operands a pair ahead.  Two
// groups are a team for up to 16 rows, and the teams take the pairs in turn, so that one's ends
// pass while the other streams, or (SHARE, where a CTA has few pairs) each pair's stages; four for
// up to 32.  A stage of 32 rows takes 2000 cycles, of 24 nearly as many: it is a warp's own chain
// of some 300 instructions, with five warps on a scheduler, that counts (scores out of tensor
// memory 330 cycles, weights 450, the vote 250, their bytes 340, each wait about 150 although what
// it waits for is there).  So the threads' stores count (weights key by key, 24 bytes in 3 stores,
// instead of a byte per column: 32 rows 671 -> 603 us), waits (one for a stage's scores and for the
// tile that its weights go to: 557), and paired fp32 arithmetic.
#include "paged_stream.cuh"
#include "q8.cuh"

namespace gqa {
using namespace stream;
namespace {

constexpr int kRows = 8;             // of a group
constexpr int kStreamUnit = 128;
constexpr int kScoreTiles = 2;       // of a team, in tensor memory
constexpr int kWeightTiles = 2;      // of a team, in shared memory
static_assert(kWeightTiles == kScoreTiles, "a stage's scores and weights have tiles of one number");
constexpr int kScoreCols = 2 * kRows, kValueCols = 3 * kRows;   // columns of a group
constexpr int kChunk = 16 * kStreamUnit;      // bytes of 16 columns of the weights
constexpr float kGrow = 3.0f, kShift = 12.0f, kLargest = 32768.0f;   // log2 units; 2^(3 + 12)
// Values of powers below 2^-112 count as 2^-112 in mo, so that a weight of up to 2^3 times 2^(12 - mo)
// stays within fp32: the products of the smallest, 2^-126, are 2^-2, and lose 2^-15 of that.
constexpr float kLeast = -112.0f;

struct Q8Bars : StreamBars {
    uint64_t q_full[4], q_free[4], q_raw;
    // of a team: a stage's scores are there, and the weights before its own read; the scores read
    uint64_t s_full[4][kScoreTiles], s_free[4][kScoreTiles];
    uint64_t p_full[4][kWeightTiles], pv_done[4][kWeightTiles];   // of a team
    uint64_t gathered, taken;        // the teams' shares of a pair: written; read
    uint64_t drained[2];
    float2 share[4][8];              // (m, l) of a group's rows
    uint32_t tmem;
    int nan_any[4][2];
};

// Where a row's result goes: its dims (of a partial in fp32, else in bf16), and its sum, or its lse.
struct Place {
    void *o, *sum;
};

// TEAM groups share a pair, kRows rows each; the teams take the pairs in turn, or (SHARE) each pair's
// stages.
template <int TEAM, bool SHARE>
struct Layout {
    using S = Q8Stream<TEAM, SHARE>;
    static constexpr int kTeams = S::kTeams, kGroups = S::kGroups, kTeamRows = TEAM * kRows;
    static constexpr int kScoreWarp = S::kProducer + 1, kValueWarp = S::kProducer + 2,
                         kQueryWarp = S::kProducer + 3;
    // columns of a team's products (a multiple of 16)
    static constexpr int kScoreN = TEAM * kScoreCols, kValueN = TEAM * kValueCols;
    static constexpr int kQuerySlots = 2;
    // A pair's factors are read after its queries' tile is free again: the scores of as many stages
    // as the teams have tiles may be formed by then, and the queries of the pairs after those,
    // as many as have a tile, be there.
    static constexpr int kFactorSlots = 8;
    // tensor memory: score tiles, then outputs
    static constexpr int kOutputs = kTeams * kScoreTiles * kScoreN, kColumns = 256;
    static_assert(kOutputs + kTeams * kValueN <= kColumns, "tensor memory");
    // shared memory
    static constexpr int kQuery = kScoreN * kD, kWeights = kValueN * kD;   // bytes of a tile
    static constexpr int kQ = S::kStages * kStageBytes;
    static constexpr int kP = kQ + kQuerySlots * kQuery;
    static constexpr int kScales = kP + kTeams * kWeightTiles * kWeights;        // two bytes per key of a stage
    static constexpr int kRowFactors = kScales + S::kStages * 2 * S::kUnit;   // float [warp][2][8]
    static constexpr int kChanges = kRowFactors + kGroups * kConsumers * kRows * 8;    // float2
    static constexpr int kMost = kChanges + kGroups * kConsumers * kRows * 8;          // float2
    static constexpr int kSums = kMost + kGroups * kConsumers * kRows * 8;   // float [group][row][warp]
    static constexpr int kFactors = kSums + kGroups * kRows * kConsumers * 4;   // float [pair][row]
    static constexpr int kNan = kFactors + kFactorSlots * kTeamRows * 4;   // a bit per row and dim
    static constexpr int kRaw = kNan + kTeams * 2 * kTeamRows * 16;   // a pair's queries in bf16
    static constexpr int kPlaces = kRaw + kTeamRows * kD * 2;         // Place [pair][row]
    static constexpr int kShares = kPlaces + kFactorSlots * kTeamRows * 16;   // float [group][row][dim]
    static constexpr int kBars = kShares + (SHARE ? kGroups * kRows * kD * 4 : 0);
    static constexpr int kBytes = kBars + static_cast<int>(sizeof(Q8Bars)) + 1024;
    static_assert(kQ % 1024 == 0 && kP % 1024 == 0 && kQuery % 1024 == 0 && kWeights % 1024 == 0 &&
                  kBars % 16 == 0 && kBytes <= 232448, "shared memory");
};

// Whether a thread of the `threads` that meet at barrier `id` says so.
__device__ __forceinline__ bool group_any(int id, int threads, bool mine) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
        "barrier.cta.red.or.pred q, %2, %3, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"(static_cast<uint32_t>(mine)), "r"(id), "r"(threads)
        : "memory");
    return r != 0;
}

// 255 in the bytes that are NaN among the four e4m3 in x.
__device__ __forceinline__ uint32_t nan_bytes(uint32_t x) {
    return __vcmpeq4(x & 0x7f7f7f7fu, 0x7f7f7f7fu);
}

// Two f16 numbers less their upper bytes as such, exactly.
__device__ __forceinline__ uint32_t less_upper(uint32_t x) {
    const uint32_t u = x & 0xff00ff00u;
    const __half2 y = __hsub2(*reinterpret_cast<const __half2 *>(&x), *reinterpret_cast<const __half2 *>(&u));
    return *reinterpret_cast<const uint32_t *>(&y);
}

// (Out of line: the records of expired waits are never run in earnest.)
__device__ __noinline__ void expired(int *status, int role, int barrier, int n) {
    set_timeout(status, kDiagPagedDecode, role, barrier, n);
}

// A score that others are taken relative to.
__device__ __forceinline__ float finite(float m) { return fmaxf(m, -3.0e38f); }

// The rows' a[i] of all lanes brought together by `op`, in 9 exchanges: of halves, then whole.
// Returns the row whose value the lane has in a[0].
template <class Op>
__device__ __forceinline__ int gather_rows(float (&a)[kRows], Op op) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int n = kRows / 2, d = 16; d > 0; n >>= 1, d >>= 1) {
        if (n > 0) {
#pragma unroll
            for (int i = 0; i < n; ++i) {
                const float keep = lane & d ? a[i + n] : a[i], give = lane & d ? a[i] : a[i + n];
                a[i] = op(keep, __shfl_xor_sync(0xffffffffu, give, d));
            }
        } else {
            a[0] = op(a[0], __shfl_xor_sync(0xffffffffu, a[0], d));
        }
    }
    return lane >> 2;
}

// ---- the queries' warp: rows of bf16 to tiles of h and l, with the factor of their scores ------
template <int TEAM, bool SHARE>
__device__ __forceinline__ void bring_queries(const Params &p, Q8Bars *bars, uint8_t *smem) {
    using L = Layout<TEAM, SHARE>;
    constexpr int kSegSlots = L::S::kSegSlots;
    const int lane = threadIdx.x & 31;
    for (int k = 0;; ++k) {
        const int slot = k % kSegSlots, b = k % L::kQuerySlots;
        if (!quick_wait(&bars->seg_full[slot], (k / kSegSlots) & 1)) {
            expired(p.status, kRoleQueries, 0, k);
            return;
        }
        const Segment sg = bars->seg[slot];
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->seg_free[slot]);
        if (sg.stages < 0) return;
        if (k >= L::kQuerySlots && !quick_wait(&bars->q_free[b], (k / L::kQuerySlots - 1) & 1)) {
            expired(p.status, kRoleQueries, 1, k);
            return;
        }
        const int rows = sg.T * p.G - sg.r0;
        float *factors = reinterpret_cast<float *>(smem + L::kFactors) +
                         k % L::kFactorSlots * L::kTeamRows;
        uint8_t *tile = smem + L::kQ + b * L::kQuery;
        // The rows as they lie, a token's heads by one copy; meanwhile where their results go.
        const int n_rows = min(rows, L::kTeamRows);
        const int tok0 = token_of(p, sg.r0), toks = token_of(p, sg.r0 + n_rows - 1) - tok0 + 1;
        if (lane == 0) mbar_arrive_expect_tx(&bars->q_raw, n_rows * kD * 2);
        __syncwarp();
        if (lane < toks) {
            const int t = tok0 + lane, h0 = max(0, sg.r0 - t * p.G);
            const int h1 = min(p.G, sg.r0 + n_rows - t * p.G);
            long at = sg.row0 + t;
            if (!GQA_IN_BOUNDS(at, p.bounds.total, p.status, kSite | 8)) at = 0;
            bulk_copy_g2s(smem + L::kRaw + (t * p.G + h0 - sg.r0) * kD * 2,
                          p.q + at * p.q_stride + (sg.g * p.G + h0) * kD, (h1 - h0) * kD * 2,
                          &bars->q_raw);
        }
        if (lane < L::kTeamRows) {
            Place to{nullptr, nullptr};
            if (lane < n_rows && sg.slot >= 0) {
                const size_t rec = (size_t)sg.slot * p.rec_rows + lane;
                if (GQA_IN_BOUNDS(rec, (long)2 * p.chunks * p.rec_rows, p.status, kSite | 9))
                    to = {p.ws_o + rec * kD, p.ws_ml + rec * 2};
            } else if (lane < n_rows) {
                const int r = sg.r0 + lane, tok = token_of(p, r), head = sg.g * p.G + r - tok * p.G;
                const long at = sg.row0 + tok;
                if (GQA_IN_BOUNDS(at, p.bounds.total, p.status, kSite | 10))
                    to = {p.o + at * p.o_stride + head * kD,
                          p.lse ? p.lse + (long)head * p.bounds.total + at : nullptr};
            }
            reinterpret_cast<Place *>(smem + L::kPlaces)[k % L::kFactorSlots * L::kTeamRows + lane] = to;
        }
        if (!quick_wait(&bars->q_raw, k & 1)) {
            expired(p.status, kRoleQueries, 2, k);
            quick_wait(&bars->q_raw, k & 1);   // never leave the CTA with copies in flight
            return;
        }
        // A group's rows at a time, four lanes to a row, 4 x 8 dims each (a group without rows reads
        // nothing of its tile; two rows at a time took 5200 cycles for 32, which a kernel's first pair
        // waits for).
        const int n = lane >> 2, part = lane & 3;
#pragma unroll 1
        for (int i0 = 0; i0 < n_rows; i0 += kRows) {
            const int row = i0 + n;
            uint4 w[4];
            uint32_t most = 0;         // (magnitudes compare as their bits do, NaN above all)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                w[j] = make_uint4(0, 0, 0, 0);
                if (row < n_rows)
                    w[j] = *reinterpret_cast<const uint4 *>(smem + L::kRaw + row * kD * 2 +
                                                            16 * (part + 4 * j));
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t words[4] = {w[j].x, w[j].y, w[j].z, w[j].w};
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    most = max(most, max(words[e] << 16 & 0x7fffffffu, words[e] & 0x7fff0000u));
            }
            most = max(most, __shfl_xor_sync(0xffffffffu, most, 1));
            most = max(most, __shfl_xor_sync(0xffffffffu, most, 2));
            const uint32_t ex = max(most >> 23, 8u);
            const float up = __uint_as_float((261 - ex) << 23);   // 2^(7 - exponent)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t words[4] = {w[j].x, w[j].y, w[j].z, w[j].w};
                uint32_t h[2] = {0, 0}, l[2] = {0, 0};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float x0 = bf16lo(words[e]) * up, x1 = bf16hi(words[e]) * up;
                    const uint32_t y = to_e4m3x2(x0, x1), back = e4m3x2_f16x2(y);
                    const float2 z = __half22float2(*reinterpret_cast<const __half2 *>(&back));
                    h[e >> 1] |= y << (16 * (e & 1));
                    l[e >> 1] |= to_e4m3x2((x0 - z.x) * 16.f, (x1 - z.y) * 16.f) << (16 * (e & 1));
                }
                // row n of its group: h in the tile's row 16 g + n, l in row 16 g + 8 + n; a row with
                // an infinity or NaN: NaN
                const int c = part + 4 * j;
                uint8_t *at = tile + (2 * i0 + n) * kD + ((c >> 1 ^ n) << 4) + 8 * (c & 1);
                *reinterpret_cast<uint2 *>(at) =
                    ex == 255 ? make_uint2(0x7f7f7f7fu, 0x7f7f7f7fu) : make_uint2(h[0], h[1]);
                *reinterpret_cast<uint2 *>(at + kRows * kD) = make_uint2(l[0], l[1]);
            }
            if (part == 0) factors[row] = __uint_as_float((ex - 7) << 23) * p.scale_log2;
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
// Scores: as soon as a stage's keys, its pair's queries and a score tile of its team are there.
template <int TEAM, bool SHARE>
__device__ __forceinline__ void issue_scores(const Params &p, Q8Bars *bars, uint8_t *smem,
                                             uint32_t tmem) {
    using L = Layout<TEAM, SHARE>;
    constexpr int kStages = L::S::kStages, kSegSlots = L::S::kSegSlots;
    const uint32_t ring = smem_u32(smem);
    const uint64_t kd0 = sdesc_sw128(ring, 16, kKeyStep);
    const uint64_t qd0 = sdesc_sw128(ring + L::kQ, 16, 1024);
    constexpr uint32_t idesc = idesc_f8_f32(128, L::kScoreN, 0, 0, 0);
    uint32_t counts = 0;               // scores of each team's stages, mod 256
    for (int k = 0, u = 0;; ++k) {
        const int slot = k % kSegSlots, b = k % L::kQuerySlots;
        if (!mbar_wait(&bars->seg_full[slot], (k / kSegSlots) & 1)) {
            expired(p.status, kRoleProducts, 0, k);
            break;
        }
        const int stages = bars->seg[slot].stages;
        mbar_arrive(&bars->seg_free[slot]);
        if (stages < 0) break;
        bool ok = mbar_wait(&bars->q_full[b], (k / L::kQuerySlots) & 1);
        for (int j = 0; ok && j < stages; ++j, ++u) {
            const int team = (SHARE ? j : k) % L::kTeams, st = u % kStages;
            const uint32_t n = counts >> (8 * team) & 255, tile = n % kScoreTiles;
            counts = (counts & ~(255u << (8 * team))) | (n + 1 & 255) << (8 * team);
            // (a tile's first use waits for the phase before its first, which reads as done)
            ok = mbar_wait(&bars->s_free[team][tile], (n / kScoreTiles + 1) & 1) &&
                 mbar_wait(&bars->full[0][st], (u / kStages) & 1);
            if (!ok) break;
            tc_fence_after();
            const uint64_t kd = kd0 + st * (kStageBytes >> 4), qd = qd0 + b * (L::kQuery >> 4);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
                umma_f8_ss(tmem + (team * kScoreTiles + tile) * L::kScoreN, kd + 2 * kk, qd + 2 * kk,
                           idesc, kk > 0);
            // (this thread's own arrival hands on what it has seen: the stage's scale bytes and the
            // queries' factors)
            mbar_arrive(&bars->s_full[team][tile]);
            umma_commit(&bars->s_full[team][tile]);
        }
        if (!ok) {
            expired(p.status, kRoleProducts, 1, u);
            break;
        }
        umma_commit(&bars->q_free[b]);
    }
    umma_commit(&bars->drained[0]);    // nothing in flight when the tensor memory is freed
    if (!mbar_wait(&bars->drained[0], 0)) expired(p.status, kRoleProducts, 2, 0);
}

// Values: as soon as a stage's weights are there.
template <int TEAM, bool SHARE>
__device__ __forceinline__ void issue_values(const Params &p, Q8Bars *bars, uint8_t *smem,
                                             uint32_t tmem) {
    using L = Layout<TEAM, SHARE>;
    constexpr int kStages = L::S::kStages, kSegSlots = L::S::kSegSlots;
    const uint32_t ring = smem_u32(smem);
    const uint64_t vd0 = sdesc_sw128(ring + kTileBytes, 16, kKeyStep);
    const uint64_t pd0 = sdesc_mn(ring + L::kP, 128, kChunk);
    constexpr uint32_t idesc = idesc_f8_f32(128, L::kValueN, 1, 1, 1);
    uint32_t parity = 0, next = 0;     // of each team's tiles of weights, a bit each; its next tile
    // (no weights before a tile's first)
    for (int i = 0; i < L::kTeams * kWeightTiles; ++i)
        mbar_arrive(&bars->s_full[i / kWeightTiles][i % kWeightTiles]);
    for (int k = 0, u = 0;; ++k) {
        const int slot = k % kSegSlots;
        if (!mbar_wait(&bars->seg_full[slot], (k / kSegSlots) & 1)) {
            expired(p.status, kRoleProducts, 3, k);
            break;
        }
        const int stages = bars->seg[slot].stages;
        mbar_arrive(&bars->seg_free[slot]);
        if (stages < 0) break;
        bool ok = true;
        for (int j = 0; j < stages; ++j, ++u) {
            const int team = (SHARE ? j : k) % L::kTeams;
            const int tile = next >> team & 1, at = team * kWeightTiles + tile;
            const uint64_t pd = pd0 + at * (L::kWeights >> 4);
            ok = mbar_wait(&bars->p_full[team][tile], parity >> at & 1);
            if (!ok) break;
            parity ^= 1u << at;
            next ^= 1u << team;
            tc_fence_after();
            const int st = u % kStages;
            const uint64_t vd = vd0 + st * (kStageBytes >> 4);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
                umma_f8_ss(tmem + L::kOutputs + team * L::kValueN, vd + kk * (kKeyStep >> 2), pd + 32 * kk,
                           idesc, kk > 0 || j >= (SHARE ? L::kTeams : 1));
            umma_commit(&bars->pv_done[team][tile]);
            umma_commit(&bars->s_full[team][tile]);   // of the stage whose weights go there next
            umma_commit(&bars->empty[st]);
        }
        if (!ok) {
            expired(p.status, kRoleProducts, 4, u);
            break;
        }
    }
    umma_commit(&bars->drained[1]);
    if (!mbar_wait(&bars->drained[1], 0)) expired(p.status, kRoleProducts, 5, 0);
}

// ---- a softmax group's warp ---------------------------------------------------------------------
template <int TEAM, bool SHARE>
__device__ __forceinline__ void softmax(const Params &p, Q8Bars *bars, uint8_t *smem, uint32_t tmem) {
    using L = Layout<TEAM, SHARE>;
    constexpr int kStages = L::S::kStages, kUnit = L::S::kUnit, kSegSlots = L::S::kSegSlots;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int group = warp / kConsumers, cw = warp % kConsumers, team = group / TEAM, member = group % TEAM;
    const int t = 32 * cw + lane;      // the thread's key of a stage, and its dim of the outputs
    tmem += static_cast<uint32_t>(32 * cw) << 16;
    const uint32_t outputs = tmem + L::kOutputs + team * L::kValueN + member * kValueCols;
    // the rows' -m, and then their products' factors
    float *rowf = reinterpret_cast<float *>(smem + L::kRowFactors) + warp * 2 * kRows;
    float2 *change = reinterpret_cast<float2 *>(smem + L::kChanges) + warp * kRows;
    float2 *most = reinterpret_cast<float2 *>(smem + L::kMost) + group * kConsumers * kRows;
    float *sums = reinterpret_cast<float *>(smem + L::kSums) + group * kRows * kConsumers;
    // A key's weights of 8 rows, each of their three bytes together (MN-major tiles of 16 columns, so
    // that a thread has 3 stores for 24 bytes).
    uint8_t *weights = smem + L::kP + team * kWeightTiles * L::kWeights + t * 16 +
                       member * kValueCols / 16 * kChunk + member * kValueCols % 16;
    const int second = member * kValueCols % 16 == 0 ? 8 : kChunk - 8;
    // (of its team's and group's barriers alone a warp sees every phase: a parity two phases back
    // reads as done, so tiles that the teams shared would be read too early)
    int scored = 0;                    // score tiles read
    int handed = 0;                    // weights handed over
    // The group's warps meet: whether one of them says so.  A warp whose wait has expired goes on to
    // the next meeting and says it there, so that all four leave together.
    bool ok = true;
    auto any = [&](bool mine) { return group_any(group + 1, 32 * kConsumers, mine); };
    auto products_done = [&]() {       // of all weights handed over
        return handed == 0 || quick_wait(&bars->pv_done[team][handed - 1 & 1], (handed - 1 >> 1) & 1);
    };
    auto fail = [&](int barrier, int n) { expired(p.status, kRoleConsumer, barrier, n); };
#pragma unroll 1
    for (int k = SHARE ? 0 : team, turn = 0;; k += SHARE ? 1 : L::kTeams, turn ^= 1) {
        const int slot = k % kSegSlots;
        if (!quick_wait(&bars->seg_full[slot], (k / kSegSlots) & 1)) ok = false;
        if (any(!ok)) return fail(0, k);
        // NaN among the values' numbers: a bit per row and dim of this pair (turn), and of the last
        auto nan_row = [&](int which, int r) {    // r: of the team's rows
            return reinterpret_cast<uint32_t *>(smem + L::kNan) +
                   ((2 * team + which) * L::kTeamRows + r) * 4;
        };
        if (!SHARE && cw == 0 && bars->nan_any[group][turn ^ 1]) {
            // The last pair's bits: all warps of the group have read them, and the team's first group,
            // which sets them, is not past this pair before this group has handed over its stages.
            // Here, where groups that have no rows of this pair come by, too.
            if (lane < kRows)
                *reinterpret_cast<uint4 *>(nan_row(turn ^ 1, kRows * member + lane)) =
                    make_uint4(0, 0, 0, 0);
            __syncwarp();
            if (lane == 0) bars->nan_any[group][turn ^ 1] = 0;
        }
        const Segment sg = bars->seg[slot];
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->seg_free[slot]);
        if (sg.stages < 0) return;
        const int first_row = sg.r0 + kRows * member;
        const Place *places = reinterpret_cast<const Place *>(smem + L::kPlaces) +
                              k % L::kFactorSlots * L::kTeamRows;
        const int rows = max(0, min(kRows, sg.T * p.G - first_row));   // none: no weights, O unread
        const int q_first = sg.S - sg.T;          // keys beyond are hidden from some
        const int lo = p.window > 0 ? max(0, q_first - p.window + 1) : 0;
        const int lo_all = p.window > 0 ? max(0, sg.S - p.window) : 0;
        float m = -CUDART_INF_F, mo = -CUDART_INF_F;   // of row `lane`
        bool fresh = true;             // no stage of this pair yet
        float l[kRows];
#pragma unroll
        for (int r = 0; r < kRows; ++r) l[r] = 0.f;
#pragma unroll 1
        for (int j = 0, u = sg.u0; j < sg.stages; ++j, ++u) {
            // (the first to team 0, whatever the CTA had before: the shares are added up in order)
            if (SHARE && j % L::kTeams != team) continue;
            const int st = u % kStages, si = scored % kScoreTiles;
            if (!quick_wait(&bars->s_full[team][si], (scored / kScoreTiles) & 1)) ok = false;
            ++scored;
            const int kb = (sg.unit0 + j) * kUnit, key = kb + t;
            const bool edge = kb + kUnit - 1 > q_first || kb < lo_all;   // of the mask
            if (rows > 0) {
                tc_fence_after();
                float y[kRows];
                uint32_t s[kScoreCols];
                tmem_ld16(tmem + (team * kScoreTiles + si) * L::kScoreN + member * kScoreCols, s);
                const uint32_t bytes =
                    reinterpret_cast<const uint16_t *>(smem + L::kScales)[st * kUnit + t];
                const float kf = scale_of(bytes & 255u), vf = scale_of(bytes >> 8);
                // The scores' factors, the row's times the key's: a score multiplied by one after the
                // other may leave fp32's range on the way, or, by a 0, take a hidden one to NaN.
                // (Formed while the scores are on their way: 32 rows 565 us, after them 575.)
                const float4 *factors = reinterpret_cast<const float4 *>(
                    smem + L::kFactors + (k % L::kFactorSlots * L::kTeamRows + member * kRows) * 4);
                float2 sf[kRows / 2];
#pragma unroll
                for (int i = 0; i < kRows / 2; i += 2) {
                    const float4 f = factors[i / 2];
                    sf[i] = __fmul2_rn(make_float2(f.x, f.y), make_float2(kf, kf));
                    sf[i + 1] = __fmul2_rn(make_float2(f.z, f.w), make_float2(kf, kf));
                }
                uint32_t hidden = 0;       // a bit per row
                if (edge) {
                    // a token's rows at a time
                    int tok = token_of(p, first_row), r = 0;
#pragma unroll 1
                    do {
                        const int at = q_first + min(tok, sg.T - 1), to = ++tok * p.G - first_row;
                        if (key > at || (p.window > 0 && at - key >= p.window))
                            hidden |= (1u << min(to, kRows)) - (1u << r);
                        r = to;
                    } while (r < kRows);
                }
                tmem_wait_ld();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars->s_free[team][si]);
#pragma unroll
                for (int r = 0; r < kRows; r += 2) {
                    const float2 h = make_float2(__uint_as_float(s[r]), __uint_as_float(s[r + 1])),
                                 lo16 = make_float2(__uint_as_float(s[kRows + r]),
                                                    __uint_as_float(s[kRows + r + 1])),
                                 x = __fmul2_rn(__ffma2_rn(lo16, make_float2(0.0625f, 0.0625f), h),
                                                sf[r / 2]);
                    y[r] = x.x;
                    y[r + 1] = x.y;
                }
                if (edge) {
#pragma unroll
                    for (int r = 0; r < kRows; ++r)
                        if (hidden >> r & 1) y[r] = -CUDART_INF_F;
                }
                // ---- weights w and products P, against new references where the old are passed
                float w[kRows], pw[kRows];
                bool update = fresh;
#pragma unroll 1
                while (true) {
                    if (update) {
                        const float ev = fmaxf(exponent_of(bytes >> 8), kLeast);
                        float a[kRows], b[kRows];
#pragma unroll
                        for (int r = 0; r < kRows; ++r) a[r] = y[r];
                        // (the score and exponent less the warp's largest score: next to a score of
                        // 2^24 an exponent is lost in fp32)
                        auto larger = [](float c, float d) { return fmaxf(c, d); };
                        const int row = gather_rows(a, larger);
#pragma unroll
                        for (int r = 0; r < kRows; ++r)
                            b[r] = y[r] - finite(__shfl_sync(0xffffffffu, a[0], 4 * r)) + ev;
                        gather_rows(b, larger);
                        if ((lane & 3) == 0) most[cw * kRows + row] = make_float2(a[0], b[0]);
                        if (any(!ok)) return fail(1, u);
                        if (lane < kRows) {
                            float mn = m;
#pragma unroll
                            for (int c = 0; c < kConsumers; ++c)
                                mn = fmaxf(mn, most[c * kRows + lane].x);
                            const float base = finite(mn), was = mo + (finite(m) - base);
                            float mno = was;
#pragma unroll
                            for (int c = 0; c < kConsumers; ++c) {
                                const float2 x = most[c * kRows + lane];
                                mno = fmaxf(mno, x.y + (finite(x.x) - base));
                            }
                            change[lane] =
                                make_float2(m == -CUDART_INF_F ? 0.f : ex2_approx(m - mn),
                                            mo == -CUDART_INF_F ? 1.f : ex2_approx(was - mno));
                            m = mn;
                            mo = mno;
                            rowf[lane] = -base;
                            rowf[kRows + lane] = mn == -CUDART_INF_F ? 0.f : ex2_approx(kShift - mno);
                        }
                        __syncwarp();
                        if (!fresh) {
                            if (!products_done()) ok = false;
                            tc_fence_after();
#pragma unroll 1
                            for (int c = 0; c < 3; ++c) {
                                uint32_t o[kRows];
                                tmem_ld8(outputs + c * kRows, o);
                                tmem_wait_ld();
#pragma unroll
                                for (int r = 0; r < kRows; ++r)
                                    o[r] = __float_as_uint(__uint_as_float(o[r]) * change[r].y);
                                tmem_st8(outputs + c * kRows, o);
                            }
                            tmem_wait_st();
                            tc_fence_before();
#pragma unroll
                            for (int r = 0; r < kRows; ++r) l[r] *= change[r].x;
                        }
                    }
                    float top = -CUDART_INF_F, largest = 0.f;
#pragma unroll
                    for (int r = 0; r < kRows; r += 4) {
                        const float4 ref = reinterpret_cast<const float4 *>(rowf)[r / 4],
                                     z = reinterpret_cast<const float4 *>(rowf + kRows)[r / 4];
#pragma unroll
                        for (int i = r; i < r + 4; i += 2) {
                            const float2 x = __fadd2_rn(make_float2(y[i], y[i + 1]),
                                                        i == r ? make_float2(ref.x, ref.y)
                                                               : make_float2(ref.z, ref.w));
                            w[i] = ex2_approx(x.x);
                            w[i + 1] = ex2_approx(x.y);
                            const float2 b = __fmul2_rn(
                                __fmul2_rn(make_float2(w[i], w[i + 1]),
                                           i == r ? make_float2(z.x, z.y) : make_float2(z.z, z.w)),
                                make_float2(vf, vf));
                            pw[i] = b.x;
                            pw[i + 1] = b.y;
                            top = fmax3(top, x.x, x.y);
                            largest = fmax3(largest, b.x, b.y);
                        }
                    }
                    if (update || !any(top > kGrow || largest > kLargest || !ok)) break;
                    update = true;
                }
                // ---- P, a byte per column, row and key
                if (edge) {
                    // (a hidden key's value may have a NaN for a power)
#pragma unroll
                    for (int r = 0; r < kRows; ++r)
                        if (hidden >> r & 1) pw[r] = 0.f;
                }
                uint2 c, d, f;
#pragma unroll
                for (int r = 0; r < kRows; r += 4) {
                    uint32_t x[2], x1[2], x2[2];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int k = r + 2 * i;
                        const float2 lk = __fadd2_rn(make_float2(l[k], l[k + 1]),
                                                     make_float2(w[k], w[k + 1]));
                        l[k] = lk.x;
                        l[k + 1] = lk.y;
                        const __half2 y = __floats2half2_rn(pw[k], pw[k + 1]);
                        x[i] = *reinterpret_cast<const uint32_t *>(&y);
                        x1[i] = less_upper(x[i]);
                        const uint32_t rest = less_upper(x1[i]);
                        x2[i] = to_e5m2x2(*reinterpret_cast<const __half2 *>(&rest));
                    }
                    // the upper bytes of four, of what is left of them, and the rest
                    (r ? c.y : c.x) = __byte_perm(x[0], x[1], 0x7531);
                    (r ? d.y : d.x) = __byte_perm(x1[0], x1[1], 0x7531);
                    (r ? f.y : f.x) = __byte_perm(x2[0], x2[1], 0x5410);
                }
                uint8_t *to = weights + (handed & 1) * L::kWeights;
                *reinterpret_cast<uint2 *>(to) = c;
                *reinterpret_cast<uint2 *>(to + second) = d;
                *reinterpret_cast<uint2 *>(to + kChunk) = f;
            } else {
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars->s_free[team][si]);
            }
            // ---- values that the mask hides: 0 * NaN is NaN
            if (edge && member == 0) {
                uint8_t *vr = smem + st * kStageBytes + kTileBytes + t * kD;
                if (key >= sg.S || key < lo) {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        reinterpret_cast<uint4 *>(vr)[i] = make_uint4(0, 0, 0, 0);
                } else if (key > q_first || key < lo_all) {
                    // some rows see it: its NaN are taken out, and noted for the rows that do (all
                    // numbers are looked over first, together: one after the other they took 4000
                    // cycles)
                    uint32_t nan = 0;
#pragma unroll 2
                    for (int i = 0; i < 8; ++i) {
                        const uint4 x = reinterpret_cast<const uint4 *>(vr)[i];
                        nan |= nan_bytes(x.x) | nan_bytes(x.y) | nan_bytes(x.z) | nan_bytes(x.w);
                    }
#pragma unroll 1
                    for (int i = 0; nan && i < kD / 4; ++i) {
                        uint32_t *at = reinterpret_cast<uint32_t *>(vr) + i;
                        const uint32_t x = *at, bad = nan_bytes(x);
                        if (!bad) continue;
                        *at = x & ~bad;
                        const int dim = 16 * (i >> 2 ^ (t & 7)) + 4 * (i & 3);
#pragma unroll 1
                        for (int e = 0; e < 4; ++e) {
                            if (!(bad >> (8 * e) & 1)) continue;
#pragma unroll 1
                            for (int r = 0; r < min(sg.T * p.G - sg.r0, L::kTeamRows); ++r) {
                                const int pos = q_first + token_of(p, sg.r0 + r);
                                if (key > pos || (p.window > 0 && pos - key >= p.window)) continue;
                                atomicOr(nan_row(turn, r) + (dim + e) / 32, 1u << ((dim + e) & 31));
                                bars->nan_any[team * TEAM + r / kRows][turn] = 1;
                            }
                        }
                    }
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars->p_full[team][handed & 1]);
            ++handed;
            fresh = false;
        }
        if constexpr (SHARE) {
            float *shares = reinterpret_cast<float *>(smem + L::kShares);
            bool nans = false;
            if (rows > 0) {
                // this team's share, O relative to m (times 2^(mo - 12), in two steps as that may be
                // 2^-138)
                const int row = gather_rows(l, [](float a, float b) { return a + b; });
                if ((lane & 3) == 0) sums[row * kConsumers + cw] = l[0];
                if (any(!ok)) return fail(2, k);
                if (!products_done()) ok = false;
                if (k > 0 && !quick_wait(&bars->taken, k - 1 & 1)) ok = false;
                if (lane < kRows) {
                    const float4 s = *reinterpret_cast<const float4 *>(sums + lane * kConsumers);
                    change[lane].x = mo == -CUDART_INF_F ? 1.f : ex2_approx(0.5f * (mo - kShift));
                    if (cw == 0) bars->share[group][lane] = make_float2(m, (s.x + s.y) + (s.z + s.w));
                }
                __syncwarp();
                tc_fence_after();
                uint32_t a[kRows], b[kRows], c[kRows];
                tmem_ld8(outputs, a);
                tmem_ld8(outputs + kRows, b);
                tmem_ld8(outputs + 2 * kRows, c);
                tmem_wait_ld();
                tc_fence_before();
                nans = *const_cast<volatile int *>(&bars->nan_any[group][turn]) != 0;
#pragma unroll
                for (int r = 0; r < kRows; ++r) {
                    const float f = change[r].x;
                    float x = (__uint_as_float(a[r]) + (__uint_as_float(b[r]) + __uint_as_float(c[r]))) *
                              f * f;
                    if (nans && nan_row(turn, kRows * member + r)[t / 32] >> (t & 31) & 1)
                        x = CUDART_NAN_F;
                    shares[(group * kRows + r) * kD + t] = fresh ? 0.f : x;
                }
            } else if (k > 0 && !quick_wait(&bars->taken, k - 1 & 1)) {   // (sees every phase)
                ok = false;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars->gathered);
            if (!quick_wait(&bars->gathered, k & 1)) ok = false;
            if (nans && cw == 0) {     // the bits have been read
                if (lane < kRows)
                    *reinterpret_cast<uint4 *>(nan_row(turn, kRows * member + lane)) =
                        make_uint4(0, 0, 0, 0);
                if (lane == 0) bars->nan_any[group][turn] = 0;
            }
            // a warp adds up a row, 4 dims per lane
            if (warp < L::kTeamRows && sg.r0 + warp < sg.T * p.G) {
                float2 x[L::kTeams];
                float M = -CUDART_INF_F, sum = 0.f;
#pragma unroll
                for (int i = 0; i < L::kTeams; ++i) {
                    x[i] = bars->share[i * TEAM + warp / kRows][warp % kRows];
                    M = fmaxf(M, x[i].x);
                }
                float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int i = 0; i < L::kTeams; ++i) {
                    // a share none of whose keys this row sees: m = -inf, l = 0 and O = 0 (NaN
                    // scores alone also leave m at -inf, with l and O NaN)
                    const float f = x[i].x == -CUDART_INF_F ? (x[i].y == 0.f ? 0.f : 1.f)
                                                            : ex2_approx(x[i].x - M);
                    const float4 y = reinterpret_cast<const float4 *>(
                        shares + ((i * TEAM + warp / kRows) * kRows + warp % kRows) * kD)[lane];
                    sum = fmaf(x[i].y, f, sum);
                    acc.x = fmaf(y.x, f, acc.x);
                    acc.y = fmaf(y.y, f, acc.y);
                    acc.z = fmaf(y.z, f, acc.z);
                    acc.w = fmaf(y.w, f, acc.w);
                }
                const Place to = places[warp];
                if (to.o && sg.slot >= 0) {
                    reinterpret_cast<float4 *>(to.o)[lane] = acc;
                    if (lane == 0) *reinterpret_cast<float2 *>(to.sum) = make_float2(M, sum);
                } else if (to.o) {
                    const float inv = 1.0f / sum;
                    reinterpret_cast<uint2 *>(to.o)[lane] = make_uint2(
                        pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
                    if (to.sum && lane == 0)
                        *reinterpret_cast<float *>(to.sum) = (M + __log2f(sum)) * 0.69314718055994531f;
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars->taken);
            continue;
        }
        if (rows == 0) continue;
        // ---- the pair's (or span's) result: this thread's dim of all rows
        const int row = gather_rows(l, [](float a, float b) { return a + b; });
        if ((lane & 3) == 0) sums[row * kConsumers + cw] = l[0];
        if (any(!ok)) return fail(2, k);
        if (lane < kRows) {
            // A row's factors.  O relative to m: times 2^(mo - 12), in two steps as that may be 2^-138.
            const float4 s = *reinterpret_cast<const float4 *>(sums + lane * kConsumers);
            const float sum = (s.x + s.y) + (s.z + s.w);
            change[lane] = make_float2(mo == -CUDART_INF_F ? 1.f : ex2_approx(0.5f * (mo - kShift)),
                                       sg.slot >= 0 ? 1.f : 1.0f / sum);
            void *to = places[kRows * member + lane].sum;
            if (cw == 0 && to) {
                if (sg.slot >= 0) *reinterpret_cast<float2 *>(to) = make_float2(m, sum);
                else *reinterpret_cast<float *>(to) = (m + __log2f(sum)) * 0.69314718055994531f;
            }
        }
        if (!products_done()) ok = false;
        __syncwarp();
        tc_fence_after();
        uint32_t a[kRows], b[kRows], c[kRows];
        tmem_ld8(outputs, a);
        tmem_ld8(outputs + kRows, b);
        tmem_ld8(outputs + 2 * kRows, c);
        tmem_wait_ld();
        tc_fence_before();
        const bool nans = *const_cast<volatile int *>(&bars->nan_any[group][turn]) != 0;
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            const float2 f = change[r];
            void *to = places[kRows * member + r].o;
            if (!to) continue;
            float x = (__uint_as_float(a[r]) + (__uint_as_float(b[r]) + __uint_as_float(c[r]))) * f.x *
                      f.x * f.y;
            if (nans && nan_row(turn, kRows * member + r)[t / 32] >> (t & 31) & 1) x = CUDART_NAN_F;
            if (sg.slot >= 0) reinterpret_cast<float *>(to)[t] = x;
            else reinterpret_cast<__nv_bfloat16 *>(to)[t] = __float2bfloat16_rn(x);
        }
        __syncwarp();                  // before the next pair's factors
    }
}

template <int TEAM, bool SHARE>
__global__ void __launch_bounds__((Q8Stream<TEAM, SHARE>::kThreads), 1)
    paged_q8_kernel(const __grid_constant__ CUtensorMap tmK,
                    const __grid_constant__ CUtensorMap tmV, const Params p) {
    griddep_wait();
    griddep_launch_dependents();
    using L = Layout<TEAM, SHARE>;
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
        for (int i = 0; i < S::kSegSlots; ++i) {
            mbar_init(&bars->seg_full[i], 1);
            mbar_init(&bars->seg_free[i], (SHARE ? L::kGroups : TEAM) * kConsumers + 3);
        }
        for (int g = 0; g < 4; ++g) {
            mbar_init(&bars->q_full[g], 1);
            mbar_init(&bars->q_free[g], 1);
            for (int i = 0; i < kScoreTiles; ++i) {
                mbar_init(&bars->s_full[g][i], 3);
                mbar_init(&bars->s_free[g][i], TEAM * kConsumers);
            }
            for (int i = 0; i < kWeightTiles; ++i) {
                mbar_init(&bars->p_full[g][i], TEAM * kConsumers);
                mbar_init(&bars->pv_done[g][i], 1);
            }
            for (int i = 0; i < 2; ++i) bars->nan_any[g][i] = 0;
        }
        for (int i = 0; i < 2; ++i) mbar_init(&bars->drained[i], 1);
        mbar_init(&bars->gathered, L::kGroups * kConsumers);
        mbar_init(&bars->taken, L::kGroups * kConsumers);
        mbar_init(&bars->q_raw, 1);
        mbar_init(&bars->clc_full, 1);
        fence_mbar_init();
    }
    // columns of P that no weight is written to, and the NaN bits
    for (int i = threadIdx.x; i < L::kTeams * kWeightTiles * L::kWeights / 16; i += S::kThreads)
        reinterpret_cast<uint4 *>(smem + L::kP)[i] = make_uint4(0, 0, 0, 0);
    for (int i = threadIdx.x; i < L::kTeams * 2 * L::kTeamRows; i += S::kThreads)
        reinterpret_cast<uint4 *>(smem + L::kNan)[i] = make_uint4(0, 0, 0, 0);
    fence_proxy_async_smem();
    if (warp == L::kScoreWarp) {
        tmem_alloc(&bars->tmem, L::kColumns);
        tmem_relinquish();
    }
    scan_units<S>(p, bars);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bars->tmem;
    if (warp < S::kProducer) softmax<TEAM, SHARE>(p, bars, smem, tmem);
    else if (warp == S::kProducer) produce<S>(tmK, tmV, p, bars, smem, smem + L::kScales);
    else if (warp == L::kQueryWarp) bring_queries<TEAM, SHARE>(p, bars, smem);
    else if (warp == L::kScoreWarp && lane == 0) issue_scores<TEAM, SHARE>(p, bars, smem, tmem);
    else if (warp == L::kValueWarp && lane == 0) issue_values<TEAM, SHARE>(p, bars, smem, tmem);
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == L::kScoreWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, L::kColumns);
    }
}

// How a call is taken: groups of a team (1: by the kernel for up to 8 rows; 0: by the tile kernel)
// and blocks of rows per sequence.
struct Plan {
    int team, blocks;
};
constexpr int kMostBlocks = 3;
Plan plan_of(int max_q, int Hq, int Hkv) {
    const long n = static_cast<long>(max_q) * (Hq / Hkv);
    if (n <= kRows) return {1, 1};
    if (n <= 2 * kRows) return {2, 1};
    const long blocks = (n + kBlockRows - 1) / kBlockRows;
    return blocks <= kMostBlocks ? Plan{4, static_cast<int>(blocks)} : Plan{0, 0};
}

// The call's tensor maps, {128 numbers, keys of a page, (page, KV head)}, a box of `most` keys of a page
// at most.  (One map over both pools, their distance as a dimension's stride, brought a page's keys and
// values by one copy, in pages of 16 tokens 426 instead of 522 us over 32 caches of 8k-64k.  Two runs of
// random cases with it ended in a fault, the pools small and far apart.  What in the copy did it is not
// known; what no other map here does is to span memory that is not its tensor's.)
bool make_maps(const gqa_paged_kv_q8 &c, int most, CUtensorMap *mk, CUtensorMap *mv) {
    const uint64_t page = c.page_size;
    const uint64_t dims[3] = {kD, page, (uint64_t)c.num_pages * c.Hkv}, strides[2] = {kD, page * kD};
    const uint32_t box[3] = {kD, static_cast<uint32_t>(c.page_size < most ? c.page_size : most), 1};
    return make_byte_map(mk, c.k, 3, dims, strides, box) && make_byte_map(mv, c.v, 3, dims, strides, box);
}

template <int TEAM, bool SHARE>
int launch(const CUtensorMap &mk, const CUtensorMap &mv, const Params &p, long grid, cudaStream_t s) {
    using L = Layout<TEAM, SHARE>;
    auto kern = paged_q8_kernel<TEAM, SHARE>;
    if (ensure_smem_attr(reinterpret_cast<const void *>(kern), L::kBytes) != cudaSuccess ||
        launch_pdl(kern, dim3(static_cast<unsigned>(grid)), dim3(L::S::kThreads), L::kBytes, s, mk, mv,
                   p) != cudaSuccess)
        return GQA_ERR_CUDA;
    return GQA_OK;
}

int launch_stream(const PackedAttn &a, const gqa_paged_kv_q8 &c, const Plan &plan, void *ws,
                  int *status, cudaStream_t s) {
    Params p = params_of(a, kStreamUnit, plan.team * kRows, plan.blocks, ws, status);
    p.scales = static_cast<const uint8_t *>(c.scales);
    CUtensorMap mk, mv;
    const long pairs = (long)a.nseq * a.Hkv * plan.blocks;
    // A warp per pair where there are many, or some of two steps at most (8 heads of 20-450 tokens:
    // 304 pairs 24 us and 14 with a CTA per pair, 608 26 and 22, 1024 27 and 29, 2048 39 and 57; 608
    // of 20-40 tokens 8 and 13).
    const bool each = plan.team == 1 && p.whole &&
                      pairs >= (a.max_kv <= 2 * kShortKeys ? 1 : 6) * static_cast<long>(kSMs);
    if (!make_maps(c, each ? kShortKeys : kStreamUnit, &mk, &mv)) return GQA_ERR_CUDA;
    if (each) return launch_q8_short(mk, mv, p, s);
    const long grid = !p.whole ? p.chunks : pairs < kSMs ? pairs : kSMs;
    const int rc = plan.team == 1   ? launch_q8_few(mk, mv, p, grid, s)
                   : plan.team == 4 ? launch<4, false>(mk, mv, p, grid, s)
                   : p.whole        ? launch<2, false>(mk, mv, p, grid, s)
                                    : launch<2, true>(mk, mv, p, grid, s);
    if (rc == GQA_OK && !p.whole && launch_combine(p, a.max_q, s) != cudaSuccess) return GQA_ERR_CUDA;
    return rc;
}

}  // namespace

bool paged_q8_counts_fit(int nseq, int total, int max_q, int max_kv, int Hq, int Hkv) {
    const Plan plan = plan_of(max_q, Hq, Hkv);
    if (plan.team)
        // (in the cut a pair's end counts as 6 units at most)
        return (long)Hkv * plan.blocks <= 0x7fffffffL &&
               paged_decode_counts_fit(nseq, max_kv, Hkv * plan.blocks) &&
               (long)nseq * Hkv * plan.blocks * ((max_kv - 1) / kStreamUnit + 1 + 6) <=
                   0x7fffffffL - 2 * kSMs;
    return paged_expand_counts_fit(nseq, max_kv, Hkv) &&
           packed_prefill_counts_fit(nseq, total, max_kv, Hq, Hkv);
}

size_t paged_q8_workspace_bytes(int nseq, int total, int max_q, int max_kv, int Hq, int Hkv) {
    const Plan plan = plan_of(max_q, Hq, Hkv);
    if (plan.team)
        return whole_pairs(max_kv)
                   ? 0
                   : partials_bytes(n_chunks(nseq, max_kv, Hkv * plan.blocks, 1, 0, kStreamUnit),
                                    plan.team * kRows);
    return paged_expand_q8_bytes(nseq, max_kv, Hkv) +
           packed_prefill_workspace_bytes(nseq, total, max_kv, Hq, Hkv);
}

int launch_paged_q8(const PackedAttn &a, const gqa_paged_kv_q8 &c, void *ws, int *status,
                    cudaStream_t s) {
    gqa_paged_kv pages = {c.k, c.v, c.page_table, c.kv_lens, c.num_pages, c.Hkv, c.page_size, c.d,
                          c.max_pages, 0};
    PackedAttn b = a;
    b.cache = &pages;
    const Plan plan = plan_of(a.max_q, a.Hq, a.Hkv);
    if (plan.team) return launch_stream(b, c, plan, ws, status, s);
    if (launch_paged_expand_q8(c, a, ws, &pages, status, s) != cudaSuccess) return GQA_ERR_CUDA;
    b.k = pages.k;
    b.v = pages.v;
    b.cap = (long)c.max_pages * c.page_size;
    return launch_packed_prefill(
        b, static_cast<char *>(ws) + paged_expand_q8_bytes(a.nseq, a.max_kv, a.Hkv), status, s);
}

}  // namespace gqa
