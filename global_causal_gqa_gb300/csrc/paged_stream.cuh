// paged_stream.cuh -- what the streaming kernels over a paged cache share (paged_decode.cu: bf16
// pages, paged_q8.cu: 8-bit ones): how a batch is cut into chunks of units and pairs, and the
// producer warp that finds the pairs and streams their keys and values into a ring of stages.
// The head of paged_decode.cu describes the cut and what it measured.
#pragma once
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math_constants.h>

#include "internal.h"
#include "packed.cuh"

namespace gqa {
namespace stream {

constexpr int kD = 128;
constexpr int kTileBytes = 16384;               // K or V of a stage
constexpr int kStageBytes = 2 * kTileBytes;
constexpr int kMostStages = 6;
constexpr int kConsumers = 4;                   // warps of a group of consumers
constexpr int kSMs = 152;
constexpr int kMinRun = 128;                    // units per SM from which chunks come in levels
constexpr int kKeyStep = 1024;                  // 8-bit stages: bytes of 8 keys (or values)
constexpr int kScaleCopies = 16;                // lanes that copy an 8-bit stage's scale bytes

// What the kernels differ in.  kUnit: keys of a stage.  kStages: of the ring.  kTeams: groups of
// consumers, or teams of groups, that take the pairs in turn.  kEnds: records of the end.  kProducer:
// the producer's warp.  full_of: which of its barriers a stage's load completes.  kEndCost: units
// that a pair's end counts as when the batch is cut (24 caches of 700-6000 tokens, 8 KV heads, before
// other steps: 16 to 48 rows 99.5 us at 0, 88 to 92 at 3 to 8; 16 rows 67 at 0, 53 at 6; 8 rows over
// windows of 2048 65 at 0, 61 at 4).
struct Bf16Stream {
    static constexpr bool kQ8 = false;
    static constexpr int kUnit = 64, kStages = 6, kSegSlots = 4, kTeams = 2, kEnds = kTeams;
    static constexpr int kEndCost = 0;
    static constexpr int kProducer = kTeams * kConsumers, kThreads = 32 * (kProducer + 1);
    __device__ static int full_of(int turn, int) { return turn % kTeams; }
};
template <int TEAM, bool SHARE>   // groups of a team; the teams take a pair's stages in turn
struct Q8Stream {
    static constexpr bool kQ8 = true;
    static constexpr int kGroups = 4, kTeams = kGroups / TEAM, kEnds = SHARE ? 1 : kTeams;
    static constexpr int kUnit = 128, kStages = 5, kSegSlots = 8;
    static constexpr int kEndCost = TEAM == 4 ? 4 : 6;
    static constexpr int kProducer = kGroups * kConsumers, kThreads = 32 * (kProducer + 4);
    __device__ static int full_of(int, int) { return 0; }
};
constexpr int kBlockRows = 32;                  // of a pair where sequences have more

// A run of stages of one (sequence, KV head).  stages < 0: no more.
struct Segment {
    int row0, T, S, seq, g, unit0, stages;
    int u0;     // stages of the CTA's run before it
    int slot;   // -1: all of the pair's keys; else the partial's place
    int r0;     // first of the pair's rows (8-bit pages: rows go in blocks)
};

// A pair whose keys begin in one chunk and go on in the next ones.  rows = 0: none.
struct Joint {
    int row0, g, rows, parts, r0;
};

// What the producer shares with the consumers.
struct StreamBars {
    Segment seg[8];
    uint64_t full[2][kMostStages];     // a stage's load
    uint64_t empty[kMostStages];
    uint64_t seg_full[8], seg_free[8];
    uint64_t clc_full;
    uint4 clc_resp;
    int scan[20], most[20];            // units of each warp's sequences; of a pair
};

struct Params {
    const __nv_bfloat16 *q;
    __nv_bfloat16 *o;
    float *lse;
    float *ws_o, *ws_ml;
    Joint *ws_joint;               // one per chunk
    int chunks, rec_rows;          // rows that a partial has room for
    const int32_t *cu, *kv_lens, *pages;
    const uint8_t *scales;         // of 8-bit pages
    int *status;
    long q_stride, o_stride;
    PackedBounds bounds;
    int nseq, Hq, Hkv, G, window, num_pages, page_size, page_shift, max_pages;
    uint32_t inv_g;                // 2^16 / G, rounded up
    int whole;                     // 1: CTAs take whole pairs, every gridDim.x-th one
    int blocks;                    // of kBlockRows rows, a pair each, that a sequence has at most
    float scale_log2;
};

// On the host (paged_decode.cu): the rule for whole pairs, the number of chunks, what the partials
// take, a call's parameters, and the kernel that merges the partials.
bool whole_pairs(int max_kv);
int n_chunks(int nseq, int max_kv, int Hkv, int max_q, int window, int unit);
size_t partials_bytes(int chunks, int rows);
Params params_of(const PackedAttn &a, int unit, int rec_rows, int blocks, void *ws, int *status);
cudaError_t launch_combine(const Params &p, int max_q, cudaStream_t s);
// The kernel for up to 8 rows over 8-bit pages (paged_q8_few.cu); returns a gqa_status.
int launch_q8_few(const CUtensorMap &mk, const CUtensorMap &mv, const Params &p, long grid,
                  cudaStream_t s);
// The one for many short caches among them (paged_q8_short.cu): boxes of kShortKeys keys at most.
constexpr int kShortKeys = 32;
int launch_q8_short(const CUtensorMap &mk, const CUtensorMap &mv, const Params &p, cudaStream_t s);

// r / G for a row r < 1024 of a pair (the error, r / 2^16 at most, is below 1 / G).
__device__ __forceinline__ int token_of(const Params &p, int r) {
    return static_cast<int>(r * p.inv_g >> 16);
}

// Pairs of a sequence's KV head: one, or one per block of its rows.
template <class S>
__device__ __forceinline__ int blocks_of(const Params &p, int T) {
    return S::kQ8 && p.blocks > 1 ? (T * p.G + kBlockRows - 1) / kBlockRows : 1;
}

// Units of one (sequence, KV head): [first, first + count) of `unit` keys each.
template <int unit>
__device__ __forceinline__ int first_unit(const PackedSeq &s, int window) {
    return window > 0 && s.S - s.T - window + 1 > 0 ? (s.S - s.T - window + 1) / unit : 0;
}
template <int unit>
__device__ __forceinline__ int count_units(const PackedSeq &s, int window) {
    return s.T > 0 ? (s.S + unit - 1) / unit - first_unit<unit>(s, window) : 0;
}

// The cut of all units into chunks, one level of kSMs equal chunks after the other; one level
// alone also where a pair has so much of the whole (`most` units) that hundreds of chunks would
// share it.
constexpr int kLevels = 4;
struct Cut {
    int all, size[kLevels];
    __device__ Cut(int units, int most, int chunks) : all(units) {
        const int run = all / kSMs;
        int rest = 0;
        size[0] = 0;
#pragma unroll
        for (int l = 1; l < kLevels; ++l) {
            size[l] = chunks > kSMs && run >= kMinRun && most <= all / 4 ? run >> (l + 2) : 0;
            rest += size[l];
        }
        size[0] = (all - kSMs * rest + kSMs - 1) / kSMs;
    }
    __device__ void get(int c, int &begin, int &n) const {
        begin = 0;
        n = 0;
#pragma unroll
        for (int l = 0; l < kLevels; ++l) {
            const int i = c - l * kSMs;
            if (i >= kSMs) begin += kSMs * size[l];
            else if (i >= 0) {
                begin += i * size[l];
                n = max(0, min(size[l], all - begin));
            }
        }
    }
    __device__ int chunk_of(int unit) const {
        int c = 0;
#pragma unroll
        for (int l = 0; l < kLevels; ++l) {
            if (unit < 0) continue;
            if (l + 1 == kLevels || unit < kSMs * size[l]) {
                c = l * kSMs + (size[l] > 0 ? unit / size[l] : 0);
                unit = -1;
            } else {
                unit -= kSMs * size[l];
            }
        }
        return c;
    }
};

__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity));
}

// A warp's wait for a phase that is mostly over: one test, and the loop out of line (the loops of
// every such wait are a large part of the code, and the caches of instructions are small).
static __device__ __noinline__ bool wait_on(uint64_t *bar, uint32_t parity) { return warp_wait(bar, parity); }
__device__ __forceinline__ bool quick_wait(uint64_t *bar, uint32_t parity) {
    return __all_sync(0xffffffffu, mbar_try_wait(bar, parity)) || wait_on(bar, parity);
}

__device__ __forceinline__ void prefetch_l2(const void *p) {
    asm volatile("prefetch.global.L2 [%0];" ::"l"(p) : "memory");
}

// Copies 16 bytes to shared memory, or `bytes` of them and zeros, and arrives on the barrier when
// they are there (an arrival of its own, which the barrier's count includes).
__device__ __forceinline__ void copy_async16(void *dst, const void *src, uint32_t bytes,
                                             uint64_t *bar) {
    asm volatile(
        "cp.async.cg.shared.global [%0], [%1], 16, %2;\n\t"
        "cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%3];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(smem_u32(bar))
        : "memory");
}

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
// The transpose of an 8 x 8 matrix of 16-bit values, a row in four lanes.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

enum Role { kRoleProducer = 0, kRoleProducts = 1, kRoleConsumer = 2, kRoleQueries = 3 };
constexpr int kSite = kDiagPagedDecode << 24;   // of the debug build's checks

// Sequences per thread in the sums below.
template <class S>
__device__ __forceinline__ int sequences_each(const Params &p) {
    return (p.nseq + S::kThreads - 1) / S::kThreads;
}

// The batch's units: each warp's sequences, in order (all threads; a __syncthreads() follows).
template <class S>
__device__ __forceinline__ void scan_units(const Params &p, StreamBars *bars) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, m = sequences_each<S>(p);
    if (!p.whole) {
        const int s0 = threadIdx.x * m;
        int mine = 0, most = 0;
        for (int i = s0; i < s0 + m && i < p.nseq; ++i) {
            const PackedSeq s = packed_seq(p.cu, p.kv_lens, i, p.bounds, p.status);
            const int n = count_units<S::kUnit>(s, p.window);
            mine += p.Hkv * blocks_of<S>(p, s.T) * (n > 0 ? n + S::kEndCost : 0);
            most = max(most, n);
        }
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) mine += __shfl_xor_sync(0xffffffffu, mine, d);
        most = __reduce_max_sync(0xffffffffu, most);
        if (lane == 0) {
            bars->scan[warp] = mine;
            bars->most[warp] = most;
        }
    }
}

// The producer warp's part.  `scales`: where an 8-bit stage's scale bytes go.
template <class S>
__device__ __forceinline__ void produce(const CUtensorMap &tmK, const CUtensorMap &tmV,
                                        const Params &p, StreamBars *bars, uint8_t *smem,
                                        uint8_t *scales) {
    constexpr int kUnit = S::kUnit, kThreads = S::kThreads, kStages = S::kStages;
    constexpr int kSegSlots = S::kSegSlots;
    const int lane = threadIdx.x & 31, m = sequences_each<S>(p);
    if (lane == 0) {
        tma_prefetch_desc(&tmK);
        tma_prefetch_desc(&tmV);
    }
    auto wait = [](uint64_t *bar, uint32_t parity) {
        return S::kQ8 ? quick_wait(bar, parity) : warp_wait(bar, parity);
    };
    bool ok = true;
    int u = 0;   // stages issued
    uint32_t owner = 0, phases = 0;   // a place's last group; bits 8 group + place: full's
    // boxes of a stage: one per page, or per 64 keys of a longer page
    const int box = min(p.page_size, kUnit), boxes = kUnit / box;
    // The batch as a list of items, 32 of them in the lanes at a time: sequences with all
    // their KV heads, or the CTA's whole pairs.
    const int items = !p.whole ? p.nseq
                               : (p.nseq * p.Hkv * p.blocks - static_cast<int>(blockIdx.x) +
                                  static_cast<int>(gridDim.x) - 1) / static_cast<int>(gridDim.x);
    // Pairs of an item: one, or an 8-bit stream's heads times the sequence's blocks of rows.
    int s_heads = p.whole ? 1 : p.Hkv;
    int base = 0, at = 0;      // the lanes' first item; the next one among them
    PackedSeq s{0, 0, 0};      // of this lane's item, as are the next three
    int s_seq = 0, s_head = 0, s_units = 0;
    auto load_items = [&](int first) {
        base = first;
        at = 0;
        s_units = 0;
        const int i = base + lane;
        if (i < items) {
            const int pair = p.whole ? static_cast<int>(blockIdx.x + i * gridDim.x) : 0;
            s_seq = p.whole ? pair / (p.Hkv * p.blocks) : i;
            // its first page entries, not after its lengths but with them
            if (p.whole) touch(p.pages + (long)s_seq * p.max_pages);
            s_head = p.whole ? pair - s_seq * p.Hkv * p.blocks : 0;
            s = packed_seq(p.cu, p.kv_lens, s_seq, p.bounds, p.whole ? p.status : nullptr);
            s_units = count_units<kUnit>(s, p.window);
            if constexpr (S::kQ8) {
                if (!p.whole) s_heads = p.Hkv * blocks_of<S>(p, s.T);
                else if (s_head % p.blocks >= blocks_of<S>(p, s.T)) s_units = 0;
            }
        }
    };
    int listed = 0;            // stages of the segments so far
    int head = 0, in = 0;      // the next pair's head within its item, units into it
    // The chunk at hand: its units left, the number of the next one, and the pair that goes
    // on behind it.
    int run = 0x7fffffff, chunk = blockIdx.x, pos = 0, all = 0, most = 0;
    Joint joint{0, 0, 0, 0, 0};
    if (!p.whole)
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) {
            all += bars->scan[w];
            most = max(most, bars->most[w]);
        }
    const Cut cut(all, most, p.chunks);
    auto start_chunk = [&]() {
        cut.get(chunk, pos, run);
        joint = {0, 0, 0, 0, 0};
        if (run == 0) return;
        // the warp's sequences that hold unit `pos`, and then the one
        int w = 0, before = 0;
        while (w < kThreads / 32 - 1 && pos >= before + bars->scan[w]) before += bars->scan[w++];
        int first = 32 * m * w, incl;
        while (true) {
            load_items(first);
            incl = (s_units > 0 ? s_units + S::kEndCost : 0) * s_heads;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int x = __shfl_up_sync(0xffffffffu, incl, d);
                if (lane >= d) incl += x;
            }
            const int here = __shfl_sync(0xffffffffu, incl, 31);
            if (pos < before + here || first + 32 >= items) break;
            before += here;
            first += 32;
        }
        const uint32_t behind = __ballot_sync(0xffffffffu, before + incl > pos);
        at = behind ? __ffs(behind) - 1 : 31;
        const int n = max(1, __shfl_sync(0xffffffffu, s_units, at)) + S::kEndCost;
        const int heads = S::kQ8 ? __shfl_sync(0xffffffffu, s_heads, at) : s_heads;
        const int rel = pos - before - (__shfl_sync(0xffffffffu, incl, at) - n * heads);
        head = rel / n;
        in = rel - head * n;
        if (S::kEndCost > 0 && in >= n - S::kEndCost) {   // within a pair's end: from the next one on
            pos += n - in;
            run = max(0, run - (n - in));
            in = 0;
            if (++head == heads) {
                head = 0;
                ++at;
            }
        }
    };
    int claims = 0;
    // Claims chunks until one has work; run = 0: there is none.
    auto next_chunk = [&]() {
        while (run == 0) {
            if (lane == 0 && GQA_IN_BOUNDS(chunk, p.chunks, p.status, kSite | 1))
                p.ws_joint[chunk] = joint;
            if (p.chunks == kSMs) return;   // a chunk per CTA
            if (lane == 0) {
                mbar_arrive_expect_tx(&bars->clc_full, 16);
                clc_try_cancel(&bars->clc_resp, &bars->clc_full);
            }
            if (!wait(&bars->clc_full, claims++ & 1)) {
                set_timeout(p.status, kDiagPagedDecode, kRoleProducer, 3, claims);
                ok = false;
                return;
            }
            chunk = clc_decode(&bars->clc_resp);
            fence_proxy_async_smem();   // read before the next response overwrites it
            __syncwarp();
            if (chunk < 0) return;
            start_chunk();
        }
    };
    if (p.whole) load_items(0);
    else start_chunk();
    auto next_segment = [&]() {
        Segment sg;
        sg.stages = -1;
        uint32_t with = 0;     // items with work, from the next one on
        while (run > 0) {
            with = at < 32 ? __ballot_sync(0xffffffffu, s_units > 0) >> at << at : 0u;
            if (with || base + 32 >= items) break;
            load_items(base + 32);
        }
        if (!with) return sg;
        const int l = __ffs(with) - 1;
        at = l;
        const int n = __shfl_sync(0xffffffffu, s_units, l);
        sg.row0 = __shfl_sync(0xffffffffu, s.row0, l);
        sg.T = __shfl_sync(0xffffffffu, s.T, l);
        sg.S = __shfl_sync(0xffffffffu, s.S, l);
        sg.seq = __shfl_sync(0xffffffffu, s_seq, l);
        sg.g = __shfl_sync(0xffffffffu, s_head, l) + head;
        sg.r0 = 0;
        int heads = s_heads;
        if constexpr (S::kQ8) {
            heads = __shfl_sync(0xffffffffu, s_heads, l);
            if (p.blocks > 1) {        // a head's blocks behind one another: they share its pages
                const int blocks = p.whole ? p.blocks : blocks_of<S>(p, sg.T);
                const int h = sg.g / blocks;
                sg.r0 = kBlockRows * (sg.g - h * blocks);
                sg.g = h;
            }
        }
        sg.unit0 = (p.window > 0 ? max(0, sg.S - sg.T - p.window + 1) / kUnit : 0) + in;
        sg.stages = min(run, n - in);
        sg.u0 = listed;
        listed += sg.stages;
        sg.slot = sg.stages == n ? -1 : 2 * chunk + (in == 0 ? 1 : 0);
        if (in == 0 && sg.stages < n)
            joint = {sg.row0, sg.g, S::kQ8 ? min(kBlockRows, sg.T * p.G - sg.r0) : sg.T * p.G,
                     cut.chunk_of(pos + n - 1) - chunk + 1, sg.r0};
        if (!p.whole) {
            run -= sg.stages;
            pos += sg.stages;
        }
        in += sg.stages;
        if (in == n) {
            if (S::kEndCost > 0 && !p.whole) {
                run = max(0, run - S::kEndCost);
                pos += S::kEndCost;
            }
            in = 0;
            if (++head == heads) {
                head = 0;
                ++at;
            }
        }
        return sg;
    };
    // The segment after the last one: its record out, its page entries on their way.  The
    // end is a record for each team.
    Segment ahead;
    PageWalk walk_ahead;
    int k = 0;
    auto advance = [&]() {
        if (run == 0) next_chunk();
        if (!ok) return;
        ahead = next_segment();
        const int records = ahead.stages < 0 ? S::kEnds : 1;
        for (int i = 0; i < records; ++i, ++k) {
            const int slot = k & (kSegSlots - 1);
            if (k >= kSegSlots && !wait(&bars->seg_free[slot], (k / kSegSlots - 1) & 1)) {
                set_timeout(p.status, kDiagPagedDecode, kRoleProducer, 0, k);
                ok = false;
                return;
            }
            if (lane == 0) {
                bars->seg[slot] = ahead;
                mbar_arrive(&bars->seg_full[slot]);
            }
            __syncwarp();
        }
        if (ahead.stages < 0) return;
        if (!GQA_IN_BOUNDS(ahead.S - 1 >> p.page_shift, p.max_pages, p.status, kSite | 2))
            ahead.S = 0;   // no entry is read, every key is zero fill
        walk_ahead = PageWalk(p.pages + (long)ahead.seq * p.max_pages,
                              ahead.unit0 * kUnit >> p.page_shift,
                              (ahead.S - 1 >> p.page_shift) + 1);
        // its queries on their way to L2: two 128-byte lines a row (8-bit: they are read a
        // pair ahead, by a warp of their own or by the consumers before they merge the last)
        if (!S::kQ8 && lane < 2 * ahead.T * p.G) {
            const int r = lane >> 1, t = token_of(p, r);
            prefetch_l2(p.q + (long)(ahead.row0 + t) * p.q_stride +
                        (ahead.g * p.G + r - t * p.G) * kD + 64 * (lane & 1));
        }
    };
    advance();
    Segment sg = ahead;
    PageWalk walk = walk_ahead;
    auto load = [&](int turn) {
        const int lo = p.window > 0 ? max(0, sg.S - sg.T - p.window + 1) : 0;
        for (int j = 0; j < sg.stages; ++j, ++u) {
            // the slab of this lane's box; -1 for one that no row sees or that is not in
            // the pool (its box is zero fill)
            const int unit_key = (sg.unit0 + j) * kUnit;
            const int pg = walk.get(unit_key >> p.page_shift, boxes);
            const int key0 = unit_key + lane * box;
            int slab = -1;
            if (lane < boxes && key0 < sg.S && key0 + box > lo) {
                if (pg >= 0 && pg < p.num_pages) slab = pg * p.Hkv + sg.g;
                else set_status(p.status, GQA_ERR_INVALID_ARG);
            }
            const int st = u % kStages, group = S::full_of(turn, j);
            uint64_t *full = &bars->full[group][st];
            uint8_t *dst = smem + st * kStageBytes + lane * box * (S::kQ8 ? kD : 2 * kD);
            const int row = unit_key & (p.page_size - 1);
            // every lane with a box waits, announces its bytes and loads for itself
            const bool free = u < kStages || mbar_wait(&bars->empty[st], (u / kStages - 1) & 1);
            if (free && lane < boxes) {
                if constexpr (S::kQ8) {
                    mbar_arrive_expect_tx(full, 2 * box * kD);
                    tma_load_3d(dst, &tmK, full, 0, 0, slab);
                    tma_load_3d(dst + kTileBytes, &tmV, full, 0, 0, slab);
                } else {
                    mbar_arrive_expect_tx(full, 2 * box * kD * 2);
                    tma_load_4d(dst, &tmK, full, 0, row, 0, slab);
                    tma_load_4d(dst + kTileBytes, &tmV, full, 0, row, 0, slab);
                }
            }
            if constexpr (S::kQ8) {
                // the bytes of 8 keys per lane (a page is a box: it has kUnit keys at most)
                const int key = 8 * lane & (kUnit - 1);
                const int at = __shfl_sync(0xffffffffu, slab, key >> p.page_shift);
                if (free && lane < kScaleCopies)
                    copy_async16(scales + (st * kUnit + key) * 2,
                                 p.scales + ((long)max(at, 0) * p.page_size + (key & (p.page_size - 1))) * 2,
                                 at >= 0 ? 16 : 0, full);
            }
            if (!__all_sync(0xffffffffu, free)) {
                set_timeout(p.status, kDiagPagedDecode, kRoleProducer, 1, u);
                ok = false;
                return;
            }
            owner = (owner & ~(1u << st)) | group << st;
            phases ^= 1u << (8 * group + st);
        }
    };
    // A segment is looked up ahead of the loads of the one before it; not the second one,
    // as the first one's loads wait for nothing that they can do without, and not a chunk's
    // first one, as chunks are claimed when they can be loaded.
#pragma unroll 1
    for (int turn = 0; ok && ahead.stages >= 0; ++turn) {
        sg = ahead;
        walk = walk_ahead;
        const int late = turn == 0 || run == 0 ? 1 : 0;
#pragma unroll 1
        for (int part = 0; part < 2 && ok; ++part) {
            if (part == late) advance();
            else load(turn);
        }
    }
    if (!ok) {   // never leave the CTA with copies in flight
        for (int st = 0; st < min(u, kStages); ++st) {
            const int group = owner >> st & 1;
            mbar_wait(&bars->full[group][st], (phases >> (8 * group + st) & 1) ^ 1);
        }
        if (claims > 0) mbar_wait(&bars->clc_full, (claims - 1) & 1);
    }
}

}  // namespace stream
}  // namespace gqa
