// paged_decode.cu -- attention of a few new tokens per sequence over a paged cache (d = 128):
// decode steps and short drafts, up to 16 rows (tokens x heads of a KV group) per sequence.
//
// For query token t of a sequence with S keys and T new tokens, at position i = S - T + t
// ("PLaMo 3アーキテクチャ徹底解析" §4.5, §5.1):
//   o = sum_j softmax_j(scale q . k_j) v_j  over j <= i (and i - j < W with a window).
// Every key and value is read once for all rows of its KV head, 512 bytes per key and head,
// and feeds 4 * 128 flops per row: the call is bound by memory, and the kernel is built to
// keep HBM busy.
//
// Work split.  The unit is 64 keys of one (sequence, KV head).  All units of the batch, in
// the order (sequence, KV head, keys), are cut into chunks whatever the lengths.  A pair of
// (sequence, KV head) that lies within one chunk is finished there; one that spans several
// leaves a partial (m, l, O) per chunk, at most two per chunk (its first and its last pair), and
// the combine kernel merges them.  A small batch has one chunk per SM.  Equal chunks are not
// equal times, though: over 32 caches of 8k-64k tokens the median SM was done at 703 us, the
// slowest at 791.  So a long batch has four levels of 152 chunks, of about 25/32, 1/8, 1/16 and
// 1/32 of an SM's share, which the CTAs claim in this order as they come free: 757 instead of
// 785 us (762 with three levels, 761 with five; below 128 units per SM the chunks' ends cost what
// the levels give: 88 for 89.5 us at 111 units, 68 for 67 at 70).  The cut is a function of the
// lengths alone, and so are the results.  Calls whose keys are few per pair take one CTA per
// pair and no second kernel.  The lengths are read on the device: every CTA sums the units of all
// sequences (a thread per sequence), and a chunk's start is found from those sums.
//
// A producer warp streams K and V by TMA into a ring of 6 stages of 64 keys (192 KB in
// flight per SM) and runs ahead over the ends of pairs; it looks pairs up 32 sequences at a time
// and a pair ahead of its loads (1024 caches of 100 tokens: 130 -> 119 us).  A box is one page
// with both halves of the head dimension (their rows 128-byte swizzled): for 64 windows of 2048
// keys in pages of 16, 98 us; with a box per half 121 us.  Two groups of four consumer warps take
// the pairs in turn, so that one group's ends (queries in, merge, outputs) pass while the other
// streams (the 1024 short caches: 115 -> 100 us, of which 79 are their whole pages at HBM's rate;
// long pairs do not care).  Each warp takes 16 keys of each stage.  S^T = K Q^T and O^T += V^T P^T
// are m16n8k16 bf16 MMAs with the keys, and then the dims, as M and 8 rows as N: half the
// products that the rows as M would take for up to 8 rows.  P leaves the score product
// transposed, 8 x 8 values at a time, as a B operand.  Accumulators and softmax statistics are
// fp32, P is rounded to bf16 for its product, and the row maximum moves only when a score exceeds
// it by 2^8 (exact: sum and O share the reference).  At the end of a pair a group's warps merge
// through shared memory.
//
// Measured (GB300): 32 caches of 8k-64k tokens, 8 KV heads, 64-token pages: 740-752 us, 7.2-7.3 TB/s.
//
// Hidden keys have weight 0, but 0 * NaN is NaN: in blocks that straddle an edge of the mask
// the values of keys that no row sees are zeroed on their way into the product, and
// non-finite ones that only some rows see are taken out and added to the rows that do.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math_constants.h>

#include "internal.h"
#include "packed.cuh"
#include "q8.cuh"

namespace gqa {
namespace {

constexpr int kD = 128;
constexpr int kTileBytes = 16384;               // K or V of a stage
constexpr int kStageBytes = 2 * kTileBytes;
constexpr int kMostStages = 6;
constexpr int kConsumers = 4;                   // warps of a group, a quarter of a stage's keys each
constexpr int kGroups = 2;                      // groups of consumers, which take the pairs in turn
constexpr int kThreads = 32 * (kGroups * kConsumers + 1);
constexpr int kMaxRows = 16;
constexpr int kScaleCopies = 16;                // lanes that copy an 8-bit stage's 256 scale bytes

// What the two kinds of cache differ in: keys of a stage (a unit), stages of the ring, and shared
// memory, in which an 8-bit cache's ring is followed by its stages' scale bytes.
template <bool Q8>
struct Ring {
    static constexpr int kUnit = Q8 ? 128 : 64;
    static constexpr int kStages = Q8 ? 5 : 6;
    static constexpr int kScales = kStages * kStageBytes;
    static constexpr int kXchg = kScales + (Q8 ? kStages * 2 * kUnit : 0);
    static constexpr int kBar = kXchg + kGroups * kConsumers * 8 * kD * 4;
    static constexpr int kBytes = kBar + 1536 + 1024;
};
constexpr float kRescaleThreshold = 8.0f;       // log2 units
// An 8-bit cache's weights go into their product as f16: up to 2^(9 + 6), and no less than 2^-24,
// 2^-33 of the reference.
constexpr float kGrow8 = 6.0f, kShift8 = 9.0f;
constexpr int kSegSlots = 4;
constexpr int kSMs = 152;
constexpr int kMinRun = 128;                    // units per SM from which chunks come in levels

// A run of stages of one (sequence, KV head).  stages < 0: no more.
struct Segment {
    int row0, T, S, seq, g, unit0, stages;
    int u0;     // stages of the CTA's run before it
    int slot;   // -1: all of the pair's keys; else the partial's place
};

// A pair whose keys begin in one chunk and go on in the next ones.  rows = 0: none.
struct Joint {
    int row0, g, rows, parts;
};

struct Bars {
    Segment seg[kSegSlots];
    uint64_t full[kGroups][kMostStages];   // a stage's load, for the group that takes it
    uint64_t empty[kMostStages];
    uint64_t seg_full[kSegSlots], seg_free[kSegSlots];
    uint64_t merge[kGroups];    // a group's warps meet (a barrier with a bounded wait)
    float2 ml[kGroups][kConsumers][8];
    uint4 clc_resp;
    uint64_t clc_full;
    int scan[kThreads / 32], most[kThreads / 32];   // units of each warp's sequences; of a pair
};
static_assert(sizeof(Bars) <= 1536, "barrier block");

struct Params {
    const __nv_bfloat16 *q;
    __nv_bfloat16 *o;
    float *lse;
    float *ws_o, *ws_ml;
    Joint *ws_joint;               // one per chunk
    int chunks;
    const int32_t *cu, *kv_lens, *pages;
    const uint8_t *scales;         // of an 8-bit cache
    int joint, v_first;            // an 8-bit cache's box has keys and values, these first
    int *status;
    long q_stride, o_stride;
    PackedBounds bounds;
    int nseq, Hq, Hkv, G, window, num_pages, page_size, page_shift, max_pages;
    uint32_t inv_g;                // 2^16 / G, rounded up
    int whole;                     // 1: CTAs take whole pairs, every gridDim.x-th one
    float scale_log2;
};

// r / G for a row r <= kMaxRows of a pair (the error, r / 2^16 at most, is below 1 / G).
__device__ __forceinline__ int token_of(const Params &p, int r) {
    return static_cast<int>(r * p.inv_g >> 16);
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

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
        "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma16816_f16(float (&c)[4], uint32_t a0, uint32_t a1,
                                             uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
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
// byte - 127, the exponent that a scale byte stands for; NaN for 255.
__device__ __forceinline__ float exponent_of(uint32_t byte) {
    return byte == kScaleNan ? CUDART_NAN_F : __uint_as_float(0x4b000000u | byte) - 8388735.0f;
}
// Clears the NaN among the four e4m3 in w; true if there was one.
__device__ __forceinline__ bool strip_nan(uint32_t &w) {
    const uint32_t nan = __vcmpeq4(w & 0x7f7f7f7fu, 0x7f7f7f7fu);
    w &= ~nan;
    return nan != 0;
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm4_trans(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

// Clears the non-finite ones of the two bf16 in w; true if there was one.
__device__ __forceinline__ bool strip_nonfinite(uint32_t &w) {
    const bool lo = (w & 0x7f80u) == 0x7f80u, hi = (w & 0x7f800000u) == 0x7f800000u;
    if (lo) w &= 0xffff0000u;
    if (hi) w &= 0x0000ffffu;
    return lo || hi;
}

// The transpose of an 8 x 8 matrix of 16-bit values, a row in four lanes.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
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

enum Role { kRoleProducer = 0, kRoleConsumer = 2 };
constexpr int kSite = kDiagPagedDecode << 24;   // of the debug build's checks

// ROWS: the most rows of a pair, 8 or 16.  Q8: an 8-bit cache.
template <int ROWS, bool Q8>
__global__ void __launch_bounds__(kThreads, 1)
    paged_decode_kernel(const __grid_constant__ CUtensorMap tmK,
                        const __grid_constant__ CUtensorMap tmV, const Params p) {
    griddep_wait();
    griddep_launch_dependents();
    constexpr int kUnit = Ring<Q8>::kUnit, kStages = Ring<Q8>::kStages;
    constexpr int kRow = Q8 ? kD : 2 * kD;   // bytes of a key or value
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_addr = smem_u32(smem_raw);
    uint8_t *smem = smem_raw + (((raw_addr + 1023u) & ~1023u) - raw_addr);
    Bars *bars = reinterpret_cast<Bars *>(smem + Ring<Q8>::kBar);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // The groups take a pair's stages in turn, or the pairs.
    const bool both = Q8 && !p.whole;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            for (int g = 0; g < kGroups; ++g)
                mbar_init(&bars->full[g][i],
                          kUnit / min(p.page_size, kUnit) + (Q8 ? kScaleCopies : 0));
            mbar_init(&bars->empty[i], kConsumers);
        }
        for (int i = 0; i < kSegSlots; ++i) {
            mbar_init(&bars->seg_full[i], 1);
            mbar_init(&bars->seg_free[i], both ? kGroups * kConsumers : kConsumers);
        }
        for (int g = 0; g < kGroups; ++g)
            mbar_init(&bars->merge[g], both ? kGroups * kConsumers : kConsumers);
        mbar_init(&bars->clc_full, 1);
        fence_mbar_init();
    }
    // ---- the batch's units: each warp's sequences, in order
    const int m = (p.nseq + kThreads - 1) / kThreads;   // sequences per thread
    if (!p.whole) {
        const int s0 = threadIdx.x * m;
        int mine = 0, most = 0;
        for (int i = s0; i < s0 + m && i < p.nseq; ++i) {
            const int n = count_units<kUnit>(packed_seq(p.cu, p.kv_lens, i, p.bounds, p.status), p.window);
            mine += p.Hkv * n;
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
    __syncthreads();

    if (warp == kGroups * kConsumers) {
        // ================= producer =================
        if (lane == 0) {
            tma_prefetch_desc(&tmK);
            tma_prefetch_desc(&tmV);
        }
        bool ok = true;
        int u = 0;   // stages issued
        uint32_t owner = 0, phases = 0;   // a place's last group; bits 8 group + place: full's
        // boxes of a stage: one per page, or per 64 keys of a longer page
        const int box = min(p.page_size, kUnit), boxes = kUnit / box;
        // The batch as a list of items, 32 of them in the lanes at a time: sequences with all
        // their KV heads, or the CTA's whole pairs.
        const int items = !p.whole ? p.nseq
                                   : (p.nseq * p.Hkv - static_cast<int>(blockIdx.x) +
                                      static_cast<int>(gridDim.x) - 1) / static_cast<int>(gridDim.x);
        const int heads = p.whole ? 1 : p.Hkv;
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
                s_seq = p.whole ? pair / p.Hkv : i;
                // its first page entries, not after its lengths but with them
                if (p.whole) touch(p.pages + (long)s_seq * p.max_pages);
                s_head = p.whole ? pair - s_seq * p.Hkv : 0;
                s = packed_seq(p.cu, p.kv_lens, s_seq, p.bounds, p.whole ? p.status : nullptr);
                s_units = count_units<kUnit>(s, p.window);
            }
        };
        int listed = 0;            // stages of the segments so far
        int head = 0, in = 0;      // the next pair's head within its item, units into it
        // The chunk at hand: its units left, the number of the next one, and the pair that goes
        // on behind it.
        int run = 0x7fffffff, chunk = blockIdx.x, pos = 0, all = 0, most = 0;
        Joint joint{0, 0, 0, 0};
        if (!p.whole)
#pragma unroll
            for (int w = 0; w < kThreads / 32; ++w) {
                all += bars->scan[w];
                most = max(most, bars->most[w]);
            }
        const Cut cut(all, most, p.chunks);
        auto start_chunk = [&]() {
            cut.get(chunk, pos, run);
            joint = {0, 0, 0, 0};
            if (run == 0) return;
            // the warp's sequences that hold unit `pos`, and then the one
            int w = 0, before = 0;
            while (w < kThreads / 32 - 1 && pos >= before + bars->scan[w]) before += bars->scan[w++];
            int first = 32 * m * w, incl;
            while (true) {
                load_items(first);
                incl = s_units * heads;
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
            const int n = max(1, __shfl_sync(0xffffffffu, s_units, at));
            const int rel = pos - before - (__shfl_sync(0xffffffffu, incl, at) - n * heads);
            head = rel / n;
            in = rel - head * n;
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
                if (!warp_wait(&bars->clc_full, claims++ & 1)) {
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
            sg.unit0 = (p.window > 0 ? max(0, sg.S - sg.T - p.window + 1) / kUnit : 0) + in;
            sg.stages = min(run, n - in);
            sg.u0 = listed;
            listed += sg.stages;
            sg.slot = sg.stages == n ? -1 : 2 * chunk + (in == 0 ? 1 : 0);
            if (in == 0 && sg.stages < n)
                joint = {sg.row0, sg.g, sg.T * p.G, cut.chunk_of(pos + n - 1) - chunk + 1};
            if (!p.whole) {
                run -= sg.stages;
                pos += sg.stages;
            }
            in += sg.stages;
            if (in == n) {
                in = 0;
                if (++head == heads) {
                    head = 0;
                    ++at;
                }
            }
            return sg;
        };
        // The segment after the last one: its record out, its page entries on their way.  The
        // end is a record for each group.
        Segment ahead;
        PageWalk walk_ahead;
        int k = 0;
        auto advance = [&]() {
            if (run == 0) next_chunk();
            if (!ok) return;
            ahead = next_segment();
            const int records = ahead.stages < 0 && !both ? kGroups : 1;
            for (int i = 0; i < records; ++i, ++k) {
                const int slot = k & (kSegSlots - 1);
                if (k >= kSegSlots && !warp_wait(&bars->seg_free[slot], (k / kSegSlots - 1) & 1)) {
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
            // its queries on their way to L2: two 128-byte lines a row
            if (lane < 2 * ahead.T * p.G) {
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
                const int st = u % kStages, group = (both ? j : turn) % kGroups;
                uint64_t *full = &bars->full[group][st];
                uint8_t *dst = smem + st * kStageBytes + lane * box * kRow * (Q8 ? 2 : 1);
                const int row = unit_key & (p.page_size - 1);
                // every lane with a box waits, announces its bytes and loads for itself
                const bool free = u < kStages || mbar_wait(&bars->empty[st], (u / kStages - 1) & 1);
                if (free && lane < boxes) {
                    mbar_arrive_expect_tx(full, 2 * box * kRow);
                    if constexpr (Q8) {
                        tma_load_4d(dst, &tmK, full, 0, row, slab, 0);
                        if (!p.joint) tma_load_4d(dst + box * kRow, &tmV, full, 0, row, slab, 0);
                    } else {
                        tma_load_4d(dst, &tmK, full, 0, row, 0, slab);
                        tma_load_4d(dst + kTileBytes, &tmV, full, 0, row, 0, slab);
                    }
                }
                if constexpr (Q8) {
                    // the bytes of 8 keys per lane (a third copy per page by TMA took longer than
                    // the keys: windows of 2048 in pages of 16 @@)
                    const int key = 8 * lane & (kUnit - 1), from = key / box;
                    const int at = __shfl_sync(0xffffffffu, slab, from);
                    if (free && lane < kScaleCopies)
                        copy_async16(smem + Ring<Q8>::kScales + (st * kUnit + key) * 2,
                                     p.scales + ((long)max(at, 0) * p.page_size + row + key % box) * 2,
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
        return;
    }

    // ================= consumers =================
    const int gq = lane >> 2, tq = lane & 3;
    constexpr int HR = ROWS / 8;                  // row halves in use
    const uint32_t ring = smem_u32(smem);
    const int group = warp / kConsumers, cw = warp % kConsumers;
    float *xchg = reinterpret_cast<float *>(smem + Ring<Q8>::kXchg) + group * kConsumers * 8 * kD;
    float2(*ml)[8] = bars->ml[group];
    // ldmatrix rows, both operands A: K: matrices (chunk 2ks | 2ks + 1) x (keys 0-7 | 8-15);
    // V transposed: (keys 0-7 | 8-15) x (dim chunk 2nn | 2nn + 1)
    const int mat = lane >> 3, l7 = lane & 7;
    const int box = min(p.page_size, kUnit);
    const uint32_t half = box * 128;          // a box: its rows' dims 0-63, then 64-127
    const int part = kUnit / kConsumers * cw;   // first of this warp's keys in a stage
    const uint32_t rows16 = part / box * 2 * half + part % box * 128;
    const uint32_t k_row = rows16 + (((mat & 1) << 3) + l7) * 128;
    const uint32_t v_row = kTileBytes + rows16 + (((mat >> 1) << 3) + l7) * 128;
    // swizzled place of chunk 2i (or 2i + 1) of a half, i = 0..3
    uint32_t k_off[4], v_off[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        k_off[i] = k_row + (((2 * i + (mat >> 1)) ^ l7) << 4);
        v_off[i] = v_row + (((2 * i + (mat & 1)) ^ l7) << 4);
    }
    // An 8-bit cache's: rows of 128 bytes, 128-byte swizzled.  A block of 16 keys has the keys
    // 0-7 and 8 + (0-7 ^ 4) as the rows 0-7 and 8-15 of the score product's A operand.  There
    // each four numbers of a lane are two of the product's k-steps' pairs: the queries' dims are
    // taken in the same order.  V's 16 x 16 matrices, transposed, bring a lane four rows, which
    // are the keys of its pairs 2tq, + 1 and 8 + 2tq, + 1 in the value product: rows 4i .. 4i + 3
    // are the score rows 2i, 2i + 1, 8 + 2i, 8 + 2i + 1.  (The ^ 4: eight rows of either operand
    // lie in eight different swizzled columns.)
    // A box of a stage has the keys of a page (or a unit's rows of it) and their values.
    uint32_t k8[2] = {0, 0}, v8 = 0, block8[2] = {0, 0};
    const uint32_t values8 = p.v_first ? 0 : box * kD, keys8 = box * kD - values8;
    if constexpr (Q8) {
        const int kk = mat & 1 ? 8 + (l7 ^ 4) : l7;
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            block8[b] = (part + 16 * b) / box * 2 * box * kD + (part + 16 * b) % box * kD;
            k8[b] = block8[b] + keys8 + kk * kD + (((mat >> 1) ^ (kk & 7)) << 4);
        }
        const int rho = lane & 15, i = 2 * (rho >> 2) + (rho & 1);
        const int vk = rho & 2 ? 8 + (i ^ 4) : i;
        v8 = block8[lane >> 4] + values8 + vk * kD + ((vk & 7) << 4);
    }
    int meets = 0;
    auto meet = [&]() {
        __syncwarp();
        uint64_t *bar = &bars->merge[both ? 0 : group];
        if (lane == 0) mbar_arrive(bar);
        if (warp_wait(bar, meets++ & 1)) return true;
        set_timeout(p.status, kDiagPagedDecode, kRoleConsumer, 2, meets);
        return false;
    };
    // Segment k and this thread's part of its queries, rows gq and gq + 8 (rows past the last
    // one are zero).
    Segment sg;
    uint32_t qb[8][2 * HR];
    float sl_next[HR][2];   // an 8-bit cache's: the factor of a score of this thread's columns
    auto next_segment = [&](int k) {
        const int slot = k & (kSegSlots - 1);
        if (!warp_wait(&bars->seg_full[slot], (k / kSegSlots) & 1)) {
            set_timeout(p.status, kDiagPagedDecode, kRoleConsumer, 0, k);
            return false;
        }
        sg = bars->seg[slot];
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->seg_free[slot]);
        const int rows = sg.stages < 0 ? 0 : sg.T * p.G;   // <= ROWS (the host's rule on max_q)
#pragma unroll
        for (int h = 0; h < HR; ++h) {
            const int r = gq + 8 * h, t = token_of(p, r);
            const __nv_bfloat16 *qr = p.q + (long)(sg.row0 + t) * p.q_stride +
                                      (sg.g * p.G + (r - t * p.G)) * kD + (Q8 ? 4 : 2) * tq;
#pragma unroll
            for (int ks = 0; ks < 8; ++ks) {
                qb[ks][h] = qb[ks][HR + h] = 0u;
                if (r < rows && GQA_IN_BOUNDS(sg.row0 + t, p.bounds.total, p.status, kSite | 3)) {
                    if constexpr (Q8) {
                        const uint2 w = __ldg(reinterpret_cast<const uint2 *>(qr + 16 * ks));
                        qb[ks][h] = w.x;
                        qb[ks][HR + h] = w.y;
                    } else {
                        qb[ks][h] = __ldg(reinterpret_cast<const uint32_t *>(qr + 16 * ks));
                        qb[ks][HR + h] = __ldg(reinterpret_cast<const uint32_t *>(qr + 16 * ks + 8));
                    }
                }
            }
            if constexpr (Q8) {
                // To f16, the row's largest element brought to [2^14, 2^15): what that leaves of
                // a number below 2^-14 is a multiple of 2^-24, 2^-38 of the largest at most.
                float most = 0.f;
#pragma unroll
                for (int ks = 0; ks < 8; ++ks)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const uint32_t w = qb[ks][HR * i + h];
                        most = amax_nan(most, amax_nan(bf16lo(w), bf16hi(w)));
                    }
                most = amax_nan(most, __shfl_xor_sync(0xffffffffu, most, 1));
                most = amax_nan(most, __shfl_xor_sync(0xffffffffu, most, 2));
                const uint32_t e = max(__float_as_uint(most) >> 23, 15u);
                const float up = __uint_as_float((268 - e) << 23);
#pragma unroll
                for (int ks = 0; ks < 8; ++ks)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const uint32_t w = qb[ks][HR * i + h];
                        const __half2 y = __floats2half2_rn(bf16lo(w) * up, bf16hi(w) * up);
                        qb[ks][HR * i + h] = *reinterpret_cast<const uint32_t *>(&y);
                    }
                // the way back, from the lanes of rows 2tq, + 1
                const float down = __uint_as_float((e - 14) << 23) * p.scale_log2;
#pragma unroll
                for (int c = 0; c < 2; ++c)
                    sl_next[h][c] = __shfl_sync(0xffffffffu, down, 4 * (2 * tq + c));
            }
        }
        return true;
    };
    const int first = both ? 0 : group, step = both ? 1 : kGroups;
    if (!next_segment(first)) return;
    uint32_t phases = 0;   // of the group's full barriers, a bit each
    for (int k = first; sg.stages >= 0; k += step) {
        const int rows = sg.T * p.G;
        float sl[HR][2];        // a score's factor, in log2 units
#pragma unroll
        for (int h = 0; h < HR; ++h)
#pragma unroll
            for (int c = 0; c < 2; ++c) sl[h][c] = Q8 ? sl_next[h][c] : p.scale_log2;
        // this thread's columns of the products: rows 8h + 2tq, + 1 (positions of rows past the
        // last one: the last)
        int qpos[HR][2];
#pragma unroll
        for (int h = 0; h < HR; ++h)
#pragma unroll
            for (int c = 0; c < 2; ++c)
                qpos[h][c] = sg.S - sg.T + min(token_of(p, 8 * h + 2 * tq + c), sg.T - 1);
        const int q_first = sg.S - sg.T;          // hi_all: keys beyond are hidden from some
        const int lo = p.window > 0 ? max(0, q_first - p.window + 1) : 0;
        const int lo_all = p.window > 0 ? max(0, sg.S - p.window) : 0;
        // o[i][h]: dims 16 i + gq (+ 8 for the second pair) of those rows
        float o[8][HR][4];
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int h = 0; h < HR; ++h) o[i][h][0] = o[i][h][1] = o[i][h][2] = o[i][h][3] = 0.f;
        float m[HR][2], mr[HR][2], l[HR][2];      // mr: m, or 0 while m is -inf
        float mo[HR][2];        // an 8-bit cache's: O's reference, the weight of 1 of a value of 1
#pragma unroll
        for (int h = 0; h < HR; ++h)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                m[h][c] = mo[h][c] = -CUDART_INF_F;
                mr[h][c] = l[h][c] = 0.f;
            }
        const int j0 = both ? group : 0, dj = both ? kGroups : 1;
        for (int j = j0, u = sg.u0 + j0; j < sg.stages; j += dj, u += dj) {
            const int st = u % kStages;
            if (!warp_wait(&bars->full[group][st], phases >> st & 1)) {
                set_timeout(p.status, kDiagPagedDecode, kRoleConsumer, 1, u);
                return;
            }
            phases ^= 1u << st;
            const int kb = (sg.unit0 + j) * kUnit + part;   // this warp's keys
            if constexpr (Q8) {
                if (kb < sg.S && kb + 31 >= lo) {
                    const uint32_t base = ring + st * kStageBytes;
                    const uint16_t *bytes = reinterpret_cast<const uint16_t *>(
                                                smem + Ring<Q8>::kScales) + st * kUnit + part;
                    // ---- scores: two blocks of 16 keys x rows
                    float x[2][HR][4], xs[2][2][HR][4];
#pragma unroll
                    for (int b = 0; b < 2; ++b)
#pragma unroll
                        for (int h = 0; h < HR; ++h)
#pragma unroll
                            for (int e = 0; e < 4; ++e) xs[0][b][h][e] = xs[1][b][h][e] = 0.f;
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int b = 0; b < 2; ++b) {
                            uint32_t w[4];
                            ldsm4(w, (base + k8[b]) ^ (i << 5));
#pragma unroll
                            for (int s = 0; s < 2; ++s) {
                                const uint32_t a0 = e4m3x2_f16x2(w[2 * s]);
                                const uint32_t a1 = e4m3x2_f16x2(w[2 * s + 1]);
                                const uint32_t a2 = e4m3x2_f16x2(w[2 * s] >> 16);
                                const uint32_t a3 = e4m3x2_f16x2(w[2 * s + 1] >> 16);
#pragma unroll
                                for (int h = 0; h < HR; ++h)
                                    mma16816_f16(xs[s][b][h], a0, a1, a2, a3, qb[2 * i + s][h],
                                                 qb[2 * i + s][HR + h]);
                            }
                        }
                    // x[b][h]: keys kb + 16b + gq (rows 8h + 2tq, + 1) and + 8 + (gq ^ 4)
                    float ev[2][2];   // the values' exponents
#pragma unroll
                    for (int b = 0; b < 2; ++b)
#pragma unroll
                        for (int f = 0; f < 2; ++f) {
                            const uint32_t w = bytes[16 * b + (f ? 8 + (gq ^ 4) : gq)];
                            const float kf = scale_of(w & 255u);
                            ev[b][f] = exponent_of(w >> 8);
#pragma unroll
                            for (int h = 0; h < HR; ++h)
#pragma unroll
                                for (int c = 0; c < 2; ++c)
                                    x[b][h][2 * f + c] =
                                        (xs[0][b][h][2 * f + c] + xs[1][b][h][2 * f + c]) * kf;
                        }
                    const bool edge = kb + 31 > q_first || kb < lo_all;   // of the mask
                    uint32_t hidden = 0;   // bits 4 (2b + h) + e
                    if (edge) {
#pragma unroll
                        for (int b = 0; b < 2; ++b)
#pragma unroll
                            for (int h = 0; h < HR; ++h)
#pragma unroll
                                for (int e = 0; e < 4; ++e) {
                                    const int key = kb + 16 * b + (e >> 1 ? 8 + (gq ^ 4) : gq);
                                    const int at = qpos[h][e & 1];
                                    if (key > at || (p.window > 0 && at - key >= p.window)) {
                                        x[b][h][e] = -CUDART_INF_F;
                                        hidden |= 1u << (4 * (2 * b + h) + e);
                                    }
                                }
                    }
                    // ---- online softmax: the references move only when something exceeds them
                    // by 2^6
                    bool grow = false;
                    float top[HR][2], topo[HR][2];
#pragma unroll
                    for (int h = 0; h < HR; ++h)
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            float t = -CUDART_INF_F, to = -CUDART_INF_F;
#pragma unroll
                            for (int b = 0; b < 2; ++b)
#pragma unroll
                                for (int f = 0; f < 2; ++f) {
                                    const float y = x[b][h][2 * f + c];
                                    t = fmaxf(t, y);
                                    to = fmaxf(to, fmaf(y, sl[h][c], ev[b][f]));
                                }
                            top[h][c] = t * sl[h][c];
                            topo[h][c] = to;
                            grow |= top[h][c] > m[h][c] + kGrow8 || to > mo[h][c] + kGrow8;
                        }
                    if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
                        for (int h = 0; h < HR; ++h)
#pragma unroll
                            for (int c = 0; c < 2; ++c) {
                                float mx = top[h][c], mxo = topo[h][c];
#pragma unroll
                                for (int d = 4; d < 32; d <<= 1) {
                                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
                                    mxo = fmaxf(mxo, __shfl_xor_sync(0xffffffffu, mxo, d));
                                }
                                const float mn = fmaxf(m[h][c], mx), mno = fmaxf(mo[h][c], mxo);
                                const float f = m[h][c] == -CUDART_INF_F ? 0.f : ex2_approx(m[h][c] - mn);
                                const float fo =
                                    mo[h][c] == -CUDART_INF_F ? 1.f : ex2_approx(mo[h][c] - mno);
                                m[h][c] = mn;
                                mr[h][c] = mn == -CUDART_INF_F ? 0.f : mn;
                                l[h][c] *= f;
                                mo[h][c] = mno;
#pragma unroll
                                for (int i = 0; i < 8; ++i) {
                                    o[i][h][c] *= fo;
                                    o[i][h][2 + c] *= fo;
                                }
                            }
                    }
                    // P as the B operand: row gq of half h, the score rows 2tq, + 1 and 8 + 2tq,
                    // + 1 of a block.  The sum takes the weights, O their products with the
                    // values' powers of two, 2^9 where that is the reference.
                    uint32_t pb[2][HR][2];
#pragma unroll
                    for (int b = 0; b < 2; ++b)
#pragma unroll
                        for (int h = 0; h < HR; ++h) {
                            float w[4], wv[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const int c = e & 1;
                                const float ro = mo[h][c] == -CUDART_INF_F ? 0.f : mo[h][c] - kShift8;
                                w[e] = ex2_approx(fmaf(x[b][h][e], sl[h][c], -mr[h][c]));
                                wv[e] = ex2_approx(fmaf(x[b][h][e], sl[h][c], ev[b][e >> 1] - ro));
                            }
                            if (edge) {
#pragma unroll
                                for (int e = 0; e < 4; ++e)
                                    if (hidden >> (4 * (2 * b + h) + e) & 1) wv[e] = 0.f;
                            }
                            l[h][0] += w[0] + w[2];
                            l[h][1] += w[1] + w[3];
                            pb[b][h][0] = transpose8x8(pack_f16x2(wv[0], wv[1]));
                            pb[b][h][1] = transpose8x8(pack_f16x2(wv[2], wv[3]));
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
                        ldsm_b8_trans(w, (base + v8) ^ (nn << 4));
                        if (edge) {
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                w[i] &= seen[i >> 1];
                                if (sg.T > 1) stripped |= strip_nan(w[i]);
                            }
                        }
#pragma unroll
                        for (int b = 0; b < 2; ++b) {
                            const uint32_t a0 = e4m3x2_f16x2(w[2 * b]);
                            const uint32_t a1 = e4m3x2_f16x2(w[2 * b + 1]);
                            const uint32_t a2 = e4m3x2_f16x2(w[2 * b] >> 16);
                            const uint32_t a3 = e4m3x2_f16x2(w[2 * b + 1] >> 16);
#pragma unroll
                            for (int h = 0; h < HR; ++h)
                                mma16816_f16(o[nn][h], a0, a1, a2, a3, pb[b][h][0], pb[b][h][1]);
                        }
                    }
                    if (__any_sync(0xffffffffu, stripped)) {
                        // the NaN that were taken out, for the rows that see them
                        for (int kk = 0; kk < 32; ++kk) {
                            const int key = kb + kk;
                            if (key < lo || key >= sg.S) continue;
                            const uint8_t *vr = smem + st * kStageBytes + block8[kk >> 4] + values8 +
                                                (kk & 15) * kD + gq;
#pragma unroll
                            for (int i = 0; i < 8; ++i)
#pragma unroll
                                for (int e = 0; e < 2; ++e) {
                                    if ((vr[((i ^ (kk & 7)) << 4) + 8 * e] & 0x7f) != 0x7f) continue;
#pragma unroll
                                    for (int h = 0; h < HR; ++h)
#pragma unroll
                                        for (int c = 0; c < 2; ++c)
                                            if (key <= qpos[h][c] &&
                                                (p.window <= 0 || qpos[h][c] - key < p.window))
                                                o[i][h][2 * e + c] = CUDART_NAN_F;
                                }
                        }
                    }
                }
            } else if (kb < sg.S && kb + 15 >= lo) {
                const uint32_t base = ring + st * kStageBytes;
                // ---- scores: 16 keys x rows, in chains of four products
                constexpr int kChains = 2;
                float x[HR][4], xs[kChains][HR][4];
#pragma unroll
                for (int h = 0; h < HR; ++h)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
#pragma unroll
                        for (int c = 0; c < kChains; ++c) xs[c][h][e] = 0.f;
#pragma unroll
                for (int ks = 0; ks < 8; ++ks) {
                    uint32_t a[4];
                    ldsm4(a, (ks < 4 ? base : base + half) + k_off[ks & 3]);
#pragma unroll
                    for (int h = 0; h < HR; ++h)
                        mma16816(xs[ks % kChains][h], a[0], a[1], a[2], a[3], qb[ks][h], qb[ks][HR + h]);
                }
                // x[h]: keys kb + gq (rows 8h + 2tq, + 1), kb + gq + 8 (the same rows)
#pragma unroll
                for (int h = 0; h < HR; ++h)
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[h][e] = xs[0][h][e] + xs[1][h][e];
                const bool edge = kb + 15 > q_first || kb < lo_all;   // of the mask
                if (edge) {
#pragma unroll
                    for (int h = 0; h < HR; ++h)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int key = kb + gq + 8 * (e >> 1), at = qpos[h][e & 1];
                            if (key > at || (p.window > 0 && at - key >= p.window))
                                x[h][e] = -CUDART_INF_F;
                        }
                }
                // ---- online softmax: the maximum moves only when a score exceeds it by 2^8
                bool grow = false;
#pragma unroll
                for (int h = 0; h < HR; ++h)
#pragma unroll
                    for (int c = 0; c < 2; ++c)
                        grow |= fmaxf(x[h][c], x[h][2 + c]) * p.scale_log2 >
                                m[h][c] + kRescaleThreshold;
                if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
                    for (int h = 0; h < HR; ++h)
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            float mx = fmaxf(x[h][c], x[h][2 + c]);
#pragma unroll
                            for (int d = 4; d < 32; d <<= 1)
                                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
                            const float mn = fmaxf(m[h][c], mx * p.scale_log2);
                            const float f =
                                m[h][c] == -CUDART_INF_F ? 0.f : ex2_approx(m[h][c] - mn);
                            m[h][c] = mn;
                            mr[h][c] = mn == -CUDART_INF_F ? 0.f : mn;
                            l[h][c] *= f;
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                o[i][h][c] *= f;
                                o[i][h][2 + c] *= f;
                            }
                        }
                }
                // P as the B operand: row gq of half h, keys 2tq, + 1 and 8 + 2tq, + 1; the
                // sum takes the unrounded weights
                uint32_t pb[HR][2];
#pragma unroll
                for (int h = 0; h < HR; ++h) {
                    float w[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        w[e] = ex2_approx(fmaf(x[h][e], p.scale_log2, -mr[h][e & 1]));
                    l[h][0] += w[0] + w[2];
                    l[h][1] += w[1] + w[3];
                    pb[h][0] = transpose8x8(pack_bf16x2(w[0], w[1]));
                    pb[h][1] = transpose8x8(pack_bf16x2(w[2], w[3]));
                }
                // ---- O += V^T P
                // masks of the A fragment's keys 2tq, + 1 (and + 8): those that some row sees
                uint32_t seen0 = 0xffffffffu, seen1 = 0xffffffffu;
                if (edge) {
                    const int ka = kb + 2 * tq;
                    auto in = [&](int key) { return key >= lo && key < sg.S; };
                    seen0 = (in(ka) ? 0xffffu : 0u) | (in(ka + 1) ? 0xffff0000u : 0u);
                    seen1 = (in(ka + 8) ? 0xffffu : 0u) | (in(ka + 9) ? 0xffff0000u : 0u);
                }
                bool stripped = false;
#pragma unroll
                for (int nn = 0; nn < 8; ++nn) {
                    uint32_t a[4];
                    ldsm4_trans(a, (nn < 4 ? base : base + half) + v_off[nn & 3]);
                    if (edge) {
                        a[0] &= seen0;
                        a[1] &= seen0;
                        a[2] &= seen1;
                        a[3] &= seen1;
                        if (sg.T > 1) {   // some of the block's keys are hidden from some rows
#pragma unroll
                            for (int i = 0; i < 4; ++i) stripped |= strip_nonfinite(a[i]);
                        }
                    }
#pragma unroll
                    for (int h = 0; h < HR; ++h)
                        mma16816(o[nn][h], a[0], a[1], a[2], a[3], pb[h][0], pb[h][1]);
                }
                if (__any_sync(0xffffffffu, stripped)) {
                    // add what was taken out to the rows that see it
                    for (int kk = 0; kk < 16; ++kk) {
                        const int key = kb + kk;
                        if (key < lo || key >= sg.S) continue;
                        const uint8_t *vr = smem + st * kStageBytes + kTileBytes + rows16 +
                                            kk * 128 + 2 * gq;
#pragma unroll
                        for (int i = 0; i < 8; ++i)
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const uint32_t w = *reinterpret_cast<const uint16_t *>(
                                    vr + (i >> 2) * half + (((2 * (i & 3) + e) ^ (kk & 7)) << 4));
                                const float y = bf16lo(w);
                                if (isfinite(y)) continue;
#pragma unroll
                                for (int h = 0; h < HR; ++h)
#pragma unroll
                                    for (int c = 0; c < 2; ++c)
                                        if (key <= qpos[h][c] &&
                                            (p.window <= 0 || qpos[h][c] - key < p.window))
                                            o[i][h][2 * e + c] += y;
                            }
                    }
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars->empty[st]);
        }
        if constexpr (Q8) {
            // O relative to m: times 2^(mo - 9 - m), in two steps as that may be 2^-135
#pragma unroll
            for (int h = 0; h < HR; ++h)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    if (mo[h][c] == -CUDART_INF_F) continue;   // O is 0, or NaN
                    float mg = m[h][c], mog = mo[h][c];
                    const float f = ex2_approx(0.5f * (mog - kShift8 - mg));
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        o[i][h][c] = o[i][h][c] * f * f;
                        o[i][h][2 + c] = o[i][h][2 + c] * f * f;
                    }
                }
        }
        // ---- the pair's (or span's) result.  The next one's queries are on their way
        // meanwhile.
        const int row0 = sg.row0, head0 = sg.g * p.G, out = sg.slot;
        if (!next_segment(k + step)) return;
        // The warps' shares meet in shared memory, 8 rows at a time, each relative to its own
        // maximum: [warp][row][128 dims], a row's dims permuted so that the lanes (4 rows x 8
        // dims) meet 32 different banks.
#pragma unroll
        for (int h = 0; h < HR; ++h) {
            if (meets > 0 && !meet()) return;   // the last ones have been read
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int r = 2 * tq + c;
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) l[h][c] += __shfl_xor_sync(0xffffffffu, l[h][c], d);
                if (gq == 0) ml[cw][r] = make_float2(m[h][c], l[h][c]);
                float *mine = xchg + (cw * 8 + r) * kD;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    mine[(16 * i + gq) ^ (tq << 3)] = o[i][h][c];
                    mine[(16 * i + 8 + gq) ^ (tq << 3)] = o[i][h][2 + c];
                }
            }
            if (!meet()) return;
            // a warp adds up every fourth row (every eighth of the groups' together), 4 dims per
            // lane
            const float2(*mls)[8] = both ? bars->ml[0] : ml;
            const float *shares = both ? xchg - group * kConsumers * 8 * kD : xchg;
            for (int rr = both ? warp : cw; rr < min(8, rows - 8 * h);
                 rr += both ? kGroups * kConsumers : kConsumers) {
                const int r = 8 * h + rr;
                constexpr int kShares = Q8 ? kGroups * kConsumers : kConsumers;
                float2 x[kShares];
                float4 y[kConsumers];
                float M = -CUDART_INF_F, L = 0.f;
                auto share = [&](int w) {
                    return *reinterpret_cast<const float4 *>(shares + (w * 8 + rr) * kD +
                                                             ((4 * lane) ^ ((rr >> 1 & 3) << 3)));
                };
#pragma unroll
                for (int w = 0; w < kShares; ++w) {
                    if (w >= kConsumers && !both) continue;
                    x[w] = mls[w][rr];
                    if (w < kConsumers) y[w] = share(w);
                    M = fmaxf(M, x[w].x);
                }
                float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int w = 0; w < kShares; ++w) {
                    if (w >= kConsumers && !both) continue;
                    const float4 yw = w < kConsumers ? y[w % kConsumers] : share(w);
                    // a share none of whose keys this row sees: m = -inf, l = 0 and O = 0 (NaN
                    // scores alone also leave m at -inf, with l and O NaN)
                    const float f = x[w].x == -CUDART_INF_F ? (x[w].y == 0.f ? 0.f : 1.f)
                                                            : ex2_approx(x[w].x - M);
                    L = fmaf(x[w].y, f, L);
                    acc.x = fmaf(yw.x, f, acc.x);
                    acc.y = fmaf(yw.y, f, acc.y);
                    acc.z = fmaf(yw.z, f, acc.z);
                    acc.w = fmaf(yw.w, f, acc.w);
                }
                if (out >= 0) {
                    const size_t rec = (size_t)out * kMaxRows + r;
                    if (!GQA_IN_BOUNDS(rec, (long)2 * p.chunks * kMaxRows, p.status, kSite | 4)) continue;
                    reinterpret_cast<float4 *>(p.ws_o + rec * kD)[lane] = acc;
                    if (lane == 0) reinterpret_cast<float2 *>(p.ws_ml)[rec] = make_float2(M, L);
                } else {
                    const int t = token_of(p, r), head = head0 + r - t * p.G;
                    const long row = row0 + t;
                    if (!GQA_IN_BOUNDS(row, p.bounds.total, p.status, kSite | 5)) continue;
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
}

// Merges the partials of pairs that span several chunks.  Block c takes the pair that begins in
// chunk c and goes on in the next ones, blockIdx.y a few of its rows, W warps to a row.  Every
// warp forms the partials' weights, a lane per partial, and adds up every W-th partial, 4 dims
// per lane; the W sums meet in shared memory.  A warp's first weights are fetched along with
// the block's record, not after it.
// (One pair that all SMs share: 20 us with a warp per row; W = 4 where there are few pairs, else
// 2.  A pair of 10^6 keys next to 37 short ones: 146 us with levels and a partial at a time, 120
// with one level and four partials in flight per warp.)
constexpr int kCombineWarps = 8, kFlight = 4;
__global__ void __launch_bounds__(32 * kCombineWarps, 6) paged_decode_combine_kernel(const Params p, int W) {
    griddep_wait();
    griddep_launch_dependents();
    __shared__ float4 part[kCombineWarps][32];
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = w % W, c = blockIdx.x;
    const int r = blockIdx.y * (kCombineWarps / W) + w / W;
    // partial k: chunk c + k, its last pair for k = 0, its first for the others
    auto rec = [&](int k) { return (size_t)(2 * (c + k) + (k == 0 ? 1 : 0)) * kMaxRows + r; };
    const float2 *ml = reinterpret_cast<const float2 *>(p.ws_ml);
    float2 x = make_float2(-CUDART_INF_F, 0.f);
    const long n_rec = (long)2 * p.chunks * kMaxRows;
    if (r < kMaxRows && c + lane < p.chunks && GQA_IN_BOUNDS(rec(lane), n_rec, p.status, kSite | 6))
        x = ml[rec(lane)];   // used if the record says so
    const Joint j = p.ws_joint[c];
    // (a chunk that an expired wait left out has no record: what its place holds is checked)
    const bool on = r < j.rows && j.rows <= kMaxRows && j.parts >= 2 && j.parts <= p.chunks - c &&
                    j.g >= 0 && j.g < p.Hkv && j.row0 >= 0 &&
                    j.row0 < p.bounds.total - token_of(p, j.rows - 1);
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float M = -CUDART_INF_F, L = 0.f;
    if (on) {
        if (lane >= j.parts) x = make_float2(-CUDART_INF_F, 0.f);
        M = x.x;
        for (int i = 32 + lane; i < j.parts; i += 32)
            if (GQA_IN_BOUNDS(rec(i), n_rec, p.status, kSite | 6)) M = fmaxf(M, ml[rec(i)].x);
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, d));
        for (int i = 0; i < j.parts; i += 32) {
            if (i > 0)
                x = i + lane < j.parts && GQA_IN_BOUNDS(rec(i + lane), n_rec, p.status, kSite | 6)
                        ? ml[rec(i + lane)]
                        : make_float2(-CUDART_INF_F, 0.f);
            // a partial none of whose keys this row sees: m = -inf, l = 0 and O = 0 (NaN scores
            // alone also leave m at -inf, with l and O NaN)
            const float f = x.x == -CUDART_INF_F ? (x.y == 0.f ? 0.f : 1.f) : ex2_approx(x.x - M);
            L = fmaf(x.y, f, L);
            const int n = min(32, j.parts - i);
            for (int q0 = sub; q0 < n; q0 += kFlight * W) {
                float4 y[kFlight];   // all in flight together
#pragma unroll
                for (int k = 0; k < kFlight; ++k) {
                    const int q = q0 + k * W;
                    y[k] = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (q < n && GQA_IN_BOUNDS(rec(i + q), n_rec, p.status, kSite | 6))
                        y[k] = reinterpret_cast<const float4 *>(p.ws_o + rec(i + q) * kD)[lane];
                }
#pragma unroll
                for (int k = 0; k < kFlight; ++k) {
                    const float fk = __shfl_sync(0xffffffffu, f, min(q0 + k * W, 31));
                    if (q0 + k * W >= n) continue;   // (fk may be a NaN's 1)
                    acc.x = fmaf(y[k].x, fk, acc.x);
                    acc.y = fmaf(y[k].y, fk, acc.y);
                    acc.z = fmaf(y[k].z, fk, acc.z);
                    acc.w = fmaf(y[k].w, fk, acc.w);
                }
            }
        }
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) L += __shfl_xor_sync(0xffffffffu, L, d);
    }
    if (W > 1) {
        part[w][lane] = acc;
        __syncthreads();
        if (sub > 0) return;
        for (int i = 1; i < W; ++i) {
            const float4 y = part[w + i][lane];
            acc.x += y.x;
            acc.y += y.y;
            acc.z += y.z;
            acc.w += y.w;
        }
    }
    if (!on) return;
    const int t = token_of(p, r), h = j.g * p.G + r - t * p.G;
    const long row = j.row0 + t;
    if (!GQA_IN_BOUNDS(row, p.bounds.total, p.status, kSite | 7)) return;
    const float inv = 1.0f / L;
    reinterpret_cast<uint2 *>(p.o + row * p.o_stride + h * kD)[lane] =
        make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
    if (p.lse && lane == 0)
        p.lse[(long)h * p.bounds.total + row] = (M + __log2f(L)) * 0.69314718055994531f;
}

// Short caches: whole pairs per CTA, one after the other, and no combine.
bool whole_pairs(int max_kv) { return max_kv <= 512; }

}  // namespace

bool paged_decode_fits(int max_q, int G) { return static_cast<long>(max_q) * G <= kMaxRows; }

namespace {
// Chunks of a batch that is not run by whole pairs.  Equal runs are not equal times (the
// slowest SMs take a tenth longer), so the batch is cut into levels of smaller and smaller
// chunks; not where it is small, or has so few pairs that one would have hundreds of partials.
int n_chunks(int nseq, int max_kv, int Hkv, int max_q, int window, int unit) {
    const long pairs = (long)nseq * Hkv, all = (max_kv + unit - 1) / unit;
    // a span of window + max_q - 1 keys touches at most this many units
    const long most = window > 0 ? ((long)window + max_q - 2) / unit + 2 : all;
    return pairs >= kSMs / 4 && pairs * (most < all ? most : all) >= (long)kMinRun * kSMs
               ? kLevels * kSMs
               : kSMs;
}
}  // namespace

size_t paged_decode_workspace_bytes(int nseq, int max_kv, int Hkv, bool q8) {
    if (whole_pairs(max_kv)) return 0;
    const size_t chunks =
        n_chunks(nseq, max_kv, Hkv, 1, 0, q8 ? Ring<true>::kUnit : Ring<false>::kUnit);
    return 2 * chunks * kMaxRows * (kD + 2) * sizeof(float) + chunks * sizeof(Joint);
}

// Units are counted in 32 bits (the last level of chunks may pass the end by kSMs - 1).
bool paged_decode_counts_fit(int nseq, int max_kv, int Hkv) {
    const long pairs = (long)nseq * Hkv, most = 0x7fffffffL - kSMs;
    constexpr int unit = Ring<false>::kUnit;   // the smaller one
    return pairs <= most && pairs * ((max_kv + unit - 1) / unit) <= most;
}

namespace {
template <bool Q8>
int launch_decode_of(const PackedAttn &a, const void *scales, void *ws, int *status,
                     cudaStream_t s) {
    constexpr int kUnit = Ring<Q8>::kUnit, kSmemBytes = Ring<Q8>::kBytes;
    const gqa_paged_kv &c = *a.cache;
    Params p{};
    p.q = static_cast<const __nv_bfloat16 *>(a.q);
    p.o = static_cast<__nv_bfloat16 *>(a.o);
    p.lse = a.lse;
    p.cu = a.cu;
    p.kv_lens = c.kv_lens;
    p.pages = c.page_table;
    p.scales = static_cast<const uint8_t *>(scales);
    p.status = status;
    p.q_stride = a.q_stride;
    p.o_stride = a.o_stride;
    p.bounds = {a.total, a.max_q, a.max_kv, a.cap ? a.cap : (long)c.max_pages * c.page_size};
    p.nseq = a.nseq;
    p.Hq = a.Hq;
    p.Hkv = a.Hkv;
    p.G = a.Hq / a.Hkv;
    p.inv_g = (65536 + p.G - 1) / p.G;
    p.window = a.window;
    p.num_pages = c.num_pages;
    p.page_size = c.page_size;
    p.page_shift = c.page_size == 16 ? 4 : c.page_size == 32 ? 5 : c.page_size == 64 ? 6 : 7;
    p.max_pages = c.max_pages;
    p.scale_log2 = a.scale * 1.4426950408889634f;
    p.whole = whole_pairs(a.max_kv);
    if (!p.whole) {
        p.chunks = n_chunks(a.nseq, a.max_kv, a.Hkv, a.max_q, a.window, kUnit);
        const size_t rec = (size_t)2 * p.chunks * kMaxRows;
        p.ws_o = static_cast<float *>(ws);
        p.ws_ml = p.ws_o + rec * kD;
        p.ws_joint = reinterpret_cast<Joint *>(p.ws_ml + rec * 2);
    }
    // a page, or a unit's rows of it, per box
    const uint64_t page = c.page_size, slabs = (uint64_t)c.num_pages * c.Hkv;
    const uint32_t rows = page < kUnit ? page : kUnit;
    CUtensorMap mk, mv;
    if constexpr (Q8) {
        // {128 numbers, rows, (page, KV head), the two pools}: a map takes a stride from pool to
        // pool below 2^40, and then a page's keys and values come as one copy; else as two
        const uint64_t kp = reinterpret_cast<uint64_t>(c.k), vp = reinterpret_cast<uint64_t>(c.v);
        const uint64_t apart = kp < vp ? vp - kp : kp - vp;
        p.joint = apart < (1ull << 40);
        p.v_first = p.joint && vp < kp;
        const uint64_t dims[4] = {kD, page, slabs, p.joint ? 2u : 1u};
        const uint64_t strides[3] = {kD, page * kD, p.joint ? apart : slabs * page * kD};
        const uint32_t box[4] = {kD, rows, 1, p.joint ? 2u : 1u};
        if (!make_byte_map(&mk, p.v_first ? c.v : c.k, 4, dims, strides, box) ||
            !make_byte_map(&mv, c.v, 4, dims, strides, box))
            return GQA_ERR_CUDA;
    } else {              // {64 dims, rows, 2 halves, (page, KV head)}
        const uint64_t dims[4] = {64, page, 2, slabs}, strides[3] = {256, 128, page * 256};
        const uint32_t box[4] = {64, rows, 2, 1};
        if (!make_bf16_map(&mk, c.k, 4, dims, strides, box) ||
            !make_bf16_map(&mv, c.v, 4, dims, strides, box))
            return GQA_ERR_CUDA;
    }
    const long pairs = (long)a.nseq * a.Hkv;
    const long grid = !p.whole ? p.chunks : pairs < kSMs ? pairs : kSMs;
    const bool eight = static_cast<long>(a.max_q) * p.G <= 8;
    auto kern = eight ? paged_decode_kernel<8, Q8> : paged_decode_kernel<16, Q8>;
    if (ensure_smem_attr(reinterpret_cast<const void *>(kern), kSmemBytes) != cudaSuccess)
        return GQA_ERR_CUDA;
    if (launch_pdl(kern, dim3(static_cast<unsigned>(grid)), dim3(kThreads), kSmemBytes, s, mk, mv,
                   p) != cudaSuccess)
        return GQA_ERR_CUDA;
    if (!p.whole) {
        const int W = pairs < kSMs / 4 ? 4 : 2, rows = kCombineWarps / W;
        const dim3 grid(p.chunks, (a.max_q * p.G + rows - 1) / rows);
        if (launch_pdl(paged_decode_combine_kernel, grid, dim3(32 * kCombineWarps), 0, s, p, W) !=
            cudaSuccess)
            return GQA_ERR_CUDA;
    }
    return GQA_OK;
}
}  // namespace

int launch_paged_decode(const PackedAttn &a, const void *scales, void *ws, int *status,
                        cudaStream_t s) {
    return scales ? launch_decode_of<true>(a, scales, ws, status, s)
                  : launch_decode_of<false>(a, nullptr, ws, status, s);
}

}  // namespace gqa
