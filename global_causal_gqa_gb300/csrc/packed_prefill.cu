// packed_prefill.cu -- tcgen05 attention over packed prompts, and of chunks of new tokens over
// a paged cache (d = 128).
//
// Within a sequence of S keys whose last T tokens are queries ("PLaMo 3アーキテクチャ徹底解析"
// §4.2, §4.5, §5.1), for query token t at position i = S - T + t and head h of KV head g:
//   o = sum_j softmax_j(scale q . k_j) v_j  over j <= i (and i - j < W with a window).
// S = Q K^T and O += P V run as 128 x 128 tiles on the tensor cores with fp32 accumulators in
// tensor memory; the softmax is one online pass (running maximum and sum in fp32), and only
// the key tiles that some query of the block sees are loaded.
//
// Rows.  A tile's 128 rows are 128/G tokens times the G = Hq/Hkv query heads that share a KV
// head (row = token * G + head), so that a short chunk or a single token still fills rows
// with everything its keys are read for, and the keys are read once for all of them.  A work
// item is (sequence, KV head, two such tiles of consecutive tokens[, a span of the keys]): both
// tiles share every K and V load.  Q, and O on its way out, are one TMA box of {64 dims, G
// heads, 128/G tokens} per half of the head dimension.
//
// Keys come as TMA boxes of 128 rows of the packed tensor, or one box per page of a paged
// cache; a box outside the tensor (a page that is not needed, or a bad entry) is zero fill.
//
// Items are claimed with cluster launch control: the grid has an upper bound of CTAs (the
// lengths are known on the device only), the CTAs that get an SM take over the items of CTAs
// not yet launched.  The producer warp turns an item's number into its sequence, rows and
// key range (a scan over the sequences' item counts, resumed where the last one stopped,
// since the numbers only grow) and publishes it through a 4-slot ring in shared memory.
// Within a sequence the blocks with the most keys come first.
//
// Warp roles (12 warps; 96 registers for warps 0-3, 200 for the softmax warps):
//   warp 0      work claiming and TMA loads: Q of the item, K and V through a 5-slot ring.
//   warp 1      tensor-memory owner and the single MMA-issuing thread.
//   warp 2      TMA stores of O.
//   warp 3      the V guard (below).
//   warps 4-7   softmax + epilogue of tile 0, warps 8-11 of tile 1: a thread per row.
// Tensor memory: S0 [0,128), S1 [128,256), O0 [256,384), O1 [384,512); P (bf16) overwrites
// the first 64 columns of its S tile and is the PV product's operand from there; S_i(j+1) is
// issued once PV_i(j) has completed.  O is rescaled only when a row's maximum grows by more
// than 2^8 (exact: O and the sum share one reference maximum).
//
// The V guard.  A hidden key has weight 0, but 0 * NaN is NaN, so a value that a row may not
// see must not reach its product as NaN or infinity: rows past a sequence's end belong to
// another sequence or to no one.  In the tiles that straddle an edge of the mask, warp 3 looks
// at the rows that some row of the item does not see, replaces non-finite elements by 0 and
// marks the keys that others do see; the epilogue adds a marked key's non-finite elements to
// the rows that see it.  The softmax warps hand P over only when the guard is done with the
// tile, so the MMA thread, which has no time to spare, knows nothing of it.
//
// Measured (GB300, 64 heads on 8): a prompt of 16384 tokens 3.11 ms, 1410 TFLOP/s; prompts of
// 2500-8192 with a window of 2048 1.10 ms, 1245; 16 prompts of 33-2000 162 us.  A key tile's
// four products take 2048 cycles of the tensor pipe, the period is about 3300: the chain of
// one tile (score product, softmax, value product, and the next score product, which waits
// for it because P lies in S's columns), each link with its hand-over.
//
// Shared memory: Q 64 KB, ring 5 x 32 KB.  O leaves through the ring as well: after an item's
// last V tile its O tiles take a slot each, so that K and V have all five slots inside an
// item and three while O leaves.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math_constants.h>

#include <type_traits>

#include "internal.h"
#include "packed.cuh"

namespace gqa {
namespace {

constexpr int kD = 128;
constexpr int kBM = 128;
constexpr int kBN = 128;
constexpr int kSlots = 5;                     // ring: K and V tiles, O on its way out
constexpr int kBoxBytes = 128 * 128;          // 128 rows x 64 bf16 (one 128-byte swizzle span)
constexpr int kTileBytes = 2 * kBoxBytes;     // 128 rows x 128 bf16
// Where a key tile's rows lie, as its TMA boxes leave them: 8-row groups and, within a group's
// reach, the second half of the head dimension.  Packed: one box, all rows of a half, then
// the other.  Paged: a box per page, {64 dims, 8 rows, 2 halves, page / 8 groups}, so that
// the groups of successive pages lie at one distance (which a matrix descriptor needs).
template <bool PAGED>
struct KeyTile {
    static constexpr int kGroup = PAGED ? 2048 : 1024, kHalf = PAGED ? 1024 : kBoxBytes;
    static __device__ __forceinline__ int row(int r) { return (r >> 3) * kGroup + (r & 7) * 128; }
};
constexpr int kSmemQ = 0;
constexpr int kSmemRing = 2 * kTileBytes;
constexpr int kSmemBar = kSmemRing + kSlots * kTileBytes;
constexpr int kSmemBytes = kSmemBar + 1024 + 1024;  // + barriers + alignment slack
constexpr int kThreads = 384;
constexpr uint32_t kTmemCols = 512;
constexpr float kRescaleThreshold = 8.0f;     // log2 units
constexpr int kItemSlots = 4;
constexpr int kItemReaders = 11;              // MMA thread, warps 2 and 3, 8 softmax warps
constexpr int kSMs = 152;

// A work item as the producer publishes it.  n_tiles < 0: no more items.
struct ItemRec {
    int row0;       // packed row of the item's first token
    int ntok;       // its tokens
    int qpos0;      // position of the first one
    int g;          // KV head
    int kt_first;   // first key tile
    int n_tiles;
    int seq;
    int kv_row0;    // packed prompts: row of the sequence's key 0
    int split;      // span of the keys, -1: all of them (the result is final)
    int ring;       // ring position of its first load; its O tiles take those after the last
    __device__ int o_slot(int i) const { return (ring + 2 * n_tiles + i) % kSlots; }
};

struct Slot {
    ItemRec it;
    uint32_t any_bad;
    uint32_t bad[16];   // marked keys: [0, 8) after qpos0, [8, 16) from the window's lower edge
};

struct Bars {
    uint4 clc_resp;
    Slot slot[kItemSlots];
    uint64_t clc_full;
    uint64_t item_full[kItemSlots], item_free[kItemSlots];
    uint64_t q_full, q_free;
    uint64_t full[kSlots], empty[kSlots];         // K/V ring
    // A guarded V tile is on its way / clean, in turn: the ring holds three V tiles at most.
    uint64_t guard_go[4], guard[4];
    uint64_t s_full[2], p_full[2], o_done[2];     // per query tile
    uint64_t o_free[2];                           // the epilogue has read O out of TMEM
    // A ring slot is there for O / holds it, [query tile][alternate]: the ring slot of an
    // item's O is freed before that of the item after next is reached, so neither can be two
    // phases ahead of its waiter.
    uint64_t stage_go[2][2], staged[2][2];
    uint64_t mma_done;
    uint32_t tmem_base;
};
static_assert(sizeof(Bars) <= 1024, "barrier block");

struct Params {
    __nv_bfloat16 *o;
    const __nv_bfloat16 *v;        // for the marked keys of the V guard
    float *lse;
    float *ws_ml, *ws_o;           // partials of split items
    const int32_t *cu, *kv_lens, *pages;
    int *status;
    long o_stride, v_stride;
    PackedBounds bounds;
    int nseq, Hq, Hkv, G, Mt, window;    // Mt = 128 / G tokens per tile
    int num_pages, page_size, max_pages;
    int split_tiles;               // key tiles of a span; 0: items are not split
    int spans;                     // most spans of an item
    int q_box_bytes;               // bytes of one Q box
    float scale_log2;
};

// Key tiles of a block of tokens at positions [q_lo, q_hi].
__host__ __device__ __forceinline__ int first_tile(int q_lo, int window) {
    return window > 0 && q_lo - window + 1 > 0 ? (q_lo - window + 1) / kBN : 0;
}
// Most key tiles of any block of `ntok` tokens of a sequence with S keys.
__host__ __device__ __forceinline__ int most_tiles(int S, int ntok, int window) {
    const int all = (S + kBN - 1) / kBN;
    // a span of window + ntok - 1 keys touches at most this many tiles
    const long w = window > 0 ? ((long)window + ntok - 2) / kBN + 2 : all;
    return w < all ? static_cast<int>(w) : all;
}
__host__ __device__ __forceinline__ int n_spans(int tiles, int split_tiles) {
    return split_tiles > 0 ? (tiles + split_tiles - 1) / split_tiles : 1;
}

// Waits with their polling loop and their error record out of line: a dozen roles wait at
// some thirty places, and inlined the loops and records were most of the kernel's code, which
// then no longer stayed in the instruction cache between an item's parts.
__device__ __forceinline__ bool wait(uint64_t *bar, uint32_t parity) {
    return mbar_wait(bar, parity);
}
__device__ __noinline__ void expired(int *status, int role, int barrier, int at) {
    set_timeout(status, kDiagPacked, role, barrier, at);
}
// A bounded wait whose outcome every lane of the warp agrees on.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity) {
    return __all_sync(0xffffffffu, wait(bar, parity));
}

enum Role { kRoleProducer = 0, kRoleMma = 1, kRoleSoftmax = 2, kRoleAux = 3 };
constexpr int kSite = kDiagPacked << 24;   // of the debug build's checks

// The producer's walk over the sequences: one block of 32 in the lanes at a time.
struct Walk {
    int base = -32;        // first sequence of the block in the lanes
    int before = 0, here = 0;   // items before the block, in the block
    PackedSeq s{0, 0, 0};  // this lane's sequence
    int blocks = 0, spans = 1;  // its blocks of tokens, and spans of each
    int count = 0, incl = 0;    // its items, and the inclusive sum over the lanes
};

__device__ __forceinline__ void walk_to(const Params &p, Walk &w, int base) {
    const int lane = threadIdx.x & 31;
    w.before += w.here;
    w.base = base;
    const int i = base + lane;
    w.count = 0;
    if (i < p.nseq) {
        w.s = packed_seq(p.cu, p.kv_lens, i, p.bounds, p.status);
        if (w.s.T > 0) {
            const int ntok = 2 * p.Mt;
            w.blocks = (w.s.T + ntok - 1) / ntok;
            w.spans = n_spans(most_tiles(w.s.S, ntok, p.window), p.split_tiles);
            w.count = w.blocks * p.Hkv * w.spans;
        }
    }
    w.incl = w.count;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, w.incl, d);
        if (lane >= d) w.incl += x;
    }
    w.here = __shfl_sync(0xffffffffu, w.incl, 31);
}

// Item `idx` (not below the last one asked for): 1 and the item, 0 if that number has no
// work (a span past the block's keys), -1 past the last item.  Warp-collective.
__device__ __forceinline__ int find_item(const Params &p, Walk &w, int idx, ItemRec &it) {
    while (w.base < 0 || idx >= w.before + w.here) {
        if (w.base + 32 >= p.nseq) return -1;
        walk_to(p, w, w.base + 32);
    }
    const int rel = idx - w.before;
    const int lane_s = __ffs(__ballot_sync(0xffffffffu, w.incl > rel)) - 1;
    const int row0 = __shfl_sync(0xffffffffu, w.s.row0, lane_s);
    const int T = __shfl_sync(0xffffffffu, w.s.T, lane_s);
    const int S = __shfl_sync(0xffffffffu, w.s.S, lane_s);
    int r = rel - __shfl_sync(0xffffffffu, w.incl - w.count, lane_s);
    const int ntok = 2 * p.Mt, blocks = __shfl_sync(0xffffffffu, w.blocks, lane_s);
    const int spans = __shfl_sync(0xffffffffu, w.spans, lane_s);
    int split = 0;
    if (spans > 1) {
        split = r % spans;
        r /= spans;
    }
    const int back = r / p.Hkv;   // blocks from the last one
    it.g = r - back * p.Hkv;
    const int t0 = (blocks - 1 - back) * ntok;
    it.seq = w.base + lane_s;
    it.row0 = row0 + t0;
    it.ntok = min(ntok, T - t0);
    it.qpos0 = S - T + t0;
    it.kv_row0 = row0;
    it.kt_first = first_tile(it.qpos0, p.window);
    it.n_tiles = (it.qpos0 + it.ntok - 1) / kBN - it.kt_first + 1;
    it.split = -1;
    if (p.split_tiles > 0 && it.n_tiles > p.split_tiles) {
        it.split = split;
        it.kt_first += split * p.split_tiles;
        it.n_tiles = min(p.split_tiles, it.n_tiles - split * p.split_tiles);
        return it.n_tiles > 0 ? 1 : 0;
    }
    return split == 0 ? 1 : 0;
}

// Item k as a reader role sees it (false: the wait expired).
__device__ __forceinline__ bool read_item(Bars *bars, int k, ItemRec &it) {
    if (!wait(&bars->item_full[k & (kItemSlots - 1)], (k / kItemSlots) & 1)) return false;
    it = bars->slot[k & (kItemSlots - 1)].it;
    return true;
}

// What the mask makes of an item's keys: rows of V outside [lo, hi] are hidden from every
// row, those in [lo, lo_all) and (hi_all, hi] from some.
struct Edges {
    int lo, lo_all, hi_all, hi;
    __device__ Edges(const ItemRec &it, int window) {
        hi_all = it.qpos0;
        hi = it.qpos0 + it.ntok - 1;
        lo = window > 0 ? max(0, it.qpos0 - window + 1) : 0;
        lo_all = window > 0 ? max(0, hi - window + 1) : 0;
    }
    __device__ bool guarded(int n0) const { return n0 < lo_all || n0 + kBN - 1 > hi_all; }
};

__device__ __forceinline__ bool nonfinite2(uint32_t w) {   // of the two bf16 in w
    return (w & 0x7f80u) == 0x7f80u || (w & 0x7f800000u) == 0x7f800000u;
}

template <bool PAGED>
__device__ __forceinline__ const __nv_bfloat16 *value_row(const Params &p, const ItemRec &it,
                                                          int key) {
    if constexpr (!PAGED) {
        if (!GQA_IN_BOUNDS(it.kv_row0 + key, p.bounds.total, p.status, kSite | 1)) return p.v;
        return p.v + (long)(it.kv_row0 + key) * p.v_stride + it.g * kD;
    } else {
        // a marked key came from a page inside the pool (anything else is read as zeros)
        if (!GQA_IN_BOUNDS(key / p.page_size, p.max_pages, p.status, kSite | 2)) return p.v;
        const int page = p.pages[(long)it.seq * p.max_pages + key / p.page_size];
        if (!GQA_IN_BOUNDS(page, p.num_pages, p.status, kSite | 1)) return p.v;
        return p.v + (((long)page * p.Hkv + it.g) * p.page_size + key % p.page_size) * kD;
    }
}

// Adds the non-finite values of the item's marked keys to a finished row at position qpos:
// the fp32 partial at `dst` (r < 0), or row r of the bf16 tile staged there.
template <bool PAGED>
__device__ __noinline__ void add_marked(const Params &p, const Slot &slot, const ItemRec &it, int qpos,
                                        uint8_t *dst, int r) {
    for (int b = 0; b < 512; ++b) {
        if (!(slot.bad[b >> 5] >> (b & 31) & 1)) continue;
        const int key = b < 256 ? it.qpos0 + 1 + b : max(0, it.qpos0 - p.window + 1) + b - 256;
        if (key > qpos || (p.window > 0 && qpos - key >= p.window)) continue;
        const __nv_bfloat16 *v = value_row<PAGED>(p, it, key);
        for (int c = 0; c < kD; ++c) {
            const float x = __bfloat162float(v[c]);
            if (isfinite(x)) continue;
            if (r < 0) {
                reinterpret_cast<float *>(dst)[c] += x;
            } else {
                const int piece = (c >> 3 & 7) ^ (r & 7);
                __nv_bfloat16 *e = reinterpret_cast<__nv_bfloat16 *>(
                                       dst + (c >> 6) * kBoxBytes + r * 128 + piece * 16) + (c & 7);
                *e = __float2bfloat16_rn(__bfloat162float(*e) + x);
            }
        }
    }
}

template <bool PAGED>
__global__ void __launch_bounds__(kThreads, 1)
    packed_prefill_kernel(const __grid_constant__ CUtensorMap tmQ,
                          const __grid_constant__ CUtensorMap tmK,
                          const __grid_constant__ CUtensorMap tmV,
                          const __grid_constant__ CUtensorMap tmO, const Params p) {
    griddep_wait();
    extern __shared__ uint8_t smem_raw[];
    // 1024-byte alignment for the 128-byte swizzle atoms
    const uint32_t raw_addr = smem_u32(smem_raw);
    uint8_t *smem = smem_raw + (((raw_addr + 1023u) & ~1023u) - raw_addr);
    Bars *bars = reinterpret_cast<Bars *>(smem + kSmemBar);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    // the first sequences' offsets and lengths into L1 while the barriers and tensor memory are
    // set up (the producer's walk reads them first)
    if (warp == 2) {
        if (lane <= p.nseq) touch(p.cu + lane);
        if (PAGED && lane < p.nseq) touch(p.kv_lens + lane);
        if (lane == 0) {
            tma_prefetch_desc(&tmQ);
            tma_prefetch_desc(&tmK);
            tma_prefetch_desc(&tmV);
            tma_prefetch_desc(&tmO);
        }
    }
    if (threadIdx.x == 0) {
        mbar_init(&bars->clc_full, 1);
        for (int i = 0; i < kItemSlots; ++i) {
            mbar_init(&bars->item_full[i], 1);
            mbar_init(&bars->item_free[i], kItemReaders);
        }
        mbar_init(&bars->q_full, 1);
        mbar_init(&bars->q_free, 1);
        for (int s = 0; s < kSlots; ++s) {
            mbar_init(&bars->full[s], 1);
            mbar_init(&bars->empty[s], 1);
        }
        for (int i = 0; i < 2; ++i) {
            for (int a = 0; a < 4; a += 2) {
                mbar_init(&bars->guard_go[i + a], 1);
                mbar_init(&bars->guard[i + a], 32);
            }
            mbar_init(&bars->s_full[i], 1);
            mbar_init(&bars->p_full[i], 128);
            mbar_init(&bars->o_done[i], 1);
            mbar_init(&bars->o_free[i], 128);
            for (int a = 0; a < 2; ++a) {
                mbar_init(&bars->stage_go[i][a], 1);
                mbar_init(&bars->staged[i][a], 128);
            }
        }
        mbar_init(&bars->mma_done, 1);
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(&bars->tmem_base, kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bars->tmem_base;

    // Register split (launch: 384 threads x 168): 128 x 96 + 256 x 200 <= 384 x 168.
    if (warp < 4) {
        reg_dealloc<96>();
        if (warp == 0) {
            // ================= work claiming, TMA loads =================
            bool ok = true;
            int u = 0;        // ring loads issued
            int nq = 0;       // items whose Q tiles have been issued
            int claims = 0;   // responses asked for
            int gc = 0;       // guarded V tiles issued
            int ring_next = 0;   // ring position of the next item to be published
            int outs[2] = {0, 0};   // ring slots handed to O, per query tile
            Walk walk;
            auto fail = [&](int barrier, int at) {
                ok = false;
                expired(p.status, kRoleProducer, barrier, at);
            };
            auto claim = [&]() {
                if (lane == 0) {
                    mbar_arrive_expect_tx(&bars->clc_full, 16);
                    clc_try_cancel(&bars->clc_resp, &bars->clc_full);
                }
                ++claims;
            };
            // the claimed number, -1 when nothing was left
            auto claimed = [&]() {
                if (!warp_wait(&bars->clc_full, (claims - 1) & 1)) {
                    fail(3, claims);
                    return -1;
                }
                const int x = clc_decode(&bars->clc_resp);
                fence_proxy_async_smem();   // read before the next response overwrites it
                __syncwarp();
                return x;
            };
            // the next item from number `idx` on, claiming further numbers while they have no
            // work; it.n_tiles = -1 when there is none
            auto settle = [&](int idx, ItemRec &it) {
                while (true) {
                    const int r = idx < 0 ? -1 : find_item(p, walk, idx, it);
                    if (r > 0) return;
                    if (r < 0) break;
                    claim();
                    idx = claimed();
                    if (!ok) break;
                }
                it.n_tiles = -1;
            };
            // O tiles of an item that go through the ring (partials go straight out)
            auto n_out = [&](const ItemRec &it) { return it.split >= 0 ? 0 : it.ntok > p.Mt ? 2 : 1; };
            auto publish = [&](int k, const ItemRec &it) {
                Slot &s = bars->slot[k & (kItemSlots - 1)];
                if (k >= kItemSlots &&
                    !warp_wait(&bars->item_free[k & (kItemSlots - 1)], (k / kItemSlots - 1) & 1)) {
                    fail(2, k);
                    return;
                }
                if (lane < 16) s.bad[lane] = 0;
                if (lane == 0) {
                    s.it = it;
                    s.it.ring = ring_next;
                    s.any_bad = 0;
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars->item_full[k & (kItemSlots - 1)]);
                ring_next += 2 * it.n_tiles + n_out(it);
            };
            auto load_q = [&](int k, const ItemRec &it) {
                if (k >= 1 && !warp_wait(&bars->q_free, (k - 1) & 1)) {
                    fail(0, k);
                    return;
                }
                const int ntile = it.ntok > p.Mt ? 2 : 1;
                if (lane == 0) {
                    mbar_arrive_expect_tx(&bars->q_full, ntile * 2 * p.q_box_bytes);
                    for (int i = 0; i < ntile; ++i)
                        for (int h = 0; h < 2; ++h)
                            tma_load_3d(smem + kSmemQ + i * kTileBytes + h * kBoxBytes, &tmQ,
                                        &bars->q_full, 64 * h, it.g * p.G, it.row0 + i * p.Mt);
                }
                __syncwarp();
                nq = k + 1;
            };
            // pages of a key tile: lane i holds the tile's i-th one
            const int npg = PAGED ? kBN / p.page_size : 1;
            // Items in turn; k = -1 only finds the first one.  (One copy of everything: code
            // that an item's ends alone ran would have to be fetched again every time.)
            ItemRec it{}, next{};
            PageWalk pages(nullptr, 0, 0);
            for (int k = -1; ok; ++k) {
                if (k >= 0) claim();   // one item ahead
                const Edges e(it, p.window);
                int slab = 0;
                for (int l = k < 0 ? 2 : 0; ok; ++l) {
                    if (l == 2) {   // the next item, well before its first load
                        const int idx = k < 0 ? static_cast<int>(blockIdx.x) : claimed();
                        if (!ok) break;
                        settle(idx, next);
                        if (ok) publish(k + 1, next);
                    }
                    if (!ok || l >= 2 * it.n_tiles) break;
                    const int n0 = (it.kt_first + (l >> 1)) * kBN;
                    if (PAGED && !(l & 1)) {
                        const int pg = pages.get(n0 / p.page_size, npg);
                        const int key0 = n0 + lane * p.page_size;
                        slab = -1;   // no row sees it, or not in the pool: zero fill
                        if (lane < npg && key0 <= e.hi && key0 + p.page_size > e.lo) {
                            if (pg >= 0 && pg < p.num_pages) slab = pg * p.Hkv + it.g;
                            else set_status(p.status, GQA_ERR_INVALID_ARG);
                        }
                    }
                    const int st = u % kSlots;
                    if (u >= kSlots && !warp_wait(&bars->empty[st], (u / kSlots - 1) & 1)) {
                        fail(1, u);
                        break;
                    }
                    uint8_t *dst = smem + kSmemRing + st * kTileBytes;
                    const CUtensorMap *map = (l & 1) ? &tmV : &tmK;
                    if (lane == 0) mbar_arrive_expect_tx(&bars->full[st], kTileBytes);
                    __syncwarp();
                    if constexpr (PAGED) {
                        if (lane < npg)
                            tma_load_5d(dst + lane * p.page_size * kD * 2, map, &bars->full[st], 0,
                                        0, 0, 0, slab);
                    } else if (lane == 0) {
                        tma_load_4d(dst, map, &bars->full[st], 0, it.kv_row0 + n0, 0, it.g);
                    }
                    __syncwarp();
                    ++u;
                    if ((l & 1) && e.guarded(n0)) {
                        if (lane == 0) mbar_arrive(&bars->guard_go[gc & 3]);
                        ++gc;
                    }
                    // Q after the item's first K, whose slot was free earlier: Q's buffer is
                    // once the previous item's last score products are done
                    if (l == 0) load_q(k, it);
                }
                // ring slots for the item's O tiles
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    if (k < 0 || i >= n_out(it) || !ok) break;
                    const int st = u % kSlots;
                    if (u >= kSlots && !warp_wait(&bars->empty[st], (u / kSlots - 1) & 1)) {
                        fail(4, u);
                        break;
                    }
                    // no load: the phase completes with this arrival alone
                    if (lane == 0) {
                        mbar_arrive(&bars->full[st]);
                        mbar_arrive(&bars->stage_go[i][outs[i] & 1]);
                    }
                    __syncwarp();
                    ++outs[i];
                    ++u;
                }
                if (!ok || next.n_tiles < 0) break;
                it = next;
                if constexpr (PAGED) {
                    const int last = (it.qpos0 + it.ntok - 1) / p.page_size;
                    // (out of bounds: no entry is read, every key is zero fill)
                    const bool in = GQA_IN_BOUNDS(last, p.max_pages, p.status, kSite | 2);
                    pages = PageWalk(p.pages + (long)it.seq * p.max_pages, it.kt_first * npg,
                                     in ? last + 1 : 0);
                }
            }
            if (!ok) {
                // never leave the CTA with copies in flight
                for (int w = max(0, u - kSlots); w < u; ++w)
                    wait(&bars->full[w % kSlots], (w / kSlots) & 1);
                if (nq > 0) wait(&bars->q_full, (nq - 1) & 1);
                if (claims > 0) wait(&bars->clc_full, (claims - 1) & 1);
            }
            __syncwarp();
        } else if (warp == 1) {
            // ================= MMA issuer =================
            if (lane == 0) {
                const uint32_t idesc_s = idesc_bf16_f32(kBM, kBN, 0, 0);
                const uint32_t idesc_o = idesc_bf16_f32(kBM, kD, 0, 1);
                const uint32_t ring0 = smem_u32(smem + kSmemRing);
                const uint32_t q0 = smem_u32(smem + kSmemQ);
                bool ok = true;
                int u = 0;                 // ring slots consumed
                auto fail = [&](int barrier, int at) {
                    ok = false;
                    expired(p.status, kRoleMma, barrier, at);
                };
                auto take = [&](int &st) {
                    st = u % kSlots;
                    if (!wait(&bars->full[st], (u / kSlots) & 1)) {
                        fail(1, u);
                        return;
                    }
                    ++u;
                    tc_fence_after();
                };
                // Descriptors differ in their address field alone (16-byte units, low word).
                using T = KeyTile<PAGED>;
                const uint64_t qd0 = sdesc_sw128(q0, 16, 1024);
                const uint64_t kd0 = sdesc_sw128(ring0, 16, T::kGroup);
                const uint64_t vd0 = sdesc_sw128(ring0, T::kHalf, T::kGroup);
                auto issue_s = [&](int i, int st) {
                    const uint64_t qd = qd0 + i * (kTileBytes >> 4), kd = kd0 + st * (kTileBytes >> 4);
#pragma unroll
                    for (int kk = 0; kk < kD / 16; ++kk)
                        umma_ss(tmem + i * 128, qd + (((kk >> 2) * kBoxBytes + (kk & 3) * 32) >> 4),
                                kd + (((kk >> 2) * T::kHalf + (kk & 3) * 32) >> 4), idesc_s,
                                kk > 0 ? 1u : 0u);
                    umma_commit(&bars->s_full[i]);
                };
                auto issue_pv = [&](int i, int st, bool acc) {
                    const uint64_t vd = vd0 + st * (kTileBytes >> 4);
#pragma unroll
                    for (int kk = 0; kk < kBN / 16; ++kk)
                        umma_ts(tmem + 256 + i * 128, tmem + i * 128 + kk * 8,
                                vd + ((kk * 2 * T::kGroup) >> 4), idesc_o, (acc || kk > 0) ? 1u : 0u);
                    umma_commit(&bars->o_done[i]);
                };
                // an item's last score products: Q and their K go free when they are done
                auto s_done = [&](int st) {
                    umma_commit(&bars->q_free);
                    umma_commit(&bars->empty[st]);
                };
                int cpv[2] = {0, 0};       // PV products issued, per query tile (all items)
                int nepi[2] = {0, 0};      // items finished, per query tile
                for (int k = 0;; ++k) {
                    ItemRec it;
                    if (!read_item(bars, k, it)) {
                        fail(6, k);
                        break;
                    }
                    if (it.n_tiles < 0) break;
                    mbar_arrive(&bars->item_free[k & (kItemSlots - 1)]);
                    const bool two = it.ntok > p.Mt;
                    const int n = it.n_tiles;
                    u = it.ring;
                    int kst = 0, vst = 0, kprev = 0;
                    if (!wait(&bars->q_full, k & 1)) {
                        fail(0, k);
                        break;
                    }
                    // one query tile's turn: PV_i(j), then S_i(j + 1); j = -1 is the item's
                    // start.  (The index is a constant, so the counters stay in registers;
                    // every product is issued from one place, so that an item's first and
                    // last tiles run code that is at hand.)
                    auto turn = [&](auto I, int j) {
                        constexpr int i = decltype(I)::value;
                        const bool last = i == 1 || !two;   // of the key tile's turns
                        if (j >= 0) {
                            if (!wait(&bars->p_full[i], cpv[i] & 1)) return fail(3, cpv[i]);
                            // the first PV of an item overwrites O_i: the previous item's
                            // epilogue must have read it out
                            if (j == 0 && nepi[i] > 0 &&
                                !wait(&bars->o_free[i], (nepi[i] - 1) & 1))
                                return fail(4, nepi[i]);
                            tc_fence_after();
                            issue_pv(i, vst, j > 0);
                            ++cpv[i];
                        }
                        if (j + 1 < n) {
                            if (i == 0) take(kst);
                            if (!ok) return;
                            // S_i(j+1) overwrites the columns P_i(j) sits in (of the previous
                            // item, its last P_i)
                            if (cpv[i] > 0 && !wait(&bars->o_done[i], (cpv[i] - 1) & 1))
                                return fail(5, cpv[i]);
                            tc_fence_after();
                            // PV_i(j) has completed, and with it every earlier product:
                            // K(j) is free once PV_0(j) is, V(j) once the last tile's is
                            if (i == 0 && j >= 0) mbar_arrive(&bars->empty[kprev]);
                            if (last && j >= 0) mbar_arrive(&bars->empty[vst]);
                            issue_s(i, kst);
                            if (last && j + 2 == n) s_done(kst);
                        } else if (last) {
                            umma_commit(&bars->empty[vst]);
                        }
                    };
                    for (int j = -1; j < n && ok; ++j) {
                        if (j >= 0) take(vst);
                        if (ok) turn(std::integral_constant<int, 0>{}, j);
                        if (two && ok) turn(std::integral_constant<int, 1>{}, j);
                        kprev = kst;
                    }
                    if (!ok) break;
                    ++nepi[0];
                    if (two) ++nepi[1];
                }
                if (!ok) set_status(p.status, GQA_ERR_DEVICE_TIMEOUT);
                // every tcgen05 operation issued above completes before TMEM is released
                umma_commit(&bars->mma_done);
                wait(&bars->mma_done, 0);
            }
            __syncwarp();
        } else if (warp == 2) {
            // ================= O stores =================
            int done[2] = {0, 0};   // O tiles stored, per query tile
            for (int k = 0;; ++k) {
                ItemRec it;
                const bool got = read_item(bars, k, it);
                if (!__all_sync(0xffffffffu, got)) {
                    expired(p.status, kRoleAux, 6, k);
                    break;
                }
                __syncwarp();
                if (it.n_tiles < 0) break;
                if (lane == 0) mbar_arrive(&bars->item_free[k & (kItemSlots - 1)]);
                int left[2];   // partials are stored by the epilogue itself
                left[0] = it.split < 0 ? 1 : 0;
                left[1] = it.split < 0 && it.ntok > p.Mt ? 1 : 0;
                if (lane == 0) {
                    const uint64_t t0 = globaltimer_ns();
                    while (left[0] + left[1] > 0) {
                        for (int i = 0; i < 2; ++i) {
                            if (left[i] == 0 ||
                                !mbar_try_wait(&bars->staged[i][done[i] & 1], (done[i] >> 1) & 1))
                                continue;
                            // (a ragged tile has been stored row by row by the epilogue)
                            const int st = it.o_slot(i);
                            if (it.ntok >= (i + 1) * p.Mt) {
                                for (int h = 0; h < 2; ++h)
                                    tma_store_3d(&tmO, smem + kSmemRing + st * kTileBytes + h * kBoxBytes,
                                                 64 * h, it.g * p.G, it.row0 + i * p.Mt);
                                bulk_commit_group();
                                bulk_wait_read_all();
                            }
                            mbar_arrive(&bars->empty[st]);
                            ++done[i];
                            --left[i];
                        }
                        // a whole item may pass before its epilogue: the limit is generous,
                        // but it is one
                        if (globaltimer_ns() - t0 > 2 * GQA_WAIT_LIMIT_NS) {
                            expired(p.status, kRoleAux, 0, k);
                            break;
                        }
                    }
                }
                __syncwarp();
                if (__any_sync(0xffffffffu, lane == 0 && left[0] + left[1] > 0)) break;
            }
            if (lane == 0) bulk_wait_all();
            __syncwarp();
        } else {
            // ================= V guard =================
            int gc = 0;
            for (int k = 0;; ++k) {
                ItemRec it;
                const bool got = read_item(bars, k, it);
                if (!__all_sync(0xffffffffu, got)) {
                    expired(p.status, kRoleAux, 5, k);
                    break;
                }
                __syncwarp();
                if (it.n_tiles < 0) break;
                const Edges e(it, p.window);
                Slot &slot = bars->slot[k & (kItemSlots - 1)];
                bool ok = true;
                for (int j = 0; j < it.n_tiles; ++j) {
                    const int n0 = (it.kt_first + j) * kBN;
                    if (!e.guarded(n0)) continue;
                    // The producer has armed the slot for this tile, and its phase cannot
                    // move on before the guard is done (waiting on the slot alone could take
                    // an older phase of the same parity for this one).
                    const int uu = it.ring + 2 * j + 1, st = uu % kSlots;
                    if (!warp_wait(&bars->guard_go[gc & 3], (gc >> 2) & 1) ||
                        !warp_wait(&bars->full[st], (uu / kSlots) & 1)) {
                        expired(p.status, kRoleAux, 1, gc);
                        ok = false;
                        break;
                    }
                    uint8_t *tile = smem + kSmemRing + st * kTileBytes;
                    // rows [a, b) of the tile need a look: below the window's edge for some
                    // row, or past the diagonal for some row.  A lane holds one 16-byte piece
                    // of a row, two rows to a load (which piece is which does not matter).
                    const int pc = lane & 15;
                    using V = KeyTile<PAGED>;
                    uint8_t *col = tile + (pc >> 3) * V::kHalf + (pc & 7) * 16;
                    // 0 * x stays 0 unless x is infinite or NaN: one packed multiply-add per
                    // two elements, since this warp's instructions come off those of the
                    // softmax warps beside it
                    auto clean = [&](int a, int b) {
                        uint32_t z = 0;
                        for (int r0 = a + (lane >> 4); r0 < b; r0 += 16) {
                            uint4 x[8];
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                x[i] = make_uint4(0, 0, 0, 0);
                                if (r0 + 2 * i < b)
                                    x[i] = *reinterpret_cast<const uint4 *>(col + V::row(r0 + 2 * i));
                            }
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                z = hfma2_bf16(x[i].x, 0u, z);
                                z = hfma2_bf16(x[i].y, 0u, z);
                                z = hfma2_bf16(x[i].z, 0u, z);
                                z = hfma2_bf16(x[i].w, 0u, z);
                            }
                        }
                        return (z & 0x7fff7fffu) == 0;   // neither half is NaN
                    };
                    bool touched = false;
                    auto strip = [&](int a, int b) {
                        for (int r = a + (lane >> 4); r < b; r += 2) {
                            const uint4 x = *reinterpret_cast<const uint4 *>(col + V::row(r));
                            if (!(nonfinite2(x.x) || nonfinite2(x.y) || nonfinite2(x.z) ||
                                  nonfinite2(x.w)))
                                continue;
                            uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                            for (int q = 0; q < 4; ++q) {
                                if ((w[q] & 0x7f80u) == 0x7f80u) w[q] &= 0xffff0000u;
                                if ((w[q] & 0x7f800000u) == 0x7f800000u) w[q] &= 0xffffu;
                            }
                            *reinterpret_cast<uint4 *>(col + V::row(r)) =
                                make_uint4(w[0], w[1], w[2], w[3]);
                            touched = true;
                            const int key = n0 + r;
                            if (key < e.lo || key > e.hi) continue;
                            const int b0 = key > e.hi_all ? key - e.hi_all - 1 : 256 + key - e.lo;
                            atomicOr(&slot.bad[b0 >> 5], 1u << (b0 & 31));
                            atomicOr(&slot.any_bad, 1u);
                        }
                    };
                    const int below = min(kBN, max(0, e.lo_all - n0));
                    const int above = min(kBN, max(below, e.hi_all + 1 - n0));
#pragma unroll 1
                    for (int part = 0; part < 2; ++part) {
                        const int a = part ? above : 0, b = part ? kBN : below;
                        if (!clean(a, b)) strip(a, b);
                    }
                    if (touched) fence_proxy_async_smem();
                    mbar_arrive(&bars->guard[gc & 3]);
                    ++gc;
                }
                if (!ok) break;
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars->item_free[k & (kItemSlots - 1)]);
            }
        }
    } else {
        reg_alloc<200>();
        // ================= softmax / epilogue =================
        const int wg = (warp - 4) >> 2;        // query tile
        const int r = (warp & 3) * 32 + lane;  // row in tile == TMEM lane
        const int rtok = r / p.G, rhead = r - rtok * p.G;
        const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t tS = tmem + lane_off + wg * 128;
        const uint32_t tO = tmem + lane_off + 256 + wg * 128;
        int cs = 0;    // score tiles consumed (all items)
        int pvb = 0;   // PV products of the previous items
        int ns = 0;    // O tiles handed to the store warp
        int gc = 0;    // guarded V tiles (all items)
        bool ok = true;
        auto fail = [&](int barrier, int at) {
            ok = false;
            expired(p.status, kRoleSoftmax, barrier, at);
        };
        for (int k = 0; ok; ++k) {
            int n_tiles, n0, qpos, ntok;
            bool span;
            int g_lo, g_hi;   // V tiles that begin below g_lo or above g_hi are guarded
            {
                ItemRec it;
                const bool got = read_item(bars, k, it);
                if (!__all_sync(0xffffffffu, got)) {
                    fail(4, k);
                    break;
                }
                n_tiles = it.n_tiles;
                if (n_tiles < 0) break;
                ntok = it.ntok - wg * p.Mt;    // tokens of this tile
                n0 = it.kt_first * kBN;
                span = it.split >= 0;
                // rows behind the last token compute what the last token's would
                qpos = it.qpos0 + wg * p.Mt + min(rtok, min(ntok, p.Mt) - 1);
                const Edges e(it, p.window);
                g_lo = e.lo_all;
                g_hi = e.hi_all - kBN + 1;
            }
            auto free_item = [&]() {
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars->item_free[k & (kItemSlots - 1)]);
            };
            if (ntok <= 0) {
                for (int j = 0; j < n_tiles; ++j, n0 += kBN) gc += n0 < g_lo || n0 > g_hi;
                free_item();
                continue;
            }
            const bool valid = rtok < min(ntok, p.Mt);
            const bool warp_on = __any_sync(0xffffffffu, valid);
            float m = -CUDART_INF_F, l = 0.f;
            for (int j = 0; j < n_tiles; ++j, n0 += kBN) {
                if (!warp_wait(&bars->s_full[wg], cs & 1)) {
                    fail(0, cs);
                    break;
                }
                ++cs;
                // P is handed over only when the values that it meets are clean
                const bool guarded = n0 < g_lo || n0 > g_hi;
                auto hand_over = [&]() {
                    if (guarded) {
                        if (!warp_wait(&bars->guard[gc & 3], (gc >> 2) & 1)) fail(5, gc);
                        ++gc;
                    }
                    mbar_arrive(&bars->p_full[wg]);
                };
                if (!warp_on) {   // no row of this warp is stored: its P may be anything
                    hand_over();
                    if (!ok) break;
                    continue;
                }
                tc_fence_after();
                const bool full = (n0 + kBN - 1 <= qpos) &&
                                  (p.window <= 0 || n0 >= qpos - p.window + 1);
                // A tile visible in all 32 rows of the warp is taken whole, in registers.  One
                // at an edge of the mask goes in 32-column chunks, in loops that are not
                // unrolled: a chunk hidden in all rows is left out (P = 0), one hidden in
                // part is masked and written back before the second pass reads it.
                const bool whole_tile = __all_sync(0xffffffffu, full);
                float f = 1.0f, nmref = 0.f;
                bool need_o = false;
                // takes the tile's raw row maximum into account
                auto update = [&](float mraw) {
                    const float m_new = fmaxf(m, mraw * p.scale_log2);   // scale > 0
                    if (m_new > m + kRescaleThreshold) {   // false while both -inf
                        need_o = j > 0 && m != -CUDART_INF_F;
                        f = ex2_approx(m - m_new);         // 0 when m was -inf
                        l *= f;
                        m = m_new;
                    }
                    nmref = m == -CUDART_INF_F ? 0.f : -m;
                };
                // P = 2^(s * scale * log2e - m) as bf16 over the first 64 columns of the S
                // tile, 16 columns at a time (each piece lands on columns already read); the
                // row sum takes the unrounded weights
                float2 ls[4] = {{0.f, 0.f}, {0.f, 0.f}, {0.f, 0.f}, {0.f, 0.f}};
                auto weights = [&](auto &&score, uint32_t (&pk)[16]) {   // of 32 columns
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const float2 a = ffma2(make_float2(score(2 * i), score(2 * i + 1)),
                                               p.scale_log2, nmref);
                        const float e0 = ex2_approx(a.x), e1 = ex2_approx(a.y);
                        ls[i & 3] = fadd2(ls[i & 3], make_float2(e0, e1));
                        pk[i] = pack_bf16x2(e0, e1);
                    }
                };
                if (whole_tile) {
                    float x[128];
                    // four loads in flight, one wait
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        uint32_t rr[32];
                        tmem_ld32(tS + 32 * c, rr);
#pragma unroll
                        for (int i = 0; i < 32; ++i) x[32 * c + i] = __uint_as_float(rr[i]);
                    }
                    tmem_wait_ld();
                    // row maximum of the raw scores: 3-input max, 8 independent chains of 16
                    float mx8[8];
#pragma unroll
                    for (int kk = 0; kk < 8; ++kk) {
                        mx8[kk] = fmax3(x[kk], x[kk + 8], x[kk + 16]);
#pragma unroll
                        for (int tt = 3; tt < 15; tt += 2)
                            mx8[kk] = fmax3(mx8[kk], x[kk + 8 * tt], x[kk + 8 * tt + 8]);
                        mx8[kk] = fmaxf(mx8[kk], x[kk + 120]);
                    }
                    update(fmax3(fmax3(mx8[0], mx8[1], mx8[2]), fmax3(mx8[3], mx8[4], mx8[5]),
                                 fmaxf(mx8[6], mx8[7])));
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        uint32_t pk[16];
                        weights([&](int i) { return x[32 * c + i]; }, pk);
                        tmem_st16(tS + 16 * c, pk);
                    }
                } else {
                    uint32_t live = 0;   // chunks that some row of the warp sees
                    // visible columns of this row in the tile: [c_lo, c_hi)
                    const int c_hi = min(kBN, qpos - n0 + 1);
                    const int c_lo = p.window > 0 ? max(0, qpos - p.window + 1 - n0) : 0;
                    float mraw = -CUDART_INF_F;
#pragma unroll 1
                    for (int c = 0; c < 4; ++c) {
                        const int lo = c_lo - 32 * c, hi = c_hi - 32 * c;
                        if (!__any_sync(0xffffffffu, lo < 32 && hi > 0 && lo < hi)) continue;
                        live |= 1u << c;
                        uint32_t rr[32];
                        tmem_ld32(tS + 32 * c, rr);
                        tmem_wait_ld();
                        if (!__all_sync(0xffffffffu, lo <= 0 && hi >= 32)) {
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                if (i < lo || i >= hi) rr[i] = __float_as_uint(-CUDART_INF_F);
                            tmem_st32(tS + 32 * c, rr);
                        }
                        float m4[4] = {mraw, -CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F};
#pragma unroll
                        for (int i = 0; i < 32; i += 2)
                            m4[i / 2 & 3] = fmax3(m4[i / 2 & 3], __uint_as_float(rr[i]),
                                                  __uint_as_float(rr[i + 1]));
                        mraw = fmaxf(fmax3(m4[0], m4[1], m4[2]), m4[3]);
                    }
                    tmem_wait_st();
                    update(mraw);
#pragma unroll 1
                    for (int c = 0; c < 4; ++c) {
                        uint32_t pk[16];
                        if (live >> c & 1) {
                            uint32_t rr[32];
                            tmem_ld32(tS + 32 * c, rr);
                            tmem_wait_ld();
                            weights([&](int i) { return __uint_as_float(rr[i]); }, pk);
                        } else {
#pragma unroll
                            for (int i = 0; i < 16; ++i) pk[i] = 0u;
                        }
                        tmem_st16(tS + 16 * c, pk);
                    }
                }
                l += ((ls[0].x + ls[0].y) + (ls[1].x + ls[1].y)) +
                     ((ls[2].x + ls[2].y) + (ls[3].x + ls[3].y));
                if (__any_sync(0xffffffffu, need_o)) {
                    // O holds the product of tiles < j (already complete: S_i(j) was
                    // issued after PV_i(j-1) finished); rescale it in TMEM before this
                    // tile's PV is issued
                    if (!warp_wait(&bars->o_done[wg], (pvb + j - 1) & 1)) fail(1, pvb + j);
                    tc_fence_after();
                    const float fo = need_o ? f : 1.0f;
#pragma unroll 1
                    for (int c = 0; c < 4; ++c) {
                        uint32_t rr[32];
                        tmem_ld32(tO + 32 * c, rr);
                        tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            rr[i] = __float_as_uint(__uint_as_float(rr[i]) * fo);
                        tmem_st32(tO + 32 * c, rr);
                    }
                }
                tmem_wait_st();
                tc_fence_before();
                hand_over();
                if (!ok) break;
            }
            if (!ok) break;
            pvb += n_tiles;
            // ---- epilogue: O out of TMEM first (frees it for the next item)
            // (and, unless the item is a span, the ring slot that it leaves through)
            if (!warp_wait(&bars->o_done[wg], (pvb - 1) & 1)) {
                fail(2, pvb);
                break;
            }
            if (!span && !warp_wait(&bars->stage_go[wg][ns & 1], (ns >> 1) & 1)) {
                fail(3, ns);
                break;
            }
            tc_fence_after();
            float x[128];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                uint32_t rr[32];
                tmem_ld32(tO + 32 * c, rr);
#pragma unroll
                for (int i = 0; i < 32; ++i) x[32 * c + i] = __uint_as_float(rr[i]);
            }
            tmem_wait_ld();
            tc_fence_before();
            mbar_arrive(&bars->o_free[wg]);
            Slot &slot = bars->slot[k & (kItemSlots - 1)];
            const ItemRec it = slot.it;
            const int row = it.row0 + wg * p.Mt + rtok, head = it.g * p.G + rhead;
            if (PAGED && it.split >= 0) {
                // a span of the keys: the unnormalised row with its maximum (log2) and sum
                const bool in = GQA_IN_BOUNDS(it.split, p.spans, p.status, kSite | 3) &&
                                GQA_IN_BOUNDS(valid ? row : 0, p.bounds.total, p.status, kSite | 4);
                if (valid && in) {
                    const size_t rec = (size_t)it.split * p.bounds.total * p.Hq + (size_t)row * p.Hq + head;
                    float4 *dst = reinterpret_cast<float4 *>(p.ws_o + rec * kD);
#pragma unroll
                    for (int c = 0; c < 32; ++c)
                        dst[c] = make_float4(x[4 * c], x[4 * c + 1], x[4 * c + 2], x[4 * c + 3]);
                    p.ws_ml[2 * rec] = m;
                    p.ws_ml[2 * rec + 1] = l;
                    if (slot.any_bad)
                        add_marked<PAGED>(p, slot, it, qpos, reinterpret_cast<uint8_t *>(dst), -1);
                }
            } else {
                // (l = 0: every visible score is -inf, and 0 * inf gives the NaN of the definition,
                // as the merge of a split item's spans does)
                const float inv_l = 1.0f / l;
                const bool whole = ntok >= p.Mt;   // the tile's tokens are all there
                // through a ring slot, as two halves of the columns like a Q tile
                uint8_t *stage = smem + kSmemRing + it.o_slot(wg) * kTileBytes;
#pragma unroll
                for (int c = 0; c < 16; ++c) {
                    const float *y = x + 8 * c;
                    *reinterpret_cast<uint4 *>(stage + (c >> 3) * kBoxBytes + r * 128 +
                                               (((c & 7) ^ (r & 7)) << 4)) =
                        make_uint4(pack_bf16x2(y[0] * inv_l, y[1] * inv_l),
                                   pack_bf16x2(y[2] * inv_l, y[3] * inv_l),
                                   pack_bf16x2(y[4] * inv_l, y[5] * inv_l),
                                   pack_bf16x2(y[6] * inv_l, y[7] * inv_l));
                }
                if (valid && slot.any_bad) add_marked<PAGED>(p, slot, it, qpos, stage, r);
                if (!whole) {
                    // a ragged tile: the warp writes the rows that are there, two at a time
                    __syncwarp();
                    const int r0 = (warp & 3) * 32, c = lane & 15;
                    const int rows = min(32, min(ntok, p.Mt) * p.G - r0);
                    const long mine = (long)row * p.o_stride + head * kD;   // this thread's row
#pragma unroll 4
                    for (int i = 0; i < rows; i += 2) {
                        const int ii = i + (lane >> 4), rr = r0 + ii;
                        const long at = __shfl_sync(0xffffffffu, mine, ii);
                        if (ii >= rows || !GQA_IN_BOUNDS(at / p.o_stride, p.bounds.total, p.status, kSite | 4))
                            continue;
                        const uint4 y = *reinterpret_cast<const uint4 *>(
                            stage + (c >> 3) * kBoxBytes + rr * 128 + (((c & 7) ^ (rr & 7)) << 4));
                        *reinterpret_cast<uint4 *>(p.o + at + 8 * c) = y;
                    }
                }
                // A whole tile is read by the store warp's TMA next.  A ragged one is not, but the
                // slot then takes a K or V tile by TMA, which a barrier alone does not order
                // after this thread's stores.
                fence_proxy_async_smem();
                mbar_arrive(&bars->staged[wg][ns & 1]);
                ++ns;
                if (valid && p.lse && GQA_IN_BOUNDS(row, p.bounds.total, p.status, kSite | 4))
                    p.lse[(size_t)head * p.bounds.total + row] =
                        (m + __log2f(l)) * 0.69314718055994531f;
            }
            free_item();
        }
        if (!ok) set_status(p.status, GQA_ERR_DEVICE_TIMEOUT);
    }

    // only now: a CTA of the next kernel that came earlier would sit on an SM that this grid's
    // unclaimed CTAs need (162 us for the 16 prompts in a row became 176)
    griddep_launch_dependents();
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

// Merges the spans of split items: one warp per (token, query head), the spans' maxima and
// sums in the lanes, 4 dims of the output per lane.
constexpr int kMostSpans = 64;
constexpr int kCombineWarps = 8, kFlight = 4;   // partials in flight per warp
__global__ void __launch_bounds__(32 * kCombineWarps) packed_combine_kernel(const Params p) {
    griddep_wait();
    griddep_launch_dependents();
    const int row = blockIdx.x, h = blockIdx.y * kCombineWarps + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    const int i = packed_row_seq(p.cu, p.nseq, row);
    if (i >= p.nseq || h >= p.Hq) return;
    const PackedSeq s = packed_seq(p.cu, p.kv_lens, i, p.bounds, nullptr);
    if (row < s.row0 || row >= s.row0 + s.T) return;
    // the block of tokens that the row was computed in
    const int ntok = 2 * p.Mt, t0 = (row - s.row0) / ntok * ntok;
    const int q_lo = s.S - s.T + t0, q_hi = q_lo + min(ntok, s.T - t0) - 1;
    const int spans = n_spans(q_hi / kBN - first_tile(q_lo, p.window) + 1, p.split_tiles);
    if (spans <= 1) return;   // written by the attention kernel itself
    const size_t step = (size_t)p.bounds.total * p.Hq, rec = (size_t)row * p.Hq + h;
    const float2 *ml = reinterpret_cast<const float2 *>(p.ws_ml);
    float2 x[kMostSpans / 32];
    float M = -CUDART_INF_F, L = 0.f;
#pragma unroll
    for (int t = 0; t < kMostSpans / 32; ++t) {
        x[t] = make_float2(-CUDART_INF_F, 0.f);
        if (32 * t + lane < spans && GQA_IN_BOUNDS(32 * t + lane, p.spans, p.status, kSite | 5))
            x[t] = ml[rec + (32 * t + lane) * step];
        M = fmaxf(M, x[t].x);
    }
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, d));
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int t = 0; t < kMostSpans / 32; ++t) {
        // a span with no key that the row sees: m = -inf, l = 0 and O = 0 (NaN scores alone
        // also leave m at -inf, with l and O NaN)
        const float f = x[t].x == -CUDART_INF_F ? (x[t].y == 0.f ? 0.f : 1.f) : ex2_approx(x[t].x - M);
        L = fmaf(x[t].y, f, L);
        const int n = min(32, spans - 32 * t);
        for (int k0 = 0; k0 < n; k0 += kFlight) {
            float4 o[kFlight];   // all in flight together
#pragma unroll
            for (int k = 0; k < kFlight; ++k) {
                o[k] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (k0 + k < n && GQA_IN_BOUNDS(32 * t + k0 + k, p.spans, p.status, kSite | 5))
                    o[k] = reinterpret_cast<const float4 *>(p.ws_o + (rec + (32 * t + k0 + k) * step) * kD)[lane];
            }
#pragma unroll
            for (int k = 0; k < kFlight; ++k) {
                const float fk = __shfl_sync(0xffffffffu, f, min(k0 + k, 31));
                if (k0 + k >= n) continue;   // (fk may be a NaN's 1)
                acc.x = fmaf(o[k].x, fk, acc.x);
                acc.y = fmaf(o[k].y, fk, acc.y);
                acc.z = fmaf(o[k].z, fk, acc.z);
                acc.w = fmaf(o[k].w, fk, acc.w);
            }
        }
    }
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) L += __shfl_xor_sync(0xffffffffu, L, d);
    const float r = 1.0f / L;
    reinterpret_cast<uint2 *>(p.o + (size_t)row * p.o_stride + h * kD)[lane] =
        make_uint2(pack_bf16x2(acc.x * r, acc.y * r), pack_bf16x2(acc.z * r, acc.w * r));
    if (p.lse && lane == 0)
        p.lse[(size_t)h * p.bounds.total + row] = (M + __log2f(L)) * 0.69314718055994531f;
}

// How many key tiles a span of a split item has (0: items stay whole), and the most spans.
// The number of spans n is the one that an estimate of the time likes best.  An item of
// tiles / n key tiles takes kTileUs each and a fixed part, more where it writes a partial.
// One sequence: all items are about as long, and go in rounds over the SMs.  Several: items
// are shorter than the host's bound on the keys (kMean of it, taken together) and the longest
// may come last.  Partials cost their bytes and the combine kernel.
// (Measured, 64 heads on 8: 512 tokens over 8192 keys 116 us whole, 137 / 151 / 173 in 2 / 4 / 8
// spans; 128 over 32000: 227 / 124 / 136 us in 2 / 4 / 8; 12 chunks of 1-300 over 1000-12000:
// 272 whole, 203 / 169 / 186.)
struct SpanRule {
    int split_tiles, spans;
};
constexpr double kTileUs = 1.75, kItemUs = 5.0, kPartialUs = 8.0, kCombineUs = 4.0, kBytesPerUs = 1e7;
constexpr double kMean = 0.6;
int best_spans(int nseq, int total, int tiles, int Hq, int Hkv, int most) {
    const int ntok = 2 * (kBM / (Hq / Hkv));
    // every sequence has a block at least, and ends in half a block on average
    const long some = nseq < total ? nseq : total, on_average = total / ntok + some / 2 + 1;
    const long blocks = nseq == 1 ? (total + ntok - 1) / ntok : on_average > some ? on_average : some;
    const double items = static_cast<double>(blocks) * Hkv;
    int best = 1;
    double least = 0;
    for (int n = 1; n <= most && (n == 1 || tiles / n >= 4); ++n) {
        const double fixed = n > 1 ? kPartialUs : kItemUs;
        const double longest = kTileUs * ((tiles + n - 1) / n) + fixed;
        double us = longest;
        if (nseq == 1)
            us *= static_cast<long>((items * n + kSMs - 1) / kSMs);
        else if (items * n > kSMs)
            us += items * (kMean * kTileUs * tiles + n * fixed) / kSMs;
        if (n > 1) us += kCombineUs + 2.0 * n * total * Hq * (kD + 2) * sizeof(float) / kBytesPerUs;
        if (n == 1 || us < least) {
            best = n;
            least = us;
        }
    }
    return best;
}
// `window` only ever lowers the number of spans: the workspace is sized without it.
SpanRule span_rule(int nseq, int total, int max_kv, int Hq, int Hkv, int window) {
    const int ntok = 2 * (kBM / (Hq / Hkv));
    int n = best_spans(nseq, total, most_tiles(max_kv, ntok, 0), Hq, Hkv, kMostSpans);
    const int tiles = most_tiles(max_kv, ntok, window);
    if (window > 0) n = best_spans(nseq, total, tiles, Hq, Hkv, n);
    if (n <= 1) return {0, 1};
    const int per = (tiles + n - 1) / n;
    return {per, n_spans(tiles, per)};
}

// The numbers of a grid: an upper bound on the items (a sequence adds at most one block that is
// not full), and one more: the CTA that gets it walks past the last sequence, so that all of them
// have been looked over (one that passes the rows has no item that would lead to it).  -1: more
// than 32 bits hold.
long n_numbers(int nseq, int total, int Hq, int Hkv, int spans) {
    const int ntok = 2 * (kBM / (Hq / Hkv));
    const long blocks = (long)total / ntok + (nseq < total ? nseq : total), most = 0x7ffffffeL;
    if (blocks > most || blocks * Hkv > most || blocks * Hkv * spans > most) return -1;
    return blocks * Hkv * spans + 1;
}

}  // namespace

size_t packed_prefill_workspace_bytes(int nseq, int total, int max_kv, int Hq, int Hkv) {
    const int tiles = most_tiles(max_kv, 2 * (kBM / (Hq / Hkv)), 0);
    const int n = best_spans(nseq, total, tiles, Hq, Hkv, kMostSpans);
    return n <= 1 ? 0 : (size_t)n * total * Hq * (kD + 2) * sizeof(float);
}

bool packed_prefill_counts_fit(int nseq, int total, int max_kv, int Hq, int Hkv) {
    // packed prompts have one span; else the rule is asked only where the most would not do, and
    // without a window, which only lowers the number of spans
    if (max_kv == 0) return n_numbers(nseq, total, Hq, Hkv, 1) > 0;
    return n_numbers(nseq, total, Hq, Hkv, kMostSpans) > 0 ||
           n_numbers(nseq, total, Hq, Hkv, span_rule(nseq, total, max_kv, Hq, Hkv, 0).spans) > 0;
}

int launch_packed_prefill(const PackedAttn &a, void *ws, int *status, cudaStream_t s) {
    const bool paged = a.cache != nullptr;
    Params p{};
    p.o = static_cast<__nv_bfloat16 *>(a.o);
    p.v = static_cast<const __nv_bfloat16 *>(a.v);
    p.lse = a.lse;
    p.cu = a.cu;
    p.status = status;
    p.o_stride = a.o_stride;
    p.v_stride = a.v_stride;
    p.nseq = a.nseq;
    p.Hq = a.Hq;
    p.Hkv = a.Hkv;
    p.G = a.Hq / a.Hkv;
    p.Mt = kBM / p.G;
    p.window = a.window;
    p.scale_log2 = a.scale * 1.4426950408889634f;
    p.q_box_bytes = 64 * 2 * p.G * p.Mt;
    p.bounds = {a.total, a.max_q, a.max_kv, 0x7fffffffL};
    int spans = 1;
    CUtensorMap mq, mk, mv, mo;
    {
        // {128 dims, query heads, tokens}: half the dims of G heads of Mt tokens per box
        const uint64_t dims[3] = {kD, (uint64_t)a.Hq, (uint64_t)a.total};
        const uint64_t qs[2] = {kD * 2, (uint64_t)a.q_stride * 2};
        const uint64_t os[2] = {kD * 2, (uint64_t)a.o_stride * 2};
        const uint32_t box[3] = {64, (uint32_t)p.G, (uint32_t)p.Mt};
        if (!make_bf16_map(&mq, a.q, 3, dims, qs, box) || !make_bf16_map(&mo, a.o, 3, dims, os, box))
            return GQA_ERR_CUDA;
    }
    if (paged) {
        const gqa_paged_kv &c = *a.cache;
        p.kv_lens = c.kv_lens;
        p.pages = c.page_table;
        p.num_pages = c.num_pages;
        p.page_size = c.page_size;
        p.max_pages = c.max_pages;
        p.bounds.cap = a.cap ? a.cap : (long)c.max_pages * c.page_size;
        const SpanRule r = span_rule(a.nseq, a.total, a.max_kv, a.Hq, a.Hkv, a.window);
        p.split_tiles = r.split_tiles;
        p.spans = spans = r.spans;
        if (spans > 1) {
            // the outputs come first (16-byte aligned), then the maxima and sums
            p.ws_o = static_cast<float *>(ws);
            p.ws_ml = p.ws_o + (size_t)spans * a.total * a.Hq * kD;
        }
        // {64 dims, 8 rows, 2 halves, groups of 8 rows, (page, KV head)}, a page per box
        const uint64_t page = c.page_size;
        const uint64_t dims[5] = {64, 8, 2, page / 8, (uint64_t)c.num_pages * c.Hkv};
        const uint64_t strides[4] = {256, 128, 2048, page * 256};
        const uint32_t box[5] = {64, 8, 2, (uint32_t)(page / 8), 1};
        if (!make_bf16_map(&mk, c.k, 5, dims, strides, box) ||
            !make_bf16_map(&mv, c.v, 5, dims, strides, box))
            return GQA_ERR_CUDA;
    } else {
        // {64 dims, rows, 2 halves, KV heads}, 128 rows per box
        const uint64_t dims[4] = {64, (uint64_t)a.total, 2, (uint64_t)a.Hkv};
        const uint64_t ks[3] = {(uint64_t)a.k_stride * 2, 128, 256};
        const uint64_t vs[3] = {(uint64_t)a.v_stride * 2, 128, 256};
        const uint32_t box[4] = {64, kBN, 2, 1};
        if (!make_bf16_map(&mk, a.k, 4, dims, ks, box) || !make_bf16_map(&mv, a.v, 4, dims, vs, box))
            return GQA_ERR_CUDA;
    }
    auto kern = paged ? packed_prefill_kernel<true> : packed_prefill_kernel<false>;
    if (ensure_smem_attr(reinterpret_cast<const void *>(kern), kSmemBytes) != cudaSuccess)
        return GQA_ERR_CUDA;
    // (the entry points have seen that it fits 32 bits)
    const long grid = n_numbers(a.nseq, a.total, a.Hq, a.Hkv, spans);
    if (launch_pdl(kern, dim3(static_cast<unsigned>(grid)), dim3(kThreads), kSmemBytes, s, mq, mk,
                   mv, mo, p) != cudaSuccess)
        return GQA_ERR_CUDA;
    if (spans > 1 &&
        launch_pdl(packed_combine_kernel,
                   dim3(a.total, (a.Hq + kCombineWarps - 1) / kCombineWarps),
                   dim3(32 * kCombineWarps), 0, s, p) != cudaSuccess)
        return GQA_ERR_CUDA;
    return GQA_OK;
}

}  // namespace gqa
