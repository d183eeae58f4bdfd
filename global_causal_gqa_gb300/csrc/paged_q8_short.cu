// paged_q8_short.cu -- attention of up to 8 rows per sequence over many short 8-bit caches (d = 128):
// a warp per pair of (sequence, KV head).  paged_q8.cu has the definition, paged_q8_few.cuh the
// arithmetic.
//
// A short pair's ends (queries in, the warps' shares merged, outputs) cost as much as its keys where
// eight warps share it, and the code that only the ends run misses the instruction caches: 256 chats
// of 20-450 tokens, 8 heads, 57 us.  Here a warp takes a whole pair, 32 keys at a time, issues its
// own copies, a few steps ahead and over the ends of pairs, and writes the result from its
// registers: no warp waits for another (39 us, 3.2 TB/s; 1024 such chats 99 us, 5.3 TB/s; twelve
// warps with two steps in flight each: eight with three 45 us, nine with three 44).  It needs as many
// pairs as warps to fill the GPU.
#include "paged_q8_few.cuh"

namespace gqa {
using namespace stream;
namespace {

constexpr int kWarps = 12, kDepth = 2;       // of a CTA; steps of a warp in flight
constexpr int kKeys = kShortKeys, kStepBytes = 2 * kKeys * kD;
constexpr int kQueue = 4;                    // pairs of a warp whose steps are in flight, at most
constexpr int kByteCopies = kKeys / 8;       // lanes that copy a step's 64 scale bytes
static_assert(kQueue > kDepth + 1, "a record lives from its pair's first copy to its last step");

struct Item {
    int row0, T, S, g, kb;                   // kb: its first key
};
struct WarpBars {
    uint64_t full[kDepth];
    Item item[kQueue];
};
constexpr int kScales = kWarps * kDepth * kStepBytes;
constexpr int kBars = kScales + kWarps * kDepth * 2 * kKeys;
constexpr int kClaimed = kBars + kWarps * static_cast<int>(sizeof(WarpBars));
constexpr int kSmemBytes = kClaimed + 16 + 1024;

__global__ void __launch_bounds__(32 * kWarps, 1)
    paged_q8_short_kernel(const __grid_constant__ CUtensorMap tmK,
                          const __grid_constant__ CUtensorMap tmV, const Params p) {
    griddep_wait();
    griddep_launch_dependents();
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_addr = smem_u32(smem_raw);
    uint8_t *smem = smem_raw + (((raw_addr + 1023u) & ~1023u) - raw_addr);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gq = lane >> 2, tq = lane & 3;
    uint8_t *ring = smem + warp * kDepth * kStepBytes;
    uint8_t *ring_bytes = smem + kScales + warp * kDepth * 2 * kKeys;
    WarpBars *bars = reinterpret_cast<WarpBars *>(smem + kBars) + warp;
    if (lane == 0) {
        for (int i = 0; i < kDepth; ++i) mbar_init(&bars->full[i], 1 + kByteCopies);
        fence_mbar_init();
    }
    __syncwarp();
    const int pairs = p.nseq * p.Hkv;
    int *claimed = reinterpret_cast<int *>(smem + kClaimed);   // of the CTA's pairs
    static_assert(kKeys == 32, "box_shift");
    const int box = min(p.page_size, kKeys), box_shift = min(p.page_shift, 5), boxes = kKeys >> box_shift;
    if (threadIdx.x == 0) *claimed = 0;
    __syncthreads();
    // ---- the pair whose copies are issued, an entry of its page table per lane (max_kv <= 512: at
    // most 32 pages; entries behind its last page are read but not used)
    PackedSeq s{0, 0, 0};
    int g = 0, lo = 0, kb = 0, entry = 0, queued = 0;
    int issued = 0, done = 0;                // steps
    bool more = true;
    auto issue = [&]() {
        while (kb >= s.S) {                  // the CTA's next pair that has work
            if (!more) return;
            int pair = lane == 0 ? atomicAdd(claimed, 1) : 0;
            pair = static_cast<int>(blockIdx.x + __shfl_sync(0xffffffffu, pair, 0) * gridDim.x);
            more = pair < pairs;
            if (!more) return;
            const int seq = pair / p.Hkv;
            entry = lane < p.max_pages ? __ldg(p.pages + (long)seq * p.max_pages + lane) : -1;
            s = packed_seq(p.cu, p.kv_lens, seq, p.bounds, lane == 0 ? p.status : nullptr);
            if (s.T == 0) s.S = 0;
            g = pair - seq * p.Hkv;
            lo = p.window > 0 ? max(0, s.S - s.T - p.window + 1) : 0;
            kb = lo & ~(kKeys - 1);
            if (s.S == 0) continue;
            if (lane == 0) bars->item[queued % kQueue] = {s.row0, s.T, s.S, g, kb};
            ++queued;
            // its queries on their way to L2: two 128-byte lines a row
            if (lane < 2 * s.T * p.G) {
                const int r = lane >> 1, t = token_of(p, r);
                prefetch_l2(p.q + (long)(s.row0 + t) * p.q_stride + (g * p.G + r - t * p.G) * kD +
                            64 * (lane & 1));
            }
        }
        const int slot = issued % kDepth, key = kb + lane * box;
        uint64_t *full = &bars->full[slot];
        const int page = __shfl_sync(0xffffffffu, entry, min(key >> p.page_shift, 31));
        int slab = -1;                       // zero fill: no row sees it, or not in the pool
        if (lane < boxes && key < s.S && key + box > lo) {
            if (page >= 0 && page < p.num_pages) slab = page * p.Hkv + g;
            else set_status(p.status, GQA_ERR_INVALID_ARG);
        }
        if (lane == 0) mbar_arrive_expect_tx(full, kStepBytes);
        __syncwarp();
        uint8_t *dst = ring + slot * kStepBytes;
        if (lane < boxes) {
            const int row = key & (p.page_size - 1);
            dst += lane * box * kD;
            tma_load_3d(dst, &tmK, full, 0, row, slab);
            tma_load_3d(dst + kKeys * kD, &tmV, full, 0, row, slab);
        }
        const int bkey = 8 * (lane & (kByteCopies - 1));
        const int at = __shfl_sync(0xffffffffu, slab, bkey >> box_shift);
        if (lane < kByteCopies)
            copy_async16(ring_bytes + (slot * kKeys + bkey) * 2,
                         p.scales + ((long)max(at, 0) * p.page_size + (kb + bkey & (p.page_size - 1))) * 2,
                         at >= 0 ? 16 : 0, full);
        kb += kKeys;
        ++issued;
    };
#pragma unroll 1
    for (int i = 0; i < kDepth; ++i) issue();

    const FewAt at(0, kKeys * kD);
    FewRows x;
#pragma unroll 1
    for (int taken = 0; done < issued; ++taken) {
        __syncwarp();
        const Item it = bars->item[taken % kQueue];
        const int rows = it.T * p.G;         // <= kFewRows (the host's rule on max_q)
        const FewMask mask(p, it.S, it.T);
        x.load(p, it.row0, it.g, rows);
        x.clear();
#pragma unroll 1
        for (int k = it.kb; k < it.S; k += kKeys) {
            const int slot = done % kDepth;
            if (!warp_wait(&bars->full[slot], (done / kDepth) & 1)) {
                if (lane == 0) set_timeout(p.status, kDiagPagedDecode, kRoleConsumer, 3, done);
                for (int i = done + 1; i < issued; ++i)   // nothing in flight
                    mbar_wait(&bars->full[i % kDepth], (i / kDepth) & 1);
                return;
            }
            x.attend(at, mask, ring + slot * kStepBytes,
                     reinterpret_cast<const uint16_t *>(ring_bytes) + slot * kKeys, k);
            __syncwarp();
            ++done;
            issue();
        }
        x.finish();
        // ---- outputs: two dims of row 2tq + (gq & 1) per lane, after an exchange with the next one
        const int odd = gq & 1, r = 2 * tq + odd, t = token_of(p, r), head = it.g * p.G + r - t * p.G;
        const long row = it.row0 + t;
        const bool on = r < rows && GQA_IN_BOUNDS(row, p.bounds.total, p.status, kSite | 16);
        const float inv[2] = {1.0f / x.l[0], 1.0f / x.l[1]};
        uint32_t *to = reinterpret_cast<uint32_t *>(p.o + (on ? row * p.o_stride + head * kD : 0) +
                                                    (gq & ~1));
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float a = x.o[i][2 * h] * inv[0], b = x.o[i][2 * h + 1] * inv[1];
                const float c = __shfl_xor_sync(0xffffffffu, odd ? a : b, 4);
                if (on) to[(16 * i + 8 * h) / 2] = odd ? pack_bf16x2(c, b) : pack_bf16x2(a, c);
            }
        if (p.lse && on && gq < 2)
            p.lse[(long)head * p.bounds.total + row] =
                ((odd ? x.m[1] : x.m[0]) + __log2f(odd ? x.l[1] : x.l[0])) * 0.69314718055994531f;
    }
}

}  // namespace

int stream::launch_q8_short(const CUtensorMap &mk, const CUtensorMap &mv, const Params &p,
                            cudaStream_t s) {
    if (ensure_smem_attr(reinterpret_cast<const void *>(paged_q8_short_kernel), kSmemBytes) !=
            cudaSuccess ||
        launch_pdl(paged_q8_short_kernel, dim3(kSMs), dim3(32 * kWarps), kSmemBytes, s, mk, mv, p) !=
            cudaSuccess)
        return GQA_ERR_CUDA;
    return GQA_OK;
}

}  // namespace gqa
