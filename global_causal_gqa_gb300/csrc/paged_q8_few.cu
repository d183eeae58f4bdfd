// paged_q8_few.cu -- attention of up to 8 rows (tokens x heads of a KV group) per sequence over the
// 8-bit paged cache (d = 128): decode steps.  paged_q8.cu has the definition and takes more rows.
//
// Cut and fed as the bf16 kernel (paged_decode.cu; paged_stream.cuh), in stages of 128 keys, of
// which a warp takes 32.  S^T = Y Q^T and O^T += Z^T P^T are m16n8k16 f16 MMAs with the keys, and
// then the dims, as M and the rows as N.  The e4m3 numbers become f16 exactly, two per instruction
// in registers (mma.sync's own 8-bit form takes longer than the 16-bit one: 33 cycles against 22 in
// a chain).  A query row is brought to f16 by a power of two of its own; P = 2^(x - m + b - mo + 9)
// with b its value's exponent, so a value's power of two is in its weight and the numbers multiply as
// they are.  l sums the weights relative to 2^m, O relative to 2^(m + mo - 9), mo the largest x - m + b
// seen: either range alone may be far from the other's.  Both references move when something exceeds them
// by 2^6; P lies between 2^15 and 2^-24, 2^-33 of the reference.
//
// A stage takes a warp 1800 cycles, the copies of a stage 1365: with few pairs per CTA both groups
// of four warps take a pair's stages in turn (BOTH; 32 caches of 8k-64k tokens 529 -> 401 us, 6.8
// TB/s, which is HBM), else the pairs, so that one's ends pass while the other streams (64
// windows of 2048: 57 us in pages of 64, 4.6 TB/s, of them 5 of start and 5 of the merge; 69 in pages
// of 16, whose 16 copies a stage the producer issues one after the other).  The
// tcgen05 kernel of paged_q8.cu takes 425 us: it holds a stage 2.5 us, through a score product, a
// softmax and a value product in different warps, where this one holds it 1 us.
#include "paged_q8_few.cuh"

namespace gqa {
using namespace stream;
namespace {

// BOTH: the groups take a pair's stages in turn.
template <bool BOTH>
struct FewStream {
    static constexpr bool kQ8 = true;
    static constexpr int kUnit = 128, kStages = 5, kSegSlots = 4, kTeams = 2, kEnds = BOTH ? 1 : 2;
    static constexpr int kProducer = kTeams * kConsumers, kThreads = 32 * (kProducer + 1);
    static constexpr int kEndCost = 4;
    // the barrier of a stage's load: its group's, so that a group sees every phase of its own
    __device__ static int full_of(int turn, int j) { return (BOTH ? j : turn) % kTeams; }
};

constexpr int kRows = kFewRows, kGroups = 2, kUnit = 128, kStages = 5, kSegSlots = 4;
constexpr int kScales = kStages * kStageBytes;      // two bytes per key of a stage
constexpr int kXchg = kScales + kStages * 2 * kUnit;
constexpr int kBar = kXchg + kGroups * kConsumers * kRows * kD * 4;
constexpr int kSmemBytes = kBar + 1536 + 1024;

struct Bars : StreamBars {
    uint64_t merge[kGroups];         // the warps of a group, or of both, meet
    float2 ml[kGroups][kConsumers][kRows];
};
static_assert(sizeof(Bars) <= 1536, "barrier block");

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
    const int group = warp / kConsumers, cw = warp % kConsumers;
    float *xchg = reinterpret_cast<float *>(smem + kXchg) + group * kConsumers * kRows * kD;
    const int part = 32 * cw;                 // first of this warp's keys in a stage
    const FewAt at(part, kTileBytes);
    FewRows x;
    int meets = 0;
    auto meet = [&]() {
        __syncwarp();
        uint64_t *bar = &bars->merge[BOTH ? 0 : group];
        if (lane == 0) mbar_arrive(bar);
        if (quick_wait(bar, meets++ & 1)) return true;
        expired(p.status, 2, meets);
        return false;
    };
    // Segment k and its queries.
    Segment sg;
    auto next_segment = [&](int k) {
        const int slot = k % kSegSlots;
        if (!quick_wait(&bars->seg_full[slot], (k / kSegSlots) & 1)) {
            expired(p.status, 0, k);
            return false;
        }
        sg = bars->seg[slot];
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->seg_free[slot]);
        // (rows <= kRows: the host's rule on max_q)
        x.load(p, sg.row0, sg.g, sg.stages < 0 ? 0 : sg.T * p.G);
        return true;
    };
    const int first = BOTH ? 0 : group, next = BOTH ? 1 : kGroups;
    if (!next_segment(first)) return;
    uint32_t phases = 0;   // of the group's full barriers, a bit each
    for (int k = first; sg.stages >= 0; k += next) {
        const int rows = sg.T * p.G;
        const FewMask mask(p, sg.S, sg.T);
        x.clear();
        for (int j = BOTH ? group : 0; j < sg.stages; j += BOTH ? kGroups : 1) {
            const int u = sg.u0 + j, st = u % kStages;
            if (!quick_wait(&bars->full[group][st], phases >> st & 1)) {
                expired(p.status, 1, u);
                return;
            }
            phases ^= 1u << st;
            const int kb = (sg.unit0 + j) * kUnit + part;   // this warp's 32 keys
            if (kb < sg.S && kb + 31 >= mask.lo)
                x.attend(at, mask, smem + st * kStageBytes,
                         reinterpret_cast<const uint16_t *>(smem + kScales) + st * kUnit + part, kb);
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars->empty[st]);
        }
        x.finish();
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
            if (gq == 0) bars->ml[group][cw][r] = make_float2(x.m[c], x.l[c]);
            float *mine = xchg + (cw * kRows + r) * kD;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                mine[(16 * i + gq) ^ (tq << 3)] = x.o[i][c];
                mine[(16 * i + 8 + gq) ^ (tq << 3)] = x.o[i][2 + c];
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
                const float2 s = mls[w][r];
                const float4 y = *reinterpret_cast<const float4 *>(
                    shares + (w * kRows + r) * kD + ((4 * lane) ^ ((r >> 1 & 3) << 3)));
                // a share none of whose keys this row sees: m = -inf, l = 0 and O = 0 (NaN scores
                // alone also leave m at -inf, with l and O NaN)
                const float f =
                    s.x == -CUDART_INF_F ? (s.y == 0.f ? 0.f : 1.f) : ex2_approx(s.x - M);
                L = fmaf(s.y, f, L);
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
