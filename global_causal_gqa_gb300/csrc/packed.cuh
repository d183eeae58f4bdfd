// packed.cuh -- what the kernels over packed sequences and the paged cache share: a
// sequence's rows and lengths, checked, and the sequence that owns a packed row.
#pragma once
#include <cstdint>

#include "gqa_attn.h"
#include "ptx.cuh"

namespace gqa {

// A sequence of a packed batch: its first row, its T new tokens and its S keys.  T = 0 where
// there is nothing to do for it.
struct PackedSeq {
    int row0, T, S;
};

// Bounds on a batch's sequences: rows of the packed tensors, new tokens and keys of one
// sequence (the host's bounds), and the keys that its pages can hold.
struct PackedBounds {
    int total, max_q, max_kv;
    long cap;
};

// A sequence of rows r0 .. r1 - 1 and `keys` keys.  Numbers that contradict one another or exceed a
// bound give T = 0 and are recorded in `status` (nullable).
__device__ __forceinline__ PackedSeq check_seq(int r0, int r1, int keys, const PackedBounds &b,
                                               int *status) {
    PackedSeq s;
    s.row0 = r0;
    s.T = r1 - r0;
    if (r0 < 0 || r1 < r0 || r1 > b.total) {
        s.T = s.S = 0;
        set_status(status, GQA_ERR_INVALID_ARG);
        return s;
    }
    s.S = keys;
    if (s.T > 0) {
        if (s.S < s.T) {
            s.T = 0;
            set_status(status, GQA_ERR_INVALID_ARG);
        } else if (s.T > b.max_q || s.S > b.max_kv || s.S > b.cap) {
            s.T = 0;
            set_status(status, GQA_ERR_CAPACITY);
        }
    }
    return s;
}

// Sequence i.  kv_lens == nullptr: packed prompts, S = T.
__device__ __forceinline__ PackedSeq packed_seq(const int32_t *cu, const int32_t *kv_lens, int i,
                                                const PackedBounds &b, int *status) {
    const int r0 = __ldg(cu + i), r1 = __ldg(cu + i + 1);
    const int keys = kv_lens ? __ldg(kv_lens + i) : r1 - r0;   // in flight with the offsets
    return check_seq(r0, r1, keys, b, status);
}

// The sequence whose rows include packed row `row` (warp-collective: every lane gets it):
// the number of entries cu[1 .. nseq] that are <= row, found by 32 probes at a time (two
// loads one after the other for up to 1024 sequences).  The caller checks the row against
// that sequence's bounds, which also rejects rows behind the last sequence (the result is
// then nseq) and offsets that are not sorted.
__device__ __forceinline__ int packed_row_seq(const int32_t *cu, int nseq, int row) {
    const int lane = threadIdx.x & 31;
    int n = 0, len = nseq;   // entries known to be <= row; those after them in question
    while (len > 32) {
        const int step = (len + 31) / 32, i = step * (lane + 1);
        const int k = __popc(__ballot_sync(0xffffffffu, i <= len && __ldg(cu + n + i) <= row));
        n += k * step;
        len = min(step - 1, len - k * step);
    }
    return n + __popc(__ballot_sync(0xffffffffu, lane < len && __ldg(cu + n + 1 + lane) <= row));
}

// Starts a load of *p into L1 without waiting for it.
__device__ __forceinline__ void touch(const int32_t *p) {
    asm volatile("{\n\t.reg .b32 t;\n\tld.global.nc.b32 t, [%0];\n\t}" ::"l"(p));
}

// A producer warp's walk over the page-table entries of one sequence, in order: the lanes
// hold 32 entries and the 32 after them, so an entry has been on its way for at least 32
// pages' worth of loads when it is needed.
struct PageWalk {
    const int32_t *row;   // the sequence's entries
    int end;              // entries from here on are not needed (and not read)
    int base, cur, next;

    PageWalk() = default;
    __device__ __forceinline__ int fetch(int i) const { return i < end ? __ldg(row + i) : -1; }
    __device__ __forceinline__ PageWalk(const int32_t *r, int first, int e) : row(r), end(e) {
        const int lane = threadIdx.x & 31;
        base = first & ~31;
        cur = fetch(base + lane);
        next = fetch(base + 32 + lane);
    }
    // The entry of page `first` + i for lane i < n (n a power of two up to 32 that divides
    // `first`; warp-collective); `first` does not decrease.
    __device__ __forceinline__ int get(int first, int n) {
        const int lane = threadIdx.x & 31;
        while (first >= base + 32) {
            base += 32;
            cur = next;
            next = fetch(base + 32 + lane);
        }
        return __shfl_sync(0xffffffffu, cur, first - base + (lane & (n - 1)));
    }
};

}  // namespace gqa
