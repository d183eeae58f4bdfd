// paged_q8.cu -- attention over the 8-bit paged cache (d = 128): the choice between its ways.
//
// Up to 16 rows per sequence and KV head: the streaming kernel (paged_decode.cu), which takes the
// numbers as they lie.  More: all keys that the call sees are expanded to bf16 pages in the
// workspace (paged_read.cu), and the tile kernel takes them from there.
#include <cuda_runtime.h>

#include "internal.h"

namespace gqa {

bool paged_q8_counts_fit(int nseq, int total, int max_q, int max_kv, int Hq, int Hkv) {
    return paged_decode_fits(max_q, Hq / Hkv)
               ? paged_decode_counts_fit(nseq, max_kv, Hkv)
               : paged_expand_counts_fit(nseq, max_kv, Hkv) &&
                     packed_prefill_counts_fit(nseq, total, max_kv, Hq, Hkv);
}

size_t paged_q8_workspace_bytes(int nseq, int total, int max_q, int max_kv, int Hq, int Hkv) {
    if (paged_decode_fits(max_q, Hq / Hkv))
        return paged_decode_workspace_bytes(nseq, max_kv, Hkv, true);
    return paged_expand_q8_bytes(nseq, max_kv, Hkv) +
           packed_prefill_workspace_bytes(nseq, total, max_kv, Hq, Hkv);
}

int launch_paged_q8(const PackedAttn &a, const gqa_paged_kv_q8 &c, void *ws, int *status,
                    cudaStream_t s) {
    gqa_paged_kv pages = {c.k, c.v, c.page_table, c.kv_lens, c.num_pages, c.Hkv, c.page_size, c.d,
                          c.max_pages, 0};
    PackedAttn b = a;
    b.cache = &pages;
    if (paged_decode_fits(a.max_q, a.Hq / a.Hkv))
        return launch_paged_decode(b, c.scales, ws, status, s);
    if (launch_paged_expand_q8(c, a, ws, &pages, status, s) != cudaSuccess) return GQA_ERR_CUDA;
    b.k = pages.k;
    b.v = pages.v;
    b.cap = (long)c.max_pages * c.page_size;
    return launch_packed_prefill(
        b, static_cast<char *>(ws) + paged_expand_q8_bytes(a.nseq, a.max_kv, a.Hkv), status, s);
}

}  // namespace gqa
