// paged_q8.cu -- attention over the 8-bit paged cache (d = 128): the choice between its ways.
//
// All keys that the call sees are expanded to bf16 pages in the workspace (paged_read.cu), and the
// bf16 kernels take them from there.
#include <cuda_runtime.h>

#include "internal.h"

namespace gqa {

bool paged_q8_counts_fit(int nseq, int total, int max_q, int max_kv, int Hq, int Hkv) {
    return paged_expand_counts_fit(nseq, max_kv, Hkv) &&
           paged_counts_fit(nseq, total, max_q, max_kv, Hq, Hkv);
}

size_t paged_q8_workspace_bytes(int nseq, int total, int max_q, int max_kv, int Hq, int Hkv) {
    return paged_expand_q8_bytes(nseq, max_kv, Hkv) +
           paged_workspace_bytes(nseq, total, max_q, max_kv, Hq, Hkv);
}

int launch_paged_q8(const PackedAttn &a, const gqa_paged_kv_q8 &c, void *ws, int *status,
                    cudaStream_t s) {
    gqa_paged_kv pages;
    if (launch_paged_expand_q8(c, a, ws, &pages, status, s) != cudaSuccess) return GQA_ERR_CUDA;
    PackedAttn b = a;
    b.cache = &pages;
    b.k = pages.k;
    b.v = pages.v;
    b.cap = (long)c.max_pages * c.page_size;
    return launch_packed_attn(
        b, static_cast<char *>(ws) + paged_expand_q8_bytes(a.nseq, a.max_kv, a.Hkv), status, s);
}

}  // namespace gqa
