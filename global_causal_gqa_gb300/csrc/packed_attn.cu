// packed_attn.cu -- the host side that the attention kernels over packed sequences share: the
// choice between them, and their TMA tensor maps.
#include <cuda.h>
#include <cuda_runtime.h>

#include "internal.h"

namespace gqa {

namespace {

using EncodeTiledFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                   const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                   const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
    static EncodeTiledFn fn = [] {
        void *ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000,
                                             cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            ptr = nullptr;
        return reinterpret_cast<EncodeTiledFn>(ptr);
    }();
    return fn;
}

bool make_map(CUtensorMap *map, CUtensorMapDataType type, const void *base, int rank,
              const uint64_t *dims, const uint64_t *strides, const uint32_t *box) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    cuuint64_t d[5], s[4];
    cuuint32_t b[5], one[5];
    for (int i = 0; i < rank; ++i) {
        d[i] = dims[i];
        b[i] = box[i];
        one[i] = 1;
        if (i + 1 < rank) s[i] = strides[i];
    }
    return fn(map, type, rank, const_cast<void *>(base), d, s, b, one,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

bool make_bf16_map(CUtensorMap *map, const void *base, int rank, const uint64_t *dims,
                   const uint64_t *strides, const uint32_t *box) {
    return make_map(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, base, rank, dims, strides, box);
}
bool make_byte_map(CUtensorMap *map, const void *base, int rank, const uint64_t *dims,
                   const uint64_t *strides, const uint32_t *box) {
    return make_map(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, base, rank, dims, strides, box);
}

size_t paged_workspace_bytes(int nseq, int total, int max_q, int max_kv, int Hq, int Hkv) {
    return paged_decode_fits(max_q, Hq / Hkv)
               ? paged_decode_workspace_bytes(nseq, max_kv, Hkv)
               : packed_prefill_workspace_bytes(nseq, total, max_kv, Hq, Hkv);
}

bool paged_counts_fit(int nseq, int total, int max_q, int max_kv, int Hq, int Hkv) {
    return paged_decode_fits(max_q, Hq / Hkv)
               ? paged_decode_counts_fit(nseq, max_kv, Hkv)
               : packed_prefill_counts_fit(nseq, total, max_kv, Hq, Hkv);
}

int launch_packed_attn(const PackedAttn &a, void *ws, int *status, cudaStream_t s) {
    if (a.cache && paged_decode_fits(a.max_q, a.Hq / a.Hkv))
        return launch_paged_decode(a, ws, status, s);
    return launch_packed_prefill(a, ws, status, s);
}

}  // namespace gqa
