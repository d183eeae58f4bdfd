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

}  // namespace

bool make_rows_map(CUtensorMap *map, const void *base, long n1, long s1, long n2, long s2, int b1,
                   int b2) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)128, (cuuint64_t)n1, (cuuint64_t)n2};
    const cuuint64_t strides[2] = {(cuuint64_t)s1 * 2, (cuuint64_t)s2 * 2};
    const cuuint32_t box[3] = {64, (cuuint32_t)b1, (cuuint32_t)b2};
    const cuuint32_t estr[3] = {1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides,
              box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool make_page_map(CUtensorMap *map, const void *base, long page, long slabs, int rows) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[4] = {64, (cuuint64_t)page, 2, (cuuint64_t)slabs};
    const cuuint64_t strides[3] = {256, 128, (cuuint64_t)page * 256};
    const cuuint32_t box[4] = {64, (cuuint32_t)rows, 2, 1};
    const cuuint32_t estr[4] = {1, 1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(base), dims, strides,
              box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

size_t paged_workspace_bytes(int, int total, int max_q, int max_kv, int Hq, int Hkv, int) {
    return paged_decode_fits(max_q, Hq / Hkv)
               ? paged_decode_workspace_bytes(max_kv)
               : packed_prefill_workspace_bytes(total, max_kv, Hq, Hkv);
}

int launch_packed_attn(const PackedAttn &a, void *ws, int *status, cudaStream_t s) {
    if (a.cache && paged_decode_fits(a.max_q, a.Hq / a.Hkv))
        return launch_paged_decode(a, ws, status, s);
    return launch_packed_prefill(a, ws, status, s);
}

}  // namespace gqa
