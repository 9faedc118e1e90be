// tensor_map.cuh -- the driver's tensor-map encoder, fetched once through the runtime (no libcuda link).
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

namespace prism {

inline PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encode_fn() {
    static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
        void *ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            ptr = nullptr;
        return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
    }();
    return fn;
}

// A bf16 or fp32 tensor [B, T, heads, d] (element strides sb, st, sh; d dense) as a 4-D map {d, heads, T, B}
// with box {128 bytes, 1, rows, 1} and the 128-byte swizzle.  Where d is narrower than the box (bf16, d = 32)
// the box reaches past the tensor: loads fill zeros there, stores write nothing.
inline bool rows_map(CUtensorMap *m, const void *base, bool f32, int B, int T, int heads, int d, long long sb, long long st,
                     long long sh, int rows) {
    const auto enc = tensor_map_encode_fn();
    if (!enc) return false;
    const cuuint64_t e = f32 ? 4 : 2;
    const cuuint64_t dims[4] = {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)T, (cuuint64_t)B};
    const cuuint64_t strides[3] = {(cuuint64_t)sh * e, (cuuint64_t)st * e, (cuuint64_t)sb * e};
    const cuuint32_t box[4] = {(cuuint32_t)(128 / e), 1, (cuuint32_t)rows, 1};
    const cuuint32_t estr[4] = {1, 1, 1, 1};
    return enc(m, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(base),
               dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace prism
