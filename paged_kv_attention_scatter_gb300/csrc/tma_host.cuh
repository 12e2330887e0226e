// Host-side TMA tensor maps for bf16 rows of [rows, heads, head_dim] tensors
// (the KV pool and the q/k/v activations), encoded through the driver entry
// point fetched by the runtime, so the library needs no -lcuda.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace pkv {

inline PFN_cuTensorMapEncodeTiled_v12000 tma_encode_fn() {
    // looked up once; threads that come meanwhile wait for it
    static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        const bool found = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000,
                                                            cudaEnableDefault,
                                                            &q) == cudaSuccess &&
                           q == cudaDriverEntryPointSuccess;
        return found ? (PFN_cuTensorMapEncodeTiled_v12000)p : nullptr;
    }();
    return fn;
}

// [rows, heads, head_dim] bf16 viewed as a 3-D tensor (head_dim innermost),
// 128-byte swizzle; box = 64 elements (128 B, the swizzle width) x 1 head x
// box_rows rows.
inline bool tma_encode_rows(CUtensorMap* m, const void* base, int64_t rows, int heads,
                            int head_dim, int box_rows) {
    auto enc = tma_encode_fn();
    if (!enc) return false;
    cuuint64_t dims[3] = {(cuuint64_t)head_dim, (cuuint64_t)heads, (cuuint64_t)rows};
    cuuint64_t strides[2] = {(cuuint64_t)head_dim * 2, (cuuint64_t)heads * head_dim * 2};
    cuuint32_t box[3] = {64, 1, (cuuint32_t)box_rows};
    cuuint32_t es[3] = {1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides,
               box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace pkv
