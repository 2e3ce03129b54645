// Tensor maps of 16-bit arrays (host side).
#pragma once

#include "common.cuh"

#include <cuda.h>

namespace gmmb {

// cuTensorMapEncodeTiled, looked up through the runtime so that the library
// loads without a driver.
using EncodeFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                              const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                              const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeFn encode_fn() {
    static const EncodeFn fn = [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000,
                                             cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            p = nullptr;
        return (EncodeFn)p;
    }();
    return fn;
}

struct TensorMaps {
    gmm_dtype dt;
    bool ok = true;
    // [planes x] rows x cols, boxes of 64 columns x box_rows
    void make(CUtensorMap *m, const void *base, int64_t cols, int64_t rows, int64_t planes,
              int box_rows) {
        const EncodeFn fn = encode_fn();
        if (!fn) {
            ok = false;
            return;
        }
        const cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)planes};
        const cuuint64_t strides[2] = {(cuuint64_t)cols * 2, (cuuint64_t)cols * rows * 2};
        const cuuint32_t box[3] = {64, (cuuint32_t)box_rows, 1};
        const cuuint32_t one[3] = {1, 1, 1};
        ok = ok && fn(m, dt == GMM_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                        : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                      planes ? 3 : 2, const_cast<void *>(base), dims, strides, box, one,
                      CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                      CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                      CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
    }
};

}  // namespace gmmb
