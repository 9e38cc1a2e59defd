// Host: tensor maps of row-major matrices for TMA tile loads.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

// cuTensorMapEncodeTiled, looked up through the runtime so the library does
// not link the driver library directly (it must load on hosts without a GPU).
typedef CUresult (*encode_tiled_fn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                    const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                    const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                    CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

static inline encode_tiled_fn encode_tiled() {
    static encode_tiled_fn fn = nullptr;
    if (!fn) {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000,
                                             cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = (encode_tiled_fn)p;
    }
    return fn;
}

// 2D tensor map over a row-major byte matrix [rows][cols(elements)].
static inline bool make_map_2d(CUtensorMap *m, CUtensorMapDataType dt, const void *base, uint64_t cols,
                               uint64_t rows, uint64_t row_bytes, uint32_t box_cols,
                               uint32_t box_rows) {
    encode_tiled_fn enc = encode_tiled();
    if (!enc) return false;
    cuuint64_t gd[2] = {cols, rows};
    cuuint64_t gs[1] = {row_bytes};
    cuuint32_t bd[2] = {box_cols, box_rows};
    cuuint32_t es[2] = {1, 1};
    return enc(m, dt, 2, const_cast<void *>(base), gd, gs, bd, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
