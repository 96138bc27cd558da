// Host-side encoding of TMA tensor maps over bf16 arrays.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/shla.h"

namespace shla {

typedef CUresult (*EncodeTiledFnPtr)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                     const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                     const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                     CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeTiledFnPtr tma_encoder() {
  // looked up once (a function-local static is initialised thread-safely)
  static const EncodeTiledFnPtr fn = []() -> EncodeTiledFnPtr {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      return reinterpret_cast<EncodeTiledFnPtr>(f);
    cudaGetLastError();
    return nullptr;
  }();
  return fn;
}

// Dimensions from the innermost; byte strides of dimensions 1 .. rank-1; the
// box in elements.  The innermost box extent spans one swizzle row (64
// elements with the 128-byte swizzle, 32 with the 64-byte one).
inline int bf16_map(CUtensorMap* map, const void* base, int rank, const cuuint64_t* dims,
                    const cuuint64_t* strides_bytes, const cuuint32_t* box,
                    CUtensorMapSwizzle swz = CU_TENSOR_MAP_SWIZZLE_128B,
                    CUtensorMapL2promotion l2 = CU_TENSOR_MAP_L2_PROMOTION_L2_256B) {
  EncodeTiledFnPtr fn = tma_encoder();
  if (!fn) return MLA_ERR_CUDA;
  const cuuint32_t estr[3] = {1, 1, 1};
  const CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void*>(base), dims,
                        strides_bytes, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, swz, l2,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? MLA_OK : MLA_ERR_CUDA;
}

inline int bf16_map_2d(CUtensorMap* map, const void* base, uint64_t cols, uint64_t rows,
                       uint64_t row_bytes, uint32_t box_cols, uint32_t box_rows,
                       CUtensorMapSwizzle swz = CU_TENSOR_MAP_SWIZZLE_128B,
                       CUtensorMapL2promotion l2 = CU_TENSOR_MAP_L2_PROMOTION_L2_256B) {
  const cuuint64_t dims[2] = {cols, rows};
  const cuuint64_t strides[1] = {row_bytes};
  const cuuint32_t box[2] = {box_cols, box_rows};
  return bf16_map(map, base, 2, dims, strides, box, swz, l2);
}

inline int bf16_map_3d(CUtensorMap* map, const void* base, uint64_t d0, uint64_t d1, uint64_t d2,
                       uint64_t s1_bytes, uint64_t s2_bytes, uint32_t b0, uint32_t b1,
                       uint32_t b2) {
  const cuuint64_t dims[3] = {d0, d1, d2};
  const cuuint64_t strides[2] = {s1_bytes, s2_bytes};
  const cuuint32_t box[3] = {b0, b1, b2};
  return bf16_map(map, base, 3, dims, strides, box);
}

}  // namespace shla
