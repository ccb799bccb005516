// glr_maps.cuh -- tensor maps of the gated linear recurrence's arrays (host only).
#pragma once

#include <string.h>

#include "glr.cuh"
#include "tensor_map.cuh"

namespace kda {

// [T_total][D], rows ld elements apart: boxes of 64 tokens by 64 channels, zeros outside.
template <typename T>
bool glr_map(CUtensorMap* m, const void* base, const GlrArgs& a, long long ld) {
  const EncodeTiledFn fn = encode_tiled();
  if (!fn) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)a.D, (cuuint64_t)a.T_total};
  const cuuint64_t strides[1] = {(cuuint64_t)(a.T_total > 1 ? ld : a.D) * sizeof(T)};  // (one row's says nothing)
  const cuuint32_t boxes[2] = {kGlrCols, kGlrTile};
  const cuuint32_t estr[2] = {1, 1};
  return fn(m, sizeof(T) == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2,
            const_cast<void*>(base), dims, strides, boxes, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
template <typename T>
bool glr_maps(GlrMaps& m, const GlrArgs& a) {
  memset(&m, 0, sizeof(m));
  return a.T_total == 0 ||  // nothing is read
         (glr_map<T>(&m.la, a.la, a, a.ldla) && glr_map<T>(&m.x, a.x, a, a.ldx) &&
          (!a.gate || glr_map<T>(&m.gate, a.gate, a, a.ldg)) && (!a.dy || glr_map<T>(&m.dy, a.dy, a, a.D)));
}

}  // namespace kda
