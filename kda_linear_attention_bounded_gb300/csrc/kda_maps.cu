// Tensor maps of the calls beside the KDA layers.  The driver's encoder is looked up at run time, so that the library loads
// on a machine without one.
#include <algorithm>

#include "kda_common.cuh"
#include "kda_hybrid.h"

namespace kda {
namespace {

using EncodeFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *, const cuuint64_t *,
                              const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encoder() {
  static EncodeFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void *p = nullptr;
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &found) == cudaSuccess &&
        found == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeFn>(p);
  });
  return fn;
}

}  // namespace

bool make_bf16_map(CUtensorMap *map, const void *base, int rank, const uint64_t *dims, const uint64_t *strides,
                   const uint32_t *box) {
  const EncodeFn encode = encoder();
  if (!encode || rank > 5) return false;
  cuuint64_t d[5], st[4];
  cuuint32_t bx[5], step[5] = {1, 1, 1, 1, 1};
  for (int i = 0; i < rank; ++i) {
    d[i] = dims[i];
    bx[i] = box[i];
    if (i + 1 < rank) st[i] = strides[i];
  }
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, static_cast<cuuint32_t>(rank), const_cast<void *>(base), d, st, bx, step,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool make_tokens_map(CUtensorMap *map, const void *base, int H, int total_tokens, int64_t token_stride) {
  const uint64_t dims[3] = {kD, static_cast<uint64_t>(H), static_cast<uint64_t>(std::max(total_tokens, 1))};
  const uint64_t strides[2] = {kD * 2, static_cast<uint64_t>(token_stride) * 2};
  const uint32_t box[3] = {64, 1, 64};
  return make_bf16_map(map, base, 3, dims, strides, box);
}

}  // namespace kda
