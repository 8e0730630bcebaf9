// gdn_tma.cu -- encodes the tensor maps of gdn_tma.cuh (host).
#include <atomic>

#include "gdn_tma.cuh"

namespace gdn {

namespace {

// The driver's encoder, reached through the runtime so the library needs no link against the driver.
using Encode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                            const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                            CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

Encode encoder() {
  static std::atomic<Encode> found{nullptr};
  Encode f = found.load(std::memory_order_acquire);
  if (f) return f;
  void* fn = nullptr;
  cudaDriverEntryPointQueryResult q;
  if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q) != cudaSuccess ||
      q != cudaDriverEntryPointSuccess)
    return nullptr;
  f = reinterpret_cast<Encode>(fn);
  found.store(f, std::memory_order_release);
  return f;
}

}  // namespace

bool encode_pool_maps(const KvDev& c, int box_tokens, CUtensorMap* k, CUtensorMap* v) {
  const Encode encode = encoder();
  if (!encode) return false;
  const cuuint64_t slabs = (cuuint64_t)(c.num_pages - 1) * slabs_per_page(c) + c.Hkv, row = (cuuint64_t)c.d * 2;
  const cuuint64_t dims[5] = {64, 8, (cuuint64_t)c.d / 64, (cuuint64_t)c.page_size / 8, slabs};
  const cuuint64_t strides[4] = {row, 128, 8 * row, c.page_size * row};
  const cuuint32_t box[5] = {64, 8, (cuuint32_t)c.d / 64, (cuuint32_t)box_tokens / 8, 1};
  const cuuint32_t ones[5] = {1, 1, 1, 1, 1};
  for (int i = 0; i < 2; ++i)
    if (encode(i ? v : k, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, i ? c.v : c.k, dims, strides, box, ones,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return false;
  return true;
}

}  // namespace gdn
