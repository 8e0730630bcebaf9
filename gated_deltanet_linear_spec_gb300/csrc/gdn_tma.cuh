// gdn_tma.cuh -- tensor maps over the paged cache's pools, and the copies that use them.
//
// A pool [num_pages, Hkv, page_size, d] is a row of slabs, one per (page, head): page_size x d elements.
// Its map is 5-D: 64 columns (128 bytes, one swizzle row) | 8 tokens | the d / 64 column blocks | the
// 8-token groups of a slab | slabs.  One copy takes some tokens of a slab with all their columns and
// leaves them as [8-token group][column block][8 tokens][128 bytes]: token t's 16-byte chunk c of
// block cb at (t / 8) * d * 16 + cb * 1024 + (t % 8) * 128 + ((c ^ (t % 8)) << 4).  A slab past the
// pool reads as zeros: that is how NULL pages are fetched.
#pragma once

#include <cuda.h>

#include "gdn_kv.cuh"
#include "gdn_tc.cuh"

namespace gdn {

// Slabs from one page to the next.
__host__ __device__ inline int slabs_per_page(const KvDev& c) {
  return (int)(c.page_stride / ((int64_t)c.page_size * c.d));
}

// Maps of both pools with boxes of `box_tokens` tokens; false if the driver refuses.
bool encode_pool_maps(const KvDev& c, int box_tokens, CUtensorMap* k, CUtensorMap* v);

namespace tc {

// The box at token `slot` of a slab.
__device__ __forceinline__ void tma_page(void* dst, const CUtensorMap* map, int slot, int slab, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %2, %2, %3, %4}], [%5];" ::"r"(
          smem_addr(dst)),
      "l"(map), "r"(0), "r"(slot >> 3), "r"(slab), "r"(smem_addr(bar))
      : "memory");
}
__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}

}  // namespace tc
}  // namespace gdn
