// gdn_tma.cuh -- tensor maps over the paged cache's pools, and the copies that use them.
//
// A pool [num_pages, Hkv, page_size, d] is one 4-D tensor (d fastest).  A copy takes a box of 64
// elements (128 bytes, one swizzle row) by some tokens of one (page, head).  In shared memory row r
// of the box is 128 bytes at r * 128 with the 16-byte chunk c at c ^ (r % 8).  A page coordinate
// past the pool reads as zeros: that is how NULL pages are fetched.
#pragma once

#include <cuda.h>

#include "gdn_kv.cuh"
#include "gdn_tc.cuh"

namespace gdn {

// Maps of both pools with boxes of `box_tokens` tokens; false if the driver refuses.
bool encode_pool_maps(const KvDev& c, int box_tokens, CUtensorMap* k, CUtensorMap* v);

namespace tc {

__device__ __forceinline__ void tma_page(void* dst, const CUtensorMap* map, int col, int slot, int head, int page,
                                         uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(
          smem_addr(dst)),
      "l"(map), "r"(col), "r"(slot), "r"(head), "r"(page), "r"(smem_addr(bar))
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
