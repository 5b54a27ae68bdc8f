// Blackwell building blocks of the paged-cache kernels beside sm100_common.cuh.
#pragma once

#include "attend_common.cuh"
#include "paged_common.cuh"
#include "sm100_common.cuh"

namespace fkv {
namespace sm100 {

// 4-D tiled load into shared memory, completion counted in bytes on `bar`.
__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* m, uint64_t* bar, int c0,
                                            int c1, int c2, int c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
      : "memory");
}

}  // namespace sm100
}  // namespace fkv
