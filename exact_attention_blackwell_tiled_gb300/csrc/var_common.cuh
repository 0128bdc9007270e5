// var_common.cuh -- the plan of a packed call (sequences of different lengths
// in one [T, H, D] tensor), as the plan kernel writes it and the attention
// kernels read it.
#pragma once

#include "fa_internal.h"

namespace fa {

// The part of an item every kernel reads, in one 16-byte load.
__device__ __forceinline__ VarItem load_item(const VarItem* items, int i) {
  const int4 x = *reinterpret_cast<const int4*>(items + i);
  VarItem it;
  it.row0 = x.x;
  it.len = x.y;
  it.tile = x.z;
  it.b = x.w;
  return it;
}

// Orders this thread's later reads of a tensor map (by the TMA unit) after the
// plan kernel's write of it, which the grid dependency has already made visible
// to ordinary loads.
__device__ __forceinline__ void tmap_acquire(const CUtensorMap* m) {
  asm volatile("fence.proxy.tensormap::generic.acquire.gpu [%0], 128;" ::"l"(
                   reinterpret_cast<uint64_t>(m))
               : "memory");
}

}  // namespace fa
