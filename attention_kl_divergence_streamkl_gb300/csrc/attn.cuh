// The attention kernels' problem description and the device helpers they share.
#pragma once

#include "common.cuh"
#include "kernels.h"
#include "tc.cuh"

namespace skl {

// The block owns all 512 TMEM columns: ask for enough shared memory that no second block shares the SM (it would
// only wait in tcgen05.alloc).
constexpr int kOneBlockPerSmSmem = 120 * 1024;

// A sequence's length: the whole extent, or its entry of a device array, kept within the extent.
__device__ __forceinline__ int seq_len(const int* lens, int b, int n) { return lens ? min(max(lens[b], 0), n) : n; }

template <int R>
__device__ __forceinline__ void setmaxnreg_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R));
}
template <int R>
__device__ __forceinline__ void setmaxnreg_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R));
}

// True on one lane of a converged warp.  The compiler knows that a single lane follows, so the tensor-core
// instructions of that branch take their operands from uniform registers.
__device__ __forceinline__ bool elect_one() {
  uint32_t one;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(one));
  return one != 0;
}

__device__ __forceinline__ void st_shared_zero16(uint32_t addr) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(addr), "r"(0) : "memory");
}

__device__ __forceinline__ void st_shared16(uint32_t addr, uint4 v) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
  tmem_st16(taddr, *reinterpret_cast<const uint32_t(*)[16]>(&r[0]));
  tmem_st16(taddr + 16, *reinterpret_cast<const uint32_t(*)[16]>(&r[16]));
}

}  // namespace skl
