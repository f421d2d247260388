// Shared by the attention kernels that use tensor memory (attn_chunk.cu,
// attn_weights_chunk.cu).
#pragma once

#include "attn.cuh"
#include "tc.cuh"

namespace moe {

// Register shares of a warpgroup.  An increase waits until the block's own registers (threads * registers a thread at
// launch) cover it, so a kernel's shares must add up to no more than those.
template <uint32_t N>
__device__ __forceinline__ void reg_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <uint32_t N>
__device__ __forceinline__ void reg_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// place of 16-byte chunk ch (of D/8) of row r in a tile of `rows` rows: blocks of 64 columns, 128-byte swizzle
__device__ __forceinline__ uint32_t tile_offset(int r, int ch, int rows) {
  return (uint32_t)((ch >> 3) * rows * 128) + sw128_offset(r, ch & 7);
}

}  // namespace moe
