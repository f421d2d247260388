// Shared by the attention kernels that use tensor memory (attn_chunk.cu,
// attn_weights_chunk.cu).
#pragma once

#include "attn.cuh"
#include "tc.cuh"

namespace moe {

// Register shares of a warpgroup (WarpgroupRoles: what a block's add up to, and what that has to stay below).
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

// mbar_wait with its limit counted in SM cycles (some 2 s): the global timer takes so long to read that a wait which has
// to poll would wake up late.
constexpr long long kWaitCycles = 4000000000ll;
__device__ __forceinline__ bool mbar_wait_cycles(uint64_t* bar, uint32_t parity) {
  if (mbar_try_wait(bar, parity)) return true;
  const long long t0 = clock64();
  while (!mbar_try_wait(bar, parity))
    if (clock64() - t0 > kWaitCycles) return false;
  return true;
}

// One lane of a converged warp.  The products' loops run in the whole warp and only the issue itself under this, so that
// descriptors and addresses stay in uniform registers: moved there one by one from a single thread's, they made the
// issue of a tile take longer than its products.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}

// D(tmem) (+)= A(tmem) * B(smem), issued by one thread
__device__ __forceinline__ void umma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                            uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ void tmem_st4(uint32_t taddr, uint32_t r0, uint32_t r1, uint32_t r2, uint32_t r3) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1, %2, %3, %4};" ::"r"(taddr), "r"(r0), "r"(r1), "r"(r2),
               "r"(r3)
               : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

}  // namespace moe
