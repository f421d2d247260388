// Arithmetic of the attention kernels that needs no device: which rows see a
// run of cells, the size of an eviction's copy, and the registers that a
// block's roles take.  Plain C++, so that a host compiler can build it alone.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define MOE_HD __host__ __device__ __forceinline__
#else
#define MOE_HD inline
#endif

namespace moe {

struct RowSpan {
  int32_t a, b;              // rows [a, b): token by token, g heads each; a <= b <= n * g
};

// The rows of the n newest of `len` tokens that see one of the cells [j0, j0 + cells), j0 < len.  The token past the last
// one lies far below 0 for cells far before the window (down to -2^30), so it is brought into [first token, n] before it is
// multiplied by the group: n * g stays below 2^30.
MOE_HD RowSpan rows_that_see(int32_t j0, int32_t cells, int32_t n, int32_t len, int32_t window, int32_t g) {
  const int32_t base = len - n;                   // token i sits in cell base + i
  const int32_t t0 = j0 - base;
  const int32_t i0 = t0 < 0 ? 0 : t0 > n ? n : t0;
  const int64_t t1 = window ? (int64_t)j0 + cells - 1 - base + window : n;
  const int32_t i1 = t1 < i0 ? i0 : t1 > n ? n : (int32_t)t1;
  return RowSpan{i0 * g, i1 * g};
}

// Blocks of `cells` kept cells that an eviction's copy needs for a sequence: no sequence is longer than max_len < 2^30, so
// a budget near 2^31 takes no more (and at least one, as a launch does).
MOE_HD int32_t evict_copy_blocks(int32_t budget, int32_t max_len, int32_t cells) {
  const int32_t kept = budget < max_len ? budget : max_len;
  return kept > 0 ? (kept + cells - 1) / cells : 1;
}

// The roles of the kernels on tensor memory: registers that a thread of each warpgroup holds (setmaxnreg), one entry per
// warpgroup of the block.  An increase waits until the block's own registers (threads * registers a thread at launch)
// cover it, without end if they never do, so a launch whose registers are below registers() is refused.
template <int... Shares>
struct WarpgroupRoles {
  static constexpr int kThreads = 128 * sizeof...(Shares);
  static constexpr int registers() { return 128 * (0 + ... + Shares); }
};

struct ChunkRoles {
  static constexpr int kSoftmax = 152, kCells = 96, kProducts = 96;
  using Block = WarpgroupRoles<kSoftmax, kSoftmax, kCells, kProducts>;
};

struct WeightRoles {
  static constexpr int kAdd = 88, kLoad = 64, kProducts = 64;
  using Block = WarpgroupRoles<kAdd, kAdd, kAdd, kAdd, kLoad, kProducts>;
};

struct DeltaRoles {
  static constexpr int kChain = 184, kOutput = 88, kProducts = 56;
  using Block = WarpgroupRoles<kChain, kChain, kOutput, kProducts>;
};

}  // namespace moe
