// Eviction by accumulated attention weight: per sequence the newest R cells
// and the B - R largest weights of the others stay (ties to the lower index),
// in order, and move to new pages.
//
// Selection: a cluster of CTAs per sequence finds the B - R'th largest weight
// digit by digit (8 bits a pass, from the top) in an order-preserving 32-bit
// key.  Each CTA reads its slice of the weights once, keeps the keys in shared
// memory (as far as they fit) and counts digits there; the counts are added
// over the cluster through distributed shared memory, and every CTA picks the
// same digit.  Slices, and the warps' parts of a slice, are in index order, so
// prefix sums over their counts give every warp the place of its first kept
// cell and how many cells equal to the threshold it may keep: results do not
// depend on the order in which anything ran.  Bound by the latency of the
// passes and of the cluster's barriers.
//
// Copy: bound by the bytes of the kept cells, read and written once; a block
// looks up 64 cells' places and copies them as one run of 16-byte chunks.
// 32,768 of 131,072 int8 cells: 34 us, of which the copy is 12.
#include <cooperative_groups.h>

#include "attn.cuh"

namespace cg = cooperative_groups;

namespace moe {

namespace {

// CTAs per sequence.  One below kShort cells, where a cluster's barriers cost what its shorter passes save (12
// sequences of 750 to 6,000 cells: 18 us, 21 with 8 CTAs each; one of 8,192: 20 and 17, of 16,384: 26 and 18).  16, beyond
// the portable size, above kLong (131,072 cells: 45 us, 48 with 8).  No more than kWave in all, so that every cluster
// runs at once (32 sequences of 98,304 cells: 76 us with 4 CTAs each, 107 with 8, 137 with 16).
constexpr int kMaxCl = 16, kShort = 8192, kLong = 65536, kWave = 128;
constexpr int kCopies = 8, kCopyPitch = 260;
constexpr int kSel = 1024, kSelWarps = kSel / 32;
constexpr int kMaxKeys = 48 * 1024;   // keys of a slice in shared memory (the rest is read from memory in every pass)

// NaN counts as -inf, and -0 as 0
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) w = -INFINITY;
  return float_key(w + 0.f);
}

__global__ void __launch_bounds__(kSel)
    evict_select_kernel(const __grid_constant__ EvictArgs a, int cap_keys) {
  cg::cluster_group cl = cg::this_cluster();
  extern __shared__ uint32_t keys[];
  // Digit counts, twice: one is cleared while the other is read.  Weights crowd into few digits (the leading ones are
  // sign and exponent), so a count is kept in kCopies copies, 8 lanes apart and in different banks.
  __shared__ uint32_t part[kCopies][kCopyPitch], hist[2][256], tot[256], pick[2], cnt[2];
  __shared__ uint32_t wg[kSelWarps], we[kSelWarps];
  pdl_launch_dependents();
  const int kCl = (int)cl.num_blocks(), s = blockIdx.x / kCl, r = (int)cl.block_rank(), tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int L = a.b.kv_lens[s];
  const int cap = (int)min((int64_t)a.b.max_len, a.acc_stride);
  if (L < 0 || L > cap) {
    if (tid == 0) atomicOr(a.b.err, (uint32_t)ATTN_BAD_LEN);
    L = min(max(L, 0), cap);
  }
  const int R = min(a.recent, L), M = L - R;               // candidates are [0, M)
  const int kept = min(L, a.budget), need = kept - R;
  const float* acc = a.acc + (int64_t)s * a.acc_stride;
  int32_t* keep = a.keep + (int64_t)s * a.budget;
  float* out = a.acc_out + (int64_t)s * a.budget;
  // this CTA's slice [lo, hi), and the part of it that this warp owns when places are given
  const int per = (M + kCl - 1) / kCl, lo = min(M, r * per), n = min(M, lo + per) - lo;
  auto key_at = [&](int i) { return i < cap_keys ? keys[i] : weight_key(acc[lo + i]); };
  uint32_t thr = 0, above = 0;        // the threshold's digits so far; cells above them
  const bool select = need < M && need > 0;
  auto clear = [&] {
    for (int i = tid; i < kCopies * kCopyPitch; i += kSel) (&part[0][0])[i] = 0;
  };
  uint32_t* mine = part[lane & (kCopies - 1)];
  if (select) {
    clear();
    __syncthreads();
#pragma unroll 4
    for (int i = tid; i < n; i += kSel) {
      const uint32_t k = weight_key(acc[lo + i]);
      if (i < cap_keys) keys[i] = k;
      atomicAdd(&mine[k >> 24], 1u);
    }
    for (int shift = 24, p = 0;; shift -= 8, p ^= 1) {
      __syncthreads();
      if (tid < 256) {
        uint32_t t = 0;
#pragma unroll
        for (int c = 0; c < kCopies; ++c) t += part[c][tid];
        hist[p][tid] = t;
      }
      cl.sync();                      // every CTA's counts are there (and the other ones have been read)
      if (tid < 256) {
        uint32_t t = 0;
#pragma unroll
        for (int c = 0; c < kMaxCl; ++c)
          if (c < kCl) t += *cl.map_shared_rank(&hist[p][tid], c);
        tot[tid] = t;
      }
      if (shift) clear();
      __syncthreads();
      if (warp == 0) {                // digits from the top: lane l owns 255 - 8l .. 248 - 8l
        uint32_t v[8], sum = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          v[i] = tot[255 - 8 * lane - i];
          sum += v[i];
        }
        uint32_t inc = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const uint32_t x = __shfl_up_sync(0xffffffffu, inc, o);
          if (lane >= o) inc += x;
        }
        uint32_t before = above + inc - sum;
        const uint32_t target = (uint32_t)need;      // the first digit at which the count reaches it
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (before < target && before + v[i] >= target) {
            pick[0] = 255 - 8 * lane - i;
            pick[1] = before;
          }
          before += v[i];
        }
      }
      __syncthreads();
      thr |= pick[0] << shift;
      above = pick[1];
      if (shift == 0) break;
#pragma unroll 4
      for (int i = tid; i < n; i += kSel) {
        const uint32_t k = key_at(i);
        if (k >> shift == thr >> shift) atomicAdd(&mine[k >> (shift - 8) & 255], 1u);
      }
    }
  }
  // ---- cells above the threshold and equal to it, per warp (32 consecutive cells at a time) ----
  const uint32_t eq_room = select ? (uint32_t)need - above : 0u;
  const int chunk = ((n + kSelWarps - 1) / kSelWarps + 31) & ~31, w0 = min(n, warp * chunk), w1 = min(n, w0 + chunk);
  auto flags = [&](int i, bool& gt, bool& eq, uint32_t& k) {
    gt = eq = false;
    k = 0;
    if (i < w1) {
      if (!select) {
        gt = need > 0;                // all of them, or none
      } else {
        k = key_at(i);
        gt = k > thr;
        eq = k == thr;
      }
    }
  };
  uint32_t ng = 0, ne = 0;
#pragma unroll 4
  for (int i = w0; i < w1; i += 32) {
    bool gt, eq;
    uint32_t k;
    flags(i + lane, gt, eq, k);
    ng += __popc(__ballot_sync(0xffffffffu, gt));
    ne += __popc(__ballot_sync(0xffffffffu, eq));
  }
  if (lane == 0) {
    wg[warp] = ng;
    we[warp] = ne;
  }
  __syncthreads();
  uint32_t gb = 0, eb = 0;            // before this warp, first within the slice
  {
    uint32_t x = wg[lane], y = we[lane];
    const uint32_t tg = __reduce_add_sync(0xffffffffu, x), te = __reduce_add_sync(0xffffffffu, y);
    x = lane < warp ? x : 0;
    y = lane < warp ? y : 0;
    gb = __reduce_add_sync(0xffffffffu, x);
    eb = __reduce_add_sync(0xffffffffu, y);
    if (tid == 0) {
      cnt[0] = tg;
      cnt[1] = te;
    }
  }
  cl.sync();
  for (int c = 0; c < r; ++c) {
    gb += *cl.map_shared_rank(&cnt[0], c);
    eb += *cl.map_shared_rank(&cnt[1], c);
  }
  // a key stands for its weight, but for those that several weights map to
  const uint32_t key_inf = float_key(-INFINITY), key_zero = float_key(0.f);
#pragma unroll 2
  for (int i = w0; i < w1; i += 32) {
    bool gt, eq;
    uint32_t k;
    flags(i + lane, gt, eq, k);
    const uint32_t mg = __ballot_sync(0xffffffffu, gt), me = __ballot_sync(0xffffffffu, eq);
    const uint32_t lt = (1u << lane) - 1u, e = eb + __popc(me & lt);
    if (gt || (eq && e < eq_room)) {
      const uint32_t at = gb + __popc(mg & lt) + min(e, eq_room);
      const int j = lo + i + lane;
      keep[at] = j;
      out[at] = select && k != key_inf && k != key_zero ? key_float(k) : acc[j];
    }
    gb += __popc(mg);
    eb += __popc(me);
  }
  // the newest cells, then the end marks (unsigned: with a budget near 2^31 the step past the last one is beyond it)
  for (uint32_t i = need + r * kSel + tid; i < (uint32_t)a.budget; i += kCl * kSel) {
    const bool in = i < (uint32_t)kept;
    keep[i] = in ? M + (int)i - need : -1;
    out[i] = in ? acc[M + (int)i - need] : 0.f;
  }
  if (r == 0 && tid == 0) a.new_lens[s] = kept;
  cl.sync();                          // no CTA leaves while its counts are read
}

constexpr int kCopyCells = 64, kCopyThreads = 256;

__global__ void __launch_bounds__(kCopyThreads)
    evict_copy_kernel(const __grid_constant__ EvictArgs a, FastDiv chunks) {
  __shared__ const uint8_t* src[kCopyCells];
  __shared__ uint8_t* dst[kCopyCells];
  pdl_wait();
  const int s = blockIdx.y, k0 = blockIdx.x * kCopyCells;
  if (threadIdx.x < kCopyCells) {
    const int k = k0 + threadIdx.x;
    const int j = k < a.budget ? a.keep[(int64_t)s * a.budget + k] : -1;
    const uint8_t* from = nullptr;
    uint8_t* to = nullptr;
    if (j >= 0) {
      from = cell_ptr(a.b, s, j);
      const uint32_t pg = fdiv((uint32_t)k, a.b.page_div);
      const int id = a.new_table[(int64_t)s * a.new_table_pages + pg];
      if ((uint32_t)id >= (uint32_t)a.b.n_pages) {
        atomicOr(a.b.err, (uint32_t)ATTN_BAD_PAGE);
        from = nullptr;
      } else {
        to = a.b.cells + (int64_t)id * a.b.page_bytes + (int64_t)(k - (int)pg * a.b.page_cells) * a.b.cell_bytes;
      }
    }
    src[threadIdx.x] = from;
    dst[threadIdx.x] = to;
  }
  __syncthreads();
  const int total = kCopyCells * (int)chunks.d;
  for (int x0 = threadIdx.x; x0 < total; x0 += 4 * kCopyThreads) {
    uint4 v[4];
    uint8_t* to[4];
#pragma unroll
    for (int y = 0; y < 4; ++y) {
      const int x = x0 + y * kCopyThreads;
      to[y] = nullptr;
      if (x < total) {
        const int c = (int)fdiv((uint32_t)x, chunks), at = (x - c * (int)chunks.d) * 16;
        const uint8_t* from = src[c];
        if (from) {
          v[y] = *reinterpret_cast<const uint4*>(from + at);
          to[y] = dst[c] + at;
        }
      }
    }
#pragma unroll
    for (int y = 0; y < 4; ++y)
      if (to[y]) *reinterpret_cast<uint4*>(to[y]) = v[y];
  }
}

}  // namespace

cudaError_t launch_attn_evict(const EvictArgs& a, cudaStream_t s) {
  const int64_t longest = a.acc_stride < a.b.max_len ? a.acc_stride : a.b.max_len;
  int cl = longest > kLong ? kMaxCl : longest >= kShort ? 8 : 1;
  while (cl > 1 && (int64_t)a.b.n_seqs * cl > kWave) cl >>= 1;
  const int64_t slice = (longest + cl - 1) / cl;
  const int cap = (int)(slice < kMaxKeys ? slice : kMaxKeys);
  cudaError_t e = ensure_dyn_smem(reinterpret_cast<const void*>(evict_select_kernel), kMaxKeys * 4);
  if (e == cudaSuccess && cl > 8)
    e = cudaFuncSetAttribute(evict_select_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.gridDim = dim3((unsigned)(a.b.n_seqs * cl));
  cfg.blockDim = dim3(kSel);
  cfg.dynamicSmemBytes = (size_t)cap * 4;
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)cl;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  e = cudaLaunchKernelEx(&cfg, evict_select_kernel, a, cap);
  if (e != cudaSuccess) return e;
  cfg.gridDim = dim3((unsigned)evict_copy_blocks(a.budget, a.b.max_len, kCopyCells), (unsigned)a.b.n_seqs);
  cfg.blockDim = dim3(kCopyThreads);
  cfg.dynamicSmemBytes = 0;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  return cudaLaunchKernelEx(&cfg, evict_copy_kernel, a, make_fastdiv(a.b.cell_bytes / 16));
}

}  // namespace moe
