// Eviction by accumulated attention weight: per sequence the newest R cells
// and the B - R largest weights of the others stay (ties to the lower index),
// in order, and move to new pages.
//
// Selection: a cluster of CTAs per sequence finds the B - R'th largest weight
// digit by digit (8 bits a pass, from the top) in an order-preserving 32-bit
// key: each CTA counts the digits of its slice in shared memory, the counts
// are added over the cluster through distributed shared memory, and every CTA
// picks the same digit.  The slices are in index order, so a prefix over the
// cluster's counts gives each CTA the place of its first kept cell and how
// many cells equal to the threshold it may keep; results do not depend on the
// order in which CTAs ran.
#include <cooperative_groups.h>

#include "attn.cuh"

namespace cg = cooperative_groups;

namespace moe {

namespace {

constexpr int kCl = 8;                // CTAs per sequence
constexpr int kSel = 512;             // threads per CTA

// NaN counts as -inf, and -0 as 0
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) w = -INFINITY;
  return float_key(w + 0.f);
}

__global__ void __cluster_dims__(kCl, 1, 1) __launch_bounds__(kSel) evict_select_kernel(const __grid_constant__ EvictArgs a) {
  cg::cluster_group cl = cg::this_cluster();
  __shared__ uint32_t hist[256];
  __shared__ uint32_t tot[256];
  __shared__ uint32_t pick[2];        // digit, count above it
  __shared__ uint32_t cnt[2];         // above, equal in this slice
  __shared__ uint32_t wsum[2][kSel / 32];
  const int s = blockIdx.x / kCl, r = (int)cl.block_rank(), tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
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
  const int per = (M + kCl - 1) / kCl, lo = min(M, r * per), hi = min(M, lo + per);
  uint32_t prefix = 0, above = 0;     // the threshold's digits so far; cells above them
  const bool select = need < M && need > 0;
  if (select) {
    for (int shift = 24; shift >= 0; shift -= 8) {
      for (int i = tid; i < 256; i += kSel) hist[i] = 0;
      __syncthreads();
      for (int j = lo + tid; j < hi; j += kSel) {
        const uint32_t k = weight_key(acc[j]);
        if (shift == 24 || (k >> (shift + 8)) == (prefix >> (shift + 8))) atomicAdd(&hist[k >> shift & 255], 1u);
      }
      cl.sync();
      if (tid < 256) {
        uint32_t t = 0;
        for (int c = 0; c < kCl; ++c) t += *cl.map_shared_rank(&hist[tid], c);
        tot[tid] = t;
      }
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
          const uint32_t n = __shfl_up_sync(0xffffffffu, inc, o);
          if (lane >= o) inc += n;
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
      cl.sync();                      // tot and pick are read; no CTA clears hist before all have added it
      prefix |= pick[0] << shift;
      above = pick[1];
      __syncthreads();
    }
  }
  // cells above the threshold and equal to it, per slice
  const uint32_t thr = prefix, eq_room = select ? (uint32_t)need - above : 0u;
  auto flags = [&](int j, bool& g, bool& e) {
    if (j >= hi) {
      g = e = false;
    } else if (!select) {
      g = need > 0;                   // all of them, or none
      e = false;
    } else {
      const uint32_t k = weight_key(acc[j]);
      g = k > thr;
      e = k == thr;
    }
  };
  if (tid < 2) cnt[tid] = 0;
  __syncthreads();
  uint32_t ng = 0, ne = 0;
  for (int j = lo + tid; j < hi; j += kSel) {
    bool g, e;
    flags(j, g, e);
    ng += g;
    ne += e;
  }
  ng = __reduce_add_sync(0xffffffffu, ng);
  ne = __reduce_add_sync(0xffffffffu, ne);
  if (lane == 0) {
    atomicAdd(&cnt[0], ng);
    atomicAdd(&cnt[1], ne);
  }
  cl.sync();
  uint32_t g0 = 0, e0 = 0;            // of the slices before this one
  for (int c = 0; c < r; ++c) {
    g0 += *cl.map_shared_rank(&cnt[0], c);
    e0 += *cl.map_shared_rank(&cnt[1], c);
  }
  cl.sync();                          // no CTA leaves while its counts are read
  for (int base = lo; base < hi; base += kSel) {
    const int j = base + tid;
    bool g, e;
    flags(j, g, e);
    const uint32_t mg = __ballot_sync(0xffffffffu, g), me = __ballot_sync(0xffffffffu, e);
    if (lane == 0) {
      wsum[0][warp] = __popc(mg);
      wsum[1][warp] = __popc(me);
    }
    __syncthreads();
    uint32_t gb = g0, eb = e0, gt = 0, et = 0;
    for (int w = 0; w < kSel / 32; ++w) {
      if (w < warp) {
        gb += wsum[0][w];
        eb += wsum[1][w];
      }
      gt += wsum[0][w];
      et += wsum[1][w];
    }
    const uint32_t lt = (1u << lane) - 1u;
    gb += __popc(mg & lt);
    eb += __popc(me & lt);
    if (g || (e && eb < eq_room)) {
      const uint32_t at = gb + min(eb, eq_room);
      keep[at] = j;
      out[at] = acc[j];
    }
    g0 += gt;
    e0 += et;
    __syncthreads();
  }
  // the newest cells, then the end marks
  for (int i = need + r * kSel + tid; i < a.budget; i += kCl * kSel) {
    const bool in = i < kept;
    keep[i] = in ? M + i - need : -1;
    out[i] = in ? acc[M + i - need] : 0.f;
  }
  if (r == 0 && tid == 0) a.new_lens[s] = kept;
}

__global__ void __launch_bounds__(256) evict_copy_kernel(const __grid_constant__ EvictArgs a, FastDiv chunks) {
  const int64_t n = (int64_t)a.b.n_seqs * a.budget * chunks.d;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
    const int64_t row = i / chunks.d;
    const int c = (int)(i - row * chunks.d), s = (int)(row / a.budget), k = (int)(row - (int64_t)s * a.budget);
    const int j = a.keep[row];
    if (j < 0) continue;
    const uint8_t* src = cell_ptr(a.b, s, j);
    const uint32_t pg = fdiv((uint32_t)k, a.b.page_div);
    const int id = a.new_table[(int64_t)s * a.new_table_pages + pg];
    if ((uint32_t)id >= (uint32_t)a.b.n_pages) {
      atomicOr(a.b.err, (uint32_t)ATTN_BAD_PAGE);
      continue;
    }
    if (!src) continue;
    uint8_t* dst = a.b.cells + (int64_t)id * a.b.page_bytes + (int64_t)(k - (int)pg * a.b.page_cells) * a.b.cell_bytes;
    reinterpret_cast<uint4*>(dst)[c] = reinterpret_cast<const uint4*>(src)[c];
  }
}

}  // namespace

cudaError_t launch_attn_evict(const EvictArgs& a, cudaStream_t s) {
  evict_select_kernel<<<a.b.n_seqs * kCl, kSel, 0, s>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const int64_t n = (int64_t)a.b.n_seqs * a.budget * (a.b.cell_bytes / 16);
  const int64_t blocks = (n + 255) / 256, most = (int64_t)a.num_sms * 32;
  evict_copy_kernel<<<(int)(blocks < most ? blocks : most), 256, 0, s>>>(a, make_fastdiv(a.b.cell_bytes / 16));
  return cudaGetLastError();
}

}  // namespace moe
