// Norms around the blocks (moe_norm_block, moe_norm_gated): one pass over the
// rows, with a row's elements in the registers of the threads that share it.
//
// A group of TPR threads (a power of two, 2 to 1,024) takes a row, thread l the
// 8-element pieces l, l + TPR, ...  Sums of squares are fp32: over a group of up to a warp by
// shuffles, over more warps through shared memory.
//
// Bound by bytes: every input is read and every output written once.  12,288 rows of 2,048 with a gate (352 MB) 56 us, 94%
// of the copy bandwidth; 12,288 x 32 vectors of 128 (302 MB) 52 us, 87%, and 77% of the issue slots.
#include <cmath>

#include "delta.cuh"
#include "rows.h"

using namespace moe;

namespace {

// 8 elements in 32 bits, of a 16-bit or fp32 row
template <bool F32, bool BF16>
__device__ __forceinline__ void load8(const void* row, int64_t at, float (&x)[8]) {
  if constexpr (F32) {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(row) + at);
    const float4 u = __ldcs(p), v = __ldcs(p + 1);
    x[0] = u.x, x[1] = u.y, x[2] = u.z, x[3] = u.w, x[4] = v.x, x[5] = v.y, x[6] = v.z, x[7] = v.w;
  } else {
    const uint4 r = __ldcs(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(row) + at));
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 f = unpack16<BF16>(w[e]);
      x[2 * e] = f.x;
      x[2 * e + 1] = f.y;
    }
  }
}
// weights: the same for every row, so they stay in the caches
template <bool BF16>
__device__ __forceinline__ void load_w(const uint16_t* w, int at, float off, float (&x)[8]) {
  const uint4 r = __ldg(reinterpret_cast<const uint4*>(w + at));
  const uint32_t u[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 f = unpack16<BF16>(u[e]);
    x[2 * e] = f.x + off;
    x[2 * e + 1] = f.y + off;
  }
}
template <bool F32, bool BF16>
__device__ __forceinline__ void store8(void* row, int64_t at, const float (&x)[8]) {
  if constexpr (F32) {
    float4* p = reinterpret_cast<float4*>(static_cast<float*>(row) + at);
    __stcs(p, make_float4(x[0], x[1], x[2], x[3]));
    __stcs(p + 1, make_float4(x[4], x[5], x[6], x[7]));
  } else {
    __stcs(reinterpret_cast<uint4*>(static_cast<uint16_t*>(row) + at),
           make_uint4(pack16<BF16>(x[0], x[1]), pack16<BF16>(x[2], x[3]), pack16<BF16>(x[4], x[5]), pack16<BF16>(x[6], x[7])));
  }
}

// F32: for a result that stays fp32
template <bool F32>
__device__ __forceinline__ float act_of(float z, int act) {
  if (act == MOE_ACT_NONE) return z;
  const float s = F32 ? logistic32(z) : logistic(z);
  return act == MOE_ACT_SILU ? z * s : s;
}

// Sum over the tpr threads of a row; with more than a warp the whole block is one row.
__device__ __forceinline__ float row_sum(float x, int tpr, float* red) {
  for (int o = min(tpr, 32) >> 1; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  if (tpr > 32) {
    const int warps = tpr >> 5;
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = x;
    __syncthreads();
    x = (threadIdx.x & 31) < warps ? red[threadIdx.x & 31] : 0.f;
#pragma unroll
    for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  }
  return x;
}

struct BlockArgs {
  const void *y, *h, *gate;
  const uint16_t *post_w, *pre_w;
  void *h_out, *x;
  int64_t rows, y_stride, h_stride, gate_stride;
  int d, tpr, gate_cols, act;
  float scale, eps, off;
};

template <bool BF16, bool YF, bool HF, int V>
__global__ void __launch_bounds__(1024) block_kernel(const __grid_constant__ BlockArgs a) {
  __shared__ float red[2][32];
  const int l = threadIdx.x & (a.tpr - 1);
  const int64_t row = (int64_t)blockIdx.x * (blockDim.x / a.tpr) + threadIdx.x / a.tpr;
  const bool live = row < a.rows;
  const float inv_d = 1.f / (float)a.d;
  float y[V][8], h[V][8];
  uint4 gate[V];
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int at = (l + i * a.tpr) * 8;
    const bool in = live && at < a.d;
#pragma unroll
    for (int e = 0; e < 8; ++e) y[i][e] = h[i][e] = 0.f;
    gate[i] = make_uint4(0, 0, 0, 0);
    if (in) {
      load8<YF, BF16>(a.y, row * a.y_stride + at, y[i]);
      if (a.h) load8<HF, BF16>(a.h, row * a.h_stride + at, h[i]);
      if (a.gate_cols > 1) gate[i] = __ldcs(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.gate) + row * a.gate_stride + at));
    }
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
#pragma unroll
    for (int e = 0; e < 8; ++e) ss += y[i][e] * y[i][e];
  }
  float f = 1.f;
  if (a.post_w) f = rsqrtf(row_sum(ss, a.tpr, red[0]) * inv_d + a.eps);
  f *= a.scale;
  if (a.gate_cols == 1 && live) f *= act_of<HF>(load16<BF16>(static_cast<const uint16_t*>(a.gate) + row * a.gate_stride), a.act);
  ss = 0.f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int at = (l + i * a.tpr) * 8;
    if (live && at < a.d) {
      float k[8];                        // the weight times the gate
#pragma unroll
      for (int e = 0; e < 8; ++e) k[e] = 1.f;
      if (a.post_w) load_w<BF16>(a.post_w, at, a.off, k);
      if (a.gate_cols > 1) {
        const uint32_t g[4] = {gate[i].x, gate[i].y, gate[i].z, gate[i].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 f2 = unpack16<BF16>(g[e]);
          k[2 * e] *= act_of<HF>(f2.x, a.act);
          k[2 * e + 1] *= act_of<HF>(f2.y, a.act);
        }
      }
      // (y is normed before that: y times its gate may pass fp32)
#pragma unroll
      for (int e = 0; e < 8; ++e) h[i][e] += (f * y[i][e]) * k[e];
      if (a.h_out) store8<HF, BF16>(a.h_out, row * a.d + at, h[i]);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) ss += h[i][e] * h[i][e];
  }
  if (!a.x) return;
  f = rsqrtf(row_sum(ss, a.tpr, red[1]) * inv_d + a.eps);
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int at = (l + i * a.tpr) * 8;
    if (live && at < a.d) {
      float w[8];
      load_w<BF16>(a.pre_w, at, a.off, w);
#pragma unroll
      for (int e = 0; e < 8; ++e) w[e] *= f * h[i][e];
      store8<false, BF16>(a.x, row * a.d + at, w);
    }
  }
}

struct GatedArgs {
  const uint16_t *o, *z, *w;
  uint16_t* out;
  int64_t rows, o_stride, z_stride;
  int d, tpr, heads, act, gate_first;
  float eps, off;
};

// A group of threads takes ROWS rows at a time, whose loads are all under way before the first is used.
template <bool BF16, int V, int ROWS>
__global__ void __launch_bounds__(ROWS > 1 ? 128 : 1024) gated_kernel(const __grid_constant__ GatedArgs a) {
  __shared__ float red[32];
  const int l = threadIdx.x & (a.tpr - 1), groups = blockDim.x / a.tpr;
  const int64_t row0 = (int64_t)blockIdx.x * groups * ROWS + threadIdx.x / a.tpr;
  uint4 ro[ROWS][V], rz[ROWS][V];
#pragma unroll
  for (int k = 0; k < ROWS; ++k) {
    const int64_t row = row0 + k * groups, t = (uint32_t)row / (uint32_t)a.heads, hd = (row - t * a.heads) * a.d;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int at = (l + i * a.tpr) * 8;
      ro[k][i] = rz[k][i] = make_uint4(0, 0, 0, 0);
      if (row < a.rows && at < a.d) {
        ro[k][i] = __ldcs(reinterpret_cast<const uint4*>(a.o + t * a.o_stride + hd + at));
        rz[k][i] = __ldcs(reinterpret_cast<const uint4*>(a.z + t * a.z_stride + hd + at));
      }
    }
  }
  float w[V][8];                      // the same for every row of this thread
#pragma unroll
  for (int i = 0; i < V; ++i)
    if ((l + i * a.tpr) * 8 < a.d) load_w<BF16>(a.w, (l + i * a.tpr) * 8, a.off, w[i]);
#pragma unroll
  for (int k = 0; k < ROWS; ++k) {
    const int64_t row = row0 + k * groups;
    float o[V][8], g[V][8];
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const uint32_t uo[4] = {ro[k][i].x, ro[k][i].y, ro[k][i].z, ro[k][i].w}, uz[4] = {rz[k][i].x, rz[k][i].y, rz[k][i].z, rz[k][i].w};
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float2 fo = unpack16<BF16>(uo[e / 2]), fz = unpack16<BF16>(uz[e / 2]);
        o[i][e] = e & 1 ? fo.y : fo.x;
        g[i][e] = act_of<false>(e & 1 ? fz.y : fz.x, a.act);
        if (a.gate_first) {
          o[i][e] *= g[i][e];
          g[i][e] = 1.f;
        }
        ss += o[i][e] * o[i][e];
      }
    }
    const float f = rsqrtf(row_sum(ss, a.tpr, red) / (float)a.d + a.eps);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int at = (l + i * a.tpr) * 8;
      if (row < a.rows && at < a.d) {
        float y[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = (o[i][e] * f) * w[i][e] * g[i][e];   // (normed first: o times its gate may pass fp32)
        store8<false, BF16>(a.out, row * a.d + at, y);
      }
    }
  }
}

// Threads per row (a power of two, 2 to 1,024) for at most `want` pieces each where that goes, and the pieces that each takes
// (1 or 2).
void share(int d, int want, int* tpr, int* v) {
  const int pieces = d / 8;
  *tpr = 2;
  while (*tpr * want < pieces && *tpr < 1024) *tpr *= 2;
  *v = 1;
  while (*v * *tpr < pieces) *v *= 2;
}

bool mis16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }

moe_status take_desc(const moe_norm_desc* D) {
  if (!D) return set_last_error(MOE_ERR_INVALID_ARG, "NULL desc");
  if (D->d < 8 || D->d > 16384 || D->d % 8 != 0)
    return set_last_error(MOE_ERR_INVALID_ARG, "d must be a multiple of 8 in [8, 16384]");
  if (D->io_type != MOE_T_BF16 && D->io_type != MOE_T_F16)
    return set_last_error(MOE_ERR_INVALID_ARG, "io_type must be MOE_T_BF16 or MOE_T_F16");
  if (D->act < MOE_ACT_NONE || D->act > MOE_ACT_SILU) return set_last_error(MOE_ERR_INVALID_ARG, "unknown act");
  if (!std::isfinite(D->eps) || D->eps < 0.f)
    return set_last_error(MOE_ERR_INVALID_ARG, "eps must be finite and not negative");
  if (!std::isfinite(D->weight_offset)) return set_last_error(MOE_ERR_INVALID_ARG, "weight_offset must be finite");
  return MOE_OK;
}

moe_status take_rows(const void* p, int64_t stride, int64_t width, const char* what) {
  if (!p) return set_last_error(MOE_ERR_INVALID_ARG, "NULL %s", what);
  if (mis16(p) || stride % 8 != 0 || stride < width)
    return set_last_error(MOE_ERR_INVALID_ARG,
                          "%s must be 16-byte aligned, its stride a multiple of 8 elements and at least %lld", what,
                          (long long)width);
  return MOE_OK;
}

#define NORM_CHECK(call)                    \
  do {                                      \
    const moe_status st_ = (call);          \
    if (st_ != MOE_OK) return st_;          \
  } while (0)

moe_status launched(cudaError_t e, const char* what) {
  return e == cudaSuccess ? MOE_OK : set_last_error(MOE_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

template <bool BF16, bool YF, bool HF>
void block_v(const BlockArgs& a, int v, unsigned grid, int threads, cudaStream_t s) {
  if (v == 1) block_kernel<BF16, YF, HF, 1><<<grid, threads, 0, s>>>(a);
  else block_kernel<BF16, YF, HF, 2><<<grid, threads, 0, s>>>(a);
}

}  // namespace

extern "C" moe_status moe_norm_block(const moe_norm_desc* D, int64_t rows, const void* y, int64_t y_stride, const void* h,
                                     int64_t h_stride, const void* gate, int64_t gate_stride, const void* post_w,
                                     const void* pre_w, void* h_out, void* x, void* stream) {
  NORM_CHECK(take_desc(D));
  if (D->y_type != D->io_type && D->y_type != MOE_T_F32)
    return set_last_error(MOE_ERR_INVALID_ARG, "y_type must be io_type or MOE_T_F32");
  if (D->h_type != D->io_type && D->h_type != MOE_T_F32)
    return set_last_error(MOE_ERR_INVALID_ARG, "h_type must be io_type or MOE_T_F32");
  if (D->gate_cols != 0 && D->gate_cols != 1 && D->gate_cols != D->d)
    return set_last_error(MOE_ERR_INVALID_ARG, "gate_cols must be 0, 1 or d");
  if (!std::isfinite(D->scale)) return set_last_error(MOE_ERR_INVALID_ARG, "scale must be finite");
  if (rows < 0 || rows > INT32_MAX) return set_last_error(MOE_ERR_INVALID_ARG, "rows must be in [0, 2^31)");
  if (rows == 0) return MOE_OK;
  if ((x == nullptr) != (pre_w == nullptr)) return set_last_error(MOE_ERR_INVALID_ARG, "x and pre_w go together");
  if (!x && !h_out) return set_last_error(MOE_ERR_INVALID_ARG, "neither h_out nor x");
  NORM_CHECK(take_rows(y, y_stride, D->d, "y"));
  if (h) NORM_CHECK(take_rows(h, h_stride, D->d, "h"));
  if (D->gate_cols == D->d) NORM_CHECK(take_rows(gate, gate_stride, D->d, "gate"));
  if (D->gate_cols == 1 && (!gate || gate_stride < 0)) return set_last_error(MOE_ERR_INVALID_ARG, "gate is NULL or its stride negative");
  if (mis16(post_w) || mis16(pre_w) || mis16(h_out) || mis16(x))
    return set_last_error(MOE_ERR_INVALID_ARG, "post_w, pre_w, h_out or x not 16-byte aligned");
  if (h && h == h_out && h_stride != D->d)
    return set_last_error(MOE_ERR_INVALID_ARG, "h_out may be h only when h is contiguous");
  {
    const int64_t d = D->d, ys = D->y_type == MOE_T_F32 ? 4 : 2, hs = D->h_type == MOE_T_F32 ? 4 : 2;
    const Rows in[] = {{y, rows, y_stride * ys, d * ys}, {D->gate_cols ? gate : nullptr, rows, gate_stride * 2, D->gate_cols * 2ll},
                       bytes_at(post_w, d * 2), bytes_at(pre_w, d * 2)};
    const Rows hr = {h, rows, h_stride * hs, d * hs}, to = bytes_at(h_out, rows * d * hs), xr = bytes_at(x, rows * d * 2);
    bool bad = rows_meet(hr, xr) || rows_meet(to, xr) || (h != h_out && rows_meet(hr, to));
    for (const Rows& r : in) bad = bad || rows_meet(r, to) || rows_meet(r, xr);
    if (bad) return set_last_error(MOE_ERR_INVALID_ARG, "h_out or x overlaps another tensor of the call");
  }
  BlockArgs a{};
  a.y = y;
  a.h = h;
  a.gate = gate;
  a.post_w = static_cast<const uint16_t*>(post_w);
  a.pre_w = static_cast<const uint16_t*>(pre_w);
  a.h_out = h_out;
  a.x = x;
  a.rows = rows;
  a.y_stride = y_stride;
  a.h_stride = h_stride;
  a.gate_stride = gate_stride;
  a.d = D->d;
  a.gate_cols = D->gate_cols;
  a.act = D->act;
  a.scale = D->scale;
  a.eps = D->eps;
  a.off = D->weight_offset;
  // Many rows: two pieces a thread, so that more bytes are under way and fewer warps of a row have to meet; a few are over
  // sooner with one.  (Rows of 2,048 with a gate and an fp32 stream, us with one | two pieces: 16 rows 2.7 | 3.3, 256 rows 3.3 | 3.6,
  // 1,024 rows 7.7 | 6.8, 2,048 rows 13.3 | 13.4, 12,288 rows 59.6 | 55.4; four pieces' registers leave room for half the rows: 70.)
  int v;
  share(D->d, rows >= 1024 ? 2 : 1, &a.tpr, &v);
  const int threads = a.tpr > 32 ? a.tpr : 128;
  const unsigned grid = (unsigned)((rows + threads / a.tpr - 1) / (threads / a.tpr));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool bf = D->io_type == MOE_T_BF16, yf = D->y_type == MOE_T_F32, hf = D->h_type == MOE_T_F32;
  if (bf) {
    if (yf) { if (hf) block_v<true, true, true>(a, v, grid, threads, s); else block_v<true, true, false>(a, v, grid, threads, s); }
    else { if (hf) block_v<true, false, true>(a, v, grid, threads, s); else block_v<true, false, false>(a, v, grid, threads, s); }
  } else {
    if (yf) { if (hf) block_v<false, true, true>(a, v, grid, threads, s); else block_v<false, true, false>(a, v, grid, threads, s); }
    else { if (hf) block_v<false, false, true>(a, v, grid, threads, s); else block_v<false, false, false>(a, v, grid, threads, s); }
  }
  return launched(cudaGetLastError(), "moe_norm_block");
}

extern "C" moe_status moe_norm_gated(const moe_norm_desc* D, int64_t n_tokens, int32_t n_heads, const void* o,
                                     int64_t o_stride, const void* z, int64_t z_stride, const void* w, int32_t gate_first,
                                     void* out, void* stream) {
  NORM_CHECK(take_desc(D));
  if (n_heads < 1 || n_tokens < 0 || n_tokens > INT32_MAX / n_heads)
    return set_last_error(MOE_ERR_INVALID_ARG, "n_heads must be positive and n_tokens * n_heads in [0, 2^31)");
  if (n_tokens == 0) return MOE_OK;
  const int64_t width = (int64_t)n_heads * D->d;
  NORM_CHECK(take_rows(o, o_stride, width, "o"));
  NORM_CHECK(take_rows(z, z_stride, width, "z"));
  NORM_CHECK(take_rows(out, width, width, "out"));
  if (!w || mis16(w)) return set_last_error(MOE_ERR_INVALID_ARG, "w is NULL or not 16-byte aligned");
  if (o == out && o_stride != width) return set_last_error(MOE_ERR_INVALID_ARG, "out may be o only when o is contiguous");
  {
    const Rows to = bytes_at(out, n_tokens * width * 2);
    if (rows_meet(Rows{z, n_tokens, z_stride * 2, width * 2}, to) || (o != out && rows_meet(Rows{o, n_tokens, o_stride * 2, width * 2}, to)) ||
        rows_meet(bytes_at(w, D->d * 2ll), to))
      return set_last_error(MOE_ERR_INVALID_ARG, "out overlaps another tensor of the call");
  }
  GatedArgs a{};
  a.o = static_cast<const uint16_t*>(o);
  a.z = static_cast<const uint16_t*>(z);
  a.w = static_cast<const uint16_t*>(w);
  a.out = static_cast<uint16_t*>(out);
  a.rows = n_tokens * n_heads;
  a.o_stride = o_stride;
  a.z_stride = z_stride;
  a.d = D->d;
  a.heads = n_heads;
  a.act = D->act;
  a.gate_first = gate_first != 0;
  a.eps = D->eps;
  a.off = D->weight_offset;
  int v;
  share(D->d, 1, &a.tpr, &v);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool bf = D->io_type == MOE_T_BF16;
  if (a.tpr <= 32 && a.rows >= 32768) {
    // many short rows: four to a group of threads, so that enough bytes are under way; a few are over sooner with one (rows of
    // 128, us with one | four: 256 rows 1.8 | 2.8, 16,384 rows 3.8 | 4.0, 32,768 rows 6.5 | 6.3, 393,216 rows 63.4 | 51.7)
    const int per = 128 / a.tpr * 4;
    const unsigned grid = (unsigned)((a.rows + per - 1) / per);
    if (bf) gated_kernel<true, 1, 4><<<grid, 128, 0, s>>>(a);
    else gated_kernel<false, 1, 4><<<grid, 128, 0, s>>>(a);
  } else {
    const int threads = a.tpr > 32 ? a.tpr : 128;
    const unsigned grid = (unsigned)((a.rows + threads / a.tpr - 1) / (threads / a.tpr));
    if (v == 1) {
      if (bf) gated_kernel<true, 1, 1><<<grid, threads, 0, s>>>(a);
      else gated_kernel<false, 1, 1><<<grid, threads, 0, s>>>(a);
    } else {
      if (bf) gated_kernel<true, 2, 1><<<grid, threads, 0, s>>>(a);
      else gated_kernel<false, 2, 1><<<grid, threads, 0, s>>>(a);
    }
  }
  return launched(cudaGetLastError(), "moe_norm_gated");
}
