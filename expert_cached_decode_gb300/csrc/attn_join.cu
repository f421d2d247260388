// Joins the parts of the items that the attention kernels cut: the rows'
// sums, each relative to its part's maximum, in the order of the parts.
// Launched after either kernel with programmatic dependence, so its blocks
// are in place when the last part is written.  Bound by latency (a call on 300
// cells takes 9 us, both launches).
#include "attn.cuh"

namespace moe {

namespace {

// Block (c, y): rows [RB y, RB y + RB) of the cut item that begins in CTA c.  W warps share a row's parts (part k goes
// to warp k % W, five or eight loads in flight each) and join through shared memory.
template <bool BF16, int D, int RB, int W>
__global__ void __launch_bounds__(RB * W * 32) join_kernel(const __grid_constant__ AttnFwdArgs a, int rows) {
  constexpr int V = D / 32;            // elements per lane
  __shared__ float sm_m[RB][W], sm_l[RB][W];
  __shared__ float sm_o[RB][W][D];
  pdl_wait();
  const AttnCut cut = a.cuts[blockIdx.x];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, rr = warp / W, w = warp % W;
  const int r = blockIdx.y * RB + rr;
  if ((int)blockIdx.y * RB >= cut.nrows || cut.parts == 0) return;
  const bool real = r < cut.nrows;
  const float* first = a.ws + ((int64_t)blockIdx.x * 2 + 1) * a.ws_slot;
  float M = -INFINITY, L = 0.f, acc[V] = {};
  constexpr int kAt = W > 1 ? 5 : 8;
  for (int k0 = w; real && k0 < cut.parts; k0 += kAt * W) {
    float m[kAt], l[kAt], x[kAt][V];
#pragma unroll
    for (int k = 0; k < kAt; ++k) {
      const int p = k0 + k * W;
      const bool in = p < cut.parts;
      // part 0 in slot 1 of CTA c, part p in slot 0 of CTA c + p
      const float* pw = first + (in && p ? (2 * (int64_t)p - 1) * a.ws_slot : 0);
      m[k] = in ? __ldcg(pw + (int64_t)rows * D + r) : -INFINITY;
      l[k] = in ? __ldcg(pw + (int64_t)rows * (D + 1) + r) : 0.f;
      if (V == 4) {
        const float4 v = __ldcg(reinterpret_cast<const float4*>(pw + r * D) + lane);
        x[k][0] = v.x;
        x[k][1] = v.y;
        x[k][V > 2 ? 2 : 0] = v.z;
        x[k][V > 2 ? 3 : 0] = v.w;
      } else {
        const float2 v = __ldcg(reinterpret_cast<const float2*>(pw + r * D) + lane);
        x[k][0] = v.x;
        x[k][1] = v.y;
      }
    }
    float top = M;
#pragma unroll
    for (int k = 0; k < kAt; ++k) top = fmaxf(top, m[k]);
    const float f0 = M == top ? 1.f : ex2(M - top);
    M = top;
    L *= f0;
#pragma unroll
    for (int e = 0; e < V; ++e) acc[e] *= f0;
#pragma unroll
    for (int k = 0; k < kAt; ++k) {
      // a part that saw no cell (or is not there) has the maximum -inf
      const float f = m[k] == -INFINITY ? 0.f : m[k] == M ? 1.f : ex2(m[k] - M);
      L += f * l[k];
#pragma unroll
      for (int e = 0; e < V; ++e) acc[e] += f == 0.f ? 0.f : f * x[k][e];
    }
  }
  if (W > 1) {
    if (lane == 0) {
      sm_m[rr][w] = M;
      sm_l[rr][w] = L;
    }
#pragma unroll
    for (int e = 0; e < V; ++e) sm_o[rr][w][V * lane + e] = acc[e];
    __syncthreads();
    if (w != 0) return;
    const float m0 = M;
#pragma unroll
    for (int k = 1; k < W; ++k) M = fmaxf(M, sm_m[rr][k]);
    const float f0 = m0 == M ? 1.f : ex2(m0 - M);
    L *= f0;
#pragma unroll
    for (int e = 0; e < V; ++e) acc[e] *= f0;
#pragma unroll
    for (int k = 1; k < W; ++k) {
      const float f = sm_m[rr][k] == -INFINITY ? 0.f : sm_m[rr][k] == M ? 1.f : ex2(sm_m[rr][k] - M);
      L += f * sm_l[rr][k];
#pragma unroll
      for (int e = 0; e < V; ++e) acc[e] += f * sm_o[rr][k][V * lane + e];
    }
  }
  if (!real) return;
  const float inv = L > 0.f ? 1.f / L : (L == 0.f ? 0.f : L);
  const int i = (int)fdiv((uint32_t)(cut.r0 + r), a.g.gdiv);
  const int64_t at = (int64_t)(cut.q0 + i) * a.g.hq + cut.h * a.g.g + (cut.r0 + r - i * a.g.g);
  if (V == 4)
    *(reinterpret_cast<uint2*>(a.out + at * D) + lane) =
        make_uint2(Half16<BF16>::pack(acc[0] * inv, acc[1] * inv),
                   Half16<BF16>::pack(acc[V > 2 ? 2 : 0] * inv, acc[V > 2 ? 3 : 0] * inv));
  else
    *(reinterpret_cast<uint32_t*>(a.out + at * D) + lane) = Half16<BF16>::pack(acc[0] * inv, acc[1] * inv);
  if (lane == 0 && a.lse) a.lse[at] = L == 0.f ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
}

template <bool BF16, int D, int RB, int W>
cudaError_t launch(const AttnFwdArgs& a, int rows, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.num_sms, rows / RB);
  cfg.blockDim = dim3(RB * W * 32);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, join_kernel<BF16, D, RB, W>, a, rows);
}

}  // namespace

// Few rows: their parts are many (a long cache over the whole GPU), so several warps share a row; many rows: one each.
cudaError_t launch_attn_join(const AttnFwdArgs& a, int rows, cudaStream_t s) {
  const bool few = rows <= 32, bf = a.g.io == MOE_T_BF16;
#define JOIN(BF, DD) return few ? launch<BF, DD, 2, 8>(a, rows, s) : launch<BF, DD, 16, 1>(a, rows, s)
  if (a.g.D == 128) {
    if (bf) JOIN(true, 128);
    JOIN(false, 128);
  }
  if (bf) JOIN(true, 64);
  JOIN(false, 64);
#undef JOIN
}

}  // namespace moe
