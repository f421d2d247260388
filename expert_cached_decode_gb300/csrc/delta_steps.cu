// The gated delta rule token by token: single tokens, drafts, short prompts.
//
// A warp keeps 32 columns of a head's state S [k_dim][32] in registers: lane l
// holds the columns 4 (l & 7) .. + 3 of the rows l / 8, l / 8 + 4, ..., so that a
// load takes whole 128-byte lines and no two warps have to meet.  A token is
//     a = S^T k^, c = S^T q^        (one pass over the registers, both at once)
//     u = beta (v - e^g a), o = scale (e^g c + (q^.k^) u)
//     S = e^g S + k^ u^T
// with the sums over the four groups of rows by shuffles.  o needs no second pass
// over the new state: S^T q^ is e^g c + (q^.k^) u.  The tokens' keys and queries
// (normed), decays and values are brought to shared memory eight tokens at a
// time, under way together with the state.
//
// Bound by the states' bytes, which are read and written once a call: 64 sequences' token
// (32 heads of 128 x 128, 268 MB) 43 us, 93% of the copy bandwidth; with 8
// columns a warp, in 32-byte pieces of lines, 51 us.  One sequence's token takes 3.2 us, five
// tokens of eight sequences 11.5: latency.
#include "delta.cuh"

namespace moe {

namespace {

constexpr int kWarps = 2, kThreads = 32 * kWarps;   // a CTA takes 64 columns
constexpr int kBatch = 8;                           // tokens staged at a time

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

template <bool BF16, int DK>
__global__ void __launch_bounds__(kThreads) steps_kernel(const __grid_constant__ DeltaFwdArgs a) {
  constexpr int R = DK / 4, LD = R + 4;   // rows of a lane; from one group of rows to the next
  // element 4 i + r of a key or a query lies at [r][i], so that a lane reads four of its rows at a time
  __shared__ __align__(16) float ks[kBatch][4 * LD], qs[kBatch][4 * LD], vs[kBatch][32 * kWarps];
  __shared__ float qk[kBatch], decay[kBatch], beta[kBatch];
  const int s = blockIdx.z, h = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int dv = a.geo.dv, hv = a.geo.hv, col = blockIdx.x * 64 + warp * 32 + 4 * (lane & 7), rg = lane >> 3;
  const DeltaSeq q = delta_seq(a.b, s);
  if (q.n < a.n_min || q.n > a.n_max) return;
  if (q.n == 0 && (q.in == q.out || q.out < 0)) return;
  float4 S[R];
  if (q.in >= 0) {
    const float* src = a.state + (((int64_t)q.in * hv + h) * DK + rg) * dv + col;
#pragma unroll
    for (int i = 0; i < R; ++i) S[i] = __ldcs(reinterpret_cast<const float4*>(src + (int64_t)4 * i * dv));
  } else {
#pragma unroll
    for (int i = 0; i < R; ++i) S[i] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  const bool writes = __syncthreads_and(delta_writes(a.b, s, q, threadIdx.x, kThreads));
  for (int i0 = 0; i0 < q.n; i0 += kBatch) {
    const int nb = min(kBatch, q.n - i0);
    if (i0) __syncthreads();
    // a warp stages a token's key and query, in 32 bits and normed
    for (int i = warp; i < nb; i += kWarps) {
      constexpr int E = DK / 32;      // elements of a lane, next to each other
      const int64_t t = q.t0 + i0 + i;
      const float g = a.g[t * hv + h], b = a.beta[t * hv + h];
      const uint32_t v = *reinterpret_cast<const uint32_t*>(a.v + t * a.v_stride + h * dv + blockIdx.x * 64 + 2 * lane);
      float x[2][E], ss[2] = {0.f, 0.f}, dot = 0.f;
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        const uint16_t* p = (w ? a.q + t * a.q_stride : a.k + t * a.k_stride) + h / a.geo.rep * DK + lane * E;
#pragma unroll
        for (int e = 0; e < E; e += 2) {
          const float2 f = unpack16<BF16>(*reinterpret_cast<const uint32_t*>(p + e));
          x[w][e] = f.x;
          x[w][e + 1] = f.y;
        }
#pragma unroll
        for (int e = 0; e < E; ++e) ss[w] += x[w][e] * x[w][e];
      }
      float f[2] = {1.f, 1.f};
      if (a.geo.normalize) {
        f[0] = rsqrtf(warp_sum(ss[0]) + a.geo.eps);
        f[1] = rsqrtf(warp_sum(ss[1]) + a.geo.eps);
      }
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const int r = lane * E + e, at = (r & 3) * LD + (r >> 2);
        x[0][e] *= f[0];
        x[1][e] *= f[1];
        dot += x[0][e] * x[1][e];
        ks[i][at] = x[0][e];
        qs[i][at] = x[1][e];
      }
      *reinterpret_cast<float2*>(&vs[i][2 * lane]) = unpack16<BF16>(v);
      dot = warp_sum(dot);
      if (lane == 0) {
        qk[i] = dot;
        decay[i] = expf(g);
        beta[i] = b;
      }
    }
    __syncthreads();
#pragma unroll 1
    for (int i = 0; i < nb; ++i) {
      const int64_t t = q.t0 + i0 + i;
      const float d = decay[i], b = beta[i], dot = qk[i];
      const float4 v4 = *reinterpret_cast<const float4*>(&vs[i][warp * 32 + 4 * (lane & 7)]);
      float av[4] = {0.f, 0.f, 0.f, 0.f}, cv[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int r = 0; r < R; r += 4) {
        const float4 k4 = *reinterpret_cast<const float4*>(&ks[i][rg * LD + r]), q4 = *reinterpret_cast<const float4*>(&qs[i][rg * LD + r]);
        const float kk[4] = {k4.x, k4.y, k4.z, k4.w}, qq[4] = {q4.x, q4.y, q4.z, q4.w};
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          av[0] += S[r + y].x * kk[y];
          av[1] += S[r + y].y * kk[y];
          av[2] += S[r + y].z * kk[y];
          av[3] += S[r + y].w * kk[y];
          cv[0] += S[r + y].x * qq[y];
          cv[1] += S[r + y].y * qq[y];
          cv[2] += S[r + y].z * qq[y];
          cv[3] += S[r + y].w * qq[y];
        }
      }
#pragma unroll
      for (int o = 8; o <= 16; o <<= 1)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          av[e] += __shfl_xor_sync(0xffffffffu, av[e], o);
          cv[e] += __shfl_xor_sync(0xffffffffu, cv[e], o);
        }
      const float v[4] = {v4.x, v4.y, v4.z, v4.w};
      float u[4], o[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        u[e] = b * (v[e] - d * av[e]);
        o[e] = a.geo.scale * (d * cv[e] + dot * u[e]);
      }
      if (rg == 0)
        *reinterpret_cast<uint2*>(a.out + (t * hv + h) * dv + col) = make_uint2(pack16<BF16>(o[0], o[1]), pack16<BF16>(o[2], o[3]));
#pragma unroll
      for (int r = 0; r < R; r += 4) {
        const float4 k4 = *reinterpret_cast<const float4*>(&ks[i][rg * LD + r]);
        const float kk[4] = {k4.x, k4.y, k4.z, k4.w};
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          S[r + y].x = d * S[r + y].x + kk[y] * u[0];
          S[r + y].y = d * S[r + y].y + kk[y] * u[1];
          S[r + y].z = d * S[r + y].z + kk[y] * u[2];
          S[r + y].w = d * S[r + y].w + kk[y] * u[3];
        }
      }
    }
  }
  if (!writes) return;
  float* dst = a.state + (((int64_t)q.out * hv + h) * DK + rg) * dv + col;
#pragma unroll
  for (int i = 0; i < R; ++i) __stcs(reinterpret_cast<float4*>(dst + (int64_t)4 * i * dv), S[i]);
}

}  // namespace

cudaError_t launch_delta_steps(const DeltaFwdArgs& a, cudaStream_t s) {
  const dim3 grid(a.geo.dv / 64, a.geo.hv, a.b.n_seqs);
  const bool bf = a.geo.io == MOE_T_BF16;
  if (a.geo.dk == 128) {
    if (bf) steps_kernel<true, 128><<<grid, kThreads, 0, s>>>(a);
    else steps_kernel<false, 128><<<grid, kThreads, 0, s>>>(a);
  } else {
    if (bf) steps_kernel<true, 64><<<grid, kThreads, 0, s>>>(a);
    else steps_kernel<false, 64><<<grid, kThreads, 0, s>>>(a);
  }
  return cudaGetLastError();
}

}  // namespace moe
