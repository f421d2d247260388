// The gated delta rule token by token: single tokens, drafts, short prompts.
//
// A warp keeps 8 columns of a head's state S [k_dim][8] in registers: lane l
// holds the columns 4 (l & 1) .. + 3 of the rows l / 2, l / 2 + 16, ..., so that a
// load takes whole 32-byte sectors and no two warps ever have to meet.  A token
// then is
//     a = S^T k^, c = S^T q^        (one pass over the registers, both at once)
//     u = beta (v - e^g a), o = scale (e^g c + (q^.k^) u)
//     S = e^g S + k^ u^T
// with the sums over the 16 groups of rows by shuffles.  o needs no second pass
// over the new state: S^T q^ is e^g c + (q^.k^) u.
//
// Bound by the states' bytes: they are read and written once a call.
#include "delta.cuh"

namespace moe {

namespace {

constexpr int kWarps = 4, kThreads = 32 * kWarps;   // a CTA takes 32 columns
constexpr int kBatch = 8;                           // tokens staged at a time

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

template <bool BF16, int DK>
__global__ void __launch_bounds__(kThreads) steps_kernel(const __grid_constant__ DeltaFwdArgs a) {
  constexpr int R = DK / 16;          // rows of a lane
  __shared__ float ks[kBatch][DK], qs[kBatch][DK];
  __shared__ float qk[kBatch];
  const int s = blockIdx.z, h = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int dv = a.geo.dv, hv = a.geo.hv, c0 = blockIdx.x * 32 + warp * 8 + 4 * (lane & 1), r0 = lane >> 1;
  const DeltaSeq q = delta_seq(a.b, s);
  if (q.n < a.n_min || q.n > a.n_max) return;
  if (q.n == 0 && (q.in == q.out || q.out < 0)) return;
  float4 S[R];
  if (q.in >= 0) {
    const float* src = a.state + (((int64_t)q.in * hv + h) * DK + r0) * dv + c0;
#pragma unroll
    for (int i = 0; i < R; ++i) S[i] = __ldcs(reinterpret_cast<const float4*>(src + (int64_t)16 * i * dv));
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
        x[0][e] *= f[0];
        x[1][e] *= f[1];
        dot += x[0][e] * x[1][e];
        ks[i][lane * E + e] = x[0][e];
        qs[i][lane * E + e] = x[1][e];
      }
      dot = warp_sum(dot);
      if (lane == 0) qk[i] = dot;
    }
    __syncthreads();
    for (int i = 0; i < nb; ++i) {
      const int64_t t = q.t0 + i0 + i;
      const float decay = expf(a.g[t * hv + h]), beta = a.beta[t * hv + h];
      const uint2 vw = *reinterpret_cast<const uint2*>(a.v + t * a.v_stride + h * dv + c0);
      float kr[R];
      float av[4] = {0.f, 0.f, 0.f, 0.f}, cv[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int r = 0; r < R; ++r) {
        kr[r] = ks[i][r0 + 16 * r];
        const float qr = qs[i][r0 + 16 * r];
        av[0] += S[r].x * kr[r];
        av[1] += S[r].y * kr[r];
        av[2] += S[r].z * kr[r];
        av[3] += S[r].w * kr[r];
        cv[0] += S[r].x * qr;
        cv[1] += S[r].y * qr;
        cv[2] += S[r].z * qr;
        cv[3] += S[r].w * qr;
      }
#pragma unroll
      for (int o = 16; o > 1; o >>= 1)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          av[e] += __shfl_xor_sync(0xffffffffu, av[e], o);
          cv[e] += __shfl_xor_sync(0xffffffffu, cv[e], o);
        }
      const float2 v0 = unpack16<BF16>(vw.x), v1 = unpack16<BF16>(vw.y);
      const float v[4] = {v0.x, v0.y, v1.x, v1.y};
      float u[4], o[4];
      const float d = qk[i];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        u[e] = beta * (v[e] - decay * av[e]);
        o[e] = a.geo.scale * (decay * cv[e] + d * u[e]);
      }
      if (r0 == 0)
        *reinterpret_cast<uint2*>(a.out + (t * hv + h) * dv + c0) =
            make_uint2(pack16<BF16>(o[0], o[1]), pack16<BF16>(o[2], o[3]));
#pragma unroll
      for (int r = 0; r < R; ++r) {
        S[r].x = decay * S[r].x + kr[r] * u[0];
        S[r].y = decay * S[r].y + kr[r] * u[1];
        S[r].z = decay * S[r].z + kr[r] * u[2];
        S[r].w = decay * S[r].w + kr[r] * u[3];
      }
    }
  }
  if (!writes) return;
  float* dst = a.state + (((int64_t)q.out * hv + h) * DK + r0) * dv + c0;
#pragma unroll
  for (int i = 0; i < R; ++i) __stcs(reinterpret_cast<float4*>(dst + (int64_t)16 * i * dv), S[i]);
}

}  // namespace

cudaError_t launch_delta_steps(const DeltaFwdArgs& a, cudaStream_t s) {
  const dim3 grid(a.geo.dv / 32, a.geo.hv, a.b.n_seqs);
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
