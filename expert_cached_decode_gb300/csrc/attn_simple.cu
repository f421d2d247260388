// The accumulated weights in their plainest form: one thread per cell.
#include "attn.cuh"

namespace moe {

namespace {

// element e of head vector h (K heads, then V heads) of a cell
template <bool BF16, bool I8>
__device__ __forceinline__ float cell_value(const uint8_t* cell, int hkv, int D, int h, int e) {
  if (I8)
    return (float)reinterpret_cast<const int8_t*>(cell)[h * D + e] *
           reinterpret_cast<const float*>(cell + (size_t)2 * hkv * D)[h];
  const uint32_t u = reinterpret_cast<const uint16_t*>(cell)[h * D + e];
  return Half16<BF16>::unpack(u).x;
}

template <bool BF16, int D, bool I8>
__global__ void __launch_bounds__(128) weights_simple_kernel(const __grid_constant__ AttnWgtArgs a) {
  __shared__ float q[D];
  const int s = blockIdx.y, j = blockIdx.x * 128 + threadIdx.x;
  const SeqInfo si = seq_info(a.b, s);
  if ((int)blockIdx.x * 128 >= si.len) return;
  const uint8_t* c = j < si.len ? cell_ptr(a.b, s, j) : nullptr;
  float sum = 0.f;
  for (int h = 0; h < a.g.hq; ++h) {
    float k[D];
    for (int e = 0; e < D; ++e) k[e] = c ? cell_value<BF16, I8>(c, a.g.hkv, D, h / a.g.g, e) : 0.f;
    for (int i = 0; i < si.n; ++i) {
      int lo, hi;
      row_range(si, a.b.window, i, lo, hi);
      if (hi <= (int)blockIdx.x * 128 || lo >= (int)blockIdx.x * 128 + 128) continue;
      const int64_t t = si.q0 + i;
      __syncthreads();
      if (threadIdx.x < D) q[threadIdx.x] = Half16<BF16>::unpack(a.q[t * a.q_stride + h * D + threadIdx.x]).x * a.g.scale_log2;
      __syncthreads();
      const float lse = a.lse[t * a.g.hq + h];
      float x = 0.f;
      for (int e = 0; e < D; ++e) x += q[e] * k[e];
      if (c && j >= lo && j < hi && lse != -INFINITY) sum += exp2f(x - lse * 1.4426950408889634f);
    }
  }
  if (j < si.len && j < a.max_kv) {
    const int64_t at = (int64_t)s * a.acc_stride + j;
    a.acc_out[at] = (a.acc_in ? a.acc_in[at] * a.decay : 0.f) + sum;
  }
}

}  // namespace

#define ATTN_BY_TYPE(CALL)                                             \
  do {                                                                 \
    const bool bf = a.g.io == MOE_T_BF16, i8 = a.g.kv == MOE_T_I8;     \
    if (a.g.D == 128) {                                                \
      if (bf) { if (i8) CALL(true, 128, true); else CALL(true, 128, false); }      \
      else { if (i8) CALL(false, 128, true); else CALL(false, 128, false); }       \
    } else {                                                           \
      if (bf) { if (i8) CALL(true, 64, true); else CALL(true, 64, false); }        \
      else { if (i8) CALL(false, 64, true); else CALL(false, 64, false); }         \
    }                                                                  \
  } while (0)

cudaError_t launch_attn_weights(const AttnWgtArgs& a, int max_q, cudaStream_t s) {
  if ((int64_t)max_q * a.g.g <= 32) return launch_attn_weights_rows(a, max_q, s);
  const dim3 grid((a.max_kv + 127) / 128, a.b.n_seqs);
#define CALL(BF, DD, I) weights_simple_kernel<BF, DD, I><<<grid, 128, 0, s>>>(a)
  ATTN_BY_TYPE(CALL);
#undef CALL
  return cudaGetLastError();
}

}  // namespace moe
