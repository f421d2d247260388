// The short convolution and the gates in front of the gated delta rule
// (moe_delta_prepare).
//
// A thread takes 8 channels of a run of tokens and slides the last taps inputs
// along in registers, so that every input is read once (and `taps - 1` more
// where a run begins inside a sequence).  Inputs before a sequence's first
// token come from its state, which the thread that owns the sequence's first
// token alone reads and then writes: it goes on past its run while a token still
// sees the state (the run behind leaves those out), and the state's slot may
// therefore be the one it came from.
//
// Bound by issue slots (69%: eight channels' products and two special functions each) next to
// the bytes, x read and y written once: 12,288 tokens of 8,192 channels 77 us, 79% of the copy bandwidth.
#include "delta.cuh"

namespace moe {

namespace {

constexpr int kThreads = 64;

struct Vec8 {
  float x[8];
};
template <bool BF16>
__device__ __forceinline__ Vec8 unpack8(const uint4& r) {
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
  Vec8 v;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 f = unpack16<BF16>(w[e]);
    v.x[2 * e] = f.x;
    v.x[2 * e + 1] = f.y;
  }
  return v;
}
template <bool BF16>
__device__ __forceinline__ Vec8 load8(const uint16_t* p) {
  return unpack8<BF16>(*reinterpret_cast<const uint4*>(p));
}

// One sequence's tokens [i0, i1) (counted from its first), 8 channels at c.  first: the run that begins the sequence, which
// takes the state's inputs and leaves the new ones.
template <bool BF16, int TAPS>
__device__ __forceinline__ void run_of(const DeltaPrepArgs& a, const DeltaSeq& q, int i0, int i1, int c, bool first, bool writes,
                                       const float (&w)[8][TAPS], const Vec8& bias) {
  Vec8 win[TAPS];                     // the inputs of the last TAPS tokens, oldest first
  const uint16_t* x = a.x + (int64_t)q.t0 * a.x_stride + c;
  const uint16_t* old = a.conv + (int64_t)max(q.in, 0) * (TAPS - 1) * a.channels + c;
  uint4 kept[TAPS - 1];               // what a state without new inputs would be
  if (first) {
#pragma unroll
    for (int j = 0; j < TAPS - 1; ++j)
      kept[j] = q.in >= 0 ? *reinterpret_cast<const uint4*>(old + (int64_t)j * a.channels) : make_uint4(0, 0, 0, 0);
  }
#pragma unroll
  for (int j = 1; j < TAPS; ++j) {    // input of token i0 - TAPS + j
    if (first) {
      win[j] = unpack8<BF16>(kept[j - 1]);
    } else {
      win[j] = load8<BF16>(x + (int64_t)(i0 - TAPS + j) * a.x_stride);
    }
  }
  if (first && writes) {
    // the state's new inputs, before any token is overwritten elsewhere: y is not x
    uint16_t* to = a.conv + (int64_t)q.out * (TAPS - 1) * a.channels + c;
#pragma unroll
    for (int j = 0; j < TAPS - 1; ++j) {
      const int i = q.n - (TAPS - 1) + j;
      uint4 r;
      if (i >= 0) {
        r = *reinterpret_cast<const uint4*>(x + (int64_t)i * a.x_stride);
      } else {                        // kept[j + n], n < TAPS - 1 (with four taps in a stack frame of 48 bytes)
        r = kept[0];
#pragma unroll
        for (int m = 1; m < TAPS - 1; ++m)
          if (TAPS - 1 + i == m) r = kept[m];
      }
      *reinterpret_cast<uint4*>(to + (int64_t)j * a.channels) = r;
    }
  }
  // four tokens' inputs go ahead of the four that are summed
  auto fetch = [&](int i, uint4 (&r)[4]) {
#pragma unroll
    for (int y = 0; y < 4; ++y)
      if (i + y < i1) r[y] = *reinterpret_cast<const uint4*>(x + (int64_t)(i + y) * a.x_stride);
  };
  uint4 next[4];
  fetch(i0, next);
#pragma unroll 1
  for (int i = i0; i < i1; i += 4) {
    const uint4 now[4] = {next[0], next[1], next[2], next[3]};
    fetch(i + 4, next);
#pragma unroll
    for (int y = 0; y < 4; ++y) {
      if (i + y >= i1) break;
#pragma unroll
      for (int j = 0; j < TAPS - 1; ++j) win[j] = win[j + 1];
      win[TAPS - 1] = unpack8<BF16>(now[y]);
      float o[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        float z = bias.x[e];
#pragma unroll
        for (int j = 0; j < TAPS; ++j) z += w[e][j] * win[j].x[e];
        o[e] = z * logistic(z);
      }
      *reinterpret_cast<uint4*>(a.y + (int64_t)(q.t0 + i + y) * a.channels + c) =
          make_uint4(pack16<BF16>(o[0], o[1]), pack16<BF16>(o[2], o[3]), pack16<BF16>(o[4], o[5]), pack16<BF16>(o[6], o[7]));
    }
  }
}

// Blocks: `runs` runs of `run` tokens, gx blocks of 8 * kThreads channels each; then the sequences without tokens, 32 at a
// time (gx blocks each; with the gates alone one each, which looks at all of them); then the gates, a thread per token and head.
template <bool BF16, int TAPS>
__global__ void __launch_bounds__(kThreads, 8) prepare_kernel(const __grid_constant__ DeltaPrepArgs a, int run, int runs, int empties, int gx) {
  const int64_t conv_blocks = (int64_t)(runs + empties) * gx;
  if (blockIdx.x >= conv_blocks) {
    const int64_t i = (blockIdx.x - conv_blocks) * kThreads + threadIdx.x;
    if (i >= (int64_t)a.b.n_tokens * a.hv) return;
    const int t = (int)(i / a.hv), h = (int)(i - (int64_t)t * a.hv), s = delta_seq_from(a.b, t);
    if (s == a.b.n_seqs || a.b.cu[s] > t) return;
    const float z = load16<BF16>(a.a + t * a.ab_stride + h) + a.dt_bias[h], b = load16<BF16>(a.gb + t * a.ab_stride + h);
    // softplus without overflow: max(z, 0) + log(1 + e^-|z|); a NaN stays one
    a.g[i] = -expf(a.a_log[h]) * (fmaxf(z, 0.f) + log1pf(expf(-fabsf(z))));
    a.beta[i] = 1.f / (1.f + expf(-b));
    return;
  }
  int y = blockIdx.x / gx;
  const int c = ((blockIdx.x - y * gx) * kThreads + threadIdx.x) * 8;
  const bool live = c < a.channels;
  if (y < runs) {                     // the convolution
    const int t0 = y * run, t1 = min(t0 + run, a.b.n_tokens);
    float w[8][TAPS];
    Vec8 bias;
    if (live) {
      const uint32_t* p = reinterpret_cast<const uint32_t*>(a.w + (int64_t)c * TAPS);
      float f[8 * TAPS];
#pragma unroll
      for (int e = 0; e < 4 * TAPS; ++e) {
        const float2 v = unpack16<BF16>(p[e]);
        f[2 * e] = v.x;
        f[2 * e + 1] = v.y;
      }
#pragma unroll
      for (int e = 0; e < 8; ++e)
#pragma unroll
        for (int j = 0; j < TAPS; ++j) w[e][j] = f[e * TAPS + j];
      if (a.bias) {
        bias = load8<BF16>(a.bias + c);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) bias.x[e] = 0.f;
      }
    }
    for (int s = delta_seq_from(a.b, t0); s < a.b.n_seqs && a.b.cu[s] < t1; ++s) {
      const DeltaSeq q = delta_seq(a.b, s);
      if (q.n == 0 || q.t0 >= t1 || q.t0 + q.n <= t0) continue;
      const int b = t0 - q.t0;        // this run's first token, counted from the sequence's
      const bool first = b <= 0;
      const int i0 = first ? 0 : max(b, min(q.n, TAPS - 1)), i1 = min(q.n, first ? max(t1 - q.t0, TAPS - 1) : t1 - q.t0);
      const bool writes = first && __syncthreads_and(delta_writes(a.b, s, q, threadIdx.x, kThreads));
      if (live && i0 < i1) run_of<BF16, TAPS>(a, q, i0, i1, c, first, writes, w, bias);
    }
    return;
  }
  y -= runs;
  if (!a.conv_on) {                   // the gates alone touch no slot, but offsets out of range are reported all the same
    const int s = y * 32 + threadIdx.x;
    if (threadIdx.x < 32 && s < a.b.n_seqs) {
      const int from = a.b.cu[s], to = a.b.cu[s + 1];
      if (from < 0 || to < from || to > a.b.n_tokens) atomicOr(a.b.err, (uint32_t)DELTA_BAD_LEN);
    }
    return;
  }
  // sequences without tokens carry their state over
  for (int s = y * 32; s < min(a.b.n_seqs, (y + 1) * 32); ++s) {
    if (a.b.cu[s + 1] > a.b.cu[s] && a.b.cu[s] >= 0 && a.b.cu[s] < a.b.n_tokens) continue;
    const DeltaSeq q = delta_seq(a.b, s);
    if (q.n > 0 || !__syncthreads_and(delta_writes(a.b, s, q, threadIdx.x, kThreads)) || !live) continue;
#pragma unroll
    for (int j = 0; j < TAPS - 1; ++j) {
      const uint4 r = q.in >= 0 ? *reinterpret_cast<const uint4*>(a.conv + ((int64_t)q.in * (TAPS - 1) + j) * a.channels + c)
                                : make_uint4(0, 0, 0, 0);
      *reinterpret_cast<uint4*>(a.conv + ((int64_t)q.out * (TAPS - 1) + j) * a.channels + c) = r;
    }
  }
}

template <bool BF16, int TAPS>
cudaError_t launch(const DeltaPrepArgs& a, cudaStream_t s, int num_sms) {
  int run = 1, runs = 0, gx = 1;
  if (a.conv_on) {
    gx = (a.channels / 8 + kThreads - 1) / kThreads;
    // (12,288 tokens of 8,192 channels: runs of 8 to 128 tokens 124, 93, 80, 76, 90 us)
    while (run < 64 && (int64_t)a.b.n_tokens * gx > (int64_t)num_sms * 32 * run) run *= 2;
    runs = (a.b.n_tokens + run - 1) / run;
  }
  const int empties = (a.b.n_seqs + 31) / 32;
  int64_t blocks = (int64_t)(runs + empties) * gx;
  if (a.gates_on) blocks += ((int64_t)a.b.n_tokens * a.hv + kThreads - 1) / kThreads;
  if (blocks > 0) prepare_kernel<BF16, TAPS><<<(unsigned)blocks, kThreads, 0, s>>>(a, run, runs, empties, gx);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_delta_prepare(const DeltaPrepArgs& a, int io, cudaStream_t s, int num_sms) {
  if (io == MOE_T_BF16)
    return a.taps == 4 ? launch<true, 4>(a, s, num_sms) : a.taps == 3 ? launch<true, 3>(a, s, num_sms) : launch<true, 2>(a, s, num_sms);
  return a.taps == 4 ? launch<false, 4>(a, s, num_sms) : a.taps == 3 ? launch<false, 3>(a, s, num_sms) : launch<false, 2>(a, s, num_sms);
}

}  // namespace moe
