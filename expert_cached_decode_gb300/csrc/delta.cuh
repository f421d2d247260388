// Shared by the kernels of the gated delta rule (delta_*.cu): the call's
// sequences, their state slots, and the kernels' arguments.
#pragma once

#include "common.cuh"
#include "delta_plan.h"
#include "internal.h"

namespace moe {

// Bits of a handle's error word.
enum DeltaErr : uint32_t {
  DELTA_BAD_SLOT = 1,    // a slot outside [-1, n_slots)
  DELTA_BAD_LEN = 2,     // offsets that fall or pass n_tokens
  DELTA_TIMEOUT = 4,     // a bounded device wait gave up
  DELTA_CLASH = 8,       // a slot that one sequence writes and another reads or writes
};

struct DeltaBatch {
  const int32_t *cu, *slots_in, *slots_out;
  uint32_t* err;
  int32_t n_seqs, n_tokens, n_slots;
};

struct DeltaSeq {
  int32_t t0, n;             // first token, tokens
  int32_t in, out;           // slots, -1: none
};

// Sequence s with its values cut to their ranges (and reported when they were not in them).
__device__ __forceinline__ DeltaSeq delta_seq(const DeltaBatch& b, int s) {
  const int a = b.cu[s], e = b.cu[s + 1], i = b.slots_in[s], o = b.slots_out[s];
  DeltaSeq q;
  q.t0 = min(max(a, 0), b.n_tokens);
  q.n = min(max(e, q.t0), b.n_tokens) - q.t0;
  q.in = i >= 0 && i < b.n_slots ? i : -1;
  q.out = o >= 0 && o < b.n_slots ? o : -1;
  uint32_t bad = 0;
  if (q.t0 != a || q.t0 + q.n != e) bad |= DELTA_BAD_LEN;
  if ((q.in != i && i != -1) || (q.out != o && o != -1)) bad |= DELTA_BAD_SLOT;
  if (bad) atomicOr(b.err, bad);
  return q;
}

// Whether sequence s' keeps slot `out` from being written by sequence s: it reads it, or is an earlier one that writes it.
// (Sequences without tokens whose two slots are the same neither read nor write.)
__device__ __forceinline__ bool delta_clash(const DeltaBatch& b, int s, int out, int other) {
  if (other == s) return false;
  const int i = b.slots_in[other], o = b.slots_out[other];
  if (i != out && (o != out || other > s)) return false;
  return i != o || b.cu[other + 1] > b.cu[other];
}

// Whether slot q.out may be written, found by the threads t = 0 .. nt - 1 that share the work: true in each of them that
// saw no clash.
__device__ __forceinline__ bool delta_writes(const DeltaBatch& b, int s, const DeltaSeq& q, int t, int nt) {
  if (q.out < 0 || (q.n == 0 && q.in == q.out)) return false;
  for (int o = t; o < b.n_seqs; o += nt)
    if (delta_clash(b, s, q.out, o)) {
      atomicOr(b.err, (uint32_t)DELTA_CLASH);
      return false;
    }
  return true;
}

// The first sequence that ends behind token t (n_seqs: none does); cu ascending.
__device__ __forceinline__ int delta_seq_from(const DeltaBatch& b, int t) {
  int lo = 0, hi = b.n_seqs;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (b.cu[mid + 1] > t) hi = mid;
    else lo = mid + 1;
  }
  return lo;
}

// 16-bit element types: two values of a word, the first in the low half
template <bool BF16>
__device__ __forceinline__ float2 unpack16(uint32_t u) {
  if constexpr (BF16) return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
  else return __half22float2(*reinterpret_cast<const __half2*>(&u));
}
template <bool BF16>
__device__ __forceinline__ uint32_t pack16(float a, float b) {
  uint32_t d;
  if constexpr (BF16) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(b), "f"(a));
  else asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(b), "f"(a));
  return d;
}
template <bool BF16>
__device__ __forceinline__ float load16(const uint16_t* p) {
  if constexpr (BF16) return __uint_as_float((uint32_t)*p << 16);
  else return __half2float(*reinterpret_cast<const __half*>(p));
}

// 1 / (1 + t), t = e^-z: by quarters, so that the reciprocal stays a normal number (those below 2^-126 would come as 0)
__device__ __forceinline__ float logistic_of(float t) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(fmaf(t, 0.25f, 0.25f)));
  return 0.25f * y;
}
// 1 / (1 + e^-z) for results that are rounded to 16 bits: to 3 units of fp32's last place from z = 0 on, below it with the
// error of the exponent's product, some |z| units (2^-17 at -88).  e^-z beyond fp32's range (z below -88.7) gives 0.
__device__ __forceinline__ float logistic(float z) {
  float t;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(t) : "f"(z * -1.44269504f));
  return logistic_of(t);
}
// The same for results in fp32, to 5 units: the exponent's product with what its rounding left out
__device__ __forceinline__ float logistic32(float z) {
  float c, t;                        // z brought into [-256, 256] with its sign; a NaN stays one
  asm("min.NaN.xorsign.abs.f32 %0, %1, %2;" : "=f"(c) : "f"(z), "f"(256.f));
  const float p = c * -1.44269502f, rest = fmaf(c, -1.92596303e-8f, fmaf(c, -1.44269502f, -p));
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(t) : "f"(p));
  return logistic_of(t * fmaf(rest, 0.693147181f, 1.f));
}

struct DeltaGeo {
  int hk, hv, rep;                // rep = hv / hk
  int dk, dv, io, taps, normalize;
  float eps, scale;
};

struct DeltaPrepArgs {
  DeltaBatch b;
  const uint16_t *x, *w, *bias, *a, *gb;   // gb: the gates' b
  int64_t x_stride, ab_stride;
  uint16_t *conv, *y;
  const float *a_log, *dt_bias;
  float *g, *beta;
  int channels, hv, taps;
  bool conv_on, gates_on;
};
cudaError_t launch_delta_prepare(const DeltaPrepArgs& a, int io, cudaStream_t s, int num_sms);

struct DeltaFwdArgs {
  DeltaBatch b;
  const uint16_t *q, *k, *v;
  int64_t q_stride, k_stride, v_stride;
  const float *g, *beta;
  float* state;
  uint16_t* out;
  DeltaGeo geo;
  int n_min, n_max;               // sequences of n_min <= tokens <= n_max are this kernel's
};
cudaError_t launch_delta_steps(const DeltaFwdArgs& a, cudaStream_t s);

// ---- chunks of kChunk tokens (delta_intra.cu prepares them, delta_chain.cu goes through them) ----
// Numbers of a chunk that the state's chain takes, per token: e^G fk 2^-up, scale e^G fq, scale fq / P's unit, the factor of T's
// row times 2^-up (U in the outputs' products) and times e^(G_C - G) (U' in the state's), and up: 0 unless the chunk grows (a g
// above 0), else such that e^G is 2^up at most.  The state reaches a token's Z and U with e^G; kept 2^-up as large they stay
// alike in size, and T's and P's columns are 2^up as large.  fk, fq: what a stored row of K or Q has to be multiplied with; G: sum of g in the chunk.
// And of the chunk: e^(G_C), and bounds from which the chain takes its units.  V up to v and S up to s give Z up to v + zs s,
// U up to uv v + us s, and add xv v + xs s to a number of S at most.  (U's and S's are not taken from Z's: S reaches the late
// tokens with their decay, the early ones reach the next S with theirs.)
struct DeltaScalars {
  float c[kChunk], oq[kChunk], pq[kChunk], rs[kChunk], rx[kChunk];
  uint8_t up[kChunk];
  float decay, zs, uv, us, xv, xs;
  uint32_t grows, pad[9];
};
static_assert(sizeof(DeltaScalars) % 16 == 0 && sizeof(DeltaScalars) == kScalarBytes, "copied in 16-byte pieces");
// 2^e, e in [-126, 127]
__device__ __forceinline__ float power2(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }
// A chunk's images, as they lie in shared memory too (rows of 128 bytes, swizzled; 64 columns to a block of 64 rows):
// K and Q of a key head, T's two halves and P of a value head (kTPBytes).

struct DeltaWork {
  uint8_t* kq;                    // [window][hk][2][kChunk * dk * 2]
  uint8_t* tp;                    // [window][hv][kTPBytes]
  DeltaScalars* sc;               // [window][hv]
  float* carry[2];                // [hv][dk][dv] the state of a sequence that goes on in the next window
  int first, count;               // this window's chunks
  int parity;
  // A window's chunks of a sequence cut into parts (DeltaParts): the state before part j [n_seqs][parts][hv][dk][dv], and what
  // part j makes of a state, as a matrix [n_seqs][parts][hv][dk][dk].  pass 0: not cut.
  float *part_state, *part_mat;
  int parts, front, pass;
  bool ordered;                   // blocks start with the longest sequence (delta_ordered)
};

cudaError_t launch_delta_intra(const DeltaFwdArgs& a, const DeltaWork& w, cudaStream_t s);
// with w.parts > 1 both passes and what joins them
cudaError_t launch_delta_chain(const DeltaFwdArgs& a, const DeltaWork& w, cudaStream_t s);

// Numbers of at most m brought below 2^14 by a power of two, and back (m of any size: those above fp32's range are bounds of
// numbers inside it, and those below 2^-100 leave numbers as small as 2^-126 above fp16's smallest).
struct Unit {
  float to, from;
};
__device__ __forceinline__ Unit unit_of(float m) {
  const uint32_t e = min(max(__float_as_uint(m) >> 23, 27u), 254u);
  return Unit{__uint_as_float((267u - e) << 23), __uint_as_float((e - 13u) << 23)};
}
// A pair of numbers as fp16: rounded, and what is left
__device__ __forceinline__ void halves(float a, float b, uint32_t& hi, uint32_t& lo) {
  hi = pack16<false>(a, b);
  float x, y;                        // a - (float)(its half of hi), in one instruction
  asm("{\n\t.reg .f16 p, q, m;\n\t"
      "mov.b32 {p, q}, %2;\n\t"
      "mov.b16 m, 0xbc00;\n\t"
      "fma.rn.f32.f16 %0, p, m, %3;\n\t"
      "fma.rn.f32.f16 %1, q, m, %4;\n\t}"
      : "=f"(x), "=f"(y)
      : "r"(hi), "f"(a), "f"(b));
  lo = pack16<false>(x, y);
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at) : "memory");
}
// P is kept in units that bring its largest possible value (two rows shorter than 2) to 2^15: what decays have made 2^-27
// of it is still a normal number in fp16.  In a row that decays above 1 make up to 2^m as large, the unit is 2^m as large.
constexpr float kDeltaPUnit = 8192.f;

}  // namespace moe
