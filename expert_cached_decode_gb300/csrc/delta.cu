// Host side of the gated delta rule (moe_delta_*): argument checks, the handle,
// choice of kernels.
#include <cmath>
#include <mutex>
#include <new>

#include "delta.cuh"
#include "rows.h"

using namespace moe;

namespace {
constexpr int kMaxSeqs = 4096;
constexpr int kMaxTokens = 1 << 24;
constexpr int kMaxParts = 16, kMaxCuts = 320;   // parts of a sequence; heads' parts of a call
// Tokens of a sequence that are taken one by one.  Chunk by chunk up to 64 cost the same, one by one each costs its own pass (heads
// of 128 x 128, us one by one | in a chunk): 16 tokens of 1 sequence of 32 heads 14 | 24, of 64 sequences 142 | 194; 24 tokens
// 19 | 24 and 201 | 195; 32 tokens 25 | 24 and 265 | 197; 64 tokens 47 | 24 and 501 | 202.
constexpr int kFewTokens = 24;
}  // namespace

struct moe_delta {
  DeltaGeo g{};
  int device = 0, num_sms = 0;
  uint32_t* err = nullptr;
  // work space of calls with long sequences: what a window of chunks holds, and the state that goes on in the next window
  uint8_t* ws = nullptr;
  DeltaWork work{};
  int window = 0;
  // Held while such a call enqueues its kernels: another host thread's, put between them on the same stream, would replace
  // what the later ones are to read.
  std::mutex enqueue;
};

// The handle's device as the current one, and back.
struct OnDevice {
  int was = 0;
  bool changed = false;
  explicit OnDevice(int device) { changed = cudaGetDevice(&was) == cudaSuccess && was != device && cudaSetDevice(device) == cudaSuccess; }
  ~OnDevice() {
    if (changed) cudaSetDevice(was);
  }
};

static bool mis16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }

static moe_status cuda_fail(cudaError_t e, const char* what) {
  cudaGetLastError();
  return set_last_error(e == cudaErrorMemoryAllocation ? MOE_ERR_OOM : MOE_ERR_CUDA, "%s: %s", what,
                        cudaGetErrorString(e));
}

#define DELTA_CHECK(call)                   \
  do {                                      \
    const moe_status st_ = (call);          \
    if (st_ != MOE_OK) return st_;          \
  } while (0)

static moe_status launched(cudaError_t e, const char* what) { return e == cudaSuccess ? MOE_OK : cuda_fail(e, what); }

extern "C" moe_status moe_delta_create(const moe_delta_desc* D, moe_delta** out) {
  if (!D || !out) return set_last_error(MOE_ERR_INVALID_ARG, "NULL desc or out");
  *out = nullptr;
  if (D->n_k_heads < 1 || D->n_k_heads > 64 || D->n_v_heads < 1 || D->n_v_heads > 128 || D->n_v_heads % D->n_k_heads != 0)
    return set_last_error(MOE_ERR_INVALID_ARG, "heads: n_k_heads in 1..64, n_v_heads a multiple of it, at most 128");
  if ((D->k_dim != 64 && D->k_dim != 128) || (D->v_dim != 64 && D->v_dim != 128))
    return set_last_error(MOE_ERR_UNIMPLEMENTED, "k_dim and v_dim must be 64 or 128");
  if (D->io_type != MOE_T_BF16 && D->io_type != MOE_T_F16)
    return set_last_error(MOE_ERR_INVALID_ARG, "io_type must be MOE_T_BF16 or MOE_T_F16");
  if (D->taps != 0 && (D->taps < 2 || D->taps > 4))
    return set_last_error(MOE_ERR_INVALID_ARG, "taps must be 0 or in 2..4");
  if (!std::isfinite(D->eps) || D->eps < 0.f)
    return set_last_error(MOE_ERR_INVALID_ARG, "eps must be finite and not negative");
  if (!std::isfinite(D->scale) || D->scale < 0.f)
    return set_last_error(MOE_ERR_INVALID_ARG, "scale must be finite and not negative");
  moe_delta* d = new (std::nothrow) moe_delta();
  if (!d) return set_last_error(MOE_ERR_OOM, "handle");
  d->g.hk = D->n_k_heads;
  d->g.hv = D->n_v_heads;
  d->g.rep = D->n_v_heads / D->n_k_heads;
  d->g.dk = D->k_dim;
  d->g.dv = D->v_dim;
  d->g.io = D->io_type;
  d->g.taps = D->taps;
  d->g.normalize = D->normalize != 0;
  d->g.eps = D->eps;
  d->g.scale = D->scale > 0.f ? D->scale : 1.f / std::sqrt((float)D->k_dim);
  cudaError_t e = cudaGetDevice(&d->device);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&d->num_sms, cudaDevAttrMultiProcessorCount, d->device);
  const int64_t kq = (int64_t)d->g.hk * 2 * kChunk * d->g.dk * 2, tp = (int64_t)d->g.hv * kTPBytes, sc = d->g.hv * (int64_t)sizeof(DeltaScalars);
  const int64_t carry = (int64_t)d->g.hv * d->g.dk * d->g.dv * sizeof(float);
  d->window = delta_window(d->g.hk, d->g.hv, d->g.dk);
  const int64_t mat = (int64_t)d->g.hv * d->g.dk * d->g.dk * sizeof(float);
  const int64_t cuts = kMaxCuts / d->g.hv > 0 ? kMaxCuts / d->g.hv : 0;     // (sequence, part) pairs
  const int64_t bytes = d->window * (kq + tp + sc) + 2 * carry + cuts * (carry + mat);
  if (e == cudaSuccess) e = cudaMalloc(&d->ws, bytes);
  if (e == cudaSuccess) e = cudaMemset(d->ws, 0, bytes);
  if (e == cudaSuccess) {
    d->work.kq = d->ws;
    d->work.tp = d->work.kq + d->window * kq;
    d->work.sc = reinterpret_cast<DeltaScalars*>(d->work.tp + d->window * tp);
    d->work.carry[0] = reinterpret_cast<float*>(d->work.tp + d->window * (tp + sc));
    d->work.carry[1] = d->work.carry[0] + carry / sizeof(float);
    d->work.part_state = d->work.carry[1] + carry / sizeof(float);
    d->work.part_mat = d->work.part_state + cuts * (carry / sizeof(float));
    d->work.parts = 1;
  }
  if (e == cudaSuccess) e = cudaMalloc(&d->err, sizeof(uint32_t));
  if (e == cudaSuccess) e = cudaMemset(d->err, 0, sizeof(uint32_t));
  if (e == cudaSuccess) e = cudaDeviceSynchronize();
  if (e != cudaSuccess) {
    const moe_status st = cuda_fail(e, "delta handle");
    moe_delta_destroy(d);
    return st;
  }
  *out = d;
  return MOE_OK;
}

// Checks what every call takes; fills the kernels' view.
static moe_status take_batch(moe_delta* d, const moe_delta_batch* B, DeltaBatch* b) {
  if (!d || !B) return set_last_error(MOE_ERR_INVALID_ARG, "NULL handle or batch");
  if (B->n_seqs < 0 || B->n_seqs > kMaxSeqs)
    return set_last_error(MOE_ERR_INVALID_ARG, "n_seqs must be in [0, %d]", kMaxSeqs);
  if (B->n_tokens < 0 || B->n_tokens > kMaxTokens)
    return set_last_error(MOE_ERR_INVALID_ARG, "n_tokens must be in [0, %d]", kMaxTokens);
  if (B->n_slots < 0) return set_last_error(MOE_ERR_INVALID_ARG, "n_slots < 0");
  if (B->n_seqs > 0 && (!B->cu || !B->slots_in || !B->slots_out))
    return set_last_error(MOE_ERR_INVALID_ARG, "NULL cu, slots_in or slots_out");
  int device = -1;
  const cudaError_t e = cudaGetDevice(&device);
  if (e != cudaSuccess) return cuda_fail(e, "device query");
  if (device != d->device)
    return set_last_error(MOE_ERR_INVALID_ARG, "the handle belongs to device %d, the current one is %d", d->device, device);
  b->cu = B->cu;
  b->slots_in = B->slots_in;
  b->slots_out = B->slots_out;
  b->err = d->err;
  b->n_seqs = B->n_seqs;
  b->n_tokens = B->n_tokens;
  b->n_slots = B->n_slots;
  return MOE_OK;
}

static moe_status take_rows(const void* p, int64_t stride, int64_t width, const char* what) {
  if (!p) return set_last_error(MOE_ERR_INVALID_ARG, "NULL %s", what);
  if (mis16(p) || stride % 8 != 0 || stride < width)
    return set_last_error(MOE_ERR_INVALID_ARG,
                          "%s must be 16-byte aligned, its stride a multiple of 8 elements and at least %lld", what,
                          (long long)width);
  return MOE_OK;
}

// Whether one of the n outputs shares memory with an input or with another output.
static bool overlaps(const Rows* out, int n, const Rows* in, int m) {
  for (int i = 0; i < n; ++i) {
    for (int j = 0; j < m; ++j)
      if (rows_meet(in[j], out[i])) return true;
    for (int j = 0; j < i; ++j)
      if (rows_meet(out[j], out[i])) return true;
  }
  return false;
}

extern "C" moe_status moe_delta_prepare(moe_delta* d, const moe_delta_batch* B, const void* x, int64_t x_stride,
                                        const void* w, const void* bias, void* conv_state, void* y, const void* a,
                                        const void* b, int64_t ab_stride, const float* a_log, const float* dt_bias,
                                        float* g, float* beta, void* stream) {
  DeltaPrepArgs p{};
  DELTA_CHECK(take_batch(d, B, &p.b));
  // (a call without tokens has no x, y, a or g to point to; its sequences still carry their convolution's state over)
  const bool conv = x || conv_state, gates = a || g;
  if (!conv && !gates && B->n_tokens > 0) return set_last_error(MOE_ERR_INVALID_ARG, "neither x nor a");
  p.channels = 2 * d->g.hk * d->g.dk + d->g.hv * d->g.dv;
  if (conv) {
    if (!d->g.taps) return set_last_error(MOE_ERR_INVALID_ARG, "the handle has no convolution (taps is 0)");
    if (B->n_tokens > 0) DELTA_CHECK(take_rows(x, x_stride, p.channels, "x"));
    if (!w || (!y && B->n_tokens > 0) || (!conv_state && B->n_slots > 0))
      return set_last_error(MOE_ERR_INVALID_ARG, "NULL w, conv_state or y");
    if (mis16(w) || mis16(bias) || mis16(conv_state) || mis16(y))
      return set_last_error(MOE_ERR_INVALID_ARG, "w, bias, conv_state or y not 16-byte aligned");
  }
  if (gates && B->n_tokens > 0) {
    if (!a || !b || !a_log || !dt_bias || !g || !beta)
      return set_last_error(MOE_ERR_INVALID_ARG, "NULL a, b, a_log, dt_bias, g or beta");
    if (ab_stride < d->g.hv) return set_last_error(MOE_ERR_INVALID_ARG, "ab_stride is below n_v_heads");
  }
  {
    const int64_t n = B->n_tokens, C = p.channels, hv = d->g.hv;
    const Rows out[] = {bytes_at(conv ? y : nullptr, n * C * 2), bytes_at(conv ? conv_state : nullptr, (int64_t)B->n_slots * (d->g.taps - 1) * C * 2),
                        bytes_at(gates ? g : nullptr, n * hv * 4), bytes_at(gates ? beta : nullptr, n * hv * 4)};
    const Rows in[] = {{conv ? x : nullptr, n, x_stride * 2, C * 2}, bytes_at(conv ? w : nullptr, C * d->g.taps * 2), bytes_at(conv ? bias : nullptr, C * 2),
                       {gates ? a : nullptr, n, ab_stride * 2, hv * 2}, {gates ? b : nullptr, n, ab_stride * 2, hv * 2},
                       bytes_at(gates ? a_log : nullptr, hv * 4), bytes_at(gates ? dt_bias : nullptr, hv * 4),
                       bytes_at(B->cu, (B->n_seqs + 1) * 4ll), bytes_at(B->slots_in, B->n_seqs * 4ll), bytes_at(B->slots_out, B->n_seqs * 4ll)};
    if (overlaps(out, 4, in, 10))
      return set_last_error(MOE_ERR_INVALID_ARG, "y, conv_state, g or beta overlaps another tensor of the call");
  }
  if (B->n_seqs == 0) return MOE_OK;
  p.conv_on = conv;
  p.gates_on = gates;
  p.x = static_cast<const uint16_t*>(x);
  p.w = static_cast<const uint16_t*>(w);
  p.bias = static_cast<const uint16_t*>(bias);
  p.a = static_cast<const uint16_t*>(a);
  p.gb = static_cast<const uint16_t*>(b);
  p.x_stride = x_stride;
  p.ab_stride = ab_stride;
  p.conv = static_cast<uint16_t*>(conv_state);
  p.y = static_cast<uint16_t*>(y);
  p.a_log = a_log;
  p.dt_bias = dt_bias;
  p.g = g;
  p.beta = beta;
  p.hv = d->g.hv;
  p.taps = d->g.taps;
  return launched(launch_delta_prepare(p, d->g.io, static_cast<cudaStream_t>(stream), d->num_sms), "moe_delta_prepare");
}

extern "C" moe_status moe_delta_forward(moe_delta* d, const moe_delta_batch* B, const void* q, int64_t q_stride,
                                        const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                                        const float* g, const float* beta, float* state, void* out, void* stream) {
  DeltaFwdArgs x{};
  DELTA_CHECK(take_batch(d, B, &x.b));
  if (B->n_seqs == 0) return MOE_OK;
  if ((!state && B->n_slots > 0) || mis16(state))
    return set_last_error(MOE_ERR_INVALID_ARG, "state is NULL or not 16-byte aligned");
  if (B->n_tokens > 0) {
    DELTA_CHECK(take_rows(q, q_stride, (int64_t)d->g.hk * d->g.dk, "q"));
    DELTA_CHECK(take_rows(k, k_stride, (int64_t)d->g.hk * d->g.dk, "k"));
    DELTA_CHECK(take_rows(v, v_stride, (int64_t)d->g.hv * d->g.dv, "v"));
    DELTA_CHECK(take_rows(out, (int64_t)d->g.hv * d->g.dv, (int64_t)d->g.hv * d->g.dv, "out"));
    if (!g || !beta) return set_last_error(MOE_ERR_INVALID_ARG, "NULL g or beta");
  }
  {
    const int64_t n = B->n_tokens, wide = (int64_t)d->g.hv * d->g.dv, narrow = (int64_t)d->g.hk * d->g.dk, hv = d->g.hv;
    const Rows outs[] = {bytes_at(out, n * wide * 2), bytes_at(state, B->n_slots * wide * d->g.dk * 4)};
    const Rows in[] = {{q, n, q_stride * 2, narrow * 2}, {k, n, k_stride * 2, narrow * 2}, {v, n, v_stride * 2, wide * 2},
                       bytes_at(g, n * hv * 4), bytes_at(beta, n * hv * 4), bytes_at(B->cu, (B->n_seqs + 1) * 4ll),
                       bytes_at(B->slots_in, B->n_seqs * 4ll), bytes_at(B->slots_out, B->n_seqs * 4ll)};
    if (overlaps(outs, 2, in, 8)) return set_last_error(MOE_ERR_INVALID_ARG, "out or state overlaps another tensor of the call");
  }
  x.q = static_cast<const uint16_t*>(q);
  x.k = static_cast<const uint16_t*>(k);
  x.v = static_cast<const uint16_t*>(v);
  x.q_stride = q_stride;
  x.k_stride = k_stride;
  x.v_stride = v_stride;
  x.g = g;
  x.beta = beta;
  x.state = state;
  x.out = static_cast<uint16_t*>(out);
  x.geo = d->g;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int max_q = B->max_q > 0 && B->max_q < B->n_tokens ? B->max_q : B->n_tokens;
  const bool many = max_q > kFewTokens;
  x.n_min = 0;
  x.n_max = many ? kFewTokens : INT32_MAX;
  cudaError_t e = launch_delta_steps(x, st);
  if (e == cudaSuccess && many) {
    x.n_min = kFewTokens + 1;
    x.n_max = INT32_MAX;
    // sequence s has chunk numbers from t0 / kChunk + s on, so there are at most so many
    const int chunks = B->n_tokens / kChunk + B->n_seqs;
    std::lock_guard<std::mutex> lock(d->enqueue);
    DeltaWork w = d->work;
    // parts, where the heads of all sequences leave SMs without work
    const DeltaCut cut = delta_cut(B->n_seqs, d->g.hv, d->g.dk, d->g.dv, (max_q + kChunk - 1) / kChunk, d->num_sms, kMaxCuts, kMaxParts);
    w.parts = cut.parts;
    w.front = cut.front;
    w.ordered = delta_ordered(B->n_seqs, d->g.hv, d->num_sms);
    for (w.first = 0; e == cudaSuccess && w.first < chunks; w.first += d->window) {
      w.count = chunks - w.first < d->window ? chunks - w.first : d->window;
      e = launch_delta_intra(x, w, st);
      if (e == cudaSuccess) e = launch_delta_chain(x, w, st);
      w.parity ^= 1;
    }
  }
  return launched(e, "moe_delta_forward");
}

extern "C" moe_status moe_delta_sync(moe_delta* d) {
  if (!d) return set_last_error(MOE_ERR_INVALID_ARG, "NULL handle");
  uint32_t err = 0;
  const OnDevice on(d->device);
  cudaError_t e = cudaDeviceSynchronize();
  if (e == cudaSuccess) e = cudaMemcpy(&err, d->err, sizeof(err), cudaMemcpyDeviceToHost);
  if (e == cudaSuccess && err) e = cudaMemset(d->err, 0, sizeof(err));
  if (e != cudaSuccess) return cuda_fail(e, "moe_delta_sync");
  if (err & DELTA_TIMEOUT) return set_last_error(MOE_ERR_TIMEOUT, "a device-side wait of a delta call gave up");
  if (err)
    return set_last_error(MOE_ERR_INVALID_ARG, "a call found%s%s%s on the GPU (left out there)",
                          err & DELTA_BAD_SLOT ? " [a slot out of range]" : "",
                          err & DELTA_BAD_LEN ? " [an offset out of range]" : "",
                          err & DELTA_CLASH ? " [a slot that one sequence writes and another uses]" : "");
  return MOE_OK;
}

extern "C" void moe_delta_destroy(moe_delta* d) {
  if (!d) return;
  {
    const OnDevice on(d->device);
    if (d->err || d->ws) cudaDeviceSynchronize();
    if (d->err) cudaFree(d->err);
    if (d->ws) cudaFree(d->ws);
    cudaGetLastError();
  }
  delete d;
}
