// The gated delta rule 64 tokens at a time on the tensor cores (tcgen05):
// prompts and long drafts.
//
// Within a chunk of C = 64 tokens, with G_i the sum of g up to token i, the rule is
//     A_ij = beta_i e^(G_i - G_j) k^_i.k^_j  (j < i),     T = (1 + A)^-1 diag(beta)
//     U = T (V - diag(e^G) K^ S0)
//     O = scale (diag(e^G) Q^ S0 + P U),   P_ij = e^(G_i - G_j) q^_i.k^_j  (j <= i)
//     S = e^(G_C) S0 + (diag(e^(G_C - G)) K^)^T U
// A CTA takes one head of one sequence and goes through its chunks; only S passes
// from one to the next.  The products run transposed, a row of S^T (one of the
// v_dim columns of the state) to a lane of tensor memory: Y^T = S^T K^T,
// U^T = Z^T T^T, S^T += U'^T K.  So everything that follows the state is an A
// operand in tensor memory (never in shared memory), what does not (K, Q, T, P)
// lies in shared memory, each thread keeps its row of S in registers, and a row's
// scale is a thread's own.
//
// Precision: the state stays fp32, and operands that stand for it hold 22 bits:
// a pair of fp16 numbers (x rounded, and the rest rounded) under a power of two
// per row, so a product takes two or three multiplications in fp16 (K is exact:
// bf16 rows under a power of two are fp16 numbers).  Only what reaches nothing but
// the 16-bit outputs (Q S0, P U) takes the first halves alone.  Powers of A would
// cancel where keys are alike, so T comes from forward substitution: two 32 x 32
// blocks in fp32, and T21 = -T22 A21 T11.
// G is summed in 64-bit fixed point (2^-40), so that differences far down a chunk
// are exact.
//
// Roles of a CTA's 16 warps: 0-3 the state's chain (S -> Y -> Z -> U -> S, a thread
// per row; they also issue its products), 4-7 A, P and T (none of which needs the
// state, so they run ahead), 8-11 load K and Q and their norms and decays, 12-15
// bring V and write the outputs.
#include "attn_tc.cuh"
#include "delta.cuh"

namespace moe {

namespace {

constexpr int C = 64;                  // tokens of a chunk
constexpr int kThreads = DeltaRoles::Block::kThreads;
constexpr int kStages = 3;             // of K and Q
constexpr int kLd = 68;                // floats from row to row of A and T
// P is kept in units that bring its largest possible value (two rows shorter than 2) to 2^15: what decays have made 2^-27
// of it is still a normal number in fp16.
constexpr float kPUnit = 8192.f;

// Columns of tensor memory.  SH holds S^T's halves (first 8 columns per 16 rows of K, then the second halves), and when Y
// and QS are done the update of S.  Z's pairs replace Y, U' 's replace U.
constexpr uint32_t kSH = 0, kY = 128, kU = 192, kUH = 256, kQS = 288, kPU = 352, kKK = 416;

struct Scalars {                       // of one chunk, per token
  float fk[C], fq[C];                  // K and Q rows' factors
  float gh[C], gl[C];                  // G, in turns of 2: a multiple of 2^-8, and the rest
  float beta[C];
  float c[C];                          // e^G fk
  float oq[C], pq[C];                  // scale e^G fq, scale fq / kPUnit
  float w[C];                          // e^(G_C - G)
  float decay[4];                      // e^(G_C)
};

struct Bars {
  uint64_t kq_full[kStages], kq_empty[kStages], tp_full[2], tp_empty[2], v_full[2], v_empty[2];
  uint64_t kk_full, y_full, u_full, d_full, o_full, o_empty, drained, drained_kk;
  uint32_t tmem;
};

template <int DK>
struct Cfg {
  static constexpr int kKQ = 128 * DK * 2;               // K (rows 0-63) and Q (64-127), in blocks of 64 dimensions
  static constexpr int kTP = 3 * C * 128;                // T's two halves, P
  static constexpr int kV = C / 2 * 128 * 4;             // V: [pair of tokens][dimension]
  static constexpr int oTP = kStages * kKQ;
  static constexpr int oV = oTP + 2 * kTP;
  static constexpr int oA = oV + 2 * kV;                 // A, then T, fp32 [64][kLd]; A21 T11 [32][36]
  static constexpr int oT = oA + C * kLd * 4;
  static constexpr int oM = oT + C * kLd * 4;
  static constexpr int oSc = oM + 32 * 36 * 4;
  static constexpr int oRs = oSc + kStages * (int)sizeof(Scalars);   // factors of T's rows [2][64]
  static constexpr int oLane = oRs + 2 * C * 4;          // the rows' factors of QS and PU [2][128]
  static constexpr int oBar = oLane + 2 * 128 * 4;
  static constexpr int kSmem = oBar + (int)sizeof(Bars);
};

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

// K as the B operand of the state's update: N = dimensions along the 128-byte rows (64 to a block of 128 rows), K = tokens
// down the rows.  Leading offset: to the next 64 dimensions; stride offset: to the next 8 tokens.
__device__ __forceinline__ uint64_t k_cols_desc(const void* tile) {
  uint64_t d = (smem_u32(tile) >> 4) & 0x3FFFull;
  d |= (uint64_t)((128 * 128) >> 4) << 16;
  d |= (uint64_t)(1024 >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}

// The power of two that brings numbers of at most m below 2^14, and back.
struct Unit {
  float to, from;
};
__device__ __forceinline__ Unit unit_of(float m) {
  const uint32_t e = min(max(__float_as_uint(m) >> 23, 27u), 240u);
  return Unit{__uint_as_float((267u - e) << 23), __uint_as_float((e - 13u) << 23)};
}

// A pair of numbers as fp16: rounded, and what is left
__device__ __forceinline__ void halves(uint64_t x, uint32_t& hi, uint32_t& lo) {
  const float a = lo2(x), b = hi2(x);
  hi = pack16<false>(a, b);
  const float2 h = unpack16<false>(hi);
  lo = pack16<false>(a - h.x, b - h.y);
}
__device__ __forceinline__ float max_abs(float m, uint64_t x) { return fmaxf(m, fmaxf(fabsf(lo2(x)), fabsf(hi2(x)))); }
__device__ __forceinline__ uint64_t f2u(uint32_t a, uint32_t b) { return f2(__uint_as_float(a), __uint_as_float(b)); }

// A wait that gave up turns every later wait of its warp into nothing: the roles then run through their loops (on wrong
// data, in bounds) so that every barrier is still met, and the error word says that the results are void.
template <bool BF16, int DK, int DV>
__global__ void __launch_bounds__(kThreads, 1) chunk_kernel(const __grid_constant__ DeltaFwdArgs a) {
  using L = Cfg<DK>;
  extern __shared__ __align__(1024) uint8_t smem[];
  Bars& bar = *reinterpret_cast<Bars*>(smem + L::oBar);
  Scalars* scalars = reinterpret_cast<Scalars*>(smem + L::oSc);
  float* rs = reinterpret_cast<float*>(smem + L::oRs);
  float* lane_s = reinterpret_cast<float*>(smem + L::oLane);
  float* lane_u = lane_s + 128;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, wg = tid >> 7, wt = tid & 127;
  const int h = blockIdx.x, s = blockIdx.y, hv = a.geo.hv;
  const DeltaSeq q = delta_seq(a.b, s);
  if (q.n < a.n_min || q.n > a.n_max) return;
  const int chunks = (q.n + C - 1) / C;

  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&bar.kq_full[i], 128);
      mbar_init(&bar.kq_empty[i], 129);      // the products that read it, and warps 12-15 (scalars)
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar.tp_full[i], 128);
      mbar_init(&bar.tp_empty[i], 1);
      mbar_init(&bar.v_full[i], 128);
      mbar_init(&bar.v_empty[i], 128);
    }
    mbar_init(&bar.kk_full, 1);
    mbar_init(&bar.y_full, 1);
    mbar_init(&bar.u_full, 1);
    mbar_init(&bar.d_full, 1);
    mbar_init(&bar.o_full, 129);             // the products, and warps 0-3 (the rows' factors)
    mbar_init(&bar.o_empty, 128);
    mbar_init(&bar.drained, 1);
    mbar_init(&bar.drained_kk, 1);
    mbar_init_fence();
  }
  if (warp == 0) {
    tmem_alloc(&bar.tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  const bool writes = __syncthreads_and(delta_writes(a.b, s, q, tid, kThreads));
  tc_fence_after();
  bool ok = true;
  auto wait = [&](uint64_t* b, uint32_t parity) {
    if (ok && !__all_sync(0xffffffffu, mbar_wait_cycles(b, parity))) {
      ok = false;
      if (lane == 0) atomicOr(a.b.err, (uint32_t)DELTA_TIMEOUT);
    }
  };
  const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;

  if (wg == 0) {
    // ================================ the chain ================================
    reg_inc<DeltaRoles::kChain>();
    const bool live = wt < DV;
    const int64_t col = (int64_t)h * DK * DV + wt, slot = (int64_t)hv * DK * DV;
    uint64_t S[DK / 2];
    float m = 0.f;
#pragma unroll
    for (int j = 0; j < DK / 2; ++j) {
      float x = 0.f, y = 0.f;
      if (live && q.in >= 0) {
        const float* p = a.state + q.in * slot + col + 2 * j * DV;
        x = p[0];
        y = p[DV];
      }
      S[j] = f2(x, y);
      m = max_abs(m, S[j]);
    }
    const uint32_t id_d = idesc_f16(128, DK, 0) | 1u << 16;
    const uint64_t kq0 = smem_desc_sw128(smem), kc0 = k_cols_desc(smem), tp0 = smem_desc_sw128(smem + L::oTP);
    const uint32_t* vs = reinterpret_cast<const uint32_t*>(smem + L::oV);
    float fu = 0.f;                          // of the update of S that is under way
    uint64_t gc = 0;
    for (int i = 0; i <= chunks; ++i) {
      const int st = i % kStages, ts = i & 1;
      // ---- S ----
      if (i > 0) {
        wait(&bar.d_full, (i - 1) & 1);
        tc_fence_after();
        if (live) {
          const uint64_t f = f2(fu, fu);
          m = 0.f;
#pragma unroll
          for (int b = 0; b < DK / 32; ++b) {
            uint32_t d[32];
            tmem_ld32(lane_base + kSH + 32 * b, d);
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              uint64_t& x = S[16 * b + j];
              x = fma2(x, gc, mul2(f2u(d[2 * j], d[2 * j + 1]), f));
              m = max_abs(m, x);
            }
          }
        }
      }
      if (i == chunks) break;
      const Unit us = unit_of(m);
      if (live) {
        const uint64_t to = f2(us.to, us.to);
#pragma unroll
        for (int b = 0; b < DK / 32; ++b) {
          uint32_t hi[16], lo[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) halves(mul2(S[16 * b + j], to), hi[j], lo[j]);
          tmem_st16(lane_base + kSH + 16 * b, hi);
          tmem_st16(lane_base + kSH + DK / 2 + 16 * b, lo);
        }
        tmem_st_wait();
      }
      tc_fence_before();
      named_bar(2, 128);
      if (warp == 0) {
        wait(&bar.kq_full[st], (i / kStages) & 1);
        if (i > 0) wait(&bar.o_empty, (i - 1) & 1);
        tc_fence_after();
        const uint64_t kd = kq0 + st * (L::kKQ >> 4);
        const uint32_t id = idesc_f16(128, 64, 0);
        if (ok && elect_one()) {
#pragma unroll
          for (int half = 0; half < 2; ++half)
#pragma unroll
            for (int k = 0; k < DK / 16; ++k)
              umma_f16_ts(kY, kSH + half * (DK / 2) + 8 * k, kd + ((k >> 2) * 16384 >> 4) + 2 * (k & 3), id, half | k);
          umma_commit(&bar.y_full);
#pragma unroll
          for (int k = 0; k < DK / 16; ++k)
            umma_f16_ts(kQS, kSH + 8 * k, kd + (((k >> 2) * 16384 + 8192) >> 4) + 2 * (k & 3), id, k != 0);
        }
        __syncwarp();
      }
      // ---- Z = V - diag(e^G) K^ S ----
      const Scalars& sc = scalars[st];
      wait(&bar.v_full[ts], (i >> 1) & 1);
      wait(&bar.kq_full[st], (i / kStages) & 1);
      wait(&bar.y_full, i & 1);
      tc_fence_after();
      float fz = 0.f;
      if (live) {
        uint32_t y[2][32];
        tmem_ld32(lane_base + kY, y[0]);
        tmem_ld32(lane_base + kY + 32, y[1]);
        tmem_ld_wait();
        uint64_t z[32];
        const uint64_t nf = f2(-us.from, -us.from);
        float mz = 0.f;
#pragma unroll
        for (int j = 0; j < 32; j += 2) {
          const float4 c4 = *reinterpret_cast<const float4*>(&sc.c[2 * j]);
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float2 v = unpack16<BF16>(vs[ts * (L::kV / 4) + (j + e) * 128 + wt]);
            const int t = 2 * (j + e);
            z[j + e] = fma2(mul2(e ? f2(c4.z, c4.w) : f2(c4.x, c4.y), nf), f2u(y[t >> 5][t & 31], y[t >> 5][(t & 31) + 1]), f2(v.x, v.y));
            mz = max_abs(mz, z[j + e]);
          }
        }
        const Unit uz = unit_of(mz);
        fz = uz.from;
        const uint64_t to = f2(uz.to, uz.to);
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          uint32_t hi[16], lo[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) halves(mul2(z[16 * b + j], to), hi[j], lo[j]);
          tmem_st16(lane_base + kY + 16 * b, hi);
          tmem_st16(lane_base + kY + 32 + 16 * b, lo);
        }
        tmem_st_wait();
      }
      mbar_arrive(&bar.v_empty[ts]);
      tc_fence_before();
      named_bar(2, 128);
      if (warp == 0) {
        wait(&bar.tp_full[ts], (i >> 1) & 1);
        tc_fence_after();
        const uint64_t td = tp0 + ts * (L::kTP >> 4);
        if (ok && elect_one()) {
          // tokens 16 k .. + 15 reach the tokens from 16 k on only
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint32_t id = idesc_f16(128, 64 - 16 * k, 0);
            const uint64_t row = td + (2048 * k >> 4) + 2 * k;
            umma_f16_ts(kU + 16 * k, kY + 8 * k, row, id, k != 0);
            umma_f16_ts(kU + 16 * k, kY + 32 + 8 * k, row, id, 1);
            umma_f16_ts(kU + 16 * k, kY + 8 * k, row + (C * 128 >> 4), id, 1);
          }
          umma_commit(&bar.u_full);
        }
        __syncwarp();
      }
      // ---- U ----
      wait(&bar.tp_full[ts], (i >> 1) & 1);
      wait(&bar.u_full, i & 1);
      tc_fence_after();
      if (live) {
        uint32_t y[2][32];
        tmem_ld32(lane_base + kU, y[0]);
        tmem_ld32(lane_base + kU + 32, y[1]);
        tmem_ld_wait();
        uint64_t u[32];
        const uint64_t f = f2(fz, fz);
        float mu = 0.f;
#pragma unroll
        for (int j = 0; j < 32; j += 2) {
          const float4 r4 = *reinterpret_cast<const float4*>(&rs[ts * C + 2 * j]);
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int t = 2 * (j + e);
            u[j + e] = mul2(mul2(e ? f2(r4.z, r4.w) : f2(r4.x, r4.y), f), f2u(y[t >> 5][t & 31], y[t >> 5][(t & 31) + 1]));
            mu = max_abs(mu, u[j + e]);
          }
        }
        const Unit uo = unit_of(mu);
        lane_s[wt] = us.from;
        lane_u[wt] = uo.from;
        float mw = 0.f;
        const uint64_t to = f2(uo.to, uo.to);
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          uint32_t hi[16];
#pragma unroll
          for (int j = 0; j < 16; j += 2) {
            const float4 w4 = *reinterpret_cast<const float4*>(&sc.w[32 * b + 2 * j]);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              uint64_t& x = u[16 * b + j + e];
              const uint64_t o = mul2(x, to);
              hi[j + e] = pack16<false>(lo2(o), hi2(o));
              x = mul2(x, e ? f2(w4.z, w4.w) : f2(w4.x, w4.y));
              mw = max_abs(mw, x);
            }
          }
          tmem_st16(lane_base + kUH + 16 * b, hi);
        }
        const Unit uw = unit_of(mw);
        fu = uw.from;
        const uint64_t tw = f2(uw.to, uw.to);
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          uint32_t hi[16], lo[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) halves(mul2(u[16 * b + j], tw), hi[j], lo[j]);
          tmem_st16(lane_base + kU + 16 * b, hi);
          tmem_st16(lane_base + kU + 32 + 16 * b, lo);
        }
        tmem_st_wait();
      }
      gc = f2(sc.decay[0], sc.decay[0]);
      mbar_arrive(&bar.o_full);
      tc_fence_before();
      named_bar(2, 128);
      if (warp == 0) {
        tc_fence_after();
        const uint64_t kc = kc0 + st * (L::kKQ >> 4), pd = tp0 + ((ts * L::kTP + 2 * C * 128) >> 4);
        if (ok && elect_one()) {
#pragma unroll
          for (int k = 0; k < 8; ++k) umma_f16_ts(kSH, kU + 8 * k, kc + ((k & 3) * 2048 >> 4), id_d, k != 0);
          umma_commit(&bar.d_full);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            umma_f16_ts(kPU + 16 * k, kUH + 8 * k, pd + (2048 * k >> 4) + 2 * k, idesc_f16(128, 64 - 16 * k, 0), k != 0);
          umma_commit(&bar.o_full);
          umma_commit(&bar.tp_empty[ts]);
          umma_commit(&bar.kq_empty[st]);
        }
        __syncwarp();
      }
    }
    if (live && writes) {
#pragma unroll
      for (int j = 0; j < DK / 2; ++j) {
        float* p = a.state + q.out * slot + col + 2 * j * DV;
        p[0] = lo2(S[j]);
        p[DV] = hi2(S[j]);
      }
    }
  } else if (wg == 1) {
    // ================================ A, P, T ================================
    reg_dec<DeltaRoles::kInverse>();
    const int w1 = warp & 3, r = wt & 63;
    const bool is_q = wt >= 64;
    float* A = reinterpret_cast<float*>(smem + L::oA);
    float* T = reinterpret_cast<float*>(smem + L::oT);
    float* M = reinterpret_cast<float*>(smem + L::oM);
    const uint64_t kq0 = smem_desc_sw128(smem);
    for (int i = 0; i < chunks; ++i) {
      const int st = i % kStages, ts = i & 1;
      const Scalars& sc = scalars[st];
      uint8_t* tp = smem + L::oTP + ts * L::kTP;
      wait(&bar.kq_full[st], (i / kStages) & 1);
      if (w1 == 0) {
        tc_fence_after();
        const uint64_t kd = kq0 + st * (L::kKQ >> 4);
        if (ok && elect_one()) {
#pragma unroll
          for (int k = 0; k < DK / 16; ++k) {
            const uint64_t d = kd + ((k >> 2) * 16384 >> 4) + 2 * (k & 3);
            umma_f16(kKK, d, d, idesc_f16(128, 64, 0), k != 0);
          }
          umma_commit(&bar.kk_full);
        }
        __syncwarp();
      }
      wait(&bar.kk_full, i & 1);
      tc_fence_after();
      if (i >= 2) wait(&bar.tp_empty[ts], ((i >> 1) - 1) & 1);
      const float gh = sc.gh[r], gl = sc.gl[r], row = is_q ? kPUnit : sc.beta[r] * sc.fk[r];
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        uint32_t x[32];
        tmem_ld32(lane_base + kKK + 32 * b, x);
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 32; j += 4) {
          const int c = 32 * b + j;
          const float4 h4 = *reinterpret_cast<const float4*>(&sc.gh[c]), l4 = *reinterpret_cast<const float4*>(&sc.gl[c]);
          float4 f4 = make_float4(1.f, 1.f, 1.f, 1.f);
          if (!is_q) f4 = *reinterpret_cast<const float4*>(&sc.fk[c]);
          float v[4];
          const float hh[4] = {h4.x, h4.y, h4.z, h4.w}, ll[4] = {l4.x, l4.y, l4.z, l4.w}, ff[4] = {f4.x, f4.y, f4.z, f4.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float d = ex2((gh - hh[e]) + (gl - ll[e])) * (row * ff[e]);
            v[e] = c + e < r + is_q ? __uint_as_float(x[j + e]) * d : 0.f;
            x[j + e] = __float_as_uint(v[e]);
          }
          if (!is_q) *reinterpret_cast<float4*>(&A[r * kLd + c]) = make_float4(v[0], v[1], v[2], v[3]);
        }
        if (is_q) {
#pragma unroll
          for (int j = 0; j < 32; j += 8) {
            uint32_t p[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) p[e] = pack16<false>(__uint_as_float(x[j + 2 * e]), __uint_as_float(x[j + 2 * e + 1]));
            *reinterpret_cast<uint4*>(tp + 2 * C * 128 + sw128_offset(r, 4 * b + j / 8)) = make_uint4(p[0], p[1], p[2], p[3]);
          }
        }
      }
      tc_fence_before();
      named_bar(3, 128);
      if (w1 < 2) {                          // (1 + A11)^-1 and (1 + A22)^-1, a lane per column
        const float* B = A + 32 * w1 * (kLd + 1);
        float x[32];
#pragma unroll
        for (int k = 0; k < 32; ++k) {
          float p[4] = {k == lane ? 1.f : 0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int j = 0; j < k; j += 4) {
            const float4 b4 = *reinterpret_cast<const float4*>(&B[k * kLd + j]);
            const float bb[4] = {b4.x, b4.y, b4.z, b4.w};
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (j + e < k) p[e] -= bb[e] * x[j + e];
          }
          x[k] = (p[0] + p[1]) + (p[2] + p[3]);
          T[(32 * w1 + k) * kLd + 32 * w1 + lane] = x[k];
        }
      }
      named_bar(3, 128);
      const int mi = wt >> 2, mj = (wt & 3) * 8;
      auto product = [&](const float* X, const float* Y, int ldy, float (&o)[8]) {   // row mi of X times columns mj .. + 7 of Y
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = 0.f;
#pragma unroll 2
        for (int k = 0; k < 32; k += 4) {
          const float4 x4 = *reinterpret_cast<const float4*>(&X[mi * kLd + k]);
          const float xx[4] = {x4.x, x4.y, x4.z, x4.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float4 y0 = *reinterpret_cast<const float4*>(&Y[(k + e) * ldy + mj]), y1 = *reinterpret_cast<const float4*>(&Y[(k + e) * ldy + mj + 4]);
            o[0] += xx[e] * y0.x;
            o[1] += xx[e] * y0.y;
            o[2] += xx[e] * y0.z;
            o[3] += xx[e] * y0.w;
            o[4] += xx[e] * y1.x;
            o[5] += xx[e] * y1.y;
            o[6] += xx[e] * y1.z;
            o[7] += xx[e] * y1.w;
          }
        }
      };
      float o[8];
      product(A + 32 * kLd, T, kLd, o);      // A21 T11
      *reinterpret_cast<float4*>(&M[mi * 36 + mj]) = make_float4(o[0], o[1], o[2], o[3]);
      *reinterpret_cast<float4*>(&M[mi * 36 + mj + 4]) = make_float4(o[4], o[5], o[6], o[7]);
      named_bar(3, 128);
      product(T + 32 * (kLd + 1), M, 36, o); // T22 (A21 T11)
      *reinterpret_cast<float4*>(&T[(32 + mi) * kLd + mj]) = make_float4(-o[0], -o[1], -o[2], -o[3]);
      *reinterpret_cast<float4*>(&T[(32 + mi) * kLd + mj + 4]) = make_float4(-o[4], -o[5], -o[6], -o[7]);
      named_bar(3, 128);
      // T diag(beta) as pairs, under a power of two per row; two threads a row
      {
        const int tr = wt >> 1, c0 = (wt & 1) * 32;
        float x[32], mx = 0.f;
#pragma unroll
        for (int j = 0; j < 32; j += 4) {
          float4 t4 = make_float4(0.f, 0.f, 0.f, 0.f);
          if (tr >= c0) t4 = *reinterpret_cast<const float4*>(&T[tr * kLd + c0 + j]);
          const float4 b4 = *reinterpret_cast<const float4*>(&sc.beta[c0 + j]);
          x[j] = t4.x * b4.x;
          x[j + 1] = t4.y * b4.y;
          x[j + 2] = t4.z * b4.z;
          x[j + 3] = t4.w * b4.w;
#pragma unroll
          for (int e = 0; e < 4; ++e) mx = fmaxf(mx, fabsf(x[j + e]));
        }
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        const Unit ut = unit_of(mx);
        if (!(wt & 1)) rs[ts * C + tr] = ut.from * sc.fk[tr];
#pragma unroll
        for (int j = 0; j < 32; j += 8) {
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) halves(f2(x[j + 2 * e] * ut.to, x[j + 2 * e + 1] * ut.to), hi[e], lo[e]);
          const uint32_t at = sw128_offset(tr, (c0 + j) / 8);
          *reinterpret_cast<uint4*>(tp + at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
          *reinterpret_cast<uint4*>(tp + C * 128 + at) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        }
      }
      fence_proxy_async_smem();
      mbar_arrive(&bar.tp_full[ts]);
    }
  } else if (wg == 2) {
    // ================================ K, Q, decays ================================
    reg_dec<DeltaRoles::kLoad>();
    constexpr int CH = DK / 8, RP = 128 / CH;                // 16-byte pieces of a row, rows of a pass
    const int ch = wt % CH, r0 = wt / CH;
    const int kh = h / a.geo.rep;
    for (int i = 0; i < chunks; ++i) {
      const int st = i % kStages, left = min(C, q.n - i * C);
      const int64_t t0 = (int64_t)q.t0 + i * C;
      Scalars& sc = scalars[st];
      uint8_t* kq = smem + st * L::kKQ;
      // a lane's two tokens' decays and betas (warp 8)
      float g2[2] = {0.f, 0.f}, be[2] = {0.f, 0.f};
      if (wt < 32) {
#pragma unroll
        for (int e = 0; e < 2; ++e)
          if (2 * lane + e < left) {
            g2[e] = a.g[(t0 + 2 * lane + e) * hv + h];
            be[e] = a.beta[(t0 + 2 * lane + e) * hv + h];
          }
      }
      if (i >= kStages) wait(&bar.kq_empty[st], (i / kStages - 1) & 1);
#pragma unroll 1
      for (int p = 0; p < C / RP; p += 4) {                  // four rows of K and of Q at a time
        uint4 x[2][4];
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          const int r = (p + y) * RP + r0;
          x[0][y] = x[1][y] = make_uint4(0, 0, 0, 0);
          if (r < left) {
            x[0][y] = __ldg(reinterpret_cast<const uint4*>(a.k + (t0 + r) * a.k_stride + kh * DK + 8 * ch));
            x[1][y] = __ldg(reinterpret_cast<const uint4*>(a.q + (t0 + r) * a.q_stride + kh * DK + 8 * ch));
          }
        }
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          const int r = (p + y) * RP + r0;
#pragma unroll
          for (int z = 0; z < 2; ++z) {
            const uint32_t w[4] = {x[z][y].x, x[z][y].y, x[z][y].z, x[z][y].w};
            float v[8], ss = 0.f;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float2 f = unpack16<BF16>(w[e]);
              v[2 * e] = f.x;
              v[2 * e + 1] = f.y;
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) ss += v[e] * v[e];
#pragma unroll
            for (int o = 1; o < CH; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            // under the power of two next to its length the row is fp16 (but for elements 2^-14 below it)
            const int e2 = ss > 0.f ? (int)(__float_as_uint(ss) >> 23) - 127 >> 1 : 0;
            const float down = __uint_as_float((uint32_t)(127 - e2) << 23), up = __uint_as_float((uint32_t)(127 + e2) << 23);
            uint32_t o[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) o[e] = pack16<false>(v[2 * e] * down, v[2 * e + 1] * down);
            *reinterpret_cast<uint4*>(kq + (ch >> 3) * 16384 + sw128_offset(64 * z + r, ch & 7)) = make_uint4(o[0], o[1], o[2], o[3]);
            if (ch == 0) (z ? sc.fq : sc.fk)[r] = r < left ? (a.geo.normalize ? rsqrtf(ss + a.geo.eps) * up : up) : 0.f;
          }
        }
      }
      fence_proxy_async_smem();
      named_bar(4, 128);
      if (wt < 32) {
        // G in units of 2^-40 of a factor of two: g log2(e), with the product's own rounding error
        int64_t G[2];
        bool nan = false;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float x = fminf(fmaxf(g2[e], -176.f), 176.f);            // 2^-253: nothing is left
          const float hi = x * 1.44269502f, lo = fmaf(x, 1.44269502f, -hi) + x * 1.92596303e-8f;
          G[e] = (int64_t)(hi * 1.099511627776e12f) + (int64_t)(lo * 1.099511627776e12f);
          nan |= g2[e] != g2[e];
        }
        const uint32_t bad = __ballot_sync(0xffffffffu, nan);            // a NaN reaches its token and all behind it
        G[1] += G[0];
        int64_t sum = G[1];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int64_t x = __shfl_up_sync(0xffffffffu, (long long)sum, o);
          if (lane >= o) sum += x;
        }
        const int64_t before = sum - G[1], total = __shfl_sync(0xffffffffu, (long long)sum, 31);
        const float poison = bad & (0xffffffffu >> (31 - lane)) ? __int_as_float(0x7fc00000) : 0.f;
        const float th = (float)(int)(total >> 32) * 0x1p-8f, tl = (float)(uint32_t)total * 0x1p-40f;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int t = 2 * lane + e;
          const int64_t x = before + (e ? G[1] : G[0]);
          const float gh = (float)(int)(x >> 32) * 0x1p-8f, gl = (float)(uint32_t)x * 0x1p-40f + poison;
          const float d = ex2(gh + gl);
          sc.gh[t] = gh;
          sc.gl[t] = gl;
          sc.beta[t] = be[e];
          sc.c[t] = d * sc.fk[t];
          sc.oq[t] = a.geo.scale * d * sc.fq[t];
          sc.pq[t] = a.geo.scale * sc.fq[t] * (1.f / kPUnit);
          sc.w[t] = ex2((th - gh) + (tl - gl));
        }
        if (lane == 0) sc.decay[0] = ex2(th + tl + (bad ? __int_as_float(0x7fc00000) : 0.f));
      }
      mbar_arrive(&bar.kq_full[st]);
    }
  } else {
    // ================================ V, outputs ================================
    reg_dec<DeltaRoles::kOutput>();
    const bool live = wt < DV;
    uint32_t* vs = reinterpret_cast<uint32_t*>(smem + L::oV);
    auto bring_v = [&](int i) {              // V of chunk i: a thread per dimension, two tokens to a word
      const int ts = i & 1, left = min(C, q.n - i * C);
      if (i >= 2) wait(&bar.v_empty[ts], ((i >> 1) - 1) & 1);
      if (live) {
        const uint16_t* p = a.v + ((int64_t)q.t0 + i * C) * a.v_stride + h * DV + wt;
#pragma unroll 1
        for (int b = 0; b < C; b += 32) {
          uint32_t x[32];
#pragma unroll
          for (int t = 0; t < 32; ++t) x[t] = b + t < left ? __ldg(p + (b + t) * a.v_stride) : (uint16_t)0;
#pragma unroll
          for (int t = 0; t < 32; t += 2) vs[ts * (L::kV / 4) + ((b + t) >> 1) * 128 + wt] = x[t] | x[t + 1] << 16;
        }
      }
      mbar_arrive(&bar.v_full[ts]);
    };
    bring_v(0);
    for (int i = 0; i < chunks; ++i) {
      const int st = i % kStages, left = min(C, q.n - i * C);
      if (i + 1 < chunks) bring_v(i + 1);
      const Scalars& sc = scalars[st];
      wait(&bar.kq_full[st], (i / kStages) & 1);
      wait(&bar.o_full, i & 1);
      tc_fence_after();
      if (live) {
        const float fs = lane_s[wt], fo = lane_u[wt];
        uint16_t* p = a.out + (((int64_t)q.t0 + i * C) * hv + h) * DV + wt;
#pragma unroll 1
        for (int b = 0; b < C; b += 16) {
          uint32_t x[16], y[16];
          tmem_ld16(lane_base + kQS + b, x);
          tmem_ld16(lane_base + kPU + b, y);
          tmem_ld_wait();
#pragma unroll
          for (int t = 0; t < 16; ++t) {
            const float o = sc.oq[b + t] * (fs * __uint_as_float(x[t])) + sc.pq[b + t] * (fo * __uint_as_float(y[t]));
            if (b + t < left) p[(int64_t)(b + t) * hv * DV] = (uint16_t)pack16<BF16>(o, 0.f);
          }
        }
      }
      tc_fence_before();
      mbar_arrive(&bar.o_empty);
      mbar_arrive(&bar.kq_empty[st]);
    }
  }
  // every product has ended before the tensor memory is given back, also after a wait that gave up
  if (warp == 0 || warp == 4) {
    uint64_t* b = warp ? &bar.drained_kk : &bar.drained;
    if (elect_one()) {
      umma_commit(b);
      if (!mbar_wait_cycles(b, 0)) atomicOr(a.b.err, (uint32_t)DELTA_TIMEOUT);
    }
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 0) tmem_dealloc(bar.tmem, 512);
}

template <bool BF16, int DK, int DV>
cudaError_t launch(const DeltaFwdArgs& a, cudaStream_t s) {
  constexpr int smem = Cfg<DK>::kSmem;
  static_assert(smem <= 227 * 1024, "shared memory");
  const void* fn = reinterpret_cast<const void*>(chunk_kernel<BF16, DK, DV>);
  const cudaError_t e = ensure_dyn_smem(fn, smem);
  if (e != cudaSuccess) return e;
  // the roles' registers must fit what the block is launched with
  static const int regs = [fn] {
    cudaFuncAttributes at;
    return cudaFuncGetAttributes(&at, fn) == cudaSuccess ? at.numRegs : 0;
  }();
  if (regs * kThreads < DeltaRoles::Block::registers()) return cudaErrorLaunchOutOfResources;
  chunk_kernel<BF16, DK, DV><<<dim3(a.geo.hv, a.b.n_seqs), kThreads, smem, s>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_delta_chunk(const DeltaFwdArgs& a, cudaStream_t s) {
  const bool bf = a.geo.io == MOE_T_BF16;
#define DELTA_CHUNK(DK, DV) return bf ? launch<true, DK, DV>(a, s) : launch<false, DK, DV>(a, s)
  if (a.geo.dk == 128) {
    if (a.geo.dv == 128) DELTA_CHUNK(128, 128);
    DELTA_CHUNK(128, 64);
  }
  if (a.geo.dv == 128) DELTA_CHUNK(64, 128);
  DELTA_CHUNK(64, 64);
#undef DELTA_CHUNK
}

}  // namespace moe
