// The gated delta rule's state through the chunks of a sequence
// (delta_intra.cu has prepared them):
//     Z = V - diag(e^G) K^ S      U = T Z      O = scale (diag(e^G) Q^ S + P U)
//     S <- e^(G_C) S + (diag(e^(G_C - G)) K^)^T U
// Only S passes from chunk to chunk, so the time of a long prompt is the number
// of its chunks times this chain's latency: three products that wait for one
// another.  Tensor memory's products would be four times as fast, but each
// costs some 300 cycles until its result is in registers again as an operand,
// and one head's rows would fill one SM with conversions; here the products are
// mma.sync, whose accumulators are the next product's operands, and a head is cut
// into slices of 16 state columns.  A CTA takes two slices, a pair of warps each:
// S^T (16 x k_dim), Z^T and U^T (16 x 64) lie in a pair's registers, each warp
// holding half of the columns.  What the other warp needs as an operand it finds
// in shared memory, and it multiplies its own half first, so the exchange costs
// little.
//
// Precision: S, Z and U are split into pairs of fp16 numbers (22 bits) under a
// power of two per row and half; products of two halves with different powers go
// to accumulators of their own.  S stays fp32 in registers.
#include "delta.cuh"
#include "tc.cuh"

namespace moe {

namespace {

constexpr int C = kChunk;
constexpr int kWarps = 4, kThreads = 32 * (kWarps + 1);   // and one that brings the chunks
constexpr int kStages = 3;
constexpr int kVRow = 80;              // bytes from token to token of V's 32 columns: 8 rows hit 8 different 16-byte places

template <int DK>
struct Cfg {
  static constexpr int kMat = C * DK * 2, kKQ = 2 * kMat;
  static constexpr int oTP = kKQ, oV = oTP + kTPBytes, oSc = oV + C * kVRow;
  static constexpr int kStage = (oSc + (int)sizeof(DeltaScalars) + 1023) / 1024 * 1024;
  // a pair's exchanged operands, 16 bytes a lane and fragment: S [warp][k-steps][2], Z of the first warp [2][2],
  // U' [warp][2][2], U [2]; and the rows' factors
  static constexpr int kS = 2 * (DK / 32) * 2 * 512, kZ = 4 * 512, kU = 2 * 4 * 512, kUh = 2 * 512, kF = 6 * 256;
  static constexpr int oZ = kS, oU = oZ + kZ, oUh = oU + kU, oF = oUh + kUh, kPair = oF + kF;
  static constexpr int oPair = kStages * kStage, oBar = oPair + 2 * kPair;
  static constexpr int kSmem = oBar + 2 * kStages * 8;
};

// (not volatile: a pure register operation, so independent products may be interleaved)
__device__ __forceinline__ void mma(float (&d)[4], const uint4& a, uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
}
// The largest of a row's values over the four lanes that hold it
__device__ __forceinline__ float row_max(float m) {
  m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
  return fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
}
// Two accumulator tiles (16 rows x 16 columns) as an A operand, rows g and g + 8 under u0 and u1
__device__ __forceinline__ void operand(const float (&x)[4], const float (&y)[4], const Unit& u0, const Unit& u1, uint4& hi, uint4& lo) {
  halves(x[0] * u0.to, x[1] * u0.to, hi.x, lo.x);
  halves(x[2] * u1.to, x[3] * u1.to, hi.y, lo.y);
  halves(y[0] * u0.to, y[1] * u0.to, hi.z, lo.z);
  halves(y[2] * u1.to, y[3] * u1.to, hi.w, lo.w);
}
template <int N>
__device__ __forceinline__ void clear(float (&x)[N][4]) {
#pragma unroll
  for (int n = 0; n < N; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) x[n][e] = 0.f;
}
template <int N>
__device__ __forceinline__ void rows_max(const float (&x)[N][4], float& m0, float& m1) {
  m0 = m1 = 0.f;
#pragma unroll
  for (int n = 0; n < N; ++n) {
    m0 = fmaxf(m0, fmaxf(fabsf(x[n][0]), fabsf(x[n][1])));
    m1 = fmaxf(m1, fmaxf(fabsf(x[n][2]), fabsf(x[n][3])));
  }
  m0 = row_max(m0);
  m1 = row_max(m1);
}

// A wait that gave up turns every later wait of its warp into nothing: the warps then run through their loops (on wrong
// data, in bounds) so that every barrier is still met, and the error word says that the results are void.
template <bool BF16, int DK>
__global__ void __launch_bounds__(kThreads, 1) chain_kernel(const __grid_constant__ DeltaFwdArgs a, const __grid_constant__ DeltaWork w) {
  using L = Cfg<DK>;
  constexpr int NT = DK / 16, KS = DK / 32;          // tiles of 8 columns and of 16 of this warp's half of S
  extern __shared__ __align__(1024) uint8_t smem[];
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::oBar);
  uint64_t* empty = full + kStages;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t4 = lane & 3;
  const int h = blockIdx.y, s = blockIdx.z, hv = a.geo.hv, dv = a.geo.dv;
  const DeltaSeq q = delta_seq(a.b, s);
  if (q.n < a.n_min || q.n > a.n_max) return;
  const int chunks = (q.n + C - 1) / C, base = delta_chunk_base(q.t0, s);
  // the chunks of this window
  const int c0 = max(0, w.first - base), c1 = min(chunks, w.first + w.count - base);
  if (c0 >= c1) return;
  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], kWarps);
    }
    mbar_init_fence();
  }
  const bool writes = __syncthreads_and(delta_writes(a.b, s, q, tid, kThreads));
  bool ok = true;
  auto wait = [&](uint64_t* b, uint32_t parity) {
    if (ok && !__all_sync(0xffffffffu, mbar_wait(b, parity))) {
      ok = false;
      if (lane == 0) atomicOr(a.b.err, (uint32_t)DELTA_TIMEOUT);
    }
  };

  if (warp == kWarps) {
    // ================================ the chunks ================================
    const uint16_t* v = a.v + (int64_t)q.t0 * a.v_stride + h * dv + blockIdx.x * 32;
    const uint32_t bytes = L::kKQ + kTPBytes + (uint32_t)sizeof(DeltaScalars) + C * 64;
    for (int i = c0; i < c1; ++i) {
      const int n = i - c0, st = n % kStages;
      if (n >= kStages) wait(&empty[st], (n / kStages - 1) & 1);
      uint8_t* to = smem + st * L::kStage;
      const int64_t id = base + i - w.first;
      if (lane == 0) {
        mbar_arrive_expect_tx(&full[st], bytes);
        bulk_g2s(to, w.kq + (id * a.geo.hk + h / a.geo.rep) * L::kKQ, L::kKQ, &full[st]);
        bulk_g2s(to + L::oTP, w.tp + (id * hv + h) * kTPBytes, kTPBytes, &full[st]);
        bulk_g2s(to + L::oSc, w.sc + id * hv + h, sizeof(DeltaScalars), &full[st]);
      }
      __syncwarp();
      // (rows behind the sequence's end repeat its last one; what they give is left out)
      for (int r = lane; r < C; r += 32)
        bulk_g2s(to + L::oV + r * kVRow, v + (int64_t)min(i * C + r, q.n - 1) * a.v_stride, 64, &full[st]);
    }
    // every copy has landed before the block may end (the chain waits for each; after a wait that gave up, here)
    for (int n = max(0, c1 - c0 - kStages); n < c1 - c0; ++n) wait(&full[n % kStages], (n / kStages) & 1);
    return;
  }

  // ================================ the chain ================================
  const int pair = warp >> 1, p = warp & 1;
  uint8_t* ex = smem + L::oPair + pair * L::kPair;
  auto frag = [&](int off, int k) -> uint4& { return reinterpret_cast<uint4*>(ex + off)[k * 32 + lane]; };
  auto factor = [&](int k) -> float2& { return reinterpret_cast<float2*>(ex + L::oF)[k * 32 + lane]; };
  const int col = blockIdx.x * 32 + pair * 16 + g;   // this lane's rows of S^T: the state's columns col and col + 8
  const int64_t slot = (int64_t)hv * DK * dv, at = (int64_t)h * DK * dv + col;
  float S[NT][4];
  {
    const float* src = c0 > 0 ? w.carry[w.parity] + at : q.in >= 0 ? a.state + q.in * slot + at : nullptr;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        S[n][e] = src ? src[(int64_t)(p * (DK / 2) + 8 * n + 2 * t4 + (e & 1)) * dv + 8 * (e >> 1)] : 0.f;
  }
  // this lane's place in four 8 x 8 tiles: row, piece
  const int lr = lane & 7, lm = lane >> 3;
  const int other = p ^ 1;
  const int s_own = p * KS * 2, s_other = other * KS * 2;

  for (int i = c0; i < c1; ++i) {
    const int n_ = i - c0, st = n_ % kStages, left = min(C, q.n - i * C);
    const uint8_t* stage = smem + st * L::kStage;
    const uint32_t kb = smem_u32(stage), qb = kb + L::kMat, tb = kb + L::oTP;
    const DeltaScalars& sc = *reinterpret_cast<const DeltaScalars*>(stage + L::oSc);
    // ---- S as an operand ----
    float m0, m1;
    rows_max(S, m0, m1);
    const Unit us0 = unit_of(m0), us1 = unit_of(m1);
    uint4 sh[KS], sl[KS];
#pragma unroll
    for (int k = 0; k < KS; ++k) {
      operand(S[2 * k], S[2 * k + 1], us0, us1, sh[k], sl[k]);
      frag(0, s_own + 2 * k) = sh[k];
      frag(0, s_own + 2 * k + 1) = sl[k];
    }
    factor(p) = make_float2(us0.from, us1.from);
    wait(&full[st], (n_ / kStages) & 1);
    // ---- Y^T = S^T K^T for this warp's 32 tokens, own half of the dimensions first ----
    float ya[4][4], yb[4][4], oa[4][4], ob[4][4];
    clear(ya);
    clear(yb);
    clear(oa);
    clear(ob);
    // B tiles of 8 tokens (row 32 p + 8 n) and 32 dimensions (half hf, 16-byte pieces from 4 j on)
    auto k_tiles = [&](uint32_t mat, int n, int hf, int j, uint32_t (&b)[4]) {
      const int ch = hf * (DK / 16) + 4 * j + lm;
      ldsm4(b, mat + (ch >> 3) * 8192 + sw128_offset(32 * p + 8 * n + lr, ch & 7));
    };
    // (products of one accumulator wait for one another: four tiles take turns)
    auto times = [&](float (&y)[4][4], const uint4& x0, const uint4& x1, const uint32_t (&b)[4][4]) {
#pragma unroll
      for (int n = 0; n < 4; ++n) mma(y[n], x0, b[n][0], b[n][1]);
#pragma unroll
      for (int n = 0; n < 4; ++n) mma(y[n], x1, b[n][2], b[n][3]);
    };
#pragma unroll
    for (int j = 0; j < KS / 2; ++j) {
      uint32_t b[4][4];
#pragma unroll
      for (int n = 0; n < 4; ++n) k_tiles(kb, n, p, j, b[n]);
      times(ya, sh[2 * j], sh[2 * j + 1], b);
      times(ya, sl[2 * j], sl[2 * j + 1], b);
    }
    named_bar(1 + 3 * pair, 64);
#pragma unroll
    for (int j = 0; j < KS / 2; ++j) {
      const uint4 h0 = frag(0, s_other + 4 * j), l0 = frag(0, s_other + 4 * j + 1), h1 = frag(0, s_other + 4 * j + 2),
                  l1 = frag(0, s_other + 4 * j + 3);
      uint32_t b[4][4];
#pragma unroll
      for (int n = 0; n < 4; ++n) k_tiles(kb, n, other, j, b[n]);
      times(yb, h0, h1, b);
      times(yb, l0, l1, b);
    }
    const float2 fo = factor(other);
    // ---- Q S, for the outputs only (its products run while Z is formed) ----
#pragma unroll
    for (int j = 0; j < KS / 2; ++j) {
      const uint4 h0 = frag(0, s_other + 4 * j), h1 = frag(0, s_other + 4 * j + 2);
      uint32_t b[4][4];
#pragma unroll
      for (int n = 0; n < 4; ++n) k_tiles(qb, n, p, j, b[n]);
      times(oa, sh[2 * j], sh[2 * j + 1], b);
#pragma unroll
      for (int n = 0; n < 4; ++n) k_tiles(qb, n, other, j, b[n]);
      times(ob, h0, h1, b);
    }
    // ---- Z ----
    float z[4][4];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      // V^T: tiles (tokens 16 j .. + 7, columns 0-7 | 8-15), (tokens 16 j + 8 .., the same)
      uint32_t v[4];
      ldsm4_t(v, kb + L::oV + (32 * p + 16 * j + 8 * (lm >> 1) + lr) * kVRow + pair * 32 + (lm & 1) * 16);
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const int n = 2 * j + y, tok = 32 * p + 8 * n + 2 * t4;
        const float2 c = *reinterpret_cast<const float2*>(&sc.c[tok]);
        const float2 v0 = unpack16<BF16>(v[2 * y]), v1 = unpack16<BF16>(v[2 * y + 1]);
        z[n][0] = v0.x - c.x * (us0.from * ya[n][0] + fo.x * yb[n][0]);
        z[n][1] = v0.y - c.y * (us0.from * ya[n][1] + fo.x * yb[n][1]);
        z[n][2] = v1.x - c.x * (us1.from * ya[n][2] + fo.y * yb[n][2]);
        z[n][3] = v1.y - c.y * (us1.from * ya[n][3] + fo.y * yb[n][3]);
        if (left < C) {
          if (tok >= left) z[n][0] = z[n][2] = 0.f;
          if (tok + 1 >= left) z[n][1] = z[n][3] = 0.f;
        }
      }
    }
    rows_max(z, m0, m1);
    const Unit uz0 = unit_of(m0), uz1 = unit_of(m1);
    uint4 zh[2], zl[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) operand(z[2 * k], z[2 * k + 1], uz0, uz1, zh[k], zl[k]);
    // ---- U^T = Z^T T^T: the second warp's tokens take the first one's Z too ----
    if (p == 0) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        frag(L::oZ, 2 * k) = zh[k];
        frag(L::oZ, 2 * k + 1) = zl[k];
      }
      factor(2) = make_float2(uz0.from, uz1.from);
      __threadfence_block();
      named_bar_arrive(2 + 3 * pair, 64);
    }
    float ua[4][4], ub[4][4];
    clear(ua);
    clear(ub);
    auto t_tiles = [&](uint32_t mat, int n, int half, uint32_t (&b)[4]) {      // token 32 p + 8 n, columns 32 half .. + 31
      ldsm4(b, mat + sw128_offset(32 * p + 8 * n + lr, 4 * half + lm));
    };
    {
      uint32_t bh[4][4], bl[4][4];
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        t_tiles(tb, n, p, bh[n]);
        t_tiles(tb + C * 128, n, p, bl[n]);
      }
#pragma unroll
      for (int n = 0; n < 4; ++n) mma(ua[n], zh[0], bh[n][0], bh[n][1]);
#pragma unroll
      for (int n = 0; n < 4; ++n) mma(ua[n], zl[0], bh[n][0], bh[n][1]);
#pragma unroll
      for (int n = 0; n < 4; ++n) mma(ua[n], zh[0], bl[n][0], bl[n][1]);
#pragma unroll
      for (int n = 2; n < 4; ++n) mma(ua[n], zh[1], bh[n][2], bh[n][3]);
#pragma unroll
      for (int n = 2; n < 4; ++n) mma(ua[n], zl[1], bh[n][2], bh[n][3]);
#pragma unroll
      for (int n = 2; n < 4; ++n) mma(ua[n], zh[1], bl[n][2], bl[n][3]);
    }
    float2 fz = make_float2(0.f, 0.f);
    if (p == 1) {
      named_bar(2 + 3 * pair, 64);
      const uint4 h0 = frag(L::oZ, 0), l0 = frag(L::oZ, 1), h1 = frag(L::oZ, 2), l1 = frag(L::oZ, 3);
      fz = factor(2);
      uint32_t bh[4][4], bl[4][4];
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        t_tiles(tb, n, 0, bh[n]);
        t_tiles(tb + C * 128, n, 0, bl[n]);
      }
      times(ub, h0, h1, bh);
      times(ub, l0, l1, bh);
      times(ub, h0, h1, bl);
    }
    // ---- U, and what it adds to the state ----
    float u[4][4], x[4][4];
#pragma unroll
    for (int n = 0; n < 4; ++n) {
      const int tok = 32 * p + 8 * n + 2 * t4;
      const float2 r = *reinterpret_cast<const float2*>(&sc.rs[tok]), wt = *reinterpret_cast<const float2*>(&sc.w[tok]);
      u[n][0] = r.x * (uz0.from * ua[n][0] + fz.x * ub[n][0]);
      u[n][1] = r.y * (uz0.from * ua[n][1] + fz.x * ub[n][1]);
      u[n][2] = r.x * (uz1.from * ua[n][2] + fz.y * ub[n][2]);
      u[n][3] = r.y * (uz1.from * ua[n][3] + fz.y * ub[n][3]);
      x[n][0] = wt.x * u[n][0];
      x[n][1] = wt.y * u[n][1];
      x[n][2] = wt.x * u[n][2];
      x[n][3] = wt.y * u[n][3];
    }
    rows_max(x, m0, m1);
    const Unit ux0 = unit_of(m0), ux1 = unit_of(m1);
    uint4 xh[2], xl[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      operand(x[2 * k], x[2 * k + 1], ux0, ux1, xh[k], xl[k]);
      frag(L::oU, p * 4 + 2 * k) = xh[k];
      frag(L::oU, p * 4 + 2 * k + 1) = xl[k];
    }
    factor(3 + p) = make_float2(ux0.from, ux1.from);
    rows_max(u, m0, m1);
    const Unit uu0 = unit_of(m0), uu1 = unit_of(m1);
    uint4 uh[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      uh[k].x = pack16<false>(u[2 * k][0] * uu0.to, u[2 * k][1] * uu0.to);
      uh[k].y = pack16<false>(u[2 * k][2] * uu1.to, u[2 * k][3] * uu1.to);
      uh[k].z = pack16<false>(u[2 * k + 1][0] * uu0.to, u[2 * k + 1][1] * uu0.to);
      uh[k].w = pack16<false>(u[2 * k + 1][2] * uu1.to, u[2 * k + 1][3] * uu1.to);
    }
    if (p == 0) {
      frag(L::oUh, 0) = uh[0];
      frag(L::oUh, 1) = uh[1];
      factor(5) = make_float2(uu0.from, uu1.from);
    }
    // ---- the state's update, this warp's half of the dimensions, own tokens first ----
    float da[NT][4], db[NT][4];
    clear(da);
    clear(db);
    // B tiles of 16 tokens (from row tok on) and dimensions 8 n .. + 15 of this half
    auto kt_tiles = [&](int tok, int n, uint32_t (&b)[4]) {
      const int ch = p * (DK / 16) + n + (lm >> 1);
      ldsm4_t(b, kb + (ch >> 3) * 8192 + sw128_offset(tok + 8 * (lm & 1) + lr, ch & 7));
    };
    auto add_to = [&](float (&d)[NT][4], const uint4& xh_, const uint4& xl_, int tok) {
      uint32_t b[NT / 2][4];
#pragma unroll
      for (int n = 0; n < NT; n += 2) kt_tiles(tok, n, b[n / 2]);
#pragma unroll
      for (int n = 0; n < NT; ++n) mma(d[n], xh_, b[n / 2][2 * (n & 1)], b[n / 2][2 * (n & 1) + 1]);
#pragma unroll
      for (int n = 0; n < NT; ++n) mma(d[n], xl_, b[n / 2][2 * (n & 1)], b[n / 2][2 * (n & 1) + 1]);
    };
#pragma unroll
    for (int k = 0; k < 2; ++k) add_to(da, xh[k], xl[k], 32 * p + 16 * k);
    named_bar(3 + 3 * pair, 64);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const uint4 h0 = frag(L::oU, other * 4 + 2 * k), l0 = frag(L::oU, other * 4 + 2 * k + 1);
      add_to(db, h0, l0, 32 * other + 16 * k);
    }
    const float2 fx = factor(3 + other);
    // ---- P U (these products run while S is formed) ----
    float pa[4][4], pb[4][4];
    clear(pa);
    clear(pb);
    {
      uint32_t b[4][4];
#pragma unroll
      for (int n = 0; n < 4; ++n) t_tiles(tb + 2 * C * 128, n, p, b[n]);
#pragma unroll
      for (int n = 0; n < 4; ++n) mma(pa[n], uh[0], b[n][0], b[n][1]);
#pragma unroll
      for (int n = 2; n < 4; ++n) mma(pa[n], uh[1], b[n][2], b[n][3]);
    }
    float2 fu = make_float2(0.f, 0.f);
    if (p == 1) {
      const uint4 h0 = frag(L::oUh, 0), h1 = frag(L::oUh, 1);
      fu = factor(5);
      uint32_t b[4][4];
#pragma unroll
      for (int n = 0; n < 4; ++n) t_tiles(tb + 2 * C * 128, n, 0, b[n]);
      times(pb, h0, h1, b);
    }
    const float gc = sc.decay[0];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      S[n][0] = gc * S[n][0] + (ux0.from * da[n][0] + fx.x * db[n][0]);
      S[n][1] = gc * S[n][1] + (ux0.from * da[n][1] + fx.x * db[n][1]);
      S[n][2] = gc * S[n][2] + (ux1.from * da[n][2] + fx.y * db[n][2]);
      S[n][3] = gc * S[n][3] + (ux1.from * da[n][3] + fx.y * db[n][3]);
    }
    // ---- outputs ----
#pragma unroll
    for (int n = 0; n < 4; ++n) {
      const int tok = 32 * p + 8 * n + 2 * t4;
      const float2 oq = *reinterpret_cast<const float2*>(&sc.oq[tok]), pq = *reinterpret_cast<const float2*>(&sc.pq[tok]);
      float o[4];
      o[0] = oq.x * (us0.from * oa[n][0] + fo.x * ob[n][0]) + pq.x * (uu0.from * pa[n][0] + fu.x * pb[n][0]);
      o[1] = oq.y * (us0.from * oa[n][1] + fo.x * ob[n][1]) + pq.y * (uu0.from * pa[n][1] + fu.x * pb[n][1]);
      o[2] = oq.x * (us1.from * oa[n][2] + fo.y * ob[n][2]) + pq.x * (uu1.from * pa[n][2] + fu.y * pb[n][2]);
      o[3] = oq.y * (us1.from * oa[n][3] + fo.y * ob[n][3]) + pq.y * (uu1.from * pa[n][3] + fu.y * pb[n][3]);
      // turned over: a lane gets the columns 2 t4, 2 t4 + 1 (and + 8) of token 8 n + g
      uint32_t r0 = pack16<BF16>(o[0], o[1]), r1 = pack16<BF16>(o[2], o[3]);
      asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %0;" : "+r"(r0));
      asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %0;" : "+r"(r1));
      const int row = 32 * p + 8 * n + g;
      if (row < left) {
        uint16_t* to = a.out + (((int64_t)q.t0 + i * C + row) * hv + h) * dv + blockIdx.x * 32 + pair * 16 + 2 * t4;
        *reinterpret_cast<uint32_t*>(to) = r0;
        *reinterpret_cast<uint32_t*>(to + 8) = r1;
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&empty[st]);
  }
  float* dst = c1 < chunks ? w.carry[w.parity ^ 1] + at : writes ? a.state + q.out * slot + at : nullptr;
  if (dst) {
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) dst[(int64_t)(p * (DK / 2) + 8 * n + 2 * t4 + (e & 1)) * dv + 8 * (e >> 1)] = S[n][e];
  }
}

template <bool BF16, int DK>
cudaError_t launch(const DeltaFwdArgs& a, const DeltaWork& w, cudaStream_t s) {
  constexpr int smem = Cfg<DK>::kSmem;
  static_assert(smem <= 227 * 1024, "shared memory");
  const cudaError_t e = ensure_dyn_smem(reinterpret_cast<const void*>(chain_kernel<BF16, DK>), smem);
  if (e != cudaSuccess) return e;
  chain_kernel<BF16, DK><<<dim3(a.geo.dv / 32, a.geo.hv, a.b.n_seqs), kThreads, smem, s>>>(a, w);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_delta_chain(const DeltaFwdArgs& a, const DeltaWork& w, cudaStream_t s) {
  const bool bf = a.geo.io == MOE_T_BF16;
  if (a.geo.dk == 128) return bf ? launch<true, 128>(a, w, s) : launch<false, 128>(a, w, s);
  return bf ? launch<true, 64>(a, w, s) : launch<false, 64>(a, w, s);
}

}  // namespace moe
