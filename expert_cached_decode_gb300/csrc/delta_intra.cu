// What the gated delta rule's chunks of 64 tokens hold apart from the state
// (delta_chain.cu goes through them): for all chunks at once, a CTA per chunk and
// key head, its value heads one after another.
//
// With G_i the sum of g up to token i of the chunk,
//     A_ij = beta_i e^(G_i - G_j) k^_i.k^_j  (j < i),   T = (1 + A)^-1 diag(beta)
//     P_ij = e^(G_i - G_j) q^_i.k^_j  (j <= i)
// K and Q become fp16 under a power of two per row (bf16 rows are exact so, but
// for elements 2^-14 below their row's length), what is missing to k^ and q^ is a
// factor per row, and K K^T and Q K^T are exact products (mma.sync, a warp to 16
// rows).  e^(G_i - G_j) of different 16-token blocks is a product of two factors
// below 1, e^(G_i - G_r) e^(G_r - G_j) with r the first token of i's block; within a
// block it is taken from the difference, where G is a sum in 64-bit fixed point.
// (1 + A)^-1: powers of A would cancel where keys are alike, so 16 x 16 blocks are
// solved by forward substitution in fp32 (a lane per column), and
// T21 = -T22 (A21 T11) joins them to 32 and 64, in tf32 products of two halves each
// (22 bits, fp32's range); a warp takes 8 columns through both products.
// T is kept as fp16 pairs under a power of two per row, P as fp16.  Decays above 1 (the state grows within the chunk) would
// take P out of fp16's range and leave the early tokens' Z and U, which grow most on their way, the fewest bits: there every
// token of Z and of the outputs' U has a power of two, which the columns of T and P take up, and P's rows one of their own.
//
// Bound by latency through shared memory (47% of the issue slots, 24% of the warps; 12,288 tokens of 16 key and 32 value heads
// of 128: 125 us, 54 of them the bytes').  Registers for four CTAs an SM: when they were chosen that whole call took 469 us with three, 457 with
// four, 468 with five, 499 with six.
#include "delta.cuh"
#include "tc.cuh"

namespace moe {

namespace {

constexpr int C = kChunk;
constexpr int kThreads = 128;
// A and T: the 16 x 16 blocks (I, J) up to the diagonal, I (I + 1) / 2 + J, rows of kLd floats
constexpr int kLd = 20, kBlock = 16 * kLd;
__device__ __forceinline__ int block_at(int i, int j) { return (i * (i + 1) / 2 + j) * kBlock; }
// A stored row of K is shorter than 2: its DK numbers add up to 2 DK^1/2 at most.
constexpr float kLong = 22.63f;
template <int DK>
constexpr float kRoot = DK == 128 ? 11.32f : 8.f;    // DK^1/2: from a column's largest number to its length

__device__ __forceinline__ float ex2f(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_tf32(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void halves_tf32(float x, uint32_t& hi, uint32_t& lo) {
  hi = __float_as_uint(x) & 0xffffe000u;
  lo = __float_as_uint(x - __uint_as_float(hi));
}

template <int DK>
struct IntraSmem {
  union {
    uint8_t kq[2 * C * DK * 2];        // K, then Q; once their products are in registers:
    struct {
      union {
        struct {
          float A[10 * kBlock], M[32 * 36];
        };
        uint8_t timg[2 * C * 128];     // T's two images, once A has done
      };
      float T[10 * kBlock];
      uint8_t pimg[C * 128];
    };
  };
  float fk[C], fq[C], kn[C], gh[C], gl[C], beta[C], w[C], pu[C], tab[4][C];
  float part[4][4];
  DeltaScalars sc;
};

// 16-byte multiples shared -> global, asynchronously (one group), by one thread; and until the last group's bytes have been read
__device__ __forceinline__ void bulk_s2g(void* dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(smem_u32(src)), "r"(bytes) : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }

// d (16 x 8) += X[16 x 16] Y[16 x 8]: rows x0 .. of X, rows y0 .. of Y
__device__ __forceinline__ void product8(float (&d)[4], const float* X, int ldx, const float* Y, int ldy, int lane) {
  const int g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int k = 0; k < 16; k += 8) {
    const float xs[4] = {X[g * ldx + k + t], X[(g + 8) * ldx + k + t], X[g * ldx + k + t + 4], X[(g + 8) * ldx + k + t + 4]};
    const float ys[2] = {Y[(k + t) * ldy + g], Y[(k + t + 4) * ldy + g]};
    uint32_t xh[4], xl[4], yh[2], yl[2];
#pragma unroll
    for (int e = 0; e < 4; ++e) halves_tf32(xs[e], xh[e], xl[e]);
#pragma unroll
    for (int e = 0; e < 2; ++e) halves_tf32(ys[e], yh[e], yl[e]);
    mma_tf32(d, xl, yh[0], yh[1]);
    mma_tf32(d, xh, yl[0], yl[1]);
    mma_tf32(d, xh, yh[0], yh[1]);
  }
}
__device__ __forceinline__ void put8(float* Y, int ldy, const float (&d)[4], float f, int lane) {
  const int g = lane >> 2, t = lane & 3;
  *reinterpret_cast<float2*>(&Y[g * ldy + 2 * t]) = make_float2(f * d[0], f * d[1]);
  *reinterpret_cast<float2*>(&Y[(g + 8) * ldy + 2 * t]) = make_float2(f * d[2], f * d[3]);
}

template <bool BF16, int DK>
__global__ void __launch_bounds__(kThreads, 4) intra_kernel(const __grid_constant__ DeltaFwdArgs a, const __grid_constant__ DeltaWork w) {
  extern __shared__ __align__(1024) uint8_t raw[];
  IntraSmem<DK>& sm = *reinterpret_cast<IntraSmem<DK>*>(raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t4 = lane & 3;
  const int id = w.first + blockIdx.x, kh = blockIdx.y, hv = a.geo.hv, rep = a.geo.rep;
  // the sequence: the last one whose chunks begin at or before this one
  int lo = 0, hi = a.b.n_seqs;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (delta_chunk_base(min(max(a.b.cu[mid], 0), a.b.n_tokens), mid) <= id) lo = mid + 1;
    else hi = mid;
  }
  const int s = lo - 1;
  if (s < 0) return;
  const DeltaSeq q = delta_seq(a.b, s);
  if (q.n < a.n_min || q.n > a.n_max) return;
  const int local = id - delta_chunk_base(q.t0, s);
  if (local < 0 || local * C >= q.n) return;
  const int left = min(C, q.n - local * C);
  const int64_t t0 = (int64_t)q.t0 + local * C;

  // a lane's two tokens' decays and betas, of the next head
  float g_next[2], b_next[2];
  auto load_gates = [&](int h) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const bool in = 2 * lane + e < left;
      g_next[e] = in ? a.g[(t0 + 2 * lane + e) * hv + h] : 0.f;
      b_next[e] = in ? a.beta[(t0 + 2 * lane + e) * hv + h] : 0.f;
    }
  };
  load_gates(kh * rep);

  // ---- K and Q: fp16 under a power of two per row ----
  constexpr int CH = DK / 8, RP = kThreads / CH;   // 16-byte pieces of a row, rows of a pass
  constexpr int kMat = C * DK * 2;
  {
    const int ch = tid % CH, r0 = tid / CH;
    uint4 xs[2][C / RP];                 // both tensors' rows on their way at once
#pragma unroll
    for (int z = 0; z < 2; ++z) {
      const uint16_t* src = (z ? a.q + t0 * a.q_stride : a.k + t0 * a.k_stride) + kh * DK + 8 * ch;
      const int64_t stride = z ? a.q_stride : a.k_stride;
#pragma unroll
      for (int y = 0; y < C / RP; ++y) {
        const int r = y * RP + r0;
        xs[z][y] = make_uint4(0, 0, 0, 0);
        if (r < left) xs[z][y] = *reinterpret_cast<const uint4*>(src + r * stride);
      }
    }
#pragma unroll
    for (int z = 0; z < 2; ++z) {
      const uint4 (&x)[C / RP] = xs[z];
#pragma unroll
      for (int y = 0; y < C / RP; ++y) {
        const int r = y * RP + r0;
        const uint32_t u[4] = {x[y].x, x[y].y, x[y].z, x[y].w};
        float v[8], ss = 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 f = unpack16<BF16>(u[e]);
          v[2 * e] = f.x;
          v[2 * e + 1] = f.y;
          ss += f.x * f.x + f.y * f.y;
        }
#pragma unroll
        for (int o = 1; o < CH; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        const int e2 = ss > 0.f ? ((int)(__float_as_uint(ss) >> 23) - 127) >> 1 : 0;
        const float down = __uint_as_float((uint32_t)(127 - e2) << 23), up = __uint_as_float((uint32_t)(127 + e2) << 23);
        uint32_t o[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] = pack16<false>(v[2 * e] * down, v[2 * e + 1] * down);
        const uint32_t at = z * kMat + (ch >> 3) * 8192 + sw128_offset(r, ch & 7);
        const uint4 out = make_uint4(o[0], o[1], o[2], o[3]);
        *reinterpret_cast<uint4*>(sm.kq + at) = out;
        if (ch == 0) {
          const float f = a.geo.normalize ? rsqrtf(ss + a.geo.eps) : 1.f;
          (z ? sm.fq : sm.fk)[r] = r < left ? f * up : 0.f;
          if (!z) sm.kn[r] = r < left ? f * sqrtf(ss) : 0.f;      // |k^|
        }
      }
    }
  }
  fence_proxy_async_smem();
  __syncthreads();
  if (tid == 0) {
    bulk_s2g(w.kq + ((int64_t)blockIdx.x * a.geo.hk + kh) * 2 * kMat, sm.kq, 2 * kMat);
    bulk_commit();
  }
  // ---- K K^T and Q K^T, rows 16 warp .. + 15, columns up to the diagonal ----
  float kk[8][4], qk[8][4];
#pragma unroll
  for (int n = 0; n < 8; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) kk[n][e] = qk[n][e] = 0.f;
  {
    const uint32_t base = smem_u32(sm.kq);
    const int ar = 16 * warp + (lane & 15), ac = lane >> 4;                    // this lane's row and piece of an A tile
    const int br = (lane & 7) + ((lane >> 4) << 3), bc = (lane >> 3) & 1;      // of a pair of B tiles
#pragma unroll
    for (int k = 0; k < DK / 16; ++k) {
      const uint32_t blk = (k >> 2) * 8192, ch = 2 * (k & 3);
      uint32_t ak[4], aq[4];
      ldsm4(ak, base + blk + sw128_offset(ar, ch + ac));
      ldsm4(aq, base + kMat + blk + sw128_offset(ar, ch + ac));
#pragma unroll
      for (int n = 0; n < 8; n += 2) {
        if (n > 2 * warp) break;
        uint32_t b[4];
        ldsm4(b, base + blk + sw128_offset(8 * n + br, ch + bc));
        mma_f16(kk[n], ak, b[0], b[1]);
        mma_f16(kk[n + 1], ak, b[2], b[3]);
        mma_f16(qk[n], aq, b[0], b[1]);
        mma_f16(qk[n + 1], aq, b[2], b[3]);
      }
    }
  }
  const int i0 = 16 * warp + g, i1 = i0 + 8;       // this lane's rows
#pragma unroll 1
  for (int hh = 0; hh < rep; ++hh) {
    const int h = kh * rep + hh;
    const int64_t at = (int64_t)blockIdx.x * hv + h;
    uint8_t* tp = w.tp + at * kTPBytes;
    bool grows;                          // a decay of the chunk is above 1
    bool calm;                           // no token lengthens a column of the state but by its decay and its value
    if (tid == 0) bulk_wait_read();      // (K and Q, or the last head's images, have left)
    __syncthreads();                     // (and have been read, like its A and T)
    {
      // G in units of 2^-40 of a factor of two: g log2(e), with the product's own rounding error; a lane takes two tokens.
      // Every warp does it all, the same values in the same places: none has to wait for another.
      const float g2[2] = {g_next[0], g_next[1]}, be[2] = {b_next[0], b_next[1]};
      if (hh + 1 < rep) load_gates(h + 1);
      int64_t G[2];
      bool nan = false;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float x = fminf(fmaxf(g2[e], -176.f), 176.f);              // 2^-253: nothing is left
        const float ph = x * 1.44269502f, pl = fmaf(x, 1.44269502f, -ph) + x * 1.92596303e-8f;
        G[e] = (int64_t)(ph * 1.099511627776e12f) + (int64_t)(pl * 1.099511627776e12f);
        nan |= g2[e] != g2[e];
      }
      const uint32_t bad = __ballot_sync(0xffffffffu, nan);              // a NaN reaches its token and all behind it
      grows = __any_sync(0xffffffffu, g2[0] > 0.f || g2[1] > 0.f);
      G[1] += G[0];
      int64_t sum = G[1];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t x = __shfl_up_sync(0xffffffffu, (long long)sum, o);
        if (lane >= o) sum += x;
      }
      const int64_t before = sum - G[1], total = __shfl_sync(0xffffffffu, (long long)sum, 31);
      const float poison = bad & (0xffffffffu >> (31 - lane)) ? __int_as_float(0x7fc00000) : 0.f;
      float cmax = 0.f;
      bool wild = false;
      const float th = (float)(int)(total >> 32) * 0x1p-8f, tl = (float)(uint32_t)total * 0x1p-40f;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int t = 2 * lane + e;
        const int64_t x = before + (e ? G[1] : G[0]);
        const float gh = (float)(int)(x >> 32) * 0x1p-8f, gl = (float)(uint32_t)x * 0x1p-40f + poison;
        const float d = ex2f(gh + gl);
        sm.gh[t] = gh;
        sm.gl[t] = gl;
        sm.beta[t] = be[e];
        sm.sc.c[t] = d * sm.fk[t];
        sm.sc.oq[t] = a.geo.scale * d * sm.fq[t];
        sm.sc.pq[t] = a.geo.scale * sm.fq[t] * (1.f / kDeltaPUnit);
        sm.w[t] = ex2f((th - gh) + (tl - gl));
        cmax = fmaxf(cmax, d * sm.fk[t]);
        wild |= !(be[e] >= 0.f && be[e] * sm.kn[t] * sm.kn[t] <= 2.0001f);   // (64 tokens: 1.007, below the bounds' own 1.01)
      }
#pragma unroll
      for (int o = 16; o; o >>= 1) cmax = fmaxf(cmax, __shfl_xor_sync(0xffffffffu, cmax, o));
      calm = !__any_sync(0xffffffffu, wild);
      if (lane == 0) {
        sm.sc.decay = ex2f(th + tl + (bad ? __int_as_float(0x7fc00000) : 0.f));
        sm.sc.zs = kLong * cmax;
      }
      // Where something grows, tokens have a power of two up >= e^(G_i) (DeltaScalars::up), which P's columns take up, and P's
      // row i, at most e^(G_i) / min e^(G_j) 2^-up_j then, one of its own.
      if (grows) {
        const int64_t here[2] = {before + G[0], before + G[1]};
        int up[2];
        int64_t held[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          up[e] = min(max((int)((here[e] + (1ll << 40) - 1) >> 40), 0), 120);
          held[e] = here[e] - ((int64_t)up[e] << 40);
        }
        int64_t least = held[0] < held[1] ? held[0] : held[1];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int64_t x = __shfl_up_sync(0xffffffffu, (long long)least, o);
          if (lane >= o && x < least) least = x;
        }
        const int64_t past = __shfl_up_sync(0xffffffffu, (long long)least, 1);
        held[0] = lane && past < held[0] ? past : held[0];
        held[1] = least;
        float most = 0.f;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int t = 2 * lane + e, rise = min((int)((here[e] - held[e] + (1ll << 40) - 1) >> 40), 120);
          sm.pu[t] = kDeltaPUnit * power2(-rise);
          sm.sc.pq[t] = a.geo.scale * sm.fq[t] * (1.f / kDeltaPUnit) * power2(rise);
          sm.sc.up[t] = (uint8_t)up[e];
          sm.sc.c[t] = ex2f((sm.gh[t] - (float)up[e]) + sm.gl[t]) * sm.fk[t];
          most = fmaxf(most, sm.sc.c[t]);
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
        if (lane == 0) sm.sc.zs = kLong * most;
      }
    }
    __syncwarp();
    // e^(G_r - G_j), r = 16 warp, j before it
    for (int j = lane; j < 16 * warp; j += 32) sm.tab[warp][j] = ex2f((sm.gh[16 * warp] - sm.gh[j]) + (sm.gl[16 * warp] - sm.gl[j]));
    __syncwarp();
    // ---- A and P ----
    {
      const float gh0 = sm.gh[i0], gl0 = sm.gl[i0], gh1 = sm.gh[i1], gl1 = sm.gl[i1];
      const float r0 = ex2f((gh0 - sm.gh[16 * warp]) + (gl0 - sm.gl[16 * warp]));
      const float r1 = ex2f((gh1 - sm.gh[16 * warp]) + (gl1 - sm.gl[16 * warp]));
      const float bk0 = sm.beta[i0] * sm.fk[i0], bk1 = sm.beta[i1] * sm.fk[i1];
#pragma unroll
      for (int n = 0; n < 8; ++n) {
        const int j = 8 * n + 2 * t4;
        float d[4] = {0.f, 0.f, 0.f, 0.f};
        if (n < 2 * warp) {
          const float2 tb = *reinterpret_cast<const float2*>(&sm.tab[warp][j]);
          d[0] = r0 * tb.x;
          d[1] = r0 * tb.y;
          d[2] = r1 * tb.x;
          d[3] = r1 * tb.y;
        } else if (n <= 2 * warp + 1) {
          const float2 hj = *reinterpret_cast<const float2*>(&sm.gh[j]), lj = *reinterpret_cast<const float2*>(&sm.gl[j]);
          d[0] = j <= i0 ? ex2f((gh0 - hj.x) + (gl0 - lj.x)) : 0.f;
          d[1] = j < i0 ? ex2f((gh0 - hj.y) + (gl0 - lj.y)) : 0.f;
          d[2] = j <= i1 ? ex2f((gh1 - hj.x) + (gl1 - lj.x)) : 0.f;
          d[3] = j < i1 ? ex2f((gh1 - hj.y) + (gl1 - lj.y)) : 0.f;
        }
        if (n <= 2 * warp + 1) {
          const float2 fj = *reinterpret_cast<const float2*>(&sm.fk[j]);
          float2 x0 = make_float2(kk[n][0] * d[0] * (bk0 * fj.x), kk[n][1] * d[1] * (bk0 * fj.y));
          float2 x1 = make_float2(kk[n][2] * d[2] * (bk1 * fj.x), kk[n][3] * d[3] * (bk1 * fj.y));
          if (n >= 2 * warp) {
            if (j >= i0) x0.x = 0.f;
            if (j + 1 >= i0) x0.y = 0.f;
            if (j >= i1) x1.x = 0.f;
            if (j + 1 >= i1) x1.y = 0.f;
          }
          float* to = sm.A + block_at(warp, n >> 1) + g * kLd + (j & 15);
          *reinterpret_cast<float2*>(to) = x0;
          *reinterpret_cast<float2*>(to + 8 * kLd) = x1;
        }
        // (what lies right of the diagonal's 16 x 16 block is written too: it is read as zeros)
        const bool in = n <= 2 * warp + 1;
        const uint32_t p0 = in ? pack16<false>(kDeltaPUnit * qk[n][0] * d[0], kDeltaPUnit * qk[n][1] * d[1]) : 0u;
        const uint32_t p1 = in ? pack16<false>(kDeltaPUnit * qk[n][2] * d[2], kDeltaPUnit * qk[n][3] * d[3]) : 0u;
        *reinterpret_cast<uint32_t*>(sm.pimg + sw128_offset(i0, n) + 4 * t4) = p0;
        *reinterpret_cast<uint32_t*>(sm.pimg + sw128_offset(i1, n) + 4 * t4) = p1;
      }
    }
    __syncwarp();
    // ---- the 16 x 16 blocks of the diagonal: a lane per column ----
    {
      const float* B = sm.A + block_at(warp, warp);
      const int c = lane & 15;
      float x[16];
#pragma unroll
      for (int k = 0; k < 16; ++k) {
        float p[2] = {k == c ? 1.f : 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < k; j += 4) {
          const float4 b4 = *reinterpret_cast<const float4*>(&B[k * kLd + j]);
          const float bb[4] = {b4.x, b4.y, b4.z, b4.w};
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (j + e < k) p[e & 1] -= bb[e] * x[j + e];
        }
        x[k] = p[0] + p[1];
        if (lane < 16) sm.T[block_at(warp, warp) + k * kLd + c] = x[k];
      }
    }
    __syncthreads();
    if (grows && tid < C) sm.beta[tid] *= power2(sm.sc.up[tid]);         // (A has taken it as it was)
    // ---- joined to 32 x 32: warps 0 and 1 the blocks 0 and 1, warps 2 and 3 the others; 8 columns a warp ----
    {
      const int b = 2 * (warp >> 1), c = 8 * (warp & 1);
      float d[4] = {0.f, 0.f, 0.f, 0.f};
      float* m = sm.M + 9 * warp * 32;               // (16 rows of 9, apart from the other warps')
      product8(d, sm.A + block_at(b + 1, b), kLd, sm.T + block_at(b, b) + c, kLd, lane);
      const int gg = lane >> 2, t = lane & 3;
      m[gg * 9 + 2 * t] = d[0];
      m[gg * 9 + 2 * t + 1] = d[1];
      m[(gg + 8) * 9 + 2 * t] = d[2];
      m[(gg + 8) * 9 + 2 * t + 1] = d[3];
      __syncwarp();
      float o[4] = {0.f, 0.f, 0.f, 0.f};
      product8(o, sm.T + block_at(b + 1, b + 1), kLd, m, 9, lane);
      put8(sm.T + block_at(b + 1, b) + c, kLd, o, -1.f, lane);
    }
    __syncthreads();
    // ---- and to 64 x 64: 8 of the 32 columns a warp ----
    {
      const int cb = warp >> 1, c = 8 * (warp & 1);      // the columns' block, and place there
      float d[2][4] = {};
#pragma unroll
      for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int k = 0; k < 2; ++k)
          if (k >= cb) product8(d[r], sm.A + block_at(2 + r, k), kLd, sm.T + block_at(k, cb) + c, kLd, lane);
      float* m = sm.M + 9 * warp * 32;
      const int gg = lane >> 2, t = lane & 3;
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        m[(16 * r + gg) * 9 + 2 * t] = d[r][0];
        m[(16 * r + gg) * 9 + 2 * t + 1] = d[r][1];
        m[(16 * r + gg + 8) * 9 + 2 * t] = d[r][2];
        m[(16 * r + gg + 8) * 9 + 2 * t + 1] = d[r][3];
      }
      __syncwarp();
      float o[2][4] = {};
      product8(o[0], sm.T + block_at(2, 2), kLd, m, 9, lane);
      product8(o[1], sm.T + block_at(3, 2), kLd, m, 9, lane);
      product8(o[1], sm.T + block_at(3, 3), kLd, m + 16 * 9, 9, lane);
      put8(sm.T + block_at(2, cb) + c, kLd, o[0], -1.f, lane);
      put8(sm.T + block_at(3, cb) + c, kLd, o[1], -1.f, lane);
    }
    __syncthreads();
    if (grows) {                         // P again, with its powers of two
#pragma unroll
      for (int n = 0; n < 8; ++n) {
        if (n > 2 * warp + 1) break;
        const int j = 8 * n + 2 * t4;
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const int i = r ? i1 : i0;
          float x[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float d = j + e <= i ? ex2f((sm.gh[i] - sm.gh[j + e]) + (sm.gl[i] - sm.gl[j + e])) : 0.f;
            x[e] = sm.pu[i] * qk[n][2 * r + e] * d * power2(sm.sc.up[j + e]);
          }
          *reinterpret_cast<uint32_t*>(sm.pimg + sw128_offset(i, n) + 4 * t4) = pack16<false>(x[0], x[1]);
        }
      }
    }
    // ---- T diag(beta) as pairs, under a power of two per row; two threads a row ----
    {
      const int tr = tid >> 1, c0 = (tid & 1) * 32;
      float hold = 1.f, sum_v = 0.f;     // 2^-up of U in the outputs' products; V's part of U has T's columns without theirs
      if (grows) {
        hold = power2(-sm.sc.up[tr]);
#pragma unroll 1
        for (int j = 0; j <= tr; ++j) sum_v += fabsf(sm.T[block_at(tr >> 4, j >> 4) + (tr & 15) * kLd + (j & 15)] * sm.beta[j] * power2(-sm.sc.up[j]));
      }
      float x[32], mx = 0.f, sum = 0.f, late = 0.f;
#pragma unroll
      for (int j = 0; j < 32; j += 4) {
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if ((tr >> 4) >= ((c0 + j) >> 4)) v = *reinterpret_cast<const float4*>(&sm.T[block_at(tr >> 4, (c0 + j) >> 4) + (tr & 15) * kLd + (j & 15)]);
        const float4 b4 = *reinterpret_cast<const float4*>(&sm.beta[c0 + j]), g4 = *reinterpret_cast<const float4*>(&sm.sc.c[c0 + j]);
        const float c4[4] = {g4.x, g4.y, g4.z, g4.w};
        x[j] = v.x * b4.x;
        x[j + 1] = v.y * b4.y;
        x[j + 2] = v.z * b4.z;
        x[j + 3] = v.w * b4.w;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          mx = fmaxf(mx, fabsf(x[j + e]));
          sum += fabsf(x[j + e]);
          late += fabsf(x[j + e]) * c4[e];
        }
      }
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      sum += __shfl_xor_sync(0xffffffffu, sum, 1);
      late += __shfl_xor_sync(0xffffffffu, late, 1);
      const Unit ut = unit_of(mx);
      const float fk = sm.fk[tr], wr = sm.w[tr];
      if (grows) sum = sum_v;
      if (!(tid & 1)) {
        sm.sc.rs[tr] = ut.from * (fk * hold);
        sm.sc.rx[tr] = ut.from * fk * wr;
      }
      // (each row twice in a warp, like the halves of its sums; b[2]: what values add to the next S)
      float b[3] = {sum * (fk * hold), kLong * late * (fk * hold), wr * (sm.beta[tr] * hold) * sm.kn[tr]};
#pragma unroll
      for (int o = 16; o; o >>= 1) {
        b[0] = fmaxf(b[0], __shfl_xor_sync(0xffffffffu, b[0], o));
        b[1] = fmaxf(b[1], __shfl_xor_sync(0xffffffffu, b[1], o));
        b[2] += __shfl_xor_sync(0xffffffffu, b[2], o);
      }
      if (!calm) {                       // by sums over T; a stored row's numbers are below 2
        float c[2] = {sum * fk * wr, kLong * late * fk * wr};
#pragma unroll
        for (int o = 16; o; o >>= 1) {
          c[0] += __shfl_xor_sync(0xffffffffu, c[0], o);
          c[1] += __shfl_xor_sync(0xffffffffu, c[1], o);
        }
        b[2] = c[0];
        if (lane == 0) sm.part[3][warp] = c[1];
      }
      if (lane == 0) {
#pragma unroll
        for (int e = 0; e < 3; ++e) sm.part[e][warp] = b[e];
      }
#pragma unroll
      for (int j = 0; j < 32; j += 8) {
        uint32_t vh[4], vl[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) halves(x[j + 2 * e] * ut.to, x[j + 2 * e + 1] * ut.to, vh[e], vl[e]);
        const uint32_t o = sw128_offset(tr, (c0 + j) / 8);
        *reinterpret_cast<uint4*>(sm.timg + o) = make_uint4(vh[0], vh[1], vh[2], vh[3]);
        *reinterpret_cast<uint4*>(sm.timg + C * 128 + o) = make_uint4(vl[0], vl[1], vl[2], vl[3]);
      }
    }
    fence_proxy_async_smem();
    __syncthreads();
    if (tid == 0) {
      bulk_s2g(tp, sm.timg, 2 * C * 128);
      bulk_s2g(tp + 2 * C * 128, sm.pimg, C * 128);
      bulk_commit();
    }
    for (int e = tid; e < (5 * C * 4 + C) / 16; e += kThreads) reinterpret_cast<uint4*>(w.sc + at)[e] = reinterpret_cast<const uint4*>(&sm.sc)[e];
    if (tid == kThreads - 1) {
      const float(&p)[4][4] = sm.part;
      DeltaScalars& o = w.sc[at];
      o.grows = grows;
      o.decay = sm.sc.decay;
      o.zs = sm.sc.zs;
      o.uv = fmaxf(fmaxf(p[0][0], p[0][1]), fmaxf(p[0][2], p[0][3]));
      o.us = fmaxf(fmaxf(p[1][0], p[1][1]), fmaxf(p[1][2], p[1][3]));
      // 1 - beta k^ k^T lengthens no column while beta |k^|^2 is in [0, 2], so the next S's columns are at most e^(G_C) times
      // these and v times the sum of e^(G_C - G_i) beta_i |k^_i|; twice that also covers each token's U' (below 1 + beta |k^|^2
      // times it).
      o.xv = ((p[2][0] + p[2][1]) + (p[2][2] + p[2][3])) * (calm ? 1.01f : 1.f);
      o.xs = calm ? (2.02f * kRoot<DK> - 1.f) * sm.sc.decay : (p[3][0] + p[3][1]) + (p[3][2] + p[3][3]);
    }
  }
  if (tid == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}

template <bool BF16, int DK>
cudaError_t launch(const DeltaFwdArgs& a, const DeltaWork& w, cudaStream_t s) {
  constexpr int smem = (int)sizeof(IntraSmem<DK>);
  const cudaError_t e = ensure_dyn_smem(reinterpret_cast<const void*>(intra_kernel<BF16, DK>), smem);
  if (e != cudaSuccess) return e;
  intra_kernel<BF16, DK><<<dim3(w.count, a.geo.hk), kThreads, smem, s>>>(a, w);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_delta_intra(const DeltaFwdArgs& a, const DeltaWork& w, cudaStream_t s) {
  const bool bf = a.geo.io == MOE_T_BF16;
  if (a.geo.dk == 128) return bf ? launch<true, 128>(a, w, s) : launch<false, 128>(a, w, s);
  return bf ? launch<true, 64>(a, w, s) : launch<false, 64>(a, w, s);
}

}  // namespace moe
