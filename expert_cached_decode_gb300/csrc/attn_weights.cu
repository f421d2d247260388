// Weights that a call's attention gives to the cells, few rows per K/V head:
// acc[j] = decay * acc[j] + sum over rows and heads of exp(scale q.k_j - lse).
//
// Bound by the bytes of K, which is read once.  A warp owns 64 cells of a
// sequence for all heads and rows, so a cell's sum needs no other warp: head
// by head it streams the cells' K vectors through a ring of its own (steps of
// 32 cells), multiplies them by the head's rows on mma.sync with the cells as
// columns, and adds the exponentials over the rows of a column; the eight
// lanes of a column are added once at the end.  The 64-cell units go to the
// warps of the GPU in turn, so short sequences spread over all SMs too.  One
// token of four sequences over 16,384 to 65,536 int8 cells takes 27 us, 44% of
// a copy's bandwidth: the 16 rows of a product, of which a token's eight query
// heads fill half, and their exponentials keep the issue slots half full.
#include "attn.cuh"

namespace moe {

namespace {

constexpr int kUnit = 64, kStep = 32;

template <int D, bool I8, int MT>
struct WgtCfg {
  static constexpr int kRowBytes = D * (I8 ? 1 : 2);
  static constexpr int kWarps = MT == 1 && kRowBytes <= 128 ? 16 : 8;
  static constexpr int kChunks = kRowBytes / 16;
  static constexpr int kPitch = kRowBytes + 16;               // as in attn_rows.cu
  static constexpr int kOffScale = kStep * kPitch;
  static constexpr int kStage = kOffScale + (I8 ? kStep * 4 : 0);
  static constexpr int kFit = 208 * 1024 / kWarps / kStage, kStages = kFit > 4 ? 4 : kFit;
  static constexpr int kRing = kWarps * kStages * kStage;
};

template <bool BF16, int D, bool I8, int MT>
__global__ void __launch_bounds__(WgtCfg<D, I8, MT>::kWarps * 32, 1) weights_rows_kernel(const __grid_constant__ AttnWgtArgs a) {
  using C = WgtCfg<D, I8, MT>;
  constexpr bool PBF = BF16 && !I8;                 // type of the products: the cells', fp16 for int8 cells
  constexpr int NT = C::kWarps * 32, ROWS = 16 * MT, RPI = 32 / C::kChunks, S = C::kStages;
  extern __shared__ __align__(128) uint8_t smem[];
  int32_t* first = reinterpret_cast<int32_t*>(smem + C::kRing);       // [n_seqs + 1] first unit of each sequence
  __shared__ int32_t wsum[32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c = lane & 3;
  const int G = a.g.g, HKV = a.g.hkv;
  // ---- units per sequence, as a running sum ----
  {
    const int per = (a.b.n_seqs + NT - 1) / NT, s0 = min(a.b.n_seqs, tid * per), s1 = min(a.b.n_seqs, s0 + per);
    int mine = 0;
    for (int s = s0; s < s1; ++s) mine += (min(seq_info(a.b, s).len, a.max_kv) + kUnit - 1) / kUnit;
    int inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int n = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += n;
    }
    if (lane == 31) wsum[warp] = inc;
    __syncthreads();
    int before = inc - mine;
    for (int w = 0; w < warp; ++w) before += wsum[w];
    for (int s = s0; s < s1; ++s) {
      first[s] = before;
      before += (min(seq_info(a.b, s).len, a.max_kv) + kUnit - 1) / kUnit;
    }
    if (s1 == a.b.n_seqs && s0 < s1) first[s1] = before;
    __syncthreads();
  }
  const int total = first[a.b.n_seqs];
  // Address of copies that read nothing.  It has to be aligned as the copies are (16 bytes), which the queries are checked
  // for and the call's int32 arrays are not; there are copies only where there are queries.
  const uint8_t* none = reinterpret_cast<const uint8_t*>(a.q);
  uint8_t* ring = smem + warp * S * C::kStage;
  const int v_off = 2 * HKV * C::kRowBytes;         // the K scales (int8)

  for (int u = warp * gridDim.x + blockIdx.x; u < total; u += C::kWarps * gridDim.x) {
    int s = 0, n = a.b.n_seqs;                      // the last sequence whose first unit is <= u
    while (n > 1) {
      const int h = n >> 1;
      if (first[s + h] <= u) {
        s += h;
        n -= h;
      } else {
        n = h;
      }
    }
    const SeqInfo q = seq_info(a.b, s);
    const int len = min(q.len, a.max_kv), jb = (u - first[s]) * kUnit;
    const uint8_t* cell[2];
    uint32_t vm[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int j = jb + x * kStep + lane;
      cell[x] = j < len ? cell_ptr(a.b, s, j) : nullptr;
      vm[x] = __ballot_sync(0xffffffffu, cell[x] != nullptr);
    }
    const RowSpan span = rows_that_see(jb, kUnit, q.n, q.len, a.b.window, G);
    const int ra = span.a, rb = span.b, rts = (rb - ra + ROWS - 1) / ROWS;
    const int n_steps = rts * HKV * 2;              // (row tile, head, half of the unit)
    auto issue = [&](int i) {
      uint8_t* st = ring + i % S * C::kStage;
      const int h = (i >> 1) % HKV;
      const uint8_t* mine = i & 1 ? cell[1] : cell[0];
      const int ch = lane % C::kChunks;
      const uint32_t to = smem_u32(st) + ch * 16;
#pragma unroll
      for (int x = 0; x < kStep / RPI; ++x) {
        const int row = x * RPI + lane / C::kChunks;
        const uint8_t* p = reinterpret_cast<const uint8_t*>(shfl_u64(reinterpret_cast<uint64_t>(mine), row));
        cp_async16(to + row * C::kPitch, p ? p + h * C::kRowBytes + ch * 16 : none, p ? 16 : 0);
      }
      if (I8) cp_async4(smem_u32(st + C::kOffScale) + 4 * lane, mine ? mine + v_off + 4 * h : none, mine ? 4 : 0);
    };
    float sum[2][4][2];
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
      for (int nt = 0; nt < 4; ++nt) sum[x][nt][0] = sum[x][nt][1] = 0.f;
    __syncwarp();
#pragma unroll
    for (int i = 0; i < S - 1; ++i) {
      if (i < n_steps) issue(i);
      cp_async_commit();
    }
#pragma unroll 1
    for (int i2 = 0; i2 < n_steps; i2 += 2) {
      // ---- Q fragments and row statistics of (row tile, head) ----
      const int rt = (i2 >> 1) / HKV, h = (i2 >> 1) - rt * HKV;
      uint32_t qf[MT][D / 16][4];
      float lse[MT][2], qs[MT][2];
      int rlo[MT][2], rhi[MT][2];
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int r = ra + rt * ROWS + m * 16 + g + 8 * e;
          const bool real = r < rb;
          const int t = real ? (int)fdiv((uint32_t)r, a.g.gdiv) : 0;
          const int hd = h * G + (real ? r - t * G : 0);
          row_range(q, a.b.window, t, rlo[m][e], rhi[m][e]);
          float x = INFINITY;                       // of a row that gives nothing
          if (real) x = a.lse[(int64_t)(q.q0 + t) * a.g.hq + hd];
          lse[m][e] = x == -INFINITY ? INFINITY : x * 1.4426950408889634f;
          const uint16_t* src = a.q + (int64_t)(q.q0 + t) * a.q_stride + hd * D;
#pragma unroll
          for (int p = 0; p < D / 32; ++p) {
            uint4 v = make_uint4(0, 0, 0, 0);
            if (real)
              v = *reinterpret_cast<const uint4*>(src + (I8 ? 16 * (c + 4 * (p >> 1)) + 8 * (p & 1) : 8 * (c + 4 * p)));
            qf[m][2 * p][e] = v.x;
            qf[m][2 * p][2 + e] = v.y;
            qf[m][2 * p + 1][e] = v.z;
            qf[m][2 * p + 1][2 + e] = v.w;
          }
          qs[m][e] = a.g.scale_log2;
          if (I8 && BF16) {                         // bf16 queries as fp16 in units of their row's largest
            float top = 0.f;
#pragma unroll
            for (int y = 0; y < D / 16; ++y)
#pragma unroll
              for (int z = 0; z < 2; ++z) {
                const float2 v = Half16<true>::unpack(qf[m][y][2 * z + e]);
                top = fmaxf(top, fmaxf(fabsf(v.x), fabsf(v.y)));
              }
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            const float u = row_unit(top), f = inv_pow2(u);
            qs[m][e] *= u;
#pragma unroll
            for (int y = 0; y < D / 16; ++y)
#pragma unroll
              for (int z = 0; z < 2; ++z) qf[m][y][2 * z + e] = bf16_to_f16(qf[m][y][2 * z + e], f);
          }
        }
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int i = i2 + x;
        __syncwarp();                               // the step before is done with its stage
        if (i + S - 1 < n_steps) issue(i + S - 1);
        cp_async_commit();
        cp_async_wait<S - 1>();
        __syncwarp();
        const uint8_t* st = ring + i % S * C::kStage;
        float sc[MT][4][4];
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int nt = 0; nt < 4; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) sc[m][nt][e] = 0.f;
#pragma unroll
        for (int p = 0; p < C::kChunks / 4; ++p)
#pragma unroll
          for (int nt = 0; nt < 4; ++nt) {
            const int row = 16 * (nt >> 1) + col_cell<I8>(nt & 1, g);
            const uint4 w = *reinterpret_cast<const uint4*>(st + row * C::kPitch + (c + 4 * p) * 16);
            if (!I8) {
#pragma unroll
              for (int m = 0; m < MT; ++m) {
                mma16816<PBF>(sc[m][nt], qf[m][2 * p], w.x, w.y);
                mma16816<PBF>(sc[m][nt], qf[m][2 * p + 1], w.z, w.w);
              }
            } else {
              const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
              for (int y = 0; y < 4; ++y) {
                uint32_t b0, b1;
                codes4_f16(ww[y], b0, b1);
#pragma unroll
                for (int m = 0; m < MT; ++m) mma16816<PBF>(sc[m][nt], qf[m][4 * p + y], b0, b1);
              }
            }
          }
        const int j0 = jb + x * kStep;
#pragma unroll
        for (int nt = 0; nt < 4; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int cl = 16 * (nt >> 1) + col_cell<I8>(nt & 1, 2 * c + e), j = j0 + cl;
            const float f = I8 ? reinterpret_cast<const float*>(st + C::kOffScale)[cl] : 1.f;
#pragma unroll
            for (int m = 0; m < MT; ++m) {
#pragma unroll
              for (int y = 0; y < 2; ++y) {
                const float p = ex2(fmaf(sc[m][nt][2 * y + e], I8 ? f * qs[m][y] : qs[m][y], -lse[m][y]));
                sum[x][nt][e] += j >= rlo[m][y] && j < rhi[m][y] ? p : 0.f;
              }
            }
          }
      }
    }
    cp_async_wait<0>();
    // ---- the rows of a column lie in the eight lanes of one c ----
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
      for (int nt = 0; nt < 4; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float v = sum[x][nt][e];
          v += __shfl_xor_sync(0xffffffffu, v, 4);
          v += __shfl_xor_sync(0xffffffffu, v, 8);
          v += __shfl_xor_sync(0xffffffffu, v, 16);
          const int cl = 16 * (nt >> 1) + col_cell<I8>(nt & 1, 2 * c + e), j = jb + x * kStep + cl;
          if (g == nt * 2 + e && j < len) {
            const int64_t at = (int64_t)s * a.acc_stride + j;
            a.acc_out[at] = (a.acc_in ? a.acc_in[at] * a.decay : 0.f) + (vm[x] >> cl & 1u ? v : 0.f);
          }
        }
  }
}

template <bool BF16, int D, bool I8, int MT>
cudaError_t launch_w(const AttnWgtArgs& a, cudaStream_t s) {
  using C = WgtCfg<D, I8, MT>;
  const int smem = C::kRing + (a.b.n_seqs + 1) * 4;
  static_assert(C::kRing + 4097 * 4 <= 226 * 1024, "shared memory");
  const cudaError_t e =
      ensure_dyn_smem(reinterpret_cast<const void*>(weights_rows_kernel<BF16, D, I8, MT>), C::kRing + 4097 * 4);
  if (e != cudaSuccess) return e;
  weights_rows_kernel<BF16, D, I8, MT><<<a.num_sms, C::kWarps * 32, smem, s>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attn_weights_rows(const AttnWgtArgs& a, int max_q, cudaStream_t s) {
  const int tiles = (int)((int64_t)max_q * a.g.g + 15) / 16;
  const bool bf = a.g.io == MOE_T_BF16, i8 = a.g.kv == MOE_T_I8;
#define WGT_MT(BF, DD, I)                            \
  return tiles <= 1   ? launch_w<BF, DD, I, 1>(a, s) \
         : tiles == 2 ? launch_w<BF, DD, I, 2>(a, s) \
                      : launch_w<BF, DD, I, 3>(a, s)
  if (a.g.D == 128) {
    if (bf && i8) WGT_MT(true, 128, true);
    if (bf) WGT_MT(true, 128, false);
    if (i8) WGT_MT(false, 128, true);
    WGT_MT(false, 128, false);
  }
  if (bf && i8) WGT_MT(true, 64, true);
  if (bf) WGT_MT(true, 64, false);
  if (i8) WGT_MT(false, 64, true);
  WGT_MT(false, 64, false);
#undef WGT_MT
}

}  // namespace moe
