// Attention of few rows (single tokens, short drafts) over the paged cache:
// up to 32 rows (tokens times query heads per K/V head) per K/V head.
//
// Bound by the cells' bytes: every cell is read once for all rows of its K/V
// head.  A CTA's eight warps take steps of 16 cells in turn, each through a
// ring of its own that cp.async fills, with its own running maximum, sum and
// output (online softmax), so no warp waits for another before the item's end;
// there the warps' results are joined in shared memory, and the parts of an
// item that several CTAs share in global memory, by the CTA that arrives last,
// in the order of the parts.
//
// Products on mma.sync m16n8k16: at 16 or 32 rows they need a fraction of the
// memory time, and their B fragments come straight from the rows of K and V.
// The order in which a contraction runs is free, so a lane's 16-byte piece of
// K (8 or 16 dimensions of one cell) feeds two or four products as it lies,
// with Q's fragments loaded to match, and int8 V feeds products whose column
// n of tile j is dimension n * (D / 8) + j.  int8 codes become 16-bit floats exactly; the
// K scale multiplies the score, the V scale the probability.
#include "attn.cuh"

namespace moe {

namespace {

constexpr int kWarps = 8, kNT = kWarps * 32, kStep = 16, kTK = kWarps * kStep;
// Fewest tiles of a part: joining parts costs as much as reading some 512 cells.
constexpr int kMinUnits = 4;

template <int D, bool I8>
struct RowsCfg {
  static constexpr int kRowBytes = D * (I8 ? 1 : 2);          // of one head vector
  static constexpr int kChunks = kRowBytes / 16;
  static constexpr int kMat = kStep * kRowBytes;               // K or V of a step
  static constexpr int kStage = 2 * kMat + (I8 ? 2 * kStep * 4 : 0);
  // bytes in flight per SM: (stages - 1) * 8 warps * stage, 128 KB at 16-bit D = 128
  static constexpr int kStages = (I8 || D == 64) ? 5 : 3;
  static constexpr int kRing = kStages * kStage;
  static constexpr int kSmem = kWarps * kRing;
};

// places of 16-byte chunks in a row of the ring: lanes that read together hit different banks
template <int CH>
__device__ __forceinline__ int k_chunk(int row, int c) { return CH >= 8 ? c ^ ((row & 1) << 2) : c; }
template <int CH, bool I8>
__device__ __forceinline__ int v_chunk(int row, int c) {
  if (!I8) return c ^ (row & 7);
  return CH >= 8 ? c ^ (((row >> 2) & 3) << 1) : c ^ (((row >> 2) & 1) << 1);
}

// the cell (within a step) of column n of n-tile nt: plain for 16-bit cells; for
// int8 cells the four that lane c's probabilities belong to lie next to each other
template <bool I8>
__device__ __forceinline__ int col_cell(int nt, int n) { return I8 ? 4 * (n >> 1) + 2 * nt + (n & 1) : 8 * nt + n; }

template <bool BF16, int D, bool I8, int MT>
__global__ void __launch_bounds__(kNT, 1) rows_kernel(const __grid_constant__ AttnFwdArgs a) {
  using C = RowsCfg<D, I8>;
  constexpr int ROWS = 16 * MT;
  constexpr bool PBF = I8 || BF16;       // probabilities and V: bf16 for int8 cells (range), else the cells' type
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ CursorScratch scr;
  __shared__ float sm_m[kWarps][ROWS], sm_l[kWarps][ROWS];
  __shared__ int last_flag;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c = lane & 3;
  const int G = a.g.g, HKV = a.g.hkv;
  Cursor cu;
  if (!find_part<ROWS, kTK, kNT, kMinUnits>(a.b, G, HKV, scr, cu)) return;
  const uint8_t* none = reinterpret_cast<const uint8_t*>(a.q);   // address of copies that read nothing
  uint8_t* ring = smem + warp * C::kRing;
  const uint32_t ring_a = smem_u32(ring);

  while (cu.u < cu.end) {
    const SeqInfo q = seq_info(a.b, cu.s);
    int lo, hi;
    const int units = Work<ROWS, kTK>::units(q, G, a.b.window, cu.rt, lo, hi);
    const int t0 = cu.t, t1 = (int)min((int64_t)units, t0 + (cu.end - cu.u));
    const int h = cu.h, s = cu.s, r0 = cu.rt * ROWS, nrows = min(ROWS, q.n * G - r0);
    // ---- Q fragments, scaled scores' factor stays outside (exact products) ----
    uint32_t qf[MT][D / 16][4];
    int rlo[MT][2], rhi[MT][2];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = r0 + m * 16 + g + 8 * e;
        const bool real = m * 16 + g + 8 * e < nrows;
        const int i = real ? r / G : 0;
        row_range(q, a.b.window, i, rlo[m][e], rhi[m][e]);
        if (!real) rlo[m][e] = rhi[m][e] = 0;
        const uint16_t* src = a.q + (int64_t)(q.q0 + i) * a.q_stride + (h * G + (real ? r - i * G : 0)) * D;
#pragma unroll
        for (int p = 0; p < D / 32; ++p) {
          // 16-bit cells: chunk c + 4p (8 dimensions) feeds products 2p, 2p + 1.
          // int8 cells: chunk c + 4(p/2) (16 dimensions), its words 2(p%2), 2(p%2) + 1 feed them.
          uint2 w0, w1;
          if (!I8) {
            const uint4 v = *reinterpret_cast<const uint4*>(src + 8 * (c + 4 * p));
            w0 = make_uint2(v.x, v.y);
            w1 = make_uint2(v.z, v.w);
          } else {
            const uint4 v = *reinterpret_cast<const uint4*>(src + 16 * (c + 4 * (p >> 1)) + 8 * (p & 1));
            w0 = make_uint2(v.x, v.y);
            w1 = make_uint2(v.z, v.w);
          }
          qf[m][2 * p][e] = real ? w0.x : 0u;
          qf[m][2 * p][2 + e] = real ? w0.y : 0u;
          qf[m][2 * p + 1][e] = real ? w1.x : 0u;
          qf[m][2 * p + 1][2 + e] = real ? w1.y : 0u;
        }
      }
    float o[MT][D / 8][4], mx[MT][2], l[MT][2];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
#pragma unroll
      for (int j = 0; j < D / 8; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[m][j][e] = 0.f;
      mx[m][0] = mx[m][1] = -INFINITY;
      l[m][0] = l[m][1] = 0.f;
    }
    // ---- this warp's steps: cells [j0 + 16 i, + 16), i = warp, warp + 8, ... ----
    const int jbase = (lo / kTK + t0) * kTK;
    const int jend = min(hi, jbase + (t1 - t0) * kTK);
    const int n_steps = jend > jbase ? (jend - jbase + kStep - 1) / kStep : 0;
    const int my = n_steps > warp ? (n_steps - warp + kWarps - 1) / kWarps : 0;
    const int head_off = h * C::kRowBytes, v_off = HKV * C::kRowBytes;
    const int sc_off = 2 * HKV * C::kRowBytes + 4 * h;
    // lane i < 16 finds the cell i of a step (NULL: hidden from every row)
    auto find = [&](int i) -> const uint8_t* {
      const int j = jbase + (warp + i * kWarps) * kStep + (lane & 15);
      return (i < my && j >= lo && j < jend) ? cell_ptr(a.b, s, j) : nullptr;
    };
    auto issue = [&](int i, const uint8_t* cell) {
      const uint32_t st = ring_a + (i % C::kStages) * C::kStage;
      const uint64_t p = reinterpret_cast<uint64_t>(cell);
      constexpr int per = 32 / C::kChunks;          // rows per instruction
      const int ch = lane % C::kChunks;
#pragma unroll
      for (int x = 0; x < kStep / per; ++x) {
        const int row = x * per + lane / C::kChunks;
        const uint64_t pr = shfl_u64(p, row);
        const uint8_t* src = pr ? reinterpret_cast<const uint8_t*>(pr) + head_off + ch * 16 : none;
        cp_async16(st + (row * C::kChunks + k_chunk<C::kChunks>(row, ch)) * 16, src, pr ? 16 : 0);
        cp_async16(st + C::kMat + (row * C::kChunks + v_chunk<C::kChunks, I8>(row, ch)) * 16, pr ? src + v_off : src,
                   pr ? 16 : 0);
      }
      if (I8) {                                     // lanes 0-15 the K scales, 16-31 the V scales
        const uint64_t pr = shfl_u64(p, lane & 15);
        const uint8_t* src = pr ? reinterpret_cast<const uint8_t*>(pr) + sc_off + (lane >> 4) * 4 * HKV : none;
        cp_async4(st + 2 * C::kMat + lane * 4, src, pr ? 4 : 0);
      }
    };
    uint32_t valid[C::kStages];                     // cells of the ring's steps that are there
    const uint8_t* nxt = find(0);
#pragma unroll
    for (int i = 0; i < C::kStages - 1; ++i) {
      valid[i] = __ballot_sync(0xffffffffu, nxt != nullptr) & 0xffffu;
      if (i < my) issue(i, nxt);
      cp_async_commit();
      nxt = find(i + 1);
    }
    for (int i0 = 0; i0 < my; i0 += C::kStages) {
#pragma unroll
      for (int k = 0; k < C::kStages; ++k) {        // unrolled so that `valid` stays in registers
        const int i = i0 + k;
        if (i >= my) break;
        constexpr int kAhead = C::kStages - 1;
        valid[(k + kAhead) % C::kStages] = __ballot_sync(0xffffffffu, nxt != nullptr) & 0xffffu;
        if (i + kAhead < my) issue(i + kAhead, nxt);
        cp_async_commit();
        nxt = find(i + C::kStages);
        cp_async_wait<kAhead>();
        __syncwarp();
        const uint8_t* st = ring + k * C::kStage;
        const int j0 = jbase + (warp + i * kWarps) * kStep;
        float ks[4], vs[4];
        if (I8) {                                   // of this lane's columns: [nt][e]
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const float* sc = reinterpret_cast<const float*>(st + 2 * C::kMat);
            const int cell = col_cell<I8>(x >> 1, 2 * c + (x & 1));
            ks[x] = sc[cell];
            vs[x] = sc[16 + cell];
          }
        }
        // ---- scores ----
        float sc[MT][2][4];
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int nt = 0; nt < 2; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) sc[m][nt][e] = 0.f;
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) {
          const int row = col_cell<I8>(nt, g);
          const uint8_t* rp = st + row * C::kRowBytes;
#pragma unroll
          for (int p = 0; p < C::kChunks / 4; ++p) {
            const uint4 w = *reinterpret_cast<const uint4*>(rp + k_chunk<C::kChunks>(row, c + 4 * p) * 16);
            if (!I8) {
#pragma unroll
              for (int m = 0; m < MT; ++m) {
                mma16816<BF16>(sc[m][nt], qf[m][2 * p], w.x, w.y);
                mma16816<BF16>(sc[m][nt], qf[m][2 * p + 1], w.z, w.w);
              }
            } else {
              const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
              for (int x = 0; x < 4; ++x) {
                const uint32_t b0 = codes2<BF16>(__byte_perm(ww[x], 0, 0x4140)),
                               b1 = codes2<BF16>(__byte_perm(ww[x], 0, 0x4342));
#pragma unroll
                for (int m = 0; m < MT; ++m) mma16816<BF16>(sc[m][nt], qf[m][4 * p + x], b0, b1);
              }
            }
          }
        }
        // ---- online softmax (base 2) ----
        const uint32_t vm = valid[k];
        uint32_t pf[MT][4];
        bool grew = false;
        float nm[MT][2];
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          const bool plain = vm == 0xffffu;
#pragma unroll
          for (int nt = 0; nt < 2; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int cell = col_cell<I8>(nt, 2 * c + (e & 1)), j = j0 + cell;
              float x = sc[m][nt][e] * a.g.scale_log2;
              if (I8) x *= ks[2 * nt + (e & 1)];
              const bool see = j >= rlo[m][e >> 1] && j < rhi[m][e >> 1] && (plain || (vm >> cell & 1u));
              sc[m][nt][e] = see ? x : -INFINITY;
            }
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float x = fmaxf(fmaxf(sc[m][0][2 * e], sc[m][0][2 * e + 1]), fmaxf(sc[m][1][2 * e], sc[m][1][2 * e + 1]));
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
            nm[m][e] = fmaxf(mx[m][e], x);
            grew |= nm[m][e] > mx[m][e];
          }
        }
        if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
          for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              // (-inf) - (-inf) never arises: a maximum that grew is finite or +inf
              const float f = nm[m][e] > mx[m][e] ? ex2(mx[m][e] - nm[m][e]) : 1.f;
              mx[m][e] = nm[m][e];
              l[m][e] *= f;
#pragma unroll
              for (int j = 0; j < D / 8; ++j) {
                o[m][j][2 * e] *= f;
                o[m][j][2 * e + 1] *= f;
              }
            }
        }
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          const float b0 = mx[m][0] == -INFINITY ? 0.f : mx[m][0], b1 = mx[m][1] == -INFINITY ? 0.f : mx[m][1];
          float p[2][4];
#pragma unroll
          for (int nt = 0; nt < 2; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              p[nt][e] = ex2(sc[m][nt][e] - (e < 2 ? b0 : b1));
              l[m][e >> 1] += p[nt][e];
              // a scale of a hidden cell may be anything: its probability stays zero
              if (I8) p[nt][e] = sc[m][nt][e] == -INFINITY ? 0.f : p[nt][e] * vs[2 * nt + (e & 1)];
            }
          pf[m][0] = Half16<PBF>::pack(p[0][0], p[0][1]);
          pf[m][1] = Half16<PBF>::pack(p[0][2], p[0][3]);
          pf[m][2] = Half16<PBF>::pack(p[1][0], p[1][1]);
          pf[m][3] = Half16<PBF>::pack(p[1][2], p[1][3]);
        }
        // ---- output ----
        if (!I8) {
          const uint32_t vb = smem_u32(st + C::kMat);
          const int row = lane & 15;
#pragma unroll
          for (int jj = 0; jj < D / 16; ++jj) {
            uint32_t b[4];
            const uint32_t ad = vb + (row * C::kChunks + v_chunk<C::kChunks, I8>(row, 2 * jj + (lane >> 4))) * 16;
            asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                         : "=r"(b[0]), "=r"(b[1]), "=r"(b[2]), "=r"(b[3])
                         : "r"(ad)
                         : "memory");
#pragma unroll
            for (int m = 0; m < MT; ++m) {
              mma16816<PBF>(o[m][2 * jj], pf[m], b[0], b[1]);
              mma16816<PBF>(o[m][2 * jj + 1], pf[m], b[2], b[3]);
            }
          }
        } else {
          constexpr int W = D / 32;               // words (4 dimensions each) per lane and cell
          uint32_t v[4][W];
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const int row = 4 * c + x;
            const uint8_t* vp = st + C::kMat + row * C::kRowBytes;
            if (D == 128) {
              const uint4 w = *reinterpret_cast<const uint4*>(vp + v_chunk<C::kChunks, I8>(row, g) * 16);
              v[x][0] = w.x;
              v[x][1] = w.y;
              v[x][W > 2 ? 2 : 0] = w.z;
              v[x][W > 2 ? 3 : 0] = w.w;
            } else {
              const uint2 w =
                  *reinterpret_cast<const uint2*>(vp + v_chunk<C::kChunks, I8>(row, g >> 1) * 16 + (g & 1) * 8);
              v[x][0] = w.x;
              v[x][1] = w.y;
            }
          }
#pragma unroll
          for (int w = 0; w < W; ++w)
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              const uint32_t b0 = codes2<true>(__byte_perm(v[0][w], v[1][w], (uint32_t)(y | (4 + y) << 8))),
                             b1 = codes2<true>(__byte_perm(v[2][w], v[3][w], (uint32_t)(y | (4 + y) << 8)));
#pragma unroll
              for (int m = 0; m < MT; ++m) mma16816<true>(o[m][4 * w + y], pf[m], b0, b1);
            }
        }
      }
    }
    cp_async_wait<0>();
    // ---- join the warps ----
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        l[m][e] += __shfl_xor_sync(0xffffffffu, l[m][e], 1);
        l[m][e] += __shfl_xor_sync(0xffffffffu, l[m][e], 2);
        if (c == 0) {
          sm_m[warp][m * 16 + g + 8 * e] = mx[m][e];
          sm_l[warp][m * 16 + g + 8 * e] = l[m][e];
        }
      }
    __syncthreads();                                // every warp is done with its ring
    float* so = reinterpret_cast<float*>(smem);     // [kWarps][ROWS][D]
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int j = 0; j < D / 8; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int n = 2 * c + (e & 1), dim = I8 ? n * (D / 8) + j : 8 * j + n;
          so[(warp * ROWS + m * 16 + g + 8 * (e >> 1)) * D + dim] = o[m][j][e];
        }
    __syncthreads();
    const int64_t u0 = cu.u - t0;
    const int first = unit_owner(cu, u0), last = unit_owner(cu, u0 + units - 1);
    const bool whole = first == last;
    float* part = a.ws + ((int64_t)blockIdx.x * 2 + (t0 == 0 ? 1 : 0)) * a.ws_slot;
    for (int x = tid; x < nrows * (D / 4); x += kNT) {
      const int r = x / (D / 4), d4 = x % (D / 4);
      float M = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sm_m[w][r]);
      const float base = M == -INFINITY ? 0.f : M;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
      float L = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float f = sm_m[w][r] == M ? (M == -INFINITY ? 0.f : 1.f) : ex2(sm_m[w][r] - base);
        const float4 v = *reinterpret_cast<const float4*>(so + (w * ROWS + r) * D + 4 * d4);
        L += f * sm_l[w][r];
        acc.x += f * v.x;
        acc.y += f * v.y;
        acc.z += f * v.z;
        acc.w += f * v.w;
      }
      if (whole) {
        const float inv = L > 0.f ? 1.f / L : (L == 0.f ? 0.f : L);
        const int i = (r0 + r) / G;
        const int64_t at = (int64_t)(q.q0 + i) * a.g.hq + h * G + (r0 + r - i * G);
        *reinterpret_cast<uint2*>(a.out + at * D + 4 * d4) =
            make_uint2(Half16<BF16>::pack(acc.x * inv, acc.y * inv), Half16<BF16>::pack(acc.z * inv, acc.w * inv));
        if (d4 == 0 && a.lse) a.lse[at] = L == 0.f ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
      } else {
        __stcg(reinterpret_cast<float4*>(part + r * D + 4 * d4), acc);
        if (d4 == 0) {
          __stcg(part + ROWS * D + r, M);
          __stcg(part + ROWS * D + ROWS + r, L);
        }
      }
    }
    if (!whole) {
      const int nseg = last - first + 1;
      __threadfence();
      __syncthreads();
      if (tid == 0) last_flag = atom_acq_rel_add(&a.arrived[first], 1u) == (uint32_t)(nseg - 1);
      __syncthreads();
      if (last_flag) {
        __threadfence();
        if (tid == 0) a.arrived[first] = 0;
        // slot 1 of the first part, slot 0 of the others
        const float* base_ws = a.ws + ((int64_t)first * 2 + 1) * a.ws_slot;
        for (int x = tid; x < nrows * (D / 4); x += kNT) {
          const int r = x / (D / 4), d4 = x % (D / 4);
          // sixteen parts' loads in flight at a time
          constexpr int kAt = 16;
          float M = -INFINITY, L = 0.f;
          float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
          for (int k0 = 0; k0 < nseg; k0 += kAt) {
            float m[kAt], lw[kAt];
            float4 v[kAt];
#pragma unroll
            for (int k = 0; k < kAt; ++k) {
              const int w = k0 + k;
              const float* pw = base_ws + (w ? (2 * (int64_t)w - 1) * a.ws_slot : 0);
              if (w < nseg) {
                m[k] = __ldcg(pw + ROWS * D + r);
                lw[k] = __ldcg(pw + ROWS * D + ROWS + r);
                v[k] = __ldcg(reinterpret_cast<const float4*>(pw + r * D + 4 * d4));
              } else {
                m[k] = -INFINITY;
                lw[k] = 0.f;
                v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
              }
            }
            float top = M;
#pragma unroll
            for (int k = 0; k < kAt; ++k) top = fmaxf(top, m[k]);
            const float f0 = M == top ? 1.f : ex2(M - top);
            M = top;
            L *= f0;
            acc.x *= f0;
            acc.y *= f0;
            acc.z *= f0;
            acc.w *= f0;
#pragma unroll
            for (int k = 0; k < kAt; ++k) {
              const float f = m[k] == -INFINITY ? 0.f : m[k] == M ? 1.f : ex2(m[k] - M);
              L += f * lw[k];
              acc.x += f * v[k].x;
              acc.y += f * v[k].y;
              acc.z += f * v[k].z;
              acc.w += f * v[k].w;
            }
          }
          const float inv = L > 0.f ? 1.f / L : (L == 0.f ? 0.f : L);
          const int i = (r0 + r) / G;
          const int64_t at = (int64_t)(q.q0 + i) * a.g.hq + h * G + (r0 + r - i * G);
          *reinterpret_cast<uint2*>(a.out + at * D + 4 * d4) =
              make_uint2(Half16<BF16>::pack(acc.x * inv, acc.y * inv), Half16<BF16>::pack(acc.z * inv, acc.w * inv));
          if (d4 == 0 && a.lse) a.lse[at] = L == 0.f ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
        }
      }
    }
    cu.u += t1 - t0;
    if (t1 == units) next_item<ROWS, kTK>(a.b, G, HKV, cu);
    __syncthreads();                                // `smem` goes back to the rings
  }
}

template <bool BF16, int D, bool I8, int MT>
cudaError_t launch_rows(const AttnFwdArgs& a, cudaStream_t s) {
  constexpr int smem = RowsCfg<D, I8>::kSmem > kWarps * 16 * MT * D * 4 ? RowsCfg<D, I8>::kSmem : kWarps * 16 * MT * D * 4;
  const cudaError_t e = ensure_dyn_smem(reinterpret_cast<const void*>(rows_kernel<BF16, D, I8, MT>), smem);
  if (e != cudaSuccess) return e;
  rows_kernel<BF16, D, I8, MT><<<a.num_sms, kNT, smem, s>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attn_rows(const AttnFwdArgs& a, int max_q, cudaStream_t s) {
  const bool two = (int64_t)max_q * a.g.g > 16, bf = a.g.io == MOE_T_BF16, i8 = a.g.kv == MOE_T_I8;
#define ROWS_MT(BF, DD, I) return two ? launch_rows<BF, DD, I, 2>(a, s) : launch_rows<BF, DD, I, 1>(a, s)
  if (a.g.D == 128) {
    if (bf && i8) ROWS_MT(true, 128, true);
    if (bf) ROWS_MT(true, 128, false);
    if (i8) ROWS_MT(false, 128, true);
    ROWS_MT(false, 128, false);
  }
  if (bf && i8) ROWS_MT(true, 64, true);
  if (bf) ROWS_MT(true, 64, false);
  if (i8) ROWS_MT(false, 64, true);
  ROWS_MT(false, 64, false);
#undef ROWS_MT
}

}  // namespace moe
