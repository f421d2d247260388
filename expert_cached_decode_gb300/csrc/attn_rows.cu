// Attention of few rows (single tokens, short drafts) over the paged cache:
// up to 32 rows (tokens times query heads per K/V head) per K/V head.
//
// Bound by the cells' bytes: every cell is read once for all rows of its K/V
// head.  A CTA's eight warps take steps of 16 or 32 cells in turn, each
// through a ring of its own that 16-byte asynchronous copies fill, with its
// own running maximum, sum and output (online softmax), so no warp waits for
// another before the item's end; there the warps' results are joined in shared
// memory, and the parts of an item that several CTAs share by attn_join.cu.
// One token over 524,288 cells takes 181 us in 16 bits (88% of a copy's
// bandwidth) and 108 us in int8 (76%; there the expansion of the codes fills
// more than half of the issue slots), over 131,072 int8 cells 36 us with the
// join, 13 of which do not depend on the length.  (One bulk copy per K or V
// vector instead: an SM starts some 150-165 of them a microsecond, which held
// int8 cells, 128 bytes each, to 2.9 TB/s against 4.2 TB/s at that time.)
//
// Products on mma.sync m16n8k16: at 16 or 32 rows they need a fraction of the
// memory time, and their B fragments come straight from the rows of K and V.
// The order in which a contraction runs is free, so a lane's 16-byte piece of
// K (8 or 16 dimensions of one cell) feeds two or four products as it lies,
// with Q's fragments loaded to match, and int8 V feeds products whose column
// n of tile j is dimension n * (D / 8) + j.  int8 codes become fp16 exactly;
// the K scale multiplies the score, the V scale the probability.
#include "attn.cuh"

namespace moe {

namespace {

constexpr int kWarps = 8, kNT = kWarps * 32, kTK = 128, kOvh = 1;
// Fewest units of a part: the joining kernel runs in any case, so short sequences are cut finely too.
constexpr int kMinUnits = 2;

// Rows of the ring are padded so that lanes that read together hit different
// banks.  In 16-byte chunks modulo 8 a row adds: K 1 (the two cells that eight
// lanes read lie 4 rows apart: 4 chunks), 16-bit V 1 (ldmatrix reads 8 rows of
// one chunk), int8 V 2 (four rows, two chunks each; at D = 64 half-chunks).
template <int D, bool I8, int MT>
struct RowsCfg {
  static constexpr int kRowBytes = D * (I8 ? 1 : 2);          // of one head vector
  static constexpr int kChunks = kRowBytes / 16;
  // cells of a step: 32 where the ring and the registers allow it
  static constexpr int kStep = kRowBytes == 256 || (D == 128 && MT == 2) ? 16 : 32;
  static constexpr int kPitchK = kRowBytes + 16, kPitchV = kRowBytes + (I8 ? 32 : 16);
  static constexpr int kOffV = kStep * kPitchK;
  static constexpr int kOffScale = kOffV + kStep * kPitchV;
  static constexpr int kOffValid = kOffScale + (I8 ? 2 * kStep * 4 : 0);
  static constexpr int kStage = kOffValid + 16;
  // some 26 KB a warp: 210 KB per SM in the rings, of which all but one step per warp are in flight
  static constexpr int kStages = 27000 / kStage > 6 ? 6 : 27000 / kStage;
  static constexpr int kRing = kStages * kStage;
  // a warp's output rows in shared memory: every D / 4 floats padded by 4, so that the four lanes of a row, D / 4
  // apart (int8), and the rows, hit different banks
  static constexpr int kPitchO = D + 16 + (I8 ? 0 : 8);
  static constexpr int kJoin = kWarps * 16 * MT * kPitchO * 4;
  static constexpr int kSmem = (kWarps * kRing > kJoin ? kWarps * kRing : kJoin);
  static_assert(kSmem >= 4096 * 8, "holds the sequences' units");
};

template <bool BF16, int D, bool I8, int MT>
__global__ void __launch_bounds__(kNT, 1) rows_kernel(const __grid_constant__ AttnFwdArgs a) {
  using C = RowsCfg<D, I8, MT>;
  constexpr int ROWS = 16 * MT, STEP = C::kStep, NB = STEP / 16;
  constexpr bool PBF = BF16 && !I8;      // type of the products: the cells', fp16 for int8 cells
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ CursorScratch scr;
  __shared__ float sm_m[kWarps][ROWS], sm_l[kWarps][ROWS];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c = lane & 3;
  const int G = a.g.g, HKV = a.g.hkv;
  if (tid == 0) a.cuts[blockIdx.x].parts = 0;
  pdl_launch_dependents();
  const Work<ROWS, kTK, kOvh> work{a.b, a.g.gdiv, HKV, a.rows_min, a.rows_max};
  Cursor cu;
  if (!find_part<kNT, kMinUnits>(work, scr, reinterpret_cast<int64_t*>(smem), cu)) return;
  __syncthreads();                       // `smem` held the sequences' units
  const uint8_t* none = reinterpret_cast<const uint8_t*>(a.q);   // address of copies that read nothing
  uint8_t* ring = smem + warp * C::kRing;
  uint32_t it = 0;                       // steps of this warp so far
  Segment sg;

  while (next_segment(work, cu, sg)) {
    const int h = sg.h, s = sg.s, r0 = sg.r0, nrows = sg.nrows, lo = sg.lo, jbase = sg.jbase, jend = sg.jend;
    // ---- this warp's steps: cells [jbase + STEP i, + STEP), i = warp, warp + 8, ... ----
    const int n_steps = jend > jbase ? (jend - jbase + STEP - 1) / STEP : 0;
    const int my = n_steps > warp ? (n_steps - warp + kWarps - 1) / kWarps : 0;
    const int head_off = h * C::kRowBytes, v_off = HKV * C::kRowBytes, sc_off = 2 * HKV * C::kRowBytes + 4 * h;
    constexpr int kHidden = INT32_MIN;
    auto cell_of = [&](int i) { return jbase + (warp + i * kWarps) * STEP + (lane & (STEP - 1)); };
    // page id of this lane's cell of step i
    auto page_id = [&](int i) {
      const int j = cell_of(i);
      if (i >= my || j < lo || j >= jend) return kHidden;
      return a.b.table[(int64_t)s * a.b.table_pages + fdiv((uint32_t)j, a.b.page_div)];
    };
    auto issue = [&](int i, int id) {
      uint8_t* st = ring + (it + i) % C::kStages * C::kStage;
      if (id != kHidden && (uint32_t)id >= (uint32_t)a.b.n_pages) {
        atomicOr(a.b.err, (uint32_t)ATTN_BAD_PAGE);
        id = kHidden;
      }
      const int j = cell_of(i);
      const int in = j - (int)fdiv((uint32_t)j, a.b.page_div) * a.b.page_cells;
      const uint8_t* cell = id == kHidden ? nullptr : a.b.cells + (int64_t)id * a.b.page_bytes + (int64_t)in * a.b.cell_bytes;
      const uint32_t vm = __ballot_sync(0xffffffffu, cell != nullptr);
      if (lane == 0) *reinterpret_cast<uint32_t*>(st + C::kOffValid) = vm;
      // a hidden cell is filled with zeros: its probability is zero, and 0 * NaN is not
      constexpr int RPI = 32 / C::kChunks;          // rows per instruction
      const int ch = lane % C::kChunks;
      const uint32_t to = smem_u32(st) + ch * 16;
#pragma unroll
      for (int x = 0; x < STEP / RPI; ++x) {
        const int row = x * RPI + lane / C::kChunks;
        const uint8_t* p = reinterpret_cast<const uint8_t*>(shfl_u64(reinterpret_cast<uint64_t>(cell), row));
        const int n = p ? 16 : 0;
        const uint8_t* src = p ? p + head_off + ch * 16 : none;
        cp_async16(to + row * C::kPitchK, src, n);
        cp_async16(to + C::kOffV + row * C::kPitchV, p ? src + v_off : none, n);
      }
      if (I8) {
        const int row = lane & (STEP - 1), n = cell ? 4 : 0;
        const uint32_t sc = smem_u32(st + C::kOffScale) + 4 * row;
        if (STEP == 32 || lane < 16) cp_async4(sc, cell ? cell + sc_off : none, n);
        if (STEP == 32 || lane >= 16) cp_async4(sc + 4 * STEP, cell ? cell + sc_off + 4 * HKV : none, n);
      }
    };
    // ---- Q fragments (the scale is applied to the scores: the products are exact) ----
    uint32_t qf[MT][D / 16][4];
    float qs[MT][2];                                // factor of a row's scores
    int rlo[MT][2], rhi[MT][2];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = r0 + m * 16 + g + 8 * e;
        qs[m][e] = a.g.scale_log2;
        const bool real = m * 16 + g + 8 * e < nrows;
        const int i = real ? (int)fdiv((uint32_t)r, a.g.gdiv) : 0;
        row_range(sg.q, a.b.window, i, rlo[m][e], rhi[m][e]);
        if (!real) {                               // a padding row: no mask (its result is not used)
          rlo[m][e] = 0;
          rhi[m][e] = INT32_MAX;
        }
        const uint16_t* src = a.q + (int64_t)(sg.q.q0 + i) * a.q_stride + (h * G + (real ? r - i * G : 0)) * D;
#pragma unroll
        for (int p = 0; p < D / 32; ++p) {
          // 16-bit cells: chunk c + 4p (8 dimensions) feeds products 2p, 2p + 1.
          // int8 cells: chunk c + 4(p/2) (16 dimensions), its words 2(p%2), 2(p%2) + 1 feed them.
          uint4 v = make_uint4(0, 0, 0, 0);
          if (real) v = *reinterpret_cast<const uint4*>(src + (I8 ? 16 * (c + 4 * (p >> 1)) + 8 * (p & 1) : 8 * (c + 4 * p)));
          qf[m][2 * p][e] = v.x;
          qf[m][2 * p][2 + e] = v.y;
          qf[m][2 * p + 1][e] = v.z;
          qf[m][2 * p + 1][2 + e] = v.w;
        }
      }
    int ids[C::kStages + 1];
#pragma unroll
    for (int i = 0; i <= C::kStages; ++i) ids[i] = page_id(i);     // loads that do not wait for one another
#pragma unroll
    for (int i = 0; i < C::kStages - 1; ++i) {
      if (i < my) issue(i, ids[i]);
      cp_async_commit();
    }
    int id0 = ids[C::kStages - 1], id1 = ids[C::kStages];
    auto halve_q = [&] {                            // bf16 queries as fp16 in units of their row's largest
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float top = 0.f;
#pragma unroll
          for (int x = 0; x < D / 16; ++x)
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              const float2 v = Half16<true>::unpack(qf[m][x][2 * y + e]);
              top = fmaxf(top, fmaxf(fabsf(v.x), fabsf(v.y)));
            }
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
          const float u = row_unit(top), f = inv_pow2(u);
          qs[m][e] *= u;
#pragma unroll
          for (int x = 0; x < D / 16; ++x)
#pragma unroll
            for (int y = 0; y < 2; ++y) qf[m][x][2 * y + e] = bf16_to_f16(qf[m][x][2 * y + e], f);
        }
    };
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
    if (I8 && BF16) halve_q();
#pragma unroll 1
    for (int i = 0; i < my; ++i) {
      __syncwarp();                                 // the step before is done with its stage
      if (i + C::kStages - 1 < my) issue(i + C::kStages - 1, id0);
      cp_async_commit();
      id0 = id1;
      id1 = page_id(i + C::kStages + 1);
      cp_async_wait<C::kStages - 1>();
      __syncwarp();
      const uint8_t* st = ring + (it + i) % C::kStages * C::kStage;
      const int j0 = jbase + (warp + i * kWarps) * STEP;
      const uint32_t vm = *reinterpret_cast<const uint32_t*>(st + C::kOffValid);
      const float* scl = reinterpret_cast<const float*>(st + C::kOffScale);
      // ---- scores: column (b, nt, n) is cell 16 b + col_cell ----
      float sc[MT][2 * NB][4];
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int nt = 0; nt < 2 * NB; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) sc[m][nt][e] = 0.f;
#pragma unroll
      for (int p = 0; p < C::kChunks / 4; ++p)
#pragma unroll
        for (int nt = 0; nt < 2 * NB; ++nt) {
          const int row = 16 * (nt >> 1) + col_cell<I8>(nt & 1, g);
          const uint4 w = *reinterpret_cast<const uint4*>(st + row * C::kPitchK + (c + 4 * p) * 16);
          if (!I8) {
#pragma unroll
            for (int m = 0; m < MT; ++m) {
              mma16816<PBF>(sc[m][nt], qf[m][2 * p], w.x, w.y);
              mma16816<PBF>(sc[m][nt], qf[m][2 * p + 1], w.z, w.w);
            }
          } else {
            const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              uint32_t b0, b1;
              codes4_f16(ww[x], b0, b1);
#pragma unroll
              for (int m = 0; m < MT; ++m) mma16816<PBF>(sc[m][nt], qf[m][4 * p + x], b0, b1);
            }
          }
        }
      // the cell of this lane's column e & 1 of tile nt
      auto lane_cell = [&](int nt, int e) { return 16 * (nt >> 1) + col_cell<I8>(nt & 1, 2 * c + e); };
      // ---- online softmax (base 2) ----
      uint32_t pf[MT][NB][4];
      bool grew = false;
      float nm[MT][2];
      bool plain = vm == 0xffffffffu;              // (16 cells: both half-warps' lanes say the same)
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int e = 0; e < 2; ++e) plain = plain && j0 >= rlo[m][e] && j0 + STEP <= rhi[m][e];
#pragma unroll
      for (int nt = 0; nt < 2 * NB; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float f = I8 ? scl[lane_cell(nt, e)] : 1.f;
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            sc[m][nt][e] *= I8 ? f * qs[m][0] : qs[m][0];
            sc[m][nt][2 + e] *= I8 ? f * qs[m][1] : qs[m][1];
          }
        }
      uint32_t vbits = I8 ? scale_bits(scl[STEP + (lane & (STEP - 1))]) : 0u;
      if (!__all_sync(0xffffffffu, plain)) {
        if (I8) vbits = finite_bits(vbits);       // (where every row sees every cell, all of them get its NaN)
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int nt = 0; nt < 2 * NB; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int cell = lane_cell(nt, e & 1), j = j0 + cell;
              if (!(j >= rlo[m][e >> 1] && j < rhi[m][e >> 1] && (vm >> cell & 1u))) sc[m][nt][e] = -INFINITY;
            }
      }
      // In fp16 the reference lies 2^15 below the largest probability: small ones keep their bits down to 2^-29 of it.
      const float ev = I8 ? -15.f + scale_exp(__reduce_max_sync(0xffffffffu, vbits)) : -15.f;
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float x = fmaxf(sc[m][0][2 * e], sc[m][0][2 * e + 1]);
#pragma unroll
          for (int nt = 1; nt < 2 * NB; ++nt) x = fmaxf(x, fmaxf(sc[m][nt][2 * e], sc[m][nt][2 * e + 1]));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
          nm[m][e] = fmaxf(mx[m][e], PBF ? x : x + ev);
          grew |= nm[m][e] > mx[m][e];
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
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          float p[2][4];
#pragma unroll
          for (int nt = 0; nt < 2; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float x = sc[m][2 * b + nt][e];
              p[nt][e] = ex2(x - (e < 2 ? b0 : b1));
              l[m][e >> 1] += p[nt][e];
              // a scale of a hidden cell may be anything: its probability stays zero
              if (I8) p[nt][e] = x == -INFINITY ? 0.f : p[nt][e] * scl[STEP + lane_cell(2 * b + nt, e & 1)];
            }
          pf[m][b][0] = Half16<PBF>::pack(p[0][0], p[0][1]);
          pf[m][b][1] = Half16<PBF>::pack(p[0][2], p[0][3]);
          pf[m][b][2] = Half16<PBF>::pack(p[1][0], p[1][1]);
          pf[m][b][3] = Half16<PBF>::pack(p[1][2], p[1][3]);
        }
      }
      // ---- output ----
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const uint8_t* vt = st + C::kOffV + 16 * b * C::kPitchV;
        if (!I8) {
          // product k = 8 x + n is cell 8 x + (n >> 1) + 4 (n & 1): lane i gives the row address of k = i % 16
          const int kk = lane & 7, row = (lane & 8) + (kk >> 1) + 4 * (kk & 1);
          const uint32_t vb = smem_u32(vt + row * C::kPitchV + (lane >> 4) * 16);
#pragma unroll
          for (int jj = 0; jj < D / 16; ++jj) {
            uint32_t f[4];
            asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                         : "=r"(f[0]), "=r"(f[1]), "=r"(f[2]), "=r"(f[3])
                         : "r"(vb + 32 * jj)
                         : "memory");
#pragma unroll
            for (int m = 0; m < MT; ++m) {
              mma16816<PBF>(o[m][2 * jj], pf[m][b], f[0], f[1]);
              mma16816<PBF>(o[m][2 * jj + 1], pf[m][b], f[2], f[3]);
            }
          }
        } else {
          constexpr int W = D / 32;               // words (4 dimensions each) per lane and cell
          uint32_t v[4][W];
#pragma unroll
          for (int x = 0; x < 4; ++x) {           // cells c, c + 4, c + 8, c + 12: columns (x / 2, 2c + x % 2)
            const uint8_t* vp = vt + (c + 4 * x) * C::kPitchV + g * (D / 8);
            if (D == 128) {
              const uint4 w = *reinterpret_cast<const uint4*>(vp);
              v[x][0] = w.x;
              v[x][1] = w.y;
              v[x][W > 2 ? 2 : 0] = w.z;
              v[x][W > 2 ? 3 : 0] = w.w;
            } else {
              const uint2 w = *reinterpret_cast<const uint2*>(vp);
              v[x][0] = w.x;
              v[x][1] = w.y;
            }
          }
#pragma unroll
          for (int w = 0; w < W; ++w) {
            uint32_t b0[4], b1[4];
            codes4x2_f16(v[0][w], v[1][w], b0);
            codes4x2_f16(v[2][w], v[3][w], b1);
#pragma unroll
            for (int y = 0; y < 4; ++y)
#pragma unroll
              for (int m = 0; m < MT; ++m) mma16816<PBF>(o[m][4 * w + y], pf[m][b], b0[y], b1[y]);
          }
        }
      }
    }
    it += my;
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
    float* so = reinterpret_cast<float*>(smem);     // [kWarps][ROWS][kPitchO]
    auto place = [](int dim) { return dim + 4 * (dim / (D / 4)); };
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = m * 16 + g + 8 * e;
        if (r >= nrows) continue;
        float* to = so + (warp * ROWS + r) * C::kPitchO;
        if (!I8) {
#pragma unroll
          for (int j = 0; j < D / 8; ++j)
            *reinterpret_cast<float2*>(to + place(8 * j) + 2 * c) = make_float2(o[m][j][2 * e], o[m][j][2 * e + 1]);
        } else {
#pragma unroll
          for (int y = 0; y < 2; ++y)
#pragma unroll
            for (int j = 0; j < D / 8; j += 4)
              *reinterpret_cast<float4*>(to + place((2 * c + y) * (D / 8)) + j) =
                  make_float4(o[m][j][2 * e + y], o[m][j + 1][2 * e + y], o[m][j + 2][2 * e + y], o[m][j + 3][2 * e + y]);
        }
      }
    __syncthreads();
    const bool whole = sg.parts == 1;
    float* part = a.ws + ((int64_t)blockIdx.x * 2 + (sg.starts ? 1 : 0)) * a.ws_slot;
    for (int x = tid; x < nrows * (D / 4); x += kNT) {
      const int r = x / (D / 4), d4 = x % (D / 4);
      float M = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sm_m[w][r]);
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
      float L = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float f = sm_m[w][r] == -INFINITY ? 0.f : sm_m[w][r] == M ? 1.f : ex2(sm_m[w][r] - M);
        const float4 v = *reinterpret_cast<const float4*>(so + (w * ROWS + r) * C::kPitchO + place(4 * d4));
        L += f * sm_l[w][r];
        acc.x += f * v.x;
        acc.y += f * v.y;
        acc.z += f * v.z;
        acc.w += f * v.w;
      }
      if (whole) {
        const float inv = L > 0.f ? 1.f / L : (L == 0.f ? 0.f : L);
        const int i = (int)fdiv((uint32_t)(r0 + r), a.g.gdiv);
        const int64_t at = (int64_t)(sg.q.q0 + i) * a.g.hq + h * G + (r0 + r - i * G);
        *reinterpret_cast<uint2*>(a.out + at * D + 4 * d4) =
            make_uint2(Half16<BF16>::pack(acc.x * inv, acc.y * inv), Half16<BF16>::pack(acc.z * inv, acc.w * inv));
        if (d4 == 0 && a.lse) a.lse[at] = L == 0.f ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
      } else {
        __stcg(reinterpret_cast<float4*>(part + r * D + 4 * d4), acc);
        if (d4 == 0) {
          __stcg(part + ROWS * D + r, M);
          __stcg(part + ROWS * (D + 1) + r, L);
        }
      }
    }
    if (!whole && sg.starts && tid == 0) a.cuts[blockIdx.x] = AttnCut{sg.parts, sg.q.q0, r0, nrows, h};
    __syncthreads();                                // `smem` goes back to the rings
  }
}

template <bool BF16, int D, bool I8, int MT>
cudaError_t launch_rows(const AttnFwdArgs& a, cudaStream_t s) {
  constexpr int smem = RowsCfg<D, I8, MT>::kSmem;
  static_assert(smem <= 220 * 1024, "shared memory");
  const cudaError_t e = ensure_dyn_smem(reinterpret_cast<const void*>(rows_kernel<BF16, D, I8, MT>), smem);
  if (e != cudaSuccess) return e;
  rows_kernel<BF16, D, I8, MT><<<a.num_sms, kNT, smem, s>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attn_rows(const AttnFwdArgs& a, int max_q, bool join, cudaStream_t s) {
  const bool two = (int64_t)max_q * a.g.g > 16, bf = a.g.io == MOE_T_BF16, i8 = a.g.kv == MOE_T_I8;
  cudaError_t e;
#define ROWS_MT(BF, DD, I) e = two ? launch_rows<BF, DD, I, 2>(a, s) : launch_rows<BF, DD, I, 1>(a, s)
  if (a.g.D == 128) {
    if (bf) {
      if (i8) ROWS_MT(true, 128, true);
      else ROWS_MT(true, 128, false);
    } else {
      if (i8) ROWS_MT(false, 128, true);
      else ROWS_MT(false, 128, false);
    }
  } else {
    if (bf) {
      if (i8) ROWS_MT(true, 64, true);
      else ROWS_MT(true, 64, false);
    } else {
      if (i8) ROWS_MT(false, 64, true);
      else ROWS_MT(false, 64, false);
    }
  }
#undef ROWS_MT
  return e == cudaSuccess && join ? launch_attn_join(a, two ? 32 : 16, s) : e;
}

}  // namespace moe
