// Weights that a call's attention gives to the cells, many rows per K/V head,
// on the tensor cores: acc[j] = decay * acc[j] + sum over rows and heads of
// exp(scale q.k_j - lse).
//
// The product is taken with the cells as rows, S^T = K Q^T (128 cells x 96
// query rows), so that a thread owns a cell and adds a row of S^T: the sum
// over query rows needs no exchange between threads, the query's statistics
// are the same for all threads (shared memory, broadcast), and a cell's mask
// is one range of columns.  A CTA holds two tiles of cells (256) against a
// stream of query tiles; each query tile is read from L2 once per 256 cells.
// K is the products' A operand from tensor memory, where the threads that own
// the cells put it, a row each (int8 codes as 16-bit floats): shared memory
// then feeds only the queries.  (With both operands there a product of 128 x
// 128 x 128 took 0.4 us instead of 0.27.)  96 columns, because two K tiles and
// two buffers of scores for each fill the tensor memory.
// Roles: warps 0-7 and 8-15 add up the two tiles' rows (two threads a cell, 48
// columns each: four warps a scheduler hide one another's latencies), 16-19
// load the queries where their groups do not fit TMA boxes, 20 and 22 issue the
// two tiles' products, 21 the copies of the queries and their statistics.
// 1,024 tokens of 32 heads over 16,384 bf16 cells take 156 us, 44% of the
// products' rate, with two thirds of the issue slots taken: a score costs some
// six instructions.
// An item is 256 cells of a sequence, its tiles the (head, query tile) pairs;
// items are divided over the CTAs as in the attention, and a second kernel
// joins those that were cut, in the order of their parts.
#include "attn_tc.cuh"

namespace moe {

namespace {

constexpr int kCells = 256, kQRows = kWeightQRows, kThreads = WeightRoles::Block::kThreads, kLseRing = 16;
constexpr int kOvh = 2, kMinUnits = 3;

template <int D>
struct WcCfg {
  static constexpr int kTileBytes = kQRows * D * 2;
  static constexpr int kQSlots = 8;
  static constexpr int kOffLse = kQSlots * kTileBytes;
  static constexpr int kOffQPtr = kOffLse + kLseRing * kQRows * 4;
  static constexpr int kSmem = kOffQPtr + 2 * kQRows * 8;
  static_assert(kOffLse >= 4096 * 8, "holds the sequences' units");
  // Statistics of step n + R are written once the query tile of step n + R - 1 is under way, so the product of step
  // n + R - 1 - kQSlots has ended and the scores of two steps before that have been taken out: those of n have.
  static_assert(kLseRing >= kQSlots + 4, "statistics outlive their use");
  // tensor memory: K of the two tiles, then two buffers of scores for each
  __host__ __device__ static constexpr uint32_t kCol(int w) { return (uint32_t)(w * (D / 2)); }
  __host__ __device__ static constexpr uint32_t kColS(int w, int b) { return (uint32_t)(D + (2 * w + b) * kQRows); }
};

// Two int8 codes (the low bytes of x's halves) as bf16, exactly: 0x4300 | low 7 bits is 128 + them, 0x4300 | the sign
// bit is 128 or 256, and the difference is the code.
__device__ __forceinline__ uint32_t codes2_bf16(uint32_t x) {
  const uint32_t a = lop3_and_or(x, 0x007f007fu, 0x43004300u), b = lop3_and_or(x, 0x00800080u, 0x43004300u);
  uint32_t d;
  asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// The work as find_part takes it: items are tiles of 256 cells.
struct WgtWork {
  const AttnBatch& b;
  FastDiv g;
  int hkv;                            // multiplier of an item's units: 1, the heads are counted in `units`
  int heads, max_kv;

  __device__ __forceinline__ int row_tiles(const SeqInfo& q) const { return (min(q.len, max_kv) + kCells - 1) / kCells; }
  // query rows [ra, rb) that see a cell of tile kt
  __device__ __forceinline__ void rows(const SeqInfo& q, int kt, int& ra, int& rb) const {
    const RowSpan span = rows_that_see(kt * kCells, kCells, q.n, q.len, b.window, (int)g.d);
    ra = span.a;
    rb = span.b;
  }
  __device__ __forceinline__ int tiles(const SeqInfo& q, int kt) const {
    int ra, rb;
    rows(q, kt, ra, rb);
    return max(1, heads * ((rb - ra + kQRows - 1) / kQRows));     // none: the cells still have to be written
  }
  __device__ __forceinline__ int units(const SeqInfo& q, int kt) const { return tiles(q, kt) + kOvh; }
};

struct WgtSegment {
  SeqInfo q;
  int s, j0, cells, ra, rb, rts, tiles, t0, t1, parts;
  bool starts;
};

__device__ __forceinline__ bool next_segment(const WgtWork& w, Cursor& c, WgtSegment& g) {
  while (c.u < c.end) {
    g.q = seq_info(w.b, c.s);
    g.s = c.s;
    const int kt = c.rt;
    w.rows(g.q, kt, g.ra, g.rb);
    g.rts = (g.rb - g.ra + kQRows - 1) / kQRows;
    g.tiles = max(1, w.heads * g.rts);
    const int units = g.tiles + kOvh, stop = (int)min((int64_t)units, c.t + (c.end - c.u));
    const int64_t u0 = c.u - c.t;
    g.t0 = max(0, c.t - kOvh);
    g.t1 = max(0, stop - kOvh);
    g.j0 = kt * kCells;
    g.cells = min(kCells, min(g.q.len, w.max_kv) - g.j0);
    c.u += stop - c.t;
    c.t = stop;
    if (stop == units) {
      c.t = 0;
      if (++c.rt >= w.row_tiles(g.q)) {
        c.rt = 0;
        do {
          ++c.s;
        } while (c.s < w.b.n_seqs && w.row_tiles(seq_info(w.b, c.s)) == 0);
      }
    }
    if (g.t1 <= g.t0) continue;
    g.parts = 1;
    g.starts = g.t0 == 0;
    if (g.t0 > 0 || g.t1 < g.tiles)
      g.parts = unit_owner(c, u0 + kOvh + g.tiles - 1) - unit_owner(c, u0 + kOvh) + 1;
    return true;
  }
  return false;
}

// A wait that gave up turns every later wait of its warp into nothing; the
// roles run through their loops (in bounds), and the error word says that the
// results are void.
template <bool BF16, int D, bool I8>
__global__ void __launch_bounds__(kThreads, 1)
    weights_chunk_kernel(const __grid_constant__ AttnWgtArgs a, const __grid_constant__ CUtensorMap qmap, int tma_q) {
  using C = WcCfg<D>;
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ CursorScratch scr;
  __shared__ uint64_t k_full[2], q_full[C::kQSlots], q_empty[C::kQSlots];
  __shared__ uint64_t s_full[2][2], s_empty[2][2], lse_full[kLseRing], drained;
  __shared__ uint32_t tmem_slot;
  __shared__ float half_sum[kCells];
  float* lse_ring = reinterpret_cast<float*>(smem + C::kOffLse);                    // [kLseRing][kQRows]
  const uint16_t** qptrs = reinterpret_cast<const uint16_t**>(smem + C::kOffQPtr);   // [2][kQRows]
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = a.g.g, HKV = a.g.hkv;
  if (tid == 0) a.cuts[blockIdx.x].parts = 0;
  pdl_launch_dependents();
  const WgtWork work{a.b, a.g.gdiv, 1, HKV, a.max_kv};
  Cursor cu;
  if (!find_part<kThreads, kMinUnits>(work, scr, reinterpret_cast<int64_t*>(smem), cu)) return;
  WgtSegment sg;
  __syncthreads();                       // `smem` held the sequences' units
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) mbar_init(&k_full[i], 256);
    for (int i = 0; i < C::kQSlots; ++i) {
      mbar_init(&q_full[i], tma_q ? 1 : 128);
      mbar_init(&q_empty[i], 2);
    }
    for (int w = 0; w < 2; ++w)
      for (int b = 0; b < 2; ++b) {
        mbar_init(&s_full[w][b], 1);
        mbar_init(&s_empty[w][b], 256);
      }
    for (int i = 0; i < kLseRing; ++i) mbar_init(&lse_full[i], 32);
    mbar_init(&drained, 2);
    mbar_init_fence();
  }
  if (warp == 20) {
    tmem_alloc(&tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  constexpr uint32_t tmem = 0;           // all 512 columns are this block's
  bool ok = true;

  if (warp >= 20) {
    // ================================ products ================================
    reg_dec<WeightRoles::kProducts>();
    if (warp == 20 || warp == 22) {
      // a warp per tile: one for both took 1.1 us a step in waits and issue, twice the products' time
      const int w = (warp - 20) >> 1;
      const uint32_t idesc = idesc_f16(128, kQRows, BF16);
      uint32_t nk = 0, nq = 0;            // heads (K tiles), query tiles
      const uint64_t q0d = smem_desc_sw128(smem);
      auto wait = [&](uint64_t* b, uint32_t parity) {
        if (ok && !__all_sync(0xffffffffu, mbar_wait_cycles(b, parity))) {
          ok = false;
          if (lane == 0) atomicOr(a.b.err, (uint32_t)ATTN_TIMEOUT);
        }
      };
      while (next_segment(work, cu, sg)) {
        if (sg.rts == 0) continue;
        int left = 0;                     // query tiles of the head still to come
        int first = sg.rts - sg.t0 % sg.rts;
        for (int t = sg.t0; t < sg.t1; ++t, ++nq) {
          const bool new_head = left == 0;
          if (new_head) {
            left = min(sg.t1 - t, first);
            first = sg.rts;
          }
          --left;
          wait(&q_full[nq % C::kQSlots], (nq / C::kQSlots) & 1);
          const uint32_t b = nq & 1;
          const uint64_t qd = q0d + nq % C::kQSlots * (C::kTileBytes >> 4);
          if (new_head) wait(&k_full[w], nk & 1);
          if (nq >= 2) wait(&s_empty[w][b], (nq / 2 - 1) & 1);
          tc_fence_after();
          if (ok && elect_one()) {
#pragma unroll
            for (int k = 0; k < D / 16; ++k)
              umma_f16_ts(C::kColS(0, 0) + (2 * w + b) * kQRows, C::kCol(1) * w + 8 * k,
                          qd + ((k >> 2) * (kQRows * 128) >> 4) + 2 * (k & 3), idesc, k != 0);
            umma_commit(&s_full[w][b]);
            umma_commit(&q_empty[nq % C::kQSlots]);
          }
          __syncwarp();
          if (new_head) ++nk;
        }
      }
      if (elect_one()) {
        umma_commit(&drained);
        if (!mbar_wait_cycles(&drained, 0)) atomicOr(a.b.err, (uint32_t)ATTN_TIMEOUT);
      }
    } else if (warp == 21) {
      // ========================= queries by TMA, statistics =========================
      uint32_t nq = 0;
      while (next_segment(work, cu, sg)) {
        if (sg.rts == 0) continue;
        int rt = sg.t0 % sg.rts, h = sg.t0 / sg.rts;
        // Statistics of this lane's rows 32 k + lane of a tile (three of them), negated and to base 2, a tile ahead.  A row that gives
        // nothing (no such row, or one that saw no cell) has -inf: its exponentials are 0.
        auto stats = [&](int rt_, int h_, float (&x)[3]) {
#pragma unroll
          for (int k = 0; k < 3; ++k) {
            const int row = sg.ra + rt_ * kQRows + 32 * k + lane;
            x[k] = INFINITY;
            if (row < sg.rb) {
              const int i = (int)fdiv((uint32_t)row, a.g.gdiv);
              x[k] = a.lse[(int64_t)(sg.q.q0 + i) * a.g.hq + h_ * G + row - i * G];
            }
          }
        };
        float nxt[3];
        stats(rt, h, nxt);
        for (int t = sg.t0; t < sg.t1; ++t, ++nq) {
          float* to = lse_ring + nq % kLseRing * kQRows + lane;
#pragma unroll
          for (int k = 0; k < 3; ++k) to[32 * k] = nxt[k] == -INFINITY ? -INFINITY : nxt[k] * -1.4426950408889634f;
          mbar_arrive(&lse_full[nq % kLseRing]);
          const int rt0 = rt, h0 = h;
          if (++rt == sg.rts) {
            rt = 0;
            ++h;
          }
          if (t + 1 < sg.t1) stats(rt, h, nxt);
          // (also without TMA: the ring of statistics must not run ahead of the queries)
          if (nq >= (uint32_t)C::kQSlots && ok &&
              !__all_sync(0xffffffffu, mbar_wait_cycles(&q_empty[nq % C::kQSlots], (nq / C::kQSlots - 1) & 1))) {
            ok = false;
            if (lane == 0) atomicOr(a.b.err, (uint32_t)ATTN_TIMEOUT);
          }
          if (tma_q) {
            if (lane == 0) mbar_arrive_expect_tx(&q_full[nq % C::kQSlots], C::kTileBytes);
            __syncwarp();
            // rows beyond the sequence's are another's or zero: their columns are masked
            if (lane < D / 64)
              tma_load_3d(smem + nq % C::kQSlots * C::kTileBytes + lane * (kQRows * 128), &qmap, 64 * lane, h0 * G,
                          sg.q.q0 + (int)fdiv((uint32_t)(sg.ra + rt0 * kQRows), a.g.gdiv), &q_full[nq % C::kQSlots]);
          }
        }
      }
    }
  } else if (warp >= 16) {
    // ====================== queries that TMA boxes do not fit ======================
    reg_dec<WeightRoles::kLoad>();
    const int pt = tid - 512;
    uint32_t nq = 0;
    constexpr int QCH = D / 8, QRP = 128 / QCH;           // 16-byte chunks of a query row, rows per pass
    // barriers of the copies in flight, oldest first (0: none)
    uint64_t *p0 = nullptr, *p1 = nullptr;
    auto give = [&](uint64_t*& p) {
      if (p) {
        fence_proxy_async_smem();
        mbar_arrive(p);
        p = nullptr;
      }
    };
    auto flush = [&] {
      cp_async_wait<0>();
      give(p0);
      give(p1);
    };
    while (!tma_q && next_segment(work, cu, sg)) {
      if (sg.rts == 0) continue;
      for (int t = sg.t0; t < sg.t1; ++t, ++nq) {
        const int rt = t % sg.rts, h = t / sg.rts, row = sg.ra + rt * kQRows + pt;
        if (pt < kQRows) {
          const int i = (int)fdiv((uint32_t)row, a.g.gdiv), hd = h * G + row - i * G;
          qptrs[(nq & 1) * kQRows + pt] = row < sg.rb ? a.q + (int64_t)(sg.q.q0 + i) * a.q_stride + hd * D : nullptr;
        }
        named_bar(2, 128);
        const uint32_t slot = nq % C::kQSlots, parity = (nq / C::kQSlots - 1) & 1;
        if (nq >= (uint32_t)C::kQSlots && ok && !mbar_try_wait(&q_empty[slot], parity)) {
          flush();                                        // hand over what has arrived before waiting
          if (!mbar_wait_cycles(&q_empty[slot], parity)) {
            ok = false;
            atomicOr(a.b.err, (uint32_t)ATTN_TIMEOUT);
          }
        }
        const uint32_t dst = smem_u32(smem + slot * C::kTileBytes);
        const uint16_t* const* qp = qptrs + (nq & 1) * kQRows;
        const int ch = pt % QCH, rs = pt / QCH;
#pragma unroll 4
        for (int p = 0; p < kQRows / QRP; ++p) {
          const int r = p * QRP + rs;
          const uint16_t* src = qp[r];
          cp_async16(dst + tile_offset(r, ch, kQRows), src ? src + ch * 8 : a.q, src ? 16 : 0);
        }
        cp_async_commit();
        cp_async_wait<2>();
        give(p0);
        p0 = p1;
        p1 = &q_full[slot];
      }
    }
    flush();
  } else {
    // ================================ sums ================================
    reg_inc<WeightRoles::kAdd>();
    const int w = warp >> 3, hh = warp >> 2 & 1, row = tid & 127;       // tile, half of its columns, cell
    constexpr int kHalf = kQRows / 2, kDh = D / 2;       // columns of a thread; dimensions of K that it puts in place
    const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    uint32_t nq = 0;
    auto wait = [&](uint64_t* b, uint32_t parity) {
      if (ok && !__all_sync(0xffffffffu, mbar_wait_cycles(b, parity))) {
        ok = false;
        if (lane == 0) atomicOr(a.b.err, (uint32_t)ATTN_TIMEOUT);
      }
    };
    while (next_segment(work, cu, sg)) {
      const int j = sg.j0 + w * 128 + row;
      const bool mine = w * 128 + row < sg.cells;
      const uint8_t* cell = mine ? cell_ptr(a.b, sg.s, j) : nullptr;
      const int base = sg.q.len - sg.q.n;
      float sum = 0.f, f = a.g.scale_log2;
      int rt = sg.rts ? sg.t0 % sg.rts : 0, h = sg.rts ? sg.t0 / sg.rts : 0;
      // This thread's half of the cell's K vector of a head, into tensor memory, two dimensions a column.  Every product
      // on the K before has ended: its last scores are here.  (The vector is asked for a step ahead, as far as L2: held in
      // registers meanwhile it would cost the sums theirs.)
      constexpr int kRaw = I8 ? kDh / 16 : kDh / 8;       // 16-byte pieces
      auto k_half = [&](int head) { return cell + (head * D + hh * kDh) * (I8 ? 1 : 2); };
      auto fetch = [&](int head) {
        if (cell) asm volatile("prefetch.global.L2 [%0];" ::"l"(k_half(head)));
      };
      auto put = [&](int head) {
        const uint32_t col = lanes + C::kCol(w) + hh * (kDh / 2);
        constexpr int kAt = kRaw < 4 ? kRaw : 4;
        if (I8) f = cell ? reinterpret_cast<const float*>(cell + 2 * HKV * D)[head] * a.g.scale_log2 : 0.f;
#pragma unroll
        for (int x0 = 0; x0 < kRaw; x0 += kAt) {
          uint4 kv[kAt];
#pragma unroll
          for (int x = 0; x < kAt; ++x) {
            kv[x] = make_uint4(0, 0, 0, 0);
            if (cell) kv[x] = reinterpret_cast<const uint4*>(k_half(head))[x0 + x];
          }
#pragma unroll
          for (int x = 0; x < kAt; ++x) {
            if (!I8) {
              tmem_st4(col + 4 * (x0 + x), kv[x].x, kv[x].y, kv[x].z, kv[x].w);
            } else {
              const uint32_t ww[4] = {kv[x].x, kv[x].y, kv[x].z, kv[x].w};
#pragma unroll
              for (int y = 0; y < 4; y += 2) {
                uint32_t o[4];
#pragma unroll
                for (int z = 0; z < 2; ++z) {
                  if (BF16) {
                    o[2 * z] = codes2_bf16(__byte_perm(ww[y + z], 0, 0x4140));
                    o[2 * z + 1] = codes2_bf16(__byte_perm(ww[y + z], 0, 0x4342));
                  } else {
                    codes4_f16(ww[y + z], o[2 * z], o[2 * z + 1]);
                  }
                }
                tmem_st4(col + 8 * (x0 + x) + 2 * y, o[0], o[1], o[2], o[3]);
              }
            }
          }
        }
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(&k_full[w]);
      };
      if (sg.rts) put(h);
      for (int t = sg.t0; sg.rts && t < sg.t1; ++t, ++nq) {
        const int r0 = sg.ra + rt * kQRows;
        const bool last = rt + 1 == sg.rts && t + 1 < sg.t1;     // a new head follows
        if (last) fetch(h + 1);
        if (++rt == sg.rts) {
          rt = 0;
          ++h;
        }
        // Columns that see this cell: rows of the sequence, tokens from the cell's own on, and fewer than `window` after it.
        const int64_t cmin = (int64_t)max(0, j - base) * G - r0;
        const int64_t cend = a.b.window ? min((int64_t)sg.rb, ((int64_t)j - base + a.b.window) * G) - r0 : (int64_t)sg.rb - r0;
        const int lo = (int)min(max(cmin, (int64_t)0), (int64_t)kQRows), hi = (int)min(max(cend, (int64_t)0), (int64_t)kQRows);
        const bool whole = __all_sync(0xffffffffu, lo == 0 && hi == kQRows);
        const uint32_t b = nq & 1;
        wait(&lse_full[nq % kLseRing], (nq / kLseRing) & 1);
        wait(&s_full[w][b], (nq >> 1) & 1);
        tc_fence_after();
        const float f_now = f;
        uint64_t s0 = 0, s1 = 0;
        uint32_t v0[32], v1[16];
        const uint32_t s_tm = lanes + C::kColS(w, b) + kHalf * hh;
        tmem_ld32(s_tm, v0);
        tmem_ld16(s_tm + 32, v1);
        tmem_ld_wait();
        tc_fence_before();
        mbar_arrive(&s_empty[w][b]);
        if (last) put(h);                                 // (`h` is the next head by now)
        const ulonglong2* ls = reinterpret_cast<const ulonglong2*>(lse_ring + nq % kLseRing * kQRows + kHalf * hh);
        const uint64_t ff = f2(f_now, f_now);
        if (whole) {
#pragma unroll
          for (int e = 0; e < kHalf; e += 4) {
            const ulonglong2 l4 = ls[e / 4];
            const uint32_t* x = e < 32 ? &v0[e & 31] : &v1[e & 15];
            const uint64_t t0 = fma2(f2(__uint_as_float(x[0]), __uint_as_float(x[1])), ff, l4.x);
            const uint64_t t1 = fma2(f2(__uint_as_float(x[2]), __uint_as_float(x[3])), ff, l4.y);
            s0 = add2(s0, f2(ex2(lo2(t0)), ex2(hi2(t0))));
            s1 = add2(s1, f2(ex2(lo2(t1)), ex2(hi2(t1))));
          }
        } else {
          const int c0 = kHalf * hh;
          const uint64_t bits = ((1ull << min(max(hi - c0, 0), kHalf)) - 1) & ~((1ull << min(max(lo - c0, 0), kHalf)) - 1);
          const float* l = reinterpret_cast<const float*>(ls);
#pragma unroll
          for (int e = 0; e < kHalf; ++e) {
            const float p = ex2(fmaf(__uint_as_float(e < 32 ? v0[e & 31] : v1[e & 15]), f_now, l[e]));
            sum += bits >> e & 1u ? p : 0.f;
          }
        }
        s0 = add2(s0, s1);
        sum += lo2(s0) + hi2(s0);
      }
      if (hh) half_sum[w * 128 + row] = sum;
      named_bar(3, 512);
      if (!hh) sum += half_sum[w * 128 + row];
      named_bar(3, 512);                                  // (before the next segment's)
      if (hh) continue;
      if (!cell) sum = 0.f;                               // a cell of a page that is not there
      if (sg.parts == 1) {
        if (mine) {
          const int64_t at = (int64_t)sg.s * a.acc_stride + j;
          a.acc_out[at] = (a.acc_in ? a.acc_in[at] * a.decay : 0.f) + sum;
        }
      } else {
        float* part = a.ws + ((int64_t)blockIdx.x * 2 + (sg.starts ? 1 : 0)) * a.ws_slot;
        __stcg(part + w * 128 + row, sum);
        if (tid == 0 && sg.starts) a.cuts[blockIdx.x] = AttnCut{sg.parts, sg.s, sg.j0, sg.cells, 0};
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 20) tmem_dealloc(tmem_slot, 512);
}

// Adds the parts of the item that begins in CTA `blockIdx.x`, in their order (slots as in attn_join.cu).
__global__ void __launch_bounds__(kCells) weights_join_kernel(const __grid_constant__ AttnWgtArgs a) {
  pdl_wait();
  const AttnCut cut = a.cuts[blockIdx.x];
  if (cut.parts == 0 || (int)threadIdx.x >= cut.nrows) return;
  const float* first = a.ws + ((int64_t)blockIdx.x * 2 + 1) * a.ws_slot + threadIdx.x;
  float sum = 0.f;
#pragma unroll 8
  for (int p = 0; p < cut.parts; ++p) sum += __ldcg(first + (p ? (2 * (int64_t)p - 1) * a.ws_slot : 0));
  const int64_t at = (int64_t)cut.q0 * a.acc_stride + cut.r0 + threadIdx.x;
  a.acc_out[at] = (a.acc_in ? a.acc_in[at] * a.decay : 0.f) + sum;
}

template <bool BF16, int D, bool I8>
cudaError_t launch_wc(const AttnWgtArgs& a, const CUtensorMap& qmap, int tma_q, cudaStream_t s) {
  static_assert(WcCfg<D>::kSmem <= 226 * 1024, "shared memory");
  const void* fn = reinterpret_cast<const void*>(weights_chunk_kernel<BF16, D, I8>);
  cudaError_t e = ensure_dyn_smem(fn, WcCfg<D>::kSmem);
  if (e != cudaSuccess) return e;
  // the roles' registers must fit what the block is launched with
  static const int regs = [fn] {
    cudaFuncAttributes at;
    return cudaFuncGetAttributes(&at, fn) == cudaSuccess ? at.numRegs : 0;
  }();
  if (regs * kThreads < WeightRoles::Block::registers()) return cudaErrorLaunchOutOfResources;
  weights_chunk_kernel<BF16, D, I8><<<a.num_sms, kThreads, WcCfg<D>::kSmem, s>>>(a, qmap, tma_q);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.num_sms);
  cfg.blockDim = dim3(kCells);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, weights_join_kernel, a);
}

}  // namespace

cudaError_t launch_attn_weights_chunk(const AttnWgtArgs& a, const CUtensorMap& qmap, int tma_q, cudaStream_t s) {
  const bool bf = a.g.io == MOE_T_BF16, i8 = a.g.kv == MOE_T_I8;
  if (a.g.D == 128) {
    if (bf) return i8 ? launch_wc<true, 128, true>(a, qmap, tma_q, s) : launch_wc<true, 128, false>(a, qmap, tma_q, s);
    return i8 ? launch_wc<false, 128, true>(a, qmap, tma_q, s) : launch_wc<false, 128, false>(a, qmap, tma_q, s);
  }
  if (bf) return i8 ? launch_wc<true, 64, true>(a, qmap, tma_q, s) : launch_wc<true, 64, false>(a, qmap, tma_q, s);
  return i8 ? launch_wc<false, 64, true>(a, qmap, tma_q, s) : launch_wc<false, 64, false>(a, qmap, tma_q, s);
}

}  // namespace moe
