// Shared by the attention kernels (attn_*.cu): the call's sequences, the cells
// and their types, and the row geometry.
#pragma once

#include <cuda.h>

#include "attn_plan.h"
#include "common.cuh"
#include "internal.h"

namespace moe {

// Bits of an attention handle's error word.
enum AttnErr : uint32_t {
  ATTN_BAD_PAGE = 1,     // a page id outside [0, n_pages)
  ATTN_BAD_LEN = 2,      // a length or an offset out of range
  ATTN_TIMEOUT = 4,      // a bounded device wait gave up
};

// Division of n < 2^31 by a number fixed per handle: with l = ceil(log2 d) and
// m = floor(2^32 (2^l - d) / d) + 1, n / d = (mulhi(m, n) + n) >> l.
struct FastDiv {
  uint32_t d, m, l;
};
inline FastDiv make_fastdiv(uint32_t d) {
  FastDiv f{d, 0, 0};
  while ((1ull << f.l) < d) ++f.l;
  f.m = (uint32_t)((((1ull << f.l) - d) << 32) / d + 1);
  return f;
}
__host__ __device__ __forceinline__ uint32_t fdiv(uint32_t n, const FastDiv& f) {
#ifdef __CUDA_ARCH__
  return (__umulhi(f.m, n) + n) >> f.l;
#else
  return (uint32_t)((((uint64_t)f.m * n) >> 32) + n) >> f.l;
#endif
}

// The sequences of a call and the cells, as every kernel takes them.
struct AttnBatch {
  uint8_t* cells;
  const int32_t* table;
  const int32_t* kv_lens;
  const int32_t* cu_q;
  uint32_t* err;
  int64_t page_bytes;        // page_cells * cell_bytes
  int32_t cell_bytes, page_cells, n_pages, n_seqs, table_pages, n_tokens, window;
  int32_t max_len;           // table_pages * page_cells
  FastDiv page_div;
};

struct SeqInfo {
  int32_t q0, n, len;        // first token, new tokens, cells
};

// Sequence s with its values cut to their ranges (and reported when they were not in them).
__device__ __forceinline__ SeqInfo seq_info(const AttnBatch& b, int s) {
  const int a = b.cu_q[s], e = b.cu_q[s + 1], l = b.kv_lens[s];
  SeqInfo i;
  i.q0 = min(max(a, 0), b.n_tokens);
  i.n = min(max(e, i.q0), b.n_tokens) - i.q0;
  i.len = min(max(l, 0), b.max_len);
  if (i.q0 != a || i.q0 + i.n != e || i.len != l) atomicOr(b.err, (uint32_t)ATTN_BAD_LEN);
  return i;
}

// The cells [lo, hi) that row i of n new tokens sees.
__device__ __forceinline__ void row_range(const SeqInfo& q, int window, int i, int& lo, int& hi) {
  hi = max(0, q.len - q.n + i + 1);
  lo = window ? max(0, hi - window) : 0;
}

// Row (among all cells) of cell j (0 <= j < max_len) of sequence s, or -1 when its page is out of range.
__device__ __forceinline__ int cell_row(const AttnBatch& b, int s, int j) {
  const uint32_t pg = fdiv((uint32_t)j, b.page_div);
  const int id = b.table[(int64_t)s * b.table_pages + pg];
  if ((uint32_t)id >= (uint32_t)b.n_pages) {
    atomicOr(b.err, (uint32_t)ATTN_BAD_PAGE);
    return -1;
  }
  return id * b.page_cells + (j - (int)pg * b.page_cells);
}
// The same in two steps, where the page's id is fetched ahead: the load alone (kHiddenCell for a cell outside
// [lo, hi)), and what becomes of it.
constexpr int kHiddenCell = INT32_MIN;
__device__ __forceinline__ int page_id(const AttnBatch& b, int s, int j, int lo, int hi) {
  if (j < lo || j >= hi) return kHiddenCell;
  return b.table[(int64_t)s * b.table_pages + fdiv((uint32_t)j, b.page_div)];
}
__device__ __forceinline__ int row_of_page(const AttnBatch& b, int id, int j) {
  if (id == kHiddenCell) return -1;
  if ((uint32_t)id >= (uint32_t)b.n_pages) {
    atomicOr(b.err, (uint32_t)ATTN_BAD_PAGE);
    return -1;
  }
  return id * b.page_cells + (j - (int)fdiv((uint32_t)j, b.page_div) * b.page_cells);
}
__device__ __forceinline__ uint8_t* row_ptr(const AttnBatch& b, int row) {
  return row < 0 ? nullptr : b.cells + (int64_t)row * b.cell_bytes;
}
__device__ __forceinline__ uint8_t* cell_ptr(const AttnBatch& b, int s, int j) { return row_ptr(b, cell_row(b, s, j)); }

// The sequence that token t belongs to, or -1 (cu_q ascending; empty ones are passed over).
__device__ __forceinline__ int seq_of(const AttnBatch& b, int t) {
  int lo = 0, hi = b.n_seqs;          // first s with cu_q[s + 1] > t
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (b.cu_q[mid + 1] > t) hi = mid;
    else lo = mid + 1;
  }
  return lo < b.n_seqs && b.cu_q[lo] <= t ? lo : -1;
}

// 16-bit element types
template <bool BF16>
struct Half16;
template <>
struct Half16<true> {
  static __device__ __forceinline__ float2 unpack(uint32_t u) {
    return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
  }
  static __device__ __forceinline__ uint32_t pack(float a, float b) {   // a in the low half
    uint32_t d;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(b), "f"(a));
    return d;
  }
};
template <>
struct Half16<false> {
  static __device__ __forceinline__ float2 unpack(uint32_t u) {
    return __half22float2(*reinterpret_cast<const __half2*>(&u));
  }
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    uint32_t d;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(b), "f"(a));
    return d;
  }
};

// ---- asynchronous copies and exponentials ----
// 16 bytes global -> shared; bytes beyond `valid` (0 or 16) are filled with zeros.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(valid) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src, int valid) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(valid) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// 2^x, 2 ulp
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// int8 codes -> 16-bit floats, exactly.  fp16: 0x6400 | (code ^ 0x80) is 1024 + 128 + code, so four codes take an
// exclusive or, two byte permutations that set the high bytes, and two subtractions.
__device__ __forceinline__ uint32_t sub_1152(uint32_t x) {
  uint32_t d;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(x), "r"(0x64806480u));
  return d;
}
__device__ __forceinline__ void codes4_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  const uint32_t x = w ^ 0x80808080u;
  lo = sub_1152(__byte_perm(x, 0x64646464u, 0x4140));
  hi = sub_1152(__byte_perm(x, 0x64646464u, 0x4342));
}
// the same for two cells' words: d[i] holds byte i of `u` (low half) and of `w`
__device__ __forceinline__ void codes4x2_f16(uint32_t u, uint32_t w, uint32_t (&d)[4]) {
  const uint32_t x = u ^ 0x80808080u, y = w ^ 0x80808080u;
  const uint32_t s = __byte_perm(x, y, 0x5140), t = __byte_perm(x, y, 0x7362);
  d[0] = sub_1152(__byte_perm(s, 0x64646464u, 0x4140));
  d[1] = sub_1152(__byte_perm(s, 0x64646464u, 0x4342));
  d[2] = sub_1152(__byte_perm(t, 0x64646464u, 0x4140));
  d[3] = sub_1152(__byte_perm(t, 0x64646464u, 0x4342));
}
// Against int8 cells the products run in fp16, which holds codes as cheaply
// as it gets, probabilities with 11 bits, and bf16 queries exactly once a row
// is divided by a power of two near its largest value (elements 2^-14 below
// that lose bits that no score can show).  `row_unit` gives that power from
// the largest magnitude's bits (1 for an all-zero row, and for one that is not
// finite).
__device__ __forceinline__ float row_unit(float top) {
  const uint32_t e = __float_as_uint(top) & 0x7f800000u;
  return e == 0 || e == 0x7f800000u ? 1.f : __uint_as_float(e);
}
// 1 / a power of two (of at least 2^-126 and at most 2^126; beyond, the nearest of those)
__device__ __forceinline__ float inv_pow2(float u) {
  return __uint_as_float(min(max(0x7f000000u - __float_as_uint(u), 0x00800000u), 0x7e800000u));
}
// two bf16 values times a power of two, as fp16
__device__ __forceinline__ uint32_t bf16_to_f16(uint32_t w, float f) {
  const float2 v = Half16<true>::unpack(w);
  return Half16<false>::pack(v.x * f, v.y * f);
}
// The probabilities against int8 cells carry the V scales.  To keep them in
// fp16's range whatever the scales are, a row's reference is not its largest
// score but that plus the binary exponent of the scales: x - ref + log2(scale)
// <= 0 for every cell of a step.  `scale_exp` is that exponent (rounded up),
// from the bits of the step's largest scale.  Where a row may not see some cell
// of the step, a scale that is not finite does not count (`finite_bits`): the
// rows that see its cell get NaN from the product in any case, and for the
// others it would push every probability below fp16's range.
__device__ __forceinline__ uint32_t scale_bits(float scale) { return __float_as_uint(scale) & 0x7fffffffu; }
__device__ __forceinline__ uint32_t finite_bits(uint32_t bits) { return bits < 0x7f800000u ? bits : 0u; }
__device__ __forceinline__ float scale_exp(uint32_t bits) {
  return (float)min(max((int)(bits >> 23 & 255u) - 126, -64), 64);
}

// Two fp32 operations per instruction
__device__ __forceinline__ uint64_t f2(float a, float b) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ float2 un2(uint64_t a) {
  float2 d;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(d.x), "=f"(d.y) : "l"(a));
  return d;
}
__device__ __forceinline__ float lo2(uint64_t a) { return un2(a).x; }
__device__ __forceinline__ float hi2(uint64_t a) { return un2(a).y; }

// D = A(16x16) * B(16x8) + D in 16-bit inputs, fp32 sums
template <bool BF16>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if (BF16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// With K's rows in shared memory as columns of mma.sync products: the cell
// (within 16) that column n of n-tile nt is; a lane's two columns 2c, 2c + 1
// of a tile are 4 rows apart.
template <bool I8>
__device__ __forceinline__ int col_cell(int nt, int n) {
  return I8 ? (n >> 1) + 4 * (2 * nt + (n & 1)) : 8 * nt + (n >> 1) + 4 * (n & 1);
}

// ---- division of a call's work over the CTAs ----
// An item is (sequence, tile of ROWS rows, K/V head); its tiles are those of
// TK cells that its rows see (one if they see none: their rows still have to
// be written).  Rows count token by token, a token's heads of one K/V head
// next to each other: row r is token r / g, head r % g.  An item counts OVH
// units for what it costs besides its tiles (queries, first loads, output),
// then one per tile.  The units of all items, in the order sequence, row tile,
// head, cell tile, are cut into equal consecutive parts, one per CTA, so that
// long sequences, long chunks and many short ones all balance, whatever the
// lengths are.  An item whose tiles fall into several parts is joined from
// their sums (attn_join.cu).  Sequences outside (rows_min, rows_max] rows per
// head belong to the other kernel of the call.
template <int ROWS, int TK, int OVH>
struct Work {
  const AttnBatch& b;
  FastDiv g;
  int hkv, rows_min, rows_max;

  __device__ __forceinline__ int row_tiles(const SeqInfo& q) const {
    const int rows = q.n * (int)g.d;
    return rows > rows_min && rows <= rows_max ? (rows + ROWS - 1) / ROWS : 0;
  }
  // cells [lo, hi) that row tile `rt` sees, and the number of its tiles
  __device__ __forceinline__ int tiles(const SeqInfo& q, int rt, int& lo, int& hi) const {
    const int i0 = (int)fdiv((uint32_t)(rt * ROWS), g);
    const int i1 = (int)fdiv((uint32_t)(min((rt + 1) * ROWS, q.n * (int)g.d) - 1), g);
    const int base = q.len - q.n + 1;
    hi = max(0, base + i1);
    lo = b.window ? max(0, base + i0 - b.window) : 0;
    return hi > lo ? (hi + TK - 1) / TK - lo / TK : 1;
  }
  __device__ __forceinline__ int units(const SeqInfo& q, int rt) const {
    int lo, hi;
    return tiles(q, rt, lo, hi) + OVH;
  }
};

// A CTA's place in the work.
struct Cursor {
  int64_t u, end, total;     // next unit, end of this CTA's part, units of the call
  int parts;                 // CTAs that have a part
  int s, rt, h, t;           // sequence, row tile, head, unit within the item
};

// First unit of part p, and the part that owns unit u.  total < 2^31 * 2^16 and parts < 2^15, so no product
// overflows; the usual call's fit 32 bits, whose division is several times shorter.
__device__ __forceinline__ int64_t part_begin(const Cursor& c, int p) {
  if (c.total < (1 << 20)) return (uint32_t)c.total * (uint32_t)p / (uint32_t)c.parts;
  return c.total * p / c.parts;
}
__device__ __forceinline__ int unit_owner(const Cursor& c, int64_t u) {
  if (c.total < (1 << 20)) return (int)((((uint32_t)u + 1) * (uint32_t)c.parts - 1) / (uint32_t)c.total);
  return (int)(((u + 1) * c.parts - 1) / c.total);
}

struct CursorScratch {
  int64_t warp[32];
  int32_t items[32];
  int64_t off;
  int s;
};

// Every thread of the CTA (NT of them, a multiple of 32) calls this; `scr` is
// shared scratch, `seq_n` shared memory for n_seqs numbers.  Returns false if
// the CTA has no part.  There are as many parts as CTAs unless the call has
// both fewer items and fewer than MIN units for each.  A thread counts its
// sequences' units; one of many row tiles is counted by its whole warp.
template <int NT, int MIN, class W>
__device__ __forceinline__ bool find_part(const W& w, CursorScratch& scr, int64_t* seq_n, Cursor& c) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, n_seqs = w.b.n_seqs;
  const int per = (n_seqs + NT - 1) / NT, s0 = min(n_seqs, tid * per), s1 = min(n_seqs, s0 + per);
  int64_t mine = 0;
  int items = 0;
  for (int k = 0; k < per; ++k) {
    const int s = s0 + k;
    SeqInfo q{0, 0, 0};
    if (s < s1) q = seq_info(w.b, s);
    const int rts = w.row_tiles(q);
    int64_t n = 0;
    if (rts <= 4)
      for (int rt = 0; rt < rts; ++rt) n += w.units(q, rt);
    uint32_t big = __ballot_sync(0xffffffffu, rts > 4);
    while (big) {
      const int src = __ffs(big) - 1;
      big &= big - 1;
      const SeqInfo o{0, __shfl_sync(0xffffffffu, q.n, src), __shfl_sync(0xffffffffu, q.len, src)};
      const int r = __shfl_sync(0xffffffffu, rts, src);
      int64_t part = 0;
      for (int rt = lane; rt < r; rt += 32) part += w.units(o, rt);
#pragma unroll
      for (int x = 16; x; x >>= 1) part += (int64_t)shfl_u64((uint64_t)part, lane ^ x);
      if (lane == src) n = part;
    }
    n *= w.hkv;
    if (s < s1) seq_n[s] = n;
    mine += n;
    items += rts * w.hkv;
  }
  int64_t inc = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t n = (int64_t)shfl_u64((uint64_t)inc, lane >= o ? lane - o : lane);
    if (lane >= o) inc += n;
  }
  items = __reduce_add_sync(0xffffffffu, items);
  if (lane == 31) {
    scr.warp[warp] = inc;
    scr.items[warp] = items;
  }
  __syncthreads();
  int64_t before = 0, total = 0;
  items = 0;
#pragma unroll
  for (int x = 0; x < NT / 32; ++x) {
    const int64_t v = scr.warp[x];
    if (x < warp) before += v;
    total += v;
    items += scr.items[x];
  }
  c.total = total;
  c.parts = min((int)gridDim.x, max(items, (int)min(total / MIN, (int64_t)gridDim.x)));
  if ((int)blockIdx.x >= c.parts) return false;
  c.u = part_begin(c, (int)blockIdx.x);
  c.end = part_begin(c, (int)blockIdx.x + 1);
  before += inc - mine;               // units before this thread's sequences
  if (c.u >= before && c.u < before + mine) {
    int64_t off = c.u - before;
    int s = s0;
    while (off >= seq_n[s]) off -= seq_n[s++];
    scr.s = s;
    scr.off = off;
  }
  __syncthreads();
  c.s = scr.s;
  // the row tile: every warp looks through them, 32 at a time
  int64_t off = scr.off;
  const SeqInfo q = seq_info(w.b, c.s);
  const int rts = w.row_tiles(q);
  for (int r0 = 0;; r0 += 32) {
    const int64_t n = r0 + lane < rts ? w.units(q, r0 + lane) : 0;
    int64_t sum = n * w.hkv;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t x = (int64_t)shfl_u64((uint64_t)sum, lane >= o ? lane - o : lane);
      if (lane >= o) sum += x;
    }
    const uint32_t past = __ballot_sync(0xffffffffu, sum > off);
    if (past) {
      const int at = __ffs(past) - 1;
      const int units = __shfl_sync(0xffffffffu, (int)n, at);
      off -= (int64_t)shfl_u64((uint64_t)sum, at) - (int64_t)units * w.hkv;
      c.rt = r0 + at;
      c.h = (int)((uint32_t)off / (uint32_t)units);     // off < units * hkv < 2^31
      c.t = (int)off - c.h * units;
      return true;
    }
    off -= (int64_t)shfl_u64((uint64_t)sum, 31);
  }
}

// One item as far as it lies in this CTA's part: tiles [t0, t1) of `tiles`, cells [jbase, jend); parts > 1 if it is
// cut, then `slot` is the place of this CTA's part and `starts` says that it is the first.
struct Segment {
  SeqInfo q;
  int s, rt, h, r0, nrows, lo, hi, tiles, t0, t1, jbase, jend, parts;
  bool starts;
};

// The next segment of this CTA's part; false at its end.  (A part may end or begin within an item's OVH units: those
// hold no tiles.)
template <int ROWS, int TK, int OVH>
__device__ __forceinline__ bool next_segment(const Work<ROWS, TK, OVH>& w, Cursor& c, Segment& g) {
  while (c.u < c.end) {
    g.q = seq_info(w.b, c.s);
    g.s = c.s;
    g.rt = c.rt;
    g.h = c.h;
    g.tiles = w.tiles(g.q, c.rt, g.lo, g.hi);
    const int units = g.tiles + OVH, stop = (int)min((int64_t)units, c.t + (c.end - c.u));
    const int64_t u0 = c.u - c.t;                 // the item's first unit
    g.t0 = max(0, c.t - OVH);
    g.t1 = max(0, stop - OVH);
    c.u += stop - c.t;
    c.t = stop;
    if (stop == units) {
      c.t = 0;
      if (++c.h == w.hkv) {
        c.h = 0;
        if (++c.rt >= w.row_tiles(g.q)) {
          c.rt = 0;
          do {
            ++c.s;
          } while (c.s < w.b.n_seqs && w.row_tiles(seq_info(w.b, c.s)) == 0);
        }
      }
    }
    if (g.t1 <= g.t0) continue;
    g.parts = 1;
    g.starts = g.t0 == 0;
    if (g.t0 > 0 || g.t1 < g.tiles) {
      const int first = unit_owner(c, u0 + OVH), last = unit_owner(c, u0 + OVH + g.tiles - 1);
      g.parts = last - first + 1;
    }
    g.r0 = g.rt * ROWS;
    g.nrows = min(ROWS, g.q.n * (int)w.g.d - g.r0);
    g.jbase = (g.lo / TK + g.t0) * TK;
    g.jend = min(g.hi, g.jbase + (g.t1 - g.t0) * TK);
    return true;
  }
  return false;
}

// ---- launchers (one per kernel family) ----
struct AttnGeo {
  int hq, hkv, g, D, io, kv;      // g = hq / hkv
  float scale_log2;               // scale * log2(e)
  FastDiv gdiv;                   // division by g
};

struct AppendArgs {
  AttnBatch b;
  const uint16_t *q, *k, *v;
  uint16_t* q_out;
  int64_t q_stride, k_stride, v_stride;
  const int32_t* positions;
  const uint64_t* turns;          // device [rot/2]
  int hq, hkv, rot, interleaved;
  float factor;
};
cudaError_t launch_attn_append(const AppendArgs& a, const AttnGeo& g, cudaStream_t s);
cudaError_t launch_attn_read(const AttnBatch& b, const AttnGeo& g, uint16_t* k_out, uint16_t* v_out, cudaStream_t s);

// An item that is cut, for the kernel that joins it: parts (0: none), first token, row tile and rows, K/V head.
struct AttnCut {
  int32_t parts, q0, r0, nrows, h;
};

struct AttnFwdArgs {
  AttnBatch b;
  const uint16_t* q;
  int64_t q_stride;
  uint16_t* out;
  float* lse;
  AttnGeo g;
  // parts of items that are cut: two slots of ws_slot floats per CTA, slot 0 for an item that began in an earlier
  // CTA, slot 1 for one that goes on in the next; [row][D] sums, then the rows' maxima, then their totals
  float* ws;
  AttnCut* cuts;                  // per CTA: the cut item that begins in it
  int64_t ws_slot;
  int num_sms, rows_min, rows_max;
};
// Floats of one slot of the work space: the largest row tile's sums, maxima and totals.
inline int64_t attn_ws_slot(int D) { return (int64_t)256 * (D + 2); }
// join: launch the joining kernel too
cudaError_t launch_attn_rows(const AttnFwdArgs& a, int max_q, bool join, cudaStream_t s);
cudaError_t launch_attn_join(const AttnFwdArgs& a, int rows, cudaStream_t s);
// map: the cells as a 2-D tensor of 16-bit elements, in boxes of 64 x `box`; box 0: no map
// after: may start while the kernel before it in the stream, which it does not depend on, still runs
cudaError_t launch_attn_chunk(const AttnFwdArgs& a, const CUtensorMap& map, int box, int max_q, bool after, cudaStream_t s);

struct AttnWgtArgs {
  AttnBatch b;
  const uint16_t* q;
  int64_t q_stride;
  const float* lse;
  const float* acc_in;
  float* acc_out;
  int64_t acc_stride;
  float decay;
  AttnGeo g;
  float* ws;                      // parts of cut items, slots as in AttnFwdArgs, a float per cell
  AttnCut* cuts;                  // {parts, sequence, first cell, cells}
  int64_t ws_slot;
  int max_kv, num_sms;
};
cudaError_t launch_attn_weights_rows(const AttnWgtArgs& a, int max_q, cudaStream_t s);
constexpr int kWeightQRows = 96;   // query rows of a tile
// qmap: the queries as a 3-D tensor [token][head][D] in boxes of kWeightQRows / g tokens x g heads x 64 (tma_q: there is one)
cudaError_t launch_attn_weights_chunk(const AttnWgtArgs& a, const CUtensorMap& qmap, int tma_q, cudaStream_t s);

struct EvictArgs {
  AttnBatch b;
  const float* acc;
  int64_t acc_stride;
  int32_t budget, recent;
  const int32_t* new_table;
  int32_t new_table_pages;
  int32_t* keep;
  int32_t* new_lens;
  float* acc_out;
  int num_sms;
};
cudaError_t launch_attn_evict(const EvictArgs& a, cudaStream_t s);

}  // namespace moe
