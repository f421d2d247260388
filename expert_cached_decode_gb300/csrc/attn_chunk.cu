// Attention of many rows (prompt chunks, long drafts) over the paged cache on
// the tensor cores.
//
// S = Q K^T and O += P V are tcgen05 products of 128 rows x 128 cells x D with
// accumulators in tensor memory.  Two streams, A and B, run against each other
// so that the products of one overlap the softmax of the other:
//   ROWS = 256: A and B are the two halves of a row tile and share every K and
//               V tile;
//   ROWS = 128: A takes the even cell tiles and B the odd ones of one row
//               tile, and the two are joined at the item's end (items of at
//               most 128 rows, where half of a 256-row tile would be padding).
// Roles of a CTA's warps: 0-3 softmax of A, 4-7 of B (one thread per row),
// 8-11 gather the tiles that TMA cannot copy and expand int8 ones, 12 issues
// the products (both streams': with a warp for each, a chunk took 3% longer,
// 17% against int8 cells), 13 finds the cells and issues the TMA copies.
// P goes back to tensor memory over S, as the A operand of P V; V is read as
// it lies (cells x dimensions) through a transposed descriptor.
//
// A row's reference (its largest score so far) is only raised when the scores
// outgrow it by 2^8, so the output in tensor memory is rarely rescaled.  In
// fp16 it lies 2^7 below the largest score: P then uses the type's range up to
// 2^15, and small probabilities keep their bits down to 2^-21 of the largest.
// A commit tracks all products issued before it: when S of tile j is complete,
// P V of the stream's tile before is too, and its softmax threads may rescale O
// without another barrier.
//
// Bound by the chain of a stream's softmax and products.  4,096 tokens of 32
// heads over 32,768 bf16 cells take 1,422 us (1,450 TFLOP/s; int8 cells, whose
// tiles pass through shared memory twice and whose scores take two more
// multiplications, 1,900 us; D = 64, with half the products per exponential,
// 1,234 us); five tokens of 8 sequences over 8,192 to 32,768 int8 cells 72 us,
// most of it for expanding the tiles.
#include "attn_tc.cuh"

namespace moe {

namespace {

constexpr int kTile = 128;            // cells per tile
constexpr int kThreads = ChunkRoles::Block::kThreads;
// units that an item costs besides its tiles (its first loads and products and its output overlap with nothing), and
// the fewest units of a part
constexpr int kOvh = 3, kMinUnits = 6;

struct Bars {
  uint64_t full[12], empty[12], raw_full[10], raw_empty[10], info[16], q_full[2], s_full[2], p_ready[2], o_full[2], drained;
  uint32_t tmem;
};

// Shared memory.  The ring of K and V tiles is as deep as it goes: an SM needs some 125 KB under way (45 KB a
// microsecond at 2 to 3 us) to stream the cells from memory.  Against int8 cells that is the raw tiles' ring.
template <int D, bool I8, int ROWS>
struct ChunkCfg {
  static constexpr int kMatBytes = kTile * D * 2;              // K or V tile in 16 bits
  // 3 slots are the least: a V tile and the next K tile are held at once
  static constexpr int kSlots = I8 ? (D == 128 ? 3 : 6) : (ROWS == 128 ? 6 : 5) * (128 / D);
  static constexpr int kQBytes = ROWS * D * 2;
  static constexpr int kRaw = I8 ? (ROWS == 128 ? 5 : 3) * (128 / D) : 0;
  static constexpr int kRawBytes = kTile * D;
  // Ring of the tiles' valid bits and scales.  Those of tile j + R are written once the loads of tile j + R - 1 are
  // under way, that is when the products of the loads kSlots + kRaw before have ended; two tiles of margin.
  static constexpr int kInfo = D == 128 ? 8 : 16;
  static_assert(2 * (kInfo - 2) >= kSlots + kRaw, "scales outlive their use");
  static constexpr int kInfoBytes = kInfo * ((I8 ? 2 * kTile * 4 : 0) + 48);
  static constexpr int kOff_slots = kQBytes;
  static constexpr int kOff_raw = kOff_slots + kSlots * kMatBytes;
  static constexpr int kOff_info = kOff_raw + kRaw * kRawBytes;
  static constexpr int kOff_rows = kOff_info + kInfoBytes;
  static constexpr int kOff_ml = kOff_rows + 2 * kTile * 4;    // stream B's maxima and sums (ROWS = 128)
  static constexpr int kOff_bar = kOff_ml + (ROWS == 128 ? 2 * 128 * 4 : 0);
  static constexpr int kSmem = kOff_bar + (int)sizeof(Bars);
};


__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}

// V as the B operand: N = dimensions run along the 128-byte rows (64 to a
// block of kTile rows), K = cells down the rows.  Leading offset: to the next
// 64 dimensions; stride offset: to the next 8 cells.
__device__ __forceinline__ uint64_t v_desc(const void* tile) {
  uint64_t d = (smem_u32(tile) >> 4) & 0x3FFFull;
  d |= (uint64_t)((kTile * 128) >> 4) << 16;
  d |= (uint64_t)(1024 >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}

// Load i of a segment of `tiles` tiles, in the order in which the products take them: K0, V0, K1, V1, ... (both streams
// on every tile), or K0, K1, V0, K2, V1, K3, ... and at the end the last two V (a stream per tile).
template <bool SPLIT>
__device__ __forceinline__ void load_at(int i, int tiles, bool& is_v, int& j) {
  if (!SPLIT) {
    is_v = i & 1;
    j = i >> 1;
  } else if (i < 2) {
    is_v = i == 1 && tiles == 1;
    j = is_v ? 0 : i;
  } else {
    is_v = i > 2 * tiles - 3 || !(i & 1);
    j = i > 2 * tiles - 3 ? i - tiles : is_v ? (i - 2) >> 1 : (i + 1) >> 1;
  }
}

// A wait that gave up turns every later wait of its warp into nothing: the
// roles then run through their loops (on wrong data, in bounds) so that every
// barrier is still met, and the error word says that the results are void.
template <bool BF16, int D, bool I8, int ROWS>
__global__ void __launch_bounds__(kThreads, 1)
    chunk_kernel(const __grid_constant__ AttnFwdArgs a, const __grid_constant__ CUtensorMap map, int box) {
  using C = ChunkCfg<D, I8, ROWS>;
  constexpr bool SPLIT = ROWS == 128;
  constexpr bool TBF = BF16 && !I8;      // type of the products: the cells', fp16 for int8 cells
  constexpr int kInfo = C::kInfo;
  extern __shared__ __align__(1024) uint8_t smem[];
  Bars& bar = *reinterpret_cast<Bars*>(smem + C::kOff_bar);
  CursorScratch& scr = *reinterpret_cast<CursorScratch*>(smem);       // (the queries' place, before there are any)
  uint8_t* slots = smem + C::kOff_slots;
  uint8_t* raw = smem + C::kOff_raw;
  float* info = reinterpret_cast<float*>(smem + C::kOff_info);          // [kInfo][ks 128][vs 128] (int8 cells)
  uint32_t* info_valid = reinterpret_cast<uint32_t*>(info + (I8 ? kInfo * 2 * kTile : 0));   // [kInfo][valid 4, scales' maxima 4, TMA 1, -]
  int32_t* rows = reinterpret_cast<int32_t*>(smem + C::kOff_rows);      // [2][kTile] the tiles' cells (-1: hidden)
  float* ml = reinterpret_cast<float*>(smem + C::kOff_ml);              // [2][128]
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = a.g.g, HKV = a.g.hkv;
  if (tid == 0) a.cuts[blockIdx.x].parts = 0;
  pdl_launch_dependents();
  Cursor cu;
  const Work<ROWS, kTile, kOvh> work{a.b, a.g.gdiv, HKV, a.rows_min, a.rows_max};
  if (!find_part<kThreads, kMinUnits>(work, scr, reinterpret_cast<int64_t*>(slots), cu)) {
    pdl_wait();
    return;
  }
  Segment g;

  __syncthreads();                       // `slots` held the sequences' units
  if (tid == 0) {
    for (int i = 0; i < C::kSlots; ++i) {
      mbar_init(&bar.full[i], I8 ? 128 : 129);   // warps 8-11 (and warp 13)
      mbar_init(&bar.empty[i], 1);
    }
    for (int i = 0; i < C::kRaw; ++i) {
      mbar_init(&bar.raw_full[i], 1);
      mbar_init(&bar.raw_empty[i], 128);
    }
    for (int i = 0; i < kInfo; ++i) mbar_init(&bar.info[i], 32);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar.q_full[i], 128);
      mbar_init(&bar.s_full[i], 1);
      mbar_init(&bar.p_ready[i], 128);
      mbar_init(&bar.o_full[i], 1);
    }
    mbar_init(&bar.drained, 1);
    mbar_init_fence();
  }
  if (warp == 12) {
    tmem_alloc(&bar.tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  constexpr uint32_t tmem = 0;           // all 512 columns are this block's
  bool ok = true;

  if (warp >= 12) {
    // ================================ products ================================
    reg_dec<ChunkRoles::kProducts>();
    if (warp == 12) {
      const uint32_t id_s = idesc_f16(128, kTile, TBF), id_o = idesc_f16(128, D, TBF) | 1u << 16;
      uint32_t n_load = 0, n_q[2] = {0, 0}, np[2] = {0, 0};   // loads consumed, Q tiles and P tiles taken
      auto wait = [&](uint64_t* b, uint32_t parity) {
        if (ok && !__all_sync(0xffffffffu, mbar_wait_cycles(b, parity))) {
          ok = false;
          if (lane == 0) atomicOr(a.b.err, (uint32_t)ATTN_TIMEOUT);
        }
      };
      auto wait_load = [&](uint32_t n) { wait(&bar.full[n % C::kSlots], (n / C::kSlots) & 1); };
      auto commit = [&](uint64_t* b) {
        if (ok && elect_one()) umma_commit(b);
        __syncwarp();
      };
      // descriptors are one addition away from these
      const uint64_t q0d = smem_desc_sw128(smem), k0d = smem_desc_sw128(slots), v0d = v_desc(slots);
      // S of stream w from load n (its last reader: `last`)
      auto scores = [&](int w, uint32_t n, bool last) {
        const uint64_t qd = q0d + (SPLIT ? 0 : w) * ((128 * D * 2) >> 4), kd = k0d + n % C::kSlots * (C::kMatBytes >> 4);
        tc_fence_after();
        if (ok && elect_one()) {
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            const int off = ((k >> 2) * (128 * 128) >> 4) + 2 * (k & 3);
            umma_f16(w * 128, qd + off, kd + off, id_s, k != 0);
          }
          umma_commit(&bar.s_full[w]);
          if (last) umma_commit(&bar.empty[n % C::kSlots]);
        }
        __syncwarp();
      };
      // O of stream w from load n
      auto output = [&](int w, uint32_t n, bool first, bool last) {
        const uint64_t vd = v0d + n % C::kSlots * (C::kMatBytes >> 4);
        wait(&bar.p_ready[w], np[w]++ & 1);
        tc_fence_after();
        if (ok && elect_one()) {
#pragma unroll
          for (int k = 0; k < kTile / 16; ++k)
            umma_f16_ts(256 + w * 128, w * 128 + 8 * k, vd + k * (2048 >> 4), id_o, !first || k != 0);
          if (last) umma_commit(&bar.empty[n % C::kSlots]);
        }
        __syncwarp();
      };
      while (next_segment(work, cu, g)) {
        const int tiles = g.t1 - g.t0;
        const bool two = SPLIT ? tiles > 1 : g.nrows > 128;
        wait(&bar.q_full[0], n_q[0]++ & 1);
        if (!SPLIT && two) wait(&bar.q_full[1], n_q[1]++ & 1);
        if (!SPLIT) {
          // loads: K0, V0, K1, V1, ...
          wait_load(n_load);
          scores(0, n_load, !two);
          if (two) scores(1, n_load, true);
          for (int j = 0; j < tiles; ++j) {
            const uint32_t nv = n_load + 2 * j + 1, nk = nv + 1;
            const bool more = j + 1 < tiles;
            wait_load(nv);
            if (more) wait_load(nk);
#pragma unroll
            for (int w = 0; w < 2; ++w) {
              if (w == 1 && !two) break;
              const bool last = w == (two ? 1 : 0);
              output(w, nv, j == 0, last);
              if (more) scores(w, nk, last);
              else commit(&bar.o_full[w]);
            }
          }
        } else {
          // loads: K0, K1, V0, K2, V1, K3, V2, ...; tile j belongs to stream j & 1
          auto load_k = [&](int j) { return n_load + (j < 2 ? j : 2 * j - 1); };
          auto load_v = [&](int j) { return n_load + (two ? min(2 * j + 2, tiles + j) : 1); };
          for (int j = 0; j < 2 && j < tiles; ++j) {
            wait_load(load_k(j));
            scores(j, load_k(j), true);
          }
          for (int j0 = 0; j0 < tiles; j0 += 2)
#pragma unroll
            for (int w = 0; w < 2; ++w) {
              const int j = j0 + w;
              if (j >= tiles) break;
              wait_load(load_v(j));
              output(w, load_v(j), j < 2, true);
              if (j + 2 < tiles) {
                wait_load(load_k(j + 2));
                scores(w, load_k(j + 2), true);
              } else {
                commit(&bar.o_full[w]);
              }
            }
        }
        n_load += 2 * tiles;
      }
      // every product has ended before the tensor memory is given back, also after a wait that gave up
      if (elect_one()) {
        umma_commit(&bar.drained);
        if (!mbar_wait_cycles(&bar.drained, 0)) atomicOr(a.b.err, (uint32_t)ATTN_TIMEOUT);
      }
    } else if (warp == 13) {
      // ============================== tile plan, TMA ==============================
      // Lane l finds the cells l, 32 + l, 64 + l, 96 + l of a tile: page ids two tiles ahead, scales one, so that no
      // load is waited for within a tile.
      uint32_t n = 0, n_tile = 0;
      const int v_off = HKV * D * (I8 ? 1 : 2), sc_off = 2 * v_off;
      struct Found {
        int row[4];
        float ks[4], vs[4];
      };
      while (next_segment(work, cu, g)) {
        const int tiles = g.t1 - g.t0;
        auto cell_at = [&](int j, int k) { return g.jbase + j * kTile + 32 * k + lane; };
        auto ids_of = [&](int j, int (&id)[4]) {        // loads only: nothing waits for them here
#pragma unroll
          for (int k = 0; k < 4; ++k) id[k] = page_id(a.b, g.s, cell_at(j, k), g.lo, j < tiles ? g.jend : 0);
        };
        auto rows_of = [&](int j, const int (&id)[4], int (&row)[4]) {
#pragma unroll
          for (int k = 0; k < 4; ++k) row[k] = row_of_page(a.b, id[k], cell_at(j, k));
        };
        auto scales = [&](Found& f) {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            f.ks[k] = f.vs[k] = 0.f;
            if (I8 && f.row[k] >= 0) {
              const uint8_t* cell = row_ptr(a.b, f.row[k]) + sc_off + 4 * g.h;
              f.ks[k] = *reinterpret_cast<const float*>(cell);
              f.vs[k] = *reinterpret_cast<const float*>(cell + 4 * HKV);
            }
          }
        };
        Found cur;                       // of the tile that is planned next
        int nxt[4];                      // page ids of the one after
        ids_of(0, nxt);
        rows_of(0, nxt, cur.row);
        ids_of(1, nxt);
        scales(cur);
        const int boxes = box ? kTile / box : 1, issuers = boxes * (I8 ? 1 : D / 64);
        const int blk = lane / boxes, bx = lane - blk * boxes;      // this lane's box of a tile
        int y0 = 0, y1 = 0;              // its first row, for even and odd tiles
        uint32_t tma = 0;
#pragma unroll 1
        for (int i = 0; i < 2 * tiles; ++i, ++n) {
          bool is_v;
          int j;
          load_at<SPLIT>(i, tiles, is_v, j);
          if (!is_v) {                   // plan tile j
            const uint32_t e = n_tile % kInfo;
            uint32_t all = 0xffffffffu;
            int y = 0;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const uint32_t vm = __ballot_sync(0xffffffffu, cur.row[k] >= 0);
              all &= vm;
              if (lane == k) info_valid[e * 12 + k] = vm;
              const int yk = __shfl_sync(0xffffffffu, cur.row[k], bx * box & 31);
              if ((bx * box >> 5) == k) y = yk;
              if (I8) {
                info[e * 2 * kTile + 32 * k + lane] = cur.ks[k];
                info[e * 2 * kTile + kTile + 32 * k + lane] = cur.vs[k];
                const uint32_t top = __reduce_max_sync(0xffffffffu, finite_bits(scale_bits(cur.vs[k])));
                if (lane == k) info_valid[e * 12 + 4 + k] = top;
              }
            }
            const uint32_t t = all == 0xffffffffu && box > 0;
            if (lane == 0) info_valid[e * 12 + 8] = t;
            mbar_arrive(&bar.info[e]);
            ++n_tile;
            if (j & 1) y1 = y;
            else y0 = y;
            tma = (tma & ~(1u << (j & 1))) | t << (j & 1);
            rows_of(j + 1, nxt, cur.row);
            ids_of(j + 2, nxt);
            scales(cur);
          }
          // every load passes here, so that the barriers' phases count loads; what TMA cannot copy, warps 8-11 gather
          constexpr uint32_t R = I8 ? C::kRaw : C::kSlots;
          uint64_t* eb = I8 ? &bar.raw_empty[n % R] : &bar.empty[n % R];
          uint64_t* fb = I8 ? &bar.raw_full[n % R] : &bar.full[n % R];
          if (n >= R && ok && !__all_sync(0xffffffffu, mbar_wait_cycles(eb, (n / R - 1) & 1))) {
            ok = false;
            if (lane == 0) atomicOr(a.b.err, (uint32_t)ATTN_TIMEOUT);
          }
          if (tma >> (j & 1) & 1u) {
            if (lane == 0) mbar_arrive_expect_tx(fb, I8 ? C::kRawBytes : C::kMatBytes);
            __syncwarp();
            const int off = (is_v ? v_off : 0) + g.h * D * (I8 ? 1 : 2);
            uint8_t* dst = (I8 ? raw + n % R * C::kRawBytes : slots + n % R * C::kMatBytes) +
                           blk * (kTile * 128) + bx * box * (I8 ? D : 128);
            if (lane < issuers) tma_load_2d(dst, &map, I8 ? off : (off >> 1) + 64 * blk, j & 1 ? y1 : y0, fb);
          } else if (lane == 0) {
            mbar_arrive(fb);
          }
        }
      }
    }
  } else if (warp >= 8) {
    // ================================ cells ================================
    reg_dec<ChunkRoles::kCells>();
    const int pt = tid - 256;
    // What TMA does not do: tiles that are not all there or whose pages are not cut into boxes are gathered 16 bytes at
    // a time, and int8 tiles are expanded.
    const uint8_t* none = reinterpret_cast<const uint8_t*>(a.q);   // address of copies that read nothing
    uint32_t n = 0, n_tile = 0;          // loads, tiles
    constexpr int kRowBytes = D * (I8 ? 1 : 2), CH = kRowBytes / 16, RPP = 128 / CH;   // chunks per row, rows per pass
    constexpr uint32_t R = C::kRaw ? C::kRaw : 1;
    const int ch = pt % CH, rsub = pt / CH;
    const int v_off = HKV * kRowBytes;
    auto wait = [&](uint64_t* b, uint32_t parity) {
      if (ok && !mbar_wait_cycles(b, parity)) {
        ok = false;
        atomicOr(a.b.err, (uint32_t)ATTN_TIMEOUT);
      }
    };
    auto wait_empty = [&](uint32_t i) {  // the slot of load i is free
      if (i >= (uint32_t)C::kSlots) wait(&bar.empty[i % C::kSlots], (i / C::kSlots - 1) & 1);
    };
    // load i has arrived: int8 is expanded from its raw tile into its slot, as fp16
    auto finish = [&](uint32_t i) {
      if (I8) {
        wait(&bar.raw_full[i % R], (i / R) & 1);
        const uint8_t* src = raw + i % R * C::kRawBytes + pt * 16;    // chunk ch of the rows rsub, rsub + RPP, ...
        uint8_t* dst = slots + (i % C::kSlots) * C::kMatBytes;
        // Rows whose loads go ahead of their stores (the compiler may not move them there).  With one stream's softmax
        // at work at a time that pays (eight sequences' 40 rows over 32,768 to 8,192 cells: 72 us, was 76); next to both
        // streams' it takes their issue slots (a 4,096-token chunk: 1,910 us, 2,030 with four).
        constexpr int kB = SPLIT ? 4 : 1;
        uint4 x[kB];
        auto load = [&](int p) {
#pragma unroll
          for (int y = 0; y < kB; ++y) x[y] = *reinterpret_cast<const uint4*>(src + (p + y) * RPP * CH * 16);
        };
        load(0);
        wait_empty(i);
        // the eight lanes of a row write eight different chunks modulo 8 at a time: the upper half odd ones first
        const bool up = ch & 4;
#pragma unroll (SPLIT ? 1 : 2)
        for (int p = 0; p < kTile / RPP; p += kB) {
          if (p) load(p);
#pragma unroll
          for (int y = 0; y < kB; ++y) {
            const int r = (p + y) * RPP + rsub;
            uint4 e, f;
            codes4_f16(x[y].x, e.x, e.y);
            codes4_f16(x[y].y, e.z, e.w);
            codes4_f16(x[y].z, f.x, f.y);
            codes4_f16(x[y].w, f.z, f.w);
            *reinterpret_cast<uint4*>(dst + tile_offset(r, 2 * ch + up, kTile)) = up ? f : e;
            *reinterpret_cast<uint4*>(dst + tile_offset(r, 2 * ch + !up, kTile)) = up ? e : f;
          }
        }
      }
      fence_proxy_async_smem();
      mbar_arrive(&bar.full[i % C::kSlots]);
      if (I8) mbar_arrive(&bar.raw_empty[i % R]);
    };
    uint32_t pending = 0;                // gathered loads before n that are not finished
    constexpr uint32_t kLag = I8 && C::kRaw < 3 ? 1 : 2;
    auto flush = [&] {
      cp_async_wait<0>();
      for (; pending; --pending) finish(n - pending);
    };
    while (next_segment(work, cu, g)) {
      const int tiles = g.t1 - g.t0;
      uint32_t tma = 0;
      const uint32_t b0 = n_tile;
#pragma unroll 1
      for (int i = 0; i < 2 * tiles; ++i, ++n) {
        bool is_v;
        int j;
        load_at<SPLIT>(i, tiles, is_v, j);
        int32_t* tr = rows + ((b0 + j) & 1) * kTile;
        if (!is_v) {
          const uint32_t e = n_tile % kInfo;
          wait(&bar.info[e], (n_tile / kInfo) & 1);
          const uint32_t t = info_valid[e * 12 + 8];
          ++n_tile;
          tma = (tma & ~(1u << (j & 1))) | t << (j & 1);
          if (!t) {                      // thread r finds the cell r
            const int cell = g.jbase + j * kTile + pt;
            const int row = cell >= g.lo && cell < g.jend ? cell_row(a.b, g.s, cell) : -1;
            named_bar(2, 128);           // every thread has read the cells that these replace
            tr[pt] = row;
            named_bar(2, 128);
          }
        }
        if (tma >> (j & 1) & 1u) {
          if (pending) flush();
          if (!I8) wait_empty(n);        // (an arrival counts for the load whose phase it is)
          finish(n);
          continue;
        }
        if (!I8 && n >= (uint32_t)C::kSlots) {
          // hand over what has arrived before waiting for a slot
          if (pending && !mbar_try_wait(&bar.empty[n % C::kSlots], (n / C::kSlots - 1) & 1)) flush();
          wait_empty(n);
        }
        const int off = (is_v ? v_off : 0) + g.h * kRowBytes;
        const uint32_t dst = smem_u32(I8 ? raw + n % R * C::kRawBytes : slots + n % C::kSlots * C::kMatBytes);
#pragma unroll 4
        for (int p = 0; p < kTile / RPP; ++p) {
          const int r = p * RPP + rsub;
          const uint8_t* src = row_ptr(a.b, tr[r]);
          const uint32_t to = I8 ? (uint32_t)((r * CH + ch) * 16) : tile_offset(r, ch, kTile);
          cp_async16(dst + to, src ? src + off + ch * 16 : none, src ? 16 : 0);
        }
        cp_async_commit();
        ++pending;
        if (pending > kLag) {
          cp_async_wait<kLag>();
          finish(n + 1 - pending);
          --pending;
        }
      }
    }
    flush();
  } else {
    // ================================ softmax ================================
    reg_inc<ChunkRoles::kSoftmax>();
    const int w = warp >> 2, row = tid & 127;
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t s_tm = tmem + lane_base + w * 128, o_tm = tmem + lane_base + 256 + w * 128;
    uint32_t n_s = 0, n_o = 0, n_ob = 0, n_tile = 0;     // S tiles and outputs of this stream; tiles of the CTA
    auto wait = [&](uint64_t* b, uint32_t parity) {
      if (ok && !__all_sync(0xffffffffu, mbar_wait_cycles(b, parity))) {
        ok = false;
        if (lane == 0) atomicOr(a.b.err, (uint32_t)ATTN_TIMEOUT);
      }
    };
    while (next_segment(work, cu, g)) {
      const int tiles = g.t1 - g.t0;
      const bool active = SPLIT ? w < tiles : w * 128 < g.nrows;
      const int r = (SPLIT ? 0 : w * 128) + row;             // row within the item
      const bool real = r < g.nrows;
      const int ti = real ? (int)fdiv((uint32_t)(g.r0 + r), a.g.gdiv) : 0, hd = g.h * G + (real ? g.r0 + r - ti * G : 0);
      int rlo = 0, rhi = INT32_MAX;        // a padding row: no mask (its result is not used)
      if (real) row_range(g.q, a.b.window, ti, rlo, rhi);
      const bool any_real = __any_sync(0xffffffffu, real);
      float sc = a.g.scale_log2;           // factor of this row's scores
      // ---- Q of this stream into shared memory (SPLIT: stream A's threads for both).  A stream that is idle in an
      // item does not arrive: it could run ahead of the products by more than the barrier's two phases ----
      if (SPLIT ? w == 0 : active) {
        const uint16_t* src = a.q + (int64_t)(g.q.q0 + ti) * a.q_stride + hd * D;
        uint8_t* dst = smem + (SPLIT ? 0 : w) * (128 * D * 2);
        float u = 1.f;
        if (I8 && BF16) {                  // against int8 cells bf16 queries go as fp16, in units of their row's largest
          float top = 0.f;
#pragma unroll 4
          for (int c = 0; real && c < D / 8; ++c) {
            const uint4 v = *reinterpret_cast<const uint4*>(src + 8 * c);
            const uint32_t x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              const float2 f = Half16<true>::unpack(x[y]);
              top = fmaxf(top, fmaxf(fabsf(f.x), fabsf(f.y)));
            }
          }
          u = row_unit(top);
          if (SPLIT) ml[row] = u;          // for stream B's threads
        }
        sc = a.g.scale_log2 * u;
        const float inv = inv_pow2(u);
#pragma unroll 4
        for (int c = 0; c < D / 8; ++c) {
          uint4 v = make_uint4(0, 0, 0, 0);
          if (real) v = *reinterpret_cast<const uint4*>(src + 8 * c);
          if (I8 && BF16) {
            v.x = bf16_to_f16(v.x, inv);
            v.y = bf16_to_f16(v.y, inv);
            v.z = bf16_to_f16(v.z, inv);
            v.w = bf16_to_f16(v.w, inv);
          }
          *reinterpret_cast<uint4*>(dst + tile_offset(row, c, 128)) = v;
        }
        fence_proxy_async_smem();
        mbar_arrive(&bar.q_full[w]);
      }
      if (SPLIT && I8 && BF16) {
        named_bar(3, 256);
        sc = a.g.scale_log2 * ml[row];
        if (tiles > 1) named_bar(3, 256);  // `ml` is used again at the segment's end
      }
      float m = -INFINITY, l = 0.f;
      for (int j = SPLIT ? w : 0; active && j < tiles; j += SPLIT ? 2 : 1) {
        const uint32_t in = (n_tile + j) % kInfo;
        wait(&bar.info[in], ((n_tile + j) / kInfo) & 1);
        wait(&bar.s_full[w], n_s++ & 1);
        tc_fence_after();
        if (!any_real) {                   // a warp of padding rows: whatever P holds reaches only their output
          tc_fence_before();
          mbar_arrive(&bar.p_ready[w]);
          continue;
        }
        const int j0 = g.jbase + j * kTile;
        const uint4 vw = *reinterpret_cast<const uint4*>(info_valid + in * 12);
        const bool whole = __all_sync(0xffffffffu, j0 >= rlo && j0 + kTile <= rhi) &&
                           (vw.x & vw.y & vw.z & vw.w) == 0xffffffffu;
        // S is read once, in two halves of 64 cells.  (One loop: the roles share the instruction cache, and a row's 128
        // scores in registers made the code of this one alone larger than it.)  When the reference grows at the second
        // half, the first one's probabilities are scaled down along with the output.
        uint64_t l0 = 0, l1 = 0;
#pragma unroll 1
        for (int hh = 0; hh < 2; ++hh) {
          uint32_t v[2][32];
          tmem_ld32(s_tm + 64 * hh, v[0]);
          tmem_ld32(s_tm + 64 * hh + 32, v[1]);
          tmem_ld_wait();
          if (I8) {
            const float4* ks = reinterpret_cast<const float4*>(info + in * 2 * kTile) + 16 * hh;
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
              for (int e = 0; e < 32; e += 4) {
                const float4 k4 = ks[8 * c + e / 4];
#pragma unroll
                for (int y = 0; y < 4; y += 2) {
                  const uint64_t x = mul2(f2(__uint_as_float(v[c][e + y]), __uint_as_float(v[c][e + y + 1])),
                                          y ? f2(k4.z, k4.w) : f2(k4.x, k4.y));
                  v[c][e + y] = __float_as_uint(lo2(x));
                  v[c][e + y + 1] = __float_as_uint(hi2(x));
                }
              }
          }
          if (!whole) {
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              // bit e: this row sees the cell e of the 32
              const int cl = min(max(rlo - j0 - 64 * hh - 32 * c, 0), 32), ch = min(max(rhi - j0 - 64 * hh - 32 * c, 0), 32);
              const uint32_t word = hh ? (c ? vw.w : vw.z) : (c ? vw.y : vw.x);
              const uint32_t bits = word & (uint32_t)((1ull << ch) - 1) & ~(uint32_t)((1ull << cl) - 1);
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (!(bits >> e & 1u)) v[c][e] = 0xff800000u;
            }
          }
          float mx[4];
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            const uint32_t* x = &v[y >> 1][16 * (y & 1)];
            mx[y] = fmaxf(__uint_as_float(x[0]), __uint_as_float(x[1]));
#pragma unroll
            for (int e = 2; e < 16; e += 2) mx[y] = fmaxf(mx[y], fmaxf(__uint_as_float(x[e]), __uint_as_float(x[e + 1])));
          }
          float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * sc;
          if (I8) {
            const uint4 tw = *reinterpret_cast<const uint4*>(info_valid + in * 12 + 4);
            top += scale_exp(max(max(tw.x, tw.y), max(tw.z, tw.w)));
          }
          if (!TBF) top -= 7.f;
          const bool grow = top > m + 8.f || (m == -INFINITY && top > -INFINITY);
          if (__any_sync(0xffffffffu, grow)) {
            // a whole number: probabilities that are scaled down are not rounded again
            top = ceilf(top);
            const float f = grow ? ex2(m - top) : 1.f;
            if (grow) {
              m = top;
              l *= f;
              l0 = mul2(l0, f2(f, f));
              l1 = mul2(l1, f2(f, f));
            }
            // (16 columns at a time: this half's 64 scores stay in registers)
            uint32_t t[16];
            auto st16 = [&](uint32_t to) {
#pragma unroll
              for (int e = 0; e < 16; e += 4) tmem_st4(to + e, t[e], t[e + 1], t[e + 2], t[e + 3]);
            };
            if (hh) {
              tmem_st_wait();
#pragma unroll 1
              for (int c = 0; c < 32; c += 16) {
                tmem_ld16(s_tm + c, t);
                tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                  const float2 x = Half16<TBF>::unpack(t[e]);
                  t[e] = Half16<TBF>::pack(x.x * f, x.y * f);
                }
                st16(s_tm + c);
              }
            }
            if (j >= (SPLIT ? 2 : 1)) {
#pragma unroll 1
              for (int c = 0; c < D; c += 16) {
                tmem_ld16(o_tm + c, t);
                tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 16; ++e) t[e] = __float_as_uint(__uint_as_float(t[e]) * f);
                st16(o_tm + c);
              }
            }
          }
          const float base = m == -INFINITY ? 0.f : m;
          const uint64_t sc2 = f2(sc, sc), nb2 = f2(-base, -base);
          const float4* vs = reinterpret_cast<const float4*>(info + in * 2 * kTile + kTile) + 16 * hh;
          uint32_t p[32];
#pragma unroll
          for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int e = 0; e < 32; e += 4) {
              const uint32_t* x = &v[c][e];
              const uint64_t t0 = fma2(f2(__uint_as_float(x[0]), __uint_as_float(x[1])), sc2, nb2);
              const uint64_t t1 = fma2(f2(__uint_as_float(x[2]), __uint_as_float(x[3])), sc2, nb2);
              uint64_t p0 = f2(ex2(lo2(t0)), ex2(hi2(t0))), p1 = f2(ex2(lo2(t1)), ex2(hi2(t1)));
              l0 = add2(l0, p0);
              l1 = add2(l1, p1);
              if (I8) {
                const float4 s4 = vs[8 * c + e / 4];
                p0 = mul2(p0, f2(s4.x, s4.y));
                p1 = mul2(p1, f2(s4.z, s4.w));
              }
              p[16 * c + e / 2] = Half16<TBF>::pack(lo2(p0), hi2(p0));
              p[16 * c + e / 2 + 1] = Half16<TBF>::pack(lo2(p1), hi2(p1));
            }
          tmem_st32(s_tm + 32 * hh, p);
        }
        l0 = add2(l0, l1);
        l += lo2(l0) + hi2(l0);
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(&bar.p_ready[w]);
      }
      n_tile += tiles;
      // ---- output ----
      const bool single = g.parts == 1;
      float* part = a.ws + ((int64_t)blockIdx.x * 2 + (g.starts ? 1 : 0)) * a.ws_slot;
      if (active) wait(&bar.o_full[w], n_o++ & 1);
      // SPLIT: stream A's threads also take B's output (the same lanes of tensor memory) and its m and l
      const bool both = SPLIT && tiles > 1;
      float fa = 1.f, fb = 0.f;
      if (both) {
        if (w == 1) {
          ml[row] = m;
          ml[128 + row] = l;
        }
        named_bar(3, 256);
        if (w == 0) {
          wait(&bar.o_full[1], n_ob++ & 1);
          const float mb = ml[row], M = fmaxf(m, mb);
          fa = m == M ? 1.f : ex2(m - M);
          fb = mb == M ? 1.f : ex2(mb - M);
          l = fa * l + fb * ml[128 + row];
          m = M;
        }
      }
      tc_fence_after();
      const int64_t at = (int64_t)(g.q.q0 + ti) * a.g.hq + hd;
      if (active && (!SPLIT || w == 0)) {
        const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t o[32];
          tmem_ld32(o_tm + 32 * c, o);
          tmem_ld_wait();
          if (both) {
            uint32_t ob[32];
            tmem_ld32(o_tm + 128 + 32 * c, ob);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 32; ++e)
              o[e] = __float_as_uint(__uint_as_float(o[e]) * fa + __uint_as_float(ob[e]) * fb);
          }
          if (real && single) {
#pragma unroll
            for (int e = 0; e < 32; e += 8) {
              uint32_t p[4];
#pragma unroll
              for (int y = 0; y < 4; ++y)
                p[y] = Half16<BF16>::pack(__uint_as_float(o[e + 2 * y]) * inv, __uint_as_float(o[e + 2 * y + 1]) * inv);
              *reinterpret_cast<uint4*>(a.out + at * D + 32 * c + e) = make_uint4(p[0], p[1], p[2], p[3]);
            }
          } else if (real) {
#pragma unroll
            for (int e = 0; e < 32; e += 4)
              __stcg(reinterpret_cast<float4*>(part + r * D + 32 * c + e),
                     make_float4(__uint_as_float(o[e]), __uint_as_float(o[e + 1]), __uint_as_float(o[e + 2]),
                                 __uint_as_float(o[e + 3])));
          }
        }
        if (real && single) {
          if (a.lse) a.lse[at] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
        } else if (real) {
          __stcg(part + ROWS * D + r, m);
          __stcg(part + ROWS * (D + 1) + r, l);
        }
      }
      tc_fence_before();
      if (both) named_bar(3, 256);       // B's output has been read: its next item may overwrite it
      if (tid == 0 && g.starts && !single)   // this CTA begins a cut item: what the joining kernel needs
        a.cuts[blockIdx.x] = AttnCut{g.parts, g.q.q0, g.r0, g.nrows, g.h};
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 12) tmem_dealloc(bar.tmem, 512);
  // Launched after a kernel that it does not depend on, this one may not end before it: what follows waits for this one
  // only.
  pdl_wait();
}

template <bool BF16, int D, bool I8, int ROWS>
cudaError_t launch_chunk(const AttnFwdArgs& a, const CUtensorMap& map, int box, bool after, cudaStream_t s) {
  constexpr int smem = ChunkCfg<D, I8, ROWS>::kSmem;
  static_assert(smem <= 227 * 1024, "shared memory");
  const void* fn = reinterpret_cast<const void*>(chunk_kernel<BF16, D, I8, ROWS>);
  cudaError_t e = ensure_dyn_smem(fn, smem);
  if (e != cudaSuccess) return e;
  // the roles' registers must fit what the block is launched with
  static const int regs = [fn] {
    cudaFuncAttributes at;
    return cudaFuncGetAttributes(&at, fn) == cudaSuccess ? at.numRegs : 0;
  }();
  if (regs * kThreads < ChunkRoles::Block::registers()) return cudaErrorLaunchOutOfResources;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.num_sms);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = after ? 1 : 0;
  e = cudaLaunchKernelEx(&cfg, chunk_kernel<BF16, D, I8, ROWS>, a, map, box);
  if (e != cudaSuccess) return e;
  return launch_attn_join(a, ROWS, s);
}

}  // namespace

cudaError_t launch_attn_chunk(const AttnFwdArgs& a, const CUtensorMap& map, int box, int max_q, bool after, cudaStream_t s) {
  const bool bf = a.g.io == MOE_T_BF16, i8 = a.g.kv == MOE_T_I8;
  const bool few = (int64_t)max_q * a.g.g <= 128;
#define CHUNK(BF, DD, I) \
  return few ? launch_chunk<BF, DD, I, 128>(a, map, box, after, s) : launch_chunk<BF, DD, I, 256>(a, map, box, after, s)
  if (a.g.D == 128) {
    if (bf && i8) CHUNK(true, 128, true);
    if (bf) CHUNK(true, 128, false);
    if (i8) CHUNK(false, 128, true);
    CHUNK(false, 128, false);
  }
  if (bf && i8) CHUNK(true, 64, true);
  if (bf) CHUNK(true, 64, false);
  if (i8) CHUNK(false, 64, true);
  CHUNK(false, 64, false);
#undef CHUNK
}

}  // namespace moe
