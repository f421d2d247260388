// The gated delta rule's state through the chunks of a sequence
// (delta_intra.cu has prepared them), on the tensor cores (tcgen05):
//     Z = V - diag(e^G) K^ S      U = T Z      O = scale (diag(e^G) Q^ S + P U)
//     S <- e^(G_C) S + (diag(e^(G_C - G)) K^)^T U
// A CTA takes one head of one sequence; only S passes from chunk to chunk.  The
// products run transposed, a row of S^T (one of the v_dim columns of the state) to a
// lane of tensor memory: Y^T = S^T K^T, U^T = Z^T T^T, S^T += U'^T K.  So
// everything that follows the state is an A operand in tensor memory, never in
// shared memory; what does not (K, Q, T, P) lies in shared memory as it was
// prepared; S stays in registers, and a row's scales are a thread's own.
//
// Precision: the state stays fp32, and operands that stand for it hold 22 bits:
// a pair of fp16 numbers (x rounded, and the rest rounded) under a power of two
// per row, so a product takes two or three multiplications in fp16.  Only what
// reaches nothing but the outputs holds 11 bits: P, and where those are bf16 S and U
// in Q S and P U (in fp16, whose outputs show it, S and U are pairs there too).
//
// Roles of a CTA's 16 warps: 0-3 and 4-7 the chain (S -> Y -> Z -> U -> S: two
// threads per row, one for each half of the dimensions or of the tokens), 8-11 write
// the outputs and bring V, 12 brings the chunks, 13 issues the products, 14 scales V in chunks that grow.
//
// Bound by the chain's latency, 2.5 us a chunk of a 128 x 128 head: of its 4,900 cycles three products that wait for one another
// take 840, a row's conversions and the hand-overs between them the rest (tensor pipe 30%, issue
// slots 55%; 12,288 tokens of 32 heads whole some 467 us).  What it measured on the way there: one
// kernel with the chunks' own parts 1,584 us for that call, the chain on mma.sync
// over four SMs a head 494 (915 for nine prompts, which have no SMs to spare), four warpgroups of
// chain 514 instead of two.
#include "attn_tc.cuh"
#include "delta.cuh"

namespace moe {

namespace {

constexpr int C = kChunk;
constexpr int kThreads = DeltaRoles::Block::kThreads;
constexpr int kStages = 3;

// Columns of tensor memory.  SH: S^T's pairs (for every 32 dimensions 16 columns of first numbers and 16 of second ones), and
// when Y and QS are done the update of S.  Z's pairs replace Y, U' 's replace U, each likewise for every 32 tokens.
constexpr uint32_t kSH = 0, kY = 128, kU = 192, kUH = 256, kQS = 288, kPU = 352, kUL = 416;

enum : int { kBarS = 1 /* and 2 */, kBarZ = 3, kBarX = 4, kBarU = 5, kBarP = 6 };

struct Bars {
  uint64_t full[kStages], v_full[kStages], v_seen[kStages], v_ready[kStages], empty[kStages];
  uint64_t y_full, u_full, d_full[2], o_full, o_empty, drained;
  uint32_t tmem;
};

template <int DK, int DV>
struct Cfg {
  static constexpr int kMat = C * DK * 2, kKQ = 2 * kMat;
  static constexpr int kV = C * DV * 2;                   // V as it comes
  static constexpr int oTP = kKQ, oV = oTP + kTPBytes, kStage = oV + kV;
  static constexpr int oSc = kStages * kStage;            // the stages' scalars
  static constexpr int oX = oSc + kStages * (int)sizeof(DeltaScalars);   // a row's largest numbers of S, by its two threads [2][128]
  static constexpr int oVm = oX + 2 * 512;                // the stages' largest numbers of V, by halves of the tokens [2][128] 16 bits
  static constexpr int oLane = oVm + kStages * 512;       // the rows' factors of QS and PU, of a chunk and the one before [2][2][128]
  static constexpr int oBar = oLane + 4 * 512;
  static constexpr int kSmem = oBar + (int)sizeof(Bars);
};

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

// K as the B operand of the state's update: N = dimensions along the 128-byte rows (64 to a block of 64 rows), K = tokens
// down the rows.  Leading offset: to the next 64 dimensions; stride offset: to the next 8 tokens.
__device__ __forceinline__ uint64_t k_cols_desc(const void* tile) {
  uint64_t d = (smem_u32(tile) >> 4) & 0x3FFFull;
  d |= (uint64_t)((C * 128) >> 4) << 16;
  d |= (uint64_t)(1024 >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}

__device__ __forceinline__ float max_abs(float m, uint64_t x) { return fmaxf(m, fmaxf(fabsf(lo2(x)), fabsf(hi2(x)))); }
__device__ __forceinline__ uint64_t f2u(uint32_t a, uint32_t b) { return f2(__uint_as_float(a), __uint_as_float(b)); }
// 32 numbers (16 pairs) as A operand: 16 columns of first numbers and 16 of second ones
__device__ __forceinline__ void put_pairs(uint32_t taddr, const uint64_t* x) {
  uint32_t hi[16], lo[16];
#pragma unroll
  for (int j = 0; j < 16; ++j) halves(lo2(x[j]), hi2(x[j]), hi[j], lo[j]);
  tmem_st16(taddr, hi);
  tmem_st16(taddr + 16, lo);
}
// A product of two powers of two that stays a number (what it is multiplied with is 0 where it would not)
__device__ __forceinline__ float finite(float x) { return fminf(x, 3e38f); }

// A wait that gave up turns every later wait of its warp into nothing: the roles then run through their loops (on wrong
// data, in bounds) so that every barrier is still met, and the error word says that the results are void.
template <bool BF16, int DK, int DV>
__global__ void __launch_bounds__(kThreads, 1) chain_kernel(const __grid_constant__ DeltaFwdArgs a, const __grid_constant__ DeltaWork w) {
  using L = Cfg<DK, DV>;
  extern __shared__ __align__(1024) uint8_t smem[];
  Bars& bar = *reinterpret_cast<Bars*>(smem + L::oBar);
  DeltaScalars* scalars = reinterpret_cast<DeltaScalars*>(smem + L::oSc);
  float* xch = reinterpret_cast<float*>(smem + L::oX);
  float* factors = reinterpret_cast<float*>(smem + L::oLane);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, wg = tid >> 7, wt = tid & 127;
  const int h = blockIdx.x, hv = a.geo.hv;
  int s = blockIdx.y;
  if (w.ordered) {
    // the longest sequence first (equal ones in order, so that each has a place of its own)
    int* pick = reinterpret_cast<int*>(xch);
    if (tid < a.b.n_seqs) {
      const int64_t n = (int64_t)a.b.cu[tid + 1] - a.b.cu[tid];
      int before = 0;
      for (int o = 0; o < a.b.n_seqs; ++o) {
        const int64_t m = (int64_t)a.b.cu[o + 1] - a.b.cu[o];
        before += m > n || (m == n && o < tid);
      }
      if (before == s) *pick = tid;
    }
    __syncthreads();
    s = *pick;
    __syncthreads();
  }
  const DeltaSeq q = delta_seq(a.b, s);
  if (q.n < a.n_min || q.n > a.n_max) return;
  const int chunks = (q.n + C - 1) / C, base = delta_chunk_base(q.t0, s);
  // the chunks of this window, and this block's among them
  const int w0 = max(0, w.first - base), w1 = min(chunks, w.first + w.count - base);
  if (w0 >= w1) return;
  constexpr int MH = (DK + DV - 1) / DV;     // blocks that find M: a lane for a column
  const DeltaParts pt = delta_parts(w1 - w0, w.parts, w.front);
  int part = 0, mat = -1;                    // mat: this block finds columns mat * DV .. of M
  bool real = true;                          // whether this block takes the state itself through, and writes outputs
  if (w.pass == 1 && blockIdx.z > 0) {
    part = 1 + (blockIdx.z - 1) / (1 + MH);
    mat = (int)((blockIdx.z - 1) % (1 + MH)) - 1;
    real = false;
    if (part >= pt.parts - 1) return;
  } else if (w.pass == 2) {
    part = 1 + blockIdx.z;
    if (part >= pt.parts) return;
  }
  const int c0 = w0 + (part ? pt.first + (part - 1) * pt.len : 0), c1 = min(w1, c0 + (part ? pt.len : pt.first));
  const int64_t seg = ((int64_t)s * w.parts + part) * hv + h;
  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&bar.full[i], 1);
      mbar_init(&bar.v_full[i], 128);
      mbar_init(&bar.v_seen[i], 128);
      mbar_init(&bar.v_ready[i], 1);
      mbar_init(&bar.empty[i], 129);         // the products that read it, and warps 8-11 (its scalars)
    }
    mbar_init(&bar.y_full, 1);
    mbar_init(&bar.u_full, 1);
    mbar_init(&bar.d_full[0], 1);
    mbar_init(&bar.d_full[1], 1);
    mbar_init(&bar.o_full, 129);             // the products, and warps 0-3 (the rows' factors)
    mbar_init(&bar.o_empty, 128);
    mbar_init(&bar.drained, 1);
    mbar_init_fence();
  }
  if (warp == 13) {
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
  const bool live = wt < DV;

  if (wg < 2) {
    // ================================ the chain ================================
    reg_inc<DeltaRoles::kChain>();
    constexpr int NB = DK / 64;              // blocks of 32 dimensions of this thread's half
    const int hf = wg;
    const int64_t slot = (int64_t)hv * DK * DV, at = ((int64_t)h * DK + hf * (DK / 2)) * DV + wt, row = (int64_t)hf * (DK / 2) * DV + wt;
    // Units: powers of two per row under which no number passes 2^14, known before the numbers are: from V's largest number, a
    // bound of S's, and the chunk's own bounds.  That of the next S starts from S's largest number, which is found while U's
    // products run.  So S's unit is some 2^4 too large, Z's and U's another 2^4 (S's 2^12 where beta |k^|^2 passes 2), which the
    // pairs have to spare: numbers 2^17 below a unit's range still hold 22 bits.  Those of a row that are smaller yet hold as
    // many bits less: any is off by 2^-38 of its row's bound, as of a state that decays to nothing within the chunk.
    // S is kept in its unit.
    uint64_t S[16 * NB];
    float m = 0.f;
    {
      const float* src = !live || !real      ? nullptr
                         : part > 0 ? w.part_state + seg * DK * DV + row
                         : c0 > 0   ? w.carry[w.parity] + at
                         : q.in >= 0 ? a.state + q.in * slot + at
                                     : nullptr;
      const int one = mat < 0 ? -1 : mat * DV + wt - hf * (DK / 2);      // where the identity has its 1
#pragma unroll
      for (int j = 0; j < 16 * NB; ++j) {
        S[j] = src ? f2(src[2 * j * DV], src[(2 * j + 1) * DV]) : f2(one == 2 * j ? 1.f : 0.f, one == 2 * j + 1 ? 1.f : 0.f);
        m = max_abs(m, S[j]);
      }
    }
    xch[hf * 128 + wt] = m;
    named_bar(kBarX, 256);
    float bound = fmaxf(m, xch[(hf ^ 1) * 128 + wt]);        // of S's numbers
    Unit us = unit_of(bound);
    named_bar(kBarX, 256);
#pragma unroll
    for (int j = 0; j < 16 * NB; ++j) S[j] = mul2(S[j], f2(us.to, us.to));
    uint64_t fs = 0;                         // what S is multiplied with as its update comes
    for (int i = c0; i <= c1; ++i) {
      const int n_ = i - c0, st = n_ % kStages;
      const DeltaScalars& sc = scalars[st];
      // ---- S ----
      if (n_ > 0) {
        wait(&bar.d_full[hf], (n_ - 1) & 1);
        tc_fence_after();
      }
      if (live) {
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          const uint32_t to = lane_base + kSH + 32 * (hf * NB + b);
          if (n_ > 0) {
            uint32_t d[32];
            tmem_ld32(to, d);
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 16; ++j) S[16 * b + j] = fma2(S[16 * b + j], fs, f2u(d[2 * j], d[2 * j + 1]));
          }
          if (i < c1) put_pairs(to, S + 16 * b);
        }
        tmem_st_wait();
      }
      if (i == c1) break;
      tc_fence_before();
      named_bar_arrive(kBarS + hf, 160);
      // ---- while Y's products run: Z's and U's units, V ----
      uint64_t c2[16], z[16];                // e^G K^'s factors; V
      wait(&bar.full[st], (n_ / kStages) & 1);
      wait(&bar.v_ready[st], (n_ / kStages) & 1);
      float ku = 0.f, vm = 0.f;              // U's accumulator to U in its unit; V's largest number
      Unit uz{0.f, 0.f};
      if (live) {
        const uint16_t* top = reinterpret_cast<const uint16_t*>(smem + L::oVm + st * 512) + wt;
        vm = fmaxf(load16<BF16>(top), load16<BF16>(top + 128));
        uz = unit_of(vm + sc.zs * bound);
        const Unit uo = unit_of(sc.uv * vm + sc.us * bound);
        const float ny = -finite(us.from * uz.to);
        ku = finite(uz.from * uo.to);
        if (hf == 0) {
          factors[(n_ & 1) * 256 + wt] = us.from;
          factors[(n_ & 1) * 256 + 128 + wt] = uo.from;
        }
        const uint16_t* p = reinterpret_cast<const uint16_t*>(smem + st * L::kStage + L::oV) + 32 * hf * DV + wt;
        const uint64_t n2 = f2(ny, ny), to = f2(uz.to, uz.to);
#pragma unroll
        for (int j = 0; j < 16; j += 2) {
          const float4 c4 = *reinterpret_cast<const float4*>(&sc.c[32 * hf + 2 * j]);
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            c2[j + e] = mul2(e ? f2(c4.z, c4.w) : f2(c4.x, c4.y), n2);
            z[j + e] = mul2(f2(load16<BF16>(p + 2 * (j + e) * DV), load16<BF16>(p + (2 * (j + e) + 1) * DV)), to);
          }
        }
      }
      // ---- Z = V - diag(e^G) K^ S, this thread's 32 tokens ----
      wait(&bar.y_full, n_ & 1);
      tc_fence_after();
      if (live) {
        uint32_t y[32];
        tmem_ld32(lane_base + kY + 32 * hf, y);
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 16; ++j) z[j] = fma2(c2[j], f2u(y[2 * j], y[2 * j + 1]), z[j]);
        put_pairs(lane_base + kY + 32 * hf, z);
        tmem_st_wait();
      }
      tc_fence_before();
      named_bar_arrive(kBarZ, 288);
      // ---- while U's products run: the next S's unit ----
      if (live) {
        float ms[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < 16 * NB; ++j) ms[j & 3] = max_abs(ms[j & 3], S[j]);
        m = fmaxf(fmaxf(ms[0], ms[1]), fmaxf(ms[2], ms[3]));
        xch[hf * 128 + wt] = m;
      }
      named_bar(kBarX, 256);
      float kx = 0.f;                        // U's accumulator to U' in the next S's unit
      if (live) {
        bound = sc.xv * vm + (sc.xs + sc.decay) * (fmaxf(m, xch[(hf ^ 1) * 128 + wt]) * us.from);
        const Unit next = unit_of(bound);
        const float keep = sc.decay * us.from * next.to;
        kx = finite(uz.from * next.to);
        us = next;
        fs = f2(keep, keep);
      }
      // ---- U, and what it adds to the state ----
      wait(&bar.u_full, n_ & 1);
      tc_fence_after();
      uint32_t x[32];
      if (live) {
        tmem_ld32(lane_base + kU + 32 * hf, x);
        const uint64_t x2 = f2(kx, kx);
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 16; j += 2) {
          const float4 w4 = *reinterpret_cast<const float4*>(&sc.rx[32 * hf + 2 * j]);
          z[j] = mul2(f2u(x[2 * j], x[2 * j + 1]), mul2(f2(w4.x, w4.y), x2));
          z[j + 1] = mul2(f2u(x[2 * j + 2], x[2 * j + 3]), mul2(f2(w4.z, w4.w), x2));
        }
        put_pairs(lane_base + kU + 32 * hf, z);
        tmem_st_wait();
      }
      tc_fence_before();
      named_bar_arrive(kBarU, 288);
      if (!real) continue;
      if (live) {                            // U itself for the outputs, while S's products run
        uint32_t hi[16], lo[16];
        const uint64_t u2 = f2(ku, ku);
#pragma unroll
        for (int j = 0; j < 16; j += 2) {
          const float4 r4 = *reinterpret_cast<const float4*>(&sc.rs[32 * hf + 2 * j]);
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const uint64_t o = mul2(f2u(x[2 * (j + e)], x[2 * (j + e) + 1]), mul2(e ? f2(r4.z, r4.w) : f2(r4.x, r4.y), u2));
            if constexpr (BF16) hi[j + e] = pack16<false>(lo2(o), hi2(o));
            else halves(lo2(o), hi2(o), hi[j + e], lo[j + e]);
          }
        }
        tmem_st16(lane_base + kUH + 16 * hf, hi);
        if constexpr (!BF16) tmem_st16(lane_base + kUL + 16 * hf, lo);
        tmem_st_wait();
      }
      if (hf == 0) mbar_arrive(&bar.o_full);
      tc_fence_before();
      named_bar_arrive(kBarP, 288);
    }
    float* dst = nullptr;
    int64_t ld = DV;
    if (!real) {                             // N goes where the state behind this part will be
      dst = mat < 0 ? w.part_state + (seg + hv) * DK * DV + row : w.part_mat + (seg * DK + hf * (DK / 2)) * DK + mat * DV + wt;
      if (mat >= 0) ld = DK;
    } else if (c1 < w1) {
      if (part == 0) dst = w.part_state + (seg + hv) * DK * DV + row;
    } else {
      dst = c1 < chunks ? w.carry[w.parity ^ 1] + at : writes ? a.state + q.out * slot + at : nullptr;
    }
    if (dst && live && (mat < 0 || mat * DV + wt < DK)) {
#pragma unroll
      for (int j = 0; j < 16 * NB; ++j) {
        dst[2 * j * ld] = lo2(S[j]) * us.from;
        dst[(2 * j + 1) * ld] = hi2(S[j]) * us.from;
      }
    }
  } else if (wg == 2) {
    // ================================ outputs ================================
    reg_dec<DeltaRoles::kOutput>();
    constexpr int VC = DV / 8, VR = 128 / VC;                // 16-byte pieces of a token, tokens of a pass
    auto fetch = [&](int i) {                // V of chunk i on its way; rows behind the sequence's end are zeros
      if (i >= c1) return;
      const int n_ = i - c0, st = n_ % kStages, left = mat < 0 ? q.n - i * C : 0;     // (M is found without V)
      if (n_ >= kStages) wait(&bar.empty[st], (n_ / kStages - 1) & 1);
      const uint16_t* p = a.v + ((int64_t)q.t0 + i * C) * a.v_stride + h * DV + wt % VC * 8;
      const uint32_t to = smem_u32(smem + st * L::kStage + L::oV) + wt * 16;
#pragma unroll
      for (int y = 0; y < C / VR; ++y) {
        const int r = y * VR + wt / VC;
        cp_async16(to + y * 2048, r < left ? p + r * a.v_stride : a.v, r < left ? 16 : 0);
      }
      asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(&bar.v_full[st])) : "memory");
    };
    auto look = [&](int i) {                 // V's largest numbers: without signs, 16-bit numbers are in the order of their bits
      if (i >= c1) return;
      const int n_ = i - c0, st = n_ % kStages;
      wait(&bar.v_full[st], (n_ / kStages) & 1);
      constexpr int TH = 256 / DV;           // threads of a pair of dimensions (two of them write: halves of the tokens)
      const int d2 = wt % (DV / 2), part = wt / (DV / 2);
      if (TH == 2 || part < 2) {
        const uint32_t* p = reinterpret_cast<const uint32_t*>(smem + st * L::kStage + L::oV) + part * 32 * (DV / 2) + d2;
        uint32_t top = 0;
#pragma unroll
        for (int j = 0; j < 32; ++j) asm("max.u16x2 %0, %0, %1;" : "+r"(top) : "r"(p[j * (DV / 2)] & 0x7fff7fffu));
        reinterpret_cast<uint32_t*>(smem + L::oVm + st * 512)[part * 64 + d2] = top;
      }
      mbar_arrive(&bar.v_seen[st]);
    };
    fetch(c0);
    fetch(c0 + 1);
    look(c0);
    for (int i = c0; i < c1; ++i) {
      const int n_ = i - c0, st = n_ % kStages, left = min(C, q.n - i * C);
      fetch(i + 2);
      look(i + 1);
      const DeltaScalars& sc = scalars[st];
      if (!real) {
        mbar_arrive(&bar.empty[st]);
        continue;
      }
      wait(&bar.full[st], (n_ / kStages) & 1);
      wait(&bar.o_full, n_ & 1);
      tc_fence_after();
      if (live) {
        const float s1 = factors[(n_ & 1) * 256 + wt], u1 = factors[(n_ & 1) * 256 + 128 + wt];
        const uint64_t fs = f2(s1, s1), fo = f2(u1, u1);
        const int64_t step = (int64_t)hv * DV;
        uint16_t* p = a.out + (((int64_t)q.t0 + i * C) * hv + h) * DV + wt;
#pragma unroll 1
        for (int b = 0; b < C; b += 16) {
          uint32_t x[16], y[16], r[8];
          tmem_ld16(lane_base + kQS + b, x);
          tmem_ld16(lane_base + kPU + b, y);
          tmem_ld_wait();
#pragma unroll
          for (int t = 0; t < 16; t += 4) {
            const float4 oq = *reinterpret_cast<const float4*>(&sc.oq[b + t]), pq = *reinterpret_cast<const float4*>(&sc.pq[b + t]);
#pragma unroll
            for (int e = 0; e < 4; e += 2) {
              const uint64_t o = fma2(mul2(e ? f2(oq.z, oq.w) : f2(oq.x, oq.y), fs), f2u(x[t + e], x[t + e + 1]),
                                      mul2(mul2(e ? f2(pq.z, pq.w) : f2(pq.x, pq.y), fo), f2u(y[t + e], y[t + e + 1])));
              r[(t + e) / 2] = pack16<BF16>(lo2(o), hi2(o));
            }
          }
          if (b + 16 <= left) {
#pragma unroll
            for (int t = 0; t < 16; ++t, p += step) *p = (uint16_t)(t & 1 ? r[t / 2] >> 16 : r[t / 2]);
          } else {
#pragma unroll
            for (int t = 0; t < 16; ++t, p += step)
              if (b + t < left) *p = (uint16_t)(t & 1 ? r[t / 2] >> 16 : r[t / 2]);
          }
        }
      }
      tc_fence_before();
      mbar_arrive(&bar.o_empty);
      mbar_arrive(&bar.empty[st]);
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else {
    reg_dec<DeltaRoles::kProducts>();
    if (warp == 12) {
      // ================================ the chunks ================================
      if (elect_one()) {
        delta_deliver(
            c1 - c0, kStages,
            [&](int st, uint32_t parity) {
              if (mbar_wait_cycles(&bar.empty[st], parity)) return true;
              atomicOr(a.b.err, (uint32_t)DELTA_TIMEOUT);
              return false;
            },
            [&](int n_, int st) {
              uint8_t* to = smem + st * L::kStage;
              const int64_t id = base + c0 + n_ - w.first;
              mbar_arrive_expect_tx(&bar.full[st], L::kKQ + kTPBytes + (uint32_t)sizeof(DeltaScalars));
              bulk_g2s(to, w.kq + (id * a.geo.hk + h / a.geo.rep) * L::kKQ, L::kKQ, &bar.full[st]);
              bulk_g2s(to + L::oTP, w.tp + (id * hv + h) * kTPBytes, kTPBytes, &bar.full[st]);
              bulk_g2s(&scalars[st], w.sc + id * hv + h, sizeof(DeltaScalars), &bar.full[st]);
            },
            [&](int st, uint32_t parity) {
              if (!mbar_wait_cycles(&bar.full[st], parity)) atomicOr(a.b.err, (uint32_t)DELTA_TIMEOUT);
            });
      }
    } else if (warp == 14) {
      // ================================ V of chunks that grow ================================
      for (int i = c0; i < c1; ++i) {
        const int n_ = i - c0, st = n_ % kStages;
        wait(&bar.full[st], (n_ / kStages) & 1);
        wait(&bar.v_seen[st], (n_ / kStages) & 1);
        if (scalars[st].grows) {             // as large as its tokens' Z are kept (fp16 ends at 2^-24: below 2^-8 it loses bits so)
          uint32_t* p = reinterpret_cast<uint32_t*>(smem + st * L::kStage + L::oV) + lane;
          for (int t = 0; t < C; ++t) {
            const float f = power2(-scalars[st].up[t]);
#pragma unroll
            for (int e = 0; e < DV / 64; ++e, p += 32) {
              const float2 v = unpack16<BF16>(*p);
              *p = pack16<BF16>(v.x * f, v.y * f);
            }
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar.v_ready[st]);
      }
    } else if (warp == 13) {
      // ================================ products ================================
      constexpr int kSecond = BF16 ? 1 : 2;  // numbers of a pair that the outputs take
      const uint32_t id_d = idesc_f16(128, 64, 0) | 1u << 16, id64 = idesc_f16(128, 64, 0);
      const uint64_t k0 = smem_desc_sw128(smem), kc0 = k_cols_desc(smem);
      for (int i = c0; i < c1; ++i) {
        const int n_ = i - c0, st = n_ % kStages;
        const uint64_t kd = k0 + st * (L::kStage >> 4), qd = kd + (L::kMat >> 4), td = kd + (L::oTP >> 4), kc = kc0 + st * (L::kStage >> 4);
        wait(&bar.full[st], (n_ / kStages) & 1);
        // Y: first and second numbers of S against K (16 dimensions a step), a half of the dimensions as its threads have them
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          named_bar(kBarS + hf, 160);
          tc_fence_after();
          if (ok && elect_one()) {
#pragma unroll
            for (int second = 0; second < 2; ++second)
#pragma unroll
              for (int j = 0; j < DK / 32; ++j) {
                const int k = hf * (DK / 32) + j;
                umma_f16_ts(kY, kSH + 32 * (k >> 1) + 16 * second + 8 * (k & 1), kd + ((k >> 2) * 8192 >> 4) + 2 * (k & 3), id64, hf | second | j);
              }
            if (hf) umma_commit(&bar.y_full);
          }
          __syncwarp();
        }
        named_bar(kBarZ, 288);
        tc_fence_after();
        if (ok && elect_one()) {
          // tokens 16 k .. + 15 reach the tokens from 16 k on only
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint32_t id = idesc_f16(128, 64 - 16 * k, 0), z = kY + 32 * (k >> 1) + 8 * (k & 1);
            const uint32_t to = kU + 16 * k;
            const uint64_t row = td + (2048 * k >> 4) + 2 * k;
            umma_f16_ts(to, z, row, id, k != 0);
            umma_f16_ts(to, z + 16, row, id, 1);
            umma_f16_ts(to, z, row + (C * 128 >> 4), id, 1);
          }
          umma_commit(&bar.u_full);
        }
        __syncwarp();
        // Q S, while U is formed
        if (real && n_ > 0) wait(&bar.o_empty, (n_ - 1) & 1);
        tc_fence_after();
        if (real && ok && elect_one()) {
#pragma unroll
          for (int k = 0; k < DK / 16; ++k)
#pragma unroll
            for (int second = 0; second < kSecond; ++second)
              umma_f16_ts(kQS, kSH + 32 * (k >> 1) + 16 * second + 8 * (k & 1), qd + ((k >> 2) * 8192 >> 4) + 2 * (k & 3), id64, second | k);
        }
        __syncwarp();
        named_bar(kBarU, 288);
        tc_fence_after();
        if (ok && elect_one()) {
          // by halves of 64 dimensions, so that the first one's threads go on while the other's products run
#pragma unroll
          for (int hf = 0; hf < DK / 64; ++hf) {
#pragma unroll
            for (int second = 0; second < 2; ++second)
#pragma unroll
              for (int k = 0; k < 4; ++k)
                umma_f16_ts(kSH + 64 * hf, kU + 32 * (k >> 1) + 16 * second + 8 * (k & 1), kc + ((8192 * hf + 2048 * k) >> 4), id_d, second | k);
            umma_commit(&bar.d_full[hf]);
          }
          if (DK == 64) umma_commit(&bar.d_full[1]);
        }
        __syncwarp();
        if (real) named_bar(kBarP, 288);
        tc_fence_after();
        if (real && ok && elect_one()) {
          const uint64_t pd = td + (2 * C * 128 >> 4);
#pragma unroll
          for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int second = 0; second < kSecond; ++second)
              umma_f16_ts(kPU + 16 * k, (second ? kUL : kUH) + 8 * k, pd + (2048 * k >> 4) + 2 * k, idesc_f16(128, 64 - 16 * k, 0), second | k);
          umma_commit(&bar.o_full);
        }
        __syncwarp();
        if (ok && elect_one()) umma_commit(&bar.empty[st]);
        __syncwarp();
      }
      // every product has ended before the tensor memory is given back, also after a wait that gave up
      if (elect_one()) {
        umma_commit(&bar.drained);
        if (!mbar_wait_cycles(&bar.drained, 0)) atomicOr(a.b.err, (uint32_t)DELTA_TIMEOUT);
      }
      __syncwarp();
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 13) tmem_dealloc(bar.tmem, 512);
}

// The states before the parts, one from another: S_(j+1) = M_j S_j + N_j (N_j lies in S_(j+1)'s place).  A block takes some
// columns of a head's state, a thread 8 of a row; M comes in pieces of 32 of its columns, the next one on its way.
constexpr int kJoinCols = 16;
template <int DK>
struct JoinSmem {
  static constexpr int kStages = 2, kLd = 36;    // (rows of 144 bytes: eight lanes' 16 bytes meet in no bank)
  float x[DK][kJoinCols], m[kStages][DK][kLd];
};
template <int DK>
__global__ void __launch_bounds__(DK * kJoinCols / 8) join_kernel(const __grid_constant__ DeltaFwdArgs a, const __grid_constant__ DeltaWork w) {
  constexpr int PIECES = DK / 32, NS = JoinSmem<DK>::kStages;
  extern __shared__ __align__(1024) uint8_t raw[];
  JoinSmem<DK>& sm = *reinterpret_cast<JoinSmem<DK>*>(raw);
  auto& x = sm.x;
  auto& m = sm.m;
  const int s = blockIdx.z, h = blockIdx.y, hv = a.geo.hv, dv = a.geo.dv, r = threadIdx.x % DK, c = threadIdx.x / DK * 8;
  const DeltaSeq q = delta_seq(a.b, s);
  if (q.n < a.n_min || q.n > a.n_max) return;
  const int chunks = (q.n + C - 1) / C, base = delta_chunk_base(q.t0, s);
  const int w0 = max(0, w.first - base), w1 = min(chunks, w.first + w.count - base);
  if (w0 >= w1) return;
  const DeltaParts pt = delta_parts(w1 - w0, w.parts, w.front);
  if (pt.parts < 3) return;
  const int64_t seg = ((int64_t)s * w.parts + 1) * hv + h;         // of part 1; the next part's lies hv further on
  const auto state = [&](int j) { return reinterpret_cast<float4*>(w.part_state + ((seg + (int64_t)(j - 1) * hv) * DK + r) * dv + blockIdx.x * kJoinCols + c); };
  const int pieces = (pt.parts - 2) * PIECES;
  const auto bring = [&](int i) {
    const float* from = w.part_mat + (seg + (int64_t)(i / PIECES) * hv) * DK * DK + i % PIECES * 32;
#pragma unroll
    for (int e = threadIdx.x; e < DK * 8; e += DK * kJoinCols / 8)
      cp_async16(smem_u32(&m[i % NS][e >> 3][4 * (e & 7)]), from + (e >> 3) * DK + 4 * (e & 7), 16);
  };
  for (int i = 0; i < NS - 1; ++i) {
    if (i < pieces) bring(i);
    cp_async_commit();
  }
  {
    const float4* s1 = state(1);
    const float4 u = s1[0], v = s1[1];
    *reinterpret_cast<float4*>(&x[r][c]) = u;
    *reinterpret_cast<float4*>(&x[r][c + 4]) = v;
  }
  float o[8];
  float4 n0, n1;
  for (int i = 0; i < pieces; ++i) {
    if (i % PIECES == 0) {
      const float4* n = state(i / PIECES + 2);
      n0 = n[0];
      n1 = n[1];
#pragma unroll
      for (int e = 0; e < 8; ++e) o[e] = 0.f;
    }
    cp_async_wait<NS - 2>();
    __syncthreads();                   // (this piece and x are there, the one before has been read)
    if (i + NS - 1 < pieces) bring(i + NS - 1);
    cp_async_commit();                 // (one group per piece, empty ones at the end)
    const int k0 = i % PIECES * 32;
#pragma unroll
    for (int k = 0; k < 32; k += 4) {
      const float4 f = *reinterpret_cast<const float4*>(&m[i % NS][r][k]);
      const float ff[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        const float4 u = *reinterpret_cast<const float4*>(&x[k0 + k + y][c]), v = *reinterpret_cast<const float4*>(&x[k0 + k + y][c + 4]);
        o[0] += ff[y] * u.x, o[1] += ff[y] * u.y, o[2] += ff[y] * u.z, o[3] += ff[y] * u.w;
        o[4] += ff[y] * v.x, o[5] += ff[y] * v.y, o[6] += ff[y] * v.z, o[7] += ff[y] * v.w;
      }
    }
    if (i % PIECES == PIECES - 1) {
      float4* n = state(i / PIECES + 2);
      const float4 u = make_float4(n0.x + o[0], n0.y + o[1], n0.z + o[2], n0.w + o[3]);
      const float4 v = make_float4(n1.x + o[4], n1.y + o[5], n1.z + o[6], n1.w + o[7]);
      n[0] = u;
      n[1] = v;
      __syncthreads();                 // (x has been read)
      *reinterpret_cast<float4*>(&x[r][c]) = u;
      *reinterpret_cast<float4*>(&x[r][c + 4]) = v;
    }
  }
}

template <bool BF16, int DK, int DV>
cudaError_t launch(const DeltaFwdArgs& a, const DeltaWork& w, cudaStream_t s) {
  constexpr int smem = Cfg<DK, DV>::kSmem;
  static_assert(smem <= 227 * 1024, "shared memory");
  const void* fn = reinterpret_cast<const void*>(chain_kernel<BF16, DK, DV>);
  const cudaError_t e = ensure_dyn_smem(fn, smem);
  if (e != cudaSuccess) return e;
  // the roles' registers must fit what the block is launched with
  static const int regs = [fn] {
    cudaFuncAttributes at;
    return cudaFuncGetAttributes(&at, fn) == cudaSuccess ? at.numRegs : 0;
  }();
  if (regs * kThreads < DeltaRoles::Block::registers()) return cudaErrorLaunchOutOfResources;
  if (w.parts < 3) {
    chain_kernel<BF16, DK, DV><<<dim3(a.geo.hv, a.b.n_seqs), kThreads, smem, s>>>(a, w);
    return cudaGetLastError();
  }
  const cudaError_t ej = ensure_dyn_smem(reinterpret_cast<const void*>(join_kernel<DK>), sizeof(JoinSmem<DK>));
  if (ej != cudaSuccess) return ej;
  DeltaWork p = w;
  p.pass = 1;
  chain_kernel<BF16, DK, DV><<<dim3(a.geo.hv, a.b.n_seqs, delta_pass1_blocks(w.parts, DK, DV)), kThreads, smem, s>>>(a, p);
  join_kernel<DK><<<dim3(DV / kJoinCols, a.geo.hv, a.b.n_seqs), DK * kJoinCols / 8, sizeof(JoinSmem<DK>), s>>>(a, p);
  p.pass = 2;
  chain_kernel<BF16, DK, DV><<<dim3(a.geo.hv, a.b.n_seqs, w.parts - 1), kThreads, smem, s>>>(a, p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_delta_chain(const DeltaFwdArgs& a, const DeltaWork& w, cudaStream_t s) {
  const bool bf = a.geo.io == MOE_T_BF16;
#define DELTA_CHAIN(DK, DV) return bf ? launch<true, DK, DV>(a, w, s) : launch<false, DK, DV>(a, w, s)
  if (a.geo.dk == 128) {
    if (a.geo.dv == 128) DELTA_CHAIN(128, 128);
    DELTA_CHAIN(128, 64);
  }
  if (a.geo.dv == 128) DELTA_CHAIN(64, 128);
  DELTA_CHAIN(64, 64);
#undef DELTA_CHAIN
}

}  // namespace moe
