// Rotation of q and k and the write of K and V cells (moe_attn_append), and
// the cells read back as values (moe_attn_read).
//
// A rotated pair (a, b) at position p becomes m (a cos f - b sin f, b cos f +
// a sin f), f = 2 pi p t_i.  The turns t_i are 64-bit fixed point (units of
// 2^-64), so p * t_i wraps to the part of a turn exactly; its top 32 bits
// (error 2^-33 turns) go through sincospi, whose argument then lies in
// [-1, 1).  A product p * t_i in 32-bit floats would be off by up to 2^-8
// radians at p = 131,071.
//
// Bound by bytes (q, k, v read, q and cells written once): 12,288 tokens of 32
// + 4 + 4 heads into 16-bit cells take 46 us, 81% of a copy's bandwidth; into
// int8 cells, with a maximum over each head vector first, 49 us (72%).  The cosines and
// sines of a token are the same for every head, so a CTA computes them once
// for its tokens (into shared memory) and its threads then take 16 elements of
// a head vector each as two 16-byte pieces that hold 8 pairs: (8c, rot/2 + 8c)
// in the half layout, (16c, 16c + 8) in the interleaved one and beyond the
// rotated part.
#include "attn.cuh"

namespace moe {

namespace {

constexpr int kThreads = 256;
constexpr int kTok = 4;               // tokens per CTA

// Code of x given 127 / max|x| (round to nearest even); a pair of floats -> bytes is left to the packer.
__device__ __forceinline__ uint32_t code4(float a, float b, float c, float d, float inv) {
  const int i0 = __float2int_rn(a * inv), i1 = __float2int_rn(b * inv), i2 = __float2int_rn(c * inv),
            i3 = __float2int_rn(d * inv);
  return (uint32_t)(i0 & 255) | (uint32_t)(i1 & 255) << 8 | (uint32_t)(i2 & 255) << 16 | (uint32_t)(i3 & 255) << 24;
}

// The larger one, or NaN if either is (fmaxf would drop it): a NaN in a head vector makes its scale NaN, and with it the
// values that are read back.
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

template <bool BF16, int D, bool I8>
__global__ void __launch_bounds__(kThreads) append_kernel(const __grid_constant__ AppendArgs a) {
  constexpr int C = D / 16;           // threads per head vector
  __shared__ float2 cs[kTok][D / 2];
  __shared__ uint8_t* cell[kTok];
  const int t0 = blockIdx.x * kTok, nt = min(kTok, a.b.n_tokens - t0), half = a.rot >> 1;
  if (threadIdx.x < nt) {             // one thread per token: its cell
    const int t = t0 + threadIdx.x, s = seq_of(a.b, t);
    uint8_t* p = nullptr;
    if (s >= 0) {
      const SeqInfo q = seq_info(a.b, s);
      const int j = q.len - q.n + (t - q.q0);
      if (j >= 0 && a.hkv) p = cell_ptr(a.b, s, j);
    }
    cell[threadIdx.x] = p;
  }
  for (int i = threadIdx.x; i < nt * half; i += kThreads) {
    const int tt = i / half, f = i - tt * half, t = t0 + tt;
    int pos;
    if (a.positions) {
      pos = a.positions[t];
    } else {
      const int s = seq_of(a.b, t);
      pos = 0;
      if (s >= 0) {
        const SeqInfo q = seq_info(a.b, s);
        pos = q.len - q.n + (t - q.q0);
      }
    }
    const uint64_t ph = (uint64_t)(int64_t)pos * a.turns[f];
    const float x = (float)(int32_t)(ph >> 32) * 4.656612873077393e-10f;   // half turns: 2^-31
    float sn, c;
    sincospif(x, &sn, &c);
    cs[tt][f] = make_float2(c * a.factor, sn * a.factor);
  }
  __syncthreads();
  const int vecs = a.hq + 2 * a.hkv, tasks = nt * vecs * C;
  // whole warps stay in the loop (the shuffles below take all 32 lanes); a lane past the end repeats the last task
  // and writes nothing
  for (int i0 = threadIdx.x & ~31; i0 < tasks; i0 += kThreads) {
    const bool live = i0 + (threadIdx.x & 31) < tasks;
    const int i = live ? i0 + (threadIdx.x & 31) : tasks - 1;
    const int c = i % C, u = i / C, tt = u / vecs, h = u - tt * vecs, t = t0 + tt;
    const bool isq = h < a.hq, isk = !isq && h < a.hq + a.hkv;
    const int hk = isq ? h : isk ? h - a.hq : h - a.hq - a.hkv;
    const uint16_t* src = isq ? a.q + t * a.q_stride : isk ? a.k + t * a.k_stride : a.v + t * a.v_stride;
    src += hk * D;
    const bool rotated = (isq || isk) && 16 * c < a.rot;
    const bool halves = rotated && !a.interleaved;
    const int o1 = halves ? 8 * c : 16 * c, o2 = halves ? half + 8 * c : 16 * c + 8;
    const uint4 r1 = *reinterpret_cast<const uint4*>(src + o1), r2 = *reinterpret_cast<const uint4*>(src + o2);
    float x[16];
    {
      const uint32_t w[8] = {r1.x, r1.y, r1.z, r1.w, r2.x, r2.y, r2.z, r2.w};
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float2 f = Half16<BF16>::unpack(w[e]);
        x[2 * e] = f.x;
        x[2 * e + 1] = f.y;
      }
    }
    if (rotated) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float2 f = cs[tt][8 * c + e];
        // the pair: (e, 8 + e) in the half layout, (2e, 2e + 1) in the interleaved one
        if (halves) {
          const float p = x[e], r = x[8 + e];
          x[e] = p * f.x - r * f.y;
          x[8 + e] = r * f.x + p * f.y;
        } else {
          const float p = x[2 * e], r = x[2 * e + 1];
          x[2 * e] = p * f.x - r * f.y;
          x[2 * e + 1] = r * f.x + p * f.y;
        }
      }
    }
    uint8_t* dst = isq ? nullptr : cell[tt];
    if (isq || !I8) {
      uint32_t w[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) w[e] = Half16<BF16>::pack(x[2 * e], x[2 * e + 1]);
      uint16_t* o = isq ? a.q_out + ((int64_t)t * a.hq + hk) * D
                        : reinterpret_cast<uint16_t*>(dst) + ((isk ? 0 : a.hkv) + hk) * D;
      if (live && (isq || dst)) {
        *reinterpret_cast<uint4*>(o + o1) = make_uint4(w[0], w[1], w[2], w[3]);
        *reinterpret_cast<uint4*>(o + o2) = make_uint4(w[4], w[5], w[6], w[7]);
      }
    }
    if (I8) {
      float top = 0.f;
#pragma unroll
      for (int e = 0; e < 16; ++e) top = max_nan(top, fabsf(x[e]));
      // the C threads of a head vector are neighbours (a warp's tasks start at a multiple of C)
#pragma unroll
      for (int o = 1; o < C; o <<= 1) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
      if (live && !isq && dst) {
        // 127 / top passes fp32's range where top is below 2^-121: such vectors (bf16 holds them) are lifted by 2^100 first
        const bool tiny = top < 0x1p-100f;
        if (tiny) {
#pragma unroll
          for (int e = 0; e < 16; ++e) x[e] *= 0x1p100f;
        }
        const float inv = top > 0.f ? 127.f / (tiny ? top * 0x1p100f : top) : 0.f;
        uint8_t* o = dst + ((isk ? 0 : a.hkv) + hk) * D;
        *reinterpret_cast<uint2*>(o + o1) =
            make_uint2(code4(x[0], x[1], x[2], x[3], inv), code4(x[4], x[5], x[6], x[7], inv));
        *reinterpret_cast<uint2*>(o + o2) =
            make_uint2(code4(x[8], x[9], x[10], x[11], inv), code4(x[12], x[13], x[14], x[15], inv));
        if (c == 0) reinterpret_cast<float*>(dst + 2 * a.hkv * D)[(isk ? 0 : a.hkv) + hk] = top / 127.f;
      }
    }
  }
}

// One thread takes 8 elements of a head vector.
template <bool BF16, int D, bool I8>
__global__ void __launch_bounds__(kThreads) read_kernel(const AttnBatch b, int hkv, uint16_t* k_out, uint16_t* v_out) {
  constexpr int C = D / 8;
  const int per = 2 * hkv * C;
  const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  const int t = (int)(i / per), r = (int)(i - (int64_t)t * per);
  if (t >= b.n_tokens) return;
  const int s = seq_of(b, t);
  if (s < 0) return;
  const SeqInfo q = seq_info(b, s);
  const int j = q.len - q.n + (t - q.q0);
  if (j < 0) return;
  const uint8_t* cell = cell_ptr(b, s, j);
  if (!cell) return;
  const int h = r / C, c = r - h * C;          // h: K heads, then V heads
  uint16_t* dst = (h < hkv ? k_out + ((int64_t)t * hkv + h) * D : v_out + ((int64_t)t * hkv + h - hkv) * D) + 8 * c;
  if (!I8) {
    *reinterpret_cast<uint4*>(dst) = *reinterpret_cast<const uint4*>(cell + ((size_t)h * D + 8 * c) * 2);
  } else {
    const uint2 w = *reinterpret_cast<const uint2*>(cell + (size_t)h * D + 8 * c);
    const float sc = reinterpret_cast<const float*>(cell + (size_t)2 * hkv * D)[h];
    uint32_t o[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t u = (e < 2 ? w.x : w.y) >> (16 * (e & 1));
      o[e] = Half16<BF16>::pack((float)(int8_t)(u & 255) * sc, (float)(int8_t)(u >> 8 & 255) * sc);
    }
    *reinterpret_cast<uint4*>(dst) = make_uint4(o[0], o[1], o[2], o[3]);
  }
}

}  // namespace

#define ATTN_BY_TYPE(CALL)                                             \
  do {                                                                 \
    const bool bf = g.io == MOE_T_BF16, i8 = g.kv == MOE_T_I8;         \
    if (g.D == 128) {                                                  \
      if (bf) { if (i8) CALL(true, 128, true); else CALL(true, 128, false); }      \
      else { if (i8) CALL(false, 128, true); else CALL(false, 128, false); }       \
    } else {                                                           \
      if (bf) { if (i8) CALL(true, 64, true); else CALL(true, 64, false); }        \
      else { if (i8) CALL(false, 64, true); else CALL(false, 64, false); }         \
    }                                                                  \
  } while (0)

cudaError_t launch_attn_append(const AppendArgs& a, const AttnGeo& g, cudaStream_t s) {
  const int grid = (a.b.n_tokens + kTok - 1) / kTok;
#define CALL(BF, DD, I) append_kernel<BF, DD, I><<<grid, kThreads, 0, s>>>(a)
  ATTN_BY_TYPE(CALL);
#undef CALL
  return cudaGetLastError();
}

cudaError_t launch_attn_read(const AttnBatch& b, const AttnGeo& g, uint16_t* k_out, uint16_t* v_out, cudaStream_t s) {
  const int64_t n = (int64_t)b.n_tokens * 2 * g.hkv * (g.D / 8);
  const int grid = (int)((n + kThreads - 1) / kThreads);
#define CALL(BF, DD, I) read_kernel<BF, DD, I><<<grid, kThreads, 0, s>>>(b, g.hkv, k_out, v_out)
  ATTN_BY_TYPE(CALL);
#undef CALL
  return cudaGetLastError();
}

}  // namespace moe
