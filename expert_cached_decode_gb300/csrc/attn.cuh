// Shared by the attention kernels (attn_*.cu): the call's sequences, the cells
// and their types, and the row geometry.
#pragma once

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

// Cell j (0 <= j < max_len) of sequence s, or NULL when its page is out of range.
__device__ __forceinline__ uint8_t* cell_ptr(const AttnBatch& b, int s, int j) {
  const uint32_t pg = fdiv((uint32_t)j, b.page_div);
  const int id = b.table[(int64_t)s * b.table_pages + pg];
  if ((uint32_t)id >= (uint32_t)b.n_pages) {
    atomicOr(b.err, (uint32_t)ATTN_BAD_PAGE);
    return nullptr;
  }
  return b.cells + (int64_t)id * b.page_bytes + (int64_t)(j - (int)pg * b.page_cells) * b.cell_bytes;
}

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

// ---- launchers (one per kernel family) ----
struct AttnGeo {
  int hq, hkv, g, D, io, kv;      // g = hq / hkv
  float scale_log2;               // scale * log2(e)
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

struct AttnFwdArgs {
  AttnBatch b;
  const uint16_t* q;
  int64_t q_stride;
  uint16_t* out;
  float* lse;
  AttnGeo g;
  float* ws;                      // partial results of split items
  int32_t* meta;
  int num_sms;
};
cudaError_t launch_attn_forward(const AttnFwdArgs& a, int max_q, cudaStream_t s);

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
  int max_kv, num_sms;
};
cudaError_t launch_attn_weights(const AttnWgtArgs& a, int max_q, cudaStream_t s);

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
