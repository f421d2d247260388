// Host side of the attention entry points (moe_attn_*): argument checks, the
// handle and its work space, launches.
#include <cmath>
#include <cstring>
#include <mutex>
#include <new>

#include "attn.cuh"

using namespace moe;

namespace {

constexpr int kMaxSeqs = 4096;
constexpr int kFewRows = 32;          // rows per K/V head that attn_rows.cu takes at a time
constexpr int kFewWeightRows = 48;    // that attn_weights.cu takes where there are many cells
constexpr int kMaxTokens = 1 << 24   /* times 32 heads still fits 31 bits */;

}  // namespace

struct moe_attn {
  AttnGeo g{};
  int device = 0, num_sms = 0;
  int page_cells = 0, cell_bytes = 0, window = 0, rot = 0, interleaved = 0;
  float factor = 1.f;
  uint64_t* turns = nullptr;
  float* ws = nullptr;
  AttnCut* cuts = nullptr;
  int64_t ws_slot = 0;
  uint32_t* err = nullptr;
  // Held while a call that uses the work space enqueues its kernels: another host thread's, put between them on the same
  // stream, would replace what the joining kernel is to read.
  std::mutex enqueue;
};

static bool mis16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }

static moe_status cuda_fail(cudaError_t e, const char* what) {
  cudaGetLastError();
  return set_last_error(e == cudaErrorMemoryAllocation ? MOE_ERR_OOM : MOE_ERR_CUDA, "%s: %s", what,
                        cudaGetErrorString(e));
}

extern "C" moe_status moe_attn_create(const moe_attn_desc* D, moe_attn** out) {
  if (!D || !out) return set_last_error(MOE_ERR_INVALID_ARG, "NULL desc or out");
  *out = nullptr;
  if (D->n_kv_heads < 1 || D->n_kv_heads > 64 || D->n_q_heads < 1 || D->n_q_heads % D->n_kv_heads != 0 ||
      D->n_q_heads / D->n_kv_heads > 32)
    return set_last_error(MOE_ERR_INVALID_ARG,
                          "heads: n_kv_heads in 1..64, n_q_heads a multiple of it, at most 32 per K/V head");
  if (D->head_dim != 64 && D->head_dim != 128)
    return set_last_error(MOE_ERR_UNIMPLEMENTED, "head_dim must be 64 or 128");
  if (D->page_cells < 1 || D->page_cells > 65536)
    return set_last_error(MOE_ERR_INVALID_ARG, "page_cells must be in 1..65536");
  if (D->io_type != MOE_T_BF16 && D->io_type != MOE_T_F16)
    return set_last_error(MOE_ERR_INVALID_ARG, "io_type must be MOE_T_BF16 or MOE_T_F16");
  if (D->kv_type != D->io_type && D->kv_type != MOE_T_I8)
    return set_last_error(MOE_ERR_INVALID_ARG, "kv_type must be io_type or MOE_T_I8");
  const int vec = 2 * D->n_kv_heads * D->head_dim;
  const int least = ((D->kv_type == MOE_T_I8 ? vec + 8 * D->n_kv_heads : 2 * vec) + 15) / 16 * 16;
  const int cb = D->cell_bytes ? D->cell_bytes : least;
  if (cb < least || cb % 16 != 0 || cb > (1 << 20))
    return set_last_error(MOE_ERR_INVALID_ARG, "cell_bytes must be a multiple of 16 and at least %d", least);
  if (D->window < 0) return set_last_error(MOE_ERR_INVALID_ARG, "window < 0");
  if (!std::isfinite(D->scale) || D->scale < 0.f)
    return set_last_error(MOE_ERR_INVALID_ARG, "scale must be finite and not negative");
  if (D->rot_dim < 0 || D->rot_dim > D->head_dim || D->rot_dim % 16 != 0)
    return set_last_error(MOE_ERR_INVALID_ARG, "rot_dim must be a multiple of 16 in [0, head_dim]");
  if (D->rot_dim && (!D->rot_turns || !std::isfinite(D->rot_factor)))
    return set_last_error(MOE_ERR_INVALID_ARG, "rot_turns is NULL or rot_factor not finite");
  moe_attn* a = new (std::nothrow) moe_attn();
  if (!a) return set_last_error(MOE_ERR_OOM, "handle");
  a->g.hq = D->n_q_heads;
  a->g.hkv = D->n_kv_heads;
  a->g.g = D->n_q_heads / D->n_kv_heads;
  a->g.gdiv = make_fastdiv((uint32_t)a->g.g);
  a->g.D = D->head_dim;
  a->g.io = D->io_type;
  a->g.kv = D->kv_type;
  const float scale = D->scale > 0.f ? D->scale : 1.f / std::sqrt((float)D->head_dim);
  a->g.scale_log2 = scale * 1.4426950408889634f;
  a->page_cells = D->page_cells;
  a->cell_bytes = cb;
  a->window = D->window;
  a->rot = D->rot_dim;
  a->interleaved = D->rot_interleaved != 0;
  a->factor = D->rot_factor;
  auto fail_destroy = [&](moe_status st) {
    moe_attn_destroy(a);
    return st;
  };
  cudaError_t e = cudaGetDevice(&a->device);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&a->num_sms, cudaDevAttrMultiProcessorCount, a->device);
  if (e != cudaSuccess) return fail_destroy(cuda_fail(e, "device query"));
  e = cudaMalloc(&a->err, sizeof(uint32_t));
  if (e == cudaSuccess) e = cudaMemset(a->err, 0, sizeof(uint32_t));
  if (e == cudaSuccess && a->rot) {
    e = cudaMalloc(&a->turns, a->rot / 2 * sizeof(uint64_t));
    if (e == cudaSuccess)
      e = cudaMemcpy(a->turns, D->rot_turns, a->rot / 2 * sizeof(uint64_t), cudaMemcpyHostToDevice);
  }
  a->ws_slot = attn_ws_slot(a->g.D);
  if (e == cudaSuccess) e = cudaMalloc(&a->ws, (size_t)a->num_sms * 4 * a->ws_slot * sizeof(float));
  if (e == cudaSuccess) e = cudaMalloc(&a->cuts, 2 * a->num_sms * sizeof(AttnCut));
  if (e == cudaSuccess) e = cudaDeviceSynchronize();
  if (e != cudaSuccess) return fail_destroy(cuda_fail(e, "attention handle"));
  *out = a;
  return MOE_OK;
}

// Checks what every call takes; fills the kernels' view.
static moe_status take_batch(moe_attn* a, const moe_attn_batch* B, bool need_q, AttnBatch* b) {
  if (!a || !B) return set_last_error(MOE_ERR_INVALID_ARG, "NULL handle or batch");
  if (B->n_seqs < 0 || B->n_seqs > kMaxSeqs)
    return set_last_error(MOE_ERR_INVALID_ARG, "n_seqs must be in [0, %d]", kMaxSeqs);
  if (B->n_tokens < 0 || B->n_tokens > kMaxTokens)
    return set_last_error(MOE_ERR_INVALID_ARG, "n_tokens must be in [0, %d]", kMaxTokens);
  if (B->table_pages < 0 || (int64_t)B->table_pages * a->page_cells >= 1 << 30)
    return set_last_error(MOE_ERR_INVALID_ARG, "table_pages * page_cells must be in [0, 2^30)");
  if (B->n_pages < 0 || B->n_pages > INT32_MAX || B->n_pages * a->page_cells > INT32_MAX)
    return set_last_error(MOE_ERR_INVALID_ARG, "n_pages * page_cells must be in [0, 2^31)");
  if (B->n_seqs > 0 && (!B->kv_lens || (need_q && !B->cu_q)))
    return set_last_error(MOE_ERR_INVALID_ARG, "NULL kv_lens or cu_q");
  if (B->n_seqs > 0 && B->table_pages > 0 && !B->block_table)
    return set_last_error(MOE_ERR_INVALID_ARG, "NULL block_table");
  if (B->n_pages > 0 && !B->cells) return set_last_error(MOE_ERR_INVALID_ARG, "NULL cells");
  if (mis16(B->cells)) return set_last_error(MOE_ERR_INVALID_ARG, "cells not 16-byte aligned");
  b->cells = static_cast<uint8_t*>(B->cells);
  b->table = B->block_table;
  b->kv_lens = B->kv_lens;
  b->cu_q = B->cu_q;
  b->err = a->err;
  b->page_bytes = (int64_t)a->page_cells * a->cell_bytes;
  b->cell_bytes = a->cell_bytes;
  b->page_cells = a->page_cells;
  b->n_pages = (int32_t)B->n_pages;
  b->n_seqs = B->n_seqs;
  b->table_pages = B->table_pages;
  b->n_tokens = B->n_tokens;
  b->max_len = B->table_pages * a->page_cells;
  b->window = a->window < b->max_len ? a->window : 0;
  b->page_div = make_fastdiv((uint32_t)a->page_cells);
  return MOE_OK;
}

static moe_status take_rows(const void* p, int64_t stride, int heads, int D, const char* what) {
  if (!p) return set_last_error(MOE_ERR_INVALID_ARG, "NULL %s", what);
  if (mis16(p) || stride % 8 != 0 || stride < (int64_t)heads * D)
    return set_last_error(MOE_ERR_INVALID_ARG,
                          "%s must be 16-byte aligned, its stride a multiple of 8 elements and at least %d", what,
                          heads * D);
  return MOE_OK;
}

#define ATTN_CHECK(call)                    \
  do {                                      \
    const moe_status st_ = (call);          \
    if (st_ != MOE_OK) return st_;          \
  } while (0)

static moe_status launched(cudaError_t e, const char* what) { return e == cudaSuccess ? MOE_OK : cuda_fail(e, what); }

extern "C" moe_status moe_attn_append(moe_attn* a, const moe_attn_batch* B, const void* q, int64_t q_stride,
                                      const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                                      const int32_t* positions, void* q_out, void* stream) {
  AppendArgs x{};
  ATTN_CHECK(take_batch(a, B, true, &x.b));
  if ((q == nullptr) != (q_out == nullptr)) return set_last_error(MOE_ERR_INVALID_ARG, "q and q_out go together");
  if ((k == nullptr) != (v == nullptr)) return set_last_error(MOE_ERR_INVALID_ARG, "k and v go together");
  if (B->n_tokens == 0 || B->n_seqs == 0) return MOE_OK;
  if (!q && !k) return set_last_error(MOE_ERR_INVALID_ARG, "neither q nor k");
  if (q) {
    ATTN_CHECK(take_rows(q, q_stride, a->g.hq, a->g.D, "q"));
    if (mis16(q_out)) return set_last_error(MOE_ERR_INVALID_ARG, "q_out not 16-byte aligned");
    if (q == q_out && q_stride != (int64_t)a->g.hq * a->g.D)
      return set_last_error(MOE_ERR_INVALID_ARG, "q_out may be q only when q is contiguous");
  }
  if (k) {
    ATTN_CHECK(take_rows(k, k_stride, a->g.hkv, a->g.D, "k"));
    ATTN_CHECK(take_rows(v, v_stride, a->g.hkv, a->g.D, "v"));
  }
  x.q = static_cast<const uint16_t*>(q);
  x.k = static_cast<const uint16_t*>(k);
  x.v = static_cast<const uint16_t*>(v);
  x.q_out = static_cast<uint16_t*>(q_out);
  x.q_stride = q_stride;
  x.k_stride = k_stride;
  x.v_stride = v_stride;
  x.positions = positions;
  x.turns = a->turns;
  x.hq = q ? a->g.hq : 0;
  x.hkv = k ? a->g.hkv : 0;
  x.rot = a->rot;
  x.interleaved = a->interleaved;
  x.factor = a->factor;
  return launched(launch_attn_append(x, a->g, static_cast<cudaStream_t>(stream)), "moe_attn_append");
}

extern "C" moe_status moe_attn_read(moe_attn* a, const moe_attn_batch* B, void* k_out, void* v_out, void* stream) {
  AttnBatch b;
  ATTN_CHECK(take_batch(a, B, true, &b));
  if (B->n_tokens == 0 || B->n_seqs == 0) return MOE_OK;
  ATTN_CHECK(take_rows(k_out, (int64_t)a->g.hkv * a->g.D, a->g.hkv, a->g.D, "k_out"));
  ATTN_CHECK(take_rows(v_out, (int64_t)a->g.hkv * a->g.D, a->g.hkv, a->g.D, "v_out"));
  return launched(launch_attn_read(b, a->g, static_cast<uint16_t*>(k_out), static_cast<uint16_t*>(v_out),
                                   static_cast<cudaStream_t>(stream)),
                  "moe_attn_read");
}

extern "C" moe_status moe_attn_forward(moe_attn* a, const moe_attn_batch* B, const void* q, int64_t q_stride, void* out,
                                       float* lse, void* stream) {
  AttnFwdArgs x{};
  ATTN_CHECK(take_batch(a, B, true, &x.b));
  if (B->n_tokens == 0 || B->n_seqs == 0) return MOE_OK;
  ATTN_CHECK(take_rows(q, q_stride, a->g.hq, a->g.D, "q"));
  ATTN_CHECK(take_rows(out, (int64_t)a->g.hq * a->g.D, a->g.hq, a->g.D, "out"));
  x.q = static_cast<const uint16_t*>(q);
  x.q_stride = q_stride;
  x.out = static_cast<uint16_t*>(out);
  x.lse = lse;
  x.g = a->g;
  x.ws = a->ws;
  x.cuts = a->cuts;
  x.ws_slot = a->ws_slot;
  x.num_sms = a->num_sms;
  const int max_q = B->max_q > 0 && B->max_q < B->n_tokens ? B->max_q : B->n_tokens;
  // Few rows per K/V head: bound by the cells' bytes, on mma.sync; more: on the tensor memory's products.  32 rows of
  // eight sequences, first and second kernel: 19 and 26 us over 1,000 int8 cells, 122 and 121 over 32,768, in bf16 18 and
  // 23, 112 and 96, at D = 64 over 32,768 59 and 79; 40 rows, as two row tiles that read the cells twice, over 8,192 to
  // 32,768 int8 cells 125 and 72.  So the limit by rows alone costs 17 to 32 rows over long 16-bit caches at D = 128 up to
  // 16 us of 112; it fits short caches, D = 64 and int8 cells.  A call that may have sequences of both kinds runs both kernels, each
  // on its own, the second starting as the first ends; where every sequence has max_q tokens one is enough.
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  std::lock_guard<std::mutex> lock(a->enqueue);
  x.rows_min = 0;
  x.rows_max = INT32_MAX;
  const bool many = (int64_t)max_q * a->g.g > kFewRows;
  if (!many) return launched(launch_attn_rows(x, max_q, true, st), "moe_attn_forward");
  const bool both = B->n_seqs > 1 && (int64_t)B->n_seqs * max_q != B->n_tokens;
  // Pages that are cut into boxes of at least 8 rows (the swizzle's period) that divide a tile of 128 cells are copied
  // by TMA; the tensor map's rows are 32-bit coordinates, and a row's stride is below 2^40.
  CUtensorMap map{};
  int box = 0;
  if (B->n_pages > 0) {
    box = a->page_cells & -a->page_cells;          // largest power of two that divides the page
    box = box > 128 ? 128 : box < 8 ? 0 : box;
    const int64_t rows = B->n_pages * (int64_t)a->page_cells;
    if (box)
      ATTN_CHECK(a->g.kv == MOE_T_I8
                     ? make_tmap_2d_bytes(&map, x.b.cells, rows, a->cell_bytes, a->g.D, box)
                     : make_tmap_2d(&map, x.b.cells, rows, a->cell_bytes / 2, box, a->g.io == MOE_T_BF16));
  }
  if (!both) return launched(launch_attn_chunk(x, map, box, max_q, false, st), "moe_attn_forward");
  AttnFwdArgs few = x;
  few.rows_max = kFewRows;
  few.ws = a->ws + (int64_t)a->num_sms * 2 * a->ws_slot;
  few.cuts = a->cuts + a->num_sms;
  x.rows_min = kFewRows;
  cudaError_t e = launch_attn_rows(few, kFewRows, false, st);
  if (e == cudaSuccess) e = launch_attn_chunk(x, map, box, max_q, true, st);
  if (e == cudaSuccess) e = launch_attn_join(few, 32, st);
  return launched(e, "moe_attn_forward");
}

extern "C" moe_status moe_attn_weights(moe_attn* a, const moe_attn_batch* B, const void* q, int64_t q_stride,
                                       const float* lse, const float* acc_in, float* acc_out, int64_t acc_stride,
                                       float decay, void* stream) {
  AttnWgtArgs x{};
  ATTN_CHECK(take_batch(a, B, true, &x.b));
  if (B->n_seqs == 0) return MOE_OK;
  if (!acc_out) return set_last_error(MOE_ERR_INVALID_ARG, "NULL acc_out");
  if (B->n_tokens > 0) {
    ATTN_CHECK(take_rows(q, q_stride, a->g.hq, a->g.D, "q"));
    if (!lse) return set_last_error(MOE_ERR_INVALID_ARG, "NULL lse");
  }
  x.max_kv = B->max_kv > 0 && B->max_kv < x.b.max_len ? B->max_kv : x.b.max_len;
  if (acc_stride < x.max_kv)
    return set_last_error(MOE_ERR_INVALID_ARG, "acc_stride %lld is below the longest sequence's %d cells",
                          (long long)acc_stride, x.max_kv);
  if (x.max_kv == 0) return MOE_OK;
  x.q = static_cast<const uint16_t*>(q);
  x.q_stride = q_stride;
  x.lse = lse;
  x.acc_in = acc_in;
  x.acc_out = acc_out;
  x.acc_stride = acc_stride;
  x.decay = decay;
  x.g = a->g;
  x.ws = a->ws;
  x.cuts = a->cuts;
  x.ws_slot = a->ws_slot;
  x.num_sms = a->num_sms;
  const int max_q = B->max_q > 0 && B->max_q < B->n_tokens ? B->max_q : B->n_tokens;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  std::lock_guard<std::mutex> lock(a->enqueue);
  // Few rows: a warp takes 64 cells for all rows; more: on the tensor memory's products.  Up to 32 rows the first is
  // faster over every length (32 rows of eight sequences, first and second: 17 and 18 us over 1,000 int8 cells, 82 and 144
  // over 32,768).  33 to 48 rows are, where the cells keep all its warps busy (40 rows over 32,768: int8 115 and 144, bf16
  // 93 and 138, at D = 64 76 and 73, 63 and 82; over 1,000: 25 and 18); 64 rows are not (155 and 144).
  const int64_t rows = (int64_t)max_q * a->g.g;
  const bool busy = (int64_t)B->n_seqs * x.max_kv >= (int64_t)a->num_sms * 8 * 64;
  if (rows <= (busy ? kFewWeightRows : kFewRows))
    return launched(launch_attn_weights_rows(x, max_q, st), "moe_attn_weights");
  // query tiles of kWeightQRows rows are boxes of whole tokens where the heads of a group divide them
  CUtensorMap map{};
  const int tma = kWeightQRows % a->g.g == 0 && B->n_tokens > 0;
  if (tma)
    ATTN_CHECK(make_tmap_rows(&map, q, B->n_tokens, q_stride, a->g.hq, a->g.D, kWeightQRows / a->g.g, a->g.g,
                              a->g.io == MOE_T_BF16));
  return launched(launch_attn_weights_chunk(x, map, tma, st), "moe_attn_weights");
}

extern "C" moe_status moe_attn_evict(moe_attn* a, const moe_attn_batch* B, const float* acc, int64_t acc_stride,
                                     int32_t budget, int32_t recent, const int32_t* new_table, int32_t new_table_pages,
                                     int32_t* keep, int32_t* new_lens, float* acc_out, void* stream) {
  EvictArgs x{};
  ATTN_CHECK(take_batch(a, B, false, &x.b));
  if (budget < 1 || recent < 0 || recent > budget)
    return set_last_error(MOE_ERR_INVALID_ARG, "budget must be positive and recent in [0, budget]");
  if (new_table_pages < 0 || (int64_t)new_table_pages * a->page_cells < budget ||
      (int64_t)new_table_pages * a->page_cells > INT32_MAX)
    return set_last_error(MOE_ERR_INVALID_ARG, "a row of the new table must hold budget cells (and less than 2^31)");
  if (B->n_seqs == 0) return MOE_OK;
  if (!acc || !new_table || !keep || !new_lens || !acc_out) return set_last_error(MOE_ERR_INVALID_ARG, "NULL array");
  if (acc_stride < 0) return set_last_error(MOE_ERR_INVALID_ARG, "acc_stride < 0");
  x.acc = acc;
  x.acc_stride = acc_stride;
  x.budget = budget;
  x.recent = recent;
  x.new_table = new_table;
  x.new_table_pages = new_table_pages;
  x.keep = keep;
  x.new_lens = new_lens;
  x.acc_out = acc_out;
  x.num_sms = a->num_sms;
  return launched(launch_attn_evict(x, static_cast<cudaStream_t>(stream)), "moe_attn_evict");
}

extern "C" moe_status moe_attn_sync(moe_attn* a) {
  if (!a) return set_last_error(MOE_ERR_INVALID_ARG, "NULL handle");
  uint32_t err = 0;
  cudaError_t e = cudaDeviceSynchronize();
  if (e == cudaSuccess) e = cudaMemcpy(&err, a->err, sizeof(err), cudaMemcpyDeviceToHost);
  if (e == cudaSuccess && err) e = cudaMemset(a->err, 0, sizeof(err));
  if (e != cudaSuccess) return cuda_fail(e, "moe_attn_sync");
  if (err & ATTN_TIMEOUT) return set_last_error(MOE_ERR_TIMEOUT, "a device-side wait of an attention call gave up");
  if (err)
    return set_last_error(MOE_ERR_INVALID_ARG, "a call found %s%s%s out of range on the GPU (left out there)",
                          err & ATTN_BAD_PAGE ? "a page id" : "", (err & 3u) == 3u ? " and " : "",
                          err & ATTN_BAD_LEN ? "a length or an offset" : "");
  return MOE_OK;
}

extern "C" void moe_attn_destroy(moe_attn* a) {
  if (!a) return;
  if (a->err || a->turns || a->ws) cudaDeviceSynchronize();
  if (a->ws) cudaFree(a->ws);
  if (a->cuts) cudaFree(a->cuts);
  if (a->turns) cudaFree(a->turns);
  if (a->err) cudaFree(a->err);
  cudaGetLastError();
  delete a;
}
