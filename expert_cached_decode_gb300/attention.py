"""Python binding of the attention over a paged cache (moe_attn_*).

PyTorch supplies device memory and streams only.  Tensors keep their own
strides from token to token (slices of a fused projection work); a token's
heads have to be contiguous.  Every call is asynchronous on `stream` (default:
the current stream); `moe_attn_sync` reports values that were out of range on
the GPU.
"""

import ctypes
import math
import struct

import numpy as np
import torch

from . import _abi
from ._abi import MoeAttnBatch, MoeAttnDesc, check

_BATCH = struct.Struct("PqPPPiiiii4x")        # MoeAttnBatch
assert _BATCH.size == ctypes.sizeof(MoeAttnBatch)


def _current_stream(device):
    return torch.cuda.current_stream(device).cuda_stream


# the same handle without the Stream object around it, where torch has it (as 2.9 and 2.11 do)
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _current_stream)

_TYPES = {torch.bfloat16: _abi.MOE_T_BF16, torch.float16: _abi.MOE_T_F16, torch.int8: _abi.MOE_T_I8}


class Rope:
    """Frequencies of a rotary position embedding: `turns` (uint64, turns per
    position of each pair in units of 2^-64) and the factor on cosine and sine.

    Pair i of rot_dim/2 turns by base^(-2i/rot_dim) radians per position, and
    with `scaling`, for a context `factor` times longer than original_len:
      "linear": that divided by factor (positions interpolated);
      "ntk":    the base raised to base * factor^(rot_dim/(rot_dim-2)), which
                leaves the first pair as it is and divides the last by factor;
      "yarn":   pairs that make more than beta_fast turns over original_len
                stay, those below beta_slow are divided by factor, a ramp over
                the pairs between; cosine and sine times 0.1 ln(factor) + 1.
    """

    def __init__(self, rot_dim, base=10000.0, interleaved=False, scaling="none", factor=1.0, original_len=4096,
                 beta_fast=32.0, beta_slow=1.0):
        if rot_dim < 0 or rot_dim % 16 != 0:
            raise ValueError("rot_dim must be a non-negative multiple of 16")
        if scaling not in ("none", "linear", "ntk", "yarn"):
            raise ValueError(f"unknown scaling {scaling!r}")
        if not base > 1.0 or not factor > 0.0:
            raise ValueError("base must be above 1 and factor positive")
        i = np.arange(rot_dim // 2, dtype=np.float64)
        if scaling == "ntk" and rot_dim:
            base = base * factor ** (rot_dim / (rot_dim - 2))
        f = base ** (-2.0 * i / max(rot_dim, 1))
        if scaling == "linear":
            f = f / factor
        self.factor = 1.0
        if scaling == "yarn":
            pair_of = lambda turns: rot_dim * math.log(original_len / (turns * 2 * math.pi)) / (2 * math.log(base))
            low = max(0, math.floor(pair_of(beta_fast)))
            high = min(rot_dim - 1, math.ceil(pair_of(beta_slow)))
            ramp = np.clip((i - low) / max(high - low, 1e-3), 0.0, 1.0)
            f = f * (1.0 - ramp) + f / factor * ramp
            self.factor = 0.1 * math.log(factor) + 1.0
        turns = np.mod(f / (2 * math.pi), 1.0)
        self.turns = np.minimum(np.round(turns * 2.0 ** 64), 2.0 ** 64 - 2048).astype(np.uint64)
        self.rot_dim, self.interleaved = rot_dim, bool(interleaved)


def kv_cell_bytes(n_kv_heads, head_dim, kv_dtype):
    """The least size of a cell, a multiple of 16 bytes."""
    vec = 2 * n_kv_heads * head_dim
    n = vec + 8 * n_kv_heads if kv_dtype == torch.int8 else 2 * vec
    return (n + 15) // 16 * 16


class PagedAttention:
    """One handle of moe_attn_*: a head layout, a cell format and the work
    space of its calls.  Calls on one handle must not overlap on the GPU; host
    threads that use one stream may share it.

    cells:    [n_pages, page_cells, cell_bytes] uint8 (device)
    cu_q:     [n_seqs + 1] int32 offsets of each sequence's new tokens
    kv_lens:  [n_seqs] int32 cells per sequence, the new tokens included
    table:    [n_seqs, pages] int32 page ids
    q:        [n_tokens, n_q_heads, head_dim]
    """

    def __init__(self, n_q_heads, n_kv_heads, head_dim, page_cells, kv_dtype=torch.bfloat16, dtype=torch.bfloat16,
                 cell_bytes=0, scale=0.0, window=0, rope=None):
        if dtype not in (torch.bfloat16, torch.float16):
            raise ValueError("dtype must be bfloat16 or float16")
        if kv_dtype not in (dtype, torch.int8):
            raise ValueError("kv_dtype must be dtype or int8")
        self._lib = _abi.load()
        self.attn = None
        turns = None if rope is None or not rope.rot_dim else np.ascontiguousarray(rope.turns)
        desc = MoeAttnDesc(n_q_heads=n_q_heads, n_kv_heads=n_kv_heads, head_dim=head_dim, page_cells=page_cells,
                           cell_bytes=cell_bytes, io_type=_TYPES[dtype], kv_type=_TYPES[kv_dtype], window=window,
                           scale=scale, rot_dim=0 if turns is None else rope.rot_dim,
                           rot_interleaved=0 if rope is None else int(rope.interleaved),
                           rot_factor=1.0 if rope is None else rope.factor,
                           rot_turns=None if turns is None else turns.ctypes.data)
        h = ctypes.c_void_p()
        check(self._lib.moe_attn_create(ctypes.byref(desc), ctypes.byref(h)), "moe_attn_create")
        self.attn = h
        self.n_q_heads, self.n_kv_heads, self.head_dim = n_q_heads, n_kv_heads, head_dim
        self.page_cells, self.dtype, self.kv_dtype, self.window = page_cells, dtype, kv_dtype, window
        self.cell_bytes = cell_bytes or kv_cell_bytes(n_kv_heads, head_dim, kv_dtype)

    # --- arguments --------------------------------------------------------------
    # (Small calls are over in some 10 us on the GPU, so the checks below are kept to a few attribute reads each.)
    def _fill(self, cells, kv_lens, table, cu_q, n_tokens, max_q, max_kv):
        """The call's batch.  A new one for every call: the library reads it while other threads may run, and another
        thread's call must not change it meanwhile (0.15 us more than one kept on the handle)."""
        shape = cells.shape
        if len(shape) != 3 or shape[1] != self.page_cells or shape[2] != self.cell_bytes or not cells.is_contiguous():
            raise ValueError(f"cells must be contiguous [n_pages, {self.page_cells}, {self.cell_bytes}]")
        if cells.dtype != torch.uint8 or not cells.is_cuda:
            raise ValueError("cells must be a uint8 device tensor")
        n = kv_lens.shape[0]
        return ctypes.byref(MoeAttnBatch.from_buffer_copy(_BATCH.pack(
            cells.data_ptr(), shape[0], self._ints(table, "table", n, 2), self._ints(kv_lens, "kv_lens", n),
            0 if cu_q is None else self._ints(cu_q, "cu_q", n + 1), n, table.shape[1], n_tokens, max_q or 0, max_kv or 0)))

    @staticmethod
    def _ints(t, what, n, dims=1):
        shape = t.shape
        if t.dtype != torch.int32 or len(shape) != dims or shape[0] != n or not t.is_contiguous() or not t.is_cuda:
            raise ValueError(f"{what} must be a contiguous int32 device tensor with {n} rows")
        return t.data_ptr()

    def _rows(self, t, what, heads, n_tokens=None):
        """(pointer, token stride) of a [n_tokens, heads, head_dim] tensor whose heads are contiguous."""
        shape = t.shape
        if t.dtype != self.dtype or len(shape) != 3 or not t.is_cuda:
            raise ValueError(f"{what} must be a {self.dtype} device tensor [n_tokens, {heads}, {self.head_dim}]")
        n, h, d = shape
        if h != heads or d != self.head_dim or (n_tokens is not None and n != n_tokens):
            raise ValueError(f"{what} has shape {tuple(t.shape)}, not [{n_tokens}, {heads}, {self.head_dim}]")
        st, sh, sd = t.stride()
        if n and (sd != 1 or (h > 1 and sh != d)):
            raise ValueError(f"{what}: a token's heads must be contiguous")
        return t.data_ptr(), (st if n > 1 else h * d)

    def _whole(self, t, what, shape, dtype):
        if t.dtype != dtype or t.shape != shape or not t.is_contiguous() or not t.is_cuda:
            raise ValueError(f"{what} must be a contiguous {dtype} device tensor {shape}")
        return t.data_ptr()

    @staticmethod
    def _on(stream, *tensors):
        """The stream's handle; tensors used on a stream that is not the current one are recorded on it."""
        if stream is None:
            return _current_stream(tensors[0].get_device())
        for t in tensors:
            if t is not None:
                t.record_stream(stream)
        return stream.cuda_stream

    # --- entry points -------------------------------------------------------------
    def moe_attn_append(self, cells, q, k, v, positions, cu_q, kv_lens, table, q_out, stream=None):
        """q_out <- rotated q; the tokens' cells <- rotated k, and v.  positions: [n_tokens] int32, or None for the
        cells' places; q and q_out, or k and v, may be None."""
        if q is None and k is None:
            raise ValueError("q or k is needed")
        n = (q if q is not None else k).shape[0]
        qp, qs = (None, 0) if q is None else self._rows(q, "q", self.n_q_heads)
        kp, ks = (None, 0) if k is None else self._rows(k, "k", self.n_kv_heads, n)
        vp, vs = (None, 0) if v is None else self._rows(v, "v", self.n_kv_heads, n)
        op = None if q_out is None else self._whole(q_out, "q_out", (n, self.n_q_heads, self.head_dim), self.dtype)
        pp = None if positions is None else self._ints(positions, "positions", n)
        batch = self._fill(cells, kv_lens, table, cu_q, n, 0, 0)
        s = self._on(stream, cells, q, k, v, positions, cu_q, kv_lens, table, q_out)
        check(self._lib.moe_attn_append(self.attn, batch, qp, qs, kp, ks, vp, vs, pp, op, s), "moe_attn_append")

    def moe_attn_read(self, cells, cu_q, kv_lens, table, k_out, v_out, stream=None):
        """k_out, v_out [n_tokens, n_kv_heads, head_dim] <- the values in the new tokens' cells."""
        n = k_out.shape[0]
        shape = (n, self.n_kv_heads, self.head_dim)
        kp, vp = self._whole(k_out, "k_out", shape, self.dtype), self._whole(v_out, "v_out", shape, self.dtype)
        batch = self._fill(cells, kv_lens, table, cu_q, n, 0, 0)
        s = self._on(stream, cells, cu_q, kv_lens, table, k_out, v_out)
        check(self._lib.moe_attn_read(self.attn, batch, kp, vp, s), "moe_attn_read")

    def moe_attn_forward(self, cells, q, cu_q, kv_lens, table, out, lse=None, max_q=None, max_kv=None, stream=None):
        """out [n_tokens, n_q_heads, head_dim] and lse [n_tokens, n_q_heads] (fp32) <- attention of q over the cells.
        max_q: an upper bound of the new tokens per sequence (default: all tokens); it chooses the kernel."""
        qp, qs = self._rows(q, "q", self.n_q_heads)
        n = q.shape[0]
        op = self._whole(out, "out", (n, self.n_q_heads, self.head_dim), self.dtype)
        lp = None if lse is None else self._whole(lse, "lse", (n, self.n_q_heads), torch.float32)
        batch = self._fill(cells, kv_lens, table, cu_q, n, max_q, max_kv)
        s = self._on(stream, cells, q, cu_q, kv_lens, table, out, lse)
        check(self._lib.moe_attn_forward(self.attn, batch, qp, qs, op, lp, s), "moe_attn_forward")

    def moe_attn_weights(self, cells, q, lse, cu_q, kv_lens, table, acc_in, acc_out, decay=1.0, max_q=None, max_kv=None,
                         stream=None):
        """acc_out [n_seqs, cells] (fp32) <- decay * acc_in + the weight that q's rows give to each cell; acc_in may be
        None (zeros) or acc_out."""
        qp, qs = self._rows(q, "q", self.n_q_heads)
        n, seqs = q.shape[0], kv_lens.shape[0]
        lp = self._whole(lse, "lse", (n, self.n_q_heads), torch.float32)
        width = acc_out.shape[1]
        op = self._whole(acc_out, "acc_out", (seqs, width), torch.float32)
        ip = None if acc_in is None else self._whole(acc_in, "acc_in", (seqs, width), torch.float32)
        batch = self._fill(cells, kv_lens, table, cu_q, n, max_q, max_kv or min(width, table.shape[1] * self.page_cells))
        s = self._on(stream, cells, q, lse, cu_q, kv_lens, table, acc_in, acc_out)
        check(self._lib.moe_attn_weights(self.attn, batch, qp, qs, lp, ip, op, width, decay, s),
              "moe_attn_weights")

    def moe_attn_evict(self, cells, acc, kv_lens, table, recent, new_table, keep, new_lens, acc_out, stream=None):
        """Keeps keep.shape[1] cells of each sequence at most: the newest `recent` and those of the largest acc.  The
        kept cells go to the pages of new_table, in order; keep [n_seqs, budget] int32, new_lens [n_seqs] int32,
        acc_out [n_seqs, budget] fp32."""
        seqs, budget = keep.shape
        ap = self._whole(acc, "acc", (seqs, acc.shape[1]), torch.float32)
        kp = self._whole(keep, "keep", (seqs, budget), torch.int32)
        np_ = self._whole(new_lens, "new_lens", (seqs,), torch.int32)
        op = self._whole(acc_out, "acc_out", (seqs, budget), torch.float32)
        tp = self._ints(new_table, "new_table", seqs, 2)
        batch = self._fill(cells, kv_lens, table, None, 0, 0, 0)
        if kv_lens.shape[0] != seqs:
            raise ValueError("keep and kv_lens name different numbers of sequences")
        s = self._on(stream, cells, acc, kv_lens, table, new_table, keep, new_lens, acc_out)
        check(self._lib.moe_attn_evict(self.attn, batch, ap, acc.shape[1], budget, recent, tp,
                                       new_table.shape[1], kp, np_, op, s), "moe_attn_evict")

    def moe_attn_sync(self):
        """Waits for the device; raises MoeError for what a call found out of range on the GPU."""
        check(self._lib.moe_attn_sync(self.attn), "moe_attn_sync")

    def moe_attn_destroy(self):
        if self.attn is not None and self.attn.value:
            self._lib.moe_attn_destroy(self.attn)
        self.attn = None

    close = moe_attn_destroy

    def __del__(self):
        try:
            self.moe_attn_destroy()
        except Exception:
            pass
