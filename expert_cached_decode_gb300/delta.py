"""Python binding of the gated delta rule (moe_delta_*): the convolution and the
gates in front of it, and the rule itself.

PyTorch supplies device memory and streams only.  Tensors keep their own
strides from token to token (slices of a fused projection work); a token's
heads have to be contiguous.  Every call is asynchronous on `stream` (default:
the current stream); `moe_delta_sync` reports values that were out of range on
the GPU.
"""

import ctypes
import struct

import torch

from . import _abi
from ._abi import MoeDeltaBatch, MoeDeltaDesc, check
from .attention import _TYPES, _current_stream

_BATCH = struct.Struct("PPPiiii")             # MoeDeltaBatch
assert _BATCH.size == ctypes.sizeof(MoeDeltaBatch)


class GatedDelta:
    """One handle of moe_delta_*: a head layout, and the work space of long sequences.  moe_delta_forward calls that overlap on
    the GPU (two streams, replays of two graphs) need a handle each; on one stream several threads may share one.

    cu:         [n_seqs + 1] int32 offsets of each sequence's new tokens
    slots_in:   [n_seqs] int32 slots that the states come from (-1: zeros)
    slots_out:  [n_seqs] int32 slots that they go to (-1: not kept); may be slots_in itself
    state:      [n_slots, n_v_heads, k_dim, v_dim] fp32
    conv_state: [n_slots, taps - 1, channels], channels = 2 n_k_heads k_dim + n_v_heads v_dim
    """

    def __init__(self, n_k_heads, n_v_heads, k_dim, v_dim, dtype=torch.bfloat16, taps=4, normalize=True, eps=1e-6, scale=0.0):
        if dtype not in (torch.bfloat16, torch.float16):
            raise ValueError("dtype must be bfloat16 or float16")
        self._lib = _abi.load()
        self.delta = None
        desc = MoeDeltaDesc(n_k_heads=n_k_heads, n_v_heads=n_v_heads, k_dim=k_dim, v_dim=v_dim, io_type=_TYPES[dtype],
                            taps=taps, normalize=int(normalize), eps=eps, scale=scale)
        h = ctypes.c_void_p()
        check(self._lib.moe_delta_create(ctypes.byref(desc), ctypes.byref(h)), "moe_delta_create")
        self.delta = h
        self.device = torch.cuda.current_device()
        self.n_k_heads, self.n_v_heads, self.k_dim, self.v_dim = n_k_heads, n_v_heads, k_dim, v_dim
        self.dtype, self.taps = dtype, taps
        self.channels = 2 * n_k_heads * k_dim + n_v_heads * v_dim
        self._state_shape = (n_v_heads, k_dim, v_dim)

    # --- arguments --------------------------------------------------------------
    def _fill(self, cu, slots_in, slots_out, n_slots, n_tokens, max_q):
        n = slots_in.shape[0]
        return ctypes.byref(MoeDeltaBatch.from_buffer_copy(_BATCH.pack(
            self._ints(cu, "cu", n + 1), self._ints(slots_in, "slots_in", n), self._ints(slots_out, "slots_out", n), n,
            n_tokens, n_slots, max_q or 0)))

    # (a kernel is launched on the handle's device, so every tensor has to be that device's)
    def _ints(self, t, what, n):
        shape = t.shape
        if t.dtype != torch.int32 or len(shape) != 1 or shape[0] != n or not t.is_contiguous() or t.get_device() != self.device:
            raise ValueError(f"{what} must be a contiguous int32 tensor of {n} on device {self.device}")
        return t.data_ptr()

    def _rows(self, t, what, heads, d, n_tokens=None):
        """(pointer, token stride) of a [n_tokens, heads, d] tensor whose heads are contiguous."""
        shape = t.shape
        if t.dtype != self.dtype or len(shape) != 3 or t.get_device() != self.device:
            raise ValueError(f"{what} must be a {self.dtype} tensor [n_tokens, {heads}, {d}] on device {self.device}")
        n, h, w = shape
        if h != heads or w != d or (n_tokens is not None and n != n_tokens):
            raise ValueError(f"{what} has shape {tuple(shape)}, not [{n_tokens}, {heads}, {d}]")
        st, sh, sd = t.stride()
        if n and (sd != 1 or (h > 1 and sh != d)):
            raise ValueError(f"{what}: a token's heads must be contiguous")
        return t.data_ptr(), (st if n > 1 else h * d)

    def _flat(self, t, what, width, n_tokens=None):
        """(pointer, row stride) of a [n_tokens, width] tensor with contiguous rows."""
        shape = t.shape
        if t.dtype != self.dtype or len(shape) != 2 or shape[1] != width or t.get_device() != self.device or (
                n_tokens is not None and shape[0] != n_tokens):
            raise ValueError(f"{what} must be a {self.dtype} tensor [{'n_tokens' if n_tokens is None else n_tokens}, {width}] "
                             f"on device {self.device}")
        if shape[0] and width > 1 and t.stride(1) != 1:
            raise ValueError(f"{what}: rows must be contiguous")
        return t.data_ptr(), (t.stride(0) if shape[0] > 1 else width)

    def _whole(self, t, what, shape, dtype):
        if t.dtype != dtype or t.shape != shape or not t.is_contiguous() or t.get_device() != self.device:
            raise ValueError(f"{what} must be a contiguous {dtype} tensor {tuple(shape)} on device {self.device}")
        return t.data_ptr()

    def _on(self, stream, *tensors):
        """The stream's handle; tensors used on a stream that is not the current one are recorded on it."""
        if stream is None:
            return _current_stream(self.device)
        if stream.device_index != self.device:
            raise ValueError(f"the stream is on device {stream.device_index}, the handle on device {self.device}")
        for t in tensors:
            if t is not None:
                t.record_stream(stream)
        return stream.cuda_stream

    # --- entry points -------------------------------------------------------------
    def moe_delta_prepare(self, x, conv_w, conv_bias, conv_state, y, a, b, a_log, dt_bias, g, beta, cu, slots_in, slots_out,
                          stream=None):
        """y [n_tokens, channels] <- silu of the causal convolution of x with conv_w [channels, taps] and conv_bias (or
        None), conv_state brought up to date; g, beta [n_tokens, n_v_heads] fp32 <- the gates of a and b.  x (with conv_w,
        conv_state, y) or a (with b, a_log, dt_bias, g, beta) may be None."""
        if x is None and a is None:
            raise ValueError("x or a is needed")
        n = (x if x is not None else a).shape[0]
        n_slots, xp, xs, wp, bp, cp, yp = 0, None, 0, None, None, None, None
        if x is not None:
            xp, xs = self._flat(x, "x", self.channels)
            wp = self._whole(conv_w, "conv_w", (self.channels, self.taps), self.dtype)
            bp = None if conv_bias is None else self._whole(conv_bias, "conv_bias", (self.channels,), self.dtype)
            n_slots = conv_state.shape[0]
            cp = self._whole(conv_state, "conv_state", (n_slots, self.taps - 1, self.channels), self.dtype)
            yp = self._whole(y, "y", (n, self.channels), self.dtype)
        else:
            n_slots = 2 ** 31 - 1            # no state is touched
        ap, s_ab, tp, lp, dp, gp, ep = None, 0, None, None, None, None, None
        if a is not None:
            ap, s_ab = self._flat(a, "a", self.n_v_heads, n)
            tp, s_b = self._flat(b, "b", self.n_v_heads, n)
            if s_b != s_ab:
                raise ValueError("a and b must have the same strides")
            lp = self._whole(a_log, "a_log", (self.n_v_heads,), torch.float32)
            dp = self._whole(dt_bias, "dt_bias", (self.n_v_heads,), torch.float32)
            gp = self._whole(g, "g", (n, self.n_v_heads), torch.float32)
            ep = self._whole(beta, "beta", (n, self.n_v_heads), torch.float32)
        batch = self._fill(cu, slots_in, slots_out, n_slots, n, 0)
        s = self._on(stream, cu, x, conv_w, conv_bias, conv_state, y, a, b, a_log, dt_bias, g, beta, slots_in, slots_out)
        check(self._lib.moe_delta_prepare(self.delta, batch, xp, xs, wp, bp, cp, yp, ap, tp, s_ab, lp, dp, gp, ep, s),
              "moe_delta_prepare")

    def moe_delta_forward(self, q, k, v, g, beta, state, out, cu, slots_in, slots_out, max_q=None, stream=None):
        """out [n_tokens, n_v_heads, v_dim] <- the gated delta rule over each sequence's tokens, state brought up to date.
        q, k [n_tokens, n_k_heads, k_dim], v [n_tokens, n_v_heads, v_dim], g (logarithm of the decay), beta [n_tokens,
        n_v_heads] fp32.  max_q: an upper bound of the tokens per sequence (default: all); it chooses the kernel."""
        qp, qs = self._rows(q, "q", self.n_k_heads, self.k_dim)
        n = q.shape[0]
        kp, ks = self._rows(k, "k", self.n_k_heads, self.k_dim, n)
        vp, vs = self._rows(v, "v", self.n_v_heads, self.v_dim, n)
        gp = self._whole(g, "g", (n, self.n_v_heads), torch.float32)
        bp = self._whole(beta, "beta", (n, self.n_v_heads), torch.float32)
        n_slots = state.shape[0]
        sp = self._whole(state, "state", (n_slots, *self._state_shape), torch.float32)
        op = self._whole(out, "out", (n, self.n_v_heads, self.v_dim), self.dtype)
        batch = self._fill(cu, slots_in, slots_out, n_slots, n, max_q)
        s = self._on(stream, q, k, v, g, beta, state, out, cu, slots_in, slots_out)
        check(self._lib.moe_delta_forward(self.delta, batch, qp, qs, kp, ks, vp, vs, gp, bp, sp, op, s), "moe_delta_forward")

    def moe_delta_sync(self):
        """Waits for the device; raises MoeError for what a call found out of range on the GPU."""
        check(self._lib.moe_delta_sync(self.delta), "moe_delta_sync")

    def moe_delta_destroy(self):
        if self.delta is not None and self.delta.value:
            self._lib.moe_delta_destroy(self.delta)
        self.delta = None

    close = moe_delta_destroy

    def __del__(self):
        try:
            self.moe_delta_destroy()
        except Exception:
            pass
