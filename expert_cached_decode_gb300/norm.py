"""Python binding of the norms around the blocks (moe_norm_*).

PyTorch supplies device memory and streams only.  Both calls are asynchronous
on `stream` (default: the current stream).
"""

import ctypes
import struct

import torch

from . import _abi
from ._abi import MoeNormDesc, check
from .attention import _TYPES, _current_stream

_ACTS = {None: _abi.MOE_ACT_NONE, "none": _abi.MOE_ACT_NONE, "sigmoid": _abi.MOE_ACT_SIGMOID, "silu": _abi.MOE_ACT_SILU}
_T = {**_TYPES, torch.float32: _abi.MOE_T_F32}
_DESC = struct.Struct("iiiiiifff")            # MoeNormDesc
assert _DESC.size == ctypes.sizeof(MoeNormDesc)


# without the checks around it, where torch has it (as 2.9 and 2.11 do)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


# (a kernel is launched on the current device `dev`, so every tensor has to be that device's)
def _rows(t, what, n, d, dtypes, dev):
    """(pointer, row stride) of a [n, d] tensor with contiguous rows."""
    if t.dtype not in dtypes or t.dim() != 2 or t.shape[0] != n or t.shape[1] != d or t.get_device() != dev:
        raise ValueError(f"{what} must be a tensor [{n}, {d}] of {' or '.join(str(x) for x in dtypes)} on the current device, {dev}")
    st, sd = t.stride()
    if n and d > 1 and sd != 1:
        raise ValueError(f"{what}: rows must be contiguous")
    return t.data_ptr(), (st if n > 1 else d)


def _whole(t, what, shape, dtype, dev):
    if t.dtype != dtype or t.shape != shape or not t.is_contiguous() or t.get_device() != dev:
        raise ValueError(f"{what} must be a contiguous {dtype} tensor {tuple(shape)} on the current device, {dev}")
    return t.data_ptr()


def _on(stream, dev, *tensors):
    """The stream's handle; tensors used on a stream that is not the current one are recorded on it."""
    if stream is None:
        return _current_stream(dev)
    if stream.device_index != dev:
        raise ValueError(f"the stream is on device {stream.device_index}, the current one is {dev}")
    for t in tensors:
        if t is not None:
            t.record_stream(stream)
    return stream.cuda_stream


def _io(*tensors):
    """The 16-bit type of the call: that of the first tensor that has one."""
    for t in tensors:
        if t is not None and t.dtype in (torch.bfloat16, torch.float16):
            return t.dtype
    raise ValueError("a tensor of the call must be bfloat16 or float16")


def moe_norm_block(y, h, h_out, x=None, pre_w=None, post_w=None, gate=None, act="sigmoid", scale=1.0, eps=1e-6,
                   weight_offset=0.0, stream=None):
    """h_out <- h + scale act(gate) y', y' = post_w ? rms(y) (weight_offset + post_w) : y, and x <- rms(h_out) (weight_offset
    + pre_w), in one pass.  y, h [rows, d] (fp32 or the 16-bit type of the others; h may be None: zeros), gate [rows, d] or
    [rows, 1] or None, post_w, pre_w [d]; h_out [rows, d] of h's type (may be h; None: not written), x [rows, d] of the
    16-bit type, or None with pre_w.  act: "sigmoid", "silu" or "none"."""
    n, d = y.shape
    dev = _current_device()
    io = _io(x, pre_w, post_w, gate, y, h, h_out)
    yp, ys = _rows(y, "y", n, d, (io, torch.float32), dev)
    ht = h.dtype if h is not None else h_out.dtype if h_out is not None else io
    hp, hs = (None, 0) if h is None else _rows(h, "h", n, d, (io, torch.float32), dev)
    gp, gs, cols = None, 0, 0
    if gate is not None:
        cols = 1 if gate.dim() == 2 and gate.shape[1] == 1 else d
        gp, gs = _rows(gate, "gate", n, cols, (io,), dev)
    op = None if h_out is None else _whole(h_out, "h_out", (n, d), ht, dev)
    xp = None if x is None else _whole(x, "x", (n, d), io, dev)
    pw = None if post_w is None else _whole(post_w, "post_w", (d,), io, dev)
    qw = None if pre_w is None else _whole(pre_w, "pre_w", (d,), io, dev)
    desc = MoeNormDesc.from_buffer_copy(_DESC.pack(d, _T[io], _T[y.dtype], _T.get(ht, -1), cols, _ACTS[act], scale, eps, weight_offset))
    s = _on(stream, dev, y, h, gate, post_w, pre_w, h_out, x)
    check(_abi.load().moe_norm_block(ctypes.byref(desc), n, yp, ys, hp, hs, gp, gs, pw, qw, op, xp, s), "moe_norm_block")


def moe_norm_gated(o, z, w, out, act="silu", gate_first=False, eps=1e-6, weight_offset=0.0, stream=None):
    """out [n_tokens, heads, d] <- rms(o) (weight_offset + w) act(z) per head vector, or with gate_first rms(o act(z))
    (weight_offset + w).  o, z [n_tokens, heads, d] with their own token strides, w [d]; out may be o."""
    n, heads, d = o.shape
    dev = _current_device()
    io = _io(o)
    ptrs = []
    for t, what in ((o, "o"), (z, "z")):
        if t.dtype != io or t.shape != o.shape or t.get_device() != dev:
            raise ValueError(f"{what} must be a {io} tensor {tuple(o.shape)} on the current device, {dev}")
        st, sh, sd = t.stride()
        if n and ((d > 1 and sd != 1) or (heads > 1 and sh != d)):
            raise ValueError(f"{what}: a token's heads must be contiguous")
        ptrs += [t.data_ptr(), st if n > 1 else heads * d]
    wp = _whole(w, "w", (d,), io, dev)
    op = _whole(out, "out", (n, heads, d), io, dev)
    desc = MoeNormDesc.from_buffer_copy(_DESC.pack(d, _T[io], 0, 0, 0, _ACTS[act], 1.0, eps, weight_offset))
    s = _on(stream, dev, o, z, w, out)
    check(_abi.load().moe_norm_gated(ctypes.byref(desc), n, heads, *ptrs, wp, int(gate_first), op, s), "moe_norm_gated")
