"""Tensors and streams of another device than the call's are refused before the
library is called.  Stand-ins for tensors, so this runs without a GPU."""

import ctypes
import math

import pytest
import torch

from expert_cached_decode_gb300 import delta, norm

BF, F, I = torch.bfloat16, torch.float32, torch.int32


class Fake:
    """What the binding asks of a contiguous device tensor."""
    is_cuda = True

    def __init__(self, shape, dtype, device=1):
        self.shape, self.dtype, self.device_no, self.recorded = torch.Size(shape), dtype, device, []

    def dim(self):
        return len(self.shape)

    def stride(self, i=None):
        st = tuple(math.prod(self.shape[j + 1:]) for j in range(len(self.shape)))
        return st if i is None else st[i]

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 4096

    def get_device(self):
        return self.device_no

    def record_stream(self, s):
        self.recorded.append(s)


class Stream:
    cuda_stream = 77

    def __init__(self, device):
        self.device_index = device


class Library:
    """Stands in for the loaded library: notes the calls, each of them fine."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        return lambda *a: self.calls.append((name, a)) or 0


def _op(lib):
    op = delta.GatedDelta.__new__(delta.GatedDelta)
    op._lib, op.delta, op.device = lib, ctypes.c_void_p(0), 1
    op.n_k_heads, op.n_v_heads, op.k_dim, op.v_dim, op.dtype, op.taps = 1, 2, 64, 64, BF, 2
    op.channels, op._state_shape = 256, (2, 64, 64)
    return op


def _forward():
    return dict(q=Fake((4, 1, 64), BF), k=Fake((4, 1, 64), BF), v=Fake((4, 2, 64), BF), g=Fake((4, 2), F), beta=Fake((4, 2), F),
                state=Fake((3, 2, 64, 64), F), out=Fake((4, 2, 64), BF), cu=Fake((2,), I), slots_in=Fake((1,), I), slots_out=Fake((1,), I))


def _prepare():
    return dict(x=Fake((4, 256), BF), conv_w=Fake((256, 2), BF), conv_bias=Fake((256,), BF), conv_state=Fake((3, 1, 256), BF),
                y=Fake((4, 256), BF), a=Fake((4, 2), BF), b=Fake((4, 2), BF), a_log=Fake((2,), F), dt_bias=Fake((2,), F),
                g=Fake((4, 2), F), beta=Fake((4, 2), F), cu=Fake((2,), I), slots_in=Fake((1,), I), slots_out=Fake((1,), I))


def _block():
    return dict(y=Fake((4, 64), F), h=Fake((4, 64), BF), h_out=Fake((4, 64), BF), x=Fake((4, 64), BF), pre_w=Fake((64,), BF),
                post_w=Fake((64,), BF), gate=Fake((4, 64), BF))


def _gated():
    return dict(o=Fake((4, 2, 64), BF), z=Fake((4, 2, 64), BF), w=Fake((64,), BF), out=Fake((4, 2, 64), BF))


CALLS = {"moe_delta_forward": _forward, "moe_delta_prepare": _prepare, "moe_norm_block": _block, "moe_norm_gated": _gated}


@pytest.fixture
def calls(monkeypatch):
    lib = Library()
    for m in (delta, norm):
        monkeypatch.setattr(m, "_current_stream", lambda d: 1000 + d)
    monkeypatch.setattr(norm, "_current_device", lambda: 1)
    monkeypatch.setattr(norm._abi, "load", lambda: lib)

    def call(name, **kw):
        f = getattr(_op(lib), name) if name.startswith("moe_delta") else getattr(norm, name)
        return f(**kw)

    call.lib = lib
    return call


@pytest.mark.parametrize("name", CALLS)
def test_one_device(calls, name):
    calls(name, **CALLS[name]())
    assert calls.lib.calls[-1][0] == name and calls.lib.calls[-1][1][-1] == 1001
    kw = CALLS[name]()
    s = Stream(1)
    calls(name, **kw, stream=s)
    assert calls.lib.calls[-1][1][-1] == 77 and all(t.recorded == [s] for t in kw.values())


@pytest.mark.parametrize("name,arg", [(n, a) for n, make in CALLS.items() for a in make()])
def test_a_tensor_of_another_device(calls, name, arg):
    kw = CALLS[name]()
    kw[arg].device_no = 0
    with pytest.raises(ValueError, match=f"^{arg} must be .* device,? 1"):
        calls(name, **kw)
    assert not calls.lib.calls


@pytest.mark.parametrize("name", CALLS)
def test_a_stream_of_another_device(calls, name):
    kw = CALLS[name]()
    with pytest.raises(ValueError, match="stream is on device 0"):
        calls(name, **kw, stream=Stream(0))
    assert not calls.lib.calls and not any(t.recorded for t in kw.values())


@pytest.mark.parametrize("name", ["moe_norm_block", "moe_norm_gated"])
def test_norms_where_another_device_is_current(calls, name, monkeypatch):
    monkeypatch.setattr(norm, "_current_device", lambda: 0)
    with pytest.raises(ValueError, match="on the current device, 0"):
        calls(name, **CALLS[name]())
    assert not calls.lib.calls
