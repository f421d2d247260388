"""Argument checks of the gated delta rule and of the norms (moe_delta_*,
moe_norm_*): every call below is refused before any CUDA work, so this runs
without a GPU.  And the oracle's pieces against each other."""

import ctypes
import os

import numpy as np
import pytest

from expert_cached_decode_gb300 import _abi
from oracle import delta as od

INVALID, UNIMPL = -1, -7


@pytest.fixture(scope="module")
def lib():
    from expert_cached_decode_gb300 import LIB_PATH, build_library
    if not os.path.exists(LIB_PATH):
        build_library()
    return _abi.load()


@pytest.mark.parametrize("over,status,words", [
    (dict(n_k_heads=0), INVALID, "heads"),
    (dict(n_k_heads=3), INVALID, "heads"),
    (dict(n_k_heads=65, n_v_heads=65), INVALID, "heads"),
    (dict(n_v_heads=0), INVALID, "heads"),
    (dict(n_k_heads=2, n_v_heads=130), INVALID, "heads"),
    (dict(k_dim=96), UNIMPL, "k_dim"),
    (dict(v_dim=256), UNIMPL, "v_dim"),
    (dict(io_type=2), INVALID, "io_type"),
    (dict(io_type=3), INVALID, "io_type"),
    (dict(taps=1), INVALID, "taps"),
    (dict(taps=5), INVALID, "taps"),
    (dict(eps=-1.0), INVALID, "eps"),
    (dict(eps=float("nan")), INVALID, "eps"),
    (dict(scale=-1.0), INVALID, "scale"),
    (dict(scale=float("inf")), INVALID, "scale"),
])
def test_create_refuses(lib, over, status, words):
    d = dict(n_k_heads=2, n_v_heads=4, k_dim=128, v_dim=128, io_type=0, taps=4, normalize=1, eps=1e-6, scale=0.0)
    d.update(over)
    out = ctypes.c_void_p(12345)
    assert lib.moe_delta_create(ctypes.byref(_abi.MoeDeltaDesc(**d)), ctypes.byref(out)) == status
    assert out.value is None
    assert words in lib.moe_last_error().decode()


def test_null_handles_are_refused(lib):
    b = _abi.MoeDeltaBatch()
    assert lib.moe_delta_create(None, None) == INVALID
    assert lib.moe_delta_prepare(None, ctypes.byref(b), None, 0, None, None, None, None, None, None, 0, None, None, None, None,
                                 None) == INVALID
    assert lib.moe_delta_forward(None, ctypes.byref(b), None, 0, None, 0, None, 0, None, None, None, None, None) == INVALID
    assert lib.moe_delta_sync(None) == INVALID
    lib.moe_delta_destroy(None)


def _norm(**over):
    d = dict(d=64, io_type=0, y_type=3, h_type=0, gate_cols=0, act=1, scale=1.0, eps=1e-6, weight_offset=0.0)
    d.update(over)
    return _abi.MoeNormDesc(**d)


@pytest.mark.parametrize("over,words", [
    (dict(d=0), "d must"), (dict(d=60), "d must"), (dict(d=16392), "d must"), (dict(io_type=3), "io_type"), (dict(y_type=1), "y_type"),
    (dict(h_type=2), "h_type"), (dict(gate_cols=8), "gate_cols"), (dict(act=3), "act"), (dict(scale=float("nan")), "scale"),
    (dict(eps=float("inf")), "eps"), (dict(weight_offset=float("inf")), "weight_offset"),
])
def test_norm_block_refuses_its_description(lib, over, words):
    buf = ctypes.create_string_buffer(4096)
    p = ctypes.addressof(buf) + (-ctypes.addressof(buf)) % 16
    assert lib.moe_norm_block(ctypes.byref(_norm(**over)), 2, p, 64, p, 64, None, 0, None, None, p, None, None) == INVALID
    assert words in lib.moe_last_error().decode()


def test_norm_arguments(lib):
    buf = ctypes.create_string_buffer(4096)
    p = ctypes.addressof(buf) + (-ctypes.addressof(buf)) % 16
    D = ctypes.byref(_norm())
    block = lambda rows=2, y=p, ys=64, h=p, hs=64, gate=None, gs=0, post=None, pre=None, ho=p, x=None, d=D: lib.moe_norm_block(
        d, rows, y, ys, h, hs, gate, gs, post, pre, ho, x, None)
    assert block(d=None) == INVALID
    assert block(rows=-1) == INVALID and block(rows=2 ** 31) == INVALID
    assert block(y=None) == INVALID and block(y=p + 2) == INVALID and block(ys=56) == INVALID and block(ys=68) == INVALID
    assert block(hs=72) == INVALID                     # in place, but h is not contiguous
    assert block(ho=None) == INVALID and block(pre=p) == INVALID and block(x=p) == INVALID
    assert block(post=p + 8) == INVALID
    assert block(d=ctypes.byref(_norm(gate_cols=64))) == INVALID      # no gate given
    assert block(d=ctypes.byref(_norm(gate_cols=1)), gate=p, gs=-1) == INVALID
    assert block(rows=0, y=None) == 0
    gated = lambda n=2, heads=2, o=p, os_=128, z=p, zs=128, w=p, out=p: lib.moe_norm_gated(D, n, heads, o, os_, z, zs, w, 0, out, None)
    assert gated(heads=0) == INVALID and gated(n=-1) == INVALID and gated(n=2 ** 30, heads=2) == INVALID
    assert gated(o=None) == INVALID and gated(zs=64) == INVALID and gated(w=None) == INVALID and gated(out=None) == INVALID
    assert gated(os_=136) == INVALID                   # in place, but o is not contiguous
    assert gated(n=0, o=None) == 0


def test_the_rule_solves_for_its_keys():
    # without decay and with beta = 1 the state answers the newest key with its value, whatever was there
    g = np.random.default_rng(0)
    q = k = g.standard_normal((5, 1, 8))
    v, S0 = g.standard_normal((5, 2, 4)), g.standard_normal((2, 8, 4))
    o, S, mag, size = od.rule(q, k, v, np.zeros((5, 2)), np.ones((5, 2)), S0, 1.0, eps=0.0)
    assert np.allclose(o, v)
    assert (mag >= np.abs(o) - 1e-12).all() and (size[-1] >= np.sqrt((S ** 2).sum(1)) - 1e-12).all()
    # with beta = 0 the state only decays
    o, S, _, _ = od.rule(q, k, v, np.full((5, 2), -0.5), np.zeros((5, 2)), S0, 1.0, eps=0.0)
    assert np.allclose(S, S0 * np.exp(-2.5))
    assert np.allclose(o[2], np.einsum("hkv,hk->hv", S0 * np.exp(-1.5), np.repeat(od.unit(q[2], 0.0), 2, 0)))


def test_the_rule_in_chunks():
    # the products of a chunk (64 at a time on the GPU) are the recurrence
    g = np.random.default_rng(1)
    n, dk, dv = 7, 6, 5
    q, k = (od.unit(g.standard_normal((n, dk)), 0.0) for _ in range(2))
    v, S0, dec, b = g.standard_normal((n, dv)), g.standard_normal((dk, dv)), -g.random(n), g.random(n)
    o, S, _, _ = od.rule(q[:, None], k[:, None], v[:, None], dec[:, None], b[:, None], S0[None], 0.5, normalize=False)
    G = np.cumsum(dec)
    D = np.tril(np.exp(G[:, None] - G[None]))
    A = np.tril(b[:, None] * D * (k @ k.T), -1)
    U = np.linalg.solve(np.eye(n) + A, b[:, None] * (v - np.exp(G)[:, None] * (k @ S0)))
    assert np.allclose(o[:, 0], 0.5 * (np.exp(G)[:, None] * (q @ S0) + (D * (q @ k.T)) @ U))
    assert np.allclose(S[0], np.exp(G[-1]) * S0 + (np.exp(G[-1] - G)[:, None] * k).T @ U)


def test_convolution_and_gates():
    g = np.random.default_rng(2)
    x, w, old = g.standard_normal((4, 3)), g.standard_normal((3, 4)), g.standard_normal((3, 3))
    y, new, _ = od.conv(x, w, None, old)
    both = np.concatenate([old, x])
    for t in range(4):
        for c in range(3):
            z = sum(w[c, i] * both[t + i, c] for i in range(4))
            assert np.isclose(y[t, c], z / (1 + np.exp(-z)))
    assert np.array_equal(new, x[1:])
    assert np.array_equal(od.conv(x[:1], w, None, old)[1], np.concatenate([old[1:], x[:1]]))
    a, b = od.gates(np.array([0.0]), np.array([0.0]), np.array([np.log(2.0)]), np.array([0.0]))
    assert np.isclose(a[0], -2 * np.log(2)) and b[0] == 0.5
