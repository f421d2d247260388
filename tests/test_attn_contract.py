"""Argument checks of the attention entry points (moe_attn_*): every call below
is refused before any CUDA work, so this runs without a GPU.  And the
frequency tables and cell sizes of the binding."""

import ctypes

import numpy as np
import pytest
import torch

from expert_cached_decode_gb300 import _abi
from oracle import attn as oa

INVALID, UNIMPL = -1, -7


@pytest.fixture(scope="module")
def lib():
    import os
    from expert_cached_decode_gb300 import LIB_PATH, build_library
    if not os.path.exists(LIB_PATH):
        build_library()
    return _abi.load()


def _desc(**over):
    d = dict(n_q_heads=8, n_kv_heads=2, head_dim=128, page_cells=16, cell_bytes=0, io_type=0, kv_type=0, window=0,
             scale=0.0, rot_dim=0, rot_interleaved=0, rot_factor=1.0, rot_turns=None)
    d.update(over)
    return _abi.MoeAttnDesc(**d)


@pytest.mark.parametrize("over,status,words", [
    (dict(n_kv_heads=0), INVALID, "heads"),
    (dict(n_kv_heads=3), INVALID, "heads"),
    (dict(n_q_heads=0), INVALID, "heads"),
    (dict(n_q_heads=66), INVALID, "heads"),
    (dict(n_kv_heads=65, n_q_heads=65), INVALID, "heads"),
    (dict(head_dim=96), UNIMPL, "head_dim"),
    (dict(head_dim=256), UNIMPL, "head_dim"),
    (dict(page_cells=0), INVALID, "page_cells"),
    (dict(page_cells=70000), INVALID, "page_cells"),
    (dict(io_type=2), INVALID, "io_type"),
    (dict(kv_type=1), INVALID, "kv_type"),
    (dict(kv_type=5), INVALID, "kv_type"),
    (dict(cell_bytes=1000), INVALID, "cell_bytes"),
    (dict(cell_bytes=1016), INVALID, "cell_bytes"),
    (dict(kv_type=2, cell_bytes=512), INVALID, "cell_bytes"),
    (dict(window=-1), INVALID, "window"),
    (dict(scale=-1.0), INVALID, "scale"),
    (dict(scale=float("nan")), INVALID, "scale"),
    (dict(rot_dim=24), INVALID, "rot_dim"),
    (dict(rot_dim=144), INVALID, "rot_dim"),
    (dict(rot_dim=64), INVALID, "rot_turns"),
])
def test_create_refuses(lib, over, status, words):
    out = ctypes.c_void_p(12345)
    assert lib.moe_attn_create(ctypes.byref(_desc(**over)), ctypes.byref(out)) == status
    assert out.value is None
    assert words in lib.moe_last_error().decode()


def test_null_handles_are_refused(lib):
    b = _abi.MoeAttnBatch()
    assert lib.moe_attn_create(None, None) == INVALID
    assert lib.moe_attn_append(None, ctypes.byref(b), None, 0, None, 0, None, 0, None, None, None) == INVALID
    assert lib.moe_attn_read(None, ctypes.byref(b), None, None, None) == INVALID
    assert lib.moe_attn_forward(None, ctypes.byref(b), None, 0, None, None, None) == INVALID
    assert lib.moe_attn_weights(None, ctypes.byref(b), None, 0, None, None, None, 0, 1.0, None) == INVALID
    assert lib.moe_attn_evict(None, ctypes.byref(b), None, 0, 1, 0, None, 0, None, None, None, None) == INVALID
    assert lib.moe_attn_sync(None) == INVALID
    lib.moe_attn_destroy(None)


def test_cell_sizes():
    from expert_cached_decode_gb300.attention import kv_cell_bytes
    assert kv_cell_bytes(4, 128, torch.int8) == 1056        # the int8 cell of the KV window
    assert kv_cell_bytes(4, 128, torch.bfloat16) == 2048
    assert kv_cell_bytes(1, 64, torch.int8) == 144          # 136 and padding
    assert kv_cell_bytes(3, 64, torch.float16) == 768


def test_rope_tables():
    from expert_cached_decode_gb300.attention import Rope
    r = Rope(64, base=10000.0)
    assert r.turns.shape == (32,) and r.turns.dtype == np.uint64 and r.factor == 1.0
    assert abs(float(r.turns[0]) * 2.0 ** -64 - 1 / (2 * np.pi)) < 2.0 ** -50
    # NTK keeps the first pair and divides the last by the factor
    n = Rope(64, base=10000.0, scaling="ntk", factor=4.0)
    assert n.turns[0] == r.turns[0]
    assert abs(float(n.turns[-1]) * 4 / float(r.turns[-1]) - 1) < 1e-12
    y = Rope(64, base=10000.0, scaling="yarn", factor=4.0, original_len=4096)
    assert y.turns[0] == r.turns[0] and abs(float(y.turns[-1]) * 4 / float(r.turns[-1]) - 1) < 1e-12
    assert abs(y.factor - (0.1 * np.log(4.0) + 1)) < 1e-12
    assert Rope(0).turns.size == 0
    for bad in (dict(rot_dim=20), dict(rot_dim=-16), dict(rot_dim=64, scaling="x"), dict(rot_dim=64, base=1.0),
                dict(rot_dim=64, factor=0.0)):
        with pytest.raises(ValueError):
            Rope(**bad)


def test_oracle_attention_against_a_loop():
    # the oracle's pieces against each other on a tiny case
    g = np.random.default_rng(0)
    q, k, v = g.standard_normal((3, 4, 8)), g.standard_normal((5, 2, 8)), g.standard_normal((5, 2, 8))
    out, lse, _ = oa.attention(q, k, v, 2, 0.5)
    for t in range(3):
        p = 5 - 3 + t
        for h in range(4):
            x = [0.5 * float(q[t, h] @ k[j, h // 2]) for j in range(max(0, p - 1), p + 1)]
            w = np.exp(x) / np.sum(np.exp(x))
            assert np.allclose(out[t, h], sum(a * v[j, h // 2] for a, j in zip(w, range(max(0, p - 1), p + 1))))
            assert np.isclose(lse[t, h], np.log(np.sum(np.exp(x))))
    assert np.isclose(oa.weights(q, k, lse, 2, 0.5).sum(), 12)
    assert list(oa.evict(np.array([1.0, 3.0, 3.0, 2.0, 0.0]), 3, 1)) == [1, 2, 4]
    assert list(oa.evict(np.array([np.nan, -np.inf, 0.0, 5.0]), 2, 0)) == [2, 3]
    # a rotation keeps a pair's length, and turning by two angles adds them
    x = g.standard_normal((2, 1, 8))
    f = np.array([0.3, 0.7])
    a = oa.rotate(oa.rotate(x, [1, 2], f, 1.0, 4, True), [3, 5], f, 1.0, 4, True)
    assert np.allclose(a, oa.rotate(x, [4, 7], f, 1.0, 4, True)) and np.allclose(a[..., 4:], x[..., 4:])


def test_oracle_weights_against_differences():
    # adding eps to the score of cell j changes lse by eps times the cell's weight
    g = np.random.default_rng(1)
    q, k, v = g.standard_normal((1, 1, 6)), g.standard_normal((7, 1, 6)), g.standard_normal((7, 1, 6))
    _, lse, _ = oa.attention(q, k, v, 0, 1.0)
    w = oa.weights(q, k, lse, 0, 1.0)
    for j in range(7):
        up, down = k.copy(), k.copy()
        step = 1e-5 * q[0, 0] / (q[0, 0] @ q[0, 0])
        up[j, 0] += step
        down[j, 0] -= step
        d = (oa.attention(q, up, v, 0, 1.0)[1] - oa.attention(q, down, v, 0, 1.0)[1])[0, 0] / 2e-5
        assert abs(d - w[j]) < 1e-9
