"""int8 cells as moe_attn_append writes them, code by code: head vectors of
every magnitude that the 16-bit types hold."""

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

BF, FP, I8 = torch.bfloat16, torch.float16, torch.int8


def _written(io, d, k, v):
    """Codes [T, 2, hkv, d] and scales [T, 2, hkv] of tokens' cells."""
    from expert_cached_decode_gb300.attention import PagedAttention
    n, hkv = k.shape[:2]
    att = PagedAttention(hkv, hkv, d, 16, kv_dtype=I8, dtype=io)
    pages = -(-n // 16)
    cells = torch.zeros((pages, 16, att.cell_bytes), dtype=torch.uint8, device="cuda")
    table = torch.arange(pages, dtype=torch.int32, device="cuda")[None]
    cu, lens = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0, n], [n]))
    att.moe_attn_append(cells, None, k, v, None, cu, lens, table, None)
    ko, vo = torch.empty_like(k), torch.empty_like(v)
    att.moe_attn_read(cells, cu, lens, table, ko, vo)
    att.moe_attn_sync()
    raw = cells.reshape(pages * 16, -1)[:n].cpu().numpy()
    codes = raw[:, :2 * hkv * d].view(np.int8).reshape(n, 2, hkv, d)
    scales = np.ascontiguousarray(raw[:, 2 * hkv * d:2 * hkv * d + 8 * hkv]).view(np.float32).reshape(n, 2, hkv)
    return codes, scales, torch.stack([ko, vo], 1)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("io,exponents", [(BF, (0, 60, 126, -60, -99, -100, -101, -110, -120, -121, -122, -125, -126, -130)),
                                          (FP, (0, 15, -10, -14, -20))])
def test_codes_of_every_magnitude(io, d, exponents):
    # 127 over the largest magnitude passes fp32's range below 2^-121
    g = np.random.default_rng(d)
    x = g.standard_normal((len(exponents), 2, 3, d))
    x /= np.abs(x).max(-1, keepdims=True)
    x *= 2.0 ** np.array(exponents, dtype=np.float64)[:, None, None, None]
    x[-1, 0, 0] = 0.0
    t = torch.from_numpy(x).to(io).cuda()
    if io == BF:
        t[-1, 1, 0] = 0.0
        t[-1, 1, 0, 5] = -2.0 ** -133                          # the smallest one, alone
    codes, scales, _ = _written(io, d, t[:, 0].contiguous(), t[:, 1].contiguous())
    x = t.double().cpu().numpy()
    top = np.abs(x).max(-1)
    # the scale: one division in fp32, to the nearest (below its normal numbers to 2^-150)
    assert (np.abs(scales - top / 127) <= 2.0 ** -24 * top / 127 + 2.0 ** -150).all()
    # the code: nearest to x 127 / top, which takes a quotient and a product of 2^-24 each
    exact = x * 127 / np.where(top > 0, top, 1.0)[..., None]
    assert (np.abs(codes - exact) <= 0.5 + 127 * 2.0 ** -22).all()


@pytest.mark.parametrize("io", [BF, FP])
@pytest.mark.parametrize("d", [64, 128])
def test_what_is_not_finite_is_not_hidden(io, d):
    # a NaN or an infinity anywhere in a head vector: its scale says so, and its values read as NaN; its neighbours stay
    g = np.random.default_rng(d)
    t = torch.from_numpy(g.standard_normal((6, 2, 3, d))).to(io).cuda()
    clean = _written(io, d, t[:, 0].contiguous(), t[:, 1].contiguous())
    bad = np.zeros((6, 2, 3), bool)
    for token, kv, head, at, value in ((0, 0, 0, 0, np.nan), (1, 1, 2, d - 1, np.nan), (2, 0, 1, d // 2 + 3, -np.nan),
                                       (3, 1, 1, 7, np.inf), (4, 0, 2, d // 2, -np.inf)):
        t[token, kv, head, at] = value
        bad[token, kv, head] = True
    t[5, 0, 0] = float("nan")                                  # nothing else in the vector
    bad[5, 0, 0] = True
    codes, scales, values = _written(io, d, t[:, 0].contiguous(), t[:, 1].contiguous())
    assert np.array_equal(np.isfinite(scales), ~bad)
    assert torch.isnan(values[torch.from_numpy(bad).cuda()]).all()
    for got, want in zip((codes, scales, values.cpu().float().numpy()), (*clean[:2], clean[2].cpu().float().numpy())):
        assert np.array_equal(got[~bad], want[~bad])
