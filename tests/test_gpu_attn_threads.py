"""One attention handle in several host threads on one stream: a call's kernels
stay together, so each call joins its own parts of the shared work space."""

import threading

import pytest
import torch

pytestmark = pytest.mark.gpu

BF, I8 = torch.bfloat16, torch.int8


def test_threads_on_one_stream_get_their_own_results():
    from attn_helpers import Case
    # items cut in every kernel: single tokens, two streams of a row tile, both kernels in one call, 256-row tiles
    kinds = [([1] * 3, [5000, 700, 33]), ([10] * 3, [4000, 900, 2000]), ([70, 1, 2], [3000, 5000, 64]), ([90], [6000])]
    cases = [Case(n, lens, 8, 2, 128, 32, I8, BF, seed=i) for i, (n, lens) in enumerate(kinds)]
    att = cases[0].att
    stream = torch.cuda.Stream()

    def calls(c):
        """(out, lse, weights) of one pass, on the shared stream."""
        n = max(c.n_new)
        out = torch.zeros((c.tokens, 8, 128), dtype=BF, device="cuda")
        lse = torch.zeros((c.tokens, 8), device="cuda")
        acc = torch.zeros((len(c.kv_lens), max(c.kv_lens)), device="cuda")
        torch.cuda.current_stream().synchronize()
        att.moe_attn_forward(c.cells, c.q, c.d_cu, c.d_lens, c.d_table, out, lse, max_q=n, stream=stream)
        att.moe_attn_weights(c.cells, c.q, lse, c.d_cu, c.d_lens, c.d_table, None, acc, max_q=n, stream=stream)
        return out, lse, acc

    want = [calls(c) for c in cases]
    torch.cuda.synchronize()
    wrong, errors = [], []

    def work(i):
        try:
            got = [calls(cases[i]) for _ in range(40)]
            stream.synchronize()
            wrong.extend((i, k) for g in got for k in range(3) if not torch.equal(g[k], want[i][k]))
        except Exception as e:                       # a thread's failure is the test's
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    att.moe_attn_sync()
    assert not errors and not wrong, (errors, wrong[:5])
