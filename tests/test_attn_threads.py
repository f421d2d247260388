"""One handle of the attention binding in two host threads: the arguments of a
call are its own while the library reads them.  (A stand-in for the library, so
this runs without a GPU.)"""

import threading

import torch

from expert_cached_decode_gb300 import _abi, attention


class _Tensor:
    """What the binding looks at in a device tensor."""
    is_cuda = True

    def __init__(self, ptr, shape, dtype):
        self.ptr, self.shape, self.dtype = ptr, torch.Size(shape), dtype

    def data_ptr(self):
        return self.ptr

    def is_contiguous(self):
        return True

    def record_stream(self, stream):
        pass


class _Stream:
    cuda_stream = 0


class _Library:
    """moe_attn_read waits, before it looks at its arguments, until a second call has come in."""

    def __init__(self):
        self.first, self.second = threading.Event(), threading.Event()
        self.seen = {}

    def moe_attn_create(self, desc, out):
        out._obj.value = 1
        return 0

    def moe_attn_destroy(self, handle):
        pass

    def moe_attn_read(self, handle, batch, k_out, v_out, stream):
        if not self.first.is_set():
            self.first.set()
            assert self.second.wait(10)
        b = batch._obj
        self.seen[k_out] = {name: getattr(b, name) for name, _ in _abi.MoeAttnBatch._fields_}
        self.second.set()
        return 0


def test_two_threads_keep_their_arguments(monkeypatch):
    lib = _Library()
    monkeypatch.setattr(_abi, "load", lambda: lib)
    att = attention.PagedAttention(8, 2, 128, 16)
    want = {}

    def call(i):
        base, seqs, tokens, pages = 0x1000000 * (i + 1), 3 + i, 5 + i, 7 + i
        t = lambda k, shape, dtype: _Tensor(base + 4096 * k, shape, dtype)
        want[base] = dict(cells=base + 4096, n_pages=11 + i, block_table=base + 2 * 4096, kv_lens=base + 3 * 4096,
                          cu_q=base + 4 * 4096, n_seqs=seqs, table_pages=pages, n_tokens=tokens, max_q=0, max_kv=0)
        att.moe_attn_read(t(1, (11 + i, 16, att.cell_bytes), torch.uint8), t(4, (seqs + 1,), torch.int32),
                          t(3, (seqs,), torch.int32), t(2, (seqs, pages), torch.int32),
                          t(0, (tokens, 2, 128), torch.bfloat16), t(5, (tokens, 2, 128), torch.bfloat16), stream=_Stream())

    a = threading.Thread(target=call, args=(0,))
    a.start()
    assert lib.first.wait(10)
    call(1)
    a.join(10)
    assert lib.seen == want
