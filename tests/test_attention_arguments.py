"""Arguments that say no more than they need to: large bounds, strides of axes of one (no GPU)."""
import ctypes as C

import pytest
import torch


@pytest.fixture(scope="module")
def pi():
    import __graft_entry__
    __graft_entry__._builder().build()
    import activation_sparse_rank_gb300 as pi
    return pi


@pytest.mark.parametrize("max_q", [3, 1 << 28, 2 ** 31 - 1])
def test_any_bound_above_the_rows_is_the_rows(pi, max_q):
    """A bound past what the kernels could take is no refusal: three rows are three rows (the workspace is refused)."""
    B, p = pi.binding, 1 << 20
    c = B.pi_kv_cache(4, 32, 2, 64, p, p, p, p, p)
    t = B.pi_kv_tokens(1, 3, p, p, 2, 2)
    st = (C.c_int64 * 2)(1024, 64)
    got = pi.lib.pi_kv_attention(C.byref(c), C.byref(t), p, max_q, p, st, 16, 0, 0.125, 1, p, None, None, 0, None)
    assert got == 1 and b"ws must be" in pi.lib.pi_last_error()


def test_strides_of_single_rows(pi, monkeypatch):
    """The stride of an axis of one is never used, and torch keeps whatever it was through .contiguous()."""
    ops = pi.operators
    monkeypatch.setattr(ops, "_dev", lambda t, device, name: t.device)
    cache = pi.KVCache.__new__(pi.KVCache)
    cache.device, cache._index, cache.head_dim = torch.device("cpu"), -1, 64
    base = torch.zeros(8 * 257, dtype=torch.float16)
    one = base.as_strided((1, 4, 64), (257, 64, 1))
    assert one.contiguous().stride(0) == 257
    assert list(cache._rows(one, 4, "q")) == [256, 64]
    assert list(cache._rows(base.as_strided((3, 1, 64), (64, 99, 1)), 1, "q")) == [64, 64]
    assert list(cache._rows(base.as_strided((3, 4, 64), (264, 64, 1)), 4, "q")) == [264, 64]
