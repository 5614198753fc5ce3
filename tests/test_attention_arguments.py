"""Arguments that say no more than they need to: large bounds (no GPU)."""
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
