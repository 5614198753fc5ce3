"""Page tables that are some columns of a wider one: positions past the columns are flagged, not looked up."""
import ctypes as C

import numpy as np
import pytest
import torch

from tests.kv_helpers import oracle_of, random_cache, same_cache


@pytest.fixture(scope="module")
def pi():
    import __graft_entry__
    __graft_entry__.build()
    import activation_sparse_rank_gb300 as pi
    return pi


def test_binding_passes_the_width_of_a_view(pi, monkeypatch):
    """Without a GPU: the checks of the device are left out, the arguments are the view's."""
    ops = pi.operators
    monkeypatch.setattr(ops, "_dev", lambda t, device, name: t.device)
    cache = pi.KVCache.__new__(pi.KVCache)
    cache.device = torch.device("cpu")
    wide = torch.arange(48, dtype=torch.int32).view(3, 16)
    cu, start = torch.zeros(4, dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    for view in (wide, wide[:, :4], wide[:, 12:]):
        t = cache._tokens(view, cu, start, "start", 5)
        assert (t.table_stride, t.table_pages) == (16, view.shape[1])
        assert t.page_table == view.data_ptr()
    t = cache._tokens(wide[1:2, 3:5], cu[:2], start[:1], "start", 5)
    assert t.table_pages == 2
    with pytest.raises(ValueError):
        cache._tokens(wide[:, :0], cu, start, "start", 5)


def test_negative_width_is_refused(pi):
    B, p = pi.binding, 1 << 20
    c = B.pi_kv_cache(4, 32, 2, 64, p, p, p, p, p)
    st = (C.c_int64 * 2)(128, 64)
    t = B.pi_kv_tokens(1, 3, p, p, 2, -1)
    assert pi.lib.pi_kv_write(C.byref(c), C.byref(t), p, None, st, p, st, 0, None) == 1
    assert b"table_pages" in pi.lib.pi_last_error()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.gpu
@pytest.mark.parametrize("columns", [slice(0, 2), slice(6, 8)])
def test_write_and_read_stop_at_the_view(pi, columns):
    """Two sequences of 20 tokens in one and a half pages of two; two more past their second page."""
    page, heads, dim = 16, 2, 64
    wide = torch.arange(16, dtype=torch.int32, device="cuda").view(2, 8)
    table = wide[:, columns]
    c = random_cache(pi, 16, heads, dim, page)
    ref = oracle_of(c)
    k = torch.randn(40, heads, dim, generator=torch.Generator().manual_seed(1)).half().cuda()
    cu = i32([0, 20, 40])
    c.write(k, -k, table, cu, i32([0, 0]))
    ref.write(k.double().cpu().numpy(), -k.double().cpu().numpy(), table.cpu().numpy(), [0, 20, 40], [0, 0])
    same_cache(c, ref)
    assert c.device_status() == 0
    c.write(k, -k, table, cu, i32([32, 40]))         # the next page of each would be the wider table's
    assert c.device_status() == 5
    same_cache(c, ref)
    got, _ = c.read(table, cu, i32([22, 22]), 40, dtype=torch.float32)
    assert c.device_status() == 5
    g = got.double().cpu().numpy()
    for s in range(2):
        np.testing.assert_array_equal(g[20 * s:20 * s + 10], ref.rows(0, table[s].tolist(), 22, 32))
        assert not g[20 * s + 10:20 * s + 20].any()


@pytest.mark.gpu
@pytest.mark.parametrize("columns", [slice(0, 2), slice(6, 8)])
@pytest.mark.parametrize("group,new,dim", [(1, 1, 64), (4, 20, 64), (2, 3, 256)])
def test_attention_stops_at_the_view(pi, columns, group, new, dim):
    """A length past the view's pages is flagged and cut to them; a view and its copy give the same bits."""
    page = 32
    wide = torch.arange(16, dtype=torch.int32, device="cuda").view(2, 8)
    table = wide[:, columns]
    c = random_cache(pi, 16, 2, dim, page)
    q = torch.randn(2 * new, 2 * group, dim, generator=torch.Generator().manual_seed(2)).half().cuda()
    cu = i32([0, new, 2 * new])
    for length, status in (([64, 50], 0), ([100, 50], 5)):
        out, lse = c.attention(q, table, cu, i32(length), max_q=new, want_lse=True)
        assert c.device_status() == status
        want, wlse = c.attention(q, table.contiguous(), cu, i32(length), max_q=new, want_lse=True)
        assert c.device_status() == status
        assert torch.equal(out, want) and torch.equal(lse, wlse)
        assert torch.isfinite(out).all()
