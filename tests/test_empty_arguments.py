"""Calls without tokens: torch gives an empty tensor any strides (0, 0 for one made from numpy's), and none is ever used."""
import numpy as np
import pytest
import torch


@pytest.fixture(scope="module")
def pi():
    import __graft_entry__
    __graft_entry__.build()
    import activation_sparse_rank_gb300 as pi
    return pi


def test_strides_of_empty_tensors(pi, monkeypatch):
    """Without a GPU: the checks of the device are left out."""
    ops = pi.operators
    monkeypatch.setattr(ops, "_dev", lambda t, device, name: t.device)
    cache = pi.KVCache.__new__(pi.KVCache)
    cache.device, cache._index, cache.head_dim = torch.device("cpu"), -1, 64
    empty, heads = torch.tensor(np.zeros((0, 9), np.float32)), torch.tensor(np.zeros((0, 4, 64), np.float32))
    assert empty.stride() == (0, 0) and heads.stride() == (0, 0, 0)                # torch's choice
    assert ops._probs(empty, None, None, None, "target") == 9
    assert list(ops._heads3(heads, torch.device("cpu"), "x")) == [256, 0]
    assert cache._rows(heads, 4, "q")[0] == 256
    table, none = torch.tensor(np.zeros((0, 5), np.int32)), torch.zeros(0, dtype=torch.int32)
    assert cache._tokens(table, torch.zeros(1, dtype=torch.int32), none, "start", 0).table_pages == 5
    one = torch.arange(3, dtype=torch.int32).view(1, 3).t()                        # a page a sequence, strides (1, 3)
    t = cache._tokens(one, torch.zeros(4, dtype=torch.int32), torch.zeros(3, dtype=torch.int32), "start", 0)
    assert (t.table_stride, t.table_pages) == (1, 1)
    some = torch.zeros(18, 2)
    for bad in (lambda: ops._probs(some.t(), None, None, None, "target"), lambda: cache._rows(torch.zeros(3, 64, 4).transpose(1, 2), 4, "q"),
                lambda: cache._tokens(torch.zeros(4, 3, dtype=torch.int32).t(), torch.zeros(4, dtype=torch.int32),
                                      torch.zeros(3, dtype=torch.int32), "start", 0)):
        with pytest.raises(ValueError):
            bad()


@pytest.mark.gpu
def test_calls_without_tokens(pi):
    def strange(*shape, dtype=torch.float16):
        return torch.zeros(shape, dtype=dtype, device="cuda").as_strided(shape, (0,) * len(shape))
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    c, rope, nobody = pi.KVCache(4, 2, 64, 16), pi.Rotary(64), strange(0, dtype=torch.int32)
    kv, q, table = strange(0, 2, 64), strange(0, 8, 64), ints([[1], [2]])
    start, cu = ints([3, 0]), ints([0, 0, 0])
    before = c.k_codes.clone(), c.k_scales.clone()
    assert pi.rotary(q, nobody, rope).shape == (0, 8, 64) and pi.rotary_backward(q, nobody, rope).shape == (0, 8, 64)
    c.write(kv, kv, table, cu, start)
    assert c.append(kv, kv, table, cu, start, rope, q=q).shape == (0, 8, 64)
    assert c.attention(q, table, cu, start).shape == (0, 8, 64)
    assert c.attention(q, table, cu, start, tree=strange(0, 1, dtype=torch.int32)).shape == (0, 8, 64)
    assert c.attention(q, strange(0, 4, dtype=torch.int32), ints([0]), nobody).shape == (0, 8, 64)
    p, floats = strange(0, 9, dtype=torch.float32), strange(0, dtype=torch.float32)
    for draft in (p, None):
        got = pi.verify_draft(p, draft, nobody, nobody, cu, floats, torch.zeros(2, device="cuda"))
        assert got.accepted.tolist() == [0, 0] and got.token.tolist() == [-1, -1] and got.path.tolist() == [[-1], [-1]]
    assert pi.token_logprobs(p).lse.shape == (0,)
    assert torch.equal(c.k_codes, before[0]) and torch.equal(c.k_scales, before[1]) and c.device_status() == 0
