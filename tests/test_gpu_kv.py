"""The 8-bit key/value cache against its float64 definition: values are equal, not close."""
import numpy as np
import pytest
import torch

from oracle import operators as O
from tests.kv_helpers import TORCH, batch, oracle_of, random_cache, same_cache

pytestmark = pytest.mark.gpu

START = [0, 1, 15, 16, 5, 63, 100, 9, 0]
NEW = [1, 1, 1, 1, 40, 2, 17, 0, 33]


@pytest.fixture(scope="module")
def pi():
    import __graft_entry__
    __graft_entry__.build()
    import activation_sparse_rank_gb300 as pi
    return pi


def packed(n, heads, dim, dtype, seed, offset=0):
    """k and v as views of a packed projection [n, 3 heads dim (+ offset)]."""
    g = torch.Generator().manual_seed(seed)
    w = heads * dim
    x = (torch.randn(n, 3 * w + offset, generator=g) * torch.exp2(torch.randint(-6, 7, (n, 1), generator=g))).to(TORCH[dtype])
    x = x.cuda()
    return x[:, w + offset:2 * w + offset].unflatten(1, (heads, dim)), x[:, 2 * w + offset:].unflatten(1, (heads, dim))


def f64(t):
    return t.detach().double().cpu().numpy()


@pytest.mark.parametrize("dtype", ["float16", "bfloat16", "float32"])
@pytest.mark.parametrize("heads,dim,page,offset", [(1, 64, 16, 0), (3, 96, 48, 0), (2, 128, 64, 1), (5, 64, 256, 0),
                                                   (2, 256, 32, 3)])
def test_write_and_read(pi, dtype, heads, dim, page, offset):
    b = batch(START, NEW, page, seed=dim)
    c = random_cache(pi, b["pages"], heads, dim, page)
    ref = oracle_of(c)
    d = b["dev"]
    for step in range(2):                            # the second write meets the first one's scales
        k, v = packed(b["n"], heads, dim, dtype, seed=step, offset=offset)
        c.write(k, v, d["table"], d["cu"], d["start"])
        ref.write(f64(k), f64(v), b["table"], b["cu"], START)
        same_cache(c, ref)
    got = c.read(d["table"], d["cu"], d["start"], b["n"], dtype=TORCH[dtype])
    for which, t in enumerate(got):
        want = np.concatenate([ref.rows(which, b["table"][s], START[s], START[s] + NEW[s]) for s in range(len(START))])
        np.testing.assert_array_equal(f64(t), f64(torch.from_numpy(want).to(TORCH[dtype])))
    assert c.device_status() == 0


def test_special_values(pi):
    """Zeros, the largest value of a scale and the next above, tiny and huge values, NaN and infinities."""
    rows = [[0.0] * 64, [448.0] + [1.0] * 63, [448.001] + [1.0] * 63, [1e-30] * 64, [3e38, -3e38] + [1.0] * 62,
            [float("inf"), -float("inf"), float("nan"), 3.0] + [0.5] * 60, [float("nan")] * 64, [-1.75 * 2 ** -70] * 64]
    n = len(rows)
    b = batch([0] * n, [1] * n, 16)
    c = pi.KVCache(b["pages"], 1, 64, 16)
    ref = oracle_of(c)
    x = torch.tensor(rows, dtype=torch.float32).reshape(n, 1, 64).cuda()
    d = b["dev"]
    c.write(x, -x, d["table"], d["cu"], d["start"])
    ref.write(f64(x), f64(-x), b["table"], b["cu"], [0] * n)
    same_cache(c, ref)
    # a token that raises the scale of a block that holds a NaN, an infinity and small values
    big = torch.full((n, 1, 64), 3e4, device="cuda")
    one = torch.ones(n, dtype=torch.int32, device="cuda")
    c.write(big, big, d["table"], d["cu"], one)
    ref.write(f64(big), f64(big), b["table"], b["cu"], [1] * n)
    same_cache(c, ref)


def test_token_by_token_is_close_to_at_once(pi):
    """40 single tokens of equal size end in the same cache as one call."""
    b = batch([0], [40], 16)
    k, v = packed(40, 2, 64, "bfloat16", seed=5)
    k, v = k.sign(), v.sign() * 3                    # one magnitude: no scale grows on the way
    c, e = pi.KVCache(b["pages"], 2, 64, 16), pi.KVCache(b["pages"], 2, 64, 16)
    d = b["dev"]
    c.write(k, v, d["table"], d["cu"], d["start"])
    cu = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    for i in range(40):
        e.write(k[i:i + 1], v[i:i + 1], d["table"], cu, torch.tensor([i], dtype=torch.int32, device="cuda"))
    same_cache(e, oracle_of(c))


def test_nothing_to_write(pi):
    c = random_cache(pi, 3, 2, 64, 16)
    ref = oracle_of(c)
    none = torch.zeros(0, 2, 64, dtype=torch.float16, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    c.write(none, none, torch.zeros(0, 1, **i32), torch.zeros(1, **i32), torch.zeros(0, **i32))
    c.write(none, none, torch.zeros(2, 1, **i32), torch.zeros(3, **i32), torch.zeros(2, **i32))
    same_cache(c, ref)
    k, v = c.read(torch.zeros(0, 1, **i32), torch.zeros(1, **i32), torch.zeros(0, **i32), 5)
    assert k.shape == (5, 2, 64) and not k.any() and not v.any()
    assert c.device_status() == 0


def test_bad_tables_are_flagged_and_skipped(pi):
    """Pages outside the pool, positions past the table, a negative start, rows out
    of range: flagged, nothing else touched, what can be written is written."""
    heads, dim, page = 2, 64, 16
    b = batch([0, 0, 0, 0, 3], [5, 20, 5, 5, 5], page)
    k, v = packed(b["n"], heads, dim, "float16", seed=1)
    d = b["dev"]
    table, start = b["table"].copy(), [0, 0, 0, -4, 3]
    table[0, 0], table[1, 1] = -1, b["pages"]        # a bad page; the second page of a sequence
    start[2] = page * table.shape[1]                 # past the table
    c = random_cache(pi, b["pages"], heads, dim, page)
    ref = oracle_of(c)
    dev = [torch.tensor(x, dtype=torch.int32, device="cuda") for x in (table, start)]
    c.write(k, v, dev[0], d["cu"], dev[1])
    assert c.device_status() == 5 and c.device_status() == 0
    ref.write(f64(k[5:21]), f64(v[5:21]), [table[1]], [0, 16], [0])
    ref.write(f64(k[35:]), f64(v[35:]), [table[4]], [0, 5], [3])
    same_cache(c, ref)
    got, _ = c.read(dev[0], d["cu"], dev[1], b["n"], dtype=torch.float32)
    assert c.device_status() == 5
    assert not got[:5].any() and not got[21:35].any()
    np.testing.assert_array_equal(f64(got[5:21]), ref.rows(0, table[1], 0, 16))
    np.testing.assert_array_equal(f64(got[35:]), ref.rows(0, table[4], 3, 8))
    cu = torch.tensor([0, 5, 200, 30, 35, 40], dtype=torch.int32, device="cuda")
    c.write(k, v, dev[0], cu, dev[1])
    assert c.device_status() == 5


def test_rows_of_no_sequence_read_as_zero(pi):
    c = random_cache(pi, 4, 2, 64, 16)
    i32 = dict(dtype=torch.int32, device="cuda")
    k = torch.full((12, 2, 64), 7.0, dtype=torch.float16, device="cuda")
    c.read(torch.tensor([[1]], **i32), torch.tensor([3, 8], **i32), torch.tensor([2], **i32), 12, k=k)
    assert not k[:3].any() and not k[8:].any()
    np.testing.assert_array_equal(f64(k[3:8]), oracle_of(c).rows(0, [1], 2, 7))


def test_other_stream_and_graph(pi):
    b = batch([3, 0], [1, 30], 32)
    k, v = packed(b["n"], 2, 128, "float16", seed=3)
    d = b["dev"]
    c = random_cache(pi, b["pages"], 2, 128, 32)
    e = random_cache(pi, b["pages"], 2, 128, 32)
    c.write(k, v, d["table"], d["cu"], d["start"])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    e.write(k, v, d["table"], d["cu"], d["start"], stream=s)
    rk, _ = e.read(d["table"], d["cu"], d["start"], b["n"], stream=s)
    torch.cuda.current_stream().wait_stream(s)
    same_cache(e, oracle_of(c))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        e.write(k, v, d["table"], d["cu"], d["start"])
        gk, _ = e.read(d["table"], d["cu"], d["start"], b["n"])
    g.replay()
    assert torch.equal(gk, rk)


def test_refusals(pi):
    c = pi.KVCache(4, 2, 64, 16)
    i32 = dict(dtype=torch.int32, device="cuda")
    table, cu, start = torch.zeros(1, 2, **i32), torch.tensor([0, 3], **i32), torch.zeros(1, **i32)
    k = torch.zeros(3, 2, 64, dtype=torch.float16, device="cuda")
    for bad in (k.double(), k.cpu()):
        with pytest.raises(TypeError):
            c.write(bad, bad, table, cu, start)
    for bad in (k[:, :1], k[:, :, :32], k.transpose(1, 2)):
        with pytest.raises(ValueError):
            c.write(bad, bad, table, cu, start)
    with pytest.raises(ValueError):
        c.write(k, k.float(), table, cu, start)
    with pytest.raises(ValueError):
        c.write(k, k, table.long(), cu, start)
    with pytest.raises(ValueError):
        c.write(k, k, table, cu[:1], start)
    with pytest.raises(TypeError):
        c.write(k, k, table, cu, start.float())
    with pytest.raises(TypeError):
        c.read(table, cu, start, 3, dtype=torch.float64)
    with pytest.raises(ValueError):
        pi.KVCache(4, 2, 64, 24)
    with pytest.raises(pi.PiError):
        pi.KVCache(4, 2, 80, 16)
    with pytest.raises(pi.PiError):
        pi.KVCache(4, 2, 64, 512)
