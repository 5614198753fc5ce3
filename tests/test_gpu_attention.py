"""Attention over the 8-bit cache against its float64 definition on the cache's stored values."""
import numpy as np
import pytest
import torch

from oracle import operators as O
from tests.kv_helpers import TORCH, batch, oracle_of, random_cache

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pi():
    import __graft_entry__
    __graft_entry__.build()
    import activation_sparse_rank_gb300 as pi
    return pi


def queries(n, heads, dim, dtype, seed=0, std=1.5):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(n, heads, dim, generator=g) * std).to(TORCH[dtype]).cuda()


def check(c, b, q, out, lse, length, causal=True, scale=None, rows=None):
    """Every output row within its bound; rows: only these (sequence, token) pairs."""
    ref = oracle_of(c)
    dtype = str(q.dtype).split(".")[1]
    heads, group, dim = c.heads, q.shape[1] // c.heads, c.head_dim
    scale = dim ** -0.5 if scale is None else scale
    qf, of, lf = (t.double().cpu().numpy() for t in (q, out, lse))
    for s in range(len(length)):
        r0, r1 = int(b["cu"][s]), int(b["cu"][s + 1])
        if r0 == r1:
            continue
        k, v = (ref.rows(i, b["table"][s], 0, max(0, int(length[s]))) for i in (0, 1))
        for h in range(q.shape[1]):
            want, wl, tol, tl = O.attention(qf[r0:r1, h], k[:, h // group], v[:, h // group], int(length[s]) - (r1 - r0),
                                            scale, causal)
            got, gl = of[r0:r1, h], lf[r0:r1, h]
            bound = tol + O.UNIT[dtype] * np.abs(want) * 1.001 + O.TINY[dtype]
            bad = ~((np.abs(got - want) <= bound) | (np.isnan(got) & np.isnan(want)))
            assert not bad.any(), (s, h, np.argwhere(bad)[:3], got[bad][:3], want[bad][:3], bound[bad][:3])
            same = (gl == wl) | (np.isnan(gl) & np.isnan(wl))
            assert (same | (np.abs(gl - wl) <= tl)).all(), (s, h, gl, wl, tl)


def run(pi, c, b, q, length, **kw):
    d = b["dev"]
    dl = torch.tensor(length, dtype=torch.int32, device="cuda")
    mq = int(np.diff(b["cu"]).max())
    out, lse = c.attention(q, d["table"], d["cu"], dl, max_q=mq, want_lse=True, **kw)
    again, _ = c.attention(q, d["table"], d["cu"], dl, max_q=mq, want_lse=True, **kw)
    assert torch.equal(out, again) or torch.isnan(out).any()
    return out, lse


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("heads,group,dim,page", [(1, 1, 64, 16), (2, 8, 128, 64), (1, 16, 64, 128), (3, 5, 96, 32),
                                                  (1, 7, 256, 16), (2, 4, 128, 256)])
def test_single_tokens(pi, dtype, heads, group, dim, page):
    """One new token a sequence, from an empty cache to some hundred tokens, page and tile edges among them."""
    length = [1, 2, 15, 16, 17, 64, 65, 333, 700, 48]
    b = batch([n - 1 for n in length], [1] * len(length), page, seed=dim)
    c = random_cache(pi, b["pages"], heads, dim, page, seed=group)
    q = queries(b["n"], heads * group, dim, dtype)
    out, lse = run(pi, c, b, q, length)
    check(c, b, q, out, lse, length)
    assert c.device_status() == 0


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("heads,group,dim,page,dtype", [(2, 1, 64, 16, "float16"), (1, 8, 128, 64, "bfloat16"),
                                                        (2, 3, 96, 32, "float16"), (1, 2, 256, 64, "bfloat16")])
def test_several_tokens(pi, heads, group, dim, page, dtype, causal):
    """Ragged new tokens: none, a few, more than a row tile; sequences without keys, or with fewer keys than rows."""
    new = [1, 5, 0, 33, 70, 2, 140, 3, 9]
    length = [1, 5, 20, 40, 300, 0, 141, 1, 400]     # 0: empty; 1 of 3: the first two rows see nothing
    b = batch([max(0, n - m) for n, m in zip(length, new)], new, page, seed=dim)
    c = random_cache(pi, b["pages"], heads, dim, page, seed=3)
    q = queries(b["n"], heads * group, dim, dtype, seed=1)
    out, lse = run(pi, c, b, q, length, causal=causal)
    check(c, b, q, out, lse, length, causal=causal)
    e = int(b["cu"][5])
    assert not out[e:e + 2].any() and torch.isneginf(lse[e:e + 2]).all()
    assert c.device_status() == 0


def test_up_to_sixteen_rows(pi):
    """Two to four tokens of four heads: one row tile with several positions in it."""
    new, length = [2, 4, 3, 1], [100, 64, 131, 70]
    b = batch([n - m for n, m in zip(length, new)], new, 32)
    c = random_cache(pi, b["pages"], 2, 128, 32)
    q = queries(b["n"], 8, 128, "float16")
    out, lse = run(pi, c, b, q, length)
    check(c, b, q, out, lse, length)


@pytest.mark.parametrize("length", [[9000], [4097, 1, 300], [0, 0, 0]])
@pytest.mark.parametrize("heads,group,dim", [(1, 1, 64), (2, 8, 128)])
def test_long_and_uneven(pi, length, heads, group, dim):
    """One sequence over many CTAs; a long one beside short ones; nothing at all."""
    b = batch([max(0, n - 1) for n in length], [1] * len(length), 64)
    c = random_cache(pi, b["pages"], heads, dim, 64)
    q = queries(b["n"], heads * group, dim, "float16")
    out, lse = run(pi, c, b, q, length)
    check(c, b, q, out, lse, length)


@pytest.mark.parametrize("new", [1, 40])
def test_scales_far_apart(pi, new):
    """Blocks whose scales differ by 2^40, values that only small blocks have, large and negative scales of the scores."""
    b = batch([500 - new], [new], 32)
    c = random_cache(pi, b["pages"], 2, 64, 32)
    g = torch.Generator().manual_seed(1)
    c.v_scales.copy_(torch.ldexp(torch.ones(c.v_scales.shape), torch.randint(-20, 20, c.v_scales.shape, generator=g)))
    c.k_scales.copy_(torch.ldexp(torch.ones(c.k_scales.shape), torch.randint(-30, -5, c.k_scales.shape, generator=g)))
    q = queries(new, 4, 64, "bfloat16")
    for scale in (0.125, -0.5, 0.0, 3.0):
        out, lse = run(pi, c, b, q, [500], sm_scale=scale)
        check(c, b, q, out, lse, [500], scale=scale)


@pytest.mark.parametrize("dtype,big,small", [("bfloat16", 1e30, 1e-30), ("float16", 6e4, 6e-8)])
def test_query_range(pi, dtype, big, small):
    """Query rows at the ends of their type's range, and zero."""
    b = batch([99] * 3, [1] * 3, 16)
    c = random_cache(pi, b["pages"], 1, 64, 16)
    q = queries(3, 2, 64, dtype)
    q[0] = (q[0].float() / q[0].float().abs().max() * big).to(q.dtype)
    q[1] = (q[1].float() * small).to(q.dtype)
    q[2] = 0
    for scale in (1 / big, 1.0):
        if dtype == "bfloat16" and scale == 1.0:
            continue                                 # every score overflows or only the largest counts
        out, lse = run(pi, c, b, q, [100] * 3, sm_scale=scale)
        check(c, b, q, out, lse, [100] * 3, scale=scale)


@pytest.mark.parametrize("group,new", [(1, 3), (2, 40), (8, 40)])
def test_masked_nan(pi, group, new):
    """Stale NaN codes after the last token reach no row; NaN keys and values of
    later tokens reach no earlier row and every later one."""
    length = 90
    b = batch([length - new], [new], 32)
    c = random_cache(pi, b["pages"], 1, 64, 32)
    q = queries(new, group, 64, "float16")
    last = b["table"][0, 2]
    c.k_codes[last, :, 26:] = 0x7f
    c.v_codes[last, :, 26:] = 0xff
    out, lse = run(pi, c, b, q, [length])
    check(c, b, q, out, lse, [length])
    assert torch.isfinite(out).all()
    c.v_codes[last, 0, 24, 5] = 0x7f                 # position 88: dim 5 of the last two rows
    out, lse = run(pi, c, b, q, [length])
    bad = torch.isnan(out)
    assert bad[-2:, :, 5].all() and bad.sum() == 2 * group
    c.v_codes[last, 0, 24, 5] = 0
    c.k_codes[last, 0, 25, 3] = 0x7f                 # position 89: the last row's scores
    out, lse = run(pi, c, b, q, [length])
    bad = torch.isnan(out)
    assert bad[-1].all() and not bad[:-1].any() and torch.isnan(lse[-1]).all()


def test_infinite_queries(pi):
    b = batch([63, 63], [1, 1], 64)
    c = random_cache(pi, b["pages"], 1, 64, 64)
    q = queries(2, 1, 64, "float16")
    q[0, 0, 0] = float("inf")
    q[1, 0, 3] = float("nan")
    out, lse = run(pi, c, b, q, [64, 64])
    assert torch.isnan(out).all() and torch.isnan(lse[1]).all()


def test_strided_queries_and_given_outputs(pi):
    b = batch([40, 7], [1, 1], 16)
    c = random_cache(pi, b["pages"], 2, 64, 16)
    wide = queries(2, 12, 64, "float16")
    q = wide[:, 4:8]
    d = b["dev"]
    out = torch.zeros(2, 4, 64, dtype=torch.float16, device="cuda")
    lse = torch.zeros(2, 4, device="cuda")
    r = c.attention(q, d["table"], d["cu"], d["length"], out=out, lse=lse)
    assert r[0] is out and r[1] is lse
    ref = c.attention(q.contiguous(), d["table"], d["cu"], d["length"])
    assert torch.equal(ref, out)


def test_cache_past_32_bit_offsets(pi):
    """Pages whose byte offsets pass 2^32."""
    page, heads, dim = 64, 8, 128
    pages = (1 << 32) // (page * heads * dim) + 40
    c = pi.KVCache.wrap(torch.empty(pages, heads, page, dim, dtype=torch.uint8, device="cuda"),
                        torch.ones(pages, heads, page // 16, device="cuda"),
                        torch.empty(pages, heads, page, dim, dtype=torch.uint8, device="cuda"),
                        torch.ones(pages, heads, page // 16, device="cuda"))
    i32 = dict(dtype=torch.int32, device="cuda")
    table = torch.tensor([[pages - 1, 3, pages - 20]], **i32)
    n = 150
    k, v = queries(n, heads, dim, "float16", seed=1), queries(n, heads, dim, "float16", seed=2)
    zero = torch.zeros(1, **i32)
    cu = torch.tensor([0, n], **i32)
    c.write(k, v, table, cu, zero)
    q = queries(1, heads, dim, "float16", seed=3)
    one, length = torch.tensor([0, 1], **i32), torch.tensor([n], **i32)
    out, lse = c.attention(q, table, one, length, want_lse=True)
    few = pi.KVCache(3, heads, dim, page)
    t = torch.tensor([[2, 0, 1]], **i32)
    few.write(k, v, t, cu, zero)
    ref, rlse = few.attention(q, t, one, length, want_lse=True)
    assert torch.equal(out, ref) and torch.equal(lse, rlse)
    rk, _ = c.read(table, cu, zero, n)
    fk, _ = few.read(t, cu, zero, n)
    assert torch.equal(rk, fk)
    assert c.device_status() == 0


def test_bad_tables_are_flagged(pi):
    b = batch([40, 7, 20], [1, 1, 2], 16)
    c = random_cache(pi, b["pages"], 2, 64, 16)
    q = queries(4, 4, 64, "float16")
    d = b["dev"]
    good = c.attention(q, d["table"], d["cu"], d["length"], max_q=2)
    assert c.device_status() == 0
    table = d["table"].clone()
    table[0, 1] = b["pages"]
    out = c.attention(q, table, d["cu"], d["length"], max_q=2)
    assert c.device_status() == 5 and torch.equal(out[1:], good[1:])
    length = d["length"].clone()
    length[0] = 1 << 30
    out = c.attention(q, d["table"], d["cu"], length, max_q=2)
    assert c.device_status() == 5 and torch.equal(out[1:], good[1:])
    length[0] = -5
    out = c.attention(q, d["table"], d["cu"], length, max_q=2)
    assert c.device_status() == 5 and torch.equal(out[1:], good[1:]) and not out[0].any()
    cu = d["cu"].clone()
    cu[3] = 9
    out = c.attention(q, d["table"], cu, d["length"], max_q=2)
    assert c.device_status() == 5 and torch.equal(out[:2], good[:2])
    out = c.attention(q, d["table"], d["cu"], d["length"], max_q=1)
    assert c.device_status() == 5 and torch.equal(out[:2], good[:2])


def test_other_stream_and_graph(pi):
    b = batch([700, 7], [1, 1], 16)
    c = random_cache(pi, b["pages"], 2, 64, 16)
    q = queries(2, 4, 64, "float16")
    d = b["dev"]
    ref = c.attention(q, d["table"], d["cu"], d["length"])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out = c.attention(q, d["table"], d["cu"], d["length"], stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(out, ref)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = c.attention(q, d["table"], d["cu"], d["length"])
    for _ in range(2):
        g.replay()
    assert torch.equal(out, ref)


def test_refusals(pi):
    c = pi.KVCache(4, 2, 64, 16)
    i32 = dict(dtype=torch.int32, device="cuda")
    table, cu, length = torch.zeros(1, 2, **i32), torch.tensor([0, 1], **i32), torch.ones(1, **i32)
    q = torch.zeros(1, 4, 64, dtype=torch.float16, device="cuda")
    with pytest.raises(TypeError):
        c.attention(q.float(), table, cu, length)
    with pytest.raises(TypeError):
        c.attention(q.cpu(), table, cu, length)
    with pytest.raises(ValueError):
        c.attention(q[:, :, :32], table, cu, length)
    with pytest.raises(pi.PiError):
        c.attention(q[:, :3], table, cu, length)     # not a multiple of the cache's heads
    with pytest.raises(pi.PiError):
        c.attention(q, table, cu, length, sm_scale=float("inf"))
    with pytest.raises(pi.PiError):
        c.attention(q, table, cu, length, max_q=-1)
    with pytest.raises(pi.PiError):
        c.attention(q, table, cu, length, ws=torch.empty(16, dtype=torch.uint8, device="cuda"))
    odd = torch.zeros(1, 4 * 64 + 4, dtype=torch.float16, device="cuda")[:, 4:].view(1, 4, 64)
    with pytest.raises(pi.PiError):
        c.attention(odd, table, cu, length)          # 8-byte aligned
