"""Rotary positions and keys turned on their way into the cache, against the float64 definition."""
import math

import numpy as np
import pytest
import torch

from oracle import operators as O
from tests.kv_helpers import TORCH, batch, oracle_of, random_cache, same_cache

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pi():
    import __graft_entry__
    __graft_entry__.build()
    import activation_sparse_rank_gb300 as pi
    return pi


def f64(t):
    return t.detach().double().cpu().numpy()


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def normal(*shape, dtype, seed=0):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(*shape, generator=g).to(TORCH[dtype]).cuda()


def close(got, x, pos, rope, dtype, inverse=False):
    want, tol = O.rotary(f64(x), pos, rope.inv_freq, rope.magnitude, rope.interleaved, inverse)
    tol = tol + O.UNIT[dtype] * (np.abs(want) + tol) * (tol > 0) + O.TINY[dtype]
    err = np.abs(f64(got) - want)
    assert (err <= tol).all(), (err - tol).max()


POS = [0, 1, 2, 4095, 131071, 1048575, (1 << 31) - 1, -1, -70000, 7]


@pytest.mark.parametrize("dtype", ["float16", "bfloat16", "float32"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("heads,dim,turned", [(1, 64, 64), (40, 128, 128), (5, 96, 24), (3, 80, 20), (7, 256, 64), (2, 6, 2),
                                              (71, 64, 16), (1, 600, 512)])
def test_rotary(pi, dtype, interleaved, heads, dim, turned):
    rope = pi.Rotary(turned, interleaved=interleaved)
    x = normal(len(POS), heads, dim, dtype=dtype, seed=dim)
    y = pi.rotary(x, ints(POS), rope)
    close(y, x, POS, rope, dtype)
    assert torch.equal(y[..., turned:], x[..., turned:])
    close(pi.rotary_backward(x, ints(POS), rope), x, POS, rope, dtype, inverse=True)


@pytest.mark.parametrize("tokens,heads", [(1, 1), (33, 1), (700, 3), (5000, 8), (40, 200)])
def test_counts(pi, tokens, heads):
    """From one row to more tokens and heads than a CTA takes."""
    rope = pi.Rotary(32, scaling="yarn", factor=4.0, original_length=64)
    pos = list(np.random.default_rng(tokens).integers(0, 1 << 20, tokens))
    x = normal(tokens, heads, 48, dtype="bfloat16", seed=1)
    close(pi.rotary(x, ints(pos), rope), x, pos, rope, "bfloat16")


@pytest.mark.parametrize("offset", [0, 1, 4])
@pytest.mark.parametrize("dtype", ["float16", "float32"])
def test_strides_and_in_place(pi, dtype, offset):
    """Queries and keys of a packed projection, turned where they are; what lies around them stays."""
    rope = pi.Rotary(64, interleaved=offset == 1)
    packed = normal(9, 6 * 64 + offset, dtype=dtype)
    before = packed.clone()
    qk = packed[:, offset:offset + 4 * 64].unflatten(1, (4, 64))
    pos = list(range(100, 109))
    apart = pi.rotary(qk, ints(pos), rope)
    close(apart, qk, pos, rope, dtype)
    assert pi.rotary(qk, ints(pos), rope, out=qk) is qk
    assert torch.equal(qk, apart)
    packed[:, offset:offset + 4 * 64] = before[:, offset:offset + 4 * 64]
    assert torch.equal(packed, before)
    to = torch.zeros(4, 9, 64, dtype=TORCH[dtype], device="cuda").transpose(0, 1)      # heads first
    pi.rotary(qk, ints(pos), rope, out=to)
    assert torch.equal(to, apart)
    one = normal(1, 4, 64, dtype=dtype).expand(9, 4, 64)                               # a broadcast row
    close(pi.rotary(one, ints(pos), rope), one, pos, rope, dtype)
    for out, x in ((one, qk), (one, one)):
        with pytest.raises(ValueError):
            pi.rotary(x, ints(pos), rope, out=out)
    square = normal(4, 4, 64, dtype=dtype)
    with pytest.raises(ValueError):                   # the same memory in another order
        pi.rotary(square, ints(pos[:4]), rope, out=square.transpose(0, 1))


def test_gradient(pi):
    """The gradient against differences of the float64 definition, and turning there and back."""
    rope = pi.Rotary(32, scaling="yarn", factor=8.0, original_length=128)
    pos = [3, 777, 50000]
    x, dy = normal(3, 2, 40, dtype="float32", seed=1), normal(3, 2, 40, dtype="float32", seed=2)
    dx = f64(pi.rotary_backward(dy, ints(pos), rope))
    rng = np.random.default_rng(0)
    for _ in range(20):
        d = rng.standard_normal(x.shape)
        up, _ = O.rotary(f64(x) + 0.5 * d, pos, rope.inv_freq, rope.magnitude, False)
        dn, _ = O.rotary(f64(x) - 0.5 * d, pos, rope.inv_freq, rope.magnitude, False)
        # linear, so differences are the derivative; 240 terms, each within 2^-21 of |dy| |d| magnitude
        bound = 240 * 2.0 ** -21 * rope.magnitude * np.abs(d).max() * np.abs(f64(dy)).max() * 2
        assert abs(((up - dn) * f64(dy)).sum() - (dx * d).sum()) <= bound
    back = f64(pi.rotary_backward(pi.rotary(x, ints(pos), rope), ints(pos), rope))
    tol = 2.0 ** -20 * rope.magnitude ** 2 * 2 * np.abs(f64(x)).max()
    assert np.abs(back[..., :32] - f64(x)[..., :32] * rope.magnitude ** 2).max() <= tol


def test_special_values_and_empty(pi):
    rope = pi.Rotary(4)
    x = torch.tensor([[[math.inf, 1.0, 2.0, 3.0, math.nan]], [[0.0, -0.0, 0.0, 6e4, -math.inf]]], dtype=torch.float16, device="cuda")
    y = f64(pi.rotary(x, ints([0, 1]), rope))
    assert np.isnan(y[0, 0, 2]) or np.isinf(y[0, 0, 2])              # 0 * inf is NaN: a pair spoils itself alone
    assert y[0, 0, 1] == 1.0 and y[0, 0, 3] == 3.0 and np.isnan(y[0, 0, 4]) and np.isneginf(y[1, 0, 4])
    assert y[1, 0, 0] == 0 and np.isfinite(y[1, 0, :4]).all()
    none = torch.zeros(0, 3, 64, device="cuda")
    assert pi.rotary(none, ints([]), pi.Rotary(64)).shape == (0, 3, 64)
    none = torch.zeros(3, 0, 64, device="cuda")
    assert pi.rotary(none, ints([1, 2, 3]), pi.Rotary(64)).shape == (3, 0, 64)


def test_refusals(pi):
    rope, x = pi.Rotary(64), normal(3, 2, 64, dtype="float16")
    for bad in (lambda: pi.rotary(x, ints([1, 2]), rope), lambda: pi.rotary(x[0], ints([1, 2, 3]), rope),
                lambda: pi.rotary(x, ints([1, 2, 3]), rope, out=x.float()), lambda: pi.rotary(x[..., ::2], ints([1, 2, 3]), rope),
                lambda: pi.rotary(x.cpu(), ints([1, 2, 3]), rope), lambda: pi.rotary(x, ints([1, 2, 3]).long(), rope),
                lambda: pi.rotary(x.double(), ints([1, 2, 3]), rope)):
        with pytest.raises((ValueError, TypeError)):
            bad()
    with pytest.raises(pi.PiError):
        pi.rotary(x[..., :32], ints([1, 2, 3]), rope)


def test_stream_and_graph(pi):
    rope = pi.Rotary(128)
    x, pos = normal(50, 9, 128, dtype="bfloat16"), ints(list(range(50)))
    want = pi.rotary(x, pos, rope)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = pi.rotary(x, pos, rope, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    out = torch.zeros_like(x)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pi.rotary(x, pos, rope, out=out)
    for shift in (5, 1000):
        pos += shift
        g.replay()
        assert torch.equal(out, pi.rotary(x, pos, rope))


# ---- the append ---------------------------------------------------------------------

START = [0, 1, 15, 16, 5, 63, 100, 9, 0]
NEW = [1, 1, 1, 1, 40, 2, 17, 0, 33]


@pytest.mark.parametrize("dtype", ["float16", "bfloat16", "float32"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("heads,dim,page,turned,q_heads,offset", [(1, 64, 16, 64, 1, 0), (3, 96, 48, 48, 6, 0), (2, 128, 64, 128, 16, 1),
                                                                  (5, 64, 256, 16, 35, 0), (2, 256, 32, 128, 2, 0), (1, 128, 16, 96, 0, 0)])
def test_append(pi, dtype, interleaved, heads, dim, page, turned, q_heads, offset):
    """The cache is that of turned binary32 keys written, bit for bit; the queries are those that `rotary` gives."""
    rope = pi.Rotary(turned, interleaved=interleaved, scaling="linear", factor=2.0)
    b = batch(START, NEW, page, seed=dim)
    c, ref = random_cache(pi, b["pages"], heads, dim, page), random_cache(pi, b["pages"], heads, dim, page)
    d, n = b["dev"], b["n"]
    own = ints([s + i for s, m in zip(START, NEW) for i in range(m)])
    given = ints(list(np.random.default_rng(3).integers(0, 1 << 17, n)))
    for pos in (None, given):                        # the second call meets the first one's scales
        packed = normal(n, (q_heads + 2 * heads) * dim + offset, dtype=dtype, seed=page)[:, offset:]
        qkv = packed.unflatten(1, (q_heads + 2 * heads, dim))
        q, k, v = qkv[:, :q_heads], qkv[:, q_heads:q_heads + heads], qkv[:, q_heads + heads:]
        at = own if pos is None else pos
        turned_k = pi.rotary(k.float(), at, rope)
        got = c.append(k, v, d["table"], d["cu"], d["start"], rope, positions=pos, q=q if q_heads else None)
        ref.write(turned_k, v.float(), d["table"], d["cu"], d["start"])
        same_cache(c, oracle_of(ref))
        if q_heads:
            assert torch.equal(got, pi.rotary(q.contiguous(), at, rope))
        else:
            assert got is None
    assert c.device_status() == 0


def test_append_many(pi):
    """Enough tokens that a warp does several heads of a block; queries in place."""
    rope = pi.Rotary(64)
    start, new, heads = [7, 0, 300], [3001, 2000, 1], 9
    b = batch(start, new, 32)
    c, ref = random_cache(pi, b["pages"], heads, 64, 32), random_cache(pi, b["pages"], heads, 64, 32)
    d, n = b["dev"], b["n"]
    k, v, q = (normal(n, h, 64, dtype="bfloat16", seed=h) for h in (heads, heads, 27))
    own = ints([s + i for s, m in zip(start, new) for i in range(m)])
    want = pi.rotary(q, own, rope)
    ref.write(pi.rotary(k.float(), own, rope), v.float(), d["table"], d["cu"], d["start"])
    assert c.append(k, v, d["table"], d["cu"], d["start"], rope, q=q, q_out=q) is q
    assert torch.equal(q, want)
    same_cache(c, oracle_of(ref))


def test_append_bad_tables(pi):
    """Pages outside the pool, positions past the table, a negative start: flagged, the rest as a write leaves it, queries turned."""
    rope = pi.Rotary(32)
    b = batch([0, 0, 0, 0, 3], [5, 20, 5, 5, 5], 16)
    d, n = b["dev"], b["n"]
    d["table"][0, 0] = 1 << 20
    d["table"][2, 0] = -3
    start = d["start"].clone()
    start[3] = -20
    table = d["table"][:, :1].contiguous()           # sequence 1 passes it
    c, ref = random_cache(pi, b["pages"], 2, 64, 16), random_cache(pi, b["pages"], 2, 64, 16)
    k, v, q = (normal(n, h, 64, dtype="float32", seed=h) for h in (2, 2, 4))
    pos = ints(list(range(n)))
    got = c.append(k, v, table, d["cu"], start, rope, positions=pos, q=q)
    ref.write(pi.rotary(k, pos, rope), v, table, d["cu"], start)
    same_cache(c, oracle_of(ref))
    assert torch.equal(got, pi.rotary(q, pos, rope))
    with pytest.raises(pi.PiError):
        pi.binding._check(c.device_status(), "status")


def test_append_rows_of_no_sequence_and_refusals(pi):
    rope = pi.Rotary(64)
    b = batch([3], [4], 16)
    d = b["dev"]
    c, ref = random_cache(pi, b["pages"], 2, 64, 16), random_cache(pi, b["pages"], 2, 64, 16)
    k, q = normal(9, 2, 64, dtype="float16"), normal(9, 4, 64, dtype="float16", seed=1)
    out = torch.full_like(q, 7.0)
    c.append(k, k, d["table"], d["cu"], d["start"], rope, q=q, q_out=out)
    assert (out[4:] == 7.0).all()
    assert torch.equal(out[:4], pi.rotary(q[:4], ints([3, 4, 5, 6]), rope))
    ref.write(pi.rotary(k[:4].float(), ints([3, 4, 5, 6]), rope), k[:4].float(), d["table"], d["cu"], d["start"])
    same_cache(c, oracle_of(ref))
    args = (d["table"], d["cu"], d["start"])
    for bad in (lambda: c.append(k, k, *args, None), lambda: c.append(k, k[:8], *args, rope), lambda: c.append(k, k, *args, rope, q_out=out),
                lambda: c.append(k, k, *args, rope, q=q.float()), lambda: c.append(k, k, *args, rope, q=q[:8]),
                lambda: c.append(k, k, *args, rope, positions=ints([1, 2])), lambda: c.append(k, k, *args, rope, q=q, q_out=out[:8])):
        with pytest.raises((ValueError, TypeError)):
            bad()
    with pytest.raises(pi.PiError):
        c.append(k, k, *args, pi.Rotary(24))
    none = k[:0]
    assert c.append(none, none, ints([]).view(0, 1), ints([0]), ints([]), rope, q=q[:0]).shape == (0, 4, 64)
    same_cache(c, oracle_of(ref))


def test_append_in_a_graph(pi):
    """One capture serves later steps: start and the page table are read when it is replayed."""
    rope = pi.Rotary(64, interleaved=True)
    b = batch([0, 5], [40, 40], 16)
    d = b["dev"]
    c, ref = random_cache(pi, b["pages"], 1, 64, 16), random_cache(pi, b["pages"], 1, 64, 16)
    k, q, out = normal(2, 1, 64, dtype="bfloat16"), normal(2, 8, 64, dtype="bfloat16"), torch.zeros(2, 8, 64, dtype=torch.bfloat16, device="cuda")
    cu, start = ints([0, 1, 2]), d["start"].clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.append(k, k, d["table"], cu, start, rope, q=q, q_out=out)
    for step in range(20):
        k.copy_(normal(2, 1, 64, dtype="bfloat16", seed=step))
        g.replay()
        ref.write(pi.rotary(k.float(), start, rope), k.float(), d["table"], cu, start)
        assert torch.equal(out, pi.rotary(q, start, rope))
        start += 1
    same_cache(c, oracle_of(ref))
