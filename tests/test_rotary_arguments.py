"""Rotary positions without a GPU: frequencies, refusals by the binding and by the C ABI before any launch."""
import ctypes as C
import math
import re
from pathlib import Path

import numpy as np
import pytest
import torch

ROOT = Path(__file__).resolve().parents[1]


@pytest.fixture(scope="module")
def pi():
    import __graft_entry__
    __graft_entry__._builder().build()
    import activation_sparse_rank_gb300 as pi
    return pi


def freq(pi, dim, base=10000.0, scaling=None, factor=1.0, original=None, fast=32.0, slow=1.0, magnitude=None, inv=None):
    from activation_sparse_rank_gb300 import operators
    return operators._frequencies(dim, base, scaling, factor, original, fast, slow, magnitude, inv)


def test_frequencies(pi):
    f, m = freq(pi, 64)
    np.testing.assert_allclose(f, 10000.0 ** (-np.arange(32) / 32), rtol=1e-15)
    assert m == 1.0
    g, m = freq(pi, 64, scaling="linear", factor=4.0)
    np.testing.assert_allclose(g, np.array(f) / 4, rtol=1e-15)
    g, m = freq(pi, 64, scaling="ntk", factor=8.0)
    assert g[0] == 1.0 and g[-1] == pytest.approx(f[-1] / 8, rel=1e-13) and m == 1.0
    g, m = freq(pi, 64, scaling="yarn", factor=16.0, original=4096)
    turns = 4096 * np.array(f) / (2 * math.pi)
    assert m == pytest.approx(0.1 * math.log(16) + 1)
    assert all(a == b for a, b, n in zip(g, f, turns) if n > 40)                 # fast pairs keep their own
    assert all(a == pytest.approx(b / 16) for a, b, n in zip(g, f, turns) if n < 0.7)
    assert all(b / 16 * (1 - 1e-12) <= a <= b for a, b in zip(g, f)) and sorted(g, reverse=True) == g
    assert freq(pi, 64, scaling="yarn", factor=16.0, original=4096, magnitude=1.5)[1] == 1.5
    assert freq(pi, 4, inv=torch.tensor([0.5, -7.0]))[0] == [0.5, -7.0]
    assert freq(pi, 2, scaling="ntk", factor=2.0)[0] == [1.0]


@pytest.mark.parametrize("kw", [dict(dim=63), dict(dim=0), dict(dim=514), dict(base=1.0), dict(base=math.inf), dict(factor=0.0),
                                dict(factor=math.nan), dict(scaling="cubic"), dict(scaling="yarn"), dict(inv_freq=[1.0]),
                                dict(scaling="yarn", original_length=4096, beta_fast=1.0, beta_slow=2.0),
                                dict(inv_freq=[math.nan] * 32), dict(inv_freq=[1.0] * 32, scaling="linear"),
                                dict(magnitude=math.inf)])
def test_rotary_refuses(pi, kw):
    with pytest.raises(ValueError):
        pi.Rotary(**{"dim": 64, **kw})


def test_host_tensors_are_refused(pi):
    with pytest.raises(TypeError):
        pi.Rotary(64, device="cpu")


def test_constant_matches_the_header(pi):
    text = (ROOT / "include" / "pi.h").read_text()
    assert int(re.search(r"#define\s+PI_MAX_ROTARY\s+([0-9]+)", text).group(1)) == pi.PI_MAX_ROTARY


def test_rotary_abi_refusals(pi):
    p = C.c_void_p(1 << 20)                          # never dereferenced: every call below is refused or empty
    st = (C.c_int64 * 2)(128, 64)

    def call(r=(32, 0, 1.0, 1 << 20), pos=p, n=3, heads=2, dim=64, x=p, xs=st, y=p, ys=st, dt=0, rot=True):
        r = pi.binding.pi_rotary(*r)
        return pi.lib.pi_rotary_apply(C.byref(r) if rot else None, pos, n, heads, dim, x, xs, y, ys, dt, 0, None)

    for bad in (dict(rot=False), dict(r=(66, 0, 1.0, 1 << 20)), dict(r=(32, 0, math.inf, 1 << 20)), dict(r=(32, 0, 1.0, None)),
                dict(r=(32, 0, 1.0, (1 << 20) + 4)), dict(pos=None), dict(n=-1), dict(heads=0), dict(heads=65536), dict(x=None),
                dict(y=None), dict(xs=None), dict(ys=None), dict(xs=(C.c_int64 * 2)(-1, 64)), dict(dt=3), dict(dim=16386),
                dict(x=C.c_void_p((1 << 20) + 1)), dict(pos=C.c_void_p((1 << 20) + 2))):
        assert call(**bad) == 1, bad
    assert call(r=(31, 0, 1.0, 1 << 20)) == 2 and call(r=(514, 0, 1.0, 1 << 20), dim=1024) == 2
    assert call(n=0) == 0


def test_append_abi_refusals(pi):
    fake = C.c_void_p(1 << 20)
    st = (C.c_int64 * 2)(128, 64)
    cache = pi.binding.pi_kv_cache(4, 32, 2, 64, 1 << 20, 1 << 20, 1 << 20, 1 << 20, 1 << 20)

    def call(r=(32, 0, 1.0, 1 << 20), tok=(1, 3, 1 << 20, 1 << 20, 2), k=fake, q=fake, qs=st, heads=2, out=fake, pos=None, dt=0,
             ks=st, start=fake):
        r, t = pi.binding.pi_rotary(*r), pi.binding.pi_kv_tokens(*tok)
        return pi.lib.pi_kv_append(C.byref(cache), C.byref(t), start, C.byref(r), pos, k, ks, fake, st, q, qs, heads, out, dt, None)

    for bad in (dict(r=(32, 0, math.nan, 1 << 20)), dict(r=(80, 0, 1.0, 1 << 20)), dict(k=None), dict(ks=None), dict(q=None),
                dict(out=None), dict(heads=0), dict(heads=-1), dict(heads=65536), dict(qs=None), dict(dt=5), dict(start=None),
                dict(out=C.c_void_p((1 << 20) + 8)), dict(pos=C.c_void_p((1 << 20) + 2)), dict(qs=(C.c_int64 * 2)(128, -64))):
        assert call(**bad) == 1, bad
    assert call(r=(24, 0, 1.0, 1 << 20)) == 2
    assert call(tok=(1 << 20, 1 << 28, 1 << 20, 1 << 20, 2), heads=65535) == 2
    assert call(tok=(1, 0, 1 << 20, 1 << 20, 2), q=None, heads=0, out=None) == 0
