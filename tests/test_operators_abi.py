"""The operators around the FFN without a GPU: refusals by the C ABI before any launch, constants, the binding's checks."""
import ctypes as C
import re
from pathlib import Path

import pytest
import torch

ROOT = Path(__file__).resolve().parents[1]


@pytest.fixture(scope="module")
def pi():
    import __graft_entry__
    __graft_entry__._builder().build()
    import activation_sparse_rank_gb300 as pi
    return pi


def test_constants_match_the_header(pi):
    text = (ROOT / "include" / "pi.h").read_text()
    defs = dict(re.findall(r"#define\s+(PI_[A-Z0-9_]+)\s+\(?(-?[0-9]+)", text))
    for n in ("PI_KV_BLOCK", "PI_KV_MAX_PAGE", "PI_MAX_TOP_K"):
        assert int(defs[n]) == getattr(pi, n)
    for name, value in re.findall(r"\b(PI_DT_[A-Z0-9_]+)\s*=\s*([0-9]+)", text):
        assert getattr(pi.binding, name) == int(value), name


def _cache(pi, **kw):
    f = dict(n_pages=4, page_size=32, heads=2, head_dim=64, k_codes=1 << 20, k_scales=1 << 20, v_codes=1 << 20,
             v_scales=1 << 20, status=1 << 20)
    f.update(kw)
    return pi.binding.pi_kv_cache(*f.values())


def test_cache_refusals(pi):
    lib = pi.lib
    fake = C.c_void_p(1 << 20)                       # never dereferenced: every call below is refused or empty
    st = (C.c_int64 * 2)(128, 64)
    tok = pi.binding.pi_kv_tokens(1, 3, 1 << 20, 1 << 20, 2)

    def write(c, t=tok, k=fake, s=st, dt=0, start=fake):
        return lib.pi_kv_write(c and C.byref(c), t and C.byref(t), start, k, s, fake, st, dt, None)

    good = _cache(pi)
    assert write(None) == 1 and write(good, None) == 1
    for bad in (dict(head_dim=80), dict(page_size=24), dict(page_size=512), dict(page_size=0)):
        assert write(_cache(pi, **bad)) == 2, bad
    for bad in (dict(n_pages=0), dict(heads=0), dict(k_codes=(1 << 20) + 8), dict(v_scales=(1 << 20) + 2),
                dict(k_scales=None), dict(status=None)):
        assert write(_cache(pi, **bad)) == 1, bad
    assert write(good, dt=3) == 1 and write(good, k=None) == 1 and write(good, start=None) == 1
    assert write(good, s=(C.c_int64 * 2)(-1, 64)) == 1 and write(good, s=None) == 1
    assert write(good, pi.binding.pi_kv_tokens(1, -1, 1 << 20, 1 << 20, 2)) == 1
    assert write(good, pi.binding.pi_kv_tokens(1, 3, None, 1 << 20, 2)) == 1
    assert write(good, pi.binding.pi_kv_tokens(1, 3, 1 << 20, 1 << 20, 0)) == 1
    assert write(good, pi.binding.pi_kv_tokens(0, 0, None, None, 0)) == 0      # nothing to do
    assert lib.pi_kv_read(C.byref(good), C.byref(tok), fake, None, None, 0, None) == 1
    assert lib.pi_kv_read(C.byref(good), C.byref(tok), fake, C.c_void_p((1 << 20) + 4), None, 0, None) == 1
    assert lib.pi_kv_status(None, None) == 1


def test_attention_refusals(pi):
    lib = pi.lib
    fake = C.c_void_p(1 << 20)
    c, tok = _cache(pi), pi.binding.pi_kv_tokens(1, 3, 1 << 20, 1 << 20, 2)
    assert lib.pi_kv_attention_workspace_bytes(None, 4, 1, 1) == 0
    need = lib.pi_kv_attention_workspace_bytes(C.byref(c), 4, 3, 1)
    assert need > 0

    def attend(q=fake, st=(C.c_int64 * 2)(256, 64), heads=4, dt=0, scale=0.125, out=fake, ws=fake, n=need, max_q=3):
        return lib.pi_kv_attention(C.byref(c), C.byref(tok), fake, max_q, q, st, heads, dt, scale, 1, out, None, ws, n, None)

    for bad in (dict(q=None), dict(out=None), dict(heads=3), dict(heads=0), dict(dt=2), dict(scale=float("nan")),
                dict(st=(C.c_int64 * 2)(250, 64)), dict(st=None), dict(ws=None), dict(n=need - 1), dict(max_q=-1),
                dict(q=C.c_void_p((1 << 20) + 8))):
        assert attend(**bad) == 1, bad
    assert attend(max_q=0) == 0


def test_norm_refusals(pi):
    lib = pi.lib
    p = C.c_void_p(1 << 20)

    def norm(x=p, st=64, add=None, add_dt=0, w=p, w_dt=0, rows=2, d=64, dt=0, eps=1e-5, y=p, s=None):
        return lib.pi_layer_norm(x, st, add, add_dt, w, None, w_dt, rows, d, dt, eps, y, s, None, None, None)

    for bad in (dict(x=None), dict(y=None), dict(rows=-1), dict(dt=7), dict(w_dt=9), dict(eps=-1.0), dict(st=63),
                dict(add=p), dict(s=p), dict(add=p, s=p, add_dt=4), dict(eps=float("nan")), dict(x=C.c_void_p((1 << 20) + 1))):
        assert norm(**bad) == 1, bad
    assert norm(d=0) == 2 and norm(d=16385) == 2 and norm(rows=0) == 0
    n = lib.pi_layer_norm_backward_workspace_bytes(2, 64)
    assert n > 0 and lib.pi_layer_norm_backward_workspace_bytes(2, 0) == 0

    def back(dy=p, x=p, mean=p, dx=p, dw=p, ws=p, nb=n, rows=2):
        return lib.pi_layer_norm_backward(dy, x, 64, p, 0, mean, p, None, rows, 64, 0, dx, dw, None, ws, nb, None)

    for bad in (dict(dy=None), dict(x=None), dict(mean=None), dict(dx=None), dict(ws=None), dict(nb=n - 1), dict(rows=-2)):
        assert back(**bad) == 1, bad


def test_score_refusals(pi):
    p = C.c_void_p(1 << 20)

    def score(x=p, st=100, dt=0, rows=2, vocab=100, t=p, k=2, lp=p, idx=p):
        return pi.lib.pi_token_logprobs(x, st, dt, rows, vocab, t, k, lp, None, None, idx, p, None)

    for bad in (dict(x=None), dict(st=99), dict(dt=3), dict(rows=-1), dict(vocab=0), dict(t=None), dict(k=-1), dict(k=65),
                dict(k=64, vocab=50), dict(idx=None), dict(lp=C.c_void_p((1 << 20) + 2))):
        assert score(**bad) == 1, bad
    assert score(rows=0) == 0


def test_binding_refuses_host_tensors(pi):
    x = torch.zeros(4, 64)
    with pytest.raises(TypeError):
        pi.layer_norm(x)
    with pytest.raises(TypeError):
        pi.layer_norm_backward(x, x, None, x, x)
    with pytest.raises(TypeError):
        pi.token_logprobs(x)
    with pytest.raises(TypeError):
        pi.KVCache(2, 1, 64, 16, device="cpu")
    with pytest.raises(ValueError):
        pi.KVCache(2, 1, 64, 20, device="cpu")
