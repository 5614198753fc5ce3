"""Pins of the float64 definitions in oracle/operators.py (CPU only)."""
import numpy as np
import pytest
import torch

from oracle import operators as O


def test_e4m3_against_torch():
    t = O.e4m3_table()
    ref = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(t, ref)
    x = np.concatenate([np.linspace(-450, 450, 40001), np.linspace(-0.05, 0.05, 20001), t[:127],
                        (t[:126] + t[1:127]) / 2])
    x = x[np.abs(x) <= 448].astype(np.float32)
    ref = torch.from_numpy(x).to(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(O.e4m3_round(x), ref)
    np.testing.assert_array_equal(O.e4m3_round([np.inf, -1e9, np.nan, 0.0]), [448, -448, np.nan, 0])


def test_block_scale_by_hand():
    assert O.block_scale([448.0]) == 1.0
    assert O.block_scale([448.5]) == 2.0
    assert O.block_scale([1.75, -0.1]) == 2.0 ** -8
    assert O.block_scale([0.0]) == 2.0 ** -64
    assert O.block_scale([np.inf, np.nan, 1.0]) == 2.0 ** -8


def test_cache_growth_by_hand():
    z = np.zeros((2, 1, 16, 1), np.uint8)
    c = O.CacheOracle(z, np.ones((2, 1, 1)), z, np.ones((2, 1, 1)))
    one = np.array([[[1.0]]])
    c.write(one, one, [[1]], [0, 1], [0])
    assert c.scale[0][1, 0, 0] == 2.0 ** -8 and c.value[0][1, 0, 0, 0] == 256.0
    c.write(1000 * one, one, [[1]], [0, 1], [1])                # 1000 <= 448 * 4
    assert c.scale[0][1, 0, 0] == 4.0
    assert c.value[0][1, 0, 0, 0] == 0.25 and c.value[0][1, 0, 1, 0] == O.e4m3_round(250.0)
    np.testing.assert_array_equal(c.rows(0, [1], 0, 2)[:, 0, 0], [1.0, 4 * 256.0])
    assert c.scale[1][1, 0, 0] == 2.0 ** -8                      # values: unchanged


def test_attention_against_torch():
    rng = np.random.default_rng(0)
    q, k, v = rng.normal(size=(3, 8)), rng.normal(size=(7, 8)), rng.normal(size=(7, 8))
    out, lse, _, _ = O.attention(q, k, v, 4, 0.3)
    s = torch.from_numpy(0.3 * q @ k.T)
    s = s.masked_fill(torch.arange(7)[None] > torch.arange(4, 7)[:, None], -np.inf)
    np.testing.assert_allclose(out, (torch.softmax(s, 1) @ torch.from_numpy(v)).numpy(), rtol=1e-12)
    np.testing.assert_allclose(lse, torch.logsumexp(s, 1).numpy(), rtol=1e-12)
    out, lse, _, _ = O.attention(q, k[:1], v[:1], -2, 0.3)       # the first two rows see nothing
    assert (out[:2] == 0).all() and np.isneginf(lse[:2]).all() and np.isfinite(lse[2])
    np.testing.assert_allclose(out[2], v[0])


def test_norm_and_gradient_against_differences():
    rng = np.random.default_rng(1)
    x, w, b, dy = rng.normal(size=(4, 6)), rng.normal(size=6), rng.normal(size=6), rng.normal(size=(4, 6))
    y, mean, rstd = O.layer_norm(x, w, b, 1e-5)[:3]
    ref = torch.nn.functional.layer_norm(torch.from_numpy(x), (6,), torch.from_numpy(w), torch.from_numpy(b), 1e-5)
    np.testing.assert_allclose(y, ref.numpy(), rtol=1e-10)
    dx, dw, db = O.layer_norm_backward(dy, x, w, mean, rstd)[:3]

    def loss(x, w, b):
        return (O.layer_norm(x, w, b, 1e-5)[0] * dy).sum()

    e = 1e-6
    for i in range(4):
        for j in range(6):
            d = np.zeros_like(x)
            d[i, j] = e
            assert abs((loss(x + d, w, b) - loss(x - d, w, b)) / (2 * e) - dx[i, j]) < 1e-7
    for j in range(6):
        d = np.zeros(6)
        d[j] = e
        assert abs((loss(x, w + d, b) - loss(x, w - d, b)) / (2 * e) - dw[j]) < 1e-7
        assert abs((loss(x, w, b + d) - loss(x, w, b - d)) / (2 * e) - db[j]) < 1e-7


def test_logprobs_against_torch():
    rng = np.random.default_rng(2)
    x = rng.normal(size=(5, 40)) * 3
    x[1, 7] = x[1, 3]                                             # a tie
    x[2, :30] = -np.inf
    t = np.array([3, 7, 35, -1, 40])
    logp, ent, lse, idx, val, _ = O.token_logprobs(x, t, 4)
    ref = torch.log_softmax(torch.from_numpy(x), 1)
    np.testing.assert_allclose(logp[:3], [ref[i, t[i]] for i in range(3)], rtol=1e-12)
    assert logp[3] == 0 and np.isnan(logp[4])
    p = ref.exp()
    np.testing.assert_allclose(ent, -torch.where(p > 0, p * ref, 0.0).sum(1).numpy(), rtol=1e-12)
    np.testing.assert_allclose(val, torch.topk(ref, 4, 1).values.numpy(), rtol=1e-12)
    a = np.zeros((1, 9))
    assert list(O.token_logprobs(a, None, 3)[3][0]) == [0, 1, 2]
    a[0, 4] = np.nan
    a[0, 6] = np.inf
    r = O.token_logprobs(a, None, 3)
    assert list(r[3][0]) == [4, 6, 0] and np.isnan(r[2][0])


@pytest.mark.parametrize("dim", [64, 128])
def test_attention_bound_covers_binary32(dim):
    """The bound holds for a binary32 evaluation whose weights are rounded to fp16."""
    rng = np.random.default_rng(3)
    q = rng.normal(size=(4, dim)).astype(np.float16).astype(np.float64) * 1.5
    k, v = rng.normal(size=(300, dim)), rng.normal(size=(300, dim))
    k, v = k.astype(np.float16).astype(np.float64), v.astype(np.float16).astype(np.float64)
    sc = dim ** -0.5
    out, lse, to, tl = O.attention(q, k, v, 296, sc)
    for i in range(4):
        s = np.float32(sc) * (k[:297 + i].astype(np.float32) @ q[i].astype(np.float32))
        p = np.exp(s - s.max())
        o = (p.astype(np.float16).astype(np.float32) @ v[:297 + i].astype(np.float32)) / p.sum()
        assert (np.abs(o - out[i]) <= to[i]).all()
        assert abs(s.max() + np.log(p.sum()) - lse[i]) <= tl[i]
