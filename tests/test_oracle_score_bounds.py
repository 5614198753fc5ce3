"""The bounds of the scores' definition (CPU only): each with its own terms, wide enough for binary32."""
import numpy as np

from oracle import operators as O


def rows():
    rng = np.random.default_rng(4)
    x = rng.normal(size=(6, 2000)) * 2.5
    x[1] = -65504.0
    x[2, ::2] = np.finfo(np.float32).min
    x[3] += 1e6
    x[4, 7] = 1e10
    x[5, 1:] = -np.inf
    return x.astype(np.float32)


def test_entropy_bound_has_no_size():
    """Neither an offset nor the type's lowest value widens the entropy's bound."""
    for row in rows().astype(np.float64):
        logp, ent, lse, _, _, _ = O.token_logprobs(row[None], None, 0)
        assert O.score_bounds(row[None], logp, ent, lse)[0] < 1e-4
    x = rows()[:1].astype(np.float64)
    a = O.score_bounds(x, *O.token_logprobs(x, None, 0)[:3])
    b = O.score_bounds(x + 2.0 ** 20, *O.token_logprobs(x + 2.0 ** 20, None, 0)[:3])
    np.testing.assert_allclose(a[0], b[0], rtol=1e-6)
    assert b[1] > a[1]


def test_bounds_cover_binary32():
    x = rows()
    t = np.array([5, 6, 1, 8, 7, 0])
    logp, ent, lse, _, _, _ = O.token_logprobs(x, t, 0)
    te, tl, tp = O.score_bounds(x, logp, ent, lse)
    m = x.max(1, keepdims=True)
    with np.errstate(invalid="ignore", over="ignore"):
        z = x - m
        e = np.exp(z)
        total = e.sum(1, dtype=np.float32)
        got_l = m[:, 0] + np.log(total)
        got_e = np.log(total) - np.where(e > 0, e * np.where(e > 0, z, 0), 0).sum(1, dtype=np.float32) / total
    got_p = x[np.arange(6), t] - got_l
    for got, want, tol in ((got_e, ent, te), (got_l, lse, tl), (got_p, logp, tp)):
        assert got.dtype == np.float32 and (np.abs(got - want) <= tol).all()
