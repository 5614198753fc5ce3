"""Log-probabilities of rows whose largest logit is the type's lowest value, or so large that 140 less rounds to it."""
import numpy as np
import pytest
import torch

from oracle import operators as O
from tests.kv_helpers import TORCH

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pi():
    import __graft_entry__
    __graft_entry__.build()
    import activation_sparse_rank_gb300 as pi
    return pi


def hard_rows(vocab, dtype):
    """Banned tokens as the type's lowest value and as -inf, additive masks and logits of any size."""
    info = torch.finfo(TORCH[dtype])
    far = 6e4 if dtype == "float16" else 1e10
    j = torch.arange(vocab)

    def row(*parts):
        x = torch.full((vocab,), parts[0], dtype=torch.float64)
        for where, value in parts[1:]:
            x[where] = value
        return x

    few = j < 10
    return torch.stack([
        row(info.min),
        row(info.min, (j % 2 == 1, -torch.inf)),
        row(-torch.inf, (few, info.min)),
        row(-torch.inf, (j == vocab - 1, info.min)),
        row(-torch.inf, (j == vocab // 2, info.max)),
        row(info.min, (j == 0, info.max)),
        row(0.0, (j == vocab // 3, far)),
        row(-info.max / 2, (j == vocab // 3, -info.max / 4)),
        row(-2e10 if far == 1e10 else info.min, (j == vocab // 2, -far)),
        row(info.min, (j % 7 == 0, info.min + 64 if dtype == "float16" else -1e5)),
        row(info.max),
        row(-torch.inf, (j % 3 == 0, far)),
        row(info.min, (few, 1.0), (j == 3, 2.5)),
    ]).to(TORCH[dtype])


def check(pi, x, k):
    t = torch.arange(x.shape[0], dtype=torch.int32) % x.shape[1]
    r = pi.token_logprobs(x.cuda(), t.cuda(), top_k=k)
    xd = x.double().numpy()
    logp, ent, lse, idx, val, _ = O.token_logprobs(xd, t.numpy(), k)
    tols = O.score_bounds(xd, np.where(np.isfinite(logp), logp, 0.0), ent, lse)
    for got, want, tol, name in zip((r.entropy, r.lse, r.logprob), (ent, lse, logp), tols, ("entropy", "lse", "logprob")):
        got = got.double().cpu().numpy()
        with np.errstate(invalid="ignore", over="ignore"):
            want = np.where(np.abs(want) > torch.finfo(torch.float32).max, np.sign(want) * np.inf, want)
            ok = (got == want) | (np.isnan(got) & np.isnan(want)) | (np.abs(got - want) <= tol)
        assert ok.all(), (name, np.flatnonzero(~ok)[:5], got[~ok][:5], want[~ok][:5], tol[~ok][:5])
    if k:
        np.testing.assert_array_equal(r.top_index.cpu().numpy(), idx)
    return r


@pytest.mark.parametrize("dtype", ["float16", "bfloat16", "float32"])
@pytest.mark.parametrize("vocab", [1, 3, 1003, 2000, 40001, 131072])
def test_few_rows(pi, dtype, vocab):
    x = hard_rows(vocab, dtype)
    r = check(pi, x, min(5, vocab))
    if vocab > 1:
        assert r.entropy[3] == 0 and r.logprob[3] == -torch.inf
        assert r.entropy[4] == 0 and r.entropy[6] == 0


@pytest.mark.parametrize("dtype", ["float16", "bfloat16", "float32"])
@pytest.mark.parametrize("vocab", [515, 9001, 70003])
def test_many_rows(pi, dtype, vocab):
    """The same among ordinary rows, more of them than the GPU has SMs."""
    g = torch.Generator().manual_seed(vocab)
    x = (torch.randn(330, vocab, generator=g) * 2.5).to(TORCH[dtype])
    hard = hard_rows(vocab, dtype)
    x[5:5 + 20 * len(hard):20] = hard
    check(pi, x, 3)
