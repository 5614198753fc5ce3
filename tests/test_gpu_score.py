"""Log-probabilities, entropy and top tokens against their float64 definition."""
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


def logits(rows, vocab, dtype, seed=0, std=2.5):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(rows, vocab, generator=g) * std).to(TORCH[dtype]).cuda()


@np.errstate(invalid="ignore")
def check(pi, x, t, k):
    r = pi.token_logprobs(x, None if t is None else torch.tensor(t, dtype=torch.int32, device="cuda"), top_k=k)
    logp, ent, lse, idx, val, tol = O.token_logprobs(x.double().cpu().numpy(), t, k)
    with np.errstate(over="ignore"):                 # a difference past binary32's range is infinite there
        logp, val = (v.astype(np.float32).astype(np.float64) for v in (logp, val))
    for got, want, name in ((r.entropy, ent, "entropy"), (r.lse, lse, "lse")) + (() if t is None else ((r.logprob, logp, "logprob"),)):
        got = got.double().cpu().numpy()
        ok = (got == want) | (np.isnan(got) & np.isnan(want)) | (np.abs(got - want) <= tol)
        assert ok.all(), (name, got[~ok][:4], want[~ok][:4], tol[~ok][:4])
    if k:
        np.testing.assert_array_equal(r.top_index.cpu().numpy(), idx)
        got = r.top_logprob.double().cpu().numpy()
        ok = (got == val) | (np.isnan(got) & np.isnan(val)) | (np.abs(got - val) <= tol[:, None])
        assert ok.all(), (got[~ok][:4], val[~ok][:4])
    return r


@pytest.mark.parametrize("dtype", ["float16", "bfloat16", "float32"])
@pytest.mark.parametrize("rows,vocab,k", [(1, 1, 1), (3, 5, 5), (2, 500, 0), (4, 1001, 20), (7, 32000, 5), (2, 50007, 64),
                                          (1, 131072, 20), (40, 4096, 1), (1, 150001, 32), (300, 777, 3)])
def test_values(pi, dtype, rows, vocab, k):
    x = logits(rows, vocab, dtype, seed=vocab)
    rng = np.random.default_rng(1)
    check(pi, x, rng.integers(0, vocab, rows), k)


@pytest.mark.parametrize("dtype,vocab,k", [("float16", 17003, 20), ("bfloat16", 40000, 64), ("float32", 9001, 5), ("bfloat16", 33001, 0)])
def test_many_rows(pi, dtype, vocab, k):
    """More rows than the GPU has places for, with ties, masks and special rows among them."""
    x = logits(307, vocab, dtype, seed=k)
    x[3] = 2.0
    x[4] = -torch.inf
    x[5, 1000:] = -torch.inf
    x[7] = torch.round(x[7])
    x[9, vocab - 1] = torch.nan
    x[11, 0] = torch.inf
    x[13] = torch.linspace(-90, 90, vocab).to(x.dtype)
    x[15] = torch.linspace(90, -90, vocab).to(x.dtype)
    x[17, :-1] = -torch.inf
    rng = np.random.default_rng(1)
    check(pi, x, rng.integers(0, vocab, 307), k)


@pytest.mark.parametrize("vocab", [40, 1003, 40000, 131072])
def test_ties(pi, vocab):
    """Equal logits: everywhere, in coarse steps, at the border of the top k, zeros of both signs."""
    x = logits(6, vocab, "float32")
    x[0] = 1.5
    x[1] = torch.round(x[1])
    x[2] = torch.where(torch.arange(vocab, device="cuda") % 3 == 0, 2.0, 1.0)
    x[3] = torch.where(torch.arange(vocab, device="cuda") % 2 == 0, -0.0, 0.0)
    x[4] = torch.arange(vocab, device="cuda").float() / vocab
    x[5] = -torch.arange(vocab, device="cuda").float() / vocab
    for dtype in (torch.float32, torch.bfloat16):
        check(pi, x.to(dtype), [0, 1, 2, 3, 4, 5], min(33, vocab))


@pytest.mark.parametrize("dtype", ["float16", "bfloat16", "float32"])
def test_masked_and_special_rows(pi, dtype):
    """Banned tokens (-inf, the type's lowest), all banned but one, all banned, NaN, +inf; padding and bad targets."""
    v = 2000
    x = logits(10, v, dtype)
    low = torch.finfo(TORCH[dtype]).min
    x[0, ::2] = -torch.inf
    x[1, ::2] = low
    x[2] = -torch.inf
    x[2, 77] = 3.0
    x[3] = -torch.inf
    x[4] = low
    x[5, 9] = torch.nan
    x[6, 9] = torch.inf
    x[7] = low
    x[7, 5] = torch.finfo(TORCH[dtype]).max
    r = check(pi, x, [0, 1, 77, 5, 5, 5, 9, 5, -1, v], 7)
    assert r.logprob[0] == -torch.inf and r.logprob[2] == 0 and r.entropy[2] == 0
    assert r.logprob[8] == 0 and torch.isnan(r.logprob[9]) and torch.isfinite(r.entropy[8:]).all()


def test_wide_range(pi):
    """Logits far apart and far from 0: sums relative to the running maximum."""
    x = logits(4, 30000, "float32")
    x[0] += 3e4
    x[1] *= 50
    x[2] = torch.linspace(-1000, 1000, 30000)        # the maximum moves all the time
    x[3] = torch.linspace(1000, -1000, 30000)
    check(pi, x, [5, 6, 29999, 0], 4)


def test_strided_rows(pi):
    wide = logits(5, 4096, "float16")
    for at in (0, 8, 3):
        x = wide[:, at:at + 1001]
        check(pi, x, [0, 1, 2, 3, 1000], 6)
    x = wide[::2, :1000]
    check(pi, x, [0, 1, 2], 6)
    r = pi.token_logprobs(wide[:0], torch.zeros(0, dtype=torch.int32, device="cuda"), top_k=3)
    assert r.logprob.numel() == 0 and r.top_index.shape == (0, 3)


def test_without_targets(pi):
    check(pi, logits(3, 999, "bfloat16"), None, 2)


def test_repeats_other_stream_and_graph(pi):
    x = logits(20, 30011, "bfloat16")
    t = torch.arange(20, dtype=torch.int32, device="cuda")
    a = pi.token_logprobs(x, t, top_k=9)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    b = pi.token_logprobs(x, t, top_k=9, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c = pi.token_logprobs(x, t, top_k=9)
    g.replay()
    for u, v, w in zip(a, b, c):
        assert torch.equal(u, v) and torch.equal(u, w)


def test_refusals(pi):
    x = logits(3, 50, "float16")
    t = torch.zeros(3, dtype=torch.int32, device="cuda")
    with pytest.raises(TypeError):
        pi.token_logprobs(x.double(), t)
    with pytest.raises(TypeError):
        pi.token_logprobs(x.cpu(), t)
    with pytest.raises(TypeError):
        pi.token_logprobs(x, t.long())
    with pytest.raises(ValueError):
        pi.token_logprobs(x, t[:2])
    with pytest.raises(ValueError):
        pi.token_logprobs(x.t(), t)
    for k in (-1, 51, 65):
        with pytest.raises(pi.PiError):
            pi.token_logprobs(x, t, top_k=k)
