"""Given tokens (no draft) with many refusals at a node: each takes its own share of the target along, once."""
import numpy as np
import pytest
import torch

from tests.test_gpu_draft import oracle, rows, run, same
from tests.kv_helpers import TORCH

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pi():
    import __graft_entry__
    __graft_entry__.build()
    import activation_sparse_rank_gb300 as pi
    return pi


@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("vocab", [300, 50007, 131072])
@pytest.mark.parametrize("children,sequences", [(1, 3), (40, 2), (255, 1)])
def test_stars(pi, dtype, vocab, children, sequences):
    """All children refused; some tokens twice, some outside the vocabulary; sampled early, late and between."""
    rng = np.random.default_rng(vocab + children)
    n = 1 + children
    p = torch.tensor(np.tile(rows(rng, 1, vocab, 1.5)[0], (n * sequences, 1))).to(TORCH[dtype])
    likely = torch.argsort(p[0].double(), descending=True).numpy()
    drawn = np.zeros((sequences, n), int)
    for s in range(sequences):
        drawn[s, 1:] = np.where(rng.random(children) < 0.5, likely[rng.integers(0, min(vocab, 40), children)], rng.integers(-1, vocab + 1, children))
    for u in (0.0, 0.37, 0.99999):
        c = dict(target=p, draft=None, drawn=drawn.flatten(), parent=([-1] + [0] * children) * sequences, cu=np.arange(sequences + 1) * n,
                 max_q=n, accept=np.full(n * sequences, np.float32(1 - 2.0 ** -24)), sample=np.full(sequences, u, np.float32))
        got = run(pi, c)
        same(got, oracle(c))
        assert not got.accepted.any() and not any(t in d for t, d in zip(got.token.tolist(), drawn[:, 1:]))


def test_refusals_after_an_accepted_token(pi):
    """The list of a node's refused tokens is its own: another node's sample may take them."""
    rng = np.random.default_rng(3)
    vocab, n = 1003, 60
    p = torch.tensor(rows(rng, n, vocab, 0.5)[0]).float()
    p[0] = 0.0
    p[0, :30] = 1 / 64
    p[0, 30] = 34 / 64
    p[20] = 0.0
    p[20, :20] = 1 / 32                                  # tokens refused at the root are all that node 20 has, but for one
    p[20, 700] = 12 / 32
    parent = [-1] + [0] * 20 + [20] * 39
    drawn = np.concatenate([[0], np.arange(19), [30], 100 + np.arange(39)])
    accept = np.full(n, np.float32(1 - 2.0 ** -24))
    accept[20] = 0.25                                    # 34 / 64 of the root
    for u in (0.0, 0.3, 0.6, 0.7, 0.99):
        c = dict(target=p, draft=None, drawn=drawn, parent=parent, cu=[0, n], max_q=n, accept=accept, sample=np.array([u], np.float32))
        got = run(pi, c)
        same(got, oracle(c))
        assert got.accepted.tolist() == [1] and got.path[0, 1].item() == 20
