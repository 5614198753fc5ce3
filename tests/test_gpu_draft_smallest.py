"""Verification where all that is left of a row is about 2^-60, the step of its sums: what is left is found, however
small, and what is not left is not."""
import numpy as np
import pytest
import torch

from tests.kv_helpers import TORCH
from tests.test_gpu_draft import oracle, run, same

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pi():
    import __graft_entry__
    __graft_entry__.build()
    import activation_sparse_rank_gb300 as pi
    return pi


SMALL = [2.0 ** -60, 1.5 * 2.0 ** -61, 2.0 ** -61 * (1 + 2.0 ** -7), 2.0 ** -61, 2.0 ** -61 * (1 - 2.0 ** -8), 2.0 ** -62, 2.0 ** -100]


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("small", SMALL)
@pytest.mark.parametrize("vocab,at", [(2, 1), (9, 4), (515, 514), (30011, 17000), (30011, 1)])
def test_one_token_left(pi, dtype, small, vocab, at):
    """After a refusal (drawn and given), after two, and where the row itself has no more."""
    p = torch.zeros(4, vocab, dtype=torch.float64)
    p[:, at] = small
    p[:3, 0] = 0.5
    q = torch.zeros(4, vocab, dtype=torch.float64)
    q[:, 0] = 1.0
    p, q = p.to(TORCH[dtype]), q.to(TORCH[dtype])
    assert (p[:, at].double() == small).all()            # both types hold it
    for sample in (0.0, 0.5, 0.99):
        c = dict(target=p, draft=q, drawn=np.zeros(4, int), parent=[-1, 0, 0, -1], cu=[0, 3, 4], max_q=3,
                 accept=np.full(4, 0.75, np.float32), sample=np.full(2, sample, np.float32))
        for c["draft"], c["parent"] in ((q, [-1, 0, 0, -1]), (q, [-1, 0, -1, -1])):
            got = run(pi, c)
            same(got, oracle(c))
            assert got.token.tolist() == [at, at] and got.accepted.tolist() == [0, 0]
        # a given token is refused for numbers above its probability
        c["draft"] = None
        got = run(pi, c)
        same(got, oracle(c))
        assert got.token.tolist() == [at, at]


def test_nothing_left(pi):
    """Draft and target alike: nothing is left of 2^-61 either, and the next token is the target's own."""
    p = torch.tensor([[0.5, 2.0 ** -61, 0.0]] * 2)
    c = dict(target=p, draft=p, drawn=np.array([0, 2]), parent=[-1, 0], cu=[0, 2], max_q=2, accept=np.full(2, 0.5, np.float32),
             sample=np.zeros(1, np.float32))
    got = run(pi, c)
    same(got, oracle(c))
    assert got.token.tolist() == [0] and got.accepted.tolist() == [0]
