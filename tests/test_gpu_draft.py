"""Trees of drafted tokens and their verification: whole numbers, equal to the float64 definition's."""
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


def ints(v):
    return torch.tensor(np.asarray(v, np.int32), device="cuda")


def floats(v):
    return torch.tensor(np.asarray(v, np.float32), device="cuda")


def forest(rng, new, branch):
    """Parents, packed: a node hangs on one of the `branch` nodes before it."""
    return [-1 if i == 0 else i - 1 - int(rng.integers(min(i, branch))) for m in new for i in range(m)]


def same_tree(pi, parent, cu, max_q):
    mask, depth = pi.draft_tree(ints(parent), ints(cu), max_q)
    want, deep = O.draft_tree(parent, cu, max_q)
    words = mask.cpu().numpy().view(np.uint32)
    bits = (words[:, :, None] >> np.arange(32)) & 1
    np.testing.assert_array_equal(bits.reshape(len(parent), -1).astype(bool), want)
    np.testing.assert_array_equal(depth.cpu().numpy(), deep)


@pytest.mark.parametrize("max_q", [1, 2, 31, 32, 33, 64, 65, 255, 256])
@pytest.mark.parametrize("branch", [1, 3, 300])
def test_trees(pi, max_q, branch):
    rng = np.random.default_rng(max_q)
    new = [max_q, 0, 1, max(1, max_q // 2), max_q, 0]
    same_tree(pi, forest(rng, new, branch), np.concatenate([[0], np.cumsum(new)]), max_q)


def test_trees_past_max_q_and_bad_parents(pi):
    parent = [-1, 0, 1, 2, 3, 4] + [0, 1, 1, -7, 1 << 30] + [-1]
    same_tree(pi, parent, [0, 6, 11, 12], 4)
    same_tree(pi, parent, [0, 6, 11, 12], 40)


def test_trees_bad_rows_are_left(pi):
    """A falling or too large entry of cu skips its sequences; the others are done, and rows of no sequence stay."""
    parent, cu = ints([-1, 0, 0, 2, -1, 0]), ints([0, 2, 99, 3, 5])
    pi.draft_tree(parent, cu, 3)
    lib, mask, depth = pi.lib, torch.full((6, 1), 77, dtype=torch.int32, device="cuda"), torch.full((6,), 77, dtype=torch.int32, device="cuda")
    assert lib.pi_draft_tree(parent.data_ptr(), cu.data_ptr(), 4, 6, 3, mask.data_ptr(), depth.data_ptr(), 0) == 0
    torch.cuda.synchronize()
    assert depth.tolist() == [0, 1, 77, 0, 0, 77] and mask.flatten().tolist() == [1, 3, 77, 1, 2, 77]


# ---- verification -------------------------------------------------------------------


def rows(rng, n, vocab, sharp=2.0):
    x = rng.standard_normal((n, vocab)) * sharp
    p = np.exp(x - x.max(1, keepdims=True))
    p /= p.sum(1, keepdims=True)
    y = x + rng.standard_normal((n, vocab)) * 0.7
    q = np.exp(y - y.max(1, keepdims=True))
    return p, q / q.sum(1, keepdims=True)


def case(rng, new, vocab, branch, dtype, with_draft=True, sharp=2.0):
    n = sum(new)
    p, q = rows(rng, n, vocab, sharp)
    p, q = (torch.tensor(t).to(TORCH[dtype]) for t in (p, q))
    parent = forest(rng, new, branch)
    cu = np.concatenate([[0], np.cumsum(new)])
    drawn = np.zeros(n, int)
    for s in range(len(new)):
        for i in range(1, new[s]):
            w = (q if with_draft else p)[cu[s] + parent[cu[s] + i]].double().numpy()
            drawn[cu[s] + i] = rng.choice(vocab, p=w / w.sum()) if with_draft else int(np.argsort(-w)[i % min(3, vocab)])
    return dict(target=p, draft=q if with_draft else None, drawn=drawn, parent=parent, cu=cu,
                accept=rng.random(n).astype(np.float32), sample=rng.random(len(new)).astype(np.float32), max_q=max(new + [1]))


def run(pi, c, **kw):
    cuda = dict(target=c["target"].cuda(), draft=None if c["draft"] is None else c["draft"].cuda())
    cuda.update(kw)
    return pi.verify_draft(cuda["target"], cuda["draft"], ints(c["drawn"]), ints(c["parent"]), ints(c["cu"]), floats(c["accept"]),
                           floats(c["sample"]), c["max_q"])


def oracle(c):
    f = lambda t: None if t is None else t.double().numpy()
    return O.verify_draft(f(c["target"]), f(c["draft"]), c["drawn"], c["parent"], c["cu"], c["accept"].astype(np.float64),
                          c["sample"].astype(np.float64), c["max_q"])


def same(got, want):
    for g, w, name in zip(got, want, ("accepted", "path", "token")):
        np.testing.assert_array_equal(g.cpu().numpy(), w, err_msg=name)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("with_draft", [True, False])
@pytest.mark.parametrize("new,vocab,branch", [([5], 50007, 1), ([1], 3, 1), ([8, 1, 0, 3, 7], 1000, 3), ([33, 12], 257, 4),
                                              ([6] * 40, 515, 2), ([256, 2], 64, 30), ([4] * 400, 33, 2), ([9, 9], 131072, 9)])
def test_verify(pi, dtype, with_draft, new, vocab, branch):
    rng = np.random.default_rng(vocab + branch)
    c = case(rng, new, vocab, branch, dtype, with_draft)
    same(run(pi, c), oracle(c))


@pytest.mark.parametrize("reject", [0, 1, 2, 5])
def test_many_rejections_at_a_node(pi, reject):
    """A star: the first `reject` children are refused whatever they are, the others as they come."""
    rng = np.random.default_rng(reject)
    c = case(rng, [8, 8, 8], 700, 1, "float32")
    c["parent"] = [-1] + [0] * 7 + [-1] + [0] * 7 + [-1] + [0] * 7
    c["accept"][[1 + i + 8 * s for s in range(3) for i in range(reject)]] = 1.0
    c["drawn"][9:] = rng.integers(0, 700, 15)
    same(run(pi, c), oracle(c))


def test_exact_ties(pi):
    """Powers of two: equal sides refuse, and a sum that equals its share goes on to the next token."""
    p = torch.tensor([[0.5, 0.25, 0.25, 0.0]] * 3)
    q = torch.tensor([[0.25, 0.5, 0.25, 0.0]] * 3)
    for a, u, two in [(0.5, 0.5, 1), (0.49, 0.75, 1), (0.5, 0.0, 2), (0.25, 0.999, 2), (1.0, 0.25, 0), (1.0, 0.0, 0)]:
        c = dict(target=p, draft=q, drawn=np.array([0, 1, two]), parent=[-1, 0, 0], cu=[0, 3], max_q=3,
                 accept=np.array([0, a, a], np.float32), sample=np.array([u], np.float32))
        same(run(pi, c), oracle(c))
        c["draft"] = None
        same(run(pi, c), oracle(c))


def test_smallest_numbers(pi):
    """The first token of any probability is taken for 0, however small it is; zeros and what the draft covers are not."""
    p = torch.zeros(4, 9)
    p[:, 4], p[:, 6], p[:, 8] = 1e-44, 1e-30, 1.0
    q = torch.zeros(4, 9)
    q[:, 4], q[:, 8] = 1e-40, 0.5
    c = dict(target=p, draft=q, drawn=np.array([0, 0, 4, 7]), parent=[-1, -1, 0, 0], cu=[0, 1, 2, 4], max_q=4,
             accept=np.ones(4, np.float32), sample=np.zeros(3, np.float32))
    got = run(pi, c)
    assert got.token.tolist() == [4, 4, 6] and got.accepted.tolist() == [0, 0, 0]


def test_what_is_no_distribution(pi):
    """Draft equal to target and refused; rows of zeros, NaN and negative numbers; tokens outside the vocabulary."""
    nan = float("nan")
    p = torch.tensor([[0.5, 0.25, 0.25, 0.0], [0.0, 0.0, 0.0, 0.0], [nan, -1.0, 0.25, nan], [nan] * 4, [0.5, 0.5, 0.0, 0.0],
                      [0.0, 0.0, 1.0, 0.0]])
    c = dict(target=p, draft=p, drawn=np.array([9, 0, 0, 0, 0, -1]), parent=[-1, -1, -1, -1, -1, 0], cu=[0, 1, 2, 3, 4, 6], max_q=2,
             accept=np.ones(6, np.float32), sample=np.full(5, 0.75, np.float32))
    got = run(pi, c)
    same(got, oracle(c))
    assert got.token.tolist() == [2, -1, 2, -1, 1]
    c["drawn"][5] = 4
    for draft in (p, None):
        c["draft"] = draft
        assert run(pi, c).accepted.tolist() == [0] * 5


@pytest.mark.parametrize("vocab", [1, 2, 31, 127, 128, 129, 4095, 4097, 300001])
def test_vocabularies(pi, vocab):
    """Rows around the pieces that warps share, and wider than usual."""
    rng = np.random.default_rng(vocab)
    for dtype in ("float32", "bfloat16"):
        c = case(rng, [3, 2], vocab, 2, dtype)
        same(run(pi, c), oracle(c))


def test_two_calls_at_once_and_another_stream(pi):
    """Calls on two streams that overlap: no state is shared."""
    rng = np.random.default_rng(8)
    cases = [case(rng, [5] * 30, 30011, 2, "float32") for _ in range(2)]
    tensors = [(c["target"].cuda(), c["draft"].cuda(), ints(c["drawn"]), ints(c["parent"]), ints(c["cu"]), floats(c["accept"]),
                floats(c["sample"])) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(8):
        for i, s in enumerate(streams):
            got[i].append(pi.verify_draft(*tensors[i], 5, stream=s))
    torch.cuda.synchronize()
    for c, results in zip(cases, got):
        want = oracle(c)
        for r in results:
            same(r, want)


@pytest.mark.parametrize("offset", [1, 2, 3])
def test_strides(pi, offset):
    """Rows that begin anywhere, target and draft not alike."""
    rng = np.random.default_rng(offset)
    c = case(rng, [7, 2, 5], 1301, 3, "bfloat16")
    wide = torch.zeros(14, 1301 + 9, dtype=torch.bfloat16)
    wide[:, offset:offset + 1301] = c["target"]
    same(run(pi, c, target=wide.cuda()[:, offset:offset + 1301]), oracle(c))


def test_rows_past_max_q_and_nodes_that_hang_nowhere(pi):
    rng = np.random.default_rng(1)
    c = case(rng, [9, 6], 50, 1, "float32")
    c["accept"][:] = 0.0                              # everything that may be is accepted
    c["max_q"] = 4
    same(run(pi, c), oracle(c))
    c["parent"][2] = -1
    same(run(pi, c), oracle(c))


@pytest.mark.parametrize("with_draft", [True, False])
def test_tokens_are_distributed_as_the_target(pi, with_draft):
    """The first token that comes out, of 40000 sequences with two drafted children, has the target's
    distribution: a share's standard deviation is sqrt(p (1 - p) / n), 5.5 of them are allowed."""
    rng = np.random.default_rng(4)
    n, vocab = 40000, 7
    p, q = rows(rng, 1, vocab, 1.0)
    g = torch.Generator().manual_seed(1)
    drawn = torch.zeros(n, 3, dtype=torch.int32)
    drawn[:, 1:] = torch.multinomial(torch.tensor(q[0]), 2 * n, replacement=True, generator=g).view(n, 2).int() if with_draft else torch.tensor([2, 5])
    target = torch.tensor(p, dtype=torch.float32).expand(3 * n, vocab).contiguous()
    draft = torch.tensor(q, dtype=torch.float32).expand(3 * n, vocab).contiguous() if with_draft else None
    c = dict(target=target, draft=draft, drawn=drawn.flatten().numpy(), parent=[-1, 0, 0] * n, cu=np.arange(n + 1) * 3, max_q=3,
             accept=torch.rand(3 * n, generator=g).numpy(), sample=torch.rand(n, generator=g).numpy())
    got = run(pi, c)
    took = got.path[:, 1].cpu().long()
    first = torch.where(took > 0, drawn.gather(1, took.clamp(min=0)[:, None])[:, 0].long(), got.token.cpu().long())
    share = torch.bincount(first, minlength=vocab).numpy() / n
    assert (np.abs(share - p[0]) <= 5.5 * np.sqrt(p[0] * (1 - p[0]) / n)).all()
    assert 0.3 < (got.accepted > 0).float().mean().item() < 1


def test_stream_graph_and_refusals(pi):
    rng = np.random.default_rng(2)
    c = case(rng, [5, 8, 2], 5001, 2, "float32")
    want = oracle(c)
    side = torch.cuda.Stream()
    t, q, x, up, cu, a, u = (c["target"].cuda(), c["draft"].cuda(), ints(c["drawn"]), ints(c["parent"]), ints(c["cu"]),
                             floats(c["accept"]), floats(c["sample"]))
    side.wait_stream(torch.cuda.current_stream())
    got = pi.verify_draft(t, q, x, up, cu, a, u, 8, stream=side)
    side.synchronize()
    same(got, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = pi.verify_draft(t, q, x, up, cu, a, u, 8)
    for seed in (0, 5):
        c["sample"] = np.random.default_rng(seed).random(3).astype(np.float32)
        c["accept"] = np.random.default_rng(seed).random(15).astype(np.float32)
        u.copy_(floats(c["sample"]))
        a.copy_(floats(c["accept"]))
        g.replay()
        same(out, oracle(c))
    for bad in (lambda: pi.verify_draft(t, q[:, :9], x, up, cu, a, u, 8), lambda: pi.verify_draft(t, q.half(), x, up, cu, a, u, 8),
                lambda: pi.verify_draft(t[:9], q[:9], x, up, cu, a, u, 8), lambda: pi.verify_draft(t, q, x.long(), up, cu, a, u, 8),
                lambda: pi.verify_draft(t, q, x, up[:9], cu, a, u, 8), lambda: pi.verify_draft(t, q, x, up, cu, a, u[:2], 8),
                lambda: pi.verify_draft(t, q, x, up, cu, a.double(), u, 8), lambda: pi.verify_draft(t, q, x, up, cu, a, u, 300),
                lambda: pi.verify_draft(t.t(), q, x, up, cu, a, u, 8), lambda: pi.draft_tree(up, cu, 0),
                lambda: pi.draft_tree(up.cpu(), cu, 8), lambda: pi.draft_tree(up, cu.long(), 8),
                lambda: pi.draft_tree(torch.zeros(300, dtype=torch.int32, device="cuda"), cu)):
        with pytest.raises((ValueError, TypeError)):
            bad()
    none = pi.verify_draft(t[:0], None, x[:0], up[:0], ints([0, 0, 0]), a[:0], u[:2])
    assert none.accepted.tolist() == [0, 0] and none.token.tolist() == [-1, -1] and none.path.tolist() == [[-1], [-1]]
