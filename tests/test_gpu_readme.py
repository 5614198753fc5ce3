"""The README's lines for positions and drafted tokens, run as they stand: every query is turned once."""
import re
from pathlib import Path

import numpy as np
import pytest
import torch

from oracle import operators as O
from tests.kv_helpers import batch

pytestmark = pytest.mark.gpu

ROOT = Path(__file__).resolve().parents[1]


@pytest.fixture(scope="module")
def pi():
    import __graft_entry__
    __graft_entry__.build()
    import activation_sparse_rank_gb300 as pi
    return pi


def test_positions_and_drafted_tokens(pi):
    text = (ROOT / "README.md").read_text()
    lines, = [b for b in re.findall(r"```python\n(.*?)```", text, re.S) if "pi.Rotary(" in b]
    rng, g = np.random.default_rng(0), torch.Generator().manual_seed(0)

    def ints(v):
        return torch.tensor(np.asarray(v, np.int32), device="cuda")

    # as many nodes as prompt tokens, of the same queries, keys and values: the lines may share names
    start, new, vocab = [20, 3], [5, 9], 50
    tree = [-1 if i == 0 else int(rng.integers(i)) for m in new for i in range(m)]
    b = batch(start, [2 * m for m in new], 64)
    cache, d, n = pi.KVCache(b["pages"], 8, 128), b["dev"], sum(new)
    q, k, v = (torch.randn(n, h, 128, generator=g).half().cuda() for h in (64, 8, 8))
    cu = ints([0, *np.cumsum(new)])
    target, draft = (torch.softmax(torch.randn(n, vocab, generator=g), 1).cuda() for _ in range(2))
    u = torch.rand(n, generator=g).cuda()
    names = dict(pi=pi, torch=torch, cache=cache, q=q.clone(), k=k, v=v, node_q=q.clone(), node_k=k, node_v=v, page_table=d["table"],
                 cu_tokens=cu, cu_nodes=cu, start=d["start"], new=ints(new), nodes=ints(new), length=d["start"] + ints(new),
                 parent=ints(tree), seq=ints(np.repeat([0, 1], new)), tokens=ints(rng.integers(0, vocab, n)), target=target, draft=draft,
                 u_accept=u, u_sample=u[:2].clone())
    exec(lines, names)
    assert cache.device_status() == 0
    # the tree's step from the operators one by one; its keys are in the cache
    bits, depth = O.draft_tree(tree, cu.tolist(), 16)
    at = names["length"]
    turned = pi.rotary(q, at[names["seq"]] + ints(depth), names["rope"])
    want = cache.attention(turned, d["table"], cu, at + ints(new), max_q=16, tree=names["mask"])
    assert torch.equal(names["out"], want)
    f = lambda t: t.double().cpu().numpy()
    r = O.verify_draft(f(target), f(draft), names["tokens"].tolist(), tree, cu.tolist(), f(u), f(u[:2]), 16)
    for got, w in zip(names["r"], r):
        np.testing.assert_array_equal(got.cpu().numpy(), w)
