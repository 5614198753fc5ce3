"""Drafted tokens appended into a block that has been begun, then the accepted ones over them: the cache is that of the
same writes one after the other, codes and scales, and a scale that a refused token raised stays raised."""
import numpy as np
import pytest
import torch

from oracle import operators as O
from tests.kv_helpers import TORCH, batch, oracle_of, same_cache

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pi():
    import __graft_entry__
    __graft_entry__.build()
    import activation_sparse_rank_gb300 as pi
    return pi


def ints(v):
    return torch.tensor(np.asarray(v, np.int32), device="cuda")


@pytest.mark.parametrize("dtype", ["float16", "bfloat16", "float32"])
@pytest.mark.parametrize("heads,dim,page", [(1, 64, 16), (3, 96, 48), (2, 128, 64), (1, 256, 32)])
@pytest.mark.parametrize("size", [1e-3, 1.0, 300.0])
def test_refused_tokens_leave_their_scale(pi, dtype, heads, dim, page, size):
    rng, g = np.random.default_rng(dim), torch.Generator().manual_seed(dim)
    rope, c = pi.Rotary(dim, base=1000.0), pi.KVCache(60, heads, dim, page)
    length, parent = [3, 16, 30, 8], [-1, 0, 0, 1, 2, 4, 0]
    nodes, S = len(parent), len(length)
    b = batch(length, [60] * S, page)
    table, ref = b["dev"]["table"], oracle_of(c)

    def append(lengths, new, k, v, positions):
        cu = np.concatenate([[0], np.cumsum(new)])
        c.append(k, v, table, ints(cu), ints(lengths), rope, positions=ints(positions))
        turned = pi.rotary(k.float(), ints(positions), rope)
        ref.write(*(t.double().cpu().numpy() for t in (turned, v)), b["table"], cu, lengths)
        same_cache(c, ref)

    def rows(n, by):
        return ((torch.randn(n, heads, dim, generator=g) * by).to(TORCH[dtype]).cuda() for _ in range(2))

    append([0] * S, length, *rows(sum(length), 1.0), [i for n in length for i in range(n)])
    depth = O.draft_tree(parent * S, np.arange(S + 1) * nodes, nodes)[1]
    for step in range(4):
        k, v = rows(nodes * S, size)
        at = np.repeat(length, nodes) + depth
        before = c.k_scales.clone(), c.v_scales.clone()
        append(length, [nodes] * S, k, v, at)
        # the root and a way down of any length, over the tree's place; the others are refused
        took = [[0, 2, 4, 5][:int(rng.integers(1, 5))] for _ in range(S)]
        raised = c.k_scales.clone(), c.v_scales.clone()
        keep = np.concatenate([[s * nodes + j for j in way] for s, way in enumerate(took)])
        append(length, [len(way) for way in took], k[torch.from_numpy(keep).cuda()], v[torch.from_numpy(keep).cuda()],
               np.concatenate([length[s] + np.arange(len(way)) for s, way in enumerate(took)]))
        for s, n in enumerate(length):
            if n % 16:                                   # the block that the tree met begun
                pg, blk = b["table"][s][n // page], n % page // 16
                for was, up, now in zip(before, raised, (c.k_scales, c.v_scales)):
                    # an accepted token of the next block may come into this one, and raise it further
                    assert (up[pg, :, blk] >= was[pg, :, blk]).all() and (now[pg, :, blk] >= up[pg, :, blk]).all()
                    if size == 300.0 and step == 0:
                        assert (up[pg, :, blk] > was[pg, :, blk]).all()
        length = [n + len(way) for n, way in zip(length, took)]
    assert c.device_status() == 0
