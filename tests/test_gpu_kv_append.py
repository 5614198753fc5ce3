"""Tokens appended one at a time to blocks that hold others: every lane of a block sees the scale that it had."""
import pytest
import torch

from tests.kv_helpers import TORCH, batch, oracle_of, random_cache, same_cache

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pi():
    import __graft_entry__
    __graft_entry__.build()
    import activation_sparse_rank_gb300 as pi
    return pi


@pytest.mark.parametrize("dtype", ["float16", "bfloat16", "float32"])
@pytest.mark.parametrize("dim", [64, 96, 128, 256])
def test_scales_that_grow_and_stay(pi, dtype, dim):
    """Magnitudes from 2^-10 to 2^10 in any order: a block's scale grows at some tokens and stays at the others."""
    seqs, heads, page, n = 7, 5, 32, 21
    start = [0, 1, 15, 16, 17, 31, 8]
    b = batch(start, [n] * seqs, page, seed=dim)
    c = random_cache(pi, b["pages"], heads, dim, page)
    ref = oracle_of(c)
    g = torch.Generator().manual_seed(dim)
    table, cu = b["dev"]["table"], torch.arange(seqs + 1, dtype=torch.int32, device="cuda")
    for i in range(n):
        at = torch.tensor([s + i for s in start], dtype=torch.int32, device="cuda")
        k, v = ((torch.randn(seqs, heads, dim, generator=g) *
                 torch.exp2(torch.randint(-10, 11, (seqs, heads, 1), generator=g))).to(TORCH[dtype]).cuda() for _ in range(2))
        c.write(k, v, table, cu, at)
        ref.write(k.double().cpu().numpy(), v.double().cpu().numpy(), b["table"], cu.tolist(), at.tolist())
    same_cache(c, ref)
    assert c.device_status() == 0
