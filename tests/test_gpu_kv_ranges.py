"""Reading with row ranges that leave rows to no sequence, or that do not ascend."""
import numpy as np
import pytest
import torch

from tests.kv_helpers import oracle_of, random_cache

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pi():
    import __graft_entry__
    __graft_entry__.build()
    import activation_sparse_rank_gb300 as pi
    return pi


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("heads,dim", [(1, 64), (40, 128)])
def test_bad_range_leaves_the_others(pi, heads, dim):
    """[0, 10, 5]: the first sequence's rows 5 .. 9 lie past the last entry, and are its own all the same."""
    c = random_cache(pi, 6, heads, dim, 16)
    ref = oracle_of(c)
    table = i32([[1, 2], [3, 4]])
    for n in (10, 14):
        for _ in range(20):
            k = torch.full((n, heads, dim), 7.0, device="cuda")
            c.read(table, i32([0, 10, 5]), i32([3, 0]), n, dtype=torch.float32, k=k)
            assert c.device_status() == 5
            np.testing.assert_array_equal(k[:10].double().cpu().numpy(), ref.rows(0, [1, 2], 3, 13))
            assert not k[10:].any()
    k = torch.full((12, heads, dim), 7.0, device="cuda")
    c.read(table, i32([9, 4, 6]), i32([0, 2]), 12, dtype=torch.float32, k=k)
    assert c.device_status() == 5
    np.testing.assert_array_equal(k[4:6].double().cpu().numpy(), ref.rows(0, [3], 2, 4))
    assert not k[:4].any() and not k[9:].any() and (k[6:9] == 7).all()


@pytest.mark.parametrize("seqs", [1, 31, 600])
def test_rows_of_no_sequence(pi, seqs):
    """Zero before the first and after the last row, with and without empty sequences."""
    c = random_cache(pi, 4, 2, 64, 16)
    ref = oracle_of(c)
    new = [2 if s % 3 else 0 for s in range(seqs)]
    new[0] = 1
    cu = np.concatenate([[5], 5 + np.cumsum(new)])
    n = int(cu[-1]) + 37
    k = torch.full((n, 2, 64), 7.0, device="cuda")
    v = k.clone()
    c.read(i32([[s % 4] for s in range(seqs)]), i32(cu.tolist()), i32([s % 14 for s in range(seqs)]), n, dtype=torch.float32, k=k, v=v)
    assert c.device_status() == 0
    for which, t in ((0, k), (1, v)):
        assert not t[:5].any() and not t[n - 37:].any()
        want = np.concatenate([ref.rows(which, [s % 4], s % 14, s % 14 + m) for s, m in enumerate(new) if m])
        np.testing.assert_array_equal(t[5:n - 37].double().cpu().numpy(), want)
