"""Rows of a tree whose scores are NaN or infinite, by their queries or by all the keys that they see: output and log of
the sum are NaN however many rows and CTAs share the work, and no other row notices."""
import numpy as np
import pytest
import torch

from tests.kv_helpers import batch, random_cache
from tests.test_gpu_tree_attention import check, ints, packed, queries, tree_bits

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pi():
    import __graft_entry__
    __graft_entry__.build()
    import activation_sparse_rank_gb300 as pi
    return pi


def attend(c, b, q, length, mask, max_q, pages=None):
    """With a page table of `pages` columns, where given."""
    table = b["dev"]["table"]
    if pages:
        wide = torch.zeros(table.shape[0], pages, dtype=torch.int32, device="cuda")
        wide[:, :table.shape[1]] = table
        table = wide
    return c.attention(q, table, b["dev"]["cu"], ints(length), max_q=max_q, want_lse=True, tree=mask)


# query rows a head: a few, 24 (under a narrow table and one of 4096 tokens), one row tile of 128, two, three
ROWS = [(1, 5, None), (4, 6, None), (4, 6, 64), (8, 5, None), (8, 16, None), (8, 20, None), (8, 33, None)]


@pytest.mark.parametrize("dim,dtype", [(64, "float16"), (96, "bfloat16"), (128, "bfloat16"), (128, "float16"), (256, "bfloat16")])
@pytest.mark.parametrize("group,new,pages", ROWS)
@pytest.mark.parametrize("length", [[129 + 40], [300], [3000], [100 + 3 * s for s in range(90)]])
def test_queries(pi, dim, dtype, group, new, pages, length):
    """One sequence, of which a CTA has a tile or two, and so many that a CTA has whole ones."""
    rng = np.random.default_rng(dim + new)
    b = batch([n - new for n in length], [new] * len(length), 64, seed=dim)
    c = random_cache(pi, b["pages"], 2, dim, 64)
    q = queries(b["n"], 2 * group, dim, dtype)
    bits, _ = tree_bits(rng, [new] * len(length), 3)
    good, glse = attend(c, b, q, length, packed(bits), new, pages)
    assert torch.isfinite(good).all() and torch.isfinite(glse).all()
    special = torch.zeros(b["n"], 2 * group, dtype=torch.bool, device="cuda")
    for s in range(0, len(length), 7):
        q[s * new + 3, 1, 7] = float("nan")
        q[s * new + new - 2, 2 * group - 1, 0] = float("inf")      # keys of both signs: infinite both ways
        special[s * new + 3, 1] = special[s * new + new - 2, 2 * group - 1] = True
    out, lse = attend(c, b, q, length, packed(bits), new, pages)
    assert torch.isnan(out[special]).all() and torch.isnan(lse[special]).all()
    assert torch.isfinite(out[~special]).all() and torch.isfinite(lse[~special]).all()
    check(c, b, q, out, lse, length[:1], bits)           # a special sequence and its other rows
    if dim <= 128 and (group * new > 32 or pages):
        # a row's scale is its own there; up to 32 rows those of a warp go to a new one together, and round by it
        assert torch.equal(out[~special], good[~special]) and torch.equal(lse[~special], glse[~special])


@pytest.mark.parametrize("dim", [64, 96, 128, 256])
@pytest.mark.parametrize("group,new,pages", ROWS)
@pytest.mark.parametrize("first", [0, 128, 256])
def test_tiles_of_nan_keys(pi, dim, group, new, pages, first):
    """New tokens at a tile's beginning, the first one's key NaN, which some rows see of that tile alone, some with
    others and some not at all; then a cache all of whose keys are NaN."""
    length = [first + new]
    b = batch([first], [new], 64, seed=dim)
    c = random_cache(pi, b["pages"], 1, dim, 64)
    q = queries(new, group, dim, "float16")
    bits = np.eye(new, dtype=bool)
    bits[1:, 0] = np.arange(1, new) % 3 == 0
    bits[4] = [j == 0 for j in range(new)]               # nothing but the NaN
    page = int(b["table"][0][first // 64])
    c.k_codes[page, 0, 0, 9] = 0xff
    out, lse = attend(c, b, q, length, packed(bits), new, pages)
    check(c, b, q, out, lse, length, bits)
    is_nan = torch.from_numpy(bits[:, 0]).cuda()
    assert torch.isnan(lse[is_nan]).all() and torch.isnan(out[is_nan]).all() and torch.isfinite(lse[~is_nan]).all()
    if first:
        c.k_codes[page, 0, 0, 9] = 0
        c.k_codes[int(b["table"][0][0]), 0, :, 3] = 0x7f             # the first tile, whole
        c.k_codes[int(b["table"][0][1]), 0, :, 3] = 0x7f
        out, lse = attend(c, b, q, length, packed(bits), new, pages)
        assert torch.isnan(out).all() and torch.isnan(lse).all()


def test_rows_that_see_nothing_beside_nan_rows(pi):
    """-inf is for rows that see nothing: NaN rows beside them are NaN."""
    new = 12
    b = batch([0], [new], 64)
    c = random_cache(pi, b["pages"], 1, 64, 64)
    for group in (1, 8, 20):
        q = queries(new, group, 64, "float16")
        q[5] = float("nan")
        bits = np.tri(new, dtype=bool)
        bits[[0, 6]] = False
        out, lse = attend(c, b, q, [new], packed(bits), new)
        check(c, b, q, out, lse, [new], bits)
        assert torch.isnan(lse[5]).all() and torch.isneginf(lse[[0, 6]]).all() and not out[[0, 6]].any()
