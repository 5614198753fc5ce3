"""Attention with several query rows a head: every form of the row tiles, cuts of long units, bad input among many rows."""
import numpy as np
import pytest
import torch

from tests.kv_helpers import batch, random_cache
from tests.test_gpu_attention import check, pi, queries, run  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("dim,page", [(64, 64), (96, 48), (128, 16), (256, 32)])
def test_row_counts_around_the_tiles(pi, dim, page, dtype):
    """Query rows a head at and around every size of a row tile; the key count ends inside a page and a tile."""
    heads = 2
    for group, new in ((1, 9), (8, 2), (1, 17), (8, 4), (3, 11), (16, 8), (1, 129), (8, 32), (1, 257)):
        for length in (max(new, 70), 397):
            b = batch([length - new], [new], page, seed=group)
            c = random_cache(pi, b["pages"], heads, dim, page, seed=new)
            q = queries(new, heads * group, dim, dtype, seed=length)
            out, lse = run(pi, c, b, q, [length])
            check(c, b, q, out, lse, [length])
            assert c.device_status() == 0


@pytest.mark.parametrize("dim,dtype", [(64, "bfloat16"), (128, "float16")])
def test_many_row_tiles(pi, dim, dtype):
    """More row tiles a head than a warp has lanes, with sequences beside it that need one or none."""
    new, length = [1100, 1, 0, 300], [1203, 77, 50, 150]
    b = batch([max(0, n - m) for n, m in zip(length, new)], new, 64, seed=1)
    c = random_cache(pi, b["pages"], 1, dim, 64)
    q = queries(b["n"], 8, dim, dtype, seed=2)
    out, lse = run(pi, c, b, q, length)
    check(c, b, q, out, lse, length)


@pytest.mark.parametrize("group,new,dim", [(1, 1, 128), (5, 3, 96), (8, 3, 64), (8, 5, 128), (16, 9, 64), (4, 4, 256)])
@pytest.mark.parametrize("length", [1300, 9100])
def test_units_cut_many_times(pi, group, new, dim, length):
    """One head: up to a part a CTA, of few and of many parts."""
    b = batch([length - new], [new], 64)
    c = random_cache(pi, b["pages"], 1, dim, 64)
    q = queries(new, group, dim, "float16")
    out, lse = run(pi, c, b, q, [length])
    check(c, b, q, out, lse, [length])


@pytest.mark.parametrize("dim,group", [(64, 8), (96, 4), (128, 8), (256, 3)])
@pytest.mark.parametrize("new", [5, 40, 150])
def test_masked_nan_in_many_rows(pi, dim, group, new):
    """NaN behind the last token reach no row; a NaN value of a late token reaches every later row and no other."""
    length = 330
    b = batch([length - new], [new], 32)
    c = random_cache(pi, b["pages"], 1, dim, 32)
    q = queries(new, group, dim, "float16")
    last = int(b["table"][0, length // 32])
    c.k_codes[last, :, length % 32:] = 0x7f
    c.v_codes[last, :, length % 32:] = 0xff
    out, lse = run(pi, c, b, q, [length])
    check(c, b, q, out, lse, [length])
    assert torch.isfinite(out).all()
    for dim_at, position in ((5, length - 2), (dim - 1, length - new + new // 2)):
        page = int(b["table"][0, position // 32])
        old = c.v_codes[page, 0, position % 32, dim_at].item()
        c.v_codes[page, 0, position % 32, dim_at] = 0x7f
        out, lse = run(pi, c, b, q, [length])
        seen = length - position
        bad = torch.isnan(out)
        assert bad[new - seen:, :, dim_at].all() and bad.sum() == seen * group and torch.isfinite(lse).all()
        c.v_codes[page, 0, position % 32, dim_at] = old


@pytest.mark.parametrize("dim,group,new", [(64, 2, 30), (96, 4, 40), (128, 8, 40), (256, 2, 12)])
def test_special_queries_among_many_rows(pi, dim, group, new):
    """A NaN or infinite query row is NaN; no other row notices."""
    length = 200
    b = batch([length - new], [new], 64)
    c = random_cache(pi, b["pages"], 2, dim, 64)
    q = queries(new, 2 * group, dim, "float16")
    good, glse = run(pi, c, b, q, [length])
    q[3, 1, 7] = float("nan")
    q[new - 2, 2 * group - 1, 0] = float("inf")
    out, lse = run(pi, c, b, q, [length])
    special = torch.zeros(new, 2 * group, dtype=torch.bool, device="cuda")
    special[3, 1] = special[new - 2, 2 * group - 1] = True
    assert torch.isnan(out[special]).all()
    assert torch.equal(out[~special], good[~special]) and torch.equal(lse[~special], glse[~special])


@pytest.mark.parametrize("dim,group", [(64, 8), (96, 8), (128, 3), (256, 4)])
def test_bad_tables_with_many_rows(pi, dim, group):
    """Pages and ranges out of bounds: flagged, the sequences beside it as before."""
    new, length = [20, 33, 12], [150, 40, 90]
    b = batch([n - m for n, m in zip(length, new)], new, 32)
    c = random_cache(pi, b["pages"], 2, dim, 32)
    q = queries(b["n"], 2 * group, dim, "bfloat16")
    d = b["dev"]
    good = c.attention(q, d["table"], d["cu"], d["length"], max_q=33)
    assert c.device_status() == 0
    for page in (b["pages"], -1, 1 << 30):
        table = d["table"].clone()
        table[0, 1] = page
        out = c.attention(q, table, d["cu"], d["length"], max_q=33)
        assert c.device_status() == 5 and torch.equal(out[20:], good[20:])
    for bad in (1 << 30, -5):
        at = d["length"].clone()
        at[0] = bad
        out = c.attention(q, d["table"], d["cu"], at, max_q=33)
        assert c.device_status() == 5 and torch.equal(out[20:], good[20:])
    out = c.attention(q, d["table"], d["cu"], d["length"], max_q=20)       # a sequence has more
    assert c.device_status() == 5 and torch.equal(out[:20], good[:20])


def test_all_masked_blocks(pi):
    """Many sequences of which most have no key at all, for one and for many rows."""
    for new in (1, 40):
        n = 150
        length = [0 if s % 7 else 60 + s for s in range(n)]
        b = batch([max(0, x - new) for x in length], [new] * n, 16)
        c = random_cache(pi, b["pages"], 1, 64, 16)
        q = queries(b["n"], 2, 64, "float16")
        out, lse = run(pi, c, b, q, length)
        check(c, b, q, out, lse, length)
        empty = torch.from_numpy(np.repeat(np.array(length) == 0, new)).cuda()
        assert not out[empty].any() and torch.isneginf(lse[empty]).all()


@pytest.mark.parametrize("dim,group,new", [(64, 1, 5), (64, 4, 40), (96, 8, 20), (128, 8, 40), (256, 2, 20)])
def test_sixteen_byte_alignment(pi, dim, group, new):
    """Queries, output and workspace that start 16 bytes past a 32-byte boundary, queries with an odd stride of 16
    bytes: the same bits as aligned ones."""
    heads, length = 2, 700
    b = batch([length - new], [new], 64)
    c = random_cache(pi, b["pages"], heads, dim, 64)
    n = heads * group
    q = queries(new, n, dim, "bfloat16")
    want, wlse = run(pi, c, b, q, [length])
    d = b["dev"]
    wide = torch.zeros(new * n * (dim + 8) + 8, dtype=torch.bfloat16, device="cuda")[8:].view(new, n, dim + 8)
    wide[:, :, :dim] = q
    out = torch.zeros(new * n * dim + 8, dtype=torch.bfloat16, device="cuda")[8:].view(new, n, dim)
    ws = torch.empty(c.attention_workspace(n, new, 1).numel() + 16, dtype=torch.uint8, device="cuda")[16:]
    assert wide.data_ptr() % 32 == 16 and out.data_ptr() % 32 == 16 and ws.data_ptr() % 32 == 16
    got, lse = c.attention(wide[:, :, :dim], d["table"], d["cu"], d["length"], max_q=new, out=out, want_lse=True, ws=ws)
    assert got is out and torch.equal(out, want) and torch.equal(lse, wlse)
