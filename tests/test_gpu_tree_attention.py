"""Attention for trees of drafted tokens over the 8-bit cache, against its float64 definition on the stored values."""
import numpy as np
import pytest
import torch

from oracle import operators as O
from tests.kv_helpers import TORCH, batch, oracle_of, random_cache

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pi():
    import __graft_entry__
    __graft_entry__.build()
    import activation_sparse_rank_gb300 as pi
    return pi


def ints(v):
    return torch.tensor(np.asarray(v, np.int32), device="cuda")


def queries(n, heads, dim, dtype, seed=0, std=1.5):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(n, heads, dim, generator=g) * std).to(TORCH[dtype]).cuda()


def packed(bits):
    """Rows of truth values as int32 words."""
    b = np.pad(bits, ((0, 0), (0, -bits.shape[1] % 32))).reshape(len(bits), -1, 32)
    return torch.from_numpy((b.astype(np.uint32) << np.arange(32, dtype=np.uint32)).sum(2, dtype=np.uint32).view(np.int32)).cuda()


def tree_bits(rng, new, branch):
    parent = [-1 if i == 0 else i - 1 - int(rng.integers(min(i, branch))) for m in new for i in range(m)]
    cu = np.concatenate([[0], np.cumsum(new)])
    return O.draft_tree(parent, cu, max(new))[0], parent


def check(c, b, q, out, lse, length, bits):
    """Every row against the keys that it sees.

    Beside the oracle's bound: a weight times its value scale is kept in fp16 relative to the row's largest, which
    is at 2^6 or above.  fp16's smallest step is 2^-24, so a small one is off by 2^-25 / 2^6 = 2^-31 of the largest,
    and the largest is at most 1 times the largest scale; it multiplies a code of at most 448, once a key."""
    ref = oracle_of(c)
    step = 2.0 ** -31 * c.v_scales.max().item() * 448
    dtype = str(q.dtype).split(".")[1]
    group = q.shape[1] // c.heads
    qf, of, lf = (t.double().cpu().numpy() for t in (q, out, lse))
    for s in range(len(length)):
        r0, r1 = int(b["cu"][s]), int(b["cu"][s + 1])
        n = max(0, int(length[s]))
        k, v = (ref.rows(i, b["table"][s], 0, n) for i in (0, 1))
        first = int(length[s]) - (r1 - r0)
        for i in range(r1 - r0):
            see = [p for p in range(n) if p < first or (p - first <= i and bits[r0 + i, p - first])]
            for h in range(q.shape[1]):
                want, wl, tol, tl = O.attention(qf[r0 + i:r0 + i + 1, h], k[see, h // group], v[see, h // group], len(see) - 1,
                                                c.head_dim ** -0.5)
                got, gl = of[r0 + i, h], lf[r0 + i, h]
                bound = tol[0] + step * len(see) + O.UNIT[dtype] * np.abs(want[0]) * 1.001 + O.TINY[dtype]
                bad = ~((np.abs(got - want[0]) <= bound) | (np.isnan(got) & np.isnan(want[0])))
                assert not bad.any(), (s, i, h, len(see), got[bad][:3], want[0][bad][:3], bound[bad][:3])
                assert gl == wl[0] or np.isnan(gl) and np.isnan(wl[0]) or abs(gl - wl[0]) <= tl[0], (s, i, h, gl, wl, tl)


def run(c, b, q, length, mask, max_q):
    d = b["dev"]
    dl = ints(length)
    out, lse = c.attention(q, d["table"], d["cu"], dl, max_q=max_q, want_lse=True, tree=mask)
    again, _ = c.attention(q, d["table"], d["cu"], dl, max_q=max_q, want_lse=True, tree=mask)
    assert torch.equal(out, again) or torch.isnan(out).any()
    return out, lse


SHAPES = [(1, 1, 64, 16, "float16"), (2, 2, 96, 32, "bfloat16"), (1, 8, 128, 64, "bfloat16"), (2, 1, 256, 16, "float16"),
          (1, 5, 128, 48, "float16"), (1, 3, 96, 256, "float16")]


@pytest.mark.parametrize("heads,group,dim,page,dtype", SHAPES)
@pytest.mark.parametrize("new,length", [([1, 2, 5, 8], [1, 40, 70, 64]), ([4, 0, 16, 3], [4, 9, 150, 130]),
                                        ([26, 26, 1, 11], [26, 333, 500, 12]), ([64, 33, 5], [200, 33, 3]), ([130, 7], [300, 135])])
@pytest.mark.parametrize("branch", [1, 4])
def test_trees(pi, heads, group, dim, page, dtype, new, length, branch):
    """From a few rows to several row tiles; trees at the cache's beginning, over tile and page edges, and of
    more nodes than the length says (their first rows have no place)."""
    rng = np.random.default_rng(dim + len(new) + branch)
    b = batch([max(0, n - m) for n, m in zip(length, new)], new, page, seed=dim)
    c = random_cache(pi, b["pages"], heads, dim, page, seed=group)
    q = queries(b["n"], heads * group, dim, dtype)
    bits, parent = tree_bits(rng, new, branch)
    mask, _ = pi.draft_tree(ints(parent), b["dev"]["cu"], max(new))
    out, lse = run(c, b, q, length, mask, max(new))
    check(c, b, q, out, lse, length, bits)
    assert c.device_status() == 0


@pytest.mark.parametrize("heads,group,dim,page,dtype", SHAPES)
@pytest.mark.parametrize("new,length", [([3, 9], [3, 40]), ([40, 70], [40, 160])])
def test_any_bits(pi, heads, group, dim, page, dtype, new, length):
    """Bits that make no tree: rows that see nothing at all, not even themselves; bits behind a row do not count."""
    rng = np.random.default_rng(dim)
    b = batch([n - m for n, m in zip(length, new)], new, page, seed=dim)
    c = random_cache(pi, b["pages"], heads, dim, page)
    q = queries(b["n"], heads * group, dim, dtype)
    bits = rng.random((b["n"], max(new))) < 0.3
    bits[[0, 2, new[0] - 1]] = False
    out, lse = run(c, b, q, length, packed(bits), max(new))
    check(c, b, q, out, lse, length, bits)
    for r in (0, 2, new[0] - 1):
        assert not out[r].any() and torch.isneginf(lse[r]).all()


@pytest.mark.parametrize("heads,group,dim,page,dtype", SHAPES)
@pytest.mark.parametrize("new,length", [([6, 3], [30, 150]), ([50, 90], [70, 290]), ([256], [300])])
def test_nan_among_the_nodes(pi, heads, group, dim, page, dtype, new, length):
    """A NaN in a node's key or value (or in the cache before) reaches the rows that see it, and no other."""
    rng = np.random.default_rng(dim)
    b = batch([n - m for n, m in zip(length, new)], new, page, seed=dim)
    c = random_cache(pi, b["pages"], heads, dim, page)
    q = queries(b["n"], heads * group, dim, dtype)
    bits, parent = tree_bits(rng, new, 4)
    for s, (n, m) in enumerate(zip(length, new)):
        for codes, nodes in ((c.v_codes, (1, m // 2, m - 1)), (c.k_codes, (2,))):
            for i in nodes:
                at = n - m + i
                codes[int(b["table"][s][at // page]), 0, at % page, int(rng.integers(dim))] = 0x7f if i % 2 else 0xff
    out, lse = run(c, b, q, length, packed(bits), max(new))
    check(c, b, q, out, lse, length, bits)
    assert torch.isnan(out).any() and not torch.isnan(out).all()


def test_masked_keys_of_any_size(pi):
    """Keys of the largest values that a row does not see leave its result alone; lowest scores that it sees do not."""
    b = batch([20], [12], 16)
    c = random_cache(pi, b["pages"], 1, 64, 16)
    q = queries(12, 4, 64, "bfloat16", std=30.0)
    bits = np.tri(12, dtype=bool)
    bits[1:, 0] = False
    page = int(b["table"][0][20 // 16])
    c.k_codes[page, 0, 4] = 0x7e                      # node 0
    c.k_scales[page, 0, 0] = 2.0 ** 60
    out, lse = run(c, b, q, [32], packed(bits), 12)
    check(c, b, q, out, lse, [32], bits)
    c.k_codes[page, 0, 4] = 0xfe
    out, lse = run(c, b, q, [32], packed(bits), 12)
    check(c, b, q, out, lse, [32], bits)


@pytest.mark.parametrize("heads,group,dim,page,dtype", SHAPES)
def test_a_chain_is_causal_attention(pi, heads, group, dim, page, dtype):
    """Full bits, wider than needed: what causal attention gives; up to 32 query rows a head (and of 256 dims) bit
    for bit, above within the bound of both (other kernels, other order of sums)."""
    new, length = [5, 40, 1, 17], [300, 41, 1, 2000]
    for keep in (1, 4):
        new, length = new[:keep], length[:keep]
        b = batch([n - m for n, m in zip(length, new)], new, page, seed=dim)
        c = random_cache(pi, b["pages"], heads, dim, page)
        q = queries(b["n"], heads * group, dim, dtype)
        d = b["dev"]
        want = c.attention(q, d["table"], d["cu"], ints(length), max_q=max(new), want_lse=True)
        full = torch.full((b["n"], 5), -1, dtype=torch.int32, device="cuda")
        got = c.attention(q, d["table"], d["cu"], ints(length), max_q=max(new), want_lse=True, tree=full)
        if max(new) * group <= 32 or dim == 256:
            assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
        bits = np.ones((b["n"], 160), bool)
        check(c, b, q, *got, length, bits)
        check(c, b, q, *want, length, bits)
        new, length = [5, 40, 1, 17], [300, 41, 1, 2000]


def test_cut_units_and_many_sequences(pi):
    """A long cache under one tree (its units cut over many CTAs), with few and with many rows, and more
    sequences than SMs."""
    rng = np.random.default_rng(0)
    for new, length, heads, group in (([21], [20000], 1, 8), ([3, 2], [5000, 2], 2, 8), ([20], [4100], 3, 1),
                                      ([3] * 200, list(range(3, 203)), 1, 2)):
        b = batch([n - m for n, m in zip(length, new)], new, 64)
        c = random_cache(pi, b["pages"], heads, 64, 64)
        q = queries(b["n"], heads * group, 64, "float16")
        bits, _ = tree_bits(rng, new, 3)
        out, lse = run(c, b, q, length, packed(bits), max(new))
        check(c, b, q, out, lse, length, bits)


def test_rows_past_max_q_bad_pages_and_rows_of_no_sequence(pi):
    new, length = [9, 4], [40, 30]
    b = batch([n - m for n, m in zip(length, new)], new, 16)
    c = random_cache(pi, b["pages"], 1, 64, 16)
    q = queries(b["n"] + 3, 2, 64, "float16")
    full = torch.full((b["n"] + 3, 1), -1, dtype=torch.int32, device="cuda")
    d, out = b["dev"], torch.full_like(q, 5.0)
    lse = torch.full(q.shape[:2], 5.0, device="cuda")
    c.attention(q, d["table"], d["cu"], ints(length), max_q=4, tree=full, out=out, lse=lse)
    assert not out[4:9].any() and torch.isneginf(lse[4:9]).all() and (out[13:] == 5.0).all() and (lse[13:] == 5.0).all()
    assert c.device_status() != 0
    sub = c.attention(q[9:13], d["table"][1:], ints([0, 4]), ints(length[1:]), max_q=4, tree=full[9:13], want_lse=True)
    assert torch.equal(sub[0], out[9:13]) and torch.equal(sub[1], lse[9:13])
    table = d["table"].clone()
    table[0, 1] = -5
    c.attention(q, table, d["cu"], ints(length), max_q=9, tree=full)
    assert c.device_status() != 0


def test_graph_stream_and_refusals(pi):
    new, length = [7, 12], [90, 200]
    b = batch([n - m for n, m in zip(length, new)], new, 32)
    c = random_cache(pi, b["pages"], 2, 128, 32)
    q = queries(b["n"], 8, 128, "bfloat16")
    d, dl = b["dev"], ints(length)
    rng = np.random.default_rng(1)
    mask = packed(tree_bits(rng, new, 3)[0])
    want = c.attention(q, d["table"], d["cu"], dl, max_q=12, tree=mask, want_lse=True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = c.attention(q, d["table"], d["cu"], dl, max_q=12, tree=mask, want_lse=True, stream=side)
    side.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    ws = c.attention_workspace(8, b["n"], 2)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out, lse = c.attention(q, d["table"], d["cu"], dl, max_q=12, tree=mask, want_lse=True, ws=ws)
    for seed in (2, 3):
        mask.copy_(packed(tree_bits(np.random.default_rng(seed), new, 5)[0]))
        dl -= 1
        g.replay()
        want = c.attention(q, d["table"], d["cu"], dl, max_q=12, tree=mask, want_lse=True)
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    args = (q, d["table"], d["cu"], dl)
    for bad in (dict(tree=mask.long()), dict(tree=mask[:5]), dict(tree=mask, max_q=33), dict(tree=mask.cpu()), dict(tree=mask[:, 0]),
                dict(tree=mask, causal=False), dict(tree=torch.zeros(b["n"], 9, dtype=torch.int32, device="cuda"), max_q=257)):
        with pytest.raises((ValueError, TypeError)):
            c.attention(*args, **bad)
    assert torch.equal(c.attention(*args, tree=mask), c.attention(*args, tree=mask, max_q=19))       # max_q left out: all rows
    none = c.attention(q[:0], d["table"][:0], ints([0]), ints([]), tree=mask[:0])
    assert none.shape == (0, 8, 128)


@pytest.mark.parametrize("new", [1, 12, 40])
def test_scores_past_binary32s_whole_numbers(pi, new):
    """Scores of 1e10 and more, whose last place is above any exponent: the largest alone counts."""
    b = batch([300 - new], [new], 16)
    c = random_cache(pi, b["pages"], 1, 64, 16)
    c.k_scales.mul_(2.0 ** 40)
    q = queries(new, 4, 64, "float16")
    bits = np.tri(new, dtype=bool)
    d = b["dev"]
    out, lse = c.attention(q, d["table"], d["cu"], d["length"], max_q=new, want_lse=True, tree=packed(bits))
    ref = oracle_of(c)
    k, v = (ref.rows(i, b["table"][0], 0, 300)[:, 0] for i in (0, 1))
    for i in range(new):
        score = k[:300 - new + i + 1] @ q[i].double().cpu().numpy().T / 8
        order = np.sort(score, 0)
        assert (order[-1] - order[-2] > np.abs(score).max(0) * 2.0 ** -16).all()       # no near ties: the input's own property
        got = out[i].double().cpu().numpy()
        np.testing.assert_array_equal(got, torch.from_numpy(v[score.argmax(0)]).half().double().numpy())
        assert (np.abs(lse[i].double().cpu().numpy() - score.max(0)) <= 2.0 ** -16 * np.abs(score).max(0)).all()
