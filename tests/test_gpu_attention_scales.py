"""Attention over blocks whose value scales lie at the ends of their range, for every form of the row tiles."""
import numpy as np
import pytest
import torch

from oracle import operators as O
from tests.kv_helpers import batch, oracle_of, random_cache
from tests.test_gpu_attention import pi, queries, run  # noqa: F401

pytestmark = pytest.mark.gpu

# head dim and query rows a head of each kernel and row tile
ROWS = [(64, 1), (64, 16), (128, 30), (256, 30), (64, 33), (96, 70), (128, 300)]
ONE, MINUS_72 = 0x38, 0xe9                           # codes


def check(c, b, q, out, lse, length, causal=False, scale=None):
    """One sequence within the operator's bounds.  Weights times value scales are
    held in fp16 relative to the row's largest, 2^6 there at least, so each may
    also be off by half of fp16's smallest step: 2^-31 of the largest."""
    ref = oracle_of(c)
    scale = c.head_dim ** -0.5 if scale is None else scale
    n, group = q.shape[0], q.shape[1] // c.heads
    qf, of, lf = (t.double().cpu().numpy() for t in (q, out, lse))
    k, v = (ref.rows(i, b["table"][0], 0, length) for i in (0, 1))
    pages = b["table"][0][np.arange(length) // c.page_size]
    at = np.arange(length) % c.page_size
    for h in range(q.shape[1]):
        kv = h // group
        s = ref.scale[1][pages, kv, at // 16]
        code = np.abs(ref.value[1][pages, kv, at])
        want, wl, tol, tl = O.attention(qf[:, h], k[:, kv], v[:, kv], length - n, scale, causal)
        for i in range(n):
            m = min(length, length - n + i + 1) if causal else length
            if m <= 0:
                continue
            p = np.exp(scale * (k[:m, kv] @ qf[i, h]) - wl[i])
            floor = 2.0 ** -31 * (p * s[:m]).max() * code[:m].sum(0)
            bound = tol[i] + 1.01 * floor + O.UNIT["bfloat16"] * np.abs(want[i]) * 1.001 + O.TINY["bfloat16"]
            bad = ~(np.abs(of[i, h] - want[i]) <= bound)
            assert not bad.any(), (h, i, np.flatnonzero(bad)[:3], of[i, h][bad][:3], want[i][bad][:3], bound[bad][:3])
            assert abs(lf[i, h] - wl[i]) <= tl[i], (h, i, lf[i, h], wl[i], tl[i])


def value_blocks(c, b, length, codes, exps):
    """Block i of sequence 0 gets code codes[i] throughout and scale 2^exps[i]."""
    for i in range(-(-length // 16)):
        page, at = int(b["table"][0, i * 16 // c.page_size]), i * 16 % c.page_size
        c.v_codes[page, :, at:at + 16] = codes[i]
        c.v_scales[page, :, at // 16] = 2.0 ** exps[i]


@pytest.mark.parametrize("dim,rows", ROWS)
@pytest.mark.parametrize("length,order", [(32, "large first"), (32, "small first"), (9000, "in turn"), (9000, "halves")])
def test_denominator_of_far_scales(pi, dim, rows, length, order):
    """Values of 2^100 beside zeros (which have the smallest scale), at equal scores: the zeros' weights count."""
    n = -(-length // 16)
    b = batch([max(0, length - rows)], [rows], 64)
    c = random_cache(pi, b["pages"], 1, dim, 64)
    large = [{"large first": i < 1, "small first": i >= 1, "in turn": i % 2 == 0, "halves": i < n // 2}[order] for i in range(n)]
    value_blocks(c, b, length, [ONE if x else 0 for x in large], [100 if x else -64 for x in large])
    c.k_codes.zero_()
    q = queries(rows, 1, dim, "bfloat16")
    out, lse = run(pi, c, b, q, [length], causal=False)
    check(c, b, q, out, lse, length)


@pytest.mark.parametrize("dim,rows", ROWS)
@pytest.mark.parametrize("length", [200, 5000])
def test_scales_over_their_whole_range(pi, dim, rows, length):
    """Scales from 2^-64 to 2^110 at random, with random keys."""
    length = max(length, rows)
    b = batch([length - rows], [rows], 32)
    c = random_cache(pi, b["pages"], 2, dim, 32, seed=rows)
    g = torch.Generator().manual_seed(length)
    c.v_scales.copy_(torch.ldexp(torch.ones(c.v_scales.shape), torch.randint(-64, 111, c.v_scales.shape, generator=g)))
    q = queries(rows, 2, dim, "bfloat16", seed=2)
    out, lse = run(pi, c, b, q, [length])
    check(c, b, q, out, lse, length, causal=True)


@pytest.mark.parametrize("dim,rows", ROWS)
@pytest.mark.parametrize("length", [64, 2000])
@pytest.mark.parametrize("order", ["large first", "large last"])
def test_small_weights_of_large_values(pi, dim, rows, order, length):
    """Weights of e^-72 on values of 2^104 beside weights of 1 on values of 1: both are of the result."""
    length = max(length, rows)
    b = batch([length - rows], [rows], 64)
    c = random_cache(pi, b["pages"], 1, dim, 64)
    n = -(-length // 16)
    large = [(i < n // 2) == (order == "large first") for i in range(n)]
    value_blocks(c, b, length, [ONE] * n, [104 if x else 0 for x in large])
    c.k_codes.zero_()
    c.k_scales.fill_(1.0)
    for i in range(n):
        if large[i]:
            page, at = int(b["table"][0, i * 16 // 64]), i * 16 % 64
            c.k_codes[page, :, at:at + 16, 0] = MINUS_72
    q = torch.zeros(rows, 1, dim, dtype=torch.bfloat16, device="cuda")
    q[:, :, 0] = 1
    out, lse = run(pi, c, b, q, [length], causal=False, sm_scale=1.0)
    check(c, b, q, out, lse, length, scale=1.0)
    assert ((out > 1.5) & (out < 4)).all()
