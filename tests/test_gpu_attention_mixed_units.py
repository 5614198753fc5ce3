"""NaN among the newest tokens of batches whose long prompts, short prompts and single row tiles alternate."""
import numpy as np
import pytest
import torch

from tests.kv_helpers import batch, random_cache
from tests.test_gpu_attention import check, pi, queries, run  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dim,group", [(64, 1), (128, 2), (96, 1)])
def test_nan_of_each_unit_stays_there(pi, dim, group):
    """Units of 256 rows beside units of fewer than 128 over many tiles of keys, in the same CTAs: each row that
    sees a NaN value has NaN in its dim, and every other output has the bits that it has without."""
    rng = np.random.default_rng(dim)
    new, length = [], []
    for s in range(70):
        n = [300, 40, 260, 129, 35, 500][s % 6] // group
        new.append(n)
        length.append(n + int(rng.choice([0, 5, 90, 700, 1500])))
    heads = 3
    b = batch([n - m for n, m in zip(length, new)], new, 64, seed=dim)
    c = random_cache(pi, b["pages"], heads, dim, 64)
    q = queries(b["n"], heads * group, dim, "bfloat16")
    good, lse = run(pi, c, b, q, length)
    assert torch.isfinite(good).all()
    expect = torch.zeros(good.shape, dtype=torch.bool)
    for s in range(len(new)):
        for position in rng.integers(length[s] - new[s], length[s], 3):
            h, d = int(rng.integers(heads)), int(rng.integers(dim))
            c.v_codes[int(b["table"][s, position // 64]), h, position % 64, d] = 0x7f
            first = int(b["cu"][s]) + int(position) - (length[s] - new[s])
            expect[first:int(b["cu"][s + 1]), h * group:(h + 1) * group, d] = True
    expect = expect.cuda()
    dev = b["dev"]
    for _ in range(10):
        out, again = c.attention(q, dev["table"], dev["cu"], dev["length"], max_q=max(new), want_lse=True)
        assert torch.equal(torch.isnan(out), expect)
        assert torch.equal(torch.where(expect, good, out), good) and torch.equal(again, lse)
    assert c.device_status() == 0


@pytest.mark.parametrize("causal", [True, False])
def test_mixed_units_against_the_definition(pi, causal):
    new, length = [300, 40, 1, 260, 129, 33], [310, 1500, 700, 260, 900, 40]
    b = batch([n - m for n, m in zip(length, new)], new, 32)
    c = random_cache(pi, b["pages"], 1, 64, 32)
    q = queries(b["n"], 1, 64, "float16")
    out, lse = run(pi, c, b, q, length, causal=causal)
    check(c, b, q, out, lse, length, causal=causal)
