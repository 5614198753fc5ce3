"""The bound on new tokens: left out, too small, and far too large."""
import pytest
import torch

from tests.kv_helpers import batch, random_cache
from tests.test_gpu_attention import check, pi, queries, run  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dim,group,new,length", [(64, 2, [5, 0, 3], [30, 4, 3]), (128, 8, [40, 1, 17], [300, 9, 40]),
                                                  (256, 1, [3, 2, 1], [50, 2, 7]), (64, 1, [300], [310])])
def test_without_a_bound(pi, dim, group, new, length):
    """A prompt without max_q: every row as with it."""
    b = batch([n - m for n, m in zip(length, new)], new, 32)
    c = random_cache(pi, b["pages"], 2, dim, 32)
    q = queries(b["n"], 2 * group, dim, "float16")
    d = b["dev"]
    out, lse = c.attention(q, d["table"], d["cu"], d["length"], want_lse=True)
    check(c, b, q, out, lse, length)
    assert c.device_status() == 0


@pytest.mark.parametrize("dim,group,most", [(64, 2, 1), (128, 8, 3), (96, 4, 16), (256, 2, 2), (64, 1, 129)])
def test_rows_past_the_bound(pi, dim, group, most):
    """0 and -inf for them, flagged; the others as with a large enough bound."""
    new = [most, most + 1, 0, 2 * most + 9, 1]
    length = [n + 40 for n in new]
    b = batch([40] * 5, new, 32)
    c = random_cache(pi, b["pages"], 2, dim, 32)
    q = queries(b["n"], 2 * group, dim, "bfloat16")
    d = b["dev"]
    out = torch.full_like(q, 7.0)
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    c.attention(q, d["table"], d["cu"], d["length"], max_q=most, out=out, lse=lse)
    assert c.device_status() == 5
    kept = torch.zeros(b["n"], dtype=torch.bool, device="cuda")
    for s, n in enumerate(new):
        kept[int(b["cu"][s]):int(b["cu"][s]) + min(n, most)] = True
    assert not out[~kept].any() and torch.isneginf(lse[~kept]).all()
    want, wlse = run(pi, c, b, q, length)
    check(c, b, q, torch.where(kept[:, None, None], out, want), torch.where(kept[:, None], lse, wlse), length)


def test_rows_past_the_bound_by_default(pi):
    """As many rows as sequences are taken for one each; where they are not, nothing is left unset."""
    b = batch([8, 8], [2, 0], 32)
    c = random_cache(pi, b["pages"], 1, 64, 32)
    q = queries(2, 1, 64, "float16")
    d = b["dev"]
    for bound in ({}, {"max_q": 0}):
        out, lse = c.attention(q, d["table"], d["cu"], d["length"], want_lse=True, **bound)
        assert c.device_status() == 5
        assert out[0].any() and not out[1].any() and torch.isneginf(lse[1]).all()
