"""Layer norm, forward and backward, against its float64 definition and bounds."""
import numpy as np
import pytest
import torch

from oracle import operators as O
from tests.kv_helpers import TORCH

pytestmark = pytest.mark.gpu

SHAPES = [(1, 1), (5, 7), (3, 64), (130, 96), (9, 511), (4, 512), (7, 1000), (33, 1024), (2, 2049), (5, 4096), (3, 5001),
          (4, 8192), (2, 12288), (1, 16383), (3, 16384)]


@pytest.fixture(scope="module")
def pi():
    import __graft_entry__
    __graft_entry__.build()
    import activation_sparse_rank_gb300 as pi
    return pi


def rand(shape, dtype, seed, mean=0.0, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std + mean).to(TORCH[dtype]).cuda()


def f64(t):
    return t.detach().double().cpu().numpy()


def near(got, want, bound, dtype, name):
    got, bound = f64(got), bound + O.UNIT[dtype] * np.abs(want) * 1.001 + O.TINY[dtype]
    bad = ~(np.abs(got - want) <= bound)
    assert not bad.any(), (name, np.argwhere(bad)[:3], got[bad][:3], np.asarray(want)[bad][:3], bound[bad][:3])


@pytest.mark.parametrize("dtype", ["float16", "bfloat16", "float32"])
@pytest.mark.parametrize("rows,d", SHAPES)
def test_forward(pi, rows, d, dtype):
    x = rand((rows, d), dtype, 1, mean=0.5, std=2.0)
    wt = "float32" if d % 3 else dtype
    w, b = rand(d, wt, 2, mean=1.0), rand(d, wt, 3)
    y, total, mean, rstd = pi.layer_norm(x, w, b, want_stats=True)
    assert total is None
    wy, wm, wr, ty, tm, tr = O.layer_norm(f64(x), f64(w), f64(b), 1e-5)
    near(y, wy, ty, dtype, "y")
    near(mean, wm, tm, "float32", "mean")
    near(rstd, wr, tr, "float32", "rstd")


@pytest.mark.parametrize("dtype,add_dtype", [("float16", "float32"), ("bfloat16", "bfloat16"), ("float32", "float16"),
                                             ("float16", "bfloat16")])
@pytest.mark.parametrize("rows,d", [(5, 7), (130, 96), (6, 1024), (3, 5001), (4, 8192)])
def test_forward_after_addition(pi, rows, d, dtype, add_dtype):
    x, a = rand((rows, d), dtype, 1, std=2.0), rand((rows, d), add_dtype, 2)
    w = rand(d, "float32", 3, mean=1.0)
    want = (x.float() + a.float()).to(x.dtype)       # one binary32 addition, rounded once
    y, total, mean, rstd = pi.layer_norm(x, w, None, add=a, eps=1e-3)
    assert mean is None and rstd is None
    assert torch.equal(total, want)
    wy, _, _, ty, _, _ = O.layer_norm(f64(want), f64(w), 0.0, 1e-3)
    near(y, wy, ty, dtype, "y")
    z = x.clone()
    y2, total2, _, _ = pi.layer_norm(z, w, None, add=a, sum=z, eps=1e-3)
    assert total2 is z and torch.equal(z, want) and torch.equal(y, y2)


def test_forward_hard_rows(pi):
    """A large mean, equal values, zeros, one outlier; eps 0 with a spread; NaN and infinity stay in their row."""
    d = 4096
    x = rand((7, d), "float32", 1)
    x[0] += 1e4
    x[1] = 3.0
    x[2] = 0
    x[3, 17] = 1e4
    x[5, 3] = float("nan")
    x[6, 3] = float("inf")
    y, _, mean, rstd = pi.layer_norm(x, want_stats=True)
    wy, wm, wr, ty, tm, tr = O.layer_norm(f64(x[:5]), 1.0, 0.0, 1e-5)
    near(y[:5], wy, ty, "float32", "y")
    near(mean[:5], wm, tm, "float32", "mean")
    near(rstd[:5], wr, tr, "float32", "rstd")
    assert torch.isnan(y[5:]).all()


def test_forward_strides_and_views(pi):
    """Rows of a wider tensor, aligned and not; leading dimensions; outputs given."""
    wide = rand((9, 3, 300), "bfloat16", 1)
    w, b = rand(96, "bfloat16", 2, mean=1.0), rand(96, "bfloat16", 3)
    for at in (0, 8, 5):
        x = wide[:, 1, at:at + 96]
        y = pi.layer_norm(x, w, b)[0]
        assert torch.equal(y, pi.layer_norm(x.contiguous(), w, b)[0])
    x = wide[:, :, :96].contiguous()
    y = torch.empty_like(x)
    r = pi.layer_norm(x, w, b, y=y)
    assert r[0] is y and torch.equal(y.view(-1, 96), pi.layer_norm(x.view(-1, 96), w, b)[0])
    e = pi.layer_norm(x[:0], w, b, want_stats=True)
    assert e[0].shape == (0, 3, 96) and e[2].numel() == 0


@pytest.mark.parametrize("dtype", ["float16", "bfloat16", "float32"])
@pytest.mark.parametrize("rows,d", SHAPES + [(700, 64), (1000, 520), (2000, 33)])
def test_backward(pi, rows, d, dtype):
    x, dy = rand((rows, d), dtype, 1, mean=0.5, std=2.0), rand((rows, d), dtype, 2)
    w = rand(d, "float32" if d % 3 else dtype, 3, mean=1.0)
    ds = rand((rows, d), dtype, 4) if d % 2 == 0 else None
    _, _, mean, rstd = pi.layer_norm(x, w, None, want_stats=True)
    dx, dw, db = pi.layer_norm_backward(dy, x, w, mean, rstd, d_sum=ds)
    wx, ww, wb, tx, tw, tb = O.layer_norm_backward(f64(dy), f64(x), f64(w), f64(mean), f64(rstd),
                                                   None if ds is None else f64(ds))
    near(dx, wx, tx, dtype, "dx")
    near(dw, ww, tw, "float32", "dweight")
    near(db, wb, tb, "float32", "dbias")
    again = pi.layer_norm_backward(dy, x, w, mean, rstd, d_sum=ds)
    assert all(torch.equal(a, b) for a, b in zip((dx, dw, db), again))
    z = dy.clone()
    only, nw, nb = pi.layer_norm_backward(z, x, w, mean, rstd, d_sum=ds, dx=z, want_weight_grad=False)
    assert only is z and torch.equal(z, dx) and nw is None and nb is None


def test_backward_against_differences(pi):
    """The GPU's gradient against differences of the float64 forward."""
    rows, d, e = 3, 24, 1e-6
    x, dy, w = rand((rows, d), "float32", 1), rand((rows, d), "float32", 2), rand(d, "float32", 3, mean=1.0)
    _, _, mean, rstd = pi.layer_norm(x, w, None, want_stats=True)
    dx, dw, db = (f64(t) for t in pi.layer_norm_backward(dy, x, w, mean, rstd))
    xf, wf, yf = f64(x), f64(w), f64(dy)

    def loss(x, w):
        return (O.layer_norm(x, w, 0.0, 1e-5)[0] * yf).sum()

    for i in range(rows):
        for j in range(d):
            s = np.zeros_like(xf)
            s[i, j] = e
            assert abs((loss(xf + s, wf) - loss(xf - s, wf)) / (2 * e) - dx[i, j]) < 1e-5
    for j in range(d):
        s = np.zeros(d)
        s[j] = e
        assert abs((loss(xf, wf + s) - loss(xf, wf - s)) / (2 * e) - dw[j]) < 1e-5


def test_backward_of_nothing_and_without_weight(pi):
    x = torch.zeros(0, 96, dtype=torch.float16, device="cuda")
    none = torch.zeros(0, device="cuda")
    dx, dw, db = pi.layer_norm_backward(x, x, None, none, none)
    assert dx.shape == (0, 96) and not dw.any() and not db.any()
    x, dy = rand((5, 96), "float16", 1), rand((5, 96), "float16", 2)
    _, _, mean, rstd = pi.layer_norm(x, want_stats=True)
    one = torch.ones(96, device="cuda")
    for a, b in zip(pi.layer_norm_backward(dy, x, None, mean, rstd), pi.layer_norm_backward(dy, x, one, mean, rstd)):
        assert torch.equal(a, b)


def test_backward_strided_x(pi):
    wide = rand((40, 300), "float16", 1)
    dy, w = rand((40, 96), "float16", 2), rand(96, "float32", 3)
    for at in (0, 3):
        x = wide[:, at:at + 96]
        _, _, mean, rstd = pi.layer_norm(x, w, want_stats=True)
        a = pi.layer_norm_backward(dy, x, w, mean, rstd)
        b = pi.layer_norm_backward(dy, x.contiguous(), w, mean, rstd)
        for s, t in zip(a, b):
            np.testing.assert_allclose(f64(s), f64(t), rtol=2e-3, atol=2e-3)


def test_other_stream_and_graph(pi):
    x, dy, w = rand((300, 1024), "bfloat16", 1), rand((300, 1024), "bfloat16", 2), rand(1024, "bfloat16", 3)
    y, _, mean, rstd = pi.layer_norm(x, w, want_stats=True)
    ref = pi.layer_norm_backward(dy, x, w, mean, rstd)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y2, _, m2, r2 = pi.layer_norm(x, w, want_stats=True, stream=s)
    got = pi.layer_norm_backward(dy, x, w, m2, r2, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(y, y2) and all(torch.equal(a, b) for a, b in zip(ref, got))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = pi.layer_norm_backward(dy, x, w, mean, rstd)
    g.replay()
    assert all(torch.equal(a, b) for a, b in zip(ref, got))


def test_refusals(pi):
    x, w = rand((4, 96), "float16", 1), rand(96, "float32", 2)
    m = torch.zeros(4, device="cuda")
    with pytest.raises(TypeError):
        pi.layer_norm(x.double(), w)
    with pytest.raises(TypeError):
        pi.layer_norm(x.cpu(), w)
    with pytest.raises(ValueError):
        pi.layer_norm(x, w[:95])
    with pytest.raises(TypeError):
        pi.layer_norm(x, w, w.half())
    with pytest.raises(ValueError):
        pi.layer_norm(x.t(), rand(4, "float32", 2))
    with pytest.raises(ValueError):
        pi.layer_norm(x, w, add=x[:3])
    with pytest.raises(ValueError):
        pi.layer_norm(x, w, sum=x)
    with pytest.raises(pi.PiError):
        pi.layer_norm(x, w, eps=-1.0)
    with pytest.raises(pi.PiError):
        pi.layer_norm(rand((1, 16385), "float16", 1))
    with pytest.raises(ValueError):
        pi.layer_norm_backward(x, x, w, m[:3], m)
    with pytest.raises(TypeError):
        pi.layer_norm_backward(x.float(), x, w, m, m)
    with pytest.raises(pi.PiError):
        pi.layer_norm_backward(x, x, w, m, m, ws=torch.empty(8, dtype=torch.uint8, device="cuda"))
