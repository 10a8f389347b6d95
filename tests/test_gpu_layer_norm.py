"""GPU tests of the layer norm and its backward pass against the float64 oracle.

Bounds, with u = 2^-24 and W columns: the mean is a float32 sum of W terms
(W u of the mean magnitude), the variance is centred on it, so that xh is off
by (W + 16) u (|xh| + sqrt(mean x^2) rstd) at most: far rows lose what float32
holds of x - mu and no more.  Outputs of bf16 are rounded once (2^-8).  The
weight sums add n rows in float32: n u of their terms' magnitudes."""
import numpy as np
import pytest
import torch

from oracle.molecule import layer_norm
from oracle.storage import round_bf16
from tests.molecule_util import B, U, close

pytestmark = pytest.mark.gpu


def _egat():
    from equivariant_graph_attention_b200 import egat
    return egat


def _data(n, W, dtype, seed=0, offset=0.3):
    r = np.random.default_rng(seed)
    st = round_bf16 if dtype == "bf16" else lambda a: a.astype(np.float32).astype(np.float64)
    f = lambda a: a.astype(np.float32).astype(np.float64)
    return (st(r.normal(size=(n, W)) * 1.5 + offset), st(r.normal(size=(n, W))), f(1 + 0.2 * r.normal(size=W)),
            f(0.2 * r.normal(size=W)))


def _place(a, dtype, ld=None, shift=0):
    """The rows on the GPU with this stride, `shift` elements into a buffer."""
    T = torch.bfloat16 if dtype == "bf16" else torch.float32
    n, W = a.shape
    ld = ld or W
    buf = torch.full((shift + n * ld + 8,), 99.0, dtype=T, device="cuda")
    v = buf[shift:shift + n * ld].view(n, ld)[:, :W] if n else buf[:0].view(0, W)
    v.copy_(torch.from_numpy(a))
    return buf, v


def _check(n, W, dtype, x, g, w, b, ld=None, shift=0, eps=1e-5):
    egat = _egat()
    rb = B if dtype == "bf16" else 0.0
    _, xt = _place(x, dtype, ld, shift)
    _, gt = _place(g, dtype, ld, shift)
    ybuf, yt = _place(np.zeros((n, W)), dtype, ld, shift)
    dbuf, dt = _place(np.zeros((n, W)), dtype, ld, shift)
    wt, bt = (None if a is None else torch.from_numpy(a).float().cuda() for a in (w, b))
    y, stats = egat.egat_layer_norm(xt, wt, bt, eps=eps, want_stats=True, out=yt)
    dx, dw, db = egat.egat_layer_norm_backward(xt, wt, stats, gt, out=dt)
    o = layer_norm(x, w, b, eps=eps, grad=g)
    one = np.ones(W) if w is None else np.abs(w)
    size = np.sqrt((x ** 2).mean(1, keepdims=True)) * o["rstd"][:, None]
    ez = (W + 16) * U * (np.abs(o["z"]) + size + 1)
    close(y, o["y"], ez * one + (8 * U + rb) * np.abs(o["y"]), "y")
    close(stats[:, 0], o["mu"], (W + 16) * U * np.abs(x).mean(1) + 1e-30, "mu")
    close(stats[:, 1], o["rstd"], (2 * W + 32) * U * (1 + size[:, 0] ** 2 * (W + 16) * U) * o["rstd"] * (1 + size[:, 0]), "rstd")
    top = np.abs(g).max(initial=0)
    close(dx, o["dx"], ((3 * W + 64) * U * (1 + size)) * o["abs_dx"]
          + o["rstd"][:, None] * ez.max(1, keepdims=True, initial=0) * 3 * np.abs(g * one).max(1, keepdims=True, initial=0) * (np.abs(o["z"]) + 1)
          + rb * np.abs(o["dx"]), "dx")
    close(dw, o["dweight"], (n + 16) * U * o["abs_dweight"] + ez.sum(0) * top + 1e-30, "dweight")
    close(db, o["dbias"], (n + 16) * U * o["abs_dbias"] + 1e-30, "dbias")
    if ld and ld > W and n:    # what lies between the rows stays as it was
        for buf in (ybuf, dbuf):
            gap = buf[shift:shift + n * ld].view(n, ld)[:, W:]
            assert (gap == 99).all()
        assert (ybuf[:shift] == 99).all() and (ybuf[shift + n * ld:] == 99).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n,W", [(1, 1), (3, 2), (5, 7), (33, 8), (70, 16), (1, 128), (1000, 128), (3, 100), (9, 257),
                                 (40, 1000), (7, 1022), (6, 1024), (6, 1032), (3, 2050), (5, 4096), (2, 4099),
                                 (3, 8192), (2, 16384), (2, 16383), (20000, 24)])
def test_sizes(n, W, dtype):
    x, g, w, b = _data(n, W, dtype)
    _check(n, W, dtype, x, g, w, b)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("W,ld,shift", [(128, 1152, 0), (128, 1152, 128), (128, 130, 1), (128, 131, 0), (64, 72, 8),
                                        (1000, 1001, 3), (4, 4, 1)])
def test_strides_and_alignment(W, ld, shift, dtype):
    x, g, w, b = _data(37, W, dtype)
    _check(37, W, dtype, x, g, w, b, ld, shift)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_without_weight_or_bias_and_with_other_eps(dtype):
    x, g, w, b = _data(19, 96, dtype)
    _check(19, 96, dtype, x, g, None, None)
    _check(19, 96, dtype, x, g, w, None, eps=0.0)
    _check(19, 96, dtype, x, g, None, b, eps=0.5)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rows_far_from_zero_and_constant_rows(dtype):
    x, g, w, b = _data(16, 256, dtype, offset=0.0)
    x[:8] = round_bf16(x[:8] * 64 + 16384) if dtype == "bf16" else (x[:8] + 1000).astype(np.float32)
    x[3] = 5.0
    _check(16, 256, dtype, x, g, w, b)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_in_place_and_nan_rows(dtype):
    egat = _egat()
    x, g, w, b = _data(50, 128, dtype)
    _, xt = _place(x, dtype)
    _, gt = _place(g, dtype)
    wt, bt = torch.from_numpy(w).float().cuda(), torch.from_numpy(b).float().cuda()
    y, stats = egat.egat_layer_norm(xt, wt, bt, want_stats=True)
    dx, _, _ = egat.egat_layer_norm_backward(xt, wt, stats, gt)
    bad = xt.clone()
    bad[7, 3], bad[8, 0] = float("nan"), float("inf")
    keep = [i for i in range(50) if i not in (7, 8)]
    y2, _ = egat.egat_layer_norm(bad, wt, bt)
    assert torch.equal(y2[keep], y[keep]) and torch.isnan(y2[7]).all() and torch.isnan(y2[8]).any()
    egat.egat_layer_norm_backward(xt, wt, stats, gt, out=gt)      # dx over the gradient
    assert torch.equal(gt, dx)
    egat.egat_layer_norm(xt, wt, bt, out=xt)                      # y over x
    assert torch.equal(xt, y)


def test_no_rows():
    egat = _egat()
    x = torch.empty((0, 64), device="cuda")
    y, stats = egat.egat_layer_norm(x, want_stats=True)
    dx, dw, db = egat.egat_layer_norm_backward(x, None, stats, x)
    assert y.shape == dx.shape == (0, 64) and not dw.any() and not db.any()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_captured_and_repeated(dtype):
    egat = _egat()
    x, g, w, b = _data(3001, 128, dtype)
    _, xt = _place(x, dtype, 1152)
    _, gt = _place(g, dtype)
    wt, bt = torch.from_numpy(w).float().cuda(), torch.from_numpy(b).float().cuda()

    def step():
        y, stats = egat.egat_layer_norm(xt, wt, bt, want_stats=True)
        return (y, stats) + egat.egat_layer_norm_backward(xt, wt, stats, gt)

    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for k in range(3):
        xt.mul_(-1.5)
        graph.replay()
        torch.cuda.synchronize()
        again = step()
        for a, c in zip(out, again):
            assert torch.equal(a, c)
