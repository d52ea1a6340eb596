"""Layer norm, with and without centring, and its gradients on the GPU against plain
64-bit forms."""
import math

import pytest
import torch

import decode_projection_gemms_gb300 as kda
from decode_projection_gemms_gb300 import binding
from ffn_ref import TINY, UNIT

pytestmark = pytest.mark.gpu
TYPES = (torch.bfloat16, torch.float16, torch.float32)
SIZES = [(1, 1), (1, 7168), (3, 8), (5, 255), (7, 256), (2, 257), (9, 512), (33, 520), (130, 1000), (6, 1024), (11, 1032),
         (64, 2048), (17, 2056), (40, 4096), (23, 4104), (300, 7168), (5, 8192), (3, 8200), (4, 16384), (2000, 64), (1500, 264)]
U = 2.0 ** -24


def normal(*shape, seed, dtype=torch.float32, std=1.0, mean=0.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * std + mean).to(dtype)


def rounding(ref, tol, dtype):
    return tol + UNIT.get(dtype, U) * (ref.abs() + tol) + TINY.get(dtype, 2.0 ** -149)


def strided(t, extra, offset=0):
    rows, cols = t.shape
    wide = torch.full((rows, cols + extra + offset), math.nan, dtype=t.dtype, device=t.device)
    v = wide[:, offset:offset + cols]
    v.copy_(t)
    return v


def check_forward(x, w, b, eps, center, y, mean, rstd):
    xd = x.double()
    K = x.shape[1]
    mu = xd.mean(dim=1, keepdim=True) if center else torch.zeros_like(xd[:, :1])
    # at most 64 fp32 steps in a sum of a row
    emu = 64 * U * xd.abs().mean(dim=1, keepdim=True) if center else 0 * mu
    d = xd - mu
    var = (d * d).mean(dim=1, keepdim=True)
    # squares: their own sum, and a mean that is off by emu
    evar = 70 * U * var + 2 * emu * d.abs().mean(dim=1, keepdim=True) + emu ** 2
    r = 1 / torch.sqrt(var + eps)
    er = r * (0.5 * evar / (var + eps - evar).clamp(min=1e-300) + 8 * U)
    assert ((rstd.double().unsqueeze(1) - r).abs() <= er).all()
    if center:
        assert ((mean.double().unsqueeze(1) - mu).abs() <= emu + U * mu.abs()).all()
    wd = w.double()
    ref = d * r * wd + (b.double() if b is not None else 0)
    tol = wd.abs() * (r * (emu + 2 * U * d.abs()) + d.abs() * er + 4 * U * (d * r).abs()) + 2 * U * ref.abs()
    assert ((y.double() - ref).abs() <= rounding(ref, tol, y.dtype)).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,K", SIZES)
def test_layer_norm(T, K, dtype):
    x = normal(T, K, seed=1, dtype=dtype, mean=0.5)
    w, b = normal(K, seed=2, dtype=dtype, mean=1.0), normal(K, seed=3, dtype=dtype)
    for center, bias in ((True, b), (True, None), (False, None), (False, b)):
        y, mean, rstd = kda.layer_norm(x, w, bias, eps=1e-3, center=center, save=True)
        assert (mean is None) == (not center)
        check_forward(x, w, bias, 1e-3, center, y, mean, rstd)
        assert torch.equal(kda.layer_norm(x, w, bias, eps=1e-3, center=center), y)


@pytest.mark.parametrize("dtype", TYPES)
def test_rows_far_from_zero_and_constant_rows(dtype):
    K = 4096
    x = normal(4, K, seed=1, dtype=dtype, std=4.0, mean=2000.0)    # a mean far above the spread
    x[1] = 7.0                                                     # no spread at all
    x[2] = 0.0
    x[3] = normal(K, seed=5, dtype=dtype, std=1e-3)
    w, b = normal(K, seed=2, dtype=dtype), normal(K, seed=3, dtype=dtype)
    y, mean, rstd = kda.layer_norm(x, w, b, save=True)
    check_forward(x, w, b, 1e-5, True, y, mean, rstd)
    assert torch.equal(y[1], b) and torch.equal(y[2], b)


def test_non_finite_rows_stay_by_themselves():
    x, w = normal(6, 520, seed=1, dtype=torch.bfloat16), normal(520, seed=2, dtype=torch.bfloat16)
    want = kda.layer_norm(x, w)
    x[2, 3], x[4, 519] = math.nan, math.inf
    y = kda.layer_norm(x, w)
    assert torch.isnan(y[2]).all() and torch.isnan(y[4]).any()
    keep = [0, 1, 3, 5]
    assert torch.equal(y[keep], want[keep])


def check_backward(dy, x, w, mean, rstd, got):
    """From the same statistics."""
    dx, dw, db = got
    T, K = x.shape
    d, xd, wd, r = dy.double(), x.double(), w.double(), rstd.double().unsqueeze(1)
    mu = mean.double().unsqueeze(1) if mean is not None else torch.zeros_like(r)
    xh = (xd - mu) * r
    exh = 2 * U * (xd.abs() + mu.abs()) * r
    g = d * wd
    a = g.mean(dim=1, keepdim=True) if mean is not None else 0 * r
    m = (g * xh).mean(dim=1, keepdim=True)
    # at most 64 fp32 steps in a sum of a row
    ea = 64 * U * g.abs().mean(dim=1, keepdim=True) if mean is not None else 0 * r
    em = 66 * U * (g * xh).abs().mean(dim=1, keepdim=True) + (g.abs() * exh).mean(dim=1, keepdim=True)
    ref = r * (g - a - xh * m)
    tol = r * (ea + xh.abs() * em + exh * (m.abs() + em) + 4 * U * (g.abs() + a.abs() + (xh * m).abs())) + 2 * U * ref.abs()
    assert ((dx.double() - ref).abs() <= rounding(ref, tol, dx.dtype)).all()
    # a column's sum: T / 152 rows of a block, four teams, 32 runs of blocks
    steps = T / 152 + 64
    ref = (d * xh).sum(dim=0)
    tol = steps * U * (d * xh).abs().sum(dim=0) + (d.abs() * exh).sum(dim=0)
    assert ((dw.double() - ref).abs() <= rounding(ref, tol, dw.dtype)).all()
    if db is not None:
        ref = d.sum(dim=0)
        assert ((db.double() - ref).abs() <= rounding(ref, steps * U * d.abs().sum(dim=0), db.dtype)).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,K", SIZES)
def test_layer_norm_backward(T, K, dtype):
    x, dy = normal(T, K, seed=1, dtype=dtype, mean=0.5), normal(T, K, seed=2, dtype=dtype, std=0.3)
    w = normal(K, seed=3, dtype=dtype, mean=1.0)
    for center in (True, False):
        _, mean, rstd = kda.layer_norm(x, w, eps=1e-3, center=center, save=True)
        got = kda.layer_norm_backward(dy, x, w, mean, rstd, bias=True)
        assert all(t.dtype is dtype for t in got)
        check_backward(dy, x, w, mean, rstd, got)
        again = kda.layer_norm_backward(dy, x, w, mean, rstd)
        assert again[2] is None and torch.equal(again[0], got[0]) and torch.equal(again[1], got[1])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,K", [(20000, 128), (5000, 2048), (3000, 7168)])
def test_many_rows(T, K, dtype):
    x, dy, w = normal(T, K, seed=1, dtype=dtype), normal(T, K, seed=2, dtype=dtype), normal(K, seed=3, dtype=dtype)
    y, mean, rstd = kda.layer_norm(x, w, save=True)
    check_forward(x, w, None, 1e-5, True, y, mean, rstd)
    check_backward(dy, x, w, mean, rstd, kda.layer_norm_backward(dy, x, w, mean, rstd, bias=True))


@pytest.mark.parametrize("center", [True, False])
def test_gradients_of_the_definition(center):
    """Against automatic differentiation, statistics included."""
    T, K = 37, 520
    x, dy, w, b = (normal(*s, seed=i) for i, s in enumerate(((T, K), (T, K), (K,), (K,))))
    _, mean, rstd = kda.layer_norm(x, w, b, center=center, save=True)
    got = kda.layer_norm_backward(dy, x, w, mean, rstd, bias=True)
    xd, wd, bd = (t.double().requires_grad_() for t in (x, w, b))
    d = xd - xd.mean(dim=1, keepdim=True) if center else xd
    (d / torch.sqrt((d * d).mean(dim=1, keepdim=True) + 1e-5) * wd + bd).backward(dy.double())
    for a, want in zip(got, (xd.grad, wd.grad, bd.grad)):
        assert float((a.double() - want).norm() / want.norm()) < 2.0 ** -20     # fp32 throughout


def test_gradients_against_differences():
    T, K, step = 4, 40, 1e-4
    x, dy, w = normal(T, K, seed=1), normal(T, K, seed=2), normal(K, seed=3)
    for center in (True, False):
        _, mean, rstd = kda.layer_norm(x, w, center=center, save=True)
        dx, dw, _ = kda.layer_norm_backward(dy, x, w, mean, rstd)

        def loss(xv, wv):
            d = xv - xv.mean(dim=1, keepdim=True) if center else xv
            return float((dy.double() * d / torch.sqrt((d * d).mean(dim=1, keepdim=True) + 1e-5) * wv).sum())

        u, v = normal(T, K, seed=8).double(), normal(K, seed=9).double()
        for grad, way, f in ((dx, u, lambda s: loss(x.double() + s * u, w.double())),
                             (dw, v, lambda s: loss(x.double(), w.double() + s * v))):
            slope = (f(step) - f(-step)) / (2 * step)
            # fp32 gradients; a third derivative of a few units a term
            assert abs(float((grad.double() * way).sum()) - slope) < 1e-5 * float((grad.double() * way).abs().sum()) + 1e-6 * T * K


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("extra,offset", [(8, 8), (3, 1), (8, 4)])
def test_strides_and_nothing_written_outside(extra, offset, dtype):
    for T, K in ((9, 200), (12, 1160)):
        x, dy, w = (normal(*s, seed=i, dtype=dtype) for i, s in enumerate(((T, K), (T, K), (K,))))
        want, mean, rstd = kda.layer_norm(x, w, save=True)
        y = torch.full((T + 2, K + extra + offset), 5.0, dtype=dtype, device="cuda")
        got = kda.layer_norm(strided(x, extra, offset), w, y=y[1:-1, offset:offset + K], save=True)
        check_forward(x, w, None, 1e-5, True, got[0], *got[1:])
        assert torch.equal(got[0], want)
        y[1:-1, offset:offset + K] = 5.0
        assert (y == 5.0).all()
        check_backward(dy, x, w, mean, rstd, kda.layer_norm_backward(strided(dy, extra, offset), strided(x, extra, offset), w,
                                                                     mean, rstd, bias=True))


def test_stream_graph_and_no_rows():
    T, K, dt = 700, 1032, torch.bfloat16

    def inputs(seed):
        return tuple(normal(*s, seed=seed + i, dtype=dt) for i, s in enumerate(((T, K), (T, K), (K,))))

    def step(x, dy, w, stream=None):
        y, mean, rstd = kda.layer_norm(x, w, save=True, stream=stream)
        return [y, mean, rstd, *kda.layer_norm_backward(dy, x, w, mean, rstd, bias=True, stream=stream)]

    want = step(*inputs(1))
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = step(*inputs(1), stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    static = inputs(1)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = step(*static)
    for seed in (11, 21):
        for a, b in zip(static, inputs(seed)):
            a.copy_(b)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(step(*inputs(seed)), outs))
    e = torch.empty((0, K), dtype=dt, device="cuda")
    y, mean, rstd = kda.layer_norm(e, static[2], save=True)
    dx, dw, db = kda.layer_norm_backward(e, e, static[2], mean, rstd, bias=True)
    assert y.shape == (0, K) and dx.shape == (0, K) and not dw.any() and not db.any()
    assert binding.device_error() == 0
