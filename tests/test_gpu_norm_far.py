"""Gradients of the layer norm where a row's mean is far above its spread, where its numbers are
very small or very large, and where a team of warps goes over many rows."""
import pytest
import torch

import decode_projection_gemms_gb300 as kda
from decode_projection_gemms_gb300 import binding
from test_gpu_norm import TYPES, U, normal, rounding

pytestmark = pytest.mark.gpu


def check(dy, x, w, mean, rstd, got):
    """From the same statistics: x - mean is rounded once and its product with rstd once, so
    xhat is off by a share of itself, however far the row lies from zero."""
    dx, dw, db = got
    T, K = x.shape
    d, xd, wd, r = dy.double(), x.double(), w.double(), rstd.double().unsqueeze(1)
    mu = mean.double().unsqueeze(1) if mean is not None else torch.zeros_like(r)
    xh = (xd - mu) * r
    exh = 2.01 * U * xh.abs()
    g = d * wd
    a = g.mean(dim=1, keepdim=True) if mean is not None else 0 * r
    m = (g * xh).mean(dim=1, keepdim=True)
    # a sum of a row: 32 columns of a thread at most, ten exchanges and a division; the sum of g
    # xhat has each g rounded too
    ea = 64 * U * g.abs().mean(dim=1, keepdim=True) if mean is not None else 0 * r
    em = 66 * U * (g * xh).abs().mean(dim=1, keepdim=True) + (g.abs() * exh).mean(dim=1, keepdim=True)
    ref = r * (g - a - xh * m)
    # roundings: x - mean, rstd m, g - a, their sum, the product with rstd
    tol = r * (ea + xh.abs() * em + 4 * U * (g.abs() + a.abs() + (xh * m).abs())) + 2 * U * ref.abs()
    assert ((dx.double() - ref).abs() <= rounding(ref, tol, dx.dtype)).all()
    # a column's sum: T / 152 rows of a team, sixteen teams, 32 runs of blocks
    steps = T / 152 + 64
    ref = (d * xh).sum(dim=0)
    tol = steps * U * (d * xh).abs().sum(dim=0) + (d.abs() * exh).sum(dim=0)
    assert ((dw.double() - ref).abs() <= rounding(ref, tol, dw.dtype)).all()
    ref = d.sum(dim=0)
    assert ((db.double() - ref).abs() <= rounding(ref, steps * U * d.abs().sum(dim=0), db.dtype)).all()


def run(x, dy, w, center=True, eps=1e-5):
    _, mean, rstd = kda.layer_norm(x, w, eps=eps, center=center, save=True)
    got = kda.layer_norm_backward(dy, x, w, mean, rstd, bias=True)
    check(dy, x, w, mean, rstd, got)
    return got


@pytest.mark.parametrize("center", [True, False])
@pytest.mark.parametrize("K", [8, 257, 264, 4096, 4103, 16384])
@pytest.mark.parametrize("dtype", TYPES)
def test_rows_far_from_zero(dtype, K, center):
    far, std = (1e5, 1.0) if dtype is torch.float32 else (2000.0, 16.0)
    x, dy, w = normal(9, K, seed=1, dtype=dtype, std=std, mean=far), normal(9, K, seed=2, dtype=dtype), normal(K, seed=3, dtype=dtype)
    x[3] = normal(K, seed=4, dtype=dtype, std=std, mean=-far / 7)
    x[4] = 0.3       # a mean that is rounded
    run(x, dy, w, center)


@pytest.mark.parametrize("K", [520, 1031])
@pytest.mark.parametrize("dtype", TYPES)
def test_constant_rows_have_no_gradient_of_the_weight(dtype, K):
    x = torch.full((5, K), 2000.0, device="cuda").to(dtype)      # the sum of a row is exact in fp32
    dy, w = normal(5, K, seed=2, dtype=dtype), normal(K, seed=3, dtype=dtype)
    _, dw, _ = run(x, dy, w)
    assert not dw.any()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("std", [2e-19, 1e17])
def test_rows_of_very_small_and_very_large_numbers(std, dtype):
    """rstd is 5e18 or 1e-17 and its square passes fp32's range, or nearly."""
    K = 512
    x, w = normal(6, K, seed=1, dtype=dtype, std=std), torch.ones(K, dtype=dtype, device="cuda")
    dy = (40.0 * torch.sign(x.float()) + normal(6, K, seed=2)).to(dtype)      # mean(g xhat) is about 32
    for center in (True, False):
        dx, dw, _ = run(x, dy, w, center, eps=0.0)
        assert torch.isfinite(dx).all() and torch.isfinite(dw).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,K", [(6000, 255), (2000, 4103), (1200, 8201), (1000, 16383), (1500, 8200), (1000, 16384)])
def test_many_rows_of_a_team(T, K, dtype):
    """Every team takes several rows, through shared memory and element by element."""
    run(normal(T, K, seed=1, dtype=dtype, mean=3.0), normal(T, K, seed=2, dtype=dtype), normal(K, seed=3, dtype=dtype))
    assert binding.device_error() == 0
