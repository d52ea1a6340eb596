"""Range of the gated block's gradients in fp16: the operands dG and dU leave fp16
where the gradients that they lead to do not."""
import math

import pytest
import torch

import decode_projection_gemms_gb300 as kda
from decode_projection_gemms_gb300 import binding
from ffn_ref import D1, D2, UNIT, acc_bound, act as act64, product_bounds

pytestmark = pytest.mark.gpu
ACTS = ("silu", "gelu", "gelu_tanh")
HALF = (torch.bfloat16, torch.float16)


def normal(rows, cols, seed, dtype, std):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn((rows, cols), generator=g, device="cuda") * std).to(dtype)


def reference(dh, x, Wg, Wu, act, dtype):
    """{name: (gradient, bound on its error before its own rounding)}. An operand is
    rounded to 16 bits: off by its unit, or in fp16 by 2^-39 of the largest operand
    (it is scaled to [2^14, 2^15), where a subnormal is off by at most 2^-25)."""
    dh, x, Wg, Wu = (t.double() for t in (dh, x, Wg, Wu))
    g, eg = product_bounds(x, Wg)
    u, eu = product_bounds(x, Wu)
    a, da = act64(g, act)
    dg, du = dh * u * da, dh * a
    d = dh.abs()
    fp = 2.0 ** -19 * (1 + g.abs())       # act and act' in fp32
    edg = d * (eu * D1 + (u.abs() + eu) * (D2 * eg + fp))
    edu = d * (D1 * eg + fp)
    low = 2.0 ** -39 * 1.01 * max(dg.abs().max().item(), du.abs().max().item()) if dtype is torch.float16 else 0.0
    edg = edg + UNIT[dtype] * (dg.abs() + edg) + low
    edu = edu + UNIT[dtype] * (du.abs() + edu) + low
    F, T = g.shape[1], g.shape[0]
    out = {"dx": (dg @ Wg + du @ Wu,
                  edg @ Wg.abs() + edu @ Wu.abs() + acc_bound(dg.abs() + edg, Wg, 2 * F)
                  + acc_bound(du.abs() + edu, Wu, 2 * F))}
    for key, v, e in (("dWg", dg, edg), ("dWu", du, edu)):
        out[key] = (v.t() @ x, e.t() @ x.abs() + acc_bound((v.abs() + e).t(), x, T))
    return out, max(dg.abs().max().item(), du.abs().max().item())


def check(got, ref, bound, what):
    """Against the formula within the output's rounding plus the bound, wherever the
    output's type holds the value."""
    dt = got.dtype
    tol = UNIT[dt] * (ref.abs() + bound) + bound + (2.0 ** -25 if dt is torch.float16 else 2.0 ** -134)
    fits = ref.abs() + tol < torch.finfo(dt).max
    assert fits.double().mean() > 0.99
    g = got.double()[fits]
    assert torch.isfinite(g).all(), f"{what}: not finite"
    worst = ((g - ref[fits]).abs() / tol[fits]).max().item()
    assert worst <= 1.0, f"{what}: {worst:.3f} of the tolerance"


def gradients(dh, x, Wg, Wu, act):
    _, g, u = kda.gated_ffn(x, Wg, Wu, act=act, save=True)
    return kda.gated_ffn_backward(dh, x, Wg, Wu, g, u, act=act)


SIZES = [(24, 64, 256), (1, 40, 64), (300, 264, 256), (65, 101, 256), (3, 2048, 2048), (700, 1000, 520)]


@pytest.mark.parametrize("T,F,K", SIZES)
def test_large_gradients_stay_finite(T, F, K):
    """dh in the thousands and u in the tens: dG passes 65504, its products with
    small weights and small activations do not."""
    dt, act = torch.float16, ACTS[T % 3]
    x = normal(T, K, 1, dt, 0.05)
    Wg, Wu = normal(F, K, 2, dt, 0.01 * (64 / max(F, T)) ** 0.5), normal(F, K, 3, dt, 12 * (256 / K) ** 0.5)
    dh = normal(T, F, 4, dt, 1500)
    dh[0, (x[0].double() @ Wu.double().t()).abs().argmax()] = 2e4
    ref, top = reference(dh, x, Wg, Wu, act, dt)
    assert top > 65504
    for got, name in zip(gradients(dh, x, Wg, Wu, act), ("dx", "dWg", "dWu")):
        check(got, *ref[name], f"{name} {T}x{F}x{K}")
    torch.cuda.synchronize()
    assert binding.device_error() == 0


@pytest.mark.parametrize("T,F,K", SIZES)
def test_small_gradients_keep_their_precision(T, F, K):
    """dh of a few 1e-6: dG and dU fall to fp16's subnormals, their products with
    large activations and weights do not."""
    dt, act = torch.float16, ACTS[T % 3]
    x = normal(T, K, 1, dt, 30)
    Wg, Wu = (normal(F, K, s, dt, K ** -0.5 / 30) for s in (2, 3))
    dh = normal(T, F, 4, dt, 3e-6)
    ref, top = reference(dh, x, Wg, Wu, act, dt)
    assert 0 < top < 2.0 ** -14
    for got, name in zip(gradients(dh, x, Wg, Wu, act), ("dx", "dWg", "dWu")):
        check(got, *ref[name], f"{name} {T}x{F}x{K}")


@pytest.mark.parametrize("dtype", HALF)
@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
def test_a_non_finite_gradient_reaches_its_row_and_feature_only(dtype, bad):
    T, F, K = 70, 96, 128
    x, dh = normal(T, K, 1, dtype, 1.0), normal(T, F, 2, dtype, 0.05)
    Wg, Wu = normal(F, K, 3, dtype, 0.12), normal(F, K, 4, dtype, 0.09)
    t, f = 41, 17
    dh[t, f] = 0
    ref, _ = reference(dh, x, Wg, Wu, "silu", dtype)
    dh[t, f] = bad
    dx, dWg, dWu = gradients(dh, x, Wg, Wu, "silu")
    assert not torch.isfinite(dx[t]).any()
    assert not torch.isfinite(dWg[f]).any() and not torch.isfinite(dWu[f]).any()
    for got, name, row in ((dx, "dx", t), (dWg, "dWg", f), (dWu, "dWu", f)):
        keep = torch.arange(got.shape[0], device="cuda") != row
        check(got[keep], ref[name][0][keep], ref[name][1][keep], name)


@pytest.mark.parametrize("T,F", [(1, 8), (33, 104), (33, 101)])
def test_zero_gradients(T, F):
    K = 64
    for dt in HALF:
        x, W = normal(T, K, 1, dt, 1.0), normal(F, K, 2, dt, 0.1)
        for out in gradients(torch.zeros((T, F), dtype=dt, device="cuda"), x, W, W, "silu"):
            assert (out == 0).all()
