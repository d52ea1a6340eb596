"""The activations far from zero, relative to their values: an absolute bound says
nothing where the activation itself is small. One live column for the gate and one
for its factor choose g and u = 1 exactly."""
import math

import pytest
import torch

import decode_projection_gemms_gb300 as kda
from ffn_ref import TINY, UNIT, mx4_values

pytestmark = pytest.mark.gpu
HALF = (torch.bfloat16, torch.float16)

# In fp32: an argument z of an exponential carries a few roundings of 2^-24 |z|, the
# exponential itself 2 + 1.16 |z| units of 2^-23, and the complementary error function
# (2 z^2 + 8) of them. With |z| <= 80 and z^2 <= 72 all stay below 2^-14 of the value;
# the derivative is a sum of two such terms of which one dominates below -2.
FP32 = 2.0 ** -13


def act64(g, name):
    """(act(g), act'(g)) in 64 bits, without cancellation for negative g."""
    if name == "silu":
        s = torch.special.expit(g)
        return g * s, s + g * s * torch.special.expit(-g)
    if name == "gelu":
        cdf = 0.5 * torch.special.erfc(-g / math.sqrt(2))
        return g * cdf, cdf + g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)
    c = 2 * math.sqrt(2 / math.pi)
    s = torch.special.expit(c * (g + 0.044715 * g ** 3))
    return g * s, s + g * s * torch.special.expit(-c * (g + 0.044715 * g ** 3)) * c * (1 + 3 * 0.044715 * g ** 2)


def near(got, ref, dtype, what):
    tol = (UNIT[dtype] + FP32) * 1.01 * ref.abs() + TINY[dtype]
    g = got.double()
    assert torch.isfinite(g).all(), what
    worst = ((g - ref).abs() / tol).max().item()
    assert worst <= 1.0, f"{what}: {worst:.3f} of the tolerance"


def operands(g, F, K, dtype):
    """x, Wg, Wu with x Wg^T = g and x Wu^T = 1 in every feature."""
    x = torch.zeros((g.numel(), K), dtype=dtype, device="cuda")
    x[:, 0], x[:, 32] = g.to(dtype), 1.0
    Wg, Wu = (torch.zeros((F, K), dtype=dtype, device="cuda") for _ in range(2))
    Wg[:, 0], Wu[:, 32] = 1.0, 1.0
    return x, Wg, Wu


def tail(lo, hi, n, dtype):
    return torch.linspace(lo, hi, n, dtype=torch.float64).to(dtype).cuda()


# where the 16-bit types still have values, and fp32 has normal ones
LEFT = [("silu", -80.0), ("gelu", -12.0), ("gelu_tanh", -9.5)]


@pytest.mark.parametrize("dtype", HALF)
@pytest.mark.parametrize("tokens,F", [(7, 8), (100, 40), (2500, 128)])
@pytest.mark.parametrize("act,lo", LEFT)
def test_left_tail(act, lo, tokens, F, dtype):
    g = tail(lo, -2.0, tokens, dtype)
    x, Wg, Wu = operands(g, F, 64, dtype)
    h = kda.gated_ffn(x, Wg, Wu, act=act)
    near(h, act64(g.double(), act)[0][:, None].expand(-1, F), dtype, f"{act} of {tokens} tokens")


@pytest.mark.parametrize("dtype", HALF)
@pytest.mark.parametrize("act,lo", LEFT)
def test_left_tail_gradients(act, lo, dtype):
    """One feature: dx holds act'(g) under the gate's column and act(g) under its
    factor's. fp16: one power of two scales all tokens, so as many of them as it holds
    with full precision (2^-28 of the largest)."""
    g = tail(lo if dtype is torch.bfloat16 else -4.5, -2.0, 300, dtype)
    x, Wg, Wu = operands(g, 1, 64, dtype)
    dh = torch.ones((300, 1), dtype=dtype, device="cuda")
    _, gs, us = kda.gated_ffn(x, Wg, Wu, act=act, save=True)
    dx, _, _ = kda.gated_ffn_backward(dh, x, Wg, Wu, gs, us, act=act)
    a, da = act64(g.double(), act)
    near(dx[:, 0], da, dtype, f"{act}'")
    near(dx[:, 32], a, dtype, act)


@pytest.mark.parametrize("tokens", [4, 12, 300])
@pytest.mark.parametrize("act", [a for a, _ in LEFT])
def test_left_tail_over_4_bits(act, tokens):
    g = torch.tensor([-2.0, -3.0, -4.0, -6.0, -8.0, -0.5, -1.0, -1.5, 2.0, 3.0, 6.0, 8.0], dtype=torch.float64)
    g = g.repeat(-(-tokens // 12))[:tokens].cuda()
    x, Wg, Wu = operands(g, 130, 64, torch.bfloat16)
    assert torch.equal(mx4_values(x), x.double())
    h = kda.mx4_gated_ffn(x, kda.mx4_quantize(Wg), kda.mx4_quantize(Wu), act=act)
    near(h, act64(g, act)[0][:, None].expand(-1, 130), torch.bfloat16, act)


@pytest.mark.parametrize("act", [a for a, _ in LEFT])
def test_gradients_of_huge_gates(act):
    """bf16 reaches 3e38, and g^2 and g^3 pass fp32 long before: the activation is then
    g or 0, its derivative 1 or 0."""
    g = torch.tensor([s * m for m in (30.0, 1e4, 1e12, 1e15, 1.8e19, 3e19, 1e30, 2e38) for s in (1, -1)],
                     dtype=torch.float64).to(torch.bfloat16).cuda()
    x, Wg, Wu = operands(g, 1, 64, torch.bfloat16)
    dh = torch.ones((g.numel(), 1), dtype=torch.bfloat16, device="cuda")
    h, gs, us = kda.gated_ffn(x, Wg, Wu, act=act, save=True)
    dx, _, _ = kda.gated_ffn_backward(dh, x, Wg, Wu, gs, us, act=act)
    right = g > 0
    # below 1e-12 on the left: silu's exp(-30) 30 is the largest value there
    for got, want in ((h[:, 0], g), (dx[:, 32], g), (dx[:, 0], torch.ones_like(g))):
        assert torch.equal(got[right], want[right])
        assert (got[~right].abs() < 1e-11).all()
