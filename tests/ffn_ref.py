"""Plain 64-bit forms of the feed-forward operators and the error bounds their
tests use (torch double arithmetic; nothing of the package)."""
from __future__ import annotations

import math

import torch

UNIT = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}      # rounding to nearest: half an ulp
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25}    # half the smallest subnormal
MAGS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def mx4_values(x: torch.Tensor) -> torch.Tensor:
    """What quantising x to microscaled 4 bits and back gives, element by element
    from the definition."""
    rows, cols = x.shape
    nb = -(-cols // 32)
    v = torch.zeros((rows, nb * 32), dtype=torch.float64, device=x.device)
    v[:, :cols] = x.double()
    v = v.view(rows, nb, 32)
    bad = ~torch.isfinite(v).all(dim=2, keepdim=True)
    v = torch.where(bad, torch.zeros_like(v), v)
    top = v.abs().amax(dim=2, keepdim=True)
    n = ((top.view(torch.int64) >> 52) - 1023 - 2).clamp(min=-127)     # floor(log2 top) - 2
    scale = ((n + 1023) << 52).view(torch.float64)
    a = v.abs() / scale
    q = torch.zeros_like(a)
    for i in range(1, 8):
        mid = (MAGS[i - 1] + MAGS[i]) / 2
        up = (a >= mid) if i % 2 == 0 else (a > mid)
        q = torch.where(up, torch.full_like(a, MAGS[i]), q)
    out = torch.where(bad, torch.full_like(a, math.nan), torch.sign(v) * q * scale)
    return out.view(rows, nb * 32)[:, :cols]


def act(g: torch.Tensor, name: str):
    """(act(g), act'(g))."""
    if name == "silu":
        s = torch.sigmoid(g)
        return g * s, s * (1 + g * (1 - s))
    if name == "gelu":
        cdf = 0.5 * (1 + torch.erf(g / math.sqrt(2)))
        return g * cdf, cdf + g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)
    c = math.sqrt(2 / math.pi)
    t = torch.tanh(c * (g + 0.044715 * g ** 3))
    return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * c * (1 + 3 * 0.044715 * g * g)


def acc_bound(a: torch.Tensor, b: torch.Tensor, k: int) -> torch.Tensor:
    """Bound on the fp32 error of sum_k a b: the tensor core adds at least 16
    products a step and the split-K join at most 8 partial sums, each step off by
    at most one unit 2^-23 of the sum of magnitudes."""
    return (k / 16 + 32) * 2.0 ** -23 * (a.abs() @ b.abs())


def close(got: torch.Tensor, ref: torch.Tensor, bound: torch.Tensor, what: str = ""):
    """got (16-bit) against ref within its rounding plus `bound`."""
    u = UNIT[got.dtype]
    g = got.double()
    assert torch.isfinite(g).all(), f"{what}: not finite"
    tol = u * (ref.abs() + bound) + bound + TINY[got.dtype]
    worst = ((g - ref).abs() / tol).max().item() if g.numel() else 0.0
    assert worst <= 1.0, f"{what}: {worst:.3f} of the tolerance"


def product_bounds(x, W):
    """(x W^T, its fp32 error bound) in 64 bits."""
    return x @ W.t(), acc_bound(x, W.t(), x.shape[1])


# Largest |act'| and |act''| of the three activations are below these; an
# activation in fp32 is off by at most 2^-20 of |g| (a handful of fp32 roundings
# and the hardware exponential's 2 ulps plus its argument's rounding, |z| <= 100).
D1, D2, ACT_EPS = 1.2, 1.2, 2.0 ** -20


def gated(x, Wg, Wu, name):
    """(h, bound on its fp32 error, g, dg, u, du)."""
    g, eg = product_bounds(x, Wg)
    u, eu = product_bounds(x, Wu)
    a, _ = act(g, name)
    ea = D1 * eg + ACT_EPS * g.abs()
    return a * u, ea * (u.abs() + eu) + a.abs() * eu + 2.0 ** -24 * (a * u).abs(), g, eg, u, eu


def gated_grads(dh, x, Wg, Wu, name, unit):
    """{name: (gradient, bound on its error before its own rounding)} of the gated
    block. g and u reach the backward pass in fp32; dG and dU are rounded to 16 bits
    (`unit`) as operands, and that error is carried through."""
    g, eg = product_bounds(x, Wg)
    u, eu = product_bounds(x, Wu)
    a, da = act(g, name)
    dg, du = dh * u * da, dh * a
    d = dh.abs()
    fp = 2.0 ** -19 * (1 + g.abs())       # act and act' in fp32
    edg = d * (eu * D1 + (u.abs() + eu) * (D2 * eg + fp))
    edg = edg + unit * (dg.abs() + edg)
    edu = d * (D1 * eg + fp)
    edu = edu + unit * (du.abs() + edu)
    tiny = 2.0 ** -25                     # fp16 operands below its subnormals
    edg, edu = edg + tiny, edu + tiny
    F, T = g.shape[1], g.shape[0]
    dx = dg @ Wg + du @ Wu
    edx = edg @ Wg.abs() + edu @ Wu.abs() + acc_bound(dg.abs() + edg, Wg, 2 * F) + acc_bound(du.abs() + edu, Wu, 2 * F)
    out = {"dx": (dx, edx)}
    for key, v, e in (("dWg", dg, edg), ("dWu", du, edu)):
        out[key] = (v.t() @ x, e.t() @ x.abs() + acc_bound((v.abs() + e).t(), x, T))
    return out
