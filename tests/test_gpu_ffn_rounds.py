"""Forward products of several rounds of tiles: accumulators and stages that come
round again, outputs that leave behind an earlier tile's."""
import math

import pytest
import torch

import decode_projection_gemms_gb300 as kda
from decode_projection_gemms_gb300 import binding
from ffn_cases import MANY_ROUNDS
from ffn_ref import close, gated, mx4_values, product_bounds

pytestmark = pytest.mark.gpu
HALF = (torch.bfloat16, torch.float16)


def normal(rows, cols, seed, dtype=torch.float32, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn((rows, cols), generator=g, device="cuda") * std).to(dtype)


def inside(T, F, dtype, offset):
    """A T x F view into a wider matrix, and a check that nothing around it changed."""
    wide = torch.full((T + 8, F + 21), 9.0, dtype=dtype, device="cuda")
    y = wide[4:4 + T, offset:offset + F]
    y.fill_(math.nan)

    def untouched():
        keep = torch.ones_like(wide, dtype=torch.bool)
        keep[4:4 + T, offset:offset + F] = False
        assert (wide[keep] == 9.0).all()
    return y, untouched


@pytest.mark.parametrize("dtype", HALF)
@pytest.mark.parametrize("mx4,is_gated,T,F,K", MANY_ROUNDS)
def test_many_rounds(mx4, is_gated, T, F, K, dtype):
    act = ("silu", "gelu", "gelu_tanh")[(T + K) % 3]
    x = normal(T, K, 1, dtype)
    Wg, Wu = normal(F, K, 2, dtype, K ** -0.5 * 1.5), normal(F, K, 3, dtype, K ** -0.5)
    v = mx4_values if mx4 else torch.Tensor.double
    if is_gated:
        ref, bound, rg, eg, ru, eu = gated(v(x), v(Wg), v(Wu), act)
    else:
        ref, bound = product_bounds(v(x), v(Wg))
    if mx4:
        qg, qu = kda.mx4_quantize(Wg), kda.mx4_quantize(Wu)
        run = (lambda y: kda.mx4_gated_ffn(x, qg, qu, act=act, h=y)) if is_gated else \
            (lambda y: kda.mx4_gemm(x, qg, y=y))
    else:
        run = lambda y: kda.gated_ffn(x, Wg, Wu, act=act, h=y)  # noqa: E731
        h, g, u = kda.gated_ffn(x, Wg, Wu, act=act, save=True)
        assert ((g.double() - rg).abs() <= eg).all() and ((u.double() - ru).abs() <= eu).all()
        assert torch.equal(h, run(None))
    want = run(None)
    close(want, ref, bound, f"{T}x{F}x{K}")
    for offset in (8, 3):
        y, untouched = inside(T, F, dtype, offset)
        run(y)
        assert torch.equal(y, want)
        untouched()
    torch.cuda.synchronize()
    assert binding.device_error() == 0
