"""Matrices that the element-wise kernels go over in more than one round."""
import math

import pytest
import torch

import decode_projection_gemms_gb300 as kda
from decode_projection_gemms_gb300 import binding
from ffn_ref import UNIT, close, gated_grads, mx4_values

pytestmark = pytest.mark.gpu
ALL = (torch.bfloat16, torch.float16, torch.float32)
ROWS = 8191


def normal(rows, cols, seed, dtype=torch.float32, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn((rows, cols), generator=g, device="cuda") * std).to(dtype)


def view(t, extra, offset):
    """The same matrix inside a wider one of NaN."""
    rows, cols = t.shape
    wide = torch.full((rows, cols + extra), math.nan, dtype=t.dtype, device=t.device)
    v = wide[:, offset:offset + cols]
    v.copy_(t)
    return v


# row lengths that are a multiple of four, of two and of one element, each over the
# end of a segment of 1024 columns and of a block of 32
@pytest.mark.parametrize("dtype,cols", [(torch.float32, 7156), (torch.float32, 7155), (torch.float32, 2050),
                                        (torch.bfloat16, 2056), (torch.bfloat16, 2050), (torch.bfloat16, 2049),
                                        (torch.float16, 2050), (torch.float16, 2049)])
@pytest.mark.parametrize("extra,offset", [(0, 0), (9, 4), (12, 1)])
def test_quantise_and_back(dtype, cols, extra, offset):
    x = normal(ROWS, cols, cols + offset, dtype, 0.05)
    q = kda.mx4_quantize(view(x, extra, offset) if extra else x)
    outs = {dt: kda.mx4_dequantize(q, dtype=dt) for dt in ALL}
    wide = {dt: torch.full((ROWS, cols + extra), 7.0, dtype=dt, device="cuda") for dt in ALL} if extra else {}
    for dt, w in wide.items():
        kda.mx4_dequantize(q, dtype=dt, y=w[:, offset:offset + cols])
        assert torch.equal(w[:, offset:offset + cols], outs[dt])
        assert (w[:, :offset] == 7.0).all() and (w[:, offset + cols:] == 7.0).all()
    for r in range(0, ROWS, 2048):
        want = mx4_values(x[r:r + 2048])
        for dt, y in outs.items():
            assert torch.equal(y[r:r + 2048].double(), want.to(dt).double()), f"rows from {r}, {dt}"
    torch.cuda.synchronize()
    assert binding.device_error() == 0


@pytest.mark.parametrize("dtype", ALL[:2])
@pytest.mark.parametrize("T,F,K,act", [(1800, 1424, 328, "gelu"), (1900, 1403, 328, "gelu_tanh"), (2600, 1001, 264, "silu")])
def test_backward(T, F, K, act, dtype):
    x, dh = normal(T, K, 1, dtype), normal(T, F, 2, dtype, 0.05)
    Wg, Wu = normal(F, K, 3, dtype, K ** -0.5 * 1.5), normal(F, K, 4, dtype, K ** -0.5)
    _, g, u = kda.gated_ffn(x, Wg, Wu, act=act, save=True)
    ref = gated_grads(dh.double(), x.double(), Wg.double(), Wu.double(), act, UNIT[dtype])
    for got, name in zip(kda.gated_ffn_backward(dh, x, Wg, Wu, g, u, act=act), ("dx", "dWg", "dWu")):
        close(got, *ref[name], f"{name} {T}x{F}x{K}")
    torch.cuda.synchronize()
    assert binding.device_error() == 0
