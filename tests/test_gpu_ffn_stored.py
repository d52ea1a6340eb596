"""4-bit matrices put together from stored codes and scales: the products read the
padding between a matrix's last block and the end of its last step of 64 columns."""
import pytest
import torch

import decode_projection_gemms_gb300 as kda
from ffn_ref import close, mx4_values, product_bounds

pytestmark = pytest.mark.gpu


def normal(rows, cols, seed, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn((rows, cols), generator=g, device="cuda") * std


def scale_places(rows, cols):
    """(row, block) of every scale byte, by the layout that the header describes."""
    nb = -(-cols // 32)
    kt = -(-nb // 4)
    at = torch.arange(-(-rows // 128) * kt * 512)
    tile, byte = at // 512, at % 512
    row = tile // kt * 128 + byte // 16 + byte % 16 // 4 * 32
    return row.cuda(), (tile % kt * 4 + byte % 4).cuda()


def stored(x):
    """x quantised, then put together again from parts built by hand: blocks past the
    columns 0, rows past the end (which are not used) NaN."""
    q = kda.mx4_quantize(x)
    rows, cols = x.shape
    row, block = scale_places(rows, cols)
    scales = torch.full_like(q.scales, 255)
    scales[block * 32 >= cols] = 0
    real = (row < rows) & (block * 32 < cols)
    scales[real] = q.scales[real]
    codes = torch.zeros_like(q.codes)
    codes.copy_(q.codes)
    return kda.Mx4Tensor(codes, scales, rows, cols), q


@pytest.mark.parametrize("M", [1, 5, 40, 300])
@pytest.mark.parametrize("K", [1, 31, 32, 65, 96, 160, 257, 288, 1057, 2080])
def test_stored_parts_with_padding(M, K):
    N = 200
    x, W = normal(M, K, 1).to(torch.bfloat16), normal(N, K, 2, 0.05)
    (xs, xq), (Ws, Wq) = stored(x), stored(W)
    assert torch.equal(kda.mx4_dequantize(Ws), kda.mx4_dequantize(Wq))
    ref, bound = product_bounds(mx4_values(x), mx4_values(W))
    want = kda.mx4_gemm(xq, Wq)
    close(want, ref, bound)
    assert torch.equal(kda.mx4_gemm(xs, Ws), want)
    assert torch.equal(kda.mx4_gemm(x, Ws), want)
    assert torch.equal(kda.mx4_gated_ffn(xs, Ws, Ws), kda.mx4_gated_ffn(xq, Wq, Wq))
