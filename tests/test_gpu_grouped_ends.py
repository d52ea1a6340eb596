"""The rows that an expert ends in, handed from the warps of two CTAs that clear the others'
rows among them to the MMAs of one: every remainder, time and again, with the GPU busy."""
import math

import pytest
import torch

import decode_projection_gemms_gb300 as kda
from decode_projection_gemms_gb300 import binding

pytestmark = pytest.mark.gpu


def normal(*shape, seed, dtype, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(0.0, std, generator=g)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("N,K", [(8, 8), (264, 520), (512, 136)])
def test_every_remainder_again_and_again(N, K, dtype):
    """Every second expert's rows are NaN and lie next to one that is not. What the others
    get is what they get alone, bit for bit, in every run."""
    counts = [c for r in range(1, 64) for c in (r + 64 * (r % 3), 1 + r % 16)]
    E, R = len(counts), sum(counts)
    off = torch.tensor([0] + counts).cumsum(0).to(torch.int32).cuda()
    x, dy = normal(R, K, seed=1, dtype=dtype), normal(R, N, seed=2, dtype=dtype)
    W = normal(E, N, K, seed=3, dtype=dtype, std=0.1)
    expert = torch.repeat_interleave(torch.arange(E), torch.tensor(counts)).cuda()
    bad = expert % 2 == 1
    for t in (x, dy):
        t[bad] = 0.0
    dx0, dW0 = kda.grouped_gemm_backward(dy, x, W, off)      # zeros where the NaN will be
    for t in (x, dy):
        t[bad] = math.nan
    side = torch.cuda.Stream()
    load = torch.empty(2 ** 26, dtype=torch.uint8, device="cuda")
    for _ in range(20):
        with torch.cuda.stream(side):
            load.add_(1)
        dx, dW = kda.grouped_gemm_backward(dy, x, W, off)
        assert torch.equal(dW[::2], dW0[::2]) and torch.equal(dx[~bad], dx0[~bad])
        assert torch.isnan(dW[1::2]).all() and torch.isnan(dx[bad]).all()
    torch.cuda.synchronize()
    assert binding.device_error() == 0


def test_a_contraction_of_more_than_a_second():
    """2^29 rows of one expert, which a single cluster contracts to its dW in 2.2 s: longer than
    the kernels' other waits last."""
    R, N, K, dt = 2 ** 29, 8, 8, torch.bfloat16
    off = torch.tensor([0, R], dtype=torch.int32, device="cuda")
    x, dy = torch.zeros((R, K), dtype=dt, device="cuda"), torch.zeros((R, N), dtype=dt, device="cuda")
    W = normal(1, N, K, seed=1, dtype=dt)
    at = torch.tensor([0, 1, 77, 2 ** 28 - 1, 2 ** 28, R - 64, R - 1], device="cuda")
    g = torch.Generator(device="cuda").manual_seed(2)
    for t in (x, dy):
        t[at] = torch.randint(-3, 4, (len(at), 8), generator=g, device="cuda").to(dt)
    dx, dW = kda.grouped_gemm_backward(dy, x, W, off)
    torch.cuda.synchronize()
    assert binding.device_error() == 0
    assert torch.equal(dW[0].double(), dy[at].double().t() @ x[at].double())      # whole numbers below 256
    want = dy[at].double() @ W[0].double()
    # eight products summed in fp32, rounded to bf16
    tol = 2.0 ** -21 * (dy[at].double().abs() @ W[0].double().abs())
    assert ((dx[at].double() - want).abs() <= tol + 2.0 ** -8 * (want.abs() + tol)).all()
    assert int(torch.count_nonzero(dx)) <= 8 * len(at)
