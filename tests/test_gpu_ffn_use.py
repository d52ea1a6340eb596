"""The feed-forward operators as programs use them: on a stream of their own, in
captured graphs, with sums written between other data, with infinities and NaN."""
import math

import pytest
import torch

import decode_projection_gemms_gb300 as kda
from decode_projection_gemms_gb300 import binding

pytestmark = pytest.mark.gpu
HALF = (torch.bfloat16, torch.float16)


def normal(rows, cols, seed, dtype=torch.float32, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn((rows, cols), generator=g, device="cuda") * std).to(dtype)


def parts(q):
    return [q.codes, q.scales]


def step(x, dh, Wg, Wu, stream=None):
    """Quantisation, values back and a training step."""
    q = kda.mx4_quantize(x, stream=stream)
    v = kda.mx4_dequantize(q, dtype=x.dtype, stream=stream)
    h, g, u = kda.gated_ffn(x, Wg, Wu, save=True, stream=stream)
    return [*parts(q), v, h, g, u, *kda.gated_ffn_backward(dh, x, Wg, Wu, g, u, stream=stream)]


@pytest.mark.parametrize("dtype", HALF)
@pytest.mark.parametrize("T,F,K", [(20, 264, 256), (300, 500, 520)])
def test_stream_and_graph(T, F, K, dtype):
    x, dh = normal(T, K, 1, dtype), normal(T, F, 2, dtype, 0.05)
    Wg, Wu = normal(F, K, 3, dtype, 0.1), normal(F, K, 4, dtype, 0.1)
    want = step(x, dh, Wg, Wu)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = step(x, dh, Wg, Wu, stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    xin, dhin = x.clone(), dh.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step(xin, dhin, Wg, Wu)
    for seed in (5, 6):
        x2, dh2 = normal(T, K, seed, dtype), normal(T, F, seed + 10, dtype, 40.0 * seed)
        xin.copy_(x2)
        dhin.copy_(dh2)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(step(x2, dh2, Wg, Wu), outs))
    assert binding.device_error() == 0


@pytest.mark.parametrize("T", [5, 70, 300, 1100])
@pytest.mark.parametrize("F", [203, 204, 512, 720, 1000])
def test_sums_stay_inside_their_matrices(T, F):
    """g and u for the backward pass, written between other data."""
    K, pad = 264, 64
    x, Wg, Wu = (normal(r, K, s, torch.bfloat16) for r, s in ((T, 1), (F, 2), (F, 3)))
    h, g, u = kda.gated_ffn(x, Wg, Wu, save=True)
    buf = [torch.full((T * F + 2 * pad,), 9.0, device="cuda") for _ in range(2)]
    out = torch.full((T, F), math.nan, dtype=torch.bfloat16, device="cuda")
    work, wp, wn = binding._work(binding.FFN_GATED, T, F, K, 0)
    rc = binding.load().kp_gated_ffn(x.data_ptr(), K, Wg.data_ptr(), K, Wu.data_ptr(), K, out.data_ptr(), F,
                                     buf[0].data_ptr() + 4 * pad, buf[1].data_ptr() + 4 * pad, T, F, K, 0, 0, wp, wn,
                                     torch.cuda.current_stream().cuda_stream)
    assert rc == binding.KP_OK, binding.last_error()
    assert torch.equal(out, h)
    for b, want in zip(buf, (g, u)):
        assert torch.equal(b[pad:-pad].view(T, F), want)
        assert (b[:pad] == 9.0).all() and (b[-pad:] == 9.0).all()


@pytest.mark.parametrize("dtype", HALF)
@pytest.mark.parametrize("act", sorted(binding.ACTIVATIONS))
@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("T", [3, 70, 700])
def test_non_finite_operands_reach_their_rows_and_features_only(T, bad, act, dtype):
    F, K = 200, 136
    x, Wg, Wu = normal(T, K, 1, dtype), normal(F, K, 2, dtype, 0.1), normal(F, K, 3, dtype, 0.1)
    want, g0, u0 = kda.gated_ffn(x, Wg, Wu, act=act, save=True)
    x[1, 100], Wg[7, 3], Wu[150, 135] = bad, bad, bad
    h, g, u = kda.gated_ffn(x, Wg, Wu, act=act, save=True)
    rows = torch.arange(T, device="cuda") == 1
    gate, factor = torch.arange(F, device="cuda") == 7, torch.arange(F, device="cuda") == 150
    # a gate of minus infinity is NaN times its factor, or 0 times infinity
    for got, ref, hit in ((g, g0, rows[:, None] | gate), (u, u0, rows[:, None] | factor),
                          (h, want, rows[:, None] | factor)):
        keep = ~hit if got is not h else ~(hit | gate)
        assert not torch.isfinite(got[hit]).any()
        assert torch.equal(got[keep], ref[keep])
