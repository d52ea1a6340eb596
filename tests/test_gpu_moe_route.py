"""The router on the GPU against its definition: choices, weights, order, gradient."""
import math

import pytest
import torch

import decode_projection_gemms_gb300 as kda
from decode_projection_gemms_gb300 import binding
from ffn_ref import TINY, UNIT
from moe_ref import choose, order, weights

pytestmark = pytest.mark.gpu
TYPES = (torch.bfloat16, torch.float16, torch.float32)


def normal(rows, cols, seed, dtype=torch.float32, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn((rows, cols), generator=g, device="cuda") * std).to(dtype)


def check(logits, k, score, bias=None):
    r = kda.moe_route(logits, k, score=score, bias=bias)
    T, E = logits.shape
    ids, chosen = choose(logits, bias, k, score)
    assert torch.equal(r.ids.long().cpu(), ids)
    w = weights(chosen, score)
    # expf within 2 ulps on a difference that is rounded once, twice for sigmoid; a sum of
    # k and a division; scores below 2^-126 are lost
    spread = (chosen.amax(dim=1, keepdim=True) - chosen).clamp(max=200.0).nan_to_num(200.0) + 200.0 * (score == "sigmoid")
    got = r.weights.double().cpu()
    assert ((got - w).abs() <= (spread + k + 16) * 2.0 ** -23 * w + 2.0 ** -125).all()
    offs, rows, pos = order(ids, E)
    assert r.offsets.tolist() == offs
    assert r.order.tolist() == rows
    assert torch.equal(r.position.long().cpu(), pos)
    assert (got[ids < 0] == 0).all()
    return r


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 64, 6), (2, 3, 3), (5, 33, 32), (31, 8, 2), (32, 64, 4), (33, 64, 4),
                                   (64, 65, 8), (64, 1024, 32), (65, 1024, 32), (100, 256, 8), (129, 1024, 32), (700, 17, 5), (1025, 384, 8)])
def test_route(T, E, k, score, dtype):
    check(normal(T, E, T + E, dtype), k, score)   # 16-bit logits have many ties


@pytest.mark.parametrize("T,E,k", [(1, 16, 4), (40, 96, 8), (500, 256, 8)])
def test_route_with_bias(T, E, k):
    logits = normal(T, E, 5)
    check(logits, k, "sigmoid", 0.2 * normal(1, E, 6)[0])
    bias = torch.zeros(E, device="cuda")
    check(logits, k, "sigmoid", bias)
    bias[::2] = -math.inf                           # half of the experts are switched off
    check(logits, k, "sigmoid", bias)


def test_bias_choices_that_single_precision_cannot_tell():
    """Scores plus biases that differ by less than a rounding of their fp32 sum."""
    E, k = 64, 4
    logits = normal(200, E, 7)
    bias = (2.0 - torch.sigmoid(logits[0].double())).float()     # token 0: all sums near 2
    ids, _ = choose(logits, bias, k, "sigmoid")
    r = kda.moe_route(logits, k, score="sigmoid", bias=bias)
    assert torch.equal(r.ids.long().cpu(), ids)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T", [7, 300])
def test_masked_experts_and_padded_tokens(T, score):
    logits = normal(T, 40, 8)
    logits[:, 5:9] = -math.inf
    logits[1, 3:] = -math.inf                       # three experts left for four slots
    logits[2] = -math.inf                           # none
    logits[3] = math.nan
    logits[4, 7] = math.inf
    logits[5] = -3.0e38                             # the lowest numbers are choices like others
    logits[6] = 0.0
    logits[6, 20] = -0.0                            # equal to 0
    logits[T - T // 4:] = -math.inf
    check(logits, 4, score)


def test_scores_that_vanish():
    logits = torch.full((3, 8), -1.0e4, device="cuda")
    logits[1] = torch.arange(8, device="cuda") * -100.0 - 500.0
    logits[2] = 1.0e4
    for score in ("softmax", "sigmoid"):
        r = check(logits, 3, score)
        assert torch.isfinite(r.weights).all()


def test_uneven_choices_and_strides():
    T, E, k = 2000, 32, 4
    logits = normal(T, E + 9, 9)
    logits[:, 11] += 50.0                           # everybody's first choice
    logits[:, 4] -= 50.0                            # nobody's
    v = logits[:, 3:E + 3]
    a, b = check(v, k, "softmax"), check(v.contiguous(), k, "softmax")
    assert torch.equal(a._buf, b._buf)
    assert a.offsets[9] - a.offsets[8] == T and a.offsets[2] == a.offsets[1]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 64, 6), (9, 33, 7), (50, 256, 8), (1000, 100, 32)])
def test_route_backward(T, E, k, score, dtype):
    logits = normal(T, E, T + E, dtype)
    logits[T // 2, : E - 1] = -math.inf
    dw = normal(T, k, 3)
    r = kda.moe_route(logits, k, score=score)
    got = kda.moe_route_backward(dw, logits, r)
    assert got.dtype is dtype
    ids, chosen = choose(logits, None, k, score)
    chosen.requires_grad_()
    d = dw.double().cpu()
    live = chosen > -math.inf
    lg = torch.nn.functional.logsigmoid(chosen) if score == "sigmoid" else chosen
    w = torch.softmax(torch.where(live, lg, torch.full_like(lg, -1e300)), dim=1)
    (torch.where(live, w, 0.0) * d).sum().backward()
    ref = torch.zeros((T, E), dtype=torch.float64).scatter_add_(1, ids.clamp(min=0), torch.where(live, chosen.grad, 0.0))
    # w and the sum of w dw are off by about 2^-17 of their parts at most
    wv = torch.where(live, w, 0.0).detach()
    part = wv * (d.abs() + (wv * d.abs()).sum(dim=1, keepdim=True))
    tol = torch.zeros((T, E), dtype=torch.float64).scatter_add_(1, ids.clamp(min=0), part) * 2.0 ** -17
    tol = tol + UNIT.get(dtype, 2.0 ** -24) * (ref.abs() + tol) + TINY.get(dtype, 2.0 ** -149)
    assert ((got.double().cpu() - ref).abs() <= tol).all()


def test_route_backward_against_differences():
    T, E, k = 6, 20, 5
    logits, dw = normal(T, E, 1), normal(T, k, 2)
    for score in ("softmax", "sigmoid"):
        r = kda.moe_route(logits, k, score=score)
        got = kda.moe_route_backward(dw, logits, r).double()
        step = 2.0 ** -8
        for t, e in [(0, int(r.ids[0, 0])), (3, int(r.ids[3, 4])), (5, int(r.ids[5, 2]))]:
            f = []
            for s in (step, -step):
                moved = logits.clone()
                moved[t, e] += s
                q = kda.moe_route(moved, k, score=score)
                # the same experts, in whatever order
                back = {int(i): float(v) for i, v in zip(q.ids[t], q.weights[t])}
                assert set(back) == set(r.ids[t].tolist())
                f.append(sum(back[int(i)] * float(d) for i, d in zip(r.ids[t], dw[t])))
            # third derivative below 6 |dw|: step^2; fp32 values: 2^-20 / step
            assert abs((f[0] - f[1]) / (2 * step) - float(got[t, e])) < 6 * 4 * step ** 2 + 2.0 ** -18 / step


def test_other_stream_graph_and_repeats():
    T, E, k = 600, 48, 4
    logits = normal(T, E, 1)
    want = kda.moe_route(logits, k)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = kda.moe_route(logits, k, stream=s)
    s.synchronize()
    assert torch.equal(want._buf, got._buf)
    static, dw = logits.clone(), normal(T, k, 4)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        r = kda.moe_route(static, k)
        d = kda.moe_route_backward(dw, static, r)
    for seed in (5, 6):
        new = normal(T, E, seed)
        static.copy_(new)
        g.replay()
        torch.cuda.synchronize()
        w = kda.moe_route(new, k)
        assert torch.equal(w._buf, r._buf) and torch.equal(kda.moe_route_backward(dw, new, w), d)
    assert binding.device_error() == 0


def test_no_tokens():
    r = kda.moe_route(torch.empty((0, 7), device="cuda"), 2)
    assert r.offsets.tolist() == [0] * 8 and r.ids.shape == (0, 2) and r.order.shape == (0,)
    assert kda.moe_route_backward(torch.empty((0, 2), device="cuda"), torch.empty((0, 7), device="cuda"), r).shape == (0, 7)
