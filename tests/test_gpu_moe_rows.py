"""Rows on their way to the experts and back, with their gradients, on the GPU."""
import math

import pytest
import torch

import decode_projection_gemms_gb300 as kda
from ffn_ref import close

pytestmark = pytest.mark.gpu
HALF = (torch.bfloat16, torch.float16)
SIZES = [(1, 1, 1, 1), (1, 8, 8, 64), (3, 4, 2, 9), (24, 64, 8, 7168), (130, 16, 4, 1000), (257, 40, 3, 203),
         (1000, 8, 2, 520), (70, 64, 32, 96)]


def normal(rows, cols, seed, dtype=torch.float32, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn((rows, cols), generator=g, device="cuda") * std).to(dtype)


def route(T, E, k, seed=1, padded=0):
    logits = normal(T, E, seed)
    if T > 2:
        logits[T // 2, min(1, E - 1):] = -math.inf          # fewer experts than slots
    if padded:
        logits[T - padded:] = -math.inf
    return kda.moe_route(logits, k)


def strided(t, extra, offset=0):
    rows, cols = t.shape
    wide = torch.full((rows, cols + extra + offset), math.nan, dtype=t.dtype, device=t.device)
    v = wide[:, offset:offset + cols]
    v.copy_(t)
    return v


def slots(r):
    """(position, mask) as int64."""
    p = r.position.long()
    return p.clamp(min=0), (p >= 0).unsqueeze(2)


@pytest.mark.parametrize("dtype", HALF)
@pytest.mark.parametrize("T,E,k,K", SIZES)
@pytest.mark.parametrize("layout", [None, (8, 8), (3, 1), (8, 4)])
def test_dispatch_and_back(T, E, k, K, layout, dtype):
    r = route(T, E, k, padded=T // 5)
    n = int(r.offsets[-1])
    x = normal(T, K, 2, dtype)
    if layout:
        x = strided(x, *layout)
    rows = torch.full((T * k, K), 9.0, dtype=dtype, device="cuda")
    if layout:
        rows = strided(rows, *layout)
    assert kda.moe_dispatch(x, r, rows=rows) is rows
    assert torch.equal(rows[:n], x[(r.order[:n] // k).long()])
    assert (rows[n:] == 9.0).all()                         # nobody's rows stay
    d = normal(T * k, K, 3, dtype)
    d[n:] = math.nan                                       # and are not read
    if layout:
        d = strided(d, *layout)
    at, ok = slots(r)
    v = torch.where(ok, d.double()[at], 0.0)
    close(kda.moe_dispatch_backward(d, r), v.sum(dim=1), k * 2.0 ** -24 * v.abs().sum(dim=1), "dx")


@pytest.mark.parametrize("dtype", HALF)
@pytest.mark.parametrize("T,E,k,K", SIZES)
@pytest.mark.parametrize("layout", [None, (8, 8), (3, 1), (8, 4)])
def test_combine_and_back(T, E, k, K, layout, dtype):
    r = route(T, E, k, padded=T // 5)
    n = int(r.offsets[-1])
    rows, dy = normal(T * k, K, 2, dtype), normal(T, K, 3, dtype, 0.05)
    rows[n:] = math.nan
    if layout:
        rows, dy = strided(rows, *layout), strided(dy, *layout)
    at, ok = slots(r)
    v = torch.where(ok, rows.double()[at], 0.0)
    w = r.weights.double().unsqueeze(2)
    y = kda.moe_combine(rows, r)
    close(y, (w * v).sum(dim=1), (k + 1) * 2.0 ** -24 * (w * v).abs().sum(dim=1), "y")
    empty = (r.ids < 0).all(dim=1)
    assert (y[empty] == 0).all()
    out = torch.full((T * k, K), 7.0, dtype=dtype, device="cuda")
    if layout:
        out = strided(out, *layout)
    drows, dw = kda.moe_combine_backward(dy, rows, r, drows=out)
    d = dy.double().unsqueeze(1)
    ref = (w * d).reshape(T * k, K)[r.order[:n].long()]
    close(drows[:n], ref, 2.0 ** -24 * ref.abs(), "drows")
    assert (drows[n:] == 7.0).all()
    # a lane adds K / 32 products at most, the warp's sums in five steps
    tol = (K / 32 + 16) * 2.0 ** -24 * (d * v).abs().sum(dim=2) + 2.0 ** -149
    assert ((dw.double() - (d * v).sum(dim=2)).abs() <= tol).all()
    assert (dw[r.ids < 0] == 0).all()
    again = kda.moe_combine_backward(dy, rows, r)
    assert torch.equal(again[0][:n], drows[:n]) and torch.equal(again[1], dw) and torch.equal(kda.moe_combine(rows, r), y)


@pytest.mark.parametrize("layout", [None, (3, 1)])
def test_nothing_is_written_outside(layout):
    T, E, k, K = 37, 12, 3, 203
    r = route(T, E, k)
    n = int(r.offsets[-1])
    x = normal(T, K, 2, torch.bfloat16)
    for call, rows in ((lambda y: kda.moe_dispatch(x, r, rows=y), T * k),
                       (lambda y: kda.moe_combine(normal(T * k, K, 4, torch.bfloat16), r, y=y), T),
                       (lambda y: kda.moe_combine_backward(x, normal(T * k, K, 4, torch.bfloat16), r, drows=y), T * k)):
        buf = torch.full((rows + 4, K + 24), 5.0, dtype=torch.bfloat16, device="cuda")
        call(buf[2:-2, 8:8 + K] if layout is None else buf[2:-2, 9:9 + K])
        buf[2:-2, 8 if layout is None else 9:][:, :K] = 5.0
        assert (buf == 5.0).all()
    assert n <= T * k


def test_positions_that_lead_nowhere_are_left_out():
    T, E, k, K = 20, 8, 2, 64
    r = route(T, E, k)
    r.position[3, 1] = T * k                     # past the rows
    r.position[4, 0] = -7
    x = normal(T, K, 1, torch.float16)
    rows = torch.zeros((T * k, K), dtype=torch.float16, device="cuda")
    kda.moe_dispatch(x, r, rows=rows)
    at = r.position.long()
    ok = (at >= 0) & (at < T * k)
    v = torch.where(ok.unsqueeze(2), rows.double()[at.clamp(0, T * k - 1)], 0.0)
    assert torch.equal(v[ok], x.double().unsqueeze(1).expand(T, k, K)[ok])
    close(kda.moe_dispatch_backward(rows, r), v.sum(dim=1), 2.0 ** -23 * v.abs().sum(dim=1))
    torch.cuda.synchronize()


def test_other_stream_and_graph():
    T, E, k, K = 300, 16, 4, 520

    def step(logits, x, dy, stream=None):
        r = kda.moe_route(logits, k, stream=stream)
        rows = kda.moe_dispatch(x, r, stream=stream)
        y = kda.moe_combine(rows, r, stream=stream)
        drows, dw = kda.moe_combine_backward(dy, rows, r, stream=stream)
        dl = kda.moe_route_backward(dw, logits, r, stream=stream)
        return [rows, y, drows, dw, dl, kda.moe_dispatch_backward(drows, r, stream=stream)]

    def inputs(seed):
        return normal(T, E, seed), normal(T, K, seed + 1, torch.bfloat16), normal(T, K, seed + 2, torch.bfloat16)

    want = step(*inputs(1))
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = step(*inputs(1), stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    static = inputs(1)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = step(*static)
    for seed in (11, 21):
        for a, b in zip(static, inputs(seed)):
            a.copy_(b)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(step(*inputs(seed)), outs))


def test_no_tokens():
    r = kda.moe_route(torch.empty((0, 7), device="cuda"), 2)
    e = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    assert kda.moe_dispatch(e, r).shape == (0, 64) and kda.moe_combine(e, r).shape == (0, 64)
    drows, dw = kda.moe_combine_backward(e, e, r)
    assert drows.shape == (0, 64) and dw.shape == (0, 2)
