"""Products grouped by expert on the GPU against plain 64-bit forms: ragged sizes,
experts without rows, rows without experts, strides, gradients."""
import math

import pytest
import torch

import decode_projection_gemms_gb300 as kda
from decode_projection_gemms_gb300 import binding
from ffn_ref import UNIT, close
from moe_ref import grouped, grouped_gated, grouped_gated_grads, grouped_grads, spans

pytestmark = pytest.mark.gpu
HALF = (torch.bfloat16, torch.float16)
# rows of each expert, rows behind the last one's
GROUPS = {
    "one": ([1], 0),
    "token": ([0, 1, 0, 0, 1, 1, 0], 0),
    "few": ([3, 0, 16, 1, 0, 5, 2], 3),
    "edges": ([15, 16, 17, 31, 32, 33], 1),
    "tiles": ([63, 64, 65, 0, 127, 128, 129], 5),
    "long": ([255, 256, 257, 0, 1], 0),
    "uneven": ([700, 0, 0, 3, 1, 40], 12),
    "none": ([0, 0, 0], 4),
}


def normal(*shape, seed, dtype=torch.float32, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def groups(name):
    n, behind = GROUPS[name]
    off = torch.tensor([0] + n, dtype=torch.int32).cumsum(0).to(torch.int32).cuda()
    return off, int(off[-1]) + behind, len(n)


def quiet(code=0):
    torch.cuda.synchronize()
    assert binding.device_error() == code


@pytest.mark.parametrize("dtype", HALF)
@pytest.mark.parametrize("N,K", [(1, 8), (40, 64), (128, 72), (130, 256), (257, 320), (513, 1032)])
@pytest.mark.parametrize("name", sorted(GROUPS))
def test_grouped_gemm(name, N, K, dtype):
    off, R, E = groups(name)
    x, W = normal(R, K, seed=1, dtype=dtype), normal(E, N, K, seed=2, dtype=dtype, std=0.1)
    end = int(off[-1])
    x[end:] = math.nan
    y = torch.full((R, N), 3.0, dtype=dtype, device="cuda")
    assert kda.grouped_gemm(x, W, off, y=y) is y
    ref, bound = grouped(x, W, off)
    close(y[:end], ref[:end], bound[:end], name)
    assert (y[end:] == 3.0).all()
    assert torch.equal(kda.grouped_gemm(x, W, off)[:end], y[:end])
    quiet()


# experts are looked up 32 at a time: the edges of that, runs without rows, several tiles an expert
@pytest.mark.parametrize("n", [[1] * 31, [1] * 32, [1] * 33, [0] * 31 + [3], [0] * 32 + [3], [0] * 33 + [3], [3] + [0] * 64,
                               [2] + [0] * 31 + [1], [0] * 64 + [5] + [0] * 31 + [300], [17] * 65,
                               [1] + [0] * 40 + [600] + [0] * 31 + [7], [0, 1] * 100, [0] * 1023 + [2]],
                         ids=lambda n: f"{len(n)}x{sum(n)}")
def test_many_experts(n):
    off = torch.tensor([0] + n, dtype=torch.int32).cumsum(0).to(torch.int32).cuda()
    R, E, N, K = int(off[-1]) + 2, len(n), 264, 72
    x, W = normal(R, K, seed=1, dtype=torch.bfloat16), normal(E, N, K, seed=2, dtype=torch.bfloat16, std=0.1)
    dy = normal(R, N, seed=3, dtype=torch.bfloat16, std=0.05)
    x[-2:], dy[-2:] = math.nan, math.inf
    y = torch.full((R, N), 3.0, dtype=torch.bfloat16, device="cuda")
    kda.grouped_gemm(x, W, off, y=y)
    ref, bound = grouped(x, W, off)
    close(y[:-2], ref[:-2], bound[:-2], "y")
    assert (y[-2:] == 3.0).all()
    dx, dW = kda.grouped_gemm_backward(dy, x, W, off)
    ref = grouped_grads(dy, x, W, off)
    close(dx[:-2], ref["dx"][0][:-2], ref["dx"][1][:-2], "dx")
    close(dW, *ref["dW"], "dW")
    quiet()


@pytest.mark.parametrize("dtype", HALF)
@pytest.mark.parametrize("N,K", [(8, 8), (40, 64), (136, 72), (264, 320), (520, 1032)])
@pytest.mark.parametrize("name", sorted(GROUPS))
def test_grouped_gemm_backward(name, N, K, dtype):
    off, R, E = groups(name)
    x, W = normal(R, K, seed=1, dtype=dtype), normal(E, N, K, seed=2, dtype=dtype, std=0.1)
    dy = normal(R, N, seed=3, dtype=dtype, std=0.05)
    end = int(off[-1])
    x[end:], dy[end:] = math.nan, math.inf
    dx, dW = kda.grouped_gemm_backward(dy, x, W, off)
    ref = grouped_grads(dy, x, W, off)
    close(dx[:end], ref["dx"][0][:end], ref["dx"][1][:end], "dx")
    close(dW, *ref["dW"], "dW")
    for (e, r) in spans(off):
        if r.start == r.stop:
            assert (dW[e] == 0).all()
    again = kda.grouped_gemm_backward(dy, x, W, off)
    assert torch.equal(again[0][:end], dx[:end]) and torch.equal(again[1], dW)
    quiet()


@pytest.mark.parametrize("dtype", HALF)
@pytest.mark.parametrize("F,K,act", [(1, 8, "silu"), (40, 64, "gelu"), (64, 72, "silu"), (130, 256, "gelu_tanh"),
                                     (257, 320, "silu"), (400, 1032, "gelu")])
@pytest.mark.parametrize("name", sorted(GROUPS))
def test_grouped_gated(name, F, K, act, dtype):
    off, R, E = groups(name)
    x = normal(R, K, seed=1, dtype=dtype)
    Wg, Wu = (normal(E, F, K, seed=s, dtype=dtype, std=0.1) for s in (2, 3))
    dh = normal(R, F, seed=4, dtype=dtype, std=0.05)
    end = int(off[-1])
    x[end:], dh[end:] = math.nan, math.nan
    h, g, u = kda.grouped_gated_ffn(x, Wg, Wu, off, act=act, save=True)
    rh, eh, rg, eg, ru, eu = grouped_gated(x[:end], Wg, Wu, off, act)
    close(h[:end], rh, eh, "h")
    assert ((g[:end].double() - rg).abs() <= eg).all() and ((u[:end].double() - ru).abs() <= eu).all()
    assert torch.equal(kda.grouped_gated_ffn(x, Wg, Wu, off, act=act)[:end], h[:end])
    g[end:], u[end:] = math.nan, math.nan
    got = kda.grouped_gated_ffn_backward(dh, x, Wg, Wu, off, g, u, act=act)
    ref = grouped_gated_grads(dh[:end], x[:end], Wg, Wu, off, act, UNIT[dtype])
    for key, v in zip(("dx", "dWg", "dWu"), got):
        r, b = ref[key]
        close(v[:end] if key == "dx" else v, r, b, key)
    again = kda.grouped_gated_ffn_backward(dh, x, Wg, Wu, off, g, u, act=act)
    assert torch.equal(again[0][:end], got[0][:end]) and torch.equal(again[1], got[1]) and torch.equal(again[2], got[2])
    quiet()


def views(t, extra):
    """The same rows inside wider ones, NaN around them."""
    wide = torch.full((*t.shape[:-1], t.shape[-1] + extra), math.nan, dtype=t.dtype, device=t.device)
    wide[..., extra // 2:extra // 2 + t.shape[-1]] = t
    return wide[..., extra // 2:extra // 2 + t.shape[-1]]


def test_strided_views_and_packed_weights():
    off, R, E = groups("tiles")
    F, K, dt = 136, 264, torch.bfloat16
    x, packed = views(normal(R, K, seed=1, dtype=dt), 16), normal(E, 2 * F, K, seed=2, dtype=dt, std=0.1)
    Wg, Wu = packed[:, :F], packed[:, F:]                   # halves of one matrix per expert
    dh = views(normal(R, F, seed=3, dtype=dt), 3)
    end = int(off[-1])
    a = kda.grouped_gated_ffn(x, Wg, Wu, off, save=True)
    b = kda.grouped_gated_ffn(x.contiguous(), Wg.contiguous(), Wu.contiguous(), off, save=True)
    assert all(torch.equal(p[:end], q[:end]) for p, q in zip(a, b))
    a = kda.grouped_gated_ffn_backward(dh, x, Wg, Wu, off, *a[1:])
    b = kda.grouped_gated_ffn_backward(dh.contiguous(), x.contiguous(), Wg.contiguous(), Wu.contiguous(), off, *b[1:])
    assert torch.equal(a[0][:end], b[0][:end]) and torch.equal(a[1], b[1]) and torch.equal(a[2], b[2])
    W, dy = views(normal(E, F, K, seed=4, dtype=dt, std=0.1), 32), views(normal(R, F, seed=5, dtype=dt), 16)
    assert torch.equal(kda.grouped_gemm(x, W, off)[:end], kda.grouped_gemm(x.contiguous(), W.contiguous(), off)[:end])
    a = kda.grouped_gemm_backward(dy, x, W, off)
    b = kda.grouped_gemm_backward(dy.contiguous(), x.contiguous(), W.contiguous(), off)
    assert torch.equal(a[0][:end], b[0][:end]) and torch.equal(a[1], b[1])
    # every other expert of a larger stack
    stack = normal(2 * E, F, K, seed=6, dtype=dt, std=0.1)
    assert torch.equal(kda.grouped_gemm(x, stack[::2], off)[:end], kda.grouped_gemm(x, stack[::2].contiguous(), off)[:end])
    quiet()


@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("name", ["few", "edges", "tiles", "uneven"])
def test_experts_do_not_see_each_other(name, bad):
    """NaN and infinity in one expert's rows and weights, and behind all rows, reach that
    expert's outputs and gradients alone."""
    off, R, E = groups(name)
    F, K, dt = 136, 200, torch.bfloat16
    end = int(off[-1])
    x, dy = normal(R, K, seed=1, dtype=dt), normal(R, F, seed=2, dtype=dt)
    W, V = normal(E, F, K, seed=3, dtype=dt, std=0.1), normal(E, F, K, seed=4, dtype=dt, std=0.1)

    def outputs():
        h, g, u = kda.grouped_gated_ffn(x, W, V, off, save=True)
        return [h, g, u, kda.grouped_gemm(x, W, off), *kda.grouped_gemm_backward(dy, x, W, off),
                *kda.grouped_gated_ffn_backward(dy, x, W, V, off, g, u)]

    want = outputs()
    hit = 2
    rows = dict(spans(off))[hit]
    x[rows], dy[rows], W[hit], V[hit] = bad, bad, bad, bad
    x[end:], dy[end:] = bad, bad
    keep = torch.ones(R, dtype=torch.bool, device="cuda")
    keep[rows], keep[end:] = False, False
    other = [e for e in range(E) if e != hit]
    for a, b in zip(outputs(), want):
        assert torch.equal(a[other], b[other]) if a.dim() == 3 else torch.equal(a[keep], b[keep])
    quiet()


def test_any_offsets_stay_inside():
    """Offsets that no router would make: the rows they name are within the matrix."""
    R, E, N, K = 40, 5, 64, 64
    x, W = normal(R, K, seed=1, dtype=torch.bfloat16), normal(E, N, K, seed=2, dtype=torch.bfloat16)
    buf = torch.full((R + 8, N), 5.0, dtype=torch.bfloat16, device="cuda")
    for o in ([-7, 3, 3, 90, 100, 2 ** 31 - 1], [9, 5, 0, -2 ** 31, 40, 40], [1000] * 6):
        off = torch.tensor(o, dtype=torch.int32, device="cuda")
        kda.grouped_gemm(x, W, off, y=buf[4:-4])
        assert (buf[:4] == 5.0).all() and (buf[-4:] == 5.0).all()
        kda.grouped_gemm_backward(x, x, W, off)
    quiet()


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_gated_gradients_against_differences(act):
    """Central differences of L = sum dh h in one direction of every operand."""
    off, R, E = groups("few")
    F, K, dt = 24, 40, torch.float16
    ops = {"x": normal(R, K, seed=1, dtype=dt), "Wg": normal(E, F, K, seed=2, dtype=dt, std=0.2),
           "Wu": normal(E, F, K, seed=3, dtype=dt, std=0.2)}
    dh = normal(R, F, seed=4, dtype=dt)
    end = int(off[-1])
    _, g, u = kda.grouped_gated_ffn(ops["x"], ops["Wg"], ops["Wu"], off, act=act, save=True)
    got = dict(zip(("x", "Wg", "Wu"), kda.grouped_gated_ffn_backward(dh, ops["x"], ops["Wg"], ops["Wu"], off, g, u, act=act)))
    for name, v in ops.items():
        d = normal(*v.shape, seed=9).double()
        if name == "x":
            d[end:] = 0
        f = []
        for s in (1e-4, -1e-4):
            p = {k: t.double() + (s * d if k == name else 0) for k, t in ops.items()}
            f.append(float((dh.double()[:end] * grouped_gated(p["x"][:end], p["Wg"], p["Wu"], off, act)[0]).sum()))
        slope = (f[0] - f[1]) / 2e-4
        grad = got[name].double()
        if name == "x":
            grad[end:] = 0
        # each element of a gradient is off by two roundings to 16 bits, of itself and of its operands
        tol = 4 * 2.0 ** -11 * float((grad.abs() * d.abs()).sum()) + 1e-6 * abs(slope)
        assert abs(float((grad * d).sum()) - slope) <= tol


def test_other_stream_and_graph():
    off, R, E = groups("tiles")
    F, K, dt = 136, 264, torch.float16

    def inputs(seed):
        return (normal(R, K, seed=seed, dtype=dt), normal(E, F, K, seed=seed + 1, dtype=dt, std=0.1),
                normal(E, F, K, seed=seed + 2, dtype=dt, std=0.1), normal(R, F, seed=seed + 3, dtype=dt, std=2.0 ** seed))

    def step(x, Wg, Wu, dh, off, stream=None):
        h, g, u = kda.grouped_gated_ffn(x, Wg, Wu, off, save=True, stream=stream)
        y = kda.grouped_gemm(x, Wg, off, stream=stream)
        return [h, g, u, y, *kda.grouped_gemm_backward(dh, x, Wg, off, stream=stream),
                *kda.grouped_gated_ffn_backward(dh, x, Wg, Wu, off, g, u, stream=stream)]

    def same(a, b, end):
        return all(torch.equal(p, q) if p.dim() == 3 else torch.equal(p[:end], q[:end]) for p, q in zip(a, b))

    want = step(*inputs(1), off)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = step(*inputs(1), off, stream=s)
    torch.cuda.synchronize()
    assert same(want, got, int(off[-1]))
    static, soff = inputs(1), off.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = step(*static, soff)
    for seed, sizes in ((2, [0, 300, 7, 1, 60, 0, 140]), (3, [0, 0, 0, 0, 0, 0, 0]), (4, [R, 0, 0, 0, 0, 0, 0])):
        new = inputs(seed)
        for a, b in zip(static, new):
            a.copy_(b)
        soff[1:] = torch.tensor(sizes).cumsum(0)            # other groups in the same graph
        g.replay()
        torch.cuda.synchronize()
        assert same(step(*new, soff), outs, sum(sizes))
    quiet()


def test_no_rows():
    dt = torch.bfloat16
    off = torch.zeros(4, dtype=torch.int32, device="cuda")
    x, dy = torch.empty((0, 64), dtype=dt, device="cuda"), torch.empty((0, 32), dtype=dt, device="cuda")
    W = normal(3, 32, 64, seed=1, dtype=dt)
    assert kda.grouped_gemm(x, W, off).shape == (0, 32)
    dx, dW = kda.grouped_gemm_backward(dy, x, W, off)
    assert dx.shape == (0, 64) and (dW == 0).all()
    h, g, u = kda.grouped_gated_ffn(x, W, W, off, save=True)
    _, dWg, dWu = kda.grouped_gated_ffn_backward(dy, x, W, W, off, g, u)
    assert h.shape == (0, 32) and (dWg == 0).all() and (dWu == 0).all()


def test_a_layer():
    """All of them in a row, forward and backward, against the layer's definition."""
    T, E, k, F, K, dt = 150, 12, 3, 136, 264, torch.bfloat16
    logits, x = normal(T, E, seed=1), normal(T, K, seed=2, dtype=dt)
    logits[100:] = -math.inf
    Wg, Wu = (normal(E, F, K, seed=s, dtype=dt, std=0.1) for s in (3, 4))
    Wd, dy = normal(E, K, F, seed=5, dtype=dt, std=0.1), normal(T, K, seed=6, dtype=dt)
    r = kda.moe_route(logits, k)
    rows = kda.moe_dispatch(x, r)
    h, g, u = kda.grouped_gated_ffn(rows, Wg, Wu, r.offsets, save=True)
    out = kda.grouped_gemm(h, Wd, r.offsets)
    y = kda.moe_combine(out, r)
    drows, dw = kda.moe_combine_backward(dy, out, r)
    dh, dWd = kda.grouped_gemm_backward(drows, h, Wd, r.offsets)
    dxr, dWg, dWu = kda.grouped_gated_ffn_backward(dh, rows, Wg, Wu, r.offsets, g, u)
    dx, dl = kda.moe_dispatch_backward(dxr, r), kda.moe_route_backward(dw, logits, r)
    v = {"x": x, "Wg": Wg, "Wu": Wu, "Wd": Wd, "l": logits}
    v = {n: t.double().requires_grad_() for n, t in v.items()}
    ids = r.ids.long()
    w = torch.softmax(v["l"].gather(1, ids.clamp(min=0))[:100], dim=1)
    ref = torch.zeros((T, K), dtype=torch.float64, device="cuda")
    for t in range(100):
        for s in range(k):
            e = ids[t, s]
            a = v["Wg"][e] @ v["x"][t]
            ref[t] = ref[t] + w[t, s] * (v["Wd"][e] @ (torch.nn.functional.silu(a) * (v["Wu"][e] @ v["x"][t])))
    ref.backward(dy.double())
    # a chain of products with operands and results in 16 bits: each adds at most a
    # rounding, relative to the whole
    for name, got, want in (("y", y, ref), ("dx", dx, v["x"].grad), ("dWg", dWg, v["Wg"].grad), ("dWu", dWu, v["Wu"].grad),
                            ("dWd", dWd, v["Wd"].grad), ("dlogits", dl, v["l"].grad)):
        err = float((got.double() - want.detach()).norm() / want.detach().norm())
        assert err < 6 * 2.0 ** -8, (name, err)
    assert (y[100:] == 0).all() and (dx[100:] == 0).all() and (dl[100:] == 0).all()
    quiet()
