"""The mixture-of-experts operators as programs use them: calls at once on several
streams, two graphs at a time, weights beyond 2^31 elements, the command."""
import json
import math

import pytest
import torch

import decode_projection_gemms_gb300 as kda
from decode_projection_gemms_gb300 import binding, cli
from ffn_ref import close, product_bounds

pytestmark = pytest.mark.gpu


def normal(*shape, seed, dtype=torch.float32, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(0.0, std, generator=g)


def layer(seed, T=300, E=12, F=136, K=264, dtype=torch.bfloat16):
    x, dy = normal(T, K, seed=seed, dtype=dtype), normal(T, K, seed=seed + 1, dtype=dtype)
    Wr = normal(E, K, seed=seed + 2, dtype=dtype, std=0.1)
    Wg, Wu = (normal(E, F, K, seed=seed + s, dtype=dtype, std=0.1) for s in (3, 4))
    return x, dy, Wr, Wg, Wu, normal(E, K, F, seed=seed + 5, dtype=dtype, std=0.1)


def step(x, dy, *weights):
    y, saved = cli.moe_layer(x, *weights, 3, save=True)
    return [y, *cli.moe_layer_backward(dy, x, *weights, saved)]


def same(a, b):
    return all(torch.equal(p, q) for p, q in zip(a, b))


def test_layers_share_the_gpu_across_streams():
    ops = [layer(10 * i) for i in range(4)]
    want = [step(*o) for o in ops]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ops]
    for _ in range(5):
        got = []
        for s, o in zip(streams, ops):
            with torch.cuda.stream(s):
                got.append(step(*o))
        torch.cuda.synchronize()
        assert all(same(a, b) for a, b in zip(want, got))
    assert binding.device_error() == 0


def test_two_graphs_of_a_layer():
    """Captured one behind the other from the same pool, replayed in turn and at once."""
    ops = [layer(1), layer(100)]
    want = [step(*o) for o in ops]
    graphs, outs, pool = [], [], None
    for o in ops:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(step(*o))
        graphs.append(g)
    for order in ((0, 1), (1, 0), (0, 0, 1)):
        for o in outs:
            for t in o:
                t.fill_(math.nan)
        for i in order:
            graphs[i].replay()
        torch.cuda.synchronize()
        assert all(same(a, b) for a, b in zip(want, outs))
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(3):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        assert all(same(a, b) for a, b in zip(want, outs))
    assert binding.device_error() == 0


def test_operands_on_a_stream_of_their_own():
    """Inputs freed right behind a call on another stream."""
    o = layer(7)
    want = step(*o)
    s = torch.cuda.Stream()
    for _ in range(3):
        x, Wr = o[0].clone(), o[2]
        logits = binding.skinny_gemm_ex(x, Wr)
        s.wait_stream(torch.cuda.current_stream())
        r = kda.moe_route(logits, 3, stream=s)
        rows = kda.moe_dispatch(x, r, stream=s)
        del logits, x
        torch.empty((300, 264), dtype=torch.bfloat16, device="cuda").fill_(math.nan)
        h = kda.grouped_gated_ffn(rows, o[3], o[4], r.offsets, stream=s)
        y = kda.moe_combine(kda.grouped_gemm(h, o[5], r.offsets, stream=s), r, stream=s)
        s.synchronize()
        assert torch.equal(y, want[0])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_weights_and_gradients_beyond_32_bits(dtype):
    """2.7e9 elements: the last expert's lie past 2^31."""
    E, N, K = 40, 8192, 8192
    W = normal(E, N, K, seed=1, dtype=dtype, std=0.02)
    n = torch.zeros(E, dtype=torch.int64)
    n[0], n[20], n[39] = 5, 33, 17
    off = torch.cat([torch.zeros(1, dtype=torch.int64), n.cumsum(0)]).to(torch.int32).cuda()
    R = int(off[-1])
    x, dy = normal(R, K, seed=2, dtype=dtype), normal(R, N, seed=3, dtype=dtype, std=0.05)
    y = kda.grouped_gemm(x, W, off)
    dx, dW = kda.grouped_gemm_backward(dy, x, W, off)
    for e in (0, 20, 39):
        r = slice(int(off[e]), int(off[e + 1]))
        xe, d, w = x[r].double(), dy[r].double(), W[e].double()
        close(y[r], *product_bounds(xe, w), "y")
        close(dx[r], *product_bounds(d, w.t()), "dx")
        close(dW[e], *product_bounds(d.t(), xe.t()), "dW")
    assert not dW[38].any() and not dW[1].any()
    assert binding.device_error() == 0


def test_rows_beyond_32_bits():
    """2.3e9 elements of rows; the last of them lie past 2^31."""
    T, k, K, E = 140000, 2, 8200, 4
    logits = normal(T, E, seed=1)
    r = kda.moe_route(logits, k)
    x = normal(T, K, seed=2, dtype=torch.bfloat16)
    rows = kda.moe_dispatch(x, r)
    last = slice(T * k - 300, T * k)
    assert torch.equal(rows[last], x[(r.order[last] // k).long()])
    y = kda.moe_combine(rows, r)          # weights add up to 1 within fp32's roundings
    assert ((y[-200:].float() - x[-200:].float()).abs() <= 2.0 ** -7 * x[-200:].float().abs()).all()
    W = normal(E, 128, K, seed=3, dtype=torch.bfloat16, std=0.02)
    out = kda.grouped_gemm(rows, W, r.offsets)
    close(out[last], *product_bounds(rows[last].double(), W[E - 1].double()))
    assert int(r.offsets[E]) - int(r.offsets[E - 1]) >= 300
    assert binding.device_error() == 0


def test_most_experts_and_choices():
    T, E, k, F, K = 500, 1024, 32, 64, 64
    r = kda.moe_route(normal(T, E, seed=1), k, score="sigmoid")
    x, W = normal(T, K, seed=2, dtype=torch.float16), normal(E, F, K, seed=3, dtype=torch.float16, std=0.1)
    rows = kda.moe_dispatch(x, r)
    y = kda.grouped_gemm(rows, W, r.offsets)
    h, g, u = kda.grouped_gated_ffn(rows, W, W, r.offsets, save=True)
    ids = r.ids.reshape(-1).long()[r.order.long()]
    ref = torch.einsum("rk,rfk->rf", rows.double(), W.double()[ids])
    bound = 2.0 ** -18 * torch.einsum("rk,rfk->rf", rows.double().abs(), W.double().abs()[ids])
    close(y, ref, bound)
    assert torch.equal(g, u) and torch.equal(g.to(torch.float16), y)
    dx, dW = kda.grouped_gemm_backward(y, rows, W, r.offsets)
    ref = torch.einsum("rf,rfk->rk", y.double(), W.double()[ids])
    close(dx, ref, 2.0 ** -18 * torch.einsum("rf,rfk->rk", y.double().abs(), W.double().abs()[ids]))
    for e in (0, 500, 1023):
        m = slice(int(r.offsets[e]), int(r.offsets[e + 1]))
        close(dW[e], *product_bounds(y[m].double().t(), rows[m].double().t()))
    assert binding.device_error() == 0


@pytest.mark.parametrize("shift", [1, 2, 4, 8])
@pytest.mark.parametrize("N", [64, 130, 203, 261])
def test_outputs_inside_wider_matrices(N, shift):
    """Rows that start on 2, 4, 8 and 16 bytes, guard columns and rows around them."""
    off = torch.tensor([0, 3, 3, 70, 101], dtype=torch.int32, device="cuda")
    R, E, K, pad = 104, 4, 72, 40
    x, W = normal(R, K, seed=1, dtype=torch.bfloat16), normal(E, N, K, seed=2, dtype=torch.bfloat16, std=0.1)
    V = normal(E, N, K, seed=3, dtype=torch.bfloat16, std=0.1)
    wide = N + shift + pad + (-(N + shift + pad)) % 8
    for call in (lambda y: kda.grouped_gemm(x, W, off, y=y), lambda y: kda.grouped_gated_ffn(x, W, V, off, h=y)):
        want = call(None)[:101]
        buf = torch.full((R + 6, wide), 5.0, dtype=torch.bfloat16, device="cuda")
        call(buf[3:-3, shift:shift + N])
        assert torch.equal(buf[3:3 + 101, shift:shift + N], want)
        buf[3:3 + 101, shift:shift + N] = 5.0
        assert (buf == 5.0).all()


def test_layer_function_gradients():
    """The command's layer against automatic differentiation of its definition."""
    x, dy, Wr, Wg, Wu, Wd = layer(3, T=61, E=5)
    y, saved = cli.moe_layer(x, Wr, Wg, Wu, Wd, 2, act="gelu_tanh", score="sigmoid", save=True)
    got = cli.moe_layer_backward(dy, x, Wr, Wg, Wu, Wd, saved, act="gelu_tanh")
    ops = [t.double().requires_grad_() for t in (x, Wr, Wg, Wu, Wd)]
    xd, rd, gd, ud, dd = ops
    ids = saved[1].ids.long()
    s = torch.sigmoid((xd @ rd.t()).gather(1, ids))
    w = s / s.sum(dim=1, keepdim=True)
    ref = 0
    for j in range(2):
        e = ids[:, j]
        a = torch.nn.functional.gelu(torch.einsum("tk,tfk->tf", xd, gd[e]), approximate="tanh")
        ref = ref + w[:, j:j + 1] * torch.einsum("tf,tkf->tk", a * torch.einsum("tk,tfk->tf", xd, ud[e]), dd[e])
    ref.backward(dy.double())
    # logits, rows, h and the gradients between the products are in 16 bits: each adds at
    # most a rounding, relative to the whole
    for name, a, b in zip(("y", "dx", "dWr", "dWg", "dWu", "dWd"), (y, *got), (ref.detach(), *(t.grad for t in ops))):
        err = float((a.double() - b).norm() / b.norm())
        assert err < 8 * 2.0 ** -8, (name, err)


def test_layer_behind_a_norm_gradients():
    """y = x + layer(norm(x)), with its norm's weight, against automatic differentiation."""
    x, dy, *weights = layer(5, T=50, E=4)
    gamma = normal(264, seed=77, dtype=torch.bfloat16, std=0.2) + 1
    y, saved = cli.norm_moe_layer(x, gamma, *weights, top_k=2, save=True)
    assert torch.equal(cli.norm_moe_layer(x, gamma, *weights, top_k=2)[0], y)
    got = cli.norm_moe_layer_backward(dy, x, gamma, *weights, saved=saved)
    ops = [t.double().requires_grad_() for t in (x, gamma, *weights)]
    xd, cd, rd, gd, ud, dd = ops
    z = xd / torch.sqrt((xd * xd).mean(dim=1, keepdim=True) + 1e-5) * cd
    ids = saved[2][1].ids.long()
    w = torch.softmax((z @ rd.t()).gather(1, ids), dim=1)
    ref = xd
    for j in range(2):
        e = ids[:, j]
        a = torch.nn.functional.silu(torch.einsum("tk,tfk->tf", z, gd[e]))
        ref = ref + w[:, j:j + 1] * torch.einsum("tf,tkf->tk", a * torch.einsum("tk,tfk->tf", z, ud[e]), dd[e])
    ref.backward(dy.double())
    # as above, with the norm's roundings
    for name, a, b in zip(("y", "dx", "dgamma", "dWr", "dWg", "dWu", "dWd"), (y, *got), (ref.detach(), *(t.grad for t in ops))):
        err = float((a.double() - b).norm() / b.norm())
        assert err < 10 * 2.0 ** -8, (name, err)


def test_command_trains_and_serves(capsys):
    cli.main(["--moe", "--M", "1", "37", "--experts", "6", "--top-k", "2", "--F", "136", "--K", "264", "--steps", "2",
              "--reps", "2"])
    lines = [json.loads(v) for v in capsys.readouterr().out.splitlines() if v.startswith("{")]
    assert len(lines) == 3 and len(lines[0]["training"]["losses"]) == 3
    assert all(math.isfinite(v) for v in lines[0]["training"]["losses"])
    assert [v["M"] for v in lines[1:]] == [1, 37] and [v["rows"] for v in lines[1:]] == [2, 74]
    assert all(v["device_error"] == 0 for v in lines[1:])
