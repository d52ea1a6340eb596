"""Feed-forward operators on the GPU against plain 64-bit forms: microscaled 4-bit
quantisation, its product, the gated block and its 4-bit form."""
import math

import pytest
import torch

import decode_projection_gemms_gb300 as kda
from decode_projection_gemms_gb300 import binding
from ffn_ref import UNIT, act as act64, close, gated, gated_grads, mx4_values, product_bounds

pytestmark = pytest.mark.gpu
HALF = (torch.bfloat16, torch.float16)
ALL = HALF + (torch.float32,)
ACTS = ("silu", "gelu", "gelu_tanh")


def normal(rows, cols, seed, dtype=torch.float32, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn((rows, cols), generator=g, device="cuda") * std).to(dtype)


def strided(t, extra, offset=0):
    """The same matrix as a view into a wider one, filled with NaN around it."""
    rows, cols = t.shape
    wide = torch.full((rows, cols + extra + offset), math.nan, dtype=t.dtype, device=t.device)
    v = wide[:, offset:offset + cols]
    v.copy_(t)
    return v


def quiet(code=0):
    torch.cuda.synchronize()
    assert binding.device_error() == code


# ---- quantisation ---------------------------------------------------------------

@pytest.mark.parametrize("dtype", ALL)
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 31), (3, 32), (2, 33), (5, 127), (129, 256), (64, 257),
                                       (127, 1000), (300, 7168), (1, 7156)])
def test_quantize_values(rows, cols, dtype):
    x = normal(rows, cols, rows * 7 + cols, dtype, std=0.3)
    x *= torch.exp2(torch.randint(-9, 9, (rows, 1), device="cuda")).to(dtype)
    q = kda.mx4_quantize(x)
    for out in ALL:
        v = kda.mx4_dequantize(q, dtype=out)
        assert v.dtype is out
        assert torch.equal(v.double(), mx4_values(x).to(out).double())
    quiet()


def test_quantize_ties_extremes_and_non_finite():
    rows = []
    ties = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.0]
    for e in (-126, -60, 0, 60, 120):
        rows.append([s * t * 2.0 ** e for t in ties for s in (1, -1)] + [4.0 * 2.0 ** e] * 16)
    tiny = 2.0 ** -149
    rows.append([tiny * i for i in range(32)])                       # subnormal: scale stays 2^-127
    rows.append([2.0 ** -127 * (i / 8) for i in range(32)])
    rows.append([0.0] * 32)
    rows.append([-0.0] * 32)
    rows.append([3.4028234663852886e38 * (1 if i % 2 else -0.5) for i in range(32)])
    x = torch.tensor(rows, dtype=torch.float32, device="cuda")
    v = kda.mx4_dequantize(kda.mx4_quantize(x), dtype=torch.float32)
    assert torch.equal(v.double(), mx4_values(x))
    for bad in (math.nan, math.inf, -math.inf):
        y = normal(2, 96, 3)
        y[1, 40] = bad
        v = kda.mx4_dequantize(kda.mx4_quantize(y), dtype=torch.float32)
        assert torch.isnan(v[1, 32:64]).all()
        keep = torch.ones(2, 96, dtype=torch.bool, device="cuda")
        keep[1, 32:64] = False
        assert torch.equal(v[keep].double(), mx4_values(y)[keep])


@pytest.mark.parametrize("dtype", ALL)
@pytest.mark.parametrize("extra,offset", [(1, 0), (8, 0), (3, 1), (24, 8)])
def test_quantize_strided_and_unaligned(dtype, extra, offset):
    x = normal(37, 203, 5, dtype)
    v = strided(x, extra, offset)
    a, b = kda.mx4_quantize(x), kda.mx4_quantize(v)
    assert torch.equal(a.codes, b.codes) and torch.equal(a.scales, b.scales)
    y = torch.full((37, 203 + extra + offset), 7.0, dtype=dtype, device="cuda")
    kda.mx4_dequantize(a, dtype=dtype, y=y[:, offset:offset + 203])
    assert torch.equal(y[:, offset:offset + 203], kda.mx4_dequantize(a, dtype=dtype))
    rest = torch.ones_like(y, dtype=torch.bool)
    rest[:, offset:offset + 203] = False
    assert (y[rest] == 7.0).all()


def test_quantize_pads_are_zero_and_empty_is_nothing():
    codes_nan = kda.mx4_quantize(normal(130, 40, 9))
    t = codes_nan.scales.view(2, 1, 32, 4, 4)     # row tile, column tile, r % 32, r / 32, block
    assert (t[1, 0, 2:, 0] == 0).all() and (t[1, 0, :, 1:] == 0).all()      # rows past 130
    assert (t[:, :, :, :, 2:] == 0).all()                                   # blocks past 40 columns
    assert (codes_nan.codes[:, 20:] == 0).all()
    e = kda.mx4_quantize(torch.empty((0, 64), device="cuda"))
    assert e.shape == (0, 64) and kda.mx4_dequantize(e).shape == (0, 64)


# ---- 4-bit product --------------------------------------------------------------

@pytest.mark.parametrize("dtype", HALF)
@pytest.mark.parametrize("M,N,K", [(1, 1, 1), (1, 128, 32), (1, 64, 64), (2, 129, 65), (7, 100, 127), (16, 256, 256),
                                   (17, 300, 257), (33, 127, 384), (64, 513, 640), (100, 999, 1000),
                                   (128, 128, 2048), (129, 257, 513), (1, 4096, 7168), (300, 640, 2050),
                                   (513, 1025, 777), (1100, 2050, 514),
                                   (1537, 1921, 1300), (2048, 1024, 256), (700, 3200, 100)])
def test_mx4_gemm(M, N, K, dtype):
    x = normal(M, K, M + K, dtype)
    W = normal(N, K, N + 1, torch.bfloat16, std=0.02)
    Wq = kda.mx4_quantize(W)
    y = kda.mx4_gemm(x, Wq)
    ref, bound = product_bounds(mx4_values(x), mx4_values(W))
    close(y, ref, bound, f"{M}x{N}x{K}")
    # the same product from codes given beforehand, bit for bit
    assert torch.equal(kda.mx4_gemm(kda.mx4_quantize(x), Wq, dtype=dtype), y)
    assert torch.equal(kda.mx4_gemm(x, Wq), y)
    quiet()


def test_mx4_gemm_one_hot_selects_columns():
    """x one-hot per row: the product is a column of W's values, exactly; every
    position of a 256-column stage, so a scale or a code out of place shows."""
    K, N = 515, 200
    x = torch.eye(K, device="cuda", dtype=torch.bfloat16)
    W = normal(N, K, 4) * torch.exp2(torch.randint(-6, 6, (N, K), device="cuda").float())
    y = kda.mx4_gemm(x, kda.mx4_quantize(W))
    assert torch.equal(y.double(), mx4_values(W).t().contiguous())


def test_mx4_gemm_nan_blocks_reach_their_rows_only():
    x, W = normal(9, 320, 1, torch.bfloat16), normal(40, 320, 2)
    x[4, 100] = math.nan
    W[7, 300] = math.inf
    y = kda.mx4_gemm(x, kda.mx4_quantize(W))
    bad = torch.zeros(9, 40, dtype=torch.bool, device="cuda")
    bad[4] = True
    bad[:, 7] = True
    assert torch.isnan(y[bad]).all() and torch.isfinite(y[~bad]).all()


@pytest.mark.parametrize("ldx,ldy", [(0, 0), (1, 3), (8, 8)])
def test_mx4_gemm_strided(ldx, ldy):
    x, W = normal(21, 300, 1, torch.float16), normal(70, 300, 2)
    Wq = kda.mx4_quantize(W)
    ref = kda.mx4_gemm(x, Wq)
    wide = torch.full((21, 70 + ldy), 5.0, dtype=torch.float16, device="cuda")
    out = kda.mx4_gemm(strided(x, ldx) if ldx else x, Wq, y=wide[:, :70])
    assert out.data_ptr() == wide.data_ptr()
    assert torch.equal(wide[:, :70], ref) and (wide[:, 70:] == 5.0).all()


# ---- gated block ----------------------------------------------------------------

GATED = [(1, 1, 8), (1, 128, 64), (2, 40, 72), (16, 128, 128), (17, 136, 200), (31, 264, 1032), (96, 512, 512),
         (127, 127, 136), (128, 256, 64), (129, 300, 520), (1, 2048, 7168), (300, 1000, 264), (600, 520, 1024),
         (1100, 1416, 328)]


@pytest.mark.parametrize("dtype", HALF)
@pytest.mark.parametrize("T,F,K", GATED)
def test_gated_ffn(T, F, K, dtype):
    act = ACTS[(T + F) % 3]
    x = normal(T, K, T, dtype)
    Wg, Wu = normal(F, K, 2, dtype, std=K ** -0.5 * 1.5), normal(F, K, 3, dtype, std=K ** -0.5)
    h, g, u = kda.gated_ffn(x, Wg, Wu, act=act, save=True)
    rh, eh, rg, eg, ru, eu = gated(x.double(), Wg.double(), Wu.double(), act)
    close(h, rh, eh, "h")
    assert g.dtype is torch.float32 and ((g.double() - rg).abs() <= eg).all()
    assert u.dtype is torch.float32 and ((u.double() - ru).abs() <= eu).all()
    assert torch.equal(kda.gated_ffn(x, Wg, Wu, act=act), h)
    quiet()


@pytest.mark.parametrize("act", ACTS)
def test_gated_ffn_activation_over_its_range(act):
    """K = 8 with one live column: g and u are chosen exactly, far into both tails."""
    g = torch.cat([torch.linspace(-100, 100, 401), torch.linspace(-4, 4, 200),
                   torch.tensor([0.0, -0.0, 1e-30, -1e-30, 3e4, -3e4])]).to(torch.bfloat16)
    T = g.numel()
    x = torch.zeros((T, 8), dtype=torch.bfloat16, device="cuda")
    x[:, 0] = g.cuda()
    x[:, 1] = 1.0
    Wg = torch.zeros((9, 8), dtype=torch.bfloat16, device="cuda")
    Wu = torch.zeros((9, 8), dtype=torch.bfloat16, device="cuda")
    Wg[:, 0] = 1.0
    Wu[:, 1] = 1.0
    h = kda.gated_ffn(x, Wg, Wu, act=act)
    rh, eh, *_ = gated(x.double(), Wg.double(), Wu.double(), act)
    close(h, rh, eh, act)


def test_gated_ffn_strided_views():
    T, F, K = 45, 88, 192
    x, Wp = normal(T, K, 1, torch.bfloat16), normal(2 * F, K, 2, torch.bfloat16, std=0.1)
    ref = kda.gated_ffn(x, Wp[:F].contiguous(), Wp[F:].contiguous())
    # halves of one packed weight, and rows inside wider matrices
    assert torch.equal(kda.gated_ffn(x, Wp[:F], Wp[F:]), ref)
    wide = torch.full((T, F + 5), 3.0, dtype=torch.bfloat16, device="cuda")
    kda.gated_ffn(strided(x, 8), strided(Wp[:F], 16), strided(Wp[F:], 24, 8), h=wide[:, :F])
    assert torch.equal(wide[:, :F], ref) and (wide[:, F:] == 3.0).all()


# ---- its backward pass ---------------------------------------------------------------

@pytest.mark.parametrize("dtype", HALF)
@pytest.mark.parametrize("T,F,K", [(1, 1, 8), (1, 40, 64), (2, 264, 72), (7, 13, 16), (63, 128, 256), (64, 257, 320),
                                   (65, 100, 1000), (255, 512, 264), (256, 256, 256), (300, 1000, 520),
                                   (777, 264, 2056), (1, 2048, 2048), (1030, 1416, 600)])
def test_gated_ffn_backward(T, F, K, dtype):
    act = ACTS[(T + F) % 3]
    x, dh = normal(T, K, T, dtype), normal(T, F, T + 1, dtype, std=0.05)
    Wg, Wu = normal(F, K, 2, dtype, std=K ** -0.5 * 1.5), normal(F, K, 3, dtype, std=K ** -0.5)
    _, g, u = kda.gated_ffn(x, Wg, Wu, act=act, save=True)
    grads = kda.gated_ffn_backward(dh, x, Wg, Wu, g, u, act=act)
    ref = gated_grads(dh.double(), x.double(), Wg.double(), Wu.double(), act, UNIT[dtype])
    for got, name in zip(grads, ("dx", "dWg", "dWu")):
        close(got, *ref[name], f"{name} {T}x{F}x{K}")
    again = kda.gated_ffn_backward(dh, x, Wg, Wu, g, u, act=act)
    assert all(torch.equal(a, b) for a, b in zip(grads, again))
    quiet()


@pytest.mark.parametrize("act", ACTS)
def test_gated_ffn_backward_against_differences(act):
    """<gradient, direction> against central differences of the 64-bit forward
    pass. With step e the difference is off by O(e^2) = 1e-8 of the loss's third
    derivative, far below the operands' rounding, which the bound carries."""
    T, F, K = 70, 96, 128
    dt = torch.float16
    x, dh = normal(T, K, 1, dt), normal(T, F, 2, dt, std=0.05)
    Wg, Wu = normal(F, K, 3, dt, std=0.12), normal(F, K, 4, dt, std=0.09)
    _, g, u = kda.gated_ffn(x, Wg, Wu, act=act, save=True)
    grads = kda.gated_ffn_backward(dh, x, Wg, Wu, g, u, act=act)
    p = [t.double() for t in (x, Wg, Wu)]
    ref = gated_grads(dh.double(), *p, act, UNIT[dt])

    def loss(a, b, c):
        return ((act64(a @ b.t(), act)[0] * (a @ c.t())) * dh.double()).sum()

    e = 1e-4
    for i, (got, name) in enumerate(zip(grads, ("dx", "dWg", "dWu"))):
        v = normal(*got.shape, 10 + i).double()
        hi, lo = list(p), list(p)
        hi[i], lo[i] = p[i] + e * v, p[i] - e * v
        diff = (loss(*hi) - loss(*lo)) / (2 * e)
        tol = ((ref[name][1] + UNIT[dt] * ref[name][0].abs()) * v.abs()).sum() + 1e-5 * diff.abs()
        assert ((got.double() * v).sum() - diff).abs() <= tol


def test_gated_ffn_backward_strided_and_empty():
    T, F, K = 45, 88, 192
    x, Wp, dh = normal(T, K, 1, torch.bfloat16), normal(2 * F, K, 2, torch.bfloat16, std=0.1), normal(T, F, 3, torch.bfloat16)
    _, g, u = kda.gated_ffn(x, Wp[:F], Wp[F:], save=True)
    ref = kda.gated_ffn_backward(dh, x, Wp[:F], Wp[F:], g, u)
    for extra, offset in ((8, 0), (1, 2), (3, 0)):
        got = kda.gated_ffn_backward(strided(dh, extra, offset), strided(x, 8), strided(Wp[:F], 16),
                                     strided(Wp[F:], 24, 8), g, u)
        assert all(torch.equal(a, b) for a, b in zip(ref, got))
    e = torch.empty((0, K), dtype=torch.bfloat16, device="cuda")
    ef = torch.empty((0, F), dtype=torch.bfloat16, device="cuda")
    dx, dWg, dWu = kda.gated_ffn_backward(ef, e, Wp[:F], Wp[F:], ef, ef)
    assert dx.shape == (0, K) and (dWg == 0).all() and (dWu == 0).all() and dWg.shape == (F, K)
    with pytest.raises(ValueError):
        kda.gated_ffn_backward(dh[:, :80], x, Wp[:F], Wp[F:], g, u)
    with pytest.raises(ValueError):
        kda.gated_ffn_backward(dh, x, Wp[:F], Wp[F:], g.t(), u)
    quiet()


# ---- gated block over 4-bit weights ------------------------------------------------

@pytest.mark.parametrize("dtype", HALF)
@pytest.mark.parametrize("T,F,K", [(1, 1, 1), (1, 128, 256), (3, 130, 100), (16, 256, 257), (64, 384, 1000),
                                   (100, 127, 64), (128, 128, 640), (129, 500, 513), (8, 2048, 7168),
                                   (700, 900, 1111), (1025, 1300, 390), (1300, 1030, 1024)])
def test_mx4_gated_ffn(T, F, K, dtype):
    act = ACTS[(T + F) % 3]
    x = normal(T, K, T, dtype)
    Wg, Wu = normal(F, K, 2, std=K ** -0.5 * 1.5), normal(F, K, 3, std=K ** -0.5)
    qg, qu = kda.mx4_quantize(Wg), kda.mx4_quantize(Wu)
    h = kda.mx4_gated_ffn(x, qg, qu, act=act)
    rh, eh, *_ = gated(mx4_values(x), mx4_values(Wg), mx4_values(Wu), act)
    close(h, rh, eh, "h")
    assert torch.equal(kda.mx4_gated_ffn(kda.mx4_quantize(x), qg, qu, act=act, dtype=dtype), h)
    quiet()


# ---- streams, graphs, refusals -----------------------------------------------------

def test_other_stream_and_graph_replay():
    x, Wg, Wu = normal(20, 256, 1, torch.bfloat16), normal(256, 256, 2, torch.bfloat16), normal(256, 256, 3, torch.bfloat16)
    qg, qu = kda.mx4_quantize(Wg), kda.mx4_quantize(Wu)
    want = [kda.gated_ffn(x, Wg, Wu), kda.mx4_gated_ffn(x, qg, qu), kda.mx4_gemm(x, qg)]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = [kda.gated_ffn(x, Wg, Wu, stream=s), kda.mx4_gated_ffn(x, qg, qu, stream=s), kda.mx4_gemm(x, qg, stream=s)]
    s.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a, b)
    xin = x.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = [kda.gated_ffn(xin, Wg, Wu), kda.mx4_gated_ffn(xin, qg, qu), kda.mx4_gemm(xin, qg)]
    x2 = normal(20, 256, 8, torch.bfloat16)
    xin.copy_(x2)
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(outs, [kda.gated_ffn(x2, Wg, Wu), kda.mx4_gated_ffn(x2, qg, qu), kda.mx4_gemm(x2, qg)]):
        assert torch.equal(a, b)


def test_no_tokens():
    W = normal(32, 64, 1, torch.bfloat16)
    q = kda.mx4_quantize(W)
    x = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    assert kda.gated_ffn(x, W, W).shape == (0, 32)
    assert kda.mx4_gemm(x, q).shape == (0, 32)
    assert kda.mx4_gated_ffn(x, q, q).shape == (0, 32)


def test_refusals():
    x, W = normal(4, 64, 1, torch.bfloat16), normal(32, 64, 2, torch.bfloat16)
    q = kda.mx4_quantize(W)
    with pytest.raises(TypeError):
        kda.mx4_quantize(torch.zeros((2, 32), dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        kda.mx4_quantize(torch.zeros((2, 32)))
    with pytest.raises(ValueError):
        kda.mx4_quantize(x.t())
    with pytest.raises(TypeError):
        kda.mx4_gemm(x, W)
    with pytest.raises(TypeError):
        kda.mx4_gemm(x.float(), q)
    with pytest.raises(ValueError):
        kda.mx4_gemm(x[:, :32], q)
    with pytest.raises(ValueError):
        kda.mx4_gemm(x, q, y=torch.empty((4, 31), dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(TypeError):
        kda.mx4_gemm(x, q, y=torch.empty((4, 32), dtype=torch.float16, device="cuda"))
    with pytest.raises(ValueError):
        kda.gated_ffn(x, W, W, act="relu")
    with pytest.raises(TypeError):
        kda.gated_ffn(x, W.half(), W)
    with pytest.raises(ValueError):
        kda.gated_ffn(x, W, W[:16])
    with pytest.raises(kda.KdaProjError) as e:
        kda.gated_ffn(normal(4, 60, 1, torch.bfloat16), normal(8, 60, 1, torch.bfloat16), normal(8, 60, 1, torch.bfloat16))
    assert e.value.code == binding.KP_ESHAPE
    with pytest.raises(kda.KdaProjError) as e:       # rows that do not start on 16 bytes
        kda.gated_ffn(strided(x, 7, 1), W, W)
    assert e.value.code == binding.KP_EALIGN
    quiet()


# ---- sharing an SM, guard regions, the command --------------------------------------

def test_operators_share_the_gpu_across_streams():
    """Calls on four streams at once, each with its own workspace, next to the
    projection's kernels: tensor memory is shared by what shares an SM."""
    x, Wg, Wu = normal(40, 512, 1, torch.bfloat16), normal(512, 512, 2, torch.bfloat16, 0.05), normal(512, 512, 3, torch.bfloat16, 0.05)
    q, qu = kda.mx4_quantize(Wg), kda.mx4_quantize(Wu)
    big = normal(700, 512, 4, torch.bfloat16)

    def work():
        h, g, u = kda.gated_ffn(big, Wg, Wu, save=True)
        return [kda.gated_ffn(x, Wg, Wu), kda.mx4_gemm(x, q), kda.mx4_gated_ffn(big, q, qu), h,
                *kda.gated_ffn_backward(h, big, Wg, Wu, g, u)]

    want = work()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(4)]
    got = []
    for rep in range(6):
        for s in streams:
            with torch.cuda.stream(s):
                got.append(work())
                if rep == 0:
                    kda.skinny_gemm(x[:8], Wg, cfg=kda.KpCfg.make("tc05", split_k=4))
    torch.cuda.synchronize()
    for outs in got:
        assert all(torch.equal(a, b) for a, b in zip(want, outs))
    quiet()


@pytest.mark.parametrize("T", [5, 70, 300, 1100])
@pytest.mark.parametrize("F,first,width", [(203, 30, 264), (203, 32, 264), (512, 32, 576), (720, 16, 752), (1000, 8, 1021)])
def test_nothing_is_written_outside_the_outputs(T, F, first, width):
    """Outputs as views into wider matrices, whose rows start on 32, 16, 4 or 2
    bytes: both kernels, tiles that end inside and outside the columns."""
    K = 264
    x, Wg, Wu = normal(T, K, 1, torch.bfloat16), normal(F, K, 2, torch.bfloat16), normal(F, K, 3, torch.bfloat16)
    q = kda.mx4_quantize(Wg)
    for run in (lambda y: kda.gated_ffn(x, Wg, Wu, h=y), lambda y: kda.mx4_gated_ffn(x, q, q, h=y),
                lambda y: kda.mx4_gemm(x, q, y=y)):
        want = run(None)
        guard = torch.full((T + 40, width), 9.0, dtype=torch.bfloat16, device="cuda")
        y = guard[20:20 + T, first:first + F]
        y.fill_(math.nan)
        run(y)
        assert torch.equal(y, want)
        keep = torch.ones_like(guard, dtype=torch.bool)
        keep[20:20 + T, first:first + F] = False
        assert (guard[keep] == 9.0).all()
    quiet()


def test_command_trains_and_serves(capsys):
    import json

    from decode_projection_gemms_gb300 import cli
    cli.main(["--ffn", "--M", "1", "24", "300", "--F", "256", "--K", "512", "--steps", "3", "--reps", "2"])
    lines = [json.loads(line) for line in capsys.readouterr().out.splitlines() if line.startswith("{")]
    losses = lines[0]["training"]["losses"]
    assert all(b < a for a, b in zip(losses, losses[1:]))
    assert [line["M"] for line in lines[1:]] == [1, 24, 300]
    for line in lines[1:]:
        # how far 4-bit outputs are from 16-bit ones is the format's; the operators
        # themselves are checked above
        assert line["relative_difference"] > 0 and line["device_error"] == 0
        assert line["weight_bytes_4_bit"] < 0.27 * line["weight_bytes_16_bit"]
