"""Host side of the mixture-of-experts operators: argument checks that need no device,
and the binding's refusals."""
import ctypes

import pytest
import torch

from decode_projection_gemms_gb300 import binding
from decode_projection_gemms_gb300.build import build
from test_ffn_binding_host import OnDevice, StreamOf, library  # noqa: F401


@pytest.fixture(scope="module")
def lib():
    build()
    return binding.load()


P, ODD, P8 = ctypes.c_void_p(256), ctypes.c_void_p(257), ctypes.c_void_p(264)
OK, EINVAL, EALIGN, ESHAPE = binding.KP_OK, binding.KP_EINVAL, binding.KP_EALIGN, binding.KP_ESHAPE


def test_workspace(lib):
    n = ctypes.c_size_t()
    w = lib.kp_moe_workspace
    assert w(0, -1, 4, 1, n) == EINVAL and w(0, 4, 0, 1, n) == EINVAL and w(7, 4, 4, 1, n) == EINVAL
    assert w(0, 4, 4, 1, None) == EINVAL
    assert w(0, 4, 8, 2, n) == OK and n.value == 0               # few tokens: none
    assert w(0, 10000, 64, 2, n) == OK and n.value >= 64 * 4


def test_route_argument_errors(lib):
    def call(logits=P, ld=8, bias=None, T=1, E=8, k=2, score=0, dtype=0, ids=P, weights=P, offsets=P, order=P,
             position=P, work=None, bytes=0):
        return lib.kp_moe_route(logits, ld, bias, T, E, k, score, dtype, ids, weights, offsets, order, position, work,
                                bytes, None)

    assert call(T=-1) == EINVAL and call(E=0) == EINVAL and call(k=0) == EINVAL and call(k=9) == EINVAL
    assert call(E=1025, ld=1025) == ESHAPE and call(E=64, ld=64, k=33) == ESHAPE
    assert call(T=2 ** 30, k=2) == ESHAPE
    assert call(dtype=3) == EINVAL and call(score=2) == EINVAL
    assert call(bias=P) == EINVAL                                  # a bias with softmax
    assert call(bias=ODD, score=1) == EALIGN
    assert call(logits=None) == EINVAL and call(logits=ODD) == EALIGN
    assert call(logits=ctypes.c_void_p(258), dtype=2) == EALIGN
    assert call(ld=7) == EINVAL
    assert call(T=2 ** 31 - 1, k=1) == ESHAPE                      # sums of a size and a block's pass 32 bits
    for name in ("ids", "weights", "offsets", "order", "position"):
        assert call(**{name: None}) == EINVAL and call(**{name: ODD}) == EALIGN
    assert call(T=1000) == EINVAL                                  # no workspace
    assert b"workspace" in lib.kp_last_error()

    def back(dweights=P, logits=P, ld=8, ids=P, weights=P, dlogits=P, ldd=8, T=1, E=8, k=2, score=0, dtype=0):
        return lib.kp_moe_route_backward(dweights, logits, ld, ids, weights, dlogits, ldd, T, E, k, score, dtype, None)

    assert back(T=0) == OK
    assert back(T=-1) == EINVAL and back(k=9) == EINVAL and back(score=5) == EINVAL and back(dtype=9) == EINVAL
    assert back(logits=None) == EINVAL and back(dlogits=None) == EINVAL and back(dlogits=ODD) == EALIGN
    assert back(ld=7) == EINVAL and back(ldd=7) == EINVAL
    assert back(dweights=None) == EINVAL and back(ids=ODD) == EALIGN and back(weights=None) == EINVAL


def test_rows_argument_errors(lib):
    def dispatch(x=P, ldx=8, position=P, rows=P, ldr=8, T=1, k=2, K=8, dtype=0):
        return lib.kp_moe_dispatch(x, ldx, position, rows, ldr, T, k, K, dtype, None)

    assert dispatch(T=0) == OK
    assert dispatch(T=-1) == EINVAL and dispatch(k=0) == EINVAL and dispatch(K=0) == EINVAL and dispatch(dtype=2) == EINVAL
    assert dispatch(T=2 ** 30) == ESHAPE
    assert dispatch(K=2 ** 31 - 1, ldx=2 ** 31, ldr=2 ** 31) == ESHAPE
    assert dispatch(x=None) == EINVAL and dispatch(x=ODD) == EALIGN and dispatch(ldx=7) == EINVAL
    assert dispatch(rows=None) == EINVAL and dispatch(ldr=7) == EINVAL and dispatch(position=ODD) == EALIGN

    def combine(rows=P, ldr=8, weights=P, position=P, y=P, ldy=8, T=1, k=2, K=8, dtype=0):
        return lib.kp_moe_combine(rows, ldr, weights, position, y, ldy, T, k, K, dtype, None)

    assert combine(T=0) == OK
    assert combine(T=-1) == EINVAL and combine(dtype=2) == EINVAL
    assert combine(rows=ODD) == EALIGN and combine(y=None) == EINVAL and combine(weights=ODD) == EALIGN
    assert combine(K=2 ** 31 - 8, ldr=2 ** 31, ldy=2 ** 31) == ESHAPE
    assert combine(position=None) == EINVAL and combine(ldy=4) == EINVAL

    def back(dy=P, lddy=8, rows=P, ldr=8, weights=P, position=P, drows=P, lddr=8, dweights=P, T=1, k=2, K=8, dtype=0):
        return lib.kp_moe_combine_backward(dy, lddy, rows, ldr, weights, position, drows, lddr, dweights, T, k, K, dtype,
                                           None)

    assert back(T=0) == OK
    assert back(dy=None) == EINVAL and back(rows=None) == EINVAL and back(drows=ODD) == EALIGN
    assert back(weights=None) == EINVAL and back(position=None) == EINVAL and back(dweights=ODD) == EALIGN
    assert back(lddy=7) == EINVAL and back(lddr=7) == EINVAL and back(K=-1) == EINVAL
    assert back(K=2 ** 31 - 8, lddy=2 ** 31, ldr=2 ** 31, lddr=2 ** 31) == ESHAPE


def test_norm_argument_errors(lib):
    def norm(x=P, ldx=8, weight=P, bias=None, y=P, ldy=8, mean=None, rstd=None, T=1, K=8, eps=1e-5, center=1, dtype=0):
        return lib.kp_layer_norm(x, ldx, weight, bias, y, ldy, mean, rstd, T, K, eps, center, dtype, None)

    assert norm(T=0) == OK
    assert norm(T=-1) == EINVAL and norm(K=0) == EINVAL and norm(dtype=3) == EINVAL
    assert norm(K=16385, ldx=16385, ldy=16385) == ESHAPE
    assert norm(eps=-1.0) == EINVAL and norm(eps=float("nan")) == EINVAL and norm(eps=float("inf")) == EINVAL
    assert norm(x=None) == EINVAL and norm(x=ODD) == EALIGN and norm(ldx=7) == EINVAL and norm(y=None) == EINVAL
    assert norm(x=ctypes.c_void_p(258), dtype=2) == EALIGN
    assert norm(weight=None) == EINVAL and norm(bias=ODD) == EALIGN and norm(mean=ODD) == EALIGN and norm(rstd=ODD) == EALIGN

    def back(dy=P, lddy=8, x=P, ldx=8, weight=P, mean=P, rstd=P, dx=P, lddx=8, dweight=P, dbias=None, T=1, K=8, dtype=0):
        return lib.kp_layer_norm_backward(dy, lddy, x, ldx, weight, mean, rstd, dx, lddx, dweight, dbias, T, K, dtype,
                                          None, 0, None)

    assert back(T=-1) == EINVAL and back(K=20000, ldx=20000, lddy=20000, lddx=20000) == ESHAPE and back(dtype=-1) == EINVAL
    assert back(dweight=None) == EINVAL and back(dbias=ODD) == EALIGN
    assert back(dy=None) == EINVAL and back(lddy=4) == EINVAL and back(x=ODD) == EALIGN and back(dx=None) == EINVAL
    assert back(rstd=None) == EINVAL and back(mean=ODD) == EALIGN and back(weight=None) == EINVAL


def test_norm_refusals(library):  # noqa: F811
    x, w, f = on(5, 24), on(24), on(5, dtype=torch.float32)
    binding.layer_norm(x, w, on(24), save=True)
    binding.layer_norm_backward(on(5, 24), x, w, None, f, bias=True)
    assert [c for c in library.calls if not c.endswith("workspace")] == ["kp_layer_norm", "kp_layer_norm_backward"]
    library.calls.clear()
    for call, error in ((lambda: binding.layer_norm(on(5, 24, dtype=torch.int32), w), TypeError),
                        (lambda: binding.layer_norm(x, on(23)), ValueError),
                        (lambda: binding.layer_norm(x, on(24, dtype=torch.float32)), TypeError),
                        (lambda: binding.layer_norm(x, w, on(24, 1)), ValueError),
                        (lambda: binding.layer_norm(x, w, y=on(5, 23)), ValueError),
                        (lambda: binding.layer_norm(on(24, 5).t(), w), ValueError),
                        (lambda: binding.layer_norm(x, w, stream=StreamOf(1)), ValueError),
                        (lambda: binding.layer_norm_backward(on(5, 23), x, w, f, f), ValueError),
                        (lambda: binding.layer_norm_backward(on(5, 24, dtype=torch.float16), x, w, f, f), TypeError),
                        (lambda: binding.layer_norm_backward(on(5, 24), x, w, on(5), f), TypeError),
                        (lambda: binding.layer_norm_backward(on(5, 24), x, w, f, on(4, dtype=torch.float32)), ValueError)):
        with pytest.raises(error):
            call()
    assert library.calls == []


def test_grouped_argument_errors(lib):
    def gemm(x=P, ldx=16, W=P, ldw=16, sw=128, y=P, ldy=8, offsets=P, R=1, E=3, N=8, K=16, dtype=0):
        return lib.kp_grouped_gemm(x, ldx, W, ldw, sw, y, ldy, offsets, R, E, N, K, dtype, None)

    assert gemm(R=0) == OK
    assert gemm(R=-1) == EINVAL and gemm(E=0) == EINVAL and gemm(N=0) == EINVAL and gemm(K=0) == EINVAL
    assert gemm(E=1025) == ESHAPE and gemm(K=12) == ESHAPE and gemm(dtype=2) == EINVAL
    big = 2 ** 30 + 8
    assert gemm(R=big) == ESHAPE and gemm(N=big, ldy=big) == ESHAPE
    assert gemm(K=big, ldx=big, ldw=big, sw=8 * big) == ESHAPE
    assert gemm(x=None) == EINVAL and gemm(x=P8) == EALIGN and gemm(ldx=20) == ESHAPE and gemm(ldx=8) == EINVAL
    assert gemm(W=None) == EINVAL and gemm(W=P8) == EALIGN and gemm(ldw=20) == ESHAPE
    assert gemm(sw=120) == ESHAPE and gemm(sw=132) == ESHAPE
    assert gemm(y=ODD) == EALIGN and gemm(ldy=7) == EINVAL and gemm(offsets=ODD) == EALIGN and gemm(offsets=None) == EINVAL

    def gemm_back(dy=P, lddy=8, x=P, ldx=16, W=P, ldw=16, sw=128, dx=P, lddx=16, dW=P, offsets=P, R=1, E=3, N=8, K=16,
                  dtype=0):
        return lib.kp_grouped_gemm_backward(dy, lddy, x, ldx, W, ldw, sw, dx, lddx, dW, offsets, R, E, N, K, dtype, None)

    assert gemm_back(R=-1) == EINVAL and gemm_back(K=12) == ESHAPE
    assert gemm_back(dW=None) == EINVAL and gemm_back(dW=P8) == EALIGN
    assert gemm_back(dy=P8) == EALIGN and gemm_back(lddy=12) == ESHAPE and gemm_back(lddy=4) == EINVAL
    assert gemm_back(dx=None) == EINVAL and gemm_back(lddx=8) == EINVAL and gemm_back(offsets=None) == EINVAL

    def gated(x=P, ldx=16, Wg=P, ldg=16, sg=128, Wu=P, ldu=16, su=128, h=P, ldh=8, g=None, u=None, offsets=P, R=1, E=3,
              F=8, K=16, act=0, dtype=0):
        return lib.kp_grouped_gated_ffn(x, ldx, Wg, ldg, sg, Wu, ldu, su, h, ldh, g, u, offsets, R, E, F, K, act, dtype,
                                        None)

    assert gated(R=0) == OK
    assert gated(act=3) == EINVAL and gated(F=0) == EINVAL and gated(Wu=None) == EINVAL and gated(su=64) == ESHAPE
    assert gated(h=None) == EINVAL and gated(g=P) == EINVAL and gated(g=P, u=P8) == EALIGN

    def gated_back(dh=P, lddh=8, x=P, ldx=16, Wg=P, ldg=16, sg=128, Wu=P, ldu=16, su=128, g=P, u=P, dx=P, lddx=16,
                   dWg=P, dWu=P, offsets=P, R=1, E=3, F=8, K=16, act=0, dtype=0):
        return lib.kp_grouped_gated_ffn_backward(dh, lddh, x, ldx, Wg, ldg, sg, Wu, ldu, su, g, u, dx, lddx, dWg, dWu,
                                                 offsets, R, E, F, K, act, dtype, None, 0, None)

    assert gated_back(act=-1) == EINVAL and gated_back(R=-1) == EINVAL
    assert gated_back(dWg=None) == EINVAL and gated_back(dWu=P8) == EALIGN
    assert gated_back(dh=ODD) == EALIGN and gated_back(lddh=4) == EINVAL and gated_back(g=None) == EINVAL
    assert gated_back(u=P8) == EALIGN and gated_back(dx=None) == EINVAL and gated_back(offsets=ODD) == EALIGN


def on(*shape, dtype=torch.bfloat16):
    return OnDevice(torch.zeros(shape, dtype=dtype))


def route_of(T=6, k=2, E=4):
    """A routing as the binding sees it; its parts are not read here."""
    r = binding.MoeRoute.__new__(binding.MoeRoute)
    r.tokens, r.top_k, r.experts, r.score, r._index = T, k, E, "softmax", 0
    r.device = torch.device("cuda", 0)
    r._buf, r._ptr = torch.zeros(4 * T * k + E + 1, dtype=torch.int32), 256
    return r


def grouped_operands(R=5, E=3, N=16, K=24):
    return {"x": on(R, K), "W": on(E, N, K), "offsets": on(E + 1, dtype=torch.int32)}


def test_calls_reach_the_library(library):  # noqa: F811
    p, r = grouped_operands(), route_of()
    binding.moe_route(on(6, 4), 2)
    binding.moe_route_backward(on(6, 2, dtype=torch.float32), on(6, 4), r)
    binding.moe_dispatch(on(6, 8), r)
    binding.moe_combine(on(12, 8), r)
    binding.moe_dispatch_backward(on(12, 8), r)
    binding.moe_combine_backward(on(6, 8), on(12, 8), r)
    binding.grouped_gemm(**p)
    binding.grouped_gemm_backward(on(5, 16), **p)
    _, g, u = binding.grouped_gated_ffn(p["x"], p["W"], p["W"], p["offsets"], save=True)
    f = on(5, 16, dtype=torch.float32)
    binding.grouped_gated_ffn_backward(on(5, 16), p["x"], p["W"], p["W"], p["offsets"], f, f)
    made = [c for c in library.calls if not c.endswith("workspace")]
    assert made == ["kp_moe_route", "kp_moe_route_backward", "kp_moe_dispatch", "kp_moe_combine", "kp_moe_combine",
                    "kp_moe_combine_backward", "kp_grouped_gemm", "kp_grouped_gemm_backward", "kp_grouped_gated_ffn",
                    "kp_grouped_gated_ffn_backward"]


def test_route_refusals(library):  # noqa: F811
    logits = on(6, 4)
    for call, error in ((lambda: binding.moe_route(logits, 5), ValueError),
                        (lambda: binding.moe_route(logits, 0), ValueError),
                        (lambda: binding.moe_route(logits, 2, score="tanh"), ValueError),
                        (lambda: binding.moe_route(on(6, 4, dtype=torch.float64), 2), TypeError),
                        (lambda: binding.moe_route(on(6), 2), ValueError),
                        (lambda: binding.moe_route(torch.zeros(6, 4), 2), ValueError),      # on the CPU
                        (lambda: binding.moe_route([[1.0]], 1), TypeError),
                        (lambda: binding.moe_route(logits, 2, score="sigmoid", bias=on(4)), TypeError),
                        (lambda: binding.moe_route(logits, 2, score="sigmoid", bias=on(5, dtype=torch.float32)), ValueError),
                        (lambda: binding.moe_route(logits, 2, stream=StreamOf(1)), ValueError)):
        with pytest.raises(error):
            call()
    r = route_of()
    dw = on(6, 2, dtype=torch.float32)
    for call, error in ((lambda: binding.moe_route_backward(dw, on(6, 5), r), ValueError),
                        (lambda: binding.moe_route_backward(on(6, 2), logits, r), TypeError),
                        (lambda: binding.moe_route_backward(on(2, 6, dtype=torch.float32), logits, r), ValueError),
                        (lambda: binding.moe_route_backward(dw, logits, None), TypeError)):
        with pytest.raises(error):
            call()
    assert library.calls == []


def test_rows_refusals(library):  # noqa: F811
    r = route_of()
    other = route_of()
    other._index = 1
    for call, error in ((lambda: binding.moe_dispatch(on(7, 8), r), ValueError),
                        (lambda: binding.moe_dispatch(on(6, 8, dtype=torch.float32), r), TypeError),
                        (lambda: binding.moe_dispatch(on(6, 8), "r"), TypeError),
                        (lambda: binding.moe_dispatch(on(6, 8), other), ValueError),
                        (lambda: binding.moe_dispatch(on(6, 8), r, rows=on(11, 8)), ValueError),
                        (lambda: binding.moe_dispatch(on(6, 8), r, rows=on(12, 8, dtype=torch.float16)), TypeError),
                        (lambda: binding.moe_dispatch(on(6, 16)[:, ::2], r), ValueError),
                        (lambda: binding.moe_combine(on(11, 8), r), ValueError),
                        (lambda: binding.moe_combine(on(12, 8), r, y=on(6, 9)), ValueError),
                        (lambda: binding.moe_combine_backward(on(6, 8), on(12, 9), r), ValueError),
                        (lambda: binding.moe_combine_backward(on(6, 8), on(12, 8, dtype=torch.float16), r), TypeError),
                        (lambda: binding.moe_combine(on(12, 8), r, stream=StreamOf(1)), ValueError)):
        with pytest.raises(error):
            call()
    assert library.calls == []


def test_grouped_refusals(library):  # noqa: F811
    p = grouped_operands()

    def gemm(**kw):
        return lambda: binding.grouped_gemm(**{**p, **kw})

    def gated(**kw):
        q = {"x": p["x"], "Wg": p["W"], "Wu": p["W"], "offsets": p["offsets"], **kw}
        return lambda: binding.grouped_gated_ffn(**q)

    for call, error in ((gemm(x=on(5, 24, dtype=torch.float32)), TypeError), (gemm(x=on(5, 16)), ValueError),
                        (gemm(W=on(3, 16, 24, dtype=torch.float16)), TypeError), (gemm(W=on(16, 24)), ValueError),
                        (gemm(W=on(3, 24, 16).transpose(1, 2)), ValueError),
                        (gemm(offsets=on(3, dtype=torch.int32)), ValueError),
                        (gemm(offsets=on(4, dtype=torch.int64)), TypeError),
                        (gemm(offsets=on(8, dtype=torch.int32)[::2]), ValueError),
                        (gemm(offsets=[0, 1, 2, 5]), TypeError),
                        (gemm(y=on(5, 17)), ValueError), (gemm(stream=StreamOf(1)), ValueError),
                        (gated(Wu=on(3, 17, 24)), ValueError), (gated(act="relu"), ValueError),
                        (gated(h=on(5, 16, dtype=torch.float16)), TypeError),
                        (lambda: binding.grouped_gemm_backward(on(5, 15), **p), ValueError),
                        (lambda: binding.grouped_gemm_backward(on(5, 16, dtype=torch.float16), **p), TypeError)):
        with pytest.raises(error):
            call()
    f, h = on(5, 16, dtype=torch.float32), on(5, 16)
    for g, u, dh, error in ((h, f, h, TypeError), (f, h, h, TypeError), (f, on(5, 20, dtype=torch.float32)[:, :16], h, ValueError),
                            (f, f, on(5, 17), ValueError)):
        with pytest.raises(error):
            binding.grouped_gated_ffn_backward(dh, p["x"], p["W"], p["W"], p["offsets"], g, u)
    assert library.calls == []


def test_sizes_past_32_bits_are_refused(library):  # noqa: F811
    # the entry points take sizes as int; none may arrive there without its upper bits
    def huge(*shape, dtype=torch.bfloat16):
        return OnDevice(torch.empty(shape, dtype=dtype, device="meta"))

    n = 2 ** 32 + 3
    p = grouped_operands()
    off = p["offsets"]
    r = route_of()
    r.tokens, r.top_k = 3, 1
    for call in (lambda: binding.layer_norm(huge(n, 8), on(8)), lambda: binding.moe_route(huge(n, 8), 2),
                 lambda: binding.moe_dispatch(huge(3, n), r), lambda: binding.moe_combine(huge(3, n), r),
                 lambda: binding.grouped_gemm(huge(n, 24), p["W"], off),
                 lambda: binding.grouped_gemm(p["x"], huge(3, n, 24), off),
                 lambda: binding.grouped_gemm(huge(5, n + 5), huge(3, 16, n + 5), off)):
        with pytest.raises(ValueError, match="2\\^31"):
            call()
    assert library.calls == []
    plain = torch.empty((3, n), dtype=torch.bfloat16, device="meta")   # what the quick checks take
    with pytest.raises(ValueError, match="2\\^31"):
        binding._half_rows(plain, "x", 3, plain.get_device())
    x, W = plain[:, :24].contiguous(), torch.empty((3, n, 24), dtype=torch.bfloat16, device="meta")
    with pytest.raises(ValueError, match="2\\^31"):
        binding._grouped_operands(x, W, "W", torch.zeros(4, dtype=torch.int32, device="meta"), x.get_device())
