"""Host side of the feed-forward operators: argument checks that need no device,
storage sizes, and the binding's refusals."""
import ctypes

import pytest
import torch

from decode_projection_gemms_gb300 import binding
from decode_projection_gemms_gb300.build import build


@pytest.fixture(scope="module")
def lib():
    build()
    return binding.load()


P, ODD = ctypes.c_void_p(256), ctypes.c_void_p(257)


@pytest.mark.parametrize("rows,cols,codes,scales", [(0, 1, 0, 0), (1, 1, 16, 512), (128, 128, 128 * 64, 512),
                                                    (129, 129, 129 * 80, 2 * 2 * 512), (4096, 7168, 4096 * 3584, 32 * 56 * 512)])
def test_mx4_sizes(lib, rows, cols, codes, scales):
    assert binding.Mx4Tensor.sizes(rows, cols) == (codes, scales)


def test_mx4_argument_errors(lib):
    a, b = ctypes.c_size_t(), ctypes.c_size_t()
    assert lib.kp_mx4_bytes(-1, 4, a, b) == binding.KP_EINVAL
    assert lib.kp_mx4_bytes(4, 0, a, b) == binding.KP_EINVAL
    q = lib.kp_mx4_quantize
    assert q(P, 8, 0, 8, 0, P, P, None) == binding.KP_OK                      # no rows: nothing to do
    assert q(P, 8, -1, 8, 0, P, P, None) == binding.KP_EINVAL
    assert q(P, 8, 1, 8, 3, P, P, None) == binding.KP_EINVAL                  # element type
    assert q(None, 8, 1, 8, 0, P, P, None) == binding.KP_EINVAL
    assert q(P, 7, 1, 8, 0, P, P, None) == binding.KP_EINVAL                  # stride below the columns
    assert q(ODD, 8, 1, 8, 0, P, P, None) == binding.KP_EALIGN
    assert q(ctypes.c_void_p(258), 8, 1, 8, binding.DTYPE_FP32, P, P, None) == binding.KP_EALIGN
    assert q(P, 8, 1, 8, 0, ctypes.c_void_p(264), P, None) == binding.KP_EALIGN
    assert q(P, 2 ** 31 - 1, 2 ** 31 - 1, 2 ** 30, 0, P, P, None) == binding.KP_ESHAPE
    d = lib.kp_mx4_dequantize
    assert d(P, P, 0, 8, P, 8, 0, None) == binding.KP_OK
    assert d(P, None, 1, 8, P, 8, 0, None) == binding.KP_EINVAL
    assert d(P, P, 1, 8, None, 8, 0, None) == binding.KP_EINVAL
    assert d(P, P, 1, 8, P, 4, 0, None) == binding.KP_EINVAL
    g = lib.kp_mx4_gemm
    assert g(P, 8, None, None, P, P, P, 8, 0, 8, 8, 0, None, 0, None) == binding.KP_OK
    assert g(P, 8, None, None, P, P, P, 8, 1, 0, 8, 0, None, 0, None) == binding.KP_EINVAL
    assert g(P, 8, None, None, P, P, P, 8, 1, 8, 8, binding.DTYPE_FP32, None, 0, None) == binding.KP_EINVAL
    assert g(P, 8, P, P, P, P, P, 8, 1, 8, 8, 0, None, 0, None) == binding.KP_EINVAL     # both forms of x
    assert g(None, 0, None, None, P, P, P, 8, 1, 8, 8, 0, None, 0, None) == binding.KP_EINVAL
    assert g(None, 0, P, None, P, P, P, 8, 1, 8, 8, 0, None, 0, None) == binding.KP_EINVAL
    assert g(P, 8, None, None, ctypes.c_void_p(8), P, P, 8, 1, 8, 8, 0, None, 0, None) == binding.KP_EALIGN
    assert g(P, 8, None, None, P, P, P, 7, 1, 8, 8, 0, None, 0, None) == binding.KP_EINVAL
    m = lib.kp_mx4_gated_ffn
    assert m(P, 8, None, None, P, P, P, P, P, 8, 1, 8, 8, 7, 0, None, 0, None) == binding.KP_EINVAL   # activation
    assert m(P, 8, None, None, P, P, None, P, P, 8, 1, 8, 8, 0, 0, None, 0, None) == binding.KP_EINVAL


def test_gated_argument_errors(lib):
    f = lib.kp_gated_ffn

    def call(x=P, ldx=16, Wg=P, ldg=16, Wu=P, ldu=16, h=P, ldh=8, g=None, u=None, T=1, F=8, K=16, act=0, dtype=0):
        return f(x, ldx, Wg, ldg, Wu, ldu, h, ldh, g, u, T, F, K, act, dtype, None, 0, None)

    assert call(T=0) == binding.KP_OK
    assert call(T=-1) == binding.KP_EINVAL
    assert call(act=3) == binding.KP_EINVAL
    assert call(dtype=2) == binding.KP_EINVAL
    assert call(K=12) == binding.KP_ESHAPE
    assert call(x=None) == binding.KP_EINVAL
    assert call(Wu=None) == binding.KP_EINVAL
    assert call(h=None) == binding.KP_EINVAL
    assert call(ldx=12) == binding.KP_EINVAL
    assert call(ldx=20) == binding.KP_ESHAPE
    assert call(Wg=ctypes.c_void_p(264)) == binding.KP_EALIGN
    assert call(ldh=7) == binding.KP_EINVAL
    assert call(g=P) == binding.KP_EINVAL
    assert call(g=P, u=ctypes.c_void_p(264)) == binding.KP_EALIGN
    b = lib.kp_gated_ffn_backward

    def back(dh=P, lddh=8, x=P, ldx=16, Wg=P, ldg=16, Wu=P, ldu=16, g=P, u=P, dx=P, dWg=P, dWu=P, T=1, F=8, K=16,
             act=0, dtype=0):
        return b(dh, lddh, x, ldx, Wg, ldg, Wu, ldu, g, u, dx, dWg, dWu, T, F, K, act, dtype, None, 0, None)

    assert back(T=-1) == binding.KP_EINVAL
    assert back(act=-1) == binding.KP_EINVAL
    assert back(K=20) == binding.KP_ESHAPE
    assert back(dWu=None) == binding.KP_EINVAL
    assert back(dWg=ctypes.c_void_p(264)) == binding.KP_EALIGN
    assert back(g=None) == binding.KP_EINVAL
    assert back(dx=ctypes.c_void_p(264)) == binding.KP_EALIGN
    assert back(lddh=4) == binding.KP_EINVAL
    assert b"row stride" in lib.kp_last_error()
    w = ctypes.c_size_t()
    assert lib.kp_ffn_workspace(0, -1, 1, 1, w) == binding.KP_EINVAL


def test_binding_refuses_before_the_library():
    x = torch.zeros((2, 64), dtype=torch.bfloat16)
    for call in (lambda: binding.mx4_quantize(x), lambda: binding.gated_ffn(x, x, x),
                 lambda: binding.mx4_gemm(x, x), lambda: binding.gated_ffn_backward(x, x, x, x, x, x)):
        with pytest.raises(ValueError):      # not on a CUDA device
            call()
    with pytest.raises(TypeError):
        binding.mx4_quantize([1.0])


def test_mx4_tensor_from_stored_parts(lib):
    q = binding.Mx4Tensor(torch.zeros((3, 32), dtype=torch.uint8), torch.zeros(512, dtype=torch.uint8), 3, 40)
    assert q.shape == (3, 40) and q.nbytes == 96 + 512 and q.codes.shape == (3, 32) and q.scales.numel() == 512
    with pytest.raises(ValueError):
        binding.Mx4Tensor(torch.zeros((3, 16), dtype=torch.uint8), torch.zeros(512, dtype=torch.uint8), 3, 40)
    with pytest.raises(TypeError):
        binding.Mx4Tensor(torch.zeros((3, 32)), torch.zeros(512, dtype=torch.uint8), 3, 40)
