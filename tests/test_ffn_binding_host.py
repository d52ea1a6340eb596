"""What the binding of the feed-forward operators checks before it calls the
library: no device, the library replaced by one that records its calls."""
import pytest
import torch

from decode_projection_gemms_gb300 import binding


class OnDevice(torch.Tensor):
    """A CPU tensor that says it is on CUDA device 0."""

    @staticmethod
    def __new__(cls, t):
        return t.as_subclass(cls)

    def get_device(self):
        return 0

    @property
    def device(self):
        return torch.device("cuda", 0)


class Recorder:
    """Every entry point succeeds and is noted; workspaces are empty."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append(name)
            return binding.KP_OK
        return call

    def kp_ffn_workspace(self, op, M, N, K, out):
        return binding.KP_OK


@pytest.fixture
def library(monkeypatch):
    lib = Recorder()
    monkeypatch.setattr(binding, "load", lambda path=None: lib)
    monkeypatch.setattr(binding, "_current_device", lambda: 0)
    monkeypatch.setattr(binding, "_raw_stream", lambda index: 0)
    monkeypatch.setattr(binding, "_device", lambda index: torch.device("cpu"))
    monkeypatch.setattr(binding, "_FFN_WORK", {})
    return lib


def backward_operands(T=5, F=16, K=24):
    on = OnDevice
    h = lambda *shape: on(torch.zeros(shape, dtype=torch.bfloat16))  # noqa: E731
    f = lambda: on(torch.zeros((T, F)))  # noqa: E731
    return {"dh": h(T, F), "x": h(T, K), "Wg": h(F, K), "Wu": h(F, K), "g": f(), "u": f()}


def test_backward_takes_float32_sums(library):
    binding.gated_ffn_backward(**backward_operands())
    assert library.calls == ["kp_gated_ffn_backward"]


@pytest.mark.parametrize("name", ["g", "u"])
def test_backward_refuses_dh_in_place_of_a_sum(library, name):
    """The library reads g and u as contiguous float32: dh itself, 16 bits an
    element, would be read past its end."""
    p = backward_operands()
    p[name] = p["dh"]
    with pytest.raises(TypeError):
        binding.gated_ffn_backward(**p)
    assert library.calls == []


@pytest.mark.parametrize("name", ["g", "u"])
def test_backward_refuses_strided_sums(library, name):
    p = backward_operands()
    p[name] = OnDevice(torch.zeros((5, 20))[:, :16])
    with pytest.raises(ValueError):
        binding.gated_ffn_backward(**p)
    assert library.calls == []


def test_backward_without_tokens_reads_no_sums(library):
    """With no rows there is nothing to read, and the type of g and u is free."""
    p = backward_operands(T=0)
    p["g"] = p["u"] = p["dh"]
    binding.gated_ffn_backward(**p)
    assert library.calls == ["kp_gated_ffn_backward"]


class StreamOf:
    cuda_stream = 7

    def __init__(self, index):
        self.device = torch.device("cuda", index)


@pytest.mark.parametrize("op", ["mx4_quantize", "mx4_dequantize", "mx4_gemm", "mx4_gated_ffn", "gated_ffn",
                                "gated_ffn_backward"])
def test_refuses_a_stream_of_another_device(library, op):
    """The work would otherwise run on the operands' device, on a stream that nobody
    named."""
    p = backward_operands()
    q = binding.Mx4Tensor.__new__(binding.Mx4Tensor)
    q._buf, q._scales, q._index, q.shape, q.device = p["x"], None, 0, (16, 24), torch.device("cuda", 0)
    q.code_ptr = q.scale_ptr = 256
    args = {"mx4_quantize": (p["x"],), "mx4_dequantize": (q,), "mx4_gemm": (p["x"], q),
            "mx4_gated_ffn": (p["x"], q, q), "gated_ffn": (p["x"], p["Wg"], p["Wu"]),
            "gated_ffn_backward": tuple(p[k] for k in ("dh", "x", "Wg", "Wu", "g", "u"))}[op]
    with pytest.raises(ValueError, match="stream"):
        getattr(binding, op)(*args, stream=StreamOf(1))
    assert library.calls == []
