"""ctypes binding of ``libkdaproj.so`` (argument marshalling only).

Every computation runs in the library's CUDA kernels; this module checks
tensor types and shapes, passes ``data_ptr()`` / stream handles through the C
ABI declared in ``include/kdaproj.h`` and turns non-zero status codes into
``KdaProjError``. There is no CPU or PyTorch fallback: if the library is not
built, importing the functions below raises.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
import threading

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_build", "libkdaproj.so")
TABLE_PATH = os.path.join(_HERE, "tune", "gb300_table.txt")

# enum kp_status
(KP_OK, KP_EINVAL, KP_EALIGN, KP_ESHAPE, KP_ENOPLAN, KP_ECUDA, KP_ETOOBIG, KP_ENODEV, KP_ECONFIG,
 KP_EIO, KP_EDEVICE) = (0, -1, -2, -3, -4, -5, -6, -7, -8, -9, -10)
STATUS_NAMES = {0: "KP_OK", -1: "KP_EINVAL", -2: "KP_EALIGN", -3: "KP_ESHAPE", -4: "KP_ENOPLAN",
                -5: "KP_ECUDA", -6: "KP_ETOOBIG", -7: "KP_ENODEV", -8: "KP_ECONFIG", -9: "KP_EIO",
                -10: "KP_EDEVICE"}
# enum kp_kind
KIND_AUTO, KIND_CC, KIND_TC05, KIND_SMALLK = 0, 1, 2, 3
KIND_NAMES = {0: "auto", 1: "cc", 2: "tc05", 3: "smallk"}
FLAG_PDL = 1
FLAG_FUSE_FB = 2
DTYPE_BF16, DTYPE_FP16, DTYPE_FP32 = 0, 1, 2
# enum kp_act, enum kp_ffn_op
ACTIVATIONS = {"silu": 0, "gelu": 1, "gelu_tanh": 2}
FFN_MX4_GEMM, FFN_MX4_GATED, FFN_GATED, FFN_GATED_BACKWARD = 0, 1, 2, 3
BRANCH_QKVG, BRANCH_FAB, BRANCH_FB = 0, 1, 2

# exported symbols (must match include/kdaproj.h)
EXPORTS = (
    "skinny_gemm", "kp_select_config", "kp_table_load", "kp_table_clear", "kp_table_size",
    "kda_proj_plan", "kda_proj_set_overlap", "kda_proj_get_config", "kda_proj_set_config",
    "kda_proj_overlap_at", "kda_proj_run", "kda_proj_destroy", "kp_last_error", "kp_version",
    "kp_device_error", "kp_scratch_bytes", "skinny_gemm_noalloc", "skinny_gemm_ex",
    "kp_selftest_timeout", "kp_pdl_consumer_checksum",
    "kp_ffn_workspace", "kp_mx4_bytes", "kp_mx4_quantize", "kp_mx4_dequantize", "kp_mx4_gemm",
    "kp_mx4_gated_ffn", "kp_gated_ffn", "kp_gated_ffn_backward",
)
DEV_SELFTEST = 5   # device error code of kp_selftest_timeout


class KdaProjError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"{STATUS_NAMES.get(code, code)}: {msg}")
        self.code = code


class KpCfg(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int32), ("split_k", ctypes.c_int32), ("block", ctypes.c_int32),
                ("rows", ctypes.c_int32), ("k_unroll", ctypes.c_int32), ("producers", ctypes.c_int32),
                ("stages", ctypes.c_int32), ("flags", ctypes.c_int32)]

    def as_dict(self) -> dict:
        d = {f: int(getattr(self, f)) for f, _ in self._fields_}
        d["kind"] = KIND_NAMES.get(d["kind"], d["kind"])
        return d

    @classmethod
    def make(cls, kind, split_k=1, block=256, rows=4, k_unroll=2, producers=1, stages=0,
             flags=FLAG_PDL):
        if isinstance(kind, str):
            kind = {v: k for k, v in KIND_NAMES.items()}[kind]
        return cls(int(kind), int(split_k), int(block), int(rows), int(k_unroll), int(producers),
                   int(stages), int(flags))


_lock = threading.Lock()
_lib = None


def load(path: str | None = None):
    """Load the library (once) and declare its signatures. Raises if absent."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        p = path or LIB_PATH
        if not os.path.exists(p):
            raise ImportError(f"{p} is missing: build it with decode_projection_gemms_gb300.build.build()")
        lib = ctypes.CDLL(p)
        vp, ci, cfgp = ctypes.c_void_p, ctypes.c_int, ctypes.POINTER(KpCfg)
        i64, sz = ctypes.c_int64, ctypes.c_size_t
        sig = {
            "skinny_gemm": [vp, vp, vp, ci, ci, ci, cfgp, vp],
            "kp_select_config": [ci, ci, ci, ci, cfgp],
            "kp_table_load": [ctypes.c_char_p],
            "kp_table_clear": [],
            "kp_table_size": [],
            "kda_proj_plan": [ci, ci, ci, ci, ci, ctypes.POINTER(vp)],
            "kda_proj_set_overlap": [vp, ci],
            "kda_proj_get_config": [vp, ci, ci, cfgp],
            "kda_proj_set_config": [vp, ci, ci, cfgp],
            "kda_proj_overlap_at": [vp, ci],
            "kda_proj_run": [vp, vp, vp, vp, vp, vp, vp, ci, vp, vp, ctypes.POINTER(vp)],
            "kda_proj_destroy": [vp],
            "kp_last_error": [],
            "kp_version": [],
            "kp_device_error": [ctypes.POINTER(ci)],
            "kp_scratch_bytes": [ci, ci, ci, cfgp, ci, ctypes.POINTER(ctypes.c_size_t)],
            "skinny_gemm_noalloc": [vp, vp, vp, ci, ci, ci, cfgp, vp],
            "skinny_gemm_ex": [vp, vp, vp, vp, ci, ci, ci, ci, cfgp, vp],
            "kp_selftest_timeout": [ci, vp],
            "kp_pdl_consumer_checksum": [vp, ctypes.c_int64, vp, ci, vp],
            "kp_ffn_workspace": [ci, ci, ci, ci, ctypes.POINTER(ctypes.c_size_t)],
            "kp_mx4_bytes": [ci, ci, ctypes.POINTER(ctypes.c_size_t), ctypes.POINTER(ctypes.c_size_t)],
            "kp_mx4_quantize": [vp, i64, ci, ci, ci, vp, vp, vp],
            "kp_mx4_dequantize": [vp, vp, ci, ci, vp, i64, ci, vp],
            "kp_mx4_gemm": [vp, i64, vp, vp, vp, vp, vp, i64, ci, ci, ci, ci, vp, sz, vp],
            "kp_mx4_gated_ffn": [vp, i64, vp, vp, vp, vp, vp, vp, vp, i64, ci, ci, ci, ci, ci, vp, sz, vp],
            "kp_gated_ffn": [vp, i64, vp, i64, vp, i64, vp, i64, vp, vp, ci, ci, ci, ci, ci, vp, sz, vp],
            "kp_gated_ffn_backward": [vp, i64, vp, i64, vp, i64, vp, i64, vp, vp, vp, vp, vp, ci, ci, ci, ci, ci,
                                      vp, sz, vp],
        }
        for name, args in sig.items():
            fn = getattr(lib, name)
            fn.argtypes = args
            fn.restype = ctypes.c_char_p if name == "kp_last_error" else ci
        rc = lib.kp_table_load(TABLE_PATH.encode()) if os.path.exists(TABLE_PATH) else KP_OK
        _lib = lib   # seen without the lock: only once the table is in
        if rc:
            raise KdaProjError(rc, lib.kp_last_error().decode())
        return _lib


def _check(rc: int):
    if rc != KP_OK:
        raise KdaProjError(rc, load().kp_last_error().decode())


def last_error() -> str:
    return load().kp_last_error().decode()


def _bf16_2d(t: torch.Tensor, name: str):
    # the common case in a few cheap checks; the rest only to name the problem
    if type(t) is torch.Tensor and t.dtype is torch.bfloat16 and t.is_cuda and t.dim() == 2 \
            and t.is_contiguous():
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != torch.bfloat16:
        raise TypeError(f"{name} must be bfloat16, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dim() != 2 or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous 2-D tensor")


def _stream_handle(stream) -> int:
    if stream is None:
        stream = torch.cuda.current_stream()
    return int(stream.cuda_stream)


def table_load(path: str = TABLE_PATH):
    _check(load().kp_table_load(str(path).encode()))


def table_clear():
    _check(load().kp_table_clear())


def table_size() -> int:
    return int(load().kp_table_size())


def select_config(M: int, N: int, K: int, num_sms: int = 0) -> KpCfg:
    c = KpCfg()
    _check(load().kp_select_config(M, N, K, num_sms, ctypes.byref(c)))
    return c


def scratch_bytes(M: int, N: int, K: int, cfg: KpCfg, num_sms: int) -> int:
    b = ctypes.c_size_t()
    _check(load().kp_scratch_bytes(M, N, K, ctypes.byref(cfg), num_sms, ctypes.byref(b)))
    return int(b.value)


def selftest_timeout(timeout_us: int = 2000, stream=None):
    """Launch the failure-path self-test (a wait that must run out)."""
    _check(load().kp_selftest_timeout(int(timeout_us), _stream_handle(stream)))


def pdl_consumer_checksum(t: torch.Tensor, out: torch.Tensor, pdl: bool = True, stream=None):
    """Launch the dependent checksum kernel on ``t`` (bf16/fp16, contiguous)
    adding into ``out`` (a CUDA int64 tensor of one element); ``pdl`` launches
    it with programmatic stream serialisation."""
    if t.dtype not in _DTYPES or not t.is_contiguous() or not t.is_cuda:
        raise TypeError("t must be a contiguous CUDA bf16/fp16 tensor")
    if out.dtype != torch.int64 or out.numel() != 1 or not out.is_cuda:
        raise TypeError("out must be a one-element CUDA int64 tensor")
    _check(load().kp_pdl_consumer_checksum(t.data_ptr(), t.numel(), out.data_ptr(), int(bool(pdl)),
                                           _stream_handle(stream)))


def device_error() -> int:
    """Read and clear the current device's error word (0: no kernel wait ran
    out). Does not wait for the device."""
    v = ctypes.c_int()
    _check(load().kp_device_error(ctypes.byref(v)))
    return int(v.value)


def check_device(stream=None):
    """Wait for ``stream`` (default: the current stream), then raise
    ``KdaProjError(KP_EDEVICE)`` if a kernel wait ran out meanwhile (the
    outputs of that work are undefined). Reading clears the code."""
    (stream or torch.cuda.current_stream()).synchronize()
    code = device_error()
    if code:
        raise KdaProjError(KP_EDEVICE, f"a kernel wait ran out (device error code {code}); "
                                       "the outputs of the work just run are undefined")


def skinny_gemm(x: torch.Tensor, W: torch.Tensor, y: torch.Tensor | None = None,
                cfg: KpCfg | None = None, stream=None) -> torch.Tensor:
    """``y = bf16(x @ W.T)`` with fp32 accumulation, in the library's kernels."""
    _bf16_2d(x, "x")
    _bf16_2d(W, "W")
    M, K = x.shape
    N = W.shape[0]
    if W.shape[1] != K:
        raise ValueError(f"W has K={W.shape[1]}, x has K={K}")
    if y is None:
        y = torch.empty((M, N), dtype=torch.bfloat16, device=x.device)
    _bf16_2d(y, "y")
    if tuple(y.shape) != (M, N):
        raise ValueError(f"y must be {(M, N)}")
    _check(load().skinny_gemm(x.data_ptr(), W.data_ptr(), y.data_ptr(), M, N, K,
                              ctypes.byref(cfg) if cfg is not None else None,
                              _stream_handle(stream)))
    return y


_DTYPES = {torch.bfloat16: DTYPE_BF16, torch.float16: DTYPE_FP16}


def _half_2d(t: torch.Tensor, name: str, dtype=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype not in _DTYPES or (dtype is not None and t.dtype != dtype):
        raise TypeError(f"{name} must be {dtype or 'bfloat16 or float16'}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dim() != 2 or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous 2-D tensor")


def skinny_gemm_ex(x: torch.Tensor, W: torch.Tensor, residual: torch.Tensor | None = None,
                   y: torch.Tensor | None = None, cfg: KpCfg | None = None,
                   stream=None) -> torch.Tensor:
    """``y = round(x @ W.T + residual)`` with fp32 accumulation; x, W, residual
    and y all bfloat16 or all float16 (the element type is x's). ``residual``
    may be ``y`` itself."""
    _half_2d(x, "x")
    _half_2d(W, "W", x.dtype)
    M, K = x.shape
    N = W.shape[0]
    if W.shape[1] != K:
        raise ValueError(f"W has K={W.shape[1]}, x has K={K}")
    if y is None:
        y = torch.empty((M, N), dtype=x.dtype, device=x.device)
    _half_2d(y, "y", x.dtype)
    if tuple(y.shape) != (M, N):
        raise ValueError(f"y must be {(M, N)}")
    if residual is not None:
        _half_2d(residual, "residual", x.dtype)
        if tuple(residual.shape) != (M, N):
            raise ValueError(f"residual must be {(M, N)}")
    _check(load().skinny_gemm_ex(x.data_ptr(), W.data_ptr(),
                                 residual.data_ptr() if residual is not None else None,
                                 y.data_ptr(), M, N, K, _DTYPES[x.dtype],
                                 ctypes.byref(cfg) if cfg is not None else None,
                                 _stream_handle(stream)))
    return y


def skinny_gemm_noalloc(x: torch.Tensor, W: torch.Tensor, y: torch.Tensor,
                        cfg: KpCfg | None = None, stream=None) -> torch.Tensor:
    """``y = bf16(x @ W.T)`` without any allocation by the library: the
    CUDA-core split-K kernel keeps its partial sums in a fixed device array
    (for callers that cannot allocate, e.g. during graph capture). ``y`` must
    be given; M <= 16. Concurrent calls on one device race."""
    _bf16_2d(x, "x")
    _bf16_2d(W, "W")
    _bf16_2d(y, "y")
    M, K = x.shape
    N = W.shape[0]
    if W.shape[1] != K or tuple(y.shape) != (M, N):
        raise ValueError("shape mismatch")
    _check(load().skinny_gemm_noalloc(x.data_ptr(), W.data_ptr(), y.data_ptr(), M, N, K,
                                      ctypes.byref(cfg) if cfg is not None else None,
                                      _stream_handle(stream)))
    return y


# ---- feed-forward operators ---------------------------------------------------
#
# Every function below runs on the current device and stream: when a stream or a
# tensor of another device is given, it calls itself with those made current, so
# that what it allocates is handed out in that stream's order. Single-token calls
# take a few microseconds on the device, so the checks on the common path are few.

_FFN_DTYPES = {torch.bfloat16: DTYPE_BF16, torch.float16: DTYPE_FP16, torch.float32: DTYPE_FP32}
_FFN_WORK: dict = {}   # workspace bytes by (device, operator, sizes): host arithmetic only
# the current stream's handle without a Stream object, the current device without a
# check of the CUDA state (the tensors at hand are CUDA tensors)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_DEVICES: dict = {}


def _device(index: int):
    d = _DEVICES.get(index)
    if d is None:
        d = _DEVICES[index] = torch.device("cuda", index)
    return d


def _here(t, name: str, stream) -> int:
    """The index of t's device, or -1 if the call has to move to another device or
    stream first."""
    try:
        index = t.get_device()
    except AttributeError:
        raise TypeError(f"{name} must be a torch.Tensor, got {type(t).__name__}") from None
    if index < 0:
        raise ValueError(f"{name} must be on a CUDA device")
    return index if stream is None and index == _current_device() else -1


@contextlib.contextmanager
def _on(device, stream, *inputs):
    """Make device and stream current. The inputs are marked as used on the
    stream, so memory that is freed meanwhile is not handed out under it."""
    if stream is not None and stream.device != device:
        raise ValueError(f"stream is on {stream.device}, the operands are on {device}")
    with torch.cuda.device(device):
        if stream is None:
            yield
            return
        for t in inputs:
            for part in ((t._buf, t._scales) if isinstance(t, Mx4Tensor) else (t,)):
                if isinstance(part, torch.Tensor) and part.is_cuda:
                    part.record_stream(stream)
        with torch.cuda.stream(stream):
            yield


def _rows(t, name: str, dtype, index: int) -> int:
    """Check a 2-D row-major CUDA matrix of `dtype` (None: any) whose rows may be
    strided; returns the row stride in elements."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor, got {type(t).__name__}")
    if dtype is not None and t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.get_device() != index:
        raise ValueError(f"{name} must be on CUDA device {index}, is on {t.device}")
    try:
        ld, inner = t.stride()
    except ValueError:
        raise ValueError(f"{name} must be a 2-D tensor") from None
    rows, cols = t.shape
    if rows <= 1:   # the stride of a single row says nothing
        ld = (cols + 7) // 8 * 8
    if ld < cols or (inner != 1 and cols > 1):
        raise ValueError(f"{name} must have contiguous rows (strides {tuple(t.stride())})")
    return ld


def _act_code(act: str) -> int:
    try:
        return ACTIVATIONS[act]
    except (KeyError, TypeError):
        raise ValueError(f"unknown activation {act!r}: one of {', '.join(ACTIVATIONS)}") from None


def _work(op: int, M: int, N: int, K: int, index: int):
    """(tensor or None, pointer, bytes) of this call's workspace."""
    key = (index, op, M, N, K)
    n = _FFN_WORK.get(key)
    if n is None:
        b = ctypes.c_size_t()
        _check(load().kp_ffn_workspace(op, M, N, K, ctypes.byref(b)))
        if len(_FFN_WORK) > 4096:
            _FFN_WORK.clear()
        n = _FFN_WORK[key] = int(b.value)
    if not n:
        return None, None, 0
    t = torch.empty(n, dtype=torch.uint8, device=_device(index))
    return t, t.data_ptr(), n


def _out(t, name: str, rows: int, cols: int, dtype, index: int):
    """The caller's output, checked, or a new one; returns (tensor, row stride)."""
    if t is None:
        return torch.empty((rows, cols), dtype=dtype, device=_device(index)), cols
    ld = _rows(t, name, dtype, index)
    if t.shape != (rows, cols):
        raise ValueError(f"{name} must be {(rows, cols)}, got {tuple(t.shape)}")
    return t, ld


class Mx4Tensor:
    """A matrix ``[rows, cols]`` held in microscaled 4-bit floating point: 4-bit
    codes and one power-of-two scale per 32 columns (4.25 bits an element), in
    the layout that ``include/kdaproj.h`` describes. Made by ``mx4_quantize``, or
    from stored ``codes`` and ``scales`` (uint8, of the sizes that
    ``Mx4Tensor.sizes`` gives, 16-byte aligned; codes past the columns and scales of
    blocks past them must be 0, as ``mx4_quantize`` leaves them, since the products
    read them)."""

    __slots__ = ("_index", "_buf", "_scales", "_code_bytes", "_scale_bytes", "shape", "device", "code_ptr", "scale_ptr")

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor, rows: int, cols: int):
        nc, ns = self.sizes(rows, cols)
        if codes.dtype != torch.uint8 or scales.dtype != torch.uint8:
            raise TypeError("codes and scales must be uint8")
        if codes.numel() != nc or scales.numel() != ns or not codes.is_contiguous() \
                or not scales.is_contiguous() or codes.device != scales.device:
            raise ValueError(f"codes and scales do not hold a {rows} x {cols} matrix "
                             f"({nc} and {ns} contiguous bytes on one device)")
        self._set(codes, scales, nc, ns, rows, cols, codes.data_ptr(), scales.data_ptr())

    def _set(self, buf, scales, nc, ns, rows, cols, code_ptr, scale_ptr):
        self._buf, self._scales, self._code_bytes, self._scale_bytes = buf, scales, nc, ns
        self.shape, self.device, self._index = (rows, cols), buf.device, buf.get_device()
        self.code_ptr, self.scale_ptr = code_ptr, scale_ptr

    @classmethod
    def _new(cls, rows: int, cols: int, device) -> "Mx4Tensor":
        """Uninitialised: both parts in one allocation."""
        nb = (cols + 31) >> 5
        nc = rows * nb * 16
        ns = ((rows + 127) >> 7) * ((nb + 3) >> 2) * 512
        off = (nc + 255) & ~255
        buf = torch.empty(off + ns, dtype=torch.uint8, device=device)
        q = cls.__new__(cls)
        ptr = buf.data_ptr()
        q._set(buf, None, nc, ns, rows, cols, ptr, ptr + off)
        return q

    @staticmethod
    def sizes(rows: int, cols: int):
        """Bytes of the codes and of the scales of a rows x cols matrix."""
        a, b = ctypes.c_size_t(), ctypes.c_size_t()
        _check(load().kp_mx4_bytes(rows, cols, ctypes.byref(a), ctypes.byref(b)))
        return int(a.value), int(b.value)

    def get_device(self) -> int:
        """The CUDA device's index, -1 on the CPU."""
        return self._index

    @property
    def codes(self) -> torch.Tensor:
        """[rows, ceil(cols / 32) * 16] bytes, two codes each."""
        rows, cols = self.shape
        return self._buf.view(-1)[:self._code_bytes].view(rows, (cols + 31) // 32 * 16)

    @property
    def scales(self) -> torch.Tensor:
        """The scale bytes, in tiles of 512."""
        if self._scales is not None:
            return self._scales
        off = self.scale_ptr - self.code_ptr
        return self._buf[off:off + self._scale_bytes]

    @property
    def nbytes(self) -> int:
        return self._code_bytes + self._scale_bytes

    def __repr__(self):
        return f"Mx4Tensor({self.shape[0]} x {self.shape[1]}, {self.device})"


def _mx4(q, name: str, index: int) -> Mx4Tensor:
    if not isinstance(q, Mx4Tensor):
        raise TypeError(f"{name} must be an Mx4Tensor (mx4_quantize), got {type(q).__name__}")
    if q._index != index:
        raise ValueError(f"{name} must be on CUDA device {index}, is on {q.device}")
    return q


def mx4_quantize(x: torch.Tensor, stream=None) -> Mx4Tensor:
    """Quantise ``x`` [rows, cols] (bfloat16, float16 or float32; any sizes, rows
    may be strided) to microscaled 4 bits: per 32 columns the scale
    ``2^(floor(log2 max|x|) - 2)``, elements to the nearest of 0, .5, 1, 1.5, 2,
    3, 4, 6 scales, ties to even. A block with a NaN or an infinity becomes NaN."""
    index = _here(x, "x", stream)
    if index < 0:
        with _on(x.device, stream, x):
            return mx4_quantize(x)
    ld = _rows(x, "x", None, index)
    dt = _FFN_DTYPES.get(x.dtype)
    if dt is None:
        raise TypeError(f"x must be bfloat16, float16 or float32, got {x.dtype}")
    rows, cols = x.shape
    q = Mx4Tensor._new(rows, cols, x.device)
    rc = load().kp_mx4_quantize(x.data_ptr(), ld, rows, cols, dt, q.code_ptr, q.scale_ptr, _raw_stream(index))
    if rc:
        _check(rc)
    return q


def mx4_dequantize(q: Mx4Tensor, dtype=torch.bfloat16, y: torch.Tensor | None = None,
                   stream=None) -> torch.Tensor:
    """The values that ``q`` stands for: exact in bfloat16 and float32 (float16
    rounds, and overflows to infinity)."""
    index = _here(q, "q", stream)
    if index < 0:
        with _on(q.device, stream, q, y):
            return mx4_dequantize(q, dtype, y)
    _mx4(q, "q", index)
    dt = _FFN_DTYPES.get(dtype)
    if dt is None:
        raise TypeError(f"dtype must be bfloat16, float16 or float32, got {dtype}")
    rows, cols = q.shape
    y, ld = _out(y, "y", rows, cols, dtype, index)
    rc = load().kp_mx4_dequantize(q.code_ptr, q.scale_ptr, rows, cols, y.data_ptr(), ld, dt, _raw_stream(index))
    if rc:
        _check(rc)
    return y


def _mx4_left(x, dtype, index: int):
    """(rows, cols, element type, x's arguments) of a 4-bit product's left side: a
    16-bit matrix, quantised within the call, or an Mx4Tensor."""
    if isinstance(x, Mx4Tensor):
        dt = torch.bfloat16 if dtype is None else dtype
        if dt not in _DTYPES:
            raise TypeError(f"dtype must be bfloat16 or float16, got {dt}")
        rows, cols = _mx4(x, "x", index).shape
        return rows, cols, dt, (None, 0, x.code_ptr, x.scale_ptr)
    ld = _rows(x, "x", None, index)
    dt = x.dtype
    if dt not in _DTYPES:
        raise TypeError(f"x must be bfloat16, float16 or an Mx4Tensor, got {dt}")
    if dtype is not None and dtype is not dt:
        raise TypeError(f"the output has x's type {dt}")
    rows, cols = x.shape
    return rows, cols, dt, (x.data_ptr(), ld, None, None)


def mx4_gemm(x, W: Mx4Tensor, y: torch.Tensor | None = None, dtype=None, stream=None) -> torch.Tensor:
    """``y = round(Q(x) @ Q(W).T)`` on the 4-bit tensor cores, sums in fp32. ``x``
    [M, K] is bfloat16 or float16 (quantised within the call; y has its type) or
    an ``Mx4Tensor`` (y has ``dtype``, bfloat16 unless given). ``W`` [N, K]. Any
    sizes; with ``x`` empty nothing runs."""
    index = _here(x, "x", stream)
    if index < 0:
        with _on(x.device, stream, x, W, y):
            return mx4_gemm(x, W, y, dtype)
    M, K, dt, xargs = _mx4_left(x, dtype, index)
    N, Kw = _mx4(W, "W", index).shape
    if Kw != K:
        raise ValueError(f"W has K={Kw}, x has K={K}")
    y, ld = _out(y, "y", M, N, dt, index)
    work, wp, wn = _work(FFN_MX4_GEMM, M, N, K, index)
    rc = load().kp_mx4_gemm(*xargs, W.code_ptr, W.scale_ptr, y.data_ptr(), ld, M, N, K, _DTYPES[dt], wp, wn,
                            _raw_stream(index))
    if rc:
        _check(rc)
    return y


def mx4_gated_ffn(x, Wg: Mx4Tensor, Wu: Mx4Tensor, act: str = "silu", h: torch.Tensor | None = None,
                  dtype=None, stream=None) -> torch.Tensor:
    """``h = round(act(Q(x) @ Q(Wg).T) * (Q(x) @ Q(Wu).T))``: the gated block over
    4-bit weights [F, K] and activations, in one product kernel. ``x`` as for
    ``mx4_gemm``; ``act`` as for ``gated_ffn``."""
    index = _here(x, "x", stream)
    if index < 0:
        with _on(x.device, stream, x, Wg, Wu, h):
            return mx4_gated_ffn(x, Wg, Wu, act, h, dtype)
    code = _act_code(act)
    T, K, dt, xargs = _mx4_left(x, dtype, index)
    shape = _mx4(Wg, "Wg", index).shape
    if _mx4(Wu, "Wu", index).shape != shape or shape[1] != K:
        raise ValueError(f"Wg {Wg.shape} and Wu {Wu.shape} must both be [F, {K}]")
    F = shape[0]
    h, ld = _out(h, "h", T, F, dt, index)
    work, wp, wn = _work(FFN_MX4_GATED, T, F, K, index)
    rc = load().kp_mx4_gated_ffn(*xargs, Wg.code_ptr, Wg.scale_ptr, Wu.code_ptr, Wu.scale_ptr, h.data_ptr(), ld,
                                 T, F, K, code, _DTYPES[dt], wp, wn, _raw_stream(index))
    if rc:
        _check(rc)
    return h


def _gated_operands(x, Wg, Wu, index: int):
    dt = x.dtype
    if dt not in _DTYPES:
        raise TypeError(f"x must be bfloat16 or float16, got {dt}")
    ldx = _rows(x, "x", None, index)
    ldg = _rows(Wg, "Wg", dt, index)
    ldu = _rows(Wu, "Wu", dt, index)
    T, K = x.shape
    shape = Wg.shape
    if shape != Wu.shape or shape[1] != K:
        raise ValueError(f"Wg {tuple(Wg.shape)} and Wu {tuple(Wu.shape)} must both be [F, {K}]")
    return T, shape[0], K, ldx, ldg, ldu, dt


def gated_ffn(x: torch.Tensor, Wg: torch.Tensor, Wu: torch.Tensor, act: str = "silu",
              h: torch.Tensor | None = None, save: bool = False, stream=None):
    """``h = round(act(x @ Wg.T) * (x @ Wu.T))``: both projections of a gated
    feed-forward block, the activation and the product in one kernel, sums in
    fp32. ``x`` [T, K], ``Wg`` and ``Wu`` [F, K], all bfloat16 or all float16; rows
    may be strided (strides and K multiples of 8, 16-byte aligned). ``act``:
    "silu", "gelu" (erf) or "gelu_tanh". With ``save`` returns ``(h, g, u)``, the
    two products in float32, for ``gated_ffn_backward``."""
    index = _here(x, "x", stream)
    if index < 0:
        with _on(x.device, stream, x, Wg, Wu, h):
            return gated_ffn(x, Wg, Wu, act, h, save)
    code = _act_code(act)
    T, F, K, ldx, ldg, ldu, dt = _gated_operands(x, Wg, Wu, index)
    h, ldh = _out(h, "h", T, F, dt, index)
    g = u = gp = up = None
    if save:
        g = torch.empty((T, F), dtype=torch.float32, device=_device(index))
        u = torch.empty((T, F), dtype=torch.float32, device=_device(index))
        gp, up = g.data_ptr(), u.data_ptr()
    work, wp, wn = _work(FFN_GATED, T, F, K, index)
    rc = load().kp_gated_ffn(x.data_ptr(), ldx, Wg.data_ptr(), ldg, Wu.data_ptr(), ldu, h.data_ptr(), ldh, gp, up,
                             T, F, K, code, _DTYPES[dt], wp, wn, _raw_stream(index))
    if rc:
        _check(rc)
    return (h, g, u) if save else h


def gated_ffn_backward(dh: torch.Tensor, x: torch.Tensor, Wg: torch.Tensor, Wu: torch.Tensor, g: torch.Tensor,
                       u: torch.Tensor, act: str = "silu", stream=None):
    """Gradients ``(dx, dWg, dWu)`` of ``gated_ffn`` for the gradient ``dh`` of its
    output, from its operands and the ``g`` and ``u`` it saved. ``dG = dh u act'(g)``
    and ``dU = dh act(g)`` are computed in fp32 and rounded to x's type as the
    tensor cores' operands (in float16 scaled by a power of two, so that neither
    overflows); the three products are summed in fp32. With no tokens the weights'
    gradients are zero."""
    index = _here(x, "x", stream)
    if index < 0:
        with _on(x.device, stream, dh, x, Wg, Wu, g, u):
            return gated_ffn_backward(dh, x, Wg, Wu, g, u, act)
    code = _act_code(act)
    T, F, K, ldx, ldg, ldu, dt = _gated_operands(x, Wg, Wu, index)
    lddh = _rows(dh, "dh", dt, index)
    for t, name in ((g, "g"), (u, "u")):
        _rows(t, name, torch.float32 if T else None, index)   # with no tokens nothing is read
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    for t, name in ((dh, "dh"), (g, "g"), (u, "u")):
        if t.shape != (T, F):
            raise ValueError(f"{name} must be {(T, F)}, got {tuple(t.shape)}")
    dx, dWg, dWu = x.new_empty((T, K)), x.new_empty((F, K)), x.new_empty((F, K))
    work, wp, wn = _work(FFN_GATED_BACKWARD, T, F, K, index)
    rc = load().kp_gated_ffn_backward(dh.data_ptr(), lddh, x.data_ptr(), ldx, Wg.data_ptr(), ldg, Wu.data_ptr(),
                                      ldu, g.data_ptr(), u.data_ptr(), dx.data_ptr(), dWg.data_ptr(),
                                      dWu.data_ptr(), T, F, K, code, _DTYPES[dt], wp, wn, _raw_stream(index))
    if rc:
        _check(rc)
    return dx, dWg, dWu


class KdaPlan:
    """Owns a ``kda_plan`` (scratch per branch + per-M configurations)."""

    def __init__(self, K: int = 7168, N_qkvg: int = 4096, N_fab: int = 136, N_fb: int = 1024,
                 max_M: int = 256):
        self.K, self.N_qkvg, self.N_fab, self.N_fb, self.max_M = K, N_qkvg, N_fab, N_fb, max_M
        self._lib = load()
        self._run = self._lib.kda_proj_run
        self._ev_key, self._ev_arr = None, None
        h = ctypes.c_void_p()
        _check(self._lib.kda_proj_plan(K, N_qkvg, N_fab, N_fb, max_M, ctypes.byref(h)))
        self._h = h

    @property
    def handle(self) -> int:
        return int(self._h.value or 0)

    def set_overlap(self, mode: int):
        _check(self._lib.kda_proj_set_overlap(self._h, int(mode)))

    def overlap_at(self, M: int) -> int:
        """Mode at M: 0 sequential, 1 overlapped, 2 single launch."""
        return int(self._lib.kda_proj_overlap_at(self._h, M))

    def get_config(self, branch: int, M: int) -> KpCfg:
        c = KpCfg()
        _check(self._lib.kda_proj_get_config(self._h, branch, M, ctypes.byref(c)))
        return c

    def set_config(self, branch: int, M: int, cfg: KpCfg):
        _check(self._lib.kda_proj_set_config(self._h, branch, M, ctypes.byref(cfg)))

    def outputs(self, M: int, device=None):
        dev = device or torch.device("cuda", torch.cuda.current_device())
        return (torch.empty((M, self.N_qkvg), dtype=torch.bfloat16, device=dev),
                torch.empty((M, self.N_fab), dtype=torch.bfloat16, device=dev),
                torch.empty((M, self.N_fb), dtype=torch.bfloat16, device=dev))

    def run(self, x: torch.Tensor, W_packed: torch.Tensor, W_fb: torch.Tensor,
            out_qkvg=None, out_fab=None, out_fb=None, aux_stream=None, events=None,
            stream=None, check: bool = False):
        """Enqueue the projection; returns ``(out_qkvg, out_fab, out_fb)``.

        ``aux_stream`` (torch.cuda.Stream) and ``events`` (two
        torch.cuda.Event) enable the two-stream overlap; ``stream`` is the
        main stream (default: the current stream). ``check=True`` waits for
        the main stream and raises ``KdaProjError(KP_EDEVICE)`` if a kernel
        wait ran out during the call (not usable under graph capture)."""
        _bf16_2d(x, "x")
        _bf16_2d(W_packed, "W_packed")
        _bf16_2d(W_fb, "W_fb")
        M, kx = x.shape
        if kx != self.K:
            raise ValueError(f"x must be [M, {self.K}]")
        if W_packed.shape != (self.N_qkvg + self.N_fab, self.K):
            raise ValueError(f"W_packed must be {(self.N_qkvg + self.N_fab, self.K)}")
        if W_fb.shape != (self.N_fb, 128):
            raise ValueError(f"W_fb must be {(self.N_fb, 128)}")
        if out_qkvg is None or out_fab is None or out_fb is None:
            oq, of, ob = self.outputs(M, x.device)
            out_qkvg = oq if out_qkvg is None else out_qkvg
            out_fab = of if out_fab is None else out_fab
            out_fb = ob if out_fb is None else out_fb
        for t, n, shape in ((out_qkvg, "out_qkvg", (M, self.N_qkvg)), (out_fab, "out_fab", (M, self.N_fab)),
                            (out_fb, "out_fb", (M, self.N_fb))):
            _bf16_2d(t, n)
            if t.shape != shape:
                raise ValueError(f"{n} must be {shape}")
        ev = None
        aux = None
        if aux_stream is not None and events is not None:
            aux = aux_stream.cuda_stream
            key = (events[0].cuda_event, events[1].cuda_event)
            if self._ev_key != key:   # the handle array, reused while the events are
                self._ev_key = key
                self._ev_arr = (ctypes.c_void_p * 2)(*key)
            ev = self._ev_arr
        rc = self._run(self._h, x.data_ptr(), W_packed.data_ptr(), W_fb.data_ptr(),
                       out_qkvg.data_ptr(), out_fab.data_ptr(), out_fb.data_ptr(), M,
                       _stream_handle(stream), aux, ev)
        if rc:
            _check(rc)
        if check:
            check_device(stream)
        return out_qkvg, out_fab, out_fb

    def close(self):
        if self._h is not None and self._h.value:
            self._lib.kda_proj_destroy(self._h)
            self._h = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def make_events():
    """Two timing-free CUDA events, created eagerly (a fresh torch Event only
    gets its handle when first recorded)."""
    evs = (torch.cuda.Event(enable_timing=False), torch.cuda.Event(enable_timing=False))
    for e in evs:
        e.record()
    return evs
