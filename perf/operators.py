"""Cases for the feed-forward operators: 4-bit quantisation and product, and the
gated feed-forward block in 16 and in 4 bits.

Five operators:

* ``quant``: microscaled 4-bit quantisation of a matrix and the values that the
  codes stand for (blocks of 32 along a row, one power-of-two scale a block);
* ``mx4_gemm``: ``y = round(Q(x) . Q(W)^T)`` with Q the quantisation above, the
  weight quantised beforehand, the activations within the call;
* ``gated``: ``h = round(act(x Wg^T) * (x Wu^T))`` in bf16 or fp16;
* ``gated_train``: the same with its backward pass: h, dx, dWg, dWu;
* ``mx4_gated``: the gated block over 4-bit weights and activations.

Hidden size 7168 and 4096 output features are the sizes of this package's
projection; the other sizes are generic.
"""
from __future__ import annotations

import math

import torch

own = False

BLOCK = 32            # elements that share a scale
W_STD = 0.02          # weights as the package's synthetic layers draw them
DH_STD = 0.05         # gradients after loss scaling
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
ACTS = ("silu", "gelu", "gelu_tanh")


def listed():
    return [
        # activations of a decode batch, quantised before a 4-bit product
        {"name": "quant_decode", "op": "quant", "rows": 16, "cols": 7168, "dtype": "bf16"},
        # a layer's fp32 master weights, converted for serving; the row length ends inside a block
        {"name": "quant_weights", "op": "quant", "rows": 8191, "cols": 7156, "dtype": "fp32"},
        # one decoded token through a projection
        {"name": "mx4_gemm_token", "op": "mx4_gemm", "M": 1, "N": 4096, "K": 7168, "dtype": "bf16"},
        # a decode batch, odd in every size
        {"name": "mx4_gemm_odd", "op": "mx4_gemm", "M": 77, "N": 4099, "K": 2050, "dtype": "fp16"},
        # a long prompt
        {"name": "mx4_gemm_prompt", "op": "mx4_gemm", "M": 4096, "N": 4096, "K": 7168, "dtype": "bf16"},
        # one decoded token through the gated half of a feed-forward block
        {"name": "gated_token", "op": "gated", "T": 1, "F": 2048, "K": 7168, "act": "silu", "dtype": "bf16"},
        # a decode batch
        {"name": "gated_batch", "op": "gated", "T": 96, "F": 2048, "K": 4096, "act": "gelu_tanh", "dtype": "fp16"},
        # a long prompt with a ragged end
        {"name": "gated_prompt", "op": "gated", "T": 4003, "F": 2048, "K": 7168, "act": "silu", "dtype": "bf16"},
        # a short fine-tuning sequence of odd length
        {"name": "gated_train_short", "op": "gated_train", "T": 333, "F": 1416, "K": 2048, "act": "gelu",
         "dtype": "fp16"},
        # a training batch
        {"name": "gated_train_batch", "op": "gated_train", "T": 8192, "F": 2048, "K": 7168, "act": "silu",
         "dtype": "bf16"},
        # a few decoded tokens over 4-bit weights
        {"name": "mx4_gated_decode", "op": "mx4_gated", "T": 8, "F": 2048, "K": 7168, "act": "silu",
         "dtype": "bf16"},
        # a prompt over 4-bit weights
        {"name": "mx4_gated_prompt", "op": "mx4_gated", "T": 2000, "F": 4096, "K": 7168, "act": "gelu_tanh",
         "dtype": "bf16"},
    ]


def _log(rng, lo, hi, multiple=1):
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return max(lo, min(hi, v // multiple * multiple))


def draw(rng):
    op = rng.choice(("quant", "mx4_gemm", "gated", "gated_train", "mx4_gated"))
    half = rng.choice(("bf16", "fp16"))
    if op == "quant":
        return {"op": op, "rows": _log(rng, 1, 8191), "cols": _log(rng, 32, 7156),
                "dtype": rng.choice(("bf16", "fp16", "fp32"))}
    if op == "mx4_gemm":
        return {"op": op, "M": _log(rng, 1, 4096), "N": _log(rng, 64, 4096), "K": _log(rng, 64, 7168),
                "dtype": half}
    if op == "gated":
        return {"op": op, "T": _log(rng, 1, 4003), "F": _log(rng, 128, 2048, 8), "K": _log(rng, 256, 7168, 8),
                "act": rng.choice(ACTS), "dtype": half}
    if op == "gated_train":
        return {"op": op, "T": _log(rng, 1, 4096), "F": _log(rng, 128, 4096, 8), "K": _log(rng, 256, 7168, 8),
                "act": rng.choice(ACTS), "dtype": half}
    return {"op": op, "T": _log(rng, 1, 2000), "F": _log(rng, 64, 4096), "K": _log(rng, 64, 7168),
            "act": rng.choice(ACTS), "dtype": half}


def work(case):
    op = case["op"]
    es = 4 if case["dtype"] == "fp32" else 2
    if op == "quant":
        n = case["rows"] * case["cols"]
        # read the matrix, write codes and scales, write the values in 16 bits
        return {"bytes": n * es + n // 2 + n // BLOCK + 2 * n, "flops": 2 * n}
    if op == "mx4_gemm":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": M * K * es + N * K * 17 // 32 + M * N * es, "flops": 2 * M * N * K}
    T, F, K = case["T"], case["F"], case["K"]
    if op == "gated":
        return {"bytes": es * (T * K + 2 * F * K + T * F), "flops": 4 * T * F * K}
    if op == "gated_train":
        # x, both weights and dh read; h, dx and both weight gradients written
        return {"bytes": es * (2 * T * K + 4 * F * K + 2 * T * F), "flops": 12 * T * F * K}
    return {"bytes": es * (T * K + T * F) + 2 * F * K * 17 // 32, "flops": 4 * T * F * K}


# --- inputs -------------------------------------------------------------------

def _normal(g, rows, cols, std, dtype):
    v = torch.randn((rows, cols), generator=g, device="cuda", dtype=torch.float32)
    return v.mul_(std).to(dtype)


def _activations(g, rows, cols, dtype):
    """Hidden states: unit normal, with a few channels that are much larger than
    the rest, as trained models have them."""
    v = torch.randn((rows, cols), generator=g, device="cuda", dtype=torch.float32)
    big = torch.randint(0, cols, (max(1, cols // 512),), generator=g, device="cuda")
    v[:, big] *= 12.0
    return v.to(dtype)


def _inputs(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    op = case["op"]
    if op == "quant":
        if case["dtype"] == "fp32":
            return {"x": _normal(g, case["rows"], case["cols"], W_STD, dt)}
        return {"x": _activations(g, case["rows"], case["cols"], dt)}
    if op == "mx4_gemm":
        return {"x": _activations(g, case["M"], case["K"], dt),
                "W": _normal(g, case["N"], case["K"], W_STD, dt)}
    T, F, K = case["T"], case["F"], case["K"]
    s = {"x": _activations(g, T, K, dt), "Wg": _normal(g, F, K, W_STD, dt), "Wu": _normal(g, F, K, W_STD, dt)}
    if op == "gated_train":
        s["dh"] = _normal(g, T, F, DH_STD, dt)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if case["op"] in ("mx4_gemm", "mx4_gated"):
        # a server quantises its weights once, when it loads them
        for name in ("W", "Wg", "Wu"):
            if name in s:
                if own:
                    from decode_projection_gemms_gb300 import mx4_quantize
                    s[name] = mx4_quantize(s[name])
                else:
                    s[name] = _quantize(s[name])
    s["case"] = case
    return s


# --- plain form ---------------------------------------------------------------

def _pow2(e):
    """2^e in fp32, exactly, for -126 <= e <= 127 (a power function need not be)."""
    return ((e + 127) << 23).view(torch.float32)


def _quantize(x):
    """Codes as values of the 4-bit format (fp32, [rows, blocks, 32]) and the
    blocks' scale exponents, from elementary operations in 32 bits."""
    rows, cols = x.shape
    nb = (cols + BLOCK - 1) // BLOCK
    v = torch.zeros((rows, nb * BLOCK), device=x.device, dtype=torch.float32)
    v[:, :cols] = x
    v = v.view(rows, nb, BLOCK)
    amax = v.abs().amax(dim=2)
    # frexp: amax = m * 2^e with m in [1/2, 1), so floor(log2 amax) = e - 1; the
    # format's largest exponent is 2
    e = torch.where(amax > 0, torch.frexp(amax).exponent - 3, torch.full_like(amax, -127, dtype=torch.int32))
    e = e.clamp(-127, 125)
    s = v * _pow2(-e).unsqueeze(2)
    a = s.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    q = (torch.round(a / step) * step).clamp(max=6.0)
    return {"codes": torch.copysign(q, s).to(torch.float16), "exp": e.to(torch.int16),
            "cols": cols}


def _values(q):
    e = q["exp"].to(torch.int32).unsqueeze(2)
    v = q["codes"].float() * 0.5 * _pow2(e + 1)
    return v.view(v.shape[0], -1)[:, :q["cols"]]


def _act(g, act):
    if act == "silu":
        return g / (1.0 + torch.exp(-g))
    if act == "gelu":
        return 0.5 * g * (1.0 + torch.erf(g * math.sqrt(0.5)))
    t = torch.tanh(math.sqrt(2.0 / math.pi) * (g + 0.044715 * g * g * g))
    return 0.5 * g * (1.0 + t)


def _dact(g, act):
    if act == "silu":
        s = 1.0 / (1.0 + torch.exp(-g))
        return s * (1.0 + g * (1.0 - s))
    if act == "gelu":
        phi = torch.exp(-0.5 * g * g) * (1.0 / math.sqrt(2.0 * math.pi))
        return 0.5 * (1.0 + torch.erf(g * math.sqrt(0.5))) + g * phi
    c = math.sqrt(2.0 / math.pi)
    t = torch.tanh(c * (g + 0.044715 * g * g * g))
    return 0.5 * (1.0 + t) + 0.5 * g * (1.0 - t * t) * c * (1.0 + 3.0 * 0.044715 * g * g)


def _plain(s, case):
    op = case["op"]
    dt = s["x"].dtype
    if op == "quant":
        return _values(_quantize(s["x"])).to(torch.bfloat16)
    if op == "mx4_gemm":
        return (_values(_quantize(s["x"])) @ _values(s["W"]).t()).to(dt)
    if op == "mx4_gated":
        x = _values(_quantize(s["x"]))
        return (_act(x @ _values(s["Wg"]).t(), case["act"]) * (x @ _values(s["Wu"]).t())).to(dt)
    x, Wg, Wu = s["x"].float(), s["Wg"].float(), s["Wu"].float()
    g = x @ Wg.t()
    u = x @ Wu.t()
    a = _act(g, case["act"])
    h = (a * u).to(dt)
    if op == "gated":
        return h
    dh = s["dh"].float()
    dg = dh * u * _dact(g, case["act"])
    du = dh * a
    return {"h": h, "dx": (dg @ Wg + du @ Wu).to(dt), "dWg": (dg.t() @ x).to(dt), "dWu": (du.t() @ x).to(dt)}


# --- the framework's operators --------------------------------------------------

def _own(s, case):
    import decode_projection_gemms_gb300 as kda
    op = case["op"]
    if op == "quant":
        return kda.mx4_dequantize(kda.mx4_quantize(s["x"]), dtype=torch.bfloat16)
    if op == "mx4_gemm":
        return kda.mx4_gemm(s["x"], s["W"])
    if op == "mx4_gated":
        return kda.mx4_gated_ffn(s["x"], s["Wg"], s["Wu"], act=case["act"])
    if op == "gated":
        return kda.gated_ffn(s["x"], s["Wg"], s["Wu"], act=case["act"])
    h, g, u = kda.gated_ffn(s["x"], s["Wg"], s["Wu"], act=case["act"], save=True)
    dx, dWg, dWu = kda.gated_ffn_backward(s["dh"], s["x"], s["Wg"], s["Wu"], g, u, act=case["act"])
    return {"h": h, "dx": dx, "dWg": dWg, "dWu": dWu}


def run(state):
    return (_own if own else _plain)(state, state["case"])


# --- the definition in 64 bits ----------------------------------------------------

def _exact_values(x):
    """Microscaled 4-bit values from the definition: scale 2^(floor(log2 max) - 2),
    elements to the nearest of the format's magnitudes, ties to the even code."""
    rows, cols = x.shape
    nb = -(-cols // BLOCK)
    v = torch.nn.functional.pad(x.double(), (0, nb * BLOCK - cols)).view(rows * nb, BLOCK)
    top = v.abs().max(dim=1, keepdim=True).values
    # floor(log2 top) is the exponent field of its bits; 2^n is built the same way
    n = ((top.view(torch.int64) >> 52) - 1023 - 2).clamp(min=-127)
    scale = ((n + 1023) << 52).view(torch.float64)
    mags = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
    a = v.abs() / scale
    q = torch.zeros_like(a)
    for i in range(1, 8):
        mid = 0.5 * (mags[i - 1] + mags[i])
        # a tie goes to the even code: upwards where i is even
        q = torch.where((a > mid) | ((a == mid) & (i % 2 == 0)), torch.full_like(a, mags[i]), q)
    return (torch.sign(v) * q * scale).view(rows, nb * BLOCK)[:, :cols]


def _exact_act(g, act):
    """The activation and its derivative in 64 bits."""
    if act == "silu":
        s = torch.special.expit(g)
        return g * s, s + g * s * torch.special.expit(-g)
    if act == "gelu":
        cdf = 0.5 * torch.special.erfc(-g / math.sqrt(2.0))
        return g * cdf, cdf + g * torch.exp(-g * g / 2.0) / math.sqrt(2.0 * math.pi)
    # 0.5 (1 + tanh z) is the logistic function of 2 z
    z2 = 2.0 * math.sqrt(2.0 / math.pi) * (g + 0.044715 * g ** 3)
    s = torch.special.expit(z2)
    dz2 = 2.0 * math.sqrt(2.0 / math.pi) * (1.0 + 3.0 * 0.044715 * g ** 2)
    return g * s, s + g * s * torch.special.expit(-z2) * dz2


def exact(case, seed):
    s = _inputs(case, seed)
    op = case["op"]
    if op == "quant":
        return _exact_values(s["x"])
    if op == "mx4_gemm":
        return _exact_values(s["x"]) @ _exact_values(s["W"]).t()
    if op == "mx4_gated":
        x = _exact_values(s["x"])
        return _exact_act(x @ _exact_values(s["Wg"]).t(), case["act"])[0] * (x @ _exact_values(s["Wu"]).t())
    x, wg, wu = s["x"].double(), s["Wg"].double(), s["Wu"].double()
    u = x @ wu.t()
    a, da = _exact_act(x @ wg.t(), case["act"])
    if op == "gated":
        return a * u
    dh = s["dh"].double()
    du = a.mul(dh)
    dg = da.mul(dh).mul(u)
    return {"h": a * u, "dx": dg @ wg + du @ wu, "dWg": dg.t() @ x, "dWu": du.t() @ x}
