"""Cases for the mixture-of-experts operators: the router, the way of the tokens to
their experts and back, and the products grouped by expert with ragged sizes.

Four operators, each with its gradients:

* ``route``: top-k experts of each token from its router logits, the weights of
  their outputs, and the order that puts the chosen (token, expert) pairs expert by
  expert; trained, also the logits' gradient;
* ``shuffle``: rows of the tokens in that order (``dispatch``), and each token's
  weighted sum of its experts' rows (``combine``); trained, both ways back;
* ``grouped``: y = round(x W_e^T), rows of x expert by expert, each expert with a
  matrix of its own; trained, also dx and dW;
* ``gated``: h = round(act(x Wg_e^T) * (x Wu_e^T)), the same way; trained, also dx,
  dWg and dWu;

and ``block``, all of them in a row as a mixture-of-experts layer calls them.

Hidden size 7168 and 2048 or 4096 features are sizes of this package's projection and
feed-forward block; the other sizes are generic.
"""
from __future__ import annotations

import math

import torch

own = False

W_STD = 0.02          # weights as the package's synthetic layers draw them
DH_STD = 0.05         # gradients after loss scaling
SKEW = 0.6            # how unevenly tokens go to experts: deviation of the experts' logits
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
ACTS = ("silu", "gelu", "gelu_tanh")


def listed():
    return [
        # the router of one decoded token
        {"name": "route_token", "op": "route", "T": 1, "E": 64, "k": 6, "score": "softmax", "bias": False,
         "padded": False, "dtype": "bf16", "train": False},
        # the router of a training batch whose last sequences are padded
        {"name": "route_train", "op": "route", "T": 16384, "E": 256, "k": 8, "score": "sigmoid", "bias": True,
         "padded": True, "dtype": "fp32", "train": True},
        # a decode batch on its way to its experts and back
        {"name": "shuffle_decode", "op": "shuffle", "T": 24, "E": 64, "k": 8, "K": 7168, "dtype": "bf16",
         "train": False},
        # a training batch, forward and backward
        {"name": "shuffle_train", "op": "shuffle", "T": 8192, "E": 64, "k": 4, "K": 4096, "dtype": "bf16",
         "train": True},
        # the second product of a decode batch's experts: a few rows each, some without any
        {"name": "grouped_decode", "op": "grouped", "R": 64, "E": 32, "N": 7168, "K": 2048, "dtype": "bf16",
         "train": False},
        # the same for a long prompt
        {"name": "grouped_prompt", "op": "grouped", "R": 16384, "E": 32, "N": 7168, "K": 2048, "dtype": "bf16",
         "train": False},
        # a small model's training step, odd in its rows and features
        {"name": "grouped_train", "op": "grouped", "R": 4003, "E": 8, "N": 1000, "K": 1416, "dtype": "fp16",
         "train": True},
        # the eight experts of one decoded token
        {"name": "gated_token", "op": "gated", "R": 8, "E": 32, "F": 2048, "K": 7168, "act": "silu",
         "dtype": "bf16", "train": False},
        # a long prompt
        {"name": "gated_prompt", "op": "gated", "R": 16384, "E": 32, "F": 2048, "K": 7168, "act": "silu",
         "dtype": "bf16", "train": False},
        # a short fine-tuning sequence, odd in every size
        {"name": "gated_train_odd", "op": "gated", "R": 1021, "E": 12, "F": 331, "K": 1032, "act": "gelu",
         "dtype": "fp16", "train": True},
        # a training batch
        {"name": "gated_train_batch", "op": "gated", "R": 16384, "E": 16, "F": 2048, "K": 4096, "act": "silu",
         "dtype": "bf16", "train": True},
        # a whole layer over a batch of prompts with padded ends
        {"name": "block_batch", "op": "block", "T": 4096, "E": 32, "k": 4, "F": 2048, "K": 4096, "act": "silu",
         "dtype": "bf16"},
    ]


def _log(rng, lo, hi, multiple=1):
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return max(lo, min(hi, v // multiple * multiple))


def draw(rng):
    op = rng.choice(("route", "shuffle", "grouped", "gated", "gated", "block"))
    half = rng.choice(("bf16", "fp16"))
    train = rng.random() < 0.5
    E = _log(rng, 4, 256) if op in ("route", "shuffle") else _log(rng, 2, 32)
    k = min(E, rng.randint(1, 8))
    if op == "route":
        score = rng.choice(("softmax", "sigmoid"))
        return {"op": op, "T": _log(rng, 1, 16384), "E": E, "k": k, "score": score,
                "bias": score == "sigmoid" and rng.random() < 0.5, "padded": rng.random() < 0.3,
                "dtype": rng.choice(("bf16", "fp16", "fp32")), "train": train}
    if op == "shuffle":
        return {"op": op, "T": _log(rng, 1, 8192), "E": E, "k": min(k, 4), "K": _log(rng, 64, 4096, 8),
                "dtype": half, "train": train}
    R = _log(rng, 1, 8192) if train else _log(rng, 1, 16384)
    if op == "grouped":
        return {"op": op, "R": R, "E": E, "N": _log(rng, 64, 7168, 8 if train else 1), "K": _log(rng, 64, 2048, 8),
                "dtype": half, "train": train}
    if op == "gated":
        return {"op": op, "R": R, "E": E, "F": _log(rng, 64, 2048), "K": _log(rng, 64, 4096, 8),
                "act": rng.choice(ACTS), "dtype": half, "train": train}
    return {"op": op, "T": _log(rng, 1, 4096), "E": E, "k": min(k, 4), "F": _log(rng, 64, 2048, 8),
            "K": _log(rng, 64, 4096, 8), "act": rng.choice(ACTS), "dtype": half}


def work(case):
    op = case["op"]
    es = 4 if case["dtype"] == "fp32" else 2
    E = case["E"]
    if op == "route":
        T, k = case["T"], case["k"]
        # logits read; ids, weights, order, positions and offsets written; trained, the
        # logits again, the weights' gradient, and the logits' written
        n = T * E * es + 16 * T * k + 4 * (E + 1)
        if case["train"]:
            n += 2 * T * E * es + 8 * T * k
        return {"bytes": n, "flops": 4 * T * E}
    if op == "shuffle":
        T, k, K = case["T"], case["k"], case["K"]
        rows, tok = T * k * K * es, T * K * es
        n = tok + rows + rows + tok + 12 * T * k   # dispatch writes the rows, combine reads those of the experts
        if case["train"]:
            n += 2 * rows + tok + 4 * T * k + rows + tok
        return {"bytes": n, "flops": (6 if case["train"] else 2) * T * k * K}
    if op == "block":
        R = case["T"] * case["k"]
        T, F, K = case["T"], case["F"], case["K"]
        used = min(E, R)
        return {"bytes": es * (2 * T * K + 3 * used * F * K) + T * E * 4, "flops": 6 * R * F * K}
    R, K = case["R"], case["K"]
    N = case["N"] if op == "grouped" else case["F"]
    m = 1 if op == "grouped" else 2               # matrices of an expert
    used = min(E, R)                              # experts whose weights have to be read, at most
    n = es * (R * K + m * used * N * K + R * N)
    f = 2 * m * R * N * K
    if case["train"]:
        n += es * (R * N + R * K + m * E * N * K)   # the output's gradient read, dx and the weights' written
        f *= 3
    return {"bytes": n, "flops": f}


# --- inputs -------------------------------------------------------------------

def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _weights(g, E, rows, cols, dtype):
    w = torch.empty((E, rows, cols), device="cuda", dtype=dtype)
    return w.normal_(0.0, W_STD, generator=g)


def _activations(g, rows, cols, dtype):
    """Hidden states: unit normal, with a few channels that are much larger than
    the rest, as trained models have them."""
    v = _randn(g, rows, cols)
    big = torch.randint(0, cols, (max(1, cols // 512),), generator=g, device="cuda")
    v[:, big] *= 12.0
    return v.to(dtype)


def _logits(g, T, E, dtype, padded):
    """Router logits with experts that are liked more than others; the last eighth
    of a padded batch has no expert at all."""
    v = (_randn(g, T, E) + SKEW * _randn(g, 1, E)).to(dtype)
    if padded:
        v[T - T // 8:] = -math.inf
    return v


def _offsets(g, R, E):
    """Rows of each expert: R draws from uneven probabilities."""
    p = torch.softmax(SKEW * _randn(g, E), 0)
    e = torch.multinomial(p, R, replacement=True, generator=g)
    n = torch.zeros(E + 1, device="cuda", dtype=torch.int64)
    n[1:] = torch.cumsum(torch.bincount(e, minlength=E), 0)
    return n.to(torch.int32)


def _inputs(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    op, E = case["op"], case["E"]
    s = {}
    if op == "route":
        T, k = case["T"], case["k"]
        s["logits"] = _logits(g, T, E, dt, case["padded"])
        if case["bias"]:
            s["bias"] = 0.1 * _randn(g, E)
        if case["train"]:
            s["dweights"] = _randn(g, T, k)
        return s
    if op == "shuffle":
        T, k, K = case["T"], case["k"], case["K"]
        s["logits"] = _logits(g, T, E, torch.float32, False)
        s["x"] = _activations(g, T, K, dt)
        s["rows"] = _randn(g, T * k, K).to(dt)     # what the experts made of them
        if case["train"]:
            s["dy"] = (DH_STD * _randn(g, T, K)).to(dt)
            s["drows"] = (DH_STD * _randn(g, T * k, K)).to(dt)
        return s
    if op == "block":
        T, F, K = case["T"], case["F"], case["K"]
        s["logits"] = _logits(g, T, E, torch.float32, True)
        s["x"] = _activations(g, T, K, dt)
        s["Wg"], s["Wu"] = _weights(g, E, F, K, dt), _weights(g, E, F, K, dt)
        s["Wd"] = _weights(g, E, K, F, dt)
        return s
    R, K = case["R"], case["K"]
    s["offsets"] = _offsets(g, R, E)
    if op == "grouped":
        N = case["N"]
        s["x"] = _randn(g, R, K).to(dt)
        s["W"] = _weights(g, E, N, K, dt)
    else:
        N = case["F"]
        s["x"] = _activations(g, R, K, dt)
        s["Wg"], s["Wu"] = _weights(g, E, N, K, dt), _weights(g, E, N, K, dt)
    if case["train"]:
        s["dy"] = (DH_STD * _randn(g, R, N)).to(dt)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "shuffle":
        # both directions follow a routing that the layer has made before
        if own:
            from decode_projection_gemms_gb300 import moe_route
            s["route"] = moe_route(s["logits"], case["k"])
        else:
            s["route"] = _route(s["logits"], None, case["k"], "softmax")
    if not own and "offsets" in s:
        # the plain form pads every expert's rows to the longest one's
        s["most"] = int((s["offsets"][1:] - s["offsets"][:-1]).max())
    if not own and case["op"] == "block":
        r = _route(s["logits"], None, case["k"], "softmax")
        s["most"] = int((r["offsets"][1:] - r["offsets"][:-1]).max())
    s["case"] = case
    return s


# --- plain form ---------------------------------------------------------------

def _scores(logits, score):
    v = logits.float()
    if score == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-v))
    e = torch.exp(v - v.amax(dim=1, keepdim=True).clamp(min=-1e30))
    return e / e.sum(dim=1, keepdim=True).clamp(min=1e-38)


def _chosen_scores(logits, ids, score):
    return torch.where(ids >= 0, _scores(logits, score).gather(1, ids.clamp(min=0)), 0.0)


def _route(logits, bias, k, score):
    """The k largest logits (with a bias: the largest sigmoid plus bias, in 64 bits
    where two may lie next to each other), ties to the lowest expert; experts at minus
    infinity are not chosen. The weights are the chosen scores over their sum."""
    T, E = logits.shape
    key = logits.double()
    if bias is not None:
        key = torch.where(key == -math.inf, key, 1.0 / (1.0 + torch.exp(-key)) + bias.double())
    top, ids = torch.sort(key, dim=1, descending=True, stable=True)
    ids = torch.where(top[:, :k] == -math.inf, -1, ids[:, :k])
    s = _chosen_scores(logits, ids, score)
    weights = s / s.sum(dim=1, keepdim=True).clamp(min=1e-38)
    flat = torch.where(ids < 0, E, ids).reshape(-1)
    order = torch.sort(flat, stable=True)[1]
    counts = torch.bincount(flat, minlength=E + 1)
    offsets = torch.zeros(E + 1, device=flat.device, dtype=torch.int64)
    offsets[1:] = torch.cumsum(counts[:E], 0)
    place = torch.arange(T * k, device=flat.device)
    position = torch.empty_like(order)
    position[order] = place
    order = torch.where(place < offsets[E], order, -1)
    position = torch.where(flat < E, position, -1)
    i32 = torch.int32
    return {"ids": ids.to(i32), "weights": weights, "offsets": offsets.to(i32), "order": order.to(i32),
            "position": position.view(T, k).to(i32)}


def _route_grad(dweights, logits, r, score):
    ids, w = r["ids"].long(), r["weights"]
    d = dweights - (w * dweights).sum(dim=1, keepdim=True)
    s = _chosen_scores(logits, ids, score)
    # softmax: the others' share cancels; sigmoid: s (1 - s) over the sum, s over the sum being w
    d = w * d * (1.0 - s) if score == "sigmoid" else w * d
    out = torch.zeros(logits.shape, device=logits.device, dtype=torch.float32)
    return out.scatter_add_(1, ids.clamp(min=0), torch.where(ids >= 0, d, 0.0)).to(logits.dtype)


def _dispatch(x, r):
    return x[(r["order"] // r["ids"].shape[1]).clamp(min=0).long()]


def _of_tokens(rows, r):
    """[T, k, K] in 32 bits: the rows of each token's experts, zeros where it has none."""
    at = r["position"].long()
    return torch.where((at >= 0).unsqueeze(2), rows[at.clamp(min=0)].float(), 0.0)


def _padded(x, offsets, most):
    """[E, most, cols] in 32 bits: every expert's rows, zeros behind them; and where
    they lie."""
    at = offsets[:-1].long().unsqueeze(1) + torch.arange(most, device=x.device)
    inside = at < offsets[1:].long().unsqueeze(1)
    v = torch.where(inside.unsqueeze(2), x[at.clamp(max=x.shape[0] - 1)].float(), 0.0)
    return v, at[inside], inside


def _rows_of(v, at, inside, rows, dtype):
    out = torch.zeros((rows, v.shape[2]), device=v.device, dtype=dtype)
    out[at] = v[inside].to(dtype)
    return out


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


def _grouped(x, W, offsets, most):
    xp, at, inside = _padded(x, offsets, most)
    return _rows_of(xp @ W.float().transpose(1, 2), at, inside, x.shape[0], x.dtype)


def _gated(x, Wg, Wu, offsets, most, act):
    xp, at, inside = _padded(x, offsets, most)
    h = _act(xp @ Wg.float().transpose(1, 2), act) * (xp @ Wu.float().transpose(1, 2))
    return _rows_of(h, at, inside, x.shape[0], x.dtype)


def _plain(s, case):
    op = case["op"]
    if op == "route":
        r = _route(s["logits"], s.get("bias"), case["k"], case["score"])
        if case["train"]:
            r["dlogits"] = _route_grad(s["dweights"], s["logits"], r, case["score"])
        return r
    if op == "shuffle":
        r = s["route"]
        w = r["weights"].unsqueeze(2)
        rows = _of_tokens(s["rows"], r)
        out = {"x_rows": _dispatch(s["x"], r), "y": (w * rows).sum(dim=1).to(s["x"].dtype)}
        if case["train"]:
            dy = s["dy"].float().unsqueeze(1)
            slot = r["order"].long()
            out["drows"] = (w * dy).reshape(slot.numel(), -1)[slot].to(s["dy"].dtype)
            out["dweights"] = (rows * dy).sum(dim=2)
            out["dx"] = _of_tokens(s["drows"], r).sum(dim=1).to(s["x"].dtype)
        return out
    if op == "block":
        r = _route(s["logits"], None, case["k"], "softmax")
        h = _gated(_dispatch(s["x"], r), s["Wg"], s["Wu"], r["offsets"], s["most"], case["act"])
        rows = _grouped(h, s["Wd"], r["offsets"], s["most"])
        return (r["weights"].unsqueeze(2) * _of_tokens(rows, r)).sum(dim=1).to(s["x"].dtype)
    offsets, most = s["offsets"], s["most"]
    if not case["train"]:
        if op == "grouped":
            return _grouped(s["x"], s["W"], offsets, most)
        return _gated(s["x"], s["Wg"], s["Wu"], offsets, most, case["act"])
    dt, R = s["x"].dtype, s["x"].shape[0]
    x, at, inside = _padded(s["x"], offsets, most)
    dy = _padded(s["dy"], offsets, most)[0]

    def back(v):
        return _rows_of(v, at, inside, R, dt)
    if op == "grouped":
        W = s["W"].float()
        return {"y": back(x @ W.transpose(1, 2)), "dx": back(dy @ W), "dW": (dy.transpose(1, 2) @ x).to(dt)}
    Wg, Wu = s["Wg"].float(), s["Wu"].float()
    g, u = x @ Wg.transpose(1, 2), x @ Wu.transpose(1, 2)
    a = _act(g, case["act"])
    dg, du = dy * u * _dact(g, case["act"]), dy * a
    return {"h": back(a * u), "dx": back(dg @ Wg + du @ Wu), "dWg": (dg.transpose(1, 2) @ x).to(dt),
            "dWu": (du.transpose(1, 2) @ x).to(dt)}


# --- the framework's operators --------------------------------------------------

def _own(s, case):
    import decode_projection_gemms_gb300 as kda
    op = case["op"]
    if op == "route":
        r = kda.moe_route(s["logits"], case["k"], score=case["score"], bias=s.get("bias"))
        out = {"ids": r.ids, "weights": r.weights, "offsets": r.offsets, "order": r.order, "position": r.position}
        if case["train"]:
            out["dlogits"] = kda.moe_route_backward(s["dweights"], s["logits"], r)
        return out
    if op == "shuffle":
        r = s["route"]
        out = {"x_rows": kda.moe_dispatch(s["x"], r), "y": kda.moe_combine(s["rows"], r)}
        if case["train"]:
            out["drows"], out["dweights"] = kda.moe_combine_backward(s["dy"], s["rows"], r)
            out["dx"] = kda.moe_dispatch_backward(s["drows"], r)
        return out
    if op == "block":
        r = kda.moe_route(s["logits"], case["k"])
        h = kda.grouped_gated_ffn(kda.moe_dispatch(s["x"], r), s["Wg"], s["Wu"], r.offsets, act=case["act"])
        return kda.moe_combine(kda.grouped_gemm(h, s["Wd"], r.offsets), r)
    x, offsets = s["x"], s["offsets"]
    if op == "grouped":
        y = kda.grouped_gemm(x, s["W"], offsets)
        if not case["train"]:
            return y
        dx, dW = kda.grouped_gemm_backward(s["dy"], x, s["W"], offsets)
        return {"y": y, "dx": dx, "dW": dW}
    if not case["train"]:
        return kda.grouped_gated_ffn(x, s["Wg"], s["Wu"], offsets, act=case["act"])
    h, g, u = kda.grouped_gated_ffn(x, s["Wg"], s["Wu"], offsets, act=case["act"], save=True)
    dx, dWg, dWu = kda.grouped_gated_ffn_backward(s["dy"], x, s["Wg"], s["Wu"], offsets, g, u, act=case["act"])
    return {"h": h, "dx": dx, "dWg": dWg, "dWu": dWu}


def run(state):
    return (_own if own else _plain)(state, state["case"])


# --- the definition in 64 bits ----------------------------------------------------

EXACT_FLOPS = 6e12    # products in 64 bits that take a few seconds


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


def _exact_choice(logits, bias, k, score):
    """Each token's experts by repeated choice of the largest, and their weights."""
    v = logits.double()
    key = v.clone() if bias is None else torch.where(v == -math.inf, v, torch.special.expit(v) + bias.double())
    p = torch.special.expit(v) if score == "sigmoid" else torch.softmax(v, 1).nan_to_num(0.0)
    ids, chosen = [], []
    for _ in range(k):
        top = key.max(dim=1, keepdim=True).values
        first = torch.where(key == top, torch.arange(key.shape[1], device=key.device), key.shape[1]).min(dim=1).values
        ok = top[:, 0] > -math.inf
        ids.append(torch.where(ok, first, -1))
        chosen.append(torch.where(ok, p.gather(1, first.unsqueeze(1))[:, 0], 0.0))
        key.scatter_(1, first.unsqueeze(1), -math.inf)
    s = torch.stack(chosen, 1)
    total = s.sum(dim=1, keepdim=True)
    return torch.stack(ids, 1), torch.where(total > 0, s / total, 0.0), s


def _exact_rows(ids, E):
    """For every expert the flat (token, slot) indices that chose it, in order."""
    flat = ids.reshape(-1)
    return [torch.nonzero(flat == e)[:, 0] for e in range(E)]


def exact(case, seed):
    if case["op"] in ("grouped", "gated", "block") and work(case)["flops"] > EXACT_FLOPS:
        return None
    s = _inputs(case, seed)
    op, E = case["op"], case["E"]
    if op == "route":
        ids, w, p = _exact_choice(s["logits"], s.get("bias"), case["k"], case["score"])
        out = {"weights": w}
        if case["train"]:
            dw = s["dweights"].double()
            d = w * (dw - (w * dw).sum(dim=1, keepdim=True))
            if case["score"] == "sigmoid":
                d = d * (1.0 - p)
            dl = torch.zeros(s["logits"].shape, device=d.device, dtype=torch.float64)
            for j in range(case["k"]):
                chosen = torch.nonzero(ids[:, j] >= 0)[:, 0]
                dl[chosen, ids[chosen, j]] = d[chosen, j]
            out["dlogits"] = dl
        return out
    if op in ("shuffle", "block"):
        ids, w, _ = _exact_choice(s["logits"], None, case["k"], "softmax")
        lists = _exact_rows(ids, E)
        slots = torch.cat(lists)
        token = slots // case["k"]
    if op == "shuffle":
        x = s["x"].double()
        rows = s["rows"].double()
        wr = w.reshape(-1)[slots].unsqueeze(1)
        out = {"x_rows": x[token], "y": torch.zeros_like(x).index_add_(0, token, wr * rows)}
        if case["train"]:
            dy = s["dy"].double()[token]
            dw = torch.zeros(w.numel(), device=x.device, dtype=torch.float64)
            dw[slots] = (dy * rows).sum(dim=1)
            out["drows"], out["dweights"] = wr * dy, dw.view_as(w)
            out["dx"] = torch.zeros_like(x).index_add_(0, token, s["drows"].double())
        return out
    if op == "block":
        y = torch.zeros(s["x"].shape, device="cuda", dtype=torch.float64)
        for e, mine in enumerate(lists):
            t = mine // case["k"]
            x = s["x"][t].double()
            h = _exact_act(x @ s["Wg"][e].double().t(), case["act"])[0] * (x @ s["Wu"][e].double().t())
            y.index_add_(0, t, w.reshape(-1)[mine].unsqueeze(1) * (h @ s["Wd"][e].double().t()))
        return y
    parts = {}
    ends = s["offsets"].tolist()
    for e in range(E):
        r = slice(ends[e], ends[e + 1])
        x = s["x"][r].double()
        if op == "grouped":
            W = s["W"][e].double()
            got = {"y": x @ W.t()}
            if case["train"]:
                dy = s["dy"][r].double()
                got["dx"], got["dW"] = dy @ W, dy.t() @ x
        else:
            wg, wu = s["Wg"][e].double(), s["Wu"][e].double()
            u = x @ wu.t()
            a, da = _exact_act(x @ wg.t(), case["act"])
            got = {"h": a * u}
            if case["train"]:
                dh = s["dy"][r].double()
                dg, du = dh * u * da, dh * a
                got.update(dx=dg @ wg + du @ wu, dWg=dg.t() @ x, dWu=du.t() @ x)
        for name, v in got.items():
            parts.setdefault(name, []).append(v)
    whole = {name: torch.stack(v) if name.startswith("dW") else torch.cat(v) for name, v in parts.items()}
    return whole if case["train"] else whole["y" if op == "grouped" else "h"]
