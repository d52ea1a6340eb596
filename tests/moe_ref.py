"""Plain 64-bit forms of the mixture-of-experts operators (torch double arithmetic;
nothing of the package)."""
from __future__ import annotations

import math

import torch

from ffn_ref import gated, gated_grads, product_bounds, acc_bound


def choose(logits, bias, k, score):
    """(ids [T, k], scores [T, k]) by k choices of the largest key, ties to the lowest
    expert; -1 and 0 where only minus infinity or NaN is left."""
    v = logits.double().cpu()
    v = torch.where(torch.isnan(v), -math.inf, v)
    # the largest finite number in place of plus infinity
    v = v.clamp(max=torch.finfo(torch.float32).max)
    key = v.clone()
    if bias is not None:
        key = torch.where(v > -math.inf, torch.sigmoid(v) + bias.double().cpu(), -math.inf)
        key = torch.where(torch.isnan(key), -math.inf, key)
    T, E = v.shape
    ids = torch.full((T, k), -1, dtype=torch.int64)
    for j in range(k):
        top, _ = key.max(dim=1, keepdim=True)
        first = torch.where(key == top, torch.arange(E), E).amin(dim=1)
        ids[:, j] = torch.where(top[:, 0] > -math.inf, first, -1)
        key[torch.arange(T), first] = -math.inf
    chosen = torch.where(ids >= 0, v.gather(1, ids.clamp(min=0)), -math.inf)
    return ids, chosen


def weights(chosen, score):
    """Chosen scores over their sum, from the chosen logits."""
    lg = torch.nn.functional.logsigmoid(chosen) if score == "sigmoid" else chosen
    w = torch.softmax(lg, dim=1)
    return torch.where(chosen > -math.inf, w, 0.0).nan_to_num(0.0)


def order(ids, E):
    """(offsets, order, position) of the pairs, expert by expert."""
    T, k = ids.shape
    lists = [[] for _ in range(E)]
    for i, e in enumerate(ids.reshape(-1).tolist()):
        if e >= 0:
            lists[e].append(i)
    offs, rows = [0], []
    for x in lists:
        rows += x
        offs.append(len(rows))
    pos = [-1] * (T * k)
    for r, i in enumerate(rows):
        pos[i] = r
    return offs, rows + [-1] * (T * k - len(rows)), torch.tensor(pos).view(T, k)


def spans(offsets):
    o = offsets.tolist()
    return [(e, slice(o[e], o[e + 1])) for e in range(len(o) - 1)]


def grouped(x, W, offsets):
    """(y, bound on its fp32 error) over all rows; zeros where there is no expert."""
    y = torch.zeros((x.shape[0], W.shape[1]), dtype=torch.float64, device=x.device)
    b = torch.zeros_like(y)
    for e, r in spans(offsets):
        y[r], b[r] = product_bounds(x[r].double(), W[e].double())
    return y, b


def grouped_grads(dy, x, W, offsets):
    """{name: (gradient, bound)}."""
    dx = torch.zeros(x.shape, dtype=torch.float64, device=x.device)
    ex = torch.zeros_like(dx)
    dW = torch.zeros(W.shape, dtype=torch.float64, device=x.device)
    eW = torch.zeros_like(dW)
    for e, r in spans(offsets):
        d, xe, w = dy[r].double(), x[r].double(), W[e].double()
        dx[r], ex[r] = d @ w, acc_bound(d, w, w.shape[0])
        dW[e], eW[e] = d.t() @ xe, acc_bound(d.t(), xe, xe.shape[0])
    return {"dx": (dx, ex), "dW": (dW, eW)}


def grouped_gated(x, Wg, Wu, offsets, act):
    """(h, bound, g, bound of g, u, bound of u)."""
    out = [torch.zeros((x.shape[0], Wg.shape[1]), dtype=torch.float64, device=x.device) for _ in range(6)]
    for e, r in spans(offsets):
        for o, v in zip(out, gated(x[r].double(), Wg[e].double(), Wu[e].double(), act)):
            o[r] = v
    return out


def grouped_gated_grads(dh, x, Wg, Wu, offsets, act, unit):
    dx, dg, du = (torch.zeros(t.shape, dtype=torch.float64, device=x.device) for t in (x, Wg, Wu))
    ex, eg, eu = (torch.zeros_like(t) for t in (dx, dg, du))
    for e, r in spans(offsets):
        got = gated_grads(dh[r].double(), x[r].double(), Wg[e].double(), Wu[e].double(), act, unit)
        (dx[r], ex[r]), (dg[e], eg[e]), (du[e], eu[e]) = got["dx"], got["dWg"], got["dWu"]
    return {"dx": (dx, ex), "dWg": (dg, eg), "dWu": (du, eu)}
