"""Run and time one skinny GEMM shape, or the KDA projection, with the
library's choice of kernel.

    python -m decode_projection_gemms_gb300.cli --M 4096 --N 4096 --K 7168 [--reps 5]
        [--cfg kind=cc,split_k=2,block=256,rows=4,k_unroll=1]
    python -m decode_projection_gemms_gb300.cli --kda --M 1 16 128 [--layers 4] [--reps 1]
    python -m decode_projection_gemms_gb300.cli --ffn --M 1 16 512 [--F 2048] [--K 7168]
        [--act silu] [--steps 4] [--fp16]
    python -m decode_projection_gemms_gb300.cli --moe --M 1 16 512 [--experts 32] [--top-k 4]
        [--F 1024] [--K 4096] [--score softmax] [--act silu] [--steps 4] [--fp16]

GEMM: prints the configuration used (the table's or the built-in rule's
choice, or the one given with --cfg as comma-separated kp_cfg fields) and the
device time per call over `reps` calls after one warm-up call, with CUDA
events on the launching stream. --kda: the projection of the pages' shapes
(packed [4096 + 136, 7168] weight, W_fb [1024, 128]) for each M in the
table's mode, eagerly, `reps` passes over a stack of `layers` weight layers
(one layer per call; 4 layers are 244 MB, above the L2). --ffn: a gated
feed-forward block y = (act(x Wg^T) * (x Wu^T)) Wd^T. It is trained for `steps`
steps on a batch of the largest M (towards a teacher block's outputs, on Wg and
Wu), its weights are converted to microscaled 4 bits, and both forms then serve
each M: times per call and how far the 4-bit outputs are from the 16-bit ones.
--moe: a mixture-of-experts layer behind a norm, y = x + f(z), z the root-mean-square norm
of x, f(z) the sum over a token's top-k experts e of w_e (act(z Wg_e^T) * (z Wu_e^T)) Wd_e^T
with experts and weights from router logits z Wr^T. It is trained for `steps` steps on a batch
of the largest M (towards a teacher layer's outputs, on the norm's weight and the layer's four)
and then serves each M: time per call and rows of the busiest expert.
Inputs are seeded synthetic bf16 (or fp16 with --fp16).
"""
from __future__ import annotations

import argparse
import json

import torch

from . import binding
from .binding import KpCfg
from .build import build
from .inputs import gen_w, gen_x

CFG_FIELDS = ("kind", "split_k", "block", "rows", "k_unroll", "producers", "stages", "flags")


def parse_cfg(text: str) -> KpCfg:
    """'kind=tc05,split_k=8,k_unroll=2' -> KpCfg (fields not given keep
    KpCfg.make's defaults)."""
    kw = {}
    for item in text.split(","):
        key, _, val = item.partition("=")
        key = key.strip()
        if key not in CFG_FIELDS or not val:
            raise ValueError(f"bad --cfg item {item!r}; fields: {', '.join(CFG_FIELDS)}")
        kw[key] = val.strip() if key == "kind" else int(val)
    if "kind" not in kw:
        raise ValueError("--cfg needs kind=cc|tc05|smallk")
    return KpCfg.make(**kw)


def run_kda(m_list, layers: int, reps: int):
    from .inputs import gen_kda_layer
    dev = torch.device("cuda", torch.cuda.current_device())
    K, Nq, Nfab, Nfb = 7168, 4096, 136, 1024
    stack = [tuple(t.to(dev) for t in gen_kda_layer(layer, seed=0, device="cpu" if layer == 0 else dev))
             for layer in range(layers)]
    plan = binding.KdaPlan(K, Nq, Nfab, Nfb, max_M=max(m_list))
    aux = torch.cuda.Stream()
    evs = binding.make_events()
    stream = torch.cuda.current_stream()
    try:
        for M in m_list:
            x = gen_x(M, K, seed=0, device=dev)
            outs = plan.outputs(M, dev)
            plan.run(x, *stack[0], *outs, aux_stream=aux, events=evs)   # warm-up
            torch.cuda.synchronize()
            a = torch.cuda.Event(enable_timing=True)
            b = torch.cuda.Event(enable_timing=True)
            a.record(stream)
            for _ in range(reps):
                for wp, wfb in stack:
                    plan.run(x, wp, wfb, *outs, aux_stream=aux, events=evs)
            b.record(stream)
            torch.cuda.synchronize()
            us = a.elapsed_time(b) * 1e3 / (reps * layers)
            print(json.dumps({"M": M, "mode": plan.overlap_at(M), "us_per_call_eager": round(us, 3),
                              "configs": {br: plan.get_config(i, M).as_dict()
                                          for i, br in enumerate(("qkvg", "fab", "fb"))},
                              "device_error": binding.device_error()}))
    finally:
        plan.close()


def _time_us(fn, reps: int) -> float:
    fn()   # warm-up
    torch.cuda.synchronize()
    a = torch.cuda.Event(enable_timing=True)
    b = torch.cuda.Event(enable_timing=True)
    a.record()
    for _ in range(reps):
        fn()
    b.record()
    torch.cuda.synchronize()
    return a.elapsed_time(b) * 1e3 / reps


def run_ffn(m_list, F: int, K: int, act: str, steps: int, reps: int, dtype):
    dev = torch.device("cuda", torch.cuda.current_device())
    std = K ** -0.5
    Wg, Wu = (gen_w(F, K, seed, std=std, device=dev, dtype=dtype) for seed in (1, 2))
    Wd = gen_w(K, F, 3, std=F ** -0.5, device=dev, dtype=dtype)
    Wd_t = Wd.t().contiguous()          # dh = dy Wd, a product with Wd^T's rows
    T = max(m_list)
    x = gen_x(T, K, seed=4, device=dev, dtype=dtype)

    def block(xs, g, u):
        return binding.skinny_gemm_ex(binding.gated_ffn(xs, g, u, act=act), Wd)

    # a teacher: the same block with other gate and up weights
    target = block(x, *(gen_w(F, K, seed, std=std, device=dev, dtype=dtype) for seed in (5, 6)))
    losses = []
    for step in range(steps + 1):
        h, g, u = binding.gated_ffn(x, Wg, Wu, act=act, save=True)
        diff = binding.skinny_gemm_ex(h, Wd) - target
        losses.append(float(diff.float().square().mean()))
        if step == steps:
            break
        dh = binding.skinny_gemm_ex(diff, Wd_t)
        _, dWg, dWu = binding.gated_ffn_backward(dh, x, Wg, Wu, g, u, act=act)
        for W, dW in ((Wg, dWg), (Wu, dWu)):   # a step of fixed length along the gradient
            W.add_(dW, alpha=-0.05 * float(W.float().norm() / (dW.float().norm() + 1e-30)))
    print(json.dumps({"training": {"tokens": T, "F": F, "K": K, "act": act, "losses": [round(v, 5) for v in losses]}}))

    qg, qu, qd = (binding.mx4_quantize(W) for W in (Wg, Wu, Wd))

    def block4(xs):
        return binding.mx4_gemm(binding.mx4_gated_ffn(xs, qg, qu, act=act), qd)

    for M in m_list:
        xs = x[:M]
        a, b = block(xs, Wg, Wu).float(), block4(xs).float()
        print(json.dumps({"M": M, "us_16_bit": round(_time_us(lambda: block(xs, Wg, Wu), reps), 2),
                          "us_4_bit": round(_time_us(lambda: block4(xs), reps), 2),
                          "relative_difference": round(float((a - b).norm() / a.norm()), 4),
                          "weight_bytes_16_bit": 2 * (Wg.numel() + Wu.numel() + Wd.numel()),
                          "weight_bytes_4_bit": qg.nbytes + qu.nbytes + qd.nbytes,
                          "device_error": binding.device_error()}))
    return losses


def moe_layer(x, Wr, Wg, Wu, Wd, top_k: int, act: str = "silu", score: str = "softmax", save: bool = False):
    """A mixture-of-experts layer's outputs; with ``save`` also what ``moe_layer_backward``
    needs."""
    logits = binding.skinny_gemm_ex(x, Wr)
    route = binding.moe_route(logits, top_k, score=score)
    rows = binding.moe_dispatch(x, route)
    if not save:
        h = binding.grouped_gated_ffn(rows, Wg, Wu, route.offsets, act=act)
        return binding.moe_combine(binding.grouped_gemm(h, Wd, route.offsets), route), route
    h, g, u = binding.grouped_gated_ffn(rows, Wg, Wu, route.offsets, act=act, save=True)
    out = binding.grouped_gemm(h, Wd, route.offsets)
    return binding.moe_combine(out, route), (logits, route, rows, h, g, u, out)


def moe_layer_backward(dy, x, Wr, Wg, Wu, Wd, saved, act: str = "silu"):
    """Gradients (dx, dWr, dWg, dWu, dWd) of ``moe_layer`` for the gradient of its outputs."""
    logits, route, rows, h, g, u, out = saved
    dout, dweights = binding.moe_combine_backward(dy, out, route)
    dh, dWd = binding.grouped_gemm_backward(dout, h, Wd, route.offsets)
    drows, dWg, dWu = binding.grouped_gated_ffn_backward(dh, rows, Wg, Wu, route.offsets, g, u, act=act)
    dlogits = binding.moe_route_backward(dweights, logits, route)
    # the products of the router: their contractions in whole groups of eight
    pad = torch.nn.functional.pad
    T, E = dlogits.shape
    t, e = -T % 8, -E % 8
    dWr = binding.skinny_gemm_ex(pad(dlogits.t(), (0, t)).contiguous(), pad(x.t(), (0, t)).contiguous())
    dx = binding.skinny_gemm_ex(pad(dlogits, (0, e)).contiguous(), pad(Wr.t(), (0, e)).contiguous(),
                                binding.moe_dispatch_backward(drows, route))
    return dx, dWr, dWg, dWu, dWd


def norm_moe_layer(x, gamma, *weights, top_k: int, act: str = "silu", score: str = "softmax", save: bool = False):
    """``x + moe_layer(z, *weights)`` with z the root-mean-square norm of x; with ``save`` also
    what ``norm_moe_layer_backward`` needs, else the routing."""
    if not save:
        y, route = moe_layer(binding.layer_norm(x, gamma, center=False), *weights, top_k, act, score)
        return x + y, route
    z, _, rstd = binding.layer_norm(x, gamma, center=False, save=True)
    y, saved = moe_layer(z, *weights, top_k, act, score, save=True)
    return x + y, (z, rstd, saved)


def norm_moe_layer_backward(dy, x, gamma, *weights, saved, act: str = "silu"):
    """Gradients (dx, dgamma, dWr, dWg, dWu, dWd) of ``norm_moe_layer``."""
    z, rstd, inner = saved
    dz, *grads = moe_layer_backward(dy, z, *weights, inner, act)
    dx, dgamma, _ = binding.layer_norm_backward(dz, x, gamma, None, rstd)
    return (dy + dx, dgamma, *grads)


def run_moe(m_list, E: int, top_k: int, F: int, K: int, score: str, act: str, steps: int, reps: int, dtype):
    dev = torch.device("cuda", torch.cuda.current_device())

    def layer(seed):
        g = torch.Generator(device=dev).manual_seed(seed)

        def w(*shape):
            v = torch.empty(shape, dtype=dtype, device=dev)
            return v.normal_(0.0, shape[-1] ** -0.5, generator=g)

        gamma = torch.ones(K, dtype=dtype, device=dev)
        return gamma, w(E, K), w(E, F, K), w(E, F, K), w(E, K, F)

    weights, teacher = layer(1), layer(2)
    how = {"top_k": top_k, "act": act, "score": score}
    T = max(m_list)
    x = gen_x(T, K, seed=4, device=dev, dtype=dtype)
    target, _ = norm_moe_layer(x, *weights[:2], *teacher[2:], **how)   # other experts, the same router
    losses = []
    for step in range(steps + 1):
        y, saved = norm_moe_layer(x, *weights, **how, save=True)
        diff = y - target
        losses.append(float(diff.float().square().mean()))
        if step == steps:
            break
        grads = norm_moe_layer_backward(diff, x, *weights, saved=saved, act=act)[1:]
        for W, dW in zip(weights, grads):   # a step of fixed length along the gradient
            W.add_(dW, alpha=-0.05 * float(W.float().norm() / (dW.float().norm() + 1e-30)))
    print(json.dumps({"training": {"tokens": T, "experts": E, "top_k": top_k, "F": F, "K": K, "score": score, "act": act,
                                   "losses": [round(v, 5) for v in losses]}}))
    for M in m_list:
        xs = x[:M]
        _, route = norm_moe_layer(xs, *weights, **how)
        n = (route.offsets[1:] - route.offsets[:-1]).tolist()
        us = _time_us(lambda: norm_moe_layer(xs, *weights, **how), reps)
        print(json.dumps({"M": M, "us": round(us, 2), "rows": sum(n), "busiest_expert": max(n),
                          "experts_used": sum(v > 0 for v in n),
                          "tflops": round(6.0 * sum(n) * F * K / us / 1e6, 2), "device_error": binding.device_error()}))
    return losses


def main(argv=None):
    ap = argparse.ArgumentParser()
    ap.add_argument("--kda", action="store_true", help="run the KDA projection instead of one GEMM")
    ap.add_argument("--ffn", action="store_true", help="train and serve a gated feed-forward block")
    ap.add_argument("--moe", action="store_true", help="train and serve a mixture-of-experts layer")
    ap.add_argument("--M", type=int, nargs="+", required=True)
    ap.add_argument("--F", type=int, default=None, help="--ffn, --moe: features of a block (2048, 1024)")
    ap.add_argument("--experts", type=int, default=32, help="--moe")
    ap.add_argument("--top-k", type=int, default=4, help="--moe: experts of a token")
    ap.add_argument("--score", default="softmax", choices=sorted(binding.SCORES), help="--moe")
    ap.add_argument("--act", default="silu", choices=sorted(binding.ACTIVATIONS))
    ap.add_argument("--steps", type=int, default=4, help="--ffn: training steps")
    ap.add_argument("--N", type=int)
    ap.add_argument("--K", type=int)
    ap.add_argument("--layers", type=int, default=4)
    ap.add_argument("--reps", type=int, default=5)
    ap.add_argument("--fp16", action="store_true")
    ap.add_argument("--residual", action="store_true")
    ap.add_argument("--cfg", default=None, help="explicit configuration, e.g. kind=cc,split_k=2")
    args = ap.parse_args(argv)
    cfg_in = parse_cfg(args.cfg) if args.cfg else None

    build()
    binding.load()
    if args.kda:
        run_kda(args.M, args.layers, args.reps)
        return
    if args.ffn:
        run_ffn(args.M, args.F or 2048, args.K or 7168, args.act, args.steps, args.reps,
                torch.float16 if args.fp16 else torch.bfloat16)
        return
    if args.moe:
        run_moe(args.M, args.experts, args.top_k, args.F or 1024, args.K or 4096, args.score, args.act, args.steps,
                args.reps, torch.float16 if args.fp16 else torch.bfloat16)
        return
    if args.N is None or args.K is None or len(args.M) != 1:
        ap.error("a GEMM needs one --M and --N, --K")
    args.M = args.M[0]
    dev = torch.device("cuda", torch.cuda.current_device())
    dt = torch.float16 if args.fp16 else torch.bfloat16
    x = gen_x(args.M, args.K, seed=1, device=dev, dtype=dt)
    W = gen_w(args.N, args.K, seed=2, device=dev, dtype=dt)
    r = gen_x(args.M, args.N, seed=3, device=dev, dtype=dt) if args.residual else None
    y = torch.empty((args.M, args.N), dtype=dt, device=dev)
    sms = torch.cuda.get_device_properties(dev).multi_processor_count
    cfg = cfg_in if cfg_in is not None else binding.select_config(args.M, args.N, args.K, sms)
    stream = torch.cuda.current_stream()
    binding.skinny_gemm_ex(x, W, r, y, cfg=cfg_in)   # warm-up (attributes, scratch)
    torch.cuda.synchronize()
    a = torch.cuda.Event(enable_timing=True)
    b = torch.cuda.Event(enable_timing=True)
    a.record(stream)
    for _ in range(args.reps):
        binding.skinny_gemm_ex(x, W, r, y, cfg=cfg_in)
    b.record(stream)
    torch.cuda.synchronize()
    us = a.elapsed_time(b) * 1e3 / args.reps
    flops = 2.0 * args.M * args.N * args.K
    nbytes = 2 * (args.M * args.K + args.N * args.K + args.M * args.N)
    print(json.dumps({"M": args.M, "N": args.N, "K": args.K, "config": cfg.as_dict(),
                      "us_per_call": round(us, 3), "tflops": round(flops / us / 1e6, 1),
                      "gbs": round(nbytes / us / 1e3, 1),
                      "device_error": binding.device_error()}))


if __name__ == "__main__":
    main()
