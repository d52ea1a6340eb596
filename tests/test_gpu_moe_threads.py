"""The router called from several host threads at once."""
import threading

import pytest
import torch

import decode_projection_gemms_gb300 as kda
from decode_projection_gemms_gb300 import binding

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("E,score", [(1024, "softmax"), (512, "softmax"), (1024, "sigmoid")])
def test_threads_that_route_different_sizes(E, score):
    """Few tokens and many, which need different shared memory of the same kernel: no
    call is refused, and every thread gets what it gets alone."""
    k, lib = 32, binding.load()
    tokens = (64, 24, 20, 24)
    logits = [torch.randn((T, E), generator=torch.Generator(device="cuda").manual_seed(i), device="cuda")
              for i, T in enumerate(tokens)]
    bias = torch.linspace(0.0, 0.1, E, device="cuda") if score == "sigmoid" else None
    routes = [kda.moe_route(x, k, score=score, bias=bias) for x in logits]
    want = [r._buf.clone() for r in routes]
    calls = []
    for x, r in zip(logits, routes):     # into the routes made before, so that the threads do little else
        s = torch.cuda.Stream()
        r._buf.zero_()
        calls.append((x.data_ptr(), E, None if bias is None else bias.data_ptr(), r.tokens, E, k, binding.SCORES[score],
                      binding.DTYPE_FP32, r._at(0), r._at(3), r._at(4), r._at(2), r._at(1), None, 0, s.cuda_stream, s))
    torch.cuda.synchronize()
    refused, go = [], threading.Event()

    def work(args):
        go.wait()
        for _ in range(4000):
            if lib.kp_moe_route(*args):
                refused.append(binding.last_error())

    threads = [threading.Thread(target=work, args=(c[:-1],)) for c in calls]
    for t in threads:
        t.start()
    go.set()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not refused
    assert all(torch.equal(r._buf, w) for r, w in zip(routes, want))
    assert binding.device_error() == 0
