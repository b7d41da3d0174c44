"""A whole expert layer on the library's calls: scored routing, E4M3 dispatch,
the experts' two products, combine.

    from combine_moe_plan_gb300 import layer, moe
    experts = moe.Experts(w13, s13, w2, s2)              # E4M3, fp32 scale per 128 x 128
    moe_layer = layer.ExpertLayer(experts, T_max=4096, E=256, k=8,
                                  router=moe.Router("sigmoid", n_group=8, topk_group=4, group_top=2, scale=2.5),
                                  bias=bias)
    y = moe_layer(x, logits)                             # bf16 [T, H], fp32 [T, E] -> bf16 [T, H]

``python -m combine_moe_plan_gb300.layer --tokens 96`` times one on random
weights, call by call and as one CUDA graph.
"""
from __future__ import annotations

import argparse

import torch

from . import moe


class ExpertLayer:
    """Router, pool, experts and the buffer between the experts' products.

    ``E`` logical experts on the ``experts.P`` physical ones (``rep_off`` /
    ``rep_ids``: replica map, needed where P > E).  One call at a time per
    buffer set; consecutive calls may alternate ``buf``.  A call takes bf16
    ``x`` [T, H], fp32 ``logits`` [T, E] and, if given, bf16 ``y`` [T, H], all
    contiguous and on the GPU; others are refused (ValueError)."""

    def __init__(self, experts, T_max, E, k, router, bias=None, rep_off=None, rep_ids=None, n_sets=1):
        self.experts, self.router, self.bias = experts, router, bias
        self.rep_off, self.rep_ids = rep_off, rep_ids
        self.pool = moe.Pool(T_max, experts.H, E, experts.P, k, n_sets=n_sets)
        self.inner = [experts.inner(T_max * k) for _ in range(n_sets)]
        # the pool's error word is zeroed on this stream: before another stream's call may set it
        torch.cuda.current_stream(experts.error_word.device).synchronize()

    def __call__(self, x, logits, y=None, buf=0, stream=None):
        T = x.shape[0]
        if logits.shape[0] != T:
            raise ValueError("logits and x must have the same number of tokens")
        p = self.pool
        # with these checked first (and the logits by the first call), an error leaves nothing enqueued
        moe._dense("x", x, torch.bfloat16, (T, p.H))
        if y is not None:
            moe._dense("y", y, torch.bfloat16, (T, p.H))
        p.plan_routed(logits, self.router, self.bias, self.rep_off, self.rep_ids, buf=buf, stream=stream)
        p.dispatch_f8(x, buf=buf, stream=stream)
        p.experts(self.experts, T, *self.inner[buf], buf=buf, stream=stream)
        return p.combine(T, y, buf=buf, stream=stream)

    def check(self) -> int:
        """Wait, and return the device error bits of the pool and the experts (0 = clean)."""
        return self.pool.check() | self.experts.check()


def random_experts(P, H, I, seed=0, device="cuda"):
    """Experts with N(0, 1 / inputs) weights, quantised per 128 x 128 block."""
    g = torch.Generator(device)
    g.manual_seed(seed)

    def pair(n, k):
        w = torch.empty(P, n, k, dtype=torch.float8_e4m3fn, device=device)
        s = torch.empty(P, n // 128, k // 128, device=device)
        for p in range(P):
            v = torch.randn(n // 128, 128, k // 128, 128, generator=g, device=device) * k ** -0.5
            amax = v.abs().amax((1, 3), keepdim=True)
            w[p] = (v * (448.0 / amax)).reshape(n, k).to(torch.float8_e4m3fn)
            s[p] = amax.reshape(n // 128, k // 128) / 448.0
        return w, s

    return moe.Experts(*pair(2 * I, H), *pair(H, I))


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, value in (("tokens", 96), ("hidden", 7168), ("inner", 2048), ("experts", 256), ("topk", 8), ("groups", 8),
                        ("steps", 20)):
        ap.add_argument("--" + name, type=int, default=value)
    a = ap.parse_args(argv)
    router = moe.Router("sigmoid", n_group=a.groups, topk_group=max(1, a.groups // 2), group_top=2, scale=2.5)
    layer = ExpertLayer(random_experts(a.experts, a.hidden, a.inner), a.tokens, a.experts, a.topk, router,
                        bias=torch.zeros(a.experts, device="cuda"))
    x = torch.randn(a.tokens, a.hidden, device="cuda").bfloat16()
    logits = torch.randn(a.tokens, a.experts, device="cuda")
    y = torch.empty_like(x)

    def timed(step):
        for _ in range(3):
            step()
        begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        begin.record()
        for _ in range(a.steps):
            step()
        end.record()
        torch.cuda.synchronize()
        return begin.elapsed_time(end) / a.steps * 1e3

    calls = timed(lambda: layer(x, logits, y))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer(x, logits, y)
    replay = timed(graph.replay)
    if layer.check():
        raise RuntimeError("device error word set")
    rows = a.tokens * a.topk
    print(f"{a.tokens} tokens x {a.hidden}, {a.experts} experts of {a.inner}, top-{a.topk} ({rows} rows): "
          f"{calls:.1f} us a layer call by call, {replay:.1f} us as a graph")


if __name__ == "__main__":
    main()
