"""A whole expert layer on the library's calls: scored routing, E4M3 dispatch,
the experts' two products, combine.

    from combine_moe_plan_gb300 import layer, moe
    experts = moe.Experts(w13, s13, w2, s2)              # E4M3, fp32 scale per 128 x 128
    moe_layer = layer.ExpertLayer(experts, T_max=4096, E=256, k=8,
                                  router=moe.Router("sigmoid", n_group=8, topk_group=4, group_top=2, scale=2.5),
                                  bias=bias)
    y = moe_layer(x, logits)                             # bf16 [T, H], fp32 [T, E] -> bf16 [T, H]

``python -m combine_moe_plan_gb300.layer --tokens 96`` times one on random
weights, call by call and as one CUDA graph; with ``--train`` a TrainingLayer,
forward and backward:

    net = layer.TrainingLayer(w13, w2, T_max=4096, E=64, k=6)      # bf16 weights
    y = net.forward(x, logits)                                     # bf16, fp32 -> bf16
    dx, dlogits = net.backward(dy, dw13, dw2, accumulate=True)     # fp32 gradients, added up
"""
from __future__ import annotations

import argparse
import contextlib

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


class TrainingLayer:
    """The same layer in bf16 with gradients: scored (``router``) or top-k softmax
    routing, bf16 rows, the experts' products, combine; and back.

    ``forward`` keeps, per buffer set, x (by reference: leave it alone until the
    set's ``backward``), the plan, with a router a copy of the logits, and the
    experts' gate and up values in 8 bits; rows and experts' outputs are not kept.  ``backward`` takes the gradient of y
    and returns those of x and the logits; the weights' gradients go to ``dw13``
    and ``dw2`` (fp32, added up with ``accumulate``; or bf16).  A replica's weights
    have a gradient of their own.  Several sets may be forward before the first
    goes backward (gradient accumulation, pipelining); the buffers of rows are
    shared, so all calls go to one stream, or wait for one another.  Tensors are
    contiguous, on the current GPU and on a 16-byte boundary, of the types and shapes
    of the calls they go to; others are refused (ValueError) before anything is
    enqueued."""

    def __init__(self, w13, w2, T_max, E, k, router=None, bias=None, rep_off=None, rep_ids=None, n_sets=1):
        if router is None and bias is not None:
            raise ValueError("a bias needs a router")
        self.experts = ex = moe.DenseExperts(w13, w2)
        self.router, self.bias, self.rep_off, self.rep_ids = router, bias, rep_off, rep_ids
        self.pool = moe.Pool(T_max, ex.H, E, ex.P, k, n_sets=n_sets)
        self.views = [self.pool.view(b) for b in range(n_sets)]
        n, dev = T_max * k, ex.error_word.device
        self.kept = [ex.kept(n) for _ in range(n_sets)]
        self.saved = [None] * n_sets  # x, the logits kept, and the handle of the stream that reads x
        self._streams = {}
        # the logits as the plan saw them: the caller's may be those of the next batch by the time of a backward
        self.logits = [torch.empty((T_max, E), device=dev) if router is not None else None for _ in range(n_sets)]

        def rows(width, dtype=torch.bfloat16):
            return torch.empty((n, width), dtype=dtype, device=dev)

        self.x_rows, self.d_rows = rows(ex.H), rows(ex.H)  # tokens in their windows; their gradients
        self.h, self.dgu = rows(ex.I), rows(2 * ex.I)
        self.parts = rows(ex.I // 128, torch.float32)
        self.row_gates, self.dgates = torch.empty(n, device=dev), torch.empty((T_max, k), device=dev)
        # the pool's error word is zeroed on this stream: before another stream's call may set it
        torch.cuda.current_stream(dev).synchronize()

    def forward(self, x, logits, y=None, buf=0, stream=None):
        T, p, ex = x.shape[0], self.pool, self.experts
        if not 0 <= buf < len(self.saved):
            raise ValueError(f"buf: want one of {len(self.saved)} sets, got {buf}")
        # with these checked first, an error leaves nothing enqueued
        moe._dense("x", x, torch.bfloat16, (T, p.H))
        moe._dense("logits", logits, torch.float32, (T, p.E))
        if T > p.T_max:
            raise ValueError(f"x: at most {p.T_max} tokens, got {T}")
        if y is None:
            y = moe._empty((T, p.H), torch.bfloat16, x.device, stream)
        moe._dense("y", y, torch.bfloat16, (T, p.H))
        if self.rep_off is not None and self.rep_ids is not None:
            moe._dense("rep_off", self.rep_off, torch.int32, (p.E + 1,))
            moe._dense("rep_ids", self.rep_ids, torch.int32, (p.P,))
        moe._on_one_gpu(ex.error_word, p.workspace, x, logits, y, self.bias, self.rep_off, self.rep_ids)
        moe._aligned(x=x, logits=logits, y=y)
        if abs(x.data_ptr() - y.data_ptr()) < 2 * T * p.H:
            raise ValueError("y lies in x, which is kept for the backward pass")
        self.saved[buf] = None
        on = self._reads(stream, x, logits)
        if self.router is None:
            p.plan(logits, self.rep_off, self.rep_ids, buf=buf, stream=stream)
        else:
            p.plan_routed(logits, self.router, self.bias, self.rep_off, self.rep_ids, buf=buf, stream=stream)
            kept = self.logits[buf] if T == p.T_max else self.logits[buf][:T]
            with contextlib.nullcontext() if stream is None else torch.cuda.stream(stream):
                logits = kept.copy_(logits)
        p.scatter(x, self.x_rows, buf=buf, stream=stream)
        v, n = self.views[buf], T * p.k
        ex.up(self.x_rows, v["offsets"], self.h, *self.kept[buf], rows=n, stream=stream)
        ex.down(self.h, v["offsets"], v["ex_out"], rows=n, stream=stream)
        y = p.combine(T, y, buf=buf, stream=stream)
        self.saved[buf] = x, logits if self.router is not None else None, on
        return y

    def backward(self, dy, dw13, dw2, dx=None, dlogits=None, accumulate=False, buf=0, stream=None):
        p, ex = self.pool, self.experts
        if not 0 <= buf < len(self.saved) or self.saved[buf] is None:
            raise ValueError(f"set {buf} has no forward to go back through")
        x, logits, on = self.saved[buf]
        T, n = x.shape[0], x.shape[0] * p.k
        dx = moe._empty(x.shape, x.dtype, x.device, stream) if dx is None else dx
        dlogits = moe._empty((T, p.E), torch.float32, x.device, stream) if dlogits is None else dlogits
        # all of it before the first launch: a refusal later on would leave gradients added up once already
        moe._dense("dy", dy, torch.bfloat16, (T, p.H))
        moe._dense("dx", dx, torch.bfloat16, (T, p.H))
        moe._dense("dlogits", dlogits, torch.float32, (T, p.E))
        ex._gradient("dw13", dw13, 2 * ex.I, ex.H, accumulate)
        ex._gradient("dw2", dw2, ex.H, ex.I, accumulate)
        moe._on_one_gpu(ex.error_word, dy, dx, dlogits, dw13, dw2)
        moe._aligned(dy=dy, dx=dx, dlogits=dlogits, dw13=dw13, dw2=dw2)
        if self._reads(stream, dy) != on:
            self._reads(stream, x)
        offsets, (codes, scales) = self.views[buf]["offsets"], self.kept[buf]
        p.scatter(dy, self.d_rows, self.row_gates, buf=buf, stream=stream)
        hg = self.h  # the forward's h has been read
        ex.down_backward(self.d_rows, codes, scales, self.row_gates, offsets, self.dgu, hg, self.parts, rows=n,
                         stream=stream)
        ex.down_grad(self.d_rows, hg, offsets, dw2, accumulate, rows=n, stream=stream)
        ex.up_backward(self.dgu, offsets, self.d_rows, rows=n, stream=stream)  # d_rows now by x's side
        p.scatter(x, self.x_rows, buf=buf, stream=stream)
        ex.up_grad(self.dgu, self.x_rows, offsets, dw13, accumulate, rows=n, stream=stream)
        p.gather(T, self.d_rows, dx, buf=buf, stream=stream)
        dgates = self.dgates if T == p.T_max else self.dgates[:T]
        p.gates_backward(T, self.parts, dgates, dlogits, self.router, logits, buf=buf, stream=stream)
        self.saved[buf] = None
        return dx, dlogits

    def _reads(self, stream, *tensors):
        """``stream`` (None: the current one) reads these: their memory is not handed out again before it has,
        even if the layer's is the last reference and is let go of while that work is still queued.  Returns the
        stream's handle."""
        on = moe._stream(stream)
        s = stream
        if s is None and (s := self._streams.get(on)) is None:  # a torch Stream takes as long to make as a call
            s = self._streams[on] = torch.cuda.current_stream()
        for t in tensors:
            t.record_stream(s)
        return on

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


def random_dense(P, H, I, seed=0, device="cuda"):
    """bf16 weights w13 [P, 2 I, H] and w2 [P, H, I], N(0, 1 / inputs)."""
    g = torch.Generator(device)
    g.manual_seed(seed)

    def one(n, k):
        w = torch.empty(P, n, k, dtype=torch.bfloat16, device=device)
        for p in range(P):
            w[p] = torch.randn(n, k, generator=g, device=device) * k ** -0.5
        return w

    return one(2 * I, H), one(H, I)


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, value in (("tokens", 96), ("hidden", 7168), ("inner", 2048), ("experts", 256), ("topk", 8), ("groups", 8),
                        ("steps", 20)):
        ap.add_argument("--" + name, type=int, default=value)
    ap.add_argument("--train", action="store_true", help="time a TrainingLayer")
    a = ap.parse_args(argv)
    router = moe.Router("sigmoid", n_group=a.groups, topk_group=max(1, a.groups // 2), group_top=2, scale=2.5)
    bias = torch.zeros(a.experts, device="cuda")
    if not a.train:
        layer = ExpertLayer(random_experts(a.experts, a.hidden, a.inner), a.tokens, a.experts, a.topk, router, bias=bias)
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

    rows = a.tokens * a.topk
    what = f"{a.tokens} tokens x {a.hidden}, {a.experts} experts of {a.inner}, top-{a.topk} ({rows} rows)"
    if a.train:
        w13, w2 = random_dense(a.experts, a.hidden, a.inner)
        layer = TrainingLayer(w13, w2, a.tokens, a.experts, a.topk, router, bias)
        dw13, dw2 = torch.empty_like(w13, dtype=torch.float32), torch.empty_like(w2, dtype=torch.float32)
        dx, dlogits, dy = torch.empty_like(x), torch.empty_like(logits), torch.randn_like(x)
        forward = timed(lambda: layer.forward(x, logits, y))

        def both():
            layer.forward(x, logits, y)
            layer.backward(dy, dw13, dw2, dx, dlogits)

        step = timed(both)
        if layer.check():
            raise RuntimeError("device error word set")
        flops = 18.0 * rows * a.hidden * a.inner  # three products of 6 a row and pair of sizes
        print(f"{what}: forward {forward:.1f} us, backward {step - forward:.1f} us, {flops / step / 1e6:.0f} TFLOP/s")
        return
    calls = timed(lambda: layer(x, logits, y))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer(x, logits, y)
    replay = timed(graph.replay)
    if layer.check():
        raise RuntimeError("device error word set")
    print(f"{what}: {calls:.1f} us a layer call by call, {replay:.1f} us as a graph")


if __name__ == "__main__":
    main()
