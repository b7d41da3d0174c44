"""Training an expert layer: its operators as measured workloads, each in a
plain form (elementary torch operations in 32 bits) and through the library.

``own`` chooses the side: False computes the plain form, True makes the
library's calls.  Both start from the same tensors, drawn by ``prepare`` from
the seed alone; the library's side also keeps a pool or a weights handle, as a
training program does.

Rows are copies of tokens in expert windows (expert p's rows are offsets[p] ..
offsets[p + 1] - 1), weights are bf16: w13 [P, 2 I, H], gate rows before up rows,
and w2 [P, H, I].  Operators (field ``op`` of a case):

scatter      rows[slot[t, j]] = x[t], and each row's gate beside it.
gather       y[t] = bf16(sum over j of rows[slot[t, j]]): the gradient of scatter.
up           g, u = rows gate^T, rows up^T; h = bf16(silu(g) u), and g and u kept
             for the backward pass as E4M3 codes with an fp32 scale per 128.
product      a grouped product by itself: "forward" h w2^T, "backward" dgu w13.
down_back    from the gradient of the experts' outputs and the codes of g and u:
             d = dout w2, the rows' gates' gradients by 128 columns (sum of d h),
             hg = bf16(gate h) and dgu, the gradients of g and u.
weight_grad  dw[p] = a^T b over the rows of window p: "up" (dgu, rows) or "down"
             (dout, hg), in fp32 or bf16.
gates_back   the gates' gradients summed per copy, and through the router (a
             softmax over the chosen logits, or scores over all experts) to the logits.
"""
from __future__ import annotations

import math

import torch

own = False

_DEV = "cuda"
_F8 = torch.float8_e4m3fn
_TOP = 448.0  # largest E4M3 value


# ---------------------------------------------------------------- the cases

def _case(name, op, T, H, I, E, P, k, kind=""):
    return {"name": name, "op": op, "T": T, "H": H, "I": I, "E": E, "P": P, "k": k, "kind": kind}


def listed():
    return [
        # A small batch's rows: launch latency.
        _case("scatter_t96", "scatter", 96, 7168, 0, 256, 256, 8),
        # The benchmark's batch with its redundant experts: bandwidth.
        _case("gather_t4096", "gather", 4096, 7168, 0, 256, 288, 8),
        # One token through bf16 experts (a forward without a batch): eight experts' weights pass by.
        _case("up_t1", "up", 1, 7168, 2048, 256, 256, 8),
        # A long training batch over the experts of one rank: the tensor cores' case.
        _case("up_t16384", "up", 16384, 2048, 1024, 64, 64, 6),
        # The decode batch: nearly every expert's weights, a few rows each.
        _case("down_t96", "product", 96, 7168, 2048, 256, 256, 8, "forward"),
        # The rows' gradient of the long batch.
        _case("up_back_t16384", "product", 16384, 2048, 1024, 64, 64, 6, "backward"),
        # Odd counts everywhere, sizes that end inside a tile.
        _case("down_back_t1537_odd", "down_back", 1537, 1920, 896, 40, 44, 5),
        _case("down_back_t16384", "down_back", 16384, 2048, 1024, 64, 64, 6),
        # A few hundred rows an expert, gradients kept in bf16.
        _case("down_grad_t1537_odd", "weight_grad", 1537, 1920, 896, 40, 44, 5, "down bf16"),
        # The largest gradient of the long batch, in fp32.
        _case("up_grad_t16384", "weight_grad", 16384, 2048, 1024, 64, 64, 6, "up fp32"),
        # The plan's own gates, one decode batch.
        _case("gates_back_t96", "gates_back", 96, 0, 2048, 256, 256, 8, "plan"),
        # Softmax scores over all experts, the long batch.
        _case("gates_back_t16384", "gates_back", 16384, 0, 1024, 64, 64, 6, "softmax"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


_KINDS = {"scatter": [""], "gather": [""], "up": [""], "product": ["forward", "backward"], "down_back": [""],
          "weight_grad": ["up fp32", "down fp32", "up bf16", "down bf16"],
          "gates_back": ["plan", "sigmoid", "sigmoid renormalised", "softmax", "softmax renormalised"]}


def draw(rng):
    op = rng.choice(sorted(_KINDS))
    kind = rng.choice(_KINDS[op])
    E = _log_int(rng, 4, 256)
    k = rng.randint(1, min(8, E))
    P = E + rng.randint(0, E // 8)
    H = 128 * _log_int(rng, 1, 56)
    inter = 128 * rng.choice([1, 2, 3, 4, 5, 7, 8, 9, 11, 13, 16])
    T = _log_int(rng, 1, 16384)
    if op == "gates_back":
        if kind == "plan" or kind.endswith("renormalised"):
            k = max(k, 2)  # one gate of a token is a constant
        return _drawn(op, T, 0, inter, E, E, k, kind)
    if op in ("scatter", "gather"):
        return _drawn(op, max(1, min(T, 4096 * 7168 * 9 // (H * (k + 1)))), H, 0, E, P, k, kind)
    # no more products, weights or gradients than the largest listed case of the kind
    T = max(1, min(T, int(8.0e11 / (4.0 * H * inter * k))))
    E = max(k, min(E, int((2.6e8 if op == "weight_grad" else 3.2e9) / (2.0 * H * inter))))
    P = E + min(P - E, E // 8)
    return _drawn(op, T, H, inter, E, P, k, kind)


def _drawn(op, T, H, inter, E, P, k, kind):
    c = _case("", op, T, H, inter, E, P, k, kind)
    del c["name"]
    return c


def _active(case):
    """Experts that get a row, on average over even routing."""
    E, P, k, T = case["E"], case["P"], case["k"], case["T"]
    return P * (1.0 - (1.0 - k / E * (E / P)) ** T)


def work(case):
    T, H, inter, E, P, k, op = (case[f] for f in ("T", "H", "I", "E", "P", "k", "op"))
    n, a = T * k, _active(case)
    if op == "scatter":
        return {"bytes": 2.0 * T * H + 2.0 * n * H + 12.0 * n, "flops": 0.0}
    if op == "gather":
        return {"bytes": 2.0 * n * H + 2.0 * T * H + 4.0 * n, "flops": 1.0 * n * H}
    if op == "gates_back":
        logits = 0 if case["kind"] == "plan" else 4.0 * T * E
        return {"bytes": 4.0 * n * (inter // 128) + logits + 4.0 * T * E + 16.0 * n,
                "flops": 1.0 * n * (inter // 128) + 4.0 * T * E}
    up, scales = 2.0 * inter * H, 4.0 * 2 * inter / 128
    if op == "up":
        return {"bytes": 2.0 * a * up + n * (2.0 * H + 2.0 * inter + 2.0 * inter + scales) + 4.0 * (P + 1),
                "flops": 2.0 * n * up}
    if op == "product":
        wide, w = (2, up) if case["kind"] == "backward" else (1, up / 2)
        return {"bytes": 2.0 * a * w + 2.0 * n * (wide * inter + H) + 4.0 * (P + 1), "flops": 2.0 * n * w}
    if op == "down_back":
        return {"bytes": a * up + n * (2.0 * H + 2.0 * inter + scales + 4.0 + 6.0 * inter + 4.0 * (inter // 128)) +
                4.0 * (P + 1), "flops": n * up}
    wide = 2 if case["kind"].startswith("up") else 1
    size = 4.0 if case["kind"].endswith("fp32") else 2.0
    return {"bytes": 2.0 * n * (wide * inter + H) + size * P * wide * inter * H + 4.0 * (P + 1),
            "flops": 2.0 * n * wide * inter * H}


# ---------------------------------------------------------------- the inputs

def _generator(seed):
    g = torch.Generator(device=_DEV)
    g.manual_seed(int(seed))
    return g


def _routing(g, case):
    """Router logits with some experts liked more than others, and what the plan
    makes of them: chosen experts, slots, window sizes.  The logits of a token
    are at least 2^-14 apart, so that rounded scores choose the same experts.
    Each of the P - E most liked experts has a second slot."""
    T, E, P, k = case["T"], case["E"], case["P"], case["k"]
    liked = 0.3 * torch.randn(E, generator=g, device=_DEV)
    logits = torch.round((torch.randn(T, E, generator=g, device=_DEV) + liked) * 64) / 64
    logits = logits + torch.arange(E, device=_DEV) * 2.0 ** -14
    top = torch.sort(logits, dim=-1, descending=True, stable=True).indices[:, :k]
    s = {"logits": logits, "top": top, "rep_off": None, "rep_ids": None}
    phys = top
    if P > E:
        hot = torch.sort(liked, descending=True, stable=True).indices[:P - E]
        n = torch.ones(E, dtype=torch.int64, device=_DEV)
        n[hot] = 2
        off = torch.zeros(E + 1, dtype=torch.int64, device=_DEV)
        off[1:] = n.cumsum(0)
        ids = torch.empty(P, dtype=torch.int64, device=_DEV)
        ids[off[:-1]] = torch.arange(E, device=_DEV)
        ids[off[hot] + 1] = E + torch.arange(P - E, device=_DEV)
        phys = ids[off[top] + torch.arange(T, device=_DEV)[:, None] % n[top]]
        s["rep_off"], s["rep_ids"] = off.int(), ids.int()
    flat = phys.reshape(-1)
    order = torch.sort(flat, stable=True).indices
    slot = torch.empty_like(order)
    slot[order] = torch.arange(T * k, device=_DEV)
    counts = torch.zeros(P, dtype=torch.int64, device=_DEV).index_add_(0, flat, torch.ones_like(flat))
    offsets = torch.zeros(P + 1, dtype=torch.int64, device=_DEV)
    offsets[1:] = counts.cumsum(0)
    s["slot"], s["offsets"], s["sizes"] = slot.reshape(T, k), offsets.int(), counts.tolist()
    # softmax over the chosen logits, as moe_plan's gates
    s["gates"] = torch.softmax(torch.gather(logits, 1, top).double(), -1).float()
    return s


def _normal(g, *shape, scale=1.0):
    return (scale * torch.randn(*shape, generator=g, device=_DEV)).bfloat16()


def _weights(g, P, N, K):
    w = torch.empty(P, N, K, dtype=torch.bfloat16, device=_DEV)
    for p in range(P):
        w[p] = torch.randn(N, K, generator=g, device=_DEV) * K ** -0.5
    return w


def _stride(groups):
    """Floats per row of a scale array: whole 16 bytes."""
    return (groups + 3) // 4 * 4


def _quantise(v):
    """E4M3 codes and fp32 scales of rows of 128-element groups: scale = max|v| /
    448, code = v * 448 / max|v| (a group of zeros: scale 0, codes 0)."""
    rows, n = v.shape
    grouped = v.reshape(rows, n // 128, 128)
    amax = grouped.abs().amax(-1, keepdim=True)
    codes = (grouped * _TOP / torch.where(amax > 0, amax, 1.0)).to(_F8)
    return codes.reshape(rows, n), (amax / _TOP).reshape(rows, n // 128)


def prepare(case, seed):
    g = _generator(seed)
    T, H, inter, P, k, op = (case[f] for f in ("T", "H", "I", "P", "k", "op"))
    s = {"case": case, **_routing(g, case)}
    n = T * k
    if own:
        from combine_moe_plan_gb300 import moe
    if op in ("scatter", "gather", "gates_back"):
        if op == "scatter":
            s["x"] = _normal(g, T, H)
            s["rows"] = torch.empty(n, H, dtype=torch.bfloat16, device=_DEV)
            s["row_gates"] = torch.empty(n, device=_DEV)
        elif op == "gather":
            s["rows"] = _normal(g, n, H)
            s["y"] = torch.empty(T, H, dtype=torch.bfloat16, device=_DEV)
        else:
            s["parts"] = 0.1 * torch.randn(n, inter // 128, generator=g, device=_DEV)
            s["dgates"] = torch.empty(T, k, device=_DEV)
            s["dlogits"] = torch.empty(T, case["E"], device=_DEV)
        if own:
            s["pool"] = moe.Pool(T, H or 128, case["E"], P, k, n_sets=1)
            s["router"] = None
            if op == "gates_back" and case["kind"] != "plan":
                s["router"] = moe.Router(score=case["kind"].split()[0], renorm=case["kind"].endswith("renormalised"),
                                         scale=2.5)
                s["pool"].plan_routed(s["logits"], s["router"])
            else:
                s["pool"].plan(s["logits"], s["rep_off"], s["rep_ids"])
        return s
    w13 = w2 = None
    if op == "up":
        s["x"], w13 = _normal(g, n, H), _weights(g, P, 2 * inter, H)
        s["h"] = torch.empty(n, inter, dtype=torch.bfloat16, device=_DEV)
        s["codes"] = torch.empty(n, 2 * inter, dtype=_F8, device=_DEV)
        s["scales"] = torch.empty(n, _stride(2 * inter // 128), device=_DEV)
    elif op == "product" and case["kind"] == "forward":
        s["a"], w2 = _normal(g, n, inter, scale=0.5), _weights(g, P, H, inter)
        s["out"] = torch.empty(n, H, dtype=torch.bfloat16, device=_DEV)
    elif op == "product":
        s["a"], w13 = _normal(g, n, 2 * inter, scale=0.01), _weights(g, P, 2 * inter, H)
        s["out"] = torch.empty(n, H, dtype=torch.bfloat16, device=_DEV)
    elif op == "down_back":
        s["dout"], w2 = _normal(g, n, H, scale=0.01), _weights(g, P, H, inter)
        codes, scales = _quantise(torch.randn(n, 2 * inter, generator=g, device=_DEV))
        s["codes"] = codes
        s["scales"] = torch.zeros(n, _stride(2 * inter // 128), device=_DEV)
        s["scales"][:, :2 * inter // 128] = scales
        s["row_gates"] = torch.empty(n, device=_DEV)
        s["row_gates"][s["slot"].reshape(-1)] = s["gates"].reshape(-1)
        s["dgu"] = torch.empty(n, 2 * inter, dtype=torch.bfloat16, device=_DEV)
        s["hg"] = torch.empty(n, inter, dtype=torch.bfloat16, device=_DEV)
        s["parts"] = torch.empty(n, inter // 128, device=_DEV)
    else:
        kind = torch.float32 if case["kind"].endswith("fp32") else torch.bfloat16
        if case["kind"].startswith("up"):
            s["a"], s["b"] = _normal(g, n, 2 * inter, scale=0.01), _normal(g, n, H)
        else:
            s["a"], s["b"] = _normal(g, n, H, scale=0.01), _normal(g, n, inter, scale=0.5)
        s["dw"] = torch.empty(P, s["a"].shape[1], s["b"].shape[1], dtype=kind, device=_DEV)
    if own:
        s["experts"] = moe.DenseExperts(w13=w13, w2=w2) if w13 is not None or w2 is not None else \
            moe.DenseExperts(sizes=(P, H, inter))
    s["w"] = w13 if w13 is not None else w2
    return s


# ------------------------------------------------------------ the plain forms

def _windows(s):
    """The experts that have rows, with their rows."""
    lo = 0
    for p, n in enumerate(s["sizes"]):
        if n:
            yield p, slice(lo, lo + n)
        lo += n


def _plain_scatter(s):
    k = s["case"]["k"]
    at = s["slot"].reshape(-1)
    s["rows"][at] = s["x"].repeat_interleave(k, 0)
    s["row_gates"][at] = s["gates"].reshape(-1)
    return {"rows": s["rows"], "row_gates": s["row_gates"]}


def _plain_gather(s):
    acc = s["rows"][s["slot"][:, 0]].float()
    for j in range(1, s["case"]["k"]):
        acc = acc + s["rows"][s["slot"][:, j]].float()
    s["y"].copy_(acc)
    return s["y"]


def _plain_up(s):
    inter = s["case"]["I"]
    scales = s["scales"][:, :2 * inter // 128]
    for p, at in _windows(s):
        y = s["x"][at].float() @ s["w"][p].float().T
        gate, up = y[:, :inter], y[:, inter:]
        s["h"][at] = (gate / (1.0 + torch.exp(-gate)) * up).bfloat16()
        s["codes"][at], scales[at] = _quantise(y)
    return {"h": s["h"], "codes": s["codes"], "scales": scales}


def _plain_product(s):
    for p, at in _windows(s):
        w = s["w"][p].float()
        s["out"][at] = (s["a"][at].float() @ (w.T if s["case"]["kind"] == "forward" else w)).bfloat16()
    return s["out"]


def _plain_down_back(s):
    inter = s["case"]["I"]
    for p, at in _windows(s):
        d = s["dout"][at].float() @ s["w"][p].float()
        v = s["codes"][at].float() * s["scales"][at, :2 * inter // 128].repeat_interleave(128, 1)
        g, u = v[:, :inter], v[:, inter:]
        gate = s["row_gates"][at, None]
        sig = 1.0 / (1.0 + torch.exp(-g))
        h = g * sig * u
        s["parts"][at] = (d * h).reshape(-1, inter // 128, 128).sum(-1)
        s["hg"][at] = (gate * h).bfloat16()
        dh = gate * d
        s["dgu"][at, :inter] = (dh * u * sig * (1.0 + g * (1.0 - sig))).bfloat16()
        s["dgu"][at, inter:] = (dh * g * sig).bfloat16()
    return {"dgu": s["dgu"], "hg": s["hg"], "parts": s["parts"]}


def _plain_weight_grad(s):
    lo = 0
    for p, n in enumerate(s["sizes"]):
        s["dw"][p] = s["a"][lo:lo + n].float().T @ s["b"][lo:lo + n].float()
        lo += n
    return s["dw"]


def _plain_gates_back(s):
    kind, top = s["case"]["kind"], s["top"]
    s["dgates"].copy_(s["parts"][s["slot"]].sum(-1))
    dg = s["dgates"]
    s["dlogits"].zero_()
    if kind == "plan":
        g = s["gates"]
        s["dlogits"].scatter_(1, top, g * (dg - (g * dg).sum(-1, keepdim=True)))
        return {"dgates": dg, "dlogits": s["dlogits"]}
    x = s["logits"]
    if kind.startswith("sigmoid"):
        scores = 1.0 / (1.0 + torch.exp(-x))
    else:
        scores = torch.exp(x - x.amax(-1, keepdim=True))
        scores = scores / scores.sum(-1, keepdim=True)
    chosen = torch.gather(scores, 1, top)
    ds = 2.5 * dg
    if kind.endswith("renormalised"):
        total = chosen.sum(-1, keepdim=True)
        ds = (ds - (ds * chosen).sum(-1, keepdim=True) / total) / total
    if kind.startswith("sigmoid"):
        s["dlogits"].scatter_(1, top, ds * chosen * (1.0 - chosen))
    else:
        s["dlogits"].scatter_(1, top, ds)
        s["dlogits"].copy_(scores * (s["dlogits"] - (ds * chosen).sum(-1, keepdim=True)))
    return {"dgates": dg, "dlogits": s["dlogits"]}


_PLAIN = {"scatter": _plain_scatter, "gather": _plain_gather, "up": _plain_up, "product": _plain_product,
          "down_back": _plain_down_back, "weight_grad": _plain_weight_grad, "gates_back": _plain_gates_back}


def run(s):
    case = s["case"]
    op, kind, inter = case["op"], case["kind"], case["I"]
    if not own:
        return _PLAIN[op](s)
    if op == "scatter":
        s["pool"].scatter(s["x"], s["rows"], s["row_gates"])
        return {"rows": s["rows"], "row_gates": s["row_gates"]}
    if op == "gather":
        return s["pool"].gather(case["T"], s["rows"], s["y"])
    if op == "gates_back":
        logits = None if s["router"] is None else s["logits"]
        s["pool"].gates_backward(case["T"], s["parts"], s["dgates"], s["dlogits"], s["router"], logits)
        return {"dgates": s["dgates"], "dlogits": s["dlogits"]}
    ex = s["experts"]
    if op == "up":
        ex.up(s["x"], s["offsets"], s["h"], s["codes"], s["scales"])
        return {"h": s["h"], "codes": s["codes"], "scales": s["scales"][:, :2 * inter // 128]}
    if op == "product":
        return (ex.down if kind == "forward" else ex.up_backward)(s["a"], s["offsets"], s["out"])
    if op == "down_back":
        ex.down_backward(s["dout"], s["codes"], s["scales"], s["row_gates"], s["offsets"], s["dgu"], s["hg"], s["parts"])
        return {"dgu": s["dgu"], "hg": s["hg"], "parts": s["parts"]}
    return (ex.up_grad if kind.startswith("up") else ex.down_grad)(s["a"], s["b"], s["offsets"], s["dw"])


# ------------------------------------------------------- the definitions, in 64 bits

def _silu_and_slope(g):
    sig = torch.special.expit(g)
    return g * sig, sig + g * sig * torch.special.expit(-g)


def _exact_up(s, p, at, out):
    inter = s["case"]["I"]
    y = torch.einsum("rk,nk->rn", s["x"][at].double(), s["w"][p].double())
    out["h"][at] = _silu_and_slope(y[:, :inter])[0] * y[:, inter:]
    grouped = y.view(y.shape[0], -1, 128)
    top = torch.linalg.vector_norm(grouped, math.inf, dim=-1)
    out["scales"][at] = top / _TOP
    out["codes"][at] = (grouped * (_TOP / top)[..., None]).view_as(y)  # before their rounding to E4M3


def _exact_down_back(s, p, at, out):
    inter = s["case"]["I"]
    d = torch.einsum("rn,ni->ri", s["dout"][at].double(), s["w"][p].double())
    v = s["codes"][at].double().view(d.shape[0], -1, 128) * s["scales"][at, :2 * inter // 128].double()[..., None]
    g, u = v.flatten(1).split(inter, dim=1)
    h, slope = _silu_and_slope(g)
    gate = s["row_gates"][at].double()[:, None]
    out["parts"][at] = torch.einsum("rbi,rbi->rb", d.view(-1, inter // 128, 128), (h * u).view(-1, inter // 128, 128))
    out["hg"][at] = gate * h * u
    out["dgu"][at] = torch.cat([gate * d * u * slope, gate * d * h], 1)


def _exact_gates_back(s):
    """The logits' gradients by differentiating the gates, in 64 bits."""
    kind, top = s["case"]["kind"], s["top"]
    dg = s["parts"].double()[s["slot"]].sum(-1)
    x = s["logits"].double().requires_grad_()
    if kind == "plan":
        gates = torch.softmax(x.gather(1, top), -1)
    else:
        gates = (torch.sigmoid(x) if kind.startswith("sigmoid") else torch.softmax(x, -1)).gather(1, top)
        if kind.endswith("renormalised"):
            gates = gates / gates.sum(-1, keepdim=True)
        gates = 2.5 * gates
    return {"dgates": dg, "dlogits": torch.autograd.grad(gates, x, dg)[0]}


def exact(case, seed):
    if work(case)["flops"] > 6e12:
        return None
    s = prepare(case, seed)
    op, n, inter = case["op"], case["T"] * case["k"], case["I"]

    def like(*names):
        widths = {"scales": 2 * inter // 128}
        return {name: torch.zeros(n, widths.get(name, s[name].shape[1]), dtype=torch.float64, device=_DEV) for name in names}

    if op == "scatter":
        token = torch.empty(n, dtype=torch.int64, device=_DEV)
        token[s["slot"].flatten()] = torch.arange(n, device=_DEV)
        return {"rows": s["x"].double()[token // case["k"]], "row_gates":
                torch.softmax(s["logits"].double().gather(1, s["top"]), -1).flatten()[token]}
    if op == "gather":
        y = torch.zeros(case["T"], case["H"], dtype=torch.float64, device=_DEV)
        token = torch.arange(n, device=_DEV) // case["k"]
        return y.index_add_(0, token, s["rows"].double()[s["slot"].flatten()])
    if op == "gates_back":
        return _exact_gates_back(s)
    if op in ("up", "down_back"):
        out = like("h", "codes", "scales") if op == "up" else like("dgu", "hg", "parts")
        for p, at in _windows(s):
            (_exact_up if op == "up" else _exact_down_back)(s, p, at, out)
        return out
    if op == "product":
        out = like("out")["out"]
        for p, at in _windows(s):
            out[at] = torch.einsum("rk,nk->rn" if case["kind"] == "forward" else "rk,kn->rn", s["a"][at].double(),
                                   s["w"][p].double())
        return out
    dw = torch.zeros(s["dw"].shape, dtype=torch.float64, device=_DEV)
    for p, at in _windows(s):
        dw[p] = torch.einsum("rm,rn->mn", s["a"][at].double(), s["b"][at].double())
    return dw
