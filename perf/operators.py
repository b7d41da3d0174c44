"""The expert layer's operators as measured workloads: routing with its
placement, the 8-bit floating-point dispatch, and the experts' two grouped
products, each in a plain form (elementary torch operations in 32 bits) and
through the library.

``own`` chooses the side: False computes the plain form, True makes the
library's calls.  Both start from the same tensors, drawn by ``prepare`` from
the seed alone; the library's side also keeps a pool or a weights handle, as a
serving program does.

Operators (field ``op`` of a case):

plan      router scores (sigmoid or softmax) with a balance bias, the best
          groups of experts, top-k, renormalised gates, and the placement of
          every copy in its expert's window.
dispatch  each token quantised to E4M3 codes with one fp32 scale per 128
          elements and written into its k slot rows.
up        h = E4M3(silu(rows w_gate^T) * (rows w_up^T)) per expert window;
          codes and weights E4M3, scales per 128 (rows) and 128 x 128 (weights).
down      out = bf16(h w2^T) per expert window, same formats.
"""
from __future__ import annotations

import math

import torch

own = False

_DEV = "cuda"
_F8 = torch.float8_e4m3fn
_TOP = 448.0  # largest E4M3 value


# ---------------------------------------------------------------- the cases

def _plan(name, T, E, P, k, score, n_group, topk_group, group_top, bias, renorm, scale):
    return {"name": name, "op": "plan", "T": T, "E": E, "P": P, "k": k, "score": score, "n_group": n_group,
            "topk_group": topk_group, "group_top": group_top, "bias": bias, "renorm": renorm, "scale": scale}


def _rows(name, op, T, H, E, P, k, inter):
    return {"name": name, "op": op, "T": T, "H": H, "E": E, "P": P, "k": k, "I": inter}


def listed():
    return [
        # One user's next token: launch latency is all there is.
        _plan("plan_t1", 1, 256, 256, 8, "sigmoid", 8, 4, 2, True, True, 2.5),
        # A prefill chunk with redundant experts, the benchmark's batch.
        _plan("plan_t4096", 4096, 256, 288, 8, "sigmoid", 8, 4, 2, True, True, 2.5),
        # A long prefill with few experts, plain softmax scores, no groups.
        _plan("plan_t16384", 16384, 64, 64, 6, "softmax", 1, 1, 1, False, False, 1.0),
        # One decode batch of a serving rank.
        _rows("dispatch_t96", "dispatch", 96, 7168, 256, 256, 8, 0),
        # The prefill chunk: bandwidth.
        _rows("dispatch_t4096", "dispatch", 4096, 7168, 256, 288, 8, 0),
        # One user's next token: eight experts' weights pass by for a row each.
        _rows("up_t1", "up", 1, 7168, 256, 256, 8, 2048),
        # One decode batch: nearly every expert's weights, a few rows each.
        _rows("up_t96", "up", 96, 7168, 256, 256, 8, 2048),
        # The prefill chunk: about 114 rows an expert, weights still the larger part.
        _rows("up_t4096", "up", 4096, 7168, 256, 288, 8, 2048),
        # A long prefill with few experts: about 1536 rows each, the tensor cores' case.
        _rows("up_t16384", "up", 16384, 2048, 64, 64, 6, 1024),
        _rows("down_t96", "down", 96, 7168, 256, 256, 8, 2048),
        # Odd counts everywhere, sizes that end inside a tile.
        _rows("down_t1537_odd", "down", 1537, 1920, 40, 44, 5, 896),
        _rows("down_t16384", "down", 16384, 2048, 64, 64, 6, 1024),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["plan", "dispatch", "up", "down"])
    if op == "plan":
        n_group, size = rng.choice([(1, 8), (1, 23), (4, 8), (1, 64), (4, 16), (8, 8), (6, 16), (8, 20), (1, 160),
                                    (8, 32), (16, 16)])
        E = n_group * size
        topk_group = 1 if n_group == 1 else rng.randint(1, n_group)
        k = rng.randint(1, min(8, topk_group * size, E))
        score = rng.choice(["sigmoid", "softmax"])
        return {"op": op, "T": _log_int(rng, 1, 16384), "E": E, "P": E + rng.randint(0, E // 8), "k": k,
                "score": score, "n_group": n_group, "topk_group": topk_group, "group_top": rng.choice([1, 2]),
                "bias": rng.random() < 0.5, "renorm": rng.random() < 0.7, "scale": rng.choice([1.0, 2.5])}
    E = _log_int(rng, 4, 256)
    k = rng.randint(1, min(8, E))
    P = E + rng.randint(0, E // 8)
    H = 128 * (2 * _log_int(rng, 1, 27) + 1)  # an odd number of groups
    if op == "dispatch":
        return {"op": op, "T": _log_int(rng, 1, 4096), "H": H, "E": E, "P": P, "k": k, "I": 0}
    inter = 128 * rng.choice([1, 2, 3, 4, 5, 7, 8, 9, 11, 13, 16])
    # no more rows and products than the largest listed case of the kind
    T = _log_int(rng, 1, 16384)
    per_row = 4.0 * inter * H if op == "up" else 2.0 * inter * H
    T = max(1, min(T, int(8.0e11 / (per_row * k))))
    return {"op": op, "T": T, "H": H, "E": E, "P": P, "k": k, "I": inter}


def _active(case):
    """Experts that get a row, on average over even routing."""
    E, P, k, T = case["E"], case["P"], case["k"], case["T"]
    return P * (1.0 - (1.0 - k / E * (E / P)) ** T)


def work(case):
    T, E, P, k = case["T"], case["E"], case["P"], case["k"]
    n = T * k
    if case["op"] == "plan":
        # logits (and bias) read; ids, gates, physical ids, slots and both inverse maps written
        return {"bytes": 4.0 * (T * E + (E if case["bias"] else 0) + 6 * n + 2 * P + 1), "flops": 8.0 * T * E}
    H, inter = case["H"], case["I"]
    if case["op"] == "dispatch":
        return {"bytes": 2.0 * T * H + n * (H + 4.0 * (H // 128)) + 4.0 * n, "flops": 4.0 * T * H}
    a = _active(case)
    if case["op"] == "up":
        w = a * 2 * inter * (H + 4.0 * (H // 128) / 128)
        return {"bytes": w + n * (H + 4.0 * (H // 128)) + n * (inter + 4.0 * (inter // 128)) + 4.0 * (P + 1),
                "flops": 4.0 * n * inter * H}
    w = a * H * (inter + 4.0 * (inter // 128) / 128)
    return {"bytes": w + n * (inter + 4.0 * (inter // 128)) + 2.0 * n * H + 4.0 * (P + 1),
            "flops": 2.0 * n * inter * H}


# ---------------------------------------------------------------- the inputs

def _generator(seed):
    g = torch.Generator(device=_DEV)
    g.manual_seed(int(seed))
    return g


def _replica_map(popularity, P):
    """CSR replica map: each of the P - E most popular experts has a second
    slot.  (None, None) where P equals E."""
    E = popularity.numel()
    if P == E:
        return None, None
    hot = torch.sort(popularity, descending=True, stable=True).indices[:P - E]
    n = torch.ones(E, dtype=torch.int64, device=_DEV)
    n[hot] = 2
    off = torch.zeros(E + 1, dtype=torch.int64, device=_DEV)
    off[1:] = n.cumsum(0)
    ids = torch.empty(P, dtype=torch.int64, device=_DEV)
    ids[off[:-1]] = torch.arange(E, device=_DEV)
    ids[off[hot] + 1] = E + torch.arange(P - E, device=_DEV)
    return off.int(), ids.int()


def _place(topk, rep_off, rep_ids, P):
    """Physical expert, slot, inverse maps, counts and offsets of the copies:
    a stable counting sort by (expert, token)."""
    T, k = topk.shape
    if rep_off is None:
        phys = topk
    else:
        lo = rep_off.long()[topk]
        n = rep_off.long()[topk + 1] - lo
        phys = rep_ids.long()[lo + torch.arange(T, device=_DEV)[:, None] % n]
    flat = phys.reshape(-1)
    order = torch.sort(flat, stable=True).indices
    slot = torch.empty_like(order)
    slot[order] = torch.arange(T * k, device=_DEV)
    counts = torch.zeros(P, dtype=torch.int64, device=_DEV).index_add_(0, flat, torch.ones_like(flat))
    offsets = torch.zeros(P + 1, dtype=torch.int64, device=_DEV)
    offsets[1:] = counts.cumsum(0)
    return {"phys": phys.int(), "slot": slot.reshape(T, k).int(), "counts": counts.int(), "offsets": offsets.int(),
            "src_token": (order // k).int(), "src_k": (order % k).int()}


def _logits(g, T, E, spread):
    """Router logits: N(0, 1), with some experts liked more than others."""
    popularity = spread * torch.randn(E, generator=g, device=_DEV)
    return torch.randn(T, E, generator=g, device=_DEV) + popularity, popularity


def _quantise_rows(v):
    """E4M3 codes and fp32 scales of rows of 128-element groups: scale =
    max|v| / 448, code = v * 448 / max|v| (a group of zeros: scale 0, codes 0)."""
    rows, n = v.shape
    grouped = v.reshape(rows, n // 128, 128)
    amax = grouped.abs().amax(-1, keepdim=True)
    codes = (grouped * _TOP / torch.where(amax > 0, amax, 1.0)).to(_F8)
    return codes.reshape(rows, n), (amax / _TOP).reshape(rows, n // 128)


def _weights(g, P, N, K):
    """Expert weights [P, N, K], E4M3 with one fp32 scale per 128 x 128 block."""
    codes = torch.empty(P, N, K, dtype=_F8, device=_DEV)
    scales = torch.empty(P, N // 128, K // 128, device=_DEV)
    for p in range(P):
        w = torch.randn(N, K, generator=g, device=_DEV).mul_(K ** -0.5).reshape(N // 128, 128, K // 128, 128)
        amax = w.abs().amax((1, 3), keepdim=True)
        codes[p] = w.mul_(_TOP / amax).reshape(N, K).to(_F8)
        scales[p] = amax.reshape(N // 128, K // 128) / _TOP
    return codes, scales


def _padded_stride(groups):
    """Floats per row of a scale array: the pool's rows of scales are multiples of 16 bytes."""
    return (groups + 3) // 4 * 4


def prepare(case, seed):
    g = _generator(seed)
    T, E, P, k = case["T"], case["E"], case["P"], case["k"]
    s = {"case": case}
    if case["op"] == "plan":
        # Half of the skew that the router has is taken back by the bias, which
        # training moves in steps of a thousandth.
        s["logits"], pop = _logits(g, T, E, 1.0)
        s["bias"] = (torch.round(-0.1 * pop * 1000) / 1000).contiguous() if case["bias"] else None
        s["rep_off"], s["rep_ids"] = _replica_map(pop, P)
        if own:
            from combine_moe_plan_gb300 import moe
            s["pool"] = moe.Pool(T, 128, E, P, k, n_sets=1)
            s["router"] = moe.Router(score=case["score"], n_group=case["n_group"], topk_group=case["topk_group"],
                                     group_top=case["group_top"], renorm=case["renorm"], scale=case["scale"])
            s["view"] = s["pool"].view(0)
        return s
    H, inter = case["H"], case["I"]
    logits, pop = _logits(g, T, E, 0.3)
    rep_off, rep_ids = _replica_map(pop, P)
    top = torch.sort(logits, dim=-1, descending=True, stable=True).indices[:, :k]
    placed = _place(top, rep_off, rep_ids, P)
    if case["op"] == "dispatch":
        # Activations with the occasional outlier.
        x = torch.randn(T, H, generator=g, device=_DEV)
        x = torch.where(torch.rand(T, H, generator=g, device=_DEV) < 0.001, 50 * x, x)
        s["x"], s["slot"] = x.bfloat16(), placed["slot"]
        if own:
            from combine_moe_plan_gb300 import moe
            s["pool"] = moe.Pool(T, H, E, P, k, n_sets=1)
            s["pool"].plan(logits, rep_off, rep_ids)
            s["view"] = s["pool"].view(0)
        return s
    n = T * k
    width = H if case["op"] == "up" else inter
    v = torch.randn(n, width, generator=g, device=_DEV)
    if case["op"] == "down":
        v = v * torch.randn(n, width, generator=g, device=_DEV)  # a gated product's tails
    s["codes"], scales = _quantise_rows(v)
    del v
    s["scales"] = torch.zeros(n, _padded_stride(width // 128), device=_DEV)
    s["scales"][:, :width // 128] = scales
    s["offsets"] = placed["offsets"]
    s["sizes"] = placed["counts"].tolist()
    if case["op"] == "up":
        s["w"], s["ws"] = _weights(g, P, 2 * inter, H)
        s["h"] = torch.empty(n, inter, dtype=_F8, device=_DEV)
        s["h_scales"] = torch.empty(n, _padded_stride(inter // 128), device=_DEV)
    else:
        s["w"], s["ws"] = _weights(g, P, H, inter)
        s["out"] = torch.empty(n, H, dtype=torch.bfloat16, device=_DEV)
    if own:
        from combine_moe_plan_gb300 import moe
        s["experts"] = moe.Experts(w13=s["w"], s13=s["ws"]) if case["op"] == "up" else moe.Experts(w2=s["w"], s2=s["ws"])
    return s


# ------------------------------------------------------------ the plain forms

def _scores(logits, score):
    if score == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-logits))
    e = torch.exp(logits - logits.amax(-1, keepdim=True))
    # a sum of up to a few hundred 32-bit terms whose rounding does not depend on their order
    return e / e.double().sum(-1, keepdim=True).to(logits.dtype)


def _select(scores, bias, case):
    """The k best experts of each token, best first: ties go to the lowest index."""
    T, E = scores.shape
    choice = scores if bias is None else scores + bias
    if case["n_group"] > 1:
        grouped = choice.reshape(T, case["n_group"], E // case["n_group"])
        best = torch.sort(grouped, dim=-1, descending=True, stable=True).values[..., :case["group_top"]].sum(-1)
        keep = torch.sort(best, dim=-1, descending=True, stable=True).indices[:, :case["topk_group"]]
        kept = torch.zeros_like(best, dtype=torch.bool).scatter_(1, keep, True)
        choice = torch.where(kept[..., None], grouped, -math.inf).reshape(T, E)
    return torch.sort(choice, dim=-1, descending=True, stable=True).indices[:, :case["k"]]


def _gates(scores, top, case):
    w = torch.gather(scores, 1, top)
    if case["renorm"]:
        w = w / w.sum(-1, keepdim=True)
    return w * case["scale"]


def _plain_plan(s):
    case = s["case"]
    scores = _scores(s["logits"], case["score"])
    top = _select(scores, s["bias"], case)
    return {"topk_e": top.int(), "gates": _gates(scores, top, case), **_place(top, s["rep_off"], s["rep_ids"], case["P"])}


def _plain_dispatch(s):
    codes, scales = _quantise_rows(s["x"].float())
    k = s["case"]["k"]
    slot = s["slot"].reshape(-1).long()
    out = torch.empty(slot.numel(), codes.shape[1], dtype=torch.uint8, device=codes.device)
    out[slot] = codes.view(torch.uint8).repeat_interleave(k, 0)
    out_scales = torch.empty(slot.numel(), scales.shape[1], device=codes.device)
    out_scales[slot] = scales.repeat_interleave(k, 0)
    return {"codes": out.view(_F8), "scales": out_scales}


def _plain_windows(s):
    """Each expert's window times its weights: (window, fp32 product) in turn.
    The windows are ragged, so the plain form takes them one by one."""
    width = s["codes"].shape[1]
    lo = 0
    for p, n in enumerate(s["sizes"]):
        if n:
            at = slice(lo, lo + n)
            rows = s["codes"][at].float() * s["scales"][at, :width // 128].repeat_interleave(128, 1)
            weights = s["w"][p].float() * s["ws"][p].repeat_interleave(128, 0).repeat_interleave(128, 1)
            yield at, rows @ weights.T
        lo += n


def _plain_up(s):
    inter = s["case"]["I"]
    scales = s["h_scales"][:, :inter // 128]
    for at, y in _plain_windows(s):
        gate, up = y[:, :inter], y[:, inter:]
        s["h"][at], scales[at] = _quantise_rows(gate / (1.0 + torch.exp(-gate)) * up)
    return {"h": s["h"], "scales": scales}


def _plain_down(s):
    for at, y in _plain_windows(s):
        s["out"][at] = y.bfloat16()
    return s["out"]


def run(s):
    op = s["case"]["op"]
    if not own:
        return {"plan": _plain_plan, "dispatch": _plain_dispatch, "up": _plain_up, "down": _plain_down}[op](s)
    if op == "plan":
        s["pool"].plan_routed(s["logits"], s["router"], s["bias"], s["rep_off"], s["rep_ids"])
        v = s["view"]
        return {name: v[name] for name in ("topk_e", "gates", "phys", "slot", "counts", "offsets", "src_token", "src_k")}
    if op == "dispatch":
        s["pool"].dispatch_f8(s["x"])
        return {"codes": s["view"]["codes_f8"], "scales": s["view"]["scales"][:, :s["case"]["H"] // 128]}
    if op == "up":
        s["experts"].up(s["codes"], s["scales"], s["offsets"], s["h"], s["h_scales"])
        return {"h": s["h"], "scales": s["h_scales"][:, :s["case"]["I"] // 128]}
    s["experts"].down(s["codes"], s["scales"], s["offsets"], s["out"])
    return s["out"]


# ------------------------------------------------------- the definitions, in 64 bits

def _exact_plan(s, case):
    x = s["logits"].double()
    if case["score"] == "sigmoid":
        p = torch.special.expit(x)
    else:
        p = torch.softmax(x, -1)
    c = p if s["bias"] is None else p + s["bias"].double()
    T, E = x.shape
    if case["n_group"] > 1:
        best = torch.topk(c.view(T, case["n_group"], -1), case["group_top"], dim=-1).values.sum(-1)
        cut = torch.topk(best, case["topk_group"], dim=-1).values[:, -1:]
        c = c.masked_fill((best < cut).repeat_interleave(E // case["n_group"], 1), -math.inf)
    gates = p.gather(1, torch.topk(c, case["k"], dim=-1).indices)
    if case["renorm"]:
        gates = gates / gates.sum(-1, keepdim=True)
    out = dict.fromkeys(("topk_e", "phys", "slot", "counts", "offsets", "src_token", "src_k"))
    out["gates"] = gates * case["scale"]
    return out


def _exact_dispatch(s):
    x = s["x"].double()
    T, H = x.shape
    amax = torch.linalg.vector_norm(x.view(T, -1, 128), math.inf, dim=-1)
    q = x * _TOP / amax.clamp_min(1e-300).repeat_interleave(128, 1)
    # to the nearest E4M3 value, ties to even: 2^-3 of the power of two below, not under 2^-9
    step = torch.exp2(torch.floor(torch.log2(q.abs().clamp_min(2.0 ** -6))) - 3)
    q = torch.round(q / step) * step
    token = torch.empty(s["slot"].numel(), dtype=torch.int64, device=_DEV)
    token[s["slot"].long().flatten()] = torch.arange(T, device=_DEV).repeat_interleave(s["slot"].shape[1])
    return {"codes": q[token], "scales": (amax / _TOP)[token]}


def _exact_product(s, lo, hi, p):
    a = s["codes"][lo:hi].double()
    a = a * torch.repeat_interleave(s["scales"][lo:hi, :a.shape[1] // 128].double(), 128, 1)
    w = s["w"][p].double()
    N, K = w.shape
    w = (w.view(N // 128, 128, K // 128, 128) * s["ws"][p].double()[:, None, :, None]).reshape(N, K)
    return torch.einsum("mk,nk->mn", a, w)


def exact(case, seed):
    if case["op"] in ("up", "down") and work(case)["flops"] > 6e12:
        return None
    s = prepare(case, seed)
    if case["op"] == "plan":
        return _exact_plan(s, case)
    if case["op"] == "dispatch":
        return _exact_dispatch(s)
    n = s["codes"].shape[0]
    edges = s["offsets"].tolist()
    if case["op"] == "down":
        out = torch.zeros(n, case["H"], dtype=torch.float64, device=_DEV)
        for p, (lo, hi) in enumerate(zip(edges, edges[1:])):
            if hi > lo:
                out[lo:hi] = _exact_product(s, lo, hi, p)
        return out
    inter = case["I"]
    h = torch.zeros(n, inter, dtype=torch.float64, device=_DEV)
    scales = torch.zeros(n, inter // 128, dtype=torch.float64, device=_DEV)
    for p, (lo, hi) in enumerate(zip(edges, edges[1:])):
        if hi > lo:
            y = _exact_product(s, lo, hi, p)
            v = (torch.special.expit(y[:, :inter]) * y[:, :inter] * y[:, inter:]).view(hi - lo, inter // 128, 128)
            amax = v.abs().amax(-1, keepdim=True)
            # the codes before their rounding to E4M3
            h[lo:hi] = (v * _TOP / amax).view(hi - lo, inter)
            scales[lo:hi] = amax[..., 0] / _TOP
    return {"h": h, "scales": scales}
