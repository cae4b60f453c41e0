"""Timed cases of what a layer of experts needs around its products.

Three operators with their gradients, each reached through the package's
tensor entry points:

  * run_route, run_route_grad: a token's experts and their weights from the
    router's logits, and the plan of rows sorted by expert that the ragged
    products take;
  * run_gather_rows, run_combine_rows, run_combine_rows_grad: tokens' rows into
    that order, and the experts' rows back, weighted and added to a residual;
  * run_grouped_act, run_grouped_act_grad: the experts' (or one dense) product
    with bias, activation, gate and residual in its epilogue.

How many rows each group holds follows from the case alone (so a case's work
does not depend on the seed); which group holds how many, and every value,
follow from the seed.
"""
from __future__ import annotations

import math
import random
import zlib

import numpy as np
import torch

own = False

# operands, outputs
_TYPES = {"bf16": (torch.bfloat16, torch.bfloat16), "bf16_f32": (torch.bfloat16, torch.float32),
          "f32": (torch.float32, torch.float32)}
_ACTS = ("none", "relu", "gelu", "silu", "gelu_tanh")


def _route(name, dtype, tokens, experts, top, scores, renorm, scale=1.0, bias=False, groups=1,
           top_groups=1, group_top=1, masked=0, op="route"):
    return {"name": name, "op": op, "dtype": dtype, "tokens": tokens, "experts": experts,
            "top": top, "scores": scores, "renorm": renorm, "scale": scale, "bias": bias,
            "groups": groups, "top_groups": top_groups, "group_top": group_top, "masked": masked}


def _move(name, op, dtype, tokens, top, experts, cols, weighted=True, residual=False):
    return {"name": name, "op": op, "dtype": dtype, "tokens": tokens, "top": top,
            "experts": experts, "cols": cols, "weighted": weighted, "residual": residual}


def _act(name, dtype, rows, groups, k, n, trans, act, gated, skew=0.0, bias=False, residual=False,
         keep=False):
    return {"name": name, "op": "act", "dtype": dtype, "rows": rows, "groups": groups, "k": k,
            "n": n, "trans": trans, "act": act, "gated": gated, "skew": skew, "bias": bias,
            "residual": residual, "keep": keep}


def listed():
    return [
        # one token decoding: two of eight experts
        _route("route_one_token", "bf16", 1, 8, 2, "softmax", True),
        # a decode batch padded to the size its graph was captured for
        _route("route_decode_padded", "f32", 96, 64, 4, "softmax", True, masked=13),
        # a prefill batch: many experts in groups, sigmoid scores, a bias that keeps them balanced
        _route("route_prefill_groups", "f32", 16384, 256, 8, "sigmoid", True, 2.5, True, 8, 4, 2),
        # training: the router's logits' gradient, an odd number of tokens
        _route("route_grad_odd", "bf16", 4099, 60, 4, "softmax", False, op="route_grad"),
        # a short prompt's rows to their experts, odd sizes in full precision
        _move("gather_short_prompt_odd", "gather", "f32", 509, 3, 16, 1537, weighted=False),
        # a prefill batch's rows back, added to the residual stream
        _move("combine_prefill", "combine", "bf16", 8192, 2, 8, 4096, residual=True),
        # training: the gradients of the experts' rows and of their weights
        _move("combine_grad", "combine_grad", "bf16", 4096, 4, 64, 2048),
        # one token's two experts of eight: their gated products, all weights read once
        _act("gated_one_token", "bf16", 2, 8, 2048, 1024, "T", "silu", True),
        # a decode batch of 96 tokens, four experts each, popular and idle experts
        _act("gated_decode_batch", "bf16", 384, 64, 4096, 1792, "T", "silu", True, skew=1.0),
        # a prefill batch: large products, as fast as the matrix cores go
        _act("gated_prefill", "bf16", 16384, 8, 4096, 14336, "T", "silu", True, skew=0.3),
        # a dense layer in full precision on odd sizes, with all that its epilogue has, training
        _act("dense_f32_odd", "f32", 1021, 1, 1023, 1537, "N", "gelu", False, bias=True,
             residual=True, keep=True),
        # training: the gradient of the gated activation and of the experts' biases
        {"name": "gated_grad", "op": "act_grad", "dtype": "bf16", "rows": 8192, "groups": 16,
         "n": 5632, "act": "silu", "gated": True, "skew": 0.5, "bias": True, "keep": True},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, lo, hi):
    # most widths are multiples of 64 or 8, the rest whatever they are
    v = _log_int(rng, lo, hi)
    step = rng.choice([64, 64, 8, 1])
    return max(lo, v // step * step)


def _draw_route(rng, op):
    experts = rng.choice([8, 16, 32, 60, 64, 128, 160, 256, 384, 512, rng.randint(2, 512)])
    tokens = _log_int(rng, 1, 16384)
    case = {"op": op, "dtype": rng.choice(["bf16", "f32"]), "tokens": tokens, "experts": experts,
            "top": rng.randint(1, min(experts, 10)), "scores": rng.choice(["softmax", "sigmoid"]),
            "renorm": rng.random() < 0.6, "scale": rng.choice([1.0, 1.0, 2.5]), "bias": False,
            "groups": 1, "top_groups": 1, "group_top": 1,
            "masked": rng.randint(0, tokens // 4) if rng.random() < 0.3 else 0}
    if op == "route":
        case["bias"] = rng.random() < 0.5
        if rng.random() < 0.5:
            groups = rng.choice([g for g in range(1, 17) if experts % g == 0 and experts // g >= 2]
                                or [1])
            least = -(-case["top"] // (experts // groups))     # groups that hold `top` experts
            case.update(groups=groups, top_groups=rng.randint(least, groups),
                        group_top=rng.choice([1, 2]))
    return case


def draw(rng: random.Random):
    top = work(listed()[9])
    while True:
        op = rng.choice(["route", "route", "route", "route_grad", "gather", "combine",
                         "combine_grad", "act", "act", "act", "act_grad"])
        dtype = rng.choice(["bf16", "bf16", "bf16_f32", "f32"])
        if op in ("route", "route_grad"):
            case = _draw_route(rng, op)
        elif op in ("gather", "combine", "combine_grad"):
            case = {"op": op, "tokens": _log_int(rng, 1, 8192), "top": rng.randint(1, 8),
                    "experts": rng.choice([8, 16, 64]), "cols": _width(rng, 128, 8192),
                    "dtype": dtype if op == "combine" else rng.choice(["bf16", "f32"]),
                    "weighted": op == "combine_grad" or rng.random() < 0.6,
                    "residual": op == "combine" and rng.random() < 0.6}
        else:
            dense = rng.random() < 0.25
            case = {"op": op, "dtype": dtype, "rows": _log_int(rng, 1, 16384),
                    "groups": 1 if dense else _log_int(rng, 2, 128), "n": _width(rng, 128, 14336),
                    "act": rng.choice(_ACTS), "gated": rng.random() < 0.6,
                    "skew": round(rng.uniform(0.0, 1.2), 2), "bias": rng.random() < 0.5,
                    "keep": rng.random() < 0.5}
            if op == "act":
                case.update(k=_width(rng, 128, 8192), trans=rng.choice(["N", "T", "T"]),
                            residual=rng.random() < 0.3)
        w = work(case)
        # an fp32 operation costs about ten bf16 ones
        cost = w["flops"] * (10 if case["dtype"] == "f32" else 1)
        if cost <= top["flops"] and w["bytes"] <= top["bytes"]:
            return case


def _sizes(case):
    text = repr(sorted((k, v) for k, v in case.items() if k != "name"))
    r = np.random.RandomState(zlib.crc32(text.encode()) & 0x7FFFFFFF)
    w = (1.0 + np.arange(case["groups"])) ** -case["skew"]
    return [int(x) for x in r.multinomial(case["rows"], w / w.sum())]


def work(case):
    op = case["op"]
    if op in ("route", "route_grad"):
        t, e, k = case["tokens"], case["experts"], case["top"]
        es = 4 if case["dtype"] == "f32" else 2
        if op == "route":      # logits and bias in; ids, weights, order, position and offsets out
            return {"bytes": t * e * es + (4 * e if case["bias"] else 0) + 16 * t * k + 4 * (e + 1),
                    "flops": 5 * t * e}
        return {"bytes": 2 * t * e * es + 8 * t * k, "flops": 8 * t * e}
    es, eo = (4, 4) if case["dtype"] == "f32" else (2, 2 if case["dtype"] == "bf16" else 4)
    if op in ("gather", "combine", "combine_grad"):
        t, k, n = case["tokens"], case["top"], case["cols"]
        plan = 4 * t * k * (2 if case["weighted"] else 1)
        if op == "gather":
            return {"bytes": t * n * es + t * k * n * es + plan,
                    "flops": t * k * n if case["weighted"] else 0}
        if op == "combine":
            return {"bytes": t * k * n * es + t * n * eo * (2 if case["residual"] else 1) + plan,
                    "flops": 2 * t * k * n}
        return {"bytes": t * n * es + 2 * t * k * n * es + plan + 4 * t * k, "flops": 3 * t * k * n}
    sizes = _sizes(case)
    rows, n = case["rows"], case["n"]
    busy, width = sum(1 for s in sizes if s), n * (2 if case["gated"] else 1)
    if op == "act":
        k = case["k"]
        return {"bytes": (rows * k + busy * k * width) * es + (busy * width * eo if case["bias"] else 0)
                + rows * n * eo * (2 if case["residual"] else 1)
                + (rows * width * eo if case["keep"] else 0),
                "flops": 2 * rows * width * k}
    return {"bytes": rows * (width + n) * eo + rows * width * es + (rows * n * es if case["keep"] else 0)
            + (4 * case["groups"] * width if case["bias"] else 0),
            "flops": 10 * rows * n}


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op = case["op"]
    ti, to = _TYPES[case["dtype"]]
    st = {"op": op, "case": case, "in": ti, "out": to}

    def normal(*shape, std=1.0, dtype=torch.float32):
        return torch.randn(*shape, generator=gen, device="cuda").mul_(std).to(dtype)

    if op in ("route", "route_grad"):
        t, e, k = case["tokens"], case["experts"], case["top"]
        st["logits"] = normal(t, e, std=1.5, dtype=ti)
        if case["masked"]:                       # the rows that pad the batch
            st["logits"][t - case["masked"]:] = -math.inf
        if case["bias"]:
            st["bias"] = normal(e, std=0.1)
        if op == "route_grad":
            ids = torch.argsort(st["logits"].float(), dim=1, descending=True, stable=True)[:, :k].int()
            if case["masked"]:
                ids[t - case["masked"]:] = -1
            st["ids"] = ids.contiguous()
            st["dweights"] = normal(t, k)
            st["dlogits"] = torch.empty(t, e, dtype=ti, device="cuda")
        else:
            for name, shape in (("ids", (t, k)), ("order", (t * k,)), ("position", (t, k))):
                st[name] = torch.empty(shape, dtype=torch.int32, device="cuda")
            st["weights"] = torch.empty(t, k, device="cuda")
            st["offsets"] = torch.empty(e + 1, dtype=torch.int32, device="cuda")
    elif op in ("gather", "combine", "combine_grad"):
        t, k, n = case["tokens"], case["top"], case["cols"]
        expert = torch.rand(t, case["experts"], generator=gen, device="cuda").argsort(1)[:, :k]
        order = torch.argsort(expert.reshape(-1), stable=True)
        position = torch.empty_like(order)
        position[order] = torch.arange(t * k, device="cuda")
        st["order"], st["position"] = order.int(), position.int().view(t, k)
        if case["weighted"]:
            st["weights"] = torch.rand(t, k, generator=gen, device="cuda")
        if op == "gather":
            st["X"] = normal(t, n, dtype=ti)
            st["D"] = torch.empty(t * k, n, dtype=ti, device="cuda")
        else:
            st["Y"] = normal(t * k, n, dtype=ti)
        if op == "combine":
            st["C"] = normal(t, n, dtype=to) if case["residual"] else None
            st["D"] = torch.empty(t, n, dtype=to, device="cuda")
        elif op == "combine_grad":
            st["dD"] = normal(t, n, std=0.1, dtype=ti)
            st["dY"] = torch.empty(t * k, n, dtype=ti, device="cuda")
            st["dweights"] = torch.empty(t, k, device="cuda")
    else:
        sizes = _sizes(case)
        turn = np.random.RandomState(seed & 0x7FFFFFFF).permutation(len(sizes))
        sizes = [sizes[i] for i in turn]
        rows, n, groups = case["rows"], case["n"], case["groups"]
        width = n * (2 if case["gated"] else 1)
        st["sizes"] = sizes
        st["offsets"] = torch.tensor(np.cumsum([0] + sizes).tolist(), dtype=torch.int32, device="cuda")
        if op == "act":
            k = case["k"]
            shape = (k, width) if case["trans"] == "N" else (width, k)
            st["A"] = normal(rows, k, dtype=ti)
            st["B"] = torch.empty(groups, *shape, dtype=ti, device="cuda")
            for i in range(groups):
                st["B"][i] = normal(*shape, std=1.0 / math.sqrt(k))
            st["bias"] = normal(groups, width, std=0.3, dtype=to) if case["bias"] else None
            st["R"] = normal(rows, n, dtype=to) if case["residual"] else None
            st["Z"] = torch.empty(rows, width, dtype=to, device="cuda") if case["keep"] else None
            st["D"] = torch.empty(rows, n, dtype=to, device="cuda")
        else:
            st["Z"] = normal(rows, width, dtype=to)
            st["dD"] = normal(rows, n, std=0.1, dtype=to)
            st["dZ"] = torch.empty(rows, width, dtype=ti, device="cuda")
            st["H"] = torch.empty(rows, n, dtype=ti, device="cuda") if case["keep"] else None
            st["dbias"] = torch.empty(groups, width, device="cuda") if case["bias"] else None
    if own:
        import dense_gemm_11_amd as g
        st["h"] = g.gemm_create()      # one per state, as a program keeps one
        if op == "route":
            st["ws"] = g.route_workspace(case["tokens"], case["experts"])
        if op == "act_grad" and case["bias"]:
            st["ws"] = g.act_grad_workspace(case["rows"], width, case["groups"])
    return st


# ------------------------------------------------------- the framework's calls
def _run_own(st):
    import dense_gemm_11_amd as g
    op, h, case = st["op"], st["h"], st["case"]
    if op == "route":
        g.run_route(h, st["logits"], st["ids"], st["weights"], offsets=st["offsets"],
                    order=st["order"], position=st["position"], workspace=st["ws"],
                    scores=case["scores"], bias=st.get("bias"), groups=case["groups"],
                    top_groups=case["top_groups"], group_top=case["group_top"],
                    renormalize=case["renorm"], scale=case["scale"])
        return st["ids"], st["weights"], st["offsets"], st["order"], st["position"]
    if op == "route_grad":
        g.run_route_grad(h, st["logits"], st["ids"], st["dweights"], st["dlogits"],
                         scores=case["scores"], renormalize=case["renorm"], scale=case["scale"])
        return st["dlogits"]
    if op == "gather":
        g.run_gather_rows(h, st["X"], st["D"], st["order"], case["top"], weights=st.get("weights"))
        return st["D"]
    if op == "combine":
        g.run_combine_rows(h, st["Y"], st["D"], st["position"], weights=st.get("weights"),
                           C=st["C"], beta=1.0 if st["C"] is not None else 0.0)
        return st["D"]
    if op == "combine_grad":
        g.run_combine_rows_grad(h, st["Y"], st["dD"], st["dY"], st["dweights"], st["position"],
                                st["weights"])
        return st["dY"], st["dweights"]
    if op == "act":
        g.run_grouped_act(h, st["A"], st["B"], st["D"], st["offsets"], activation=case["act"],
                          gated=case["gated"], bias=st["bias"], Z=st["Z"], R=st["R"],
                          transB=case["trans"])
        return (st["D"], st["Z"]) if case["keep"] else st["D"]
    g.run_grouped_act_grad(h, st["Z"], st["dD"], st["dZ"], st["offsets"], activation=case["act"],
                           gated=case["gated"], H=st["H"], dbias=st["dbias"],
                           workspace=st.get("ws"))
    return tuple(x for x in (st["dZ"], st["H"], st["dbias"]) if x is not None)


# ------------------------------------------------------------- the plain forms
def _plain_scores(x, kind):
    if kind == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-x))
    top = x.max(dim=1, keepdim=True).values
    e = torch.exp(x - torch.where(top.isinf(), torch.zeros_like(top), top))
    return e / e.sum(1, keepdim=True).clamp_min(1e-30)


def _plain_route(st):
    case, x = st["case"], st["logits"].float()
    t, e, k = case["tokens"], case["experts"], case["top"]
    f64, dev = torch.float64, x.device
    # what is chosen: in 64 bits, since scores next to each other decide
    choice = _plain_scores(x.to(f64), case["scores"])
    if case["bias"]:
        choice = choice + st["bias"].to(f64)
    elif case["groups"] == 1 or case["group_top"] == 1:
        choice = x.to(f64)                       # the scores rise with the logits
    low = torch.tensor(-math.inf, dtype=f64, device=dev)
    choice = torch.where(x > -math.inf, choice, low)
    if case["groups"] > 1:
        per = choice.view(t, case["groups"], -1)
        best = per.sort(dim=2, descending=True).values[:, :, :case["group_top"]].sum(2)
        kept = best.sort(dim=1, descending=True, stable=True).indices[:, :case["top_groups"]]
        keep = torch.zeros(t, case["groups"], dtype=torch.bool, device=dev).scatter_(1, kept, True)
        choice = torch.where(keep[:, :, None], per, low).view(t, e)
    best, ids = choice.sort(dim=1, descending=True, stable=True)
    best, ids = best[:, :k], ids[:, :k]
    live = best > -math.inf
    w = torch.where(live, _plain_scores(x, case["scores"]).gather(1, ids), torch.zeros((), device=dev))
    if case["renorm"]:
        w = w / w.sum(1, keepdim=True).clamp_min(1e-30)
    w = w * case["scale"]
    ids = torch.where(live, ids, torch.full_like(ids, -1))
    flat = torch.where(live, ids, torch.full_like(ids, e)).reshape(-1)
    rank, order = flat.sort(stable=True)
    offsets = torch.searchsorted(rank, torch.arange(e + 1, device=dev))
    position = torch.empty_like(order)
    position[order] = torch.arange(t * k, device=dev)
    position = torch.where(live, position.view(t, k), torch.full_like(ids, -1))
    order = torch.where(rank < e, order, torch.full_like(order, -1))
    return ids.int(), w, offsets.int(), order.int(), position.int()


def _plain_route_grad(st):
    case, x, g = st["case"], st["logits"].float(), st["dweights"]
    ids = st["ids"].long()
    live = ids >= 0
    at = ids.clamp_min(0)
    zero = torch.zeros((), device=x.device)
    s = _plain_scores(x, case["scores"])
    c = case["scale"]
    g = torch.where(live, g, zero)
    p = torch.where(live, s.gather(1, at), zero)
    if case["renorm"]:
        total = p.sum(1, keepdim=True).clamp_min(1e-30)
        q = p / total
        mixed = c * (g - (g * q).sum(1, keepdim=True))
        picked = q * mixed if case["scores"] == "softmax" else q * (1.0 - p) * mixed
        dx = torch.zeros_like(x)
    elif case["scores"] == "softmax":
        picked = c * p * g
        dx = -c * s * (p * g).sum(1, keepdim=True)
    else:
        picked = c * p * (1.0 - p) * g
        dx = torch.zeros_like(x)
    return dx.scatter_add_(1, at, torch.where(live, picked, zero)).to(st["in"])


def _plain_act(x, act):
    """The activation and its derivative."""
    if act == "none":
        return x, torch.ones_like(x)
    if act == "relu":
        on = (x > 0).to(x.dtype)
        return x * on, on
    if act == "silu":
        s = 1.0 / (1.0 + torch.exp(-x))
        return x * s, s * (1.0 + x * (1.0 - s))
    if act == "gelu":
        phi = 0.5 * (1.0 + torch.erf(x * math.sqrt(0.5)))
        return x * phi, phi + x * torch.exp(-0.5 * x * x) * (1.0 / math.sqrt(2.0 * math.pi))
    c = math.sqrt(2.0 / math.pi)
    th = torch.tanh(c * (x + 0.044715 * x * x * x))
    return 0.5 * x * (1.0 + th), 0.5 * (1.0 + th) + 0.5 * x * (1.0 - th * th) * c * (
        1.0 + 3 * 0.044715 * x * x)


def _run_plain(st):
    op, case, ti, to = st["op"], st["case"], st["in"], st["out"]
    if op == "route":
        return _plain_route(st)
    if op == "route_grad":
        return _plain_route_grad(st)
    if op == "gather":
        a = st["order"].long()
        rows = st["X"].float()[a // case["top"]]
        if case["weighted"]:
            rows = rows * st["weights"].reshape(-1)[a][:, None]
        return rows.to(ti)
    if op == "combine":
        rows = st["Y"].float()[st["position"].long()]
        if case["weighted"]:
            rows = rows * st["weights"][:, :, None]
        out = rows.sum(1)
        return (out + st["C"].float() if case["residual"] else out).to(to)
    if op == "combine_grad":
        at, dD = st["position"].long(), st["dD"].float()
        dw = (st["Y"].float()[at] * dD[:, None, :]).sum(2)
        dY = torch.empty_like(st["dY"])
        dY[at] = (st["weights"][:, :, None] * dD[:, None, :]).to(ti)
        return dY, dw
    n, lo, outs = case["n"], 0, []
    if op == "act":
        D, Z = torch.empty_like(st["D"]), None if st["Z"] is None else torch.empty_like(st["Z"])
        for i, size in enumerate(st["sizes"]):
            r = slice(lo, lo + size)
            lo += size
            w = st["B"][i].float()
            z = st["A"][r].float() @ (w if case["trans"] == "N" else w.t())
            if case["bias"]:
                z = z + st["bias"][i].float()
            d = _plain_act(z[:, :n], case["act"])[0]
            if case["gated"]:
                d = d * z[:, n:]
            if case["residual"]:
                d = d + st["R"][r].float()
            D[r] = d.to(to)
            if Z is not None:
                Z[r] = z.to(to)
        return D if Z is None else (D, Z)
    z, dD = st["Z"].float(), st["dD"].float()
    h, slope = _plain_act(z[:, :n], case["act"])
    if case["gated"]:
        dz = torch.cat([dD * z[:, n:] * slope, dD * h], 1)
        h = h * z[:, n:]
    else:
        dz = dD * slope
    outs.append(dz.to(ti))
    if case["keep"]:
        outs.append(h.to(ti))
    if case["bias"]:
        outs.append(torch.stack([x.sum(0) for x in dz.split(st["sizes"])]))
    return tuple(outs)


def run(state):
    return _run_own(state) if own else _run_plain(state)


# --------------------------------------------------- the definitions in 64 bits
def _exact_route(case, st):
    x = st["logits"].double().cpu().numpy()
    t, e, k = case["tokens"], case["experts"], case["top"]
    allowed = x > -np.inf
    any_row = allowed.any(1)
    if case["scores"] == "sigmoid":
        with np.errstate(over="ignore"):
            s = np.where(allowed, 1.0 / (1.0 + np.exp(-x)), 0.0)
    else:
        top = np.where(any_row, np.where(allowed, x, -np.inf).max(1), 0.0)
        s = np.where(allowed, np.exp(x - top[:, None]), 0.0)
        s /= np.maximum(s.sum(1, keepdims=True), 1e-300)
    c = s + (st["bias"].double().cpu().numpy() if case["bias"] else 0.0)
    if not case["bias"] and (case["groups"] == 1 or case["group_top"] == 1):
        c = x.copy()
    c = np.where(allowed, c, -np.inf)
    if case["groups"] > 1:
        per = c.reshape(t, case["groups"], -1)
        score = -np.sort(-per, axis=2)[:, :, :case["group_top"]].sum(2)
        best = np.argsort(-score, axis=1, kind="stable")
        place = np.argsort(best, axis=1, kind="stable")        # each group's rank
        c = np.where(place[:, :, None] < case["top_groups"], per, -np.inf).reshape(t, e)
    ids = np.argsort(-c, axis=1, kind="stable")[:, :k]
    live = np.take_along_axis(c, ids, 1) > -np.inf
    w = np.where(live, np.take_along_axis(s, ids, 1), 0.0)
    if case["renorm"]:
        w = w / np.maximum(w.sum(1, keepdims=True), 1e-300)
    w = w * case["scale"]
    ids = np.where(live, ids, -1)
    order = np.full(t * k, -1, np.int32)
    position = np.full(t * k, -1, np.int32)
    flat = ids.reshape(-1)
    offsets, at = np.zeros(e + 1, np.int32), 0
    for i in range(e):
        mine = np.flatnonzero(flat == i)
        order[at:at + len(mine)] = mine
        position[mine] = np.arange(at, at + len(mine))
        at += len(mine)
        offsets[i + 1] = at
    return tuple(torch.from_numpy(np.ascontiguousarray(v)) for v in
                 (ids.astype(np.int32), w, offsets, order, position.reshape(t, k)))


def _exact_route_grad(case, st):
    # the weights as a function of the logits, differentiated term by term
    x, g = st["logits"].double().cpu().numpy(), st["dweights"].double().cpu().numpy()
    ids = st["ids"].cpu().numpy()
    t, e = x.shape
    dx = np.zeros_like(x)
    rows = np.arange(t)
    live = ids >= 0
    at = np.where(live, ids, 0)
    picked = np.where(live, np.take_along_axis(x, at, 1), -np.inf)
    if case["scores"] == "softmax":
        # over all experts, or (renormalised) over the chosen ones alone
        base = x if not case["renorm"] else picked
        top = base.max(1, keepdims=True)
        top = np.where(np.isfinite(top), top, 0.0)
        total = np.exp(base - top).sum(1, keepdims=True)
        total = np.where(total > 0, total, 1.0)
        q = np.exp(picked - top) / total
        mean = (q * g * live).sum(1, keepdims=True)
        for j in range(ids.shape[1]):
            dx[rows, at[:, j]] += np.where(live[:, j], q[:, j] * g[:, j], 0.0)
        if case["renorm"]:
            for j in range(ids.shape[1]):
                dx[rows, at[:, j]] -= np.where(live[:, j], q[:, j] * mean[:, 0], 0.0)
        else:
            dx -= np.exp(x - top) / total * mean
    else:
        s = 1.0 / (1.0 + np.exp(-picked))
        ds = g * live
        if case["renorm"]:
            total = (s * live).sum(1, keepdims=True)
            total = np.where(total > 0, total, 1.0)
            ds = (g - (g * s * live).sum(1, keepdims=True) / total) / total * live
        for j in range(ids.shape[1]):
            dx[rows, at[:, j]] += np.where(live[:, j], ds[:, j] * s[:, j] * (1.0 - s[:, j]), 0.0)
    return torch.from_numpy(dx * case["scale"])


def _exact_act(x, name):
    if name == "none":
        return x
    if name == "relu":
        return x.clamp_min(0.0)
    if name == "silu":
        return x * torch.sigmoid(x)
    if name == "gelu":
        return 0.5 * x * torch.erfc(-x / math.sqrt(2.0))
    return x * torch.sigmoid(2.0 * math.sqrt(2.0 / math.pi) * (x + 0.044715 * x ** 3))


def _exact_slope(x, name):
    if name == "none":
        return torch.ones_like(x)
    if name == "relu":
        return (x > 0).double()
    if name == "silu":
        s = torch.sigmoid(x)
        return s + x * s * torch.sigmoid(-x)
    if name == "gelu":
        return 0.5 * torch.erfc(-x / math.sqrt(2.0)) + x * torch.exp(-x * x / 2) / math.sqrt(2 * math.pi)
    u = 2.0 * math.sqrt(2.0 / math.pi) * (x + 0.044715 * x ** 3)
    s = torch.sigmoid(u)
    return s + x * s * torch.sigmoid(-u) * 2.0 * math.sqrt(2.0 / math.pi) * (1.0 + 0.134145 * x ** 2)


def exact(case, seed):
    st = prepare(case, seed)
    op, f64 = case["op"], torch.float64
    if op == "route":
        return _exact_route(case, st)
    if op == "route_grad":
        return _exact_route_grad(case, st)
    if op in ("gather", "combine", "combine_grad"):
        t, k, n = case["tokens"], case["top"], case["cols"]
        w = st["weights"].to(f64) if case["weighted"] else torch.ones(t, k, dtype=f64, device="cuda")
        at = st["position"].long()
        if op == "gather":
            out = torch.zeros(t * k, n, dtype=f64, device="cuda")
            for j in range(k):
                out[at[:, j]] = w[:, j, None] * st["X"].to(f64)
            return out
        if op == "combine":
            out = st["C"].to(f64) if case["residual"] else torch.zeros(t, n, dtype=f64, device="cuda")
            for j in range(k):
                out += w[:, j, None] * st["Y"][at[:, j]].to(f64)
            return out
        dD = st["dD"].to(f64)
        dY, dw = torch.zeros(t * k, n, dtype=f64, device="cuda"), torch.zeros_like(w)
        for j in range(k):
            dY[at[:, j]] = w[:, j, None] * dD
            dw[:, j] = (st["Y"][at[:, j]].to(f64) * dD).sum(1)
        return dY, dw
    bounds, n = st["offsets"].tolist(), case["n"]
    spans = list(zip(bounds[:-1], bounds[1:]))
    if op == "act":
        D = torch.zeros(case["rows"], n, dtype=f64, device="cuda")
        Z = torch.zeros(st["Z"].shape, dtype=f64, device="cuda") if case["keep"] else None
        for i, (a, b) in enumerate(spans):
            if a == b:
                continue
            w = st["B"][i].to(f64)
            z = torch.mm(st["A"][a:b].to(f64), w if case["trans"] == "N" else w.transpose(0, 1))
            if case["bias"]:
                z += st["bias"][i].to(f64)
            D[a:b] = _exact_act(z[:, :n], case["act"])
            if case["gated"]:
                D[a:b] *= z[:, n:]
            if Z is not None:
                Z[a:b] = z
        if case["residual"]:
            D += st["R"].to(f64)
        return D if Z is None else (D, Z)
    z, dD = st["Z"].to(f64), st["dD"].to(f64)
    gate = z[:, :n]
    if case["gated"]:
        dz = torch.cat([dD * z[:, n:] * _exact_slope(gate, case["act"]),
                        dD * _exact_act(gate, case["act"])], 1)
    else:
        dz = dD * _exact_slope(gate, case["act"])
    outs = [dz]
    if case["keep"]:
        h = _exact_act(gate, case["act"])
        outs.append(h * z[:, n:] if case["gated"] else h)
    if case["bias"]:
        db = torch.zeros(case["groups"], dz.shape[1], dtype=f64, device="cuda")
        for i, (a, b) in enumerate(spans):
            db[i] = dz[a:b].sum(0)
        outs.append(db)
    return tuple(outs)
