"""Timed cases of the products over ragged groups of rows.

Three operators, each reached through the package's tensor entry points:

  * run_grouped:       D[rows of g] = alpha s_g A[rows of g] op(B_g) + beta C[rows of g]
                       (an expert's product over the rows routed to it);
  * run_grouped_wgrad: D_g = alpha s_g A[rows of g]^T B[rows of g] + beta C_g
                       (the gradient of the experts' weights);
  * run_lora:          D = alpha (X op(W) + s_a (X op(down_a)) op(up_a)) + beta C
                       (a shared projection with one low-rank adapter a per
                       segment of rows, or none).

A group is the run of rows offsets[g] .. offsets[g+1]-1, given by an int32
array on the GPU.  How many rows each group holds follows from the case alone
(so a case's work does not depend on the seed); which group holds how many,
and every value, follow from the seed.
"""
from __future__ import annotations

import math
import random
import zlib

import numpy as np
import torch

own = False

_TYPES = {"bf16": (torch.bfloat16, torch.bfloat16), "bf16_f32": (torch.bfloat16, torch.float32),
          "f32": (torch.float32, torch.float32)}


def _grouped(name, dtype, rows, groups, k, n, trans, skew):
    return {"name": name, "op": "grouped", "dtype": dtype, "rows": rows, "groups": groups, "k": k,
            "n": n, "trans": trans, "skew": skew}


def _lora(name, op, dtype, rows, segments, single, adapters, without, rank, k, n, trans):
    return {"name": name, "op": op, "dtype": dtype, "rows": rows, "segments": segments,
            "single": single, "adapters": adapters, "without": without, "rank": rank, "k": k,
            "n": n, "trans": trans}


def listed():
    return [
        # one token routed to two of eight experts: latency and two experts' weights
        _grouped("experts_one_token", "bf16", 2, 8, 2048, 1024, "T", 0.0),
        # a decode batch of 96 tokens, four experts each, popular and idle experts,
        # the weights stored as the forward pass of a training run keeps them
        _grouped("experts_decode_batch", "bf16", 384, 64, 4096, 1792, "N", 1.0),
        # a short prompt on odd sizes, fp32 results for the sum over experts
        _grouped("experts_short_prompt_odd", "bf16_f32", 1021, 16, 1537, 2051, "T", 0.6),
        # a prefill batch: large products, as fast as the matrix cores go
        _grouped("experts_prefill", "bf16", 16384, 8, 4096, 14336, "T", 0.3),
        # the same kind of layer in full precision
        _grouped("experts_f32", "f32", 2500, 12, 1024, 1408, "N", 0.5),
        # the backward pass of a layer of experts: inputs' and weights' gradients
        {"name": "experts_grad", "op": "grouped_grad", "dtype": "bf16", "rows": 8192,
         "groups": 16, "k": 2048, "n": 5632, "trans": "T", "skew": 0.5},
        # many small experts, some without a row, accumulated over micro-batches in fp32
        {"name": "experts_wgrad_accumulate", "op": "wgrad", "dtype": "bf16_f32", "rows": 4099,
         "groups": 64, "k": 2048, "n": 1408, "skew": 1.2},
        # one request decoding one token with its adapter
        _lora("adapters_one_token", "lora", "bf16", 1, 1, 1, 4, 0, 8, 2048, 2048, "T"),
        # sixty-four requests decoding, sixteen adapters in the order of arrival, some without
        _lora("adapters_decode_batch", "lora", "bf16", 64, 64, 64, 16, 9, 16, 4096, 4096, "T"),
        # prompts of odd lengths among decoding requests
        _lora("adapters_mixed_batch", "lora", "bf16", 1531, 40, 33, 24, 4, 32, 4096, 12288, "N"),
        # the same in full precision on odd sizes
        _lora("adapters_f32_odd", "lora", "f32", 517, 9, 5, 6, 1, 12, 1023, 1537, "N"),
        # fine-tuning four adapters at once: the inputs' and the adapters' gradients
        _lora("adapters_grad", "lora_grad", "bf16", 8192, 4, 0, 4, 0, 64, 4096, 4096, "T"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, lo, hi):
    # most widths are multiples of 64 or 8, the rest whatever they are
    v = _log_int(rng, lo, hi)
    step = rng.choice([64, 64, 8, 1])
    return max(lo, v // step * step)


def draw(rng: random.Random):
    top = work(listed()[3])
    while True:
        op = rng.choice(["grouped", "grouped", "grouped_grad", "wgrad", "lora", "lora", "lora_grad"])
        dtype = rng.choice(["bf16", "bf16", "bf16", "bf16_f32", "f32"])
        case = {"op": op, "dtype": dtype, "rows": _log_int(rng, 1, 16384)}
        case["k"] = _width(rng, 128, 8192)
        case["n"] = _width(rng, 128, 14336)
        if op != "wgrad":
            case["trans"] = rng.choice(["N", "T"])
        if op in ("lora", "lora_grad"):
            case["rank"] = rng.choice([4, 8, 8, 16, 16, 32, 64, rng.randint(1, 64)])
            case["adapters"] = rng.randint(1, 32)
            if op == "lora_grad":
                # the rows of each adapter together, as a training step sorts them
                case["dtype"] = dtype = rng.choice(["bf16", "bf16", "f32"])
                case["rows"] = _log_int(rng, 64, 16384)
                case["segments"] = case["adapters"]
                case["single"] = case["without"] = 0
            else:
                case["segments"] = _log_int(rng, 1, min(96, case["rows"]))
                case["single"] = (case["segments"] if case["segments"] == case["rows"]
                                  else rng.randint(0, case["segments"] - 1))
                case["without"] = rng.randint(0, case["segments"] // 4)
        else:
            case["groups"] = _log_int(rng, 1, 128)
            case["skew"] = round(rng.uniform(0.0, 1.2), 2)
        w = work(case)
        # an fp32 operation costs about ten bf16 ones
        cost = w["flops"] * (10 if dtype == "f32" else 1)
        if cost <= top["flops"] and w["bytes"] <= top["bytes"]:
            return case


def _case_rng(case):
    text = repr(sorted((k, v) for k, v in case.items() if k != "name"))
    return np.random.RandomState(zlib.crc32(text.encode()) & 0x7FFFFFFF)


def _sizes(case):
    """Rows of each group (as a list) and each segment's adapter (-1: none) or None."""
    r = _case_rng(case)
    if "groups" in case:
        w = (1.0 + np.arange(case["groups"])) ** -case["skew"]
        return [int(x) for x in r.multinomial(case["rows"], w / w.sum())], None
    segs, single = case["segments"], case["single"]
    if case["op"] == "lora_grad":
        sizes = r.multinomial(case["rows"], np.full(segs, 1.0 / segs))
        return [int(x) for x in sizes], list(range(segs))
    sizes = [1] * single
    if segs > single:
        long = segs - single
        rest = case["rows"] - single - long       # each longer segment has a row at least
        sizes += [1 + int(x) for x in r.multinomial(rest, r.dirichlet(np.full(long, 3.0)))]
    ids = [int(x) for x in r.randint(0, case["adapters"], segs)]
    for i in r.choice(segs, case["without"], replace=False):
        ids[i] = -1
    return sizes, ids


def work(case):
    es, eo = (4, 4) if case["dtype"] == "f32" else (2, 2 if case["dtype"] == "bf16" else 4)
    sizes, ids = _sizes(case)
    rows, k, n = sum(sizes), case["k"], case["n"]
    op = case["op"]
    if op in ("grouped", "grouped_grad", "wgrad"):
        busy, groups = sum(1 for s in sizes if s), len(sizes)
        if op == "grouped":
            return {"bytes": (rows * k + busy * k * n) * es + rows * n * eo,
                    "flops": 2 * rows * n * k}
        if op == "wgrad":                          # C read, D written
            return {"bytes": rows * (k + n) * es + 2 * groups * k * n * eo,
                    "flops": 2 * rows * n * k}
        return {"bytes": (rows * (k + n) + busy * k * n) * es + (rows * k + groups * k * n) * eo,
                "flops": 4 * rows * n * k}
    r = case["rank"]
    used = len({a for a, s in zip(ids, sizes) if a >= 0 and s})
    adapted = sum(s for a, s in zip(ids, sizes) if a >= 0)
    if op == "lora":
        return {"bytes": (rows * k + k * n + used * r * (k + n)) * es + rows * n * eo,
                "flops": 2 * rows * n * k + 2 * adapted * r * (k + n)}
    # both operands and W read, the gradients of X, down and up written
    return {"bytes": (rows * (k + n) + k * n + used * r * (k + n)) * es
            + (rows * k + case["adapters"] * r * (k + n)) * eo,
            "flops": 2 * rows * n * k + 6 * rows * r * (k + n)}


def prepare(case, seed):
    ti, to = _TYPES[case["dtype"]]
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def normal(*shape, std=1.0, dtype=ti):
        return torch.randn(*shape, generator=gen, device="cuda").mul_(std).to(dtype)

    sizes, ids = _sizes(case)
    if case["op"] != "lora_grad":
        order = np.random.RandomState(seed & 0x7FFFFFFF).permutation(len(sizes))
        sizes = [sizes[i] for i in order]
        ids = None if ids is None else [ids[i] for i in order]
    rows, k, n, op = case["rows"], case["k"], case["n"], case["op"]
    bounds = [0]
    for s in sizes:
        bounds.append(bounds[-1] + s)
    st = {"op": op, "sizes": sizes, "ids": ids, "trans": case.get("trans"),
          "in": ti, "out": to,
          "offsets": torch.tensor(bounds, dtype=torch.int32, device="cuda")}
    groups = len(sizes)
    w_std = 1.0 / math.sqrt(k)
    shape = (k, n) if case.get("trans") == "N" else (n, k)
    if op in ("grouped", "grouped_grad"):
        st["B"] = torch.empty(groups, *shape, dtype=ti, device="cuda")
        for g in range(groups):
            st["B"][g] = normal(*shape, std=w_std)
    if op == "grouped":
        st["A"] = normal(rows, k)
        st["D"] = torch.empty(rows, n, dtype=to, device="cuda")
    elif op in ("grouped_grad", "wgrad"):
        st["A"] = normal(rows, k)
        st["dY"] = normal(rows, n, std=0.1)
        if op == "wgrad":
            st["C"] = normal(groups, k, n, std=0.3, dtype=to)
            st["dW"] = torch.empty(groups, k, n, dtype=to, device="cuda")
        else:
            st["dA"] = torch.empty(rows, k, dtype=to, device="cuda")
            st["dB"] = torch.empty(groups, *shape, dtype=to, device="cuda")
    else:
        r = case["rank"]
        st["W"] = normal(*shape, std=w_std)
        st["down"] = normal(case["adapters"], r, k, std=w_std)
        st["up"] = normal(case["adapters"], n, r, std=1.0 / math.sqrt(r))
        st["scales"] = (0.5 + torch.rand(case["adapters"], generator=gen, device="cuda"))
        st["ids_gpu"] = torch.tensor(ids, dtype=torch.int32, device="cuda")
        st["X"] = normal(rows, k)
        if op == "lora":
            st["D"] = torch.empty(rows, n, dtype=to, device="cuda")
        else:
            st["dY"] = normal(rows, n, std=0.1)
            st["dX"] = torch.empty(rows, k, dtype=to, device="cuda")
            st["ddown"] = torch.empty(case["adapters"], r, k, dtype=to, device="cuda")
            st["dup"] = torch.empty(case["adapters"], n, r, dtype=to, device="cuda")
    if own:
        import dense_gemm_11_amd as g
        st["h"] = g.gemm_create()      # one per state, as a program keeps one
        if op in ("lora", "lora_grad"):
            st["ws"] = g.lora_workspace(rows, case["rank"])
        if op == "lora_grad":
            r, f32 = case["rank"], torch.float32
            st["TU"] = torch.empty(2, rows, r, dtype=f32, device="cuda")
            if ti is not f32:
                st["terms"] = torch.empty(2, rows, 2, r, dtype=ti, device="cuda")
                st["ddown2"] = torch.empty(case["adapters"], 2, r, k, dtype=f32, device="cuda")
                st["dup2"] = torch.empty(case["adapters"], n, 2, r, dtype=f32, device="cuda")
    return st


def _run_own(st):
    import dense_gemm_11_amd as g
    op, h, off = st["op"], st["h"], st["offsets"]
    if op == "grouped":
        g.run_grouped(h, st["A"], st["B"], st["D"], off, transB=st["trans"])
        return st["D"]
    if op == "wgrad":
        g.run_grouped_wgrad(h, st["A"], st["dY"], st["dW"], off, C=st["C"], beta=1.0)
        return st["dW"]
    flip = "T" if st["trans"] == "N" else "N"
    if op == "grouped_grad":
        g.run_grouped(h, st["dY"], st["B"], st["dA"], off, transB=flip)
        if st["trans"] == "N":
            g.run_grouped_wgrad(h, st["A"], st["dY"], st["dB"], off)
        else:
            g.run_grouped_wgrad(h, st["dY"], st["A"], st["dB"], off)
        return st["dA"], st["dB"]
    if op == "lora":
        g.run_lora(h, st["X"], st["W"], st["D"], off, st["down"], st["up"], st["ws"],
                   ids=st["ids_gpu"], scales=st["scales"], transB=st["trans"])
        return st["D"]
    # the adapters' activations T and gradients U, in fp32
    T, U = st["TU"]
    g.run_grouped(h, st["X"], st["down"], T, off, transB="T", scales=st["scales"])
    g.run_grouped(h, st["dY"], st["up"], U, off, transB="N", scales=st["scales"])
    if "terms" not in st:
        g.run_grouped_wgrad(h, U, st["X"], st["ddown"], off)
        g.run_grouped_wgrad(h, st["dY"], T, st["dup"], off)
    else:
        # as operands of bf16 products they go in as two terms side by side, hi +
        # lo (16 bits: one bf16 rounding would be as large as the gradients' own),
        # whose two fp32 products are then added and rounded once
        hi, lo = st["terms"][:, :, 0], st["terms"][:, :, 1]
        hi.copy_(st["TU"])
        torch.sub(st["TU"], hi, out=lo)
        T2, U2 = st["terms"].flatten(2)
        dd, du = st["ddown2"], st["dup2"]
        g.run_grouped_wgrad(h, U2, st["X"], dd.flatten(1, 2), off)
        g.run_grouped_wgrad(h, st["dY"], T2, du.flatten(2), off)
        torch.add(dd[:, 0], dd[:, 1], out=st["ddown"])
        torch.add(du[:, :, 0], du[:, :, 1], out=st["dup"])
    g.run_lora(h, st["dY"], st["W"], st["dX"], off, st["up"], st["down"], st["ws"],
               ids=st["ids_gpu"], scales=st["scales"], transB=flip, transDown="N", transUp="N")
    return st["dX"], st["ddown"], st["dup"]


def _op(w, trans):
    w = w.float()
    return w if trans == "N" else w.t()


def _run_plain(st):
    op, to = st["op"], st["out"]
    if op == "lora":
        X = st["X"].float()
        D = X @ _op(st["W"], st["trans"])
    elif op == "lora_grad":
        X, dY = st["X"].float(), st["dY"].float()
        dX = dY @ _op(st["W"], "T" if st["trans"] == "N" else "N")
        ddown, dup = [], []
    elif op == "grouped":
        D = []
    else:
        D, dB = [], []
    lo = 0
    for i, size in enumerate(st["sizes"]):
        rows = slice(lo, lo + size)
        lo += size
        if op == "grouped":
            D.append((st["A"][rows].float() @ _op(st["B"][i], st["trans"])).to(to))
        elif op == "wgrad":
            D.append((st["A"][rows].float().t() @ st["dY"][rows].float() + st["C"][i].float()).to(to))
        elif op == "grouped_grad":
            A, dY = st["A"][rows].float(), st["dY"][rows].float()
            D.append((dY @ _op(st["B"][i], "T" if st["trans"] == "N" else "N")).to(to))
            dB.append((A.t() @ dY if st["trans"] == "N" else dY.t() @ A).to(to))
        else:
            a = st["ids"][i]
            if a < 0:
                continue
            down, up, s = st["down"][a].float(), st["up"][a].float(), st["scales"][a]
            if op == "lora":
                D[rows] += s * ((X[rows] @ down.t()) @ up.t())
            else:
                T, U = s * (X[rows] @ down.t()), s * (dY[rows] @ up)
                dX[rows] += U @ down
                ddown.append((U.t() @ X[rows]).to(to))
                dup.append((dY[rows].t() @ T).to(to))
    if op == "grouped":
        return torch.cat(D)
    if op == "wgrad":
        return torch.stack(D)
    if op == "grouped_grad":
        return torch.cat(D), torch.stack(dB)
    if op == "lora":
        return D.to(to)
    return dX.to(to), torch.stack(ddown), torch.stack(dup)


def run(state):
    return _run_own(state) if own else _run_plain(state)


def exact(case, seed):
    st = prepare(case, seed)
    f64 = torch.float64
    bounds = st["offsets"].tolist()
    spans = list(zip(bounds[:-1], bounds[1:]))
    op = case["op"]

    def weight(i):                      # K x N of group i
        w = st["B"][i].to(f64)
        return w if case["trans"] == "N" else w.transpose(0, 1)

    if op == "grouped":
        out = torch.zeros(case["rows"], case["n"], dtype=f64, device="cuda")
        for i, (a, b) in enumerate(spans):
            if b > a:
                torch.mm(st["A"][a:b].to(f64), weight(i), out=out[a:b])
        return out
    if op == "wgrad":
        out = st["C"].to(f64)
        for i, (a, b) in enumerate(spans):
            if b > a:
                out[i].addmm_(st["A"][a:b].to(f64).transpose(0, 1), st["dY"][a:b].to(f64))
        return out
    if op == "grouped_grad":
        dA = torch.zeros(case["rows"], case["k"], dtype=f64, device="cuda")
        dB = torch.zeros(st["B"].shape, dtype=f64, device="cuda")
        for i, (a, b) in enumerate(spans):
            if b == a:
                continue
            A, dY = st["A"][a:b].to(f64), st["dY"][a:b].to(f64)
            dA[a:b] = torch.mm(dY, weight(i).transpose(0, 1))
            dB[i] = (torch.mm(A.transpose(0, 1), dY) if case["trans"] == "N"
                     else torch.mm(dY.transpose(0, 1), A))
        return dA, dB
    W = st["W"].to(f64)
    W = W if case["trans"] == "N" else W.transpose(0, 1)
    X = st["X"].to(f64)
    if op == "lora":
        out = torch.mm(X, W)
        for (a, b), i in zip(spans, st["ids_gpu"].tolist()):
            if i >= 0:
                t = torch.mm(X[a:b], st["down"][i].to(f64).transpose(0, 1))
                t *= float(st["scales"][i])
                out[a:b] += torch.mm(t, st["up"][i].to(f64).transpose(0, 1))
        return out
    dY = st["dY"].to(f64)
    dX = torch.mm(dY, W.transpose(0, 1))
    ddown = torch.zeros(st["down"].shape, dtype=f64, device="cuda")
    dup = torch.zeros(st["up"].shape, dtype=f64, device="cuda")
    for (a, b), i in zip(spans, st["ids_gpu"].tolist()):
        s, down, up = float(st["scales"][i]), st["down"][i].to(f64), st["up"][i].to(f64)
        u = s * torch.mm(dY[a:b], up)
        dX[a:b] += torch.mm(u, down)
        ddown[i] += torch.mm(u.transpose(0, 1), X[a:b])
        dup[i] += s * torch.mm(dY[a:b].transpose(0, 1),
                               torch.mm(X[a:b], down.transpose(0, 1)))
    return dX, ddown, dup
