"""Routing to experts (run_route) and its gradient (run_route_grad) against the
definition in 64 bits.

Choices, offsets, order and positions have to be equal.  Weights: with D the
largest distance of a chosen logit from the largest, e^(x - m) is off by D + 2
units of 2^-24 (the difference's rounding, the exponential's last place), a sum of
up to 1024 terms in 16 or 64 lanes of up to 32 each by at most 38 more of each
term's and the division and scale by 2: 64 + 2 D units in all.  An e^(x - m) below
2^-126, fp32's smallest normal number, may come out as 0, which is off by less than
2^-126, and the sum it is divided by is 1 at least.  The gradient adds
the products' and differences' roundings to that, 96 + 2 D units of the sum of
the magnitudes that it is a difference of, and its own rounding to the logits' type.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

from .gpu_support import announce, require_gpu

gpu = pytest.mark.gpu
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def g():
    import dense_gemm_11_amd
    return dense_gemm_11_amd


def scores_of(x, kind):
    """Scores of the logits x (float64); masked ones get 0."""
    ok = x > -np.inf
    with np.errstate(over="ignore", invalid="ignore"):
        if kind == "sigmoid":
            return np.where(ok, 1.0 / (1.0 + np.exp(-x)), 0.0)
        m = np.where(ok, x, -np.inf).max(1, keepdims=True, initial=-np.inf)
        e = np.where(ok, np.where(x == m, 1.0, np.exp(x - m)), 0.0)
        return e / np.maximum(e.sum(1, keepdims=True), 1e-300)


def choose(x, top, kind, bias=None, groups=1, top_groups=1, group_top=1):
    """ids by the definition, one token at a time."""
    s = scores_of(x, kind)
    ids = np.full((x.shape[0], top), -1, np.int32)
    for t in range(x.shape[0]):
        if bias is not None:
            c = s[t] + bias
        elif groups > 1 and group_top == 2:
            c = s[t].copy()
        else:
            c = x[t].copy()
        c[~(x[t] > -np.inf) | ~(c > -np.inf)] = -np.inf
        if groups > 1:
            per = c.reshape(groups, -1)
            best = np.sort(per, axis=1)[:, ::-1][:, :group_top]
            score = np.array([sum(v for v in b[1:] if v > -np.inf) + b[0] for b in best])
            kept = np.argsort(-score, kind="stable")[:top_groups]
            mask = np.full(groups, False)
            mask[kept] = True
            c = np.where(mask[:, None], per, -np.inf).reshape(-1)
        o = np.argsort(-c, kind="stable")[:top]
        ids[t] = np.where(c[o] > -np.inf, o, -1)
    return ids


def weights_of(x, ids, kind, renorm, scale):
    at = np.maximum(ids, 0)
    live = ids >= 0
    if renorm:
        # as ratios, so that no score is lost to underflow
        xs = np.where(live, np.take_along_axis(x, at, 1), -np.inf)
        m = xs.max(1, keepdims=True)
        if kind == "sigmoid":
            m = np.minimum(m, 0.0)
        with np.errstate(over="ignore", invalid="ignore"):
            w = np.where(xs == m, 1.0, np.exp(xs - m))
            if kind == "sigmoid":
                w = np.where(xs > 0, 1.0 / (1.0 + np.exp(-xs)), w / (1.0 + np.exp(np.minimum(xs, 0))))
        w = np.where(live, w, 0.0)
        w = w / np.where(live.any(1, keepdims=True), w.sum(1, keepdims=True), 1.0)
    else:
        w = np.where(live, np.take_along_axis(scores_of(x, kind), at, 1), 0.0)
    return w * scale


def plan_of(ids, experts):
    flat = ids.reshape(-1)
    order, position, offsets = np.full(flat.size, -1), np.full(flat.size, -1), [0]
    for e in range(experts):
        mine = np.flatnonzero(flat == e)
        order[offsets[-1]:offsets[-1] + len(mine)] = mine
        position[mine] = offsets[-1] + np.arange(len(mine))
        offsets.append(offsets[-1] + len(mine))
    return np.array(offsets), order, position.reshape(ids.shape)


def spread(x, ids):
    """64 + 2 D of the module's docstring, per token."""
    xs = np.where(ids >= 0, np.take_along_axis(x, np.maximum(ids, 0), 1), np.nan)
    m = np.where(x > -np.inf, x, -np.inf).max(1, keepdims=True, initial=-np.inf)
    with np.errstate(invalid="ignore"):
        d = np.nan_to_num(np.abs(m - xs), nan=0.0, posinf=0.0).max(1, keepdims=True)
    return d


def run(x, top, kind="softmax", renorm=False, scale=1.0, bias=None, groups=1, top_groups=1, group_top=1,
        plan=True, tokens=None):
    T, E = x.shape
    i32 = dict(dtype=torch.int32, device="cuda")
    ids, w = torch.full((T, top), 99, **i32), torch.full((T, top), 9.0, device="cuda")
    offsets, order, position = (torch.full((E + 1,), 99, **i32), torch.full((T * top,), 99, **i32),
                                torch.full((T, top), 99, **i32)) if plan else (None,) * 3
    h = g().gemm_create()
    try:
        g().run_route(h, x, ids, w, offsets, order, position, g().route_workspace(T, E), scores=kind,
                      bias=bias, groups=groups, top_groups=top_groups, group_top=group_top,
                      renormalize=renorm, scale=scale)
        torch.cuda.synchronize()
    finally:
        g().gemm_destroy(h)
    return [None if v is None else v.cpu().numpy() for v in (ids, w, offsets, order, position)]


def check(x, got, top, kind="softmax", renorm=False, scale=1.0, bias=None, groups=1, top_groups=1,
          group_top=1):
    x64 = x.double().cpu().numpy()
    b64 = None if bias is None else bias.double().cpu().numpy()
    ids, w, offsets, order, position = got
    want = choose(x64, top, kind, b64, groups, top_groups, group_top)
    assert np.array_equal(ids, want), f"{(ids != want).any(1).sum()} tokens chose otherwise"
    val = weights_of(x64, want, kind, renorm, scale)
    tol = (64 + 2 * spread(x64, want)) * 2.0 ** -24 * val + 2.0 ** -126 * scale
    assert (np.abs(w - val) <= tol).all(), (np.abs(w - val) / np.maximum(tol, 1e-300)).max()
    if offsets is not None:
        for a, b in zip((offsets, order, position), plan_of(want, x.shape[1])):
            assert np.array_equal(a, b)


CASES = [
    # tokens, experts, top, options
    (1, 8, 2, {}),
    (1, 1, 1, dict(renorm=True)),
    (16, 64, 4, dict(renorm=True)),
    (17, 64, 6, dict(kind="sigmoid", scale=2.5)),
    (65, 5, 5, dict(kind="sigmoid", renorm=True)),
    (100, 60, 4, dict(kind="sigmoid", renorm=True, bias=True)),
    (300, 7, 3, dict(bias=True)),
    (1024, 512, 16, dict(renorm=True)),
    (1025, 256, 8, dict(kind="sigmoid", renorm=True, scale=2.5, bias=True, groups=8, top_groups=4,
                        group_top=2)),
    (1100, 160, 6, dict(groups=8, top_groups=3)),
    (1200, 72, 6, dict(groups=9, top_groups=4, group_top=2)),
    (2000, 1000, 12, dict(bias=True, kind="sigmoid")),
    (70, 1024, 32, dict(kind="sigmoid", renorm=True, groups=32, top_groups=9, group_top=2)),
    (40, 990, 10, dict(groups=33, top_groups=5)),
    (4097, 33, 5, dict(renorm=True)),
    (20000, 30, 2, dict(groups=15, top_groups=7, group_top=2, bias=True)),
    (33000, 12, 3, {}),
    (6000, 512, 10, dict(bias=True)),
    (8193, 64, 15, dict(kind="sigmoid", bias=True, groups=4, top_groups=2, group_top=2)),
]


def draw(T, E, dtype, seed, ties):
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn(T, E, generator=gen) * 1.5
    if ties:                             # a few values only, so most tokens have equals
        x = (x * 2).round() / 2
    return x.to(TYPES[dtype])


@gpu
@pytest.mark.parametrize("ties", [False, True])
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("case", range(len(CASES)))
def test_route(case, dtype, ties):
    require_gpu()
    T, E, top, opt = CASES[case]
    announce("route", T, E, top, opt, dtype, ties)
    opt = dict(opt)
    x = draw(T, E, dtype, case, ties)
    if T > 9:
        x[T - T // 9:] = -float("inf")   # padding
        x[::7, ::3] = -float("inf")      # experts that some tokens may not take
    if opt.pop("bias", False):
        b = torch.randn(E, generator=torch.Generator().manual_seed(case)) * 0.2
        opt["bias"] = ((b * 8).round() / 8 if ties else b).cuda()
    # an odd row length, other data between the rows
    wide = torch.full((T, E + 3), 50.0, dtype=TYPES[dtype], device="cuda")
    view = wide[:, :E]
    view.copy_(x)
    check(x, run(view, top, **opt), top, **opt)


@gpu
@pytest.mark.parametrize("T", [5, 3000])
@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
def test_route_of_infinities_and_nan(T, kind, biased):
    require_gpu()
    announce("route infinities", T, kind, biased)
    inf, nan = float("inf"), float("nan")
    rows = [[inf, 0, inf, 1, 2, -inf], [nan, -inf, nan, -inf, -inf, nan], [nan, 3, 3, nan, -inf, 1],
            [-300, -299, -302, -inf, -301, -298], [300, 0, -300, 100, 200, -100]]
    x = torch.tensor(rows).repeat(-(-T // 5), 1)[:T].contiguous()
    bias = torch.tensor([0.5, -inf, 0.25, nan, 1.0, 0.0]).cuda() if biased else None
    for renorm in (False, True):
        got = run(x.cuda(), 4, kind, renorm, 1.0, bias)
        check(x, got, 4, kind, renorm, 1.0, bias)


@gpu
def test_route_separates_scores_that_fp32_cannot():
    require_gpu()
    announce("route near ties")
    gen = torch.Generator().manual_seed(0)
    x = torch.randn(2000, 2, generator=gen)
    s = torch.sigmoid(x.double())
    # a bias per pair of experts would make their scores equal but for its rounding
    for t in range(20):
        bias = torch.stack([(s[t, 1] - s[t, 0]).float(), torch.zeros(())]).cuda()
        one = x[t:t + 1].repeat(1500, 1)
        check(one, run(one.cuda(), 2, "sigmoid", bias=bias), 2, "sigmoid", bias=bias)


@gpu
@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
def test_route_sums_of_choices_far_larger_than_themselves(kind):
    """Groups of one bias near 1000 and one near -1000: fp32 rounds their choices to
    2^-15, the sums decide by less."""
    require_gpu()
    announce("route large biases", kind)
    x = draw(3000, 16, "f32", 3, False)
    x[:, [0, 1, 5, 8, 9, 13]] /= 64  # sums of several groups next to each other
    bias = torch.tensor([1000.0, -1000.0, -4000.0, -4000.0] * 4) + torch.tensor([0.125, -0.125, 0, 0] * 4)
    opt = dict(kind=kind, bias=bias.cuda(), groups=4, top_groups=2, group_top=2)
    check(x, run(x.cuda(), 4, **opt), 4, **opt)


@gpu
@pytest.mark.parametrize("T", [1, 90, 3000])
@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", list(TYPES))
def test_route_groups_whose_sums_pass_fp32(dtype, kind, T):
    """Biases that mask whole groups by the type's lowest numbers: two of them sum
    below -FLT_MAX, which in 64 bits is a number like any other, so these groups are
    kept where too few others are."""
    require_gpu()
    announce("route sums past fp32", dtype, kind, T)
    x = draw(T, 32, dtype, 7, False)
    low = torch.finfo(torch.float32).min
    x[::3, 4:8] = -float("inf")                      # a group of none at all
    for masks in ([low] * 7, [-3e38, low, -2.5e38, low, -2.9e38, low, -1.9e38], [low, -2.0, low, low, low, 0.0, low]):
        bias = torch.cat([torch.zeros(4), torch.tensor(masks).repeat_interleave(4)])
        for top_groups, top in ((1, 2), (3, 10), (6, 15)):
            opt = dict(kind=kind, bias=bias.cuda(), groups=8, top_groups=top_groups, group_top=2)
            check(x, run(x.cuda(), top, **opt), top, **opt)


@gpu
@pytest.mark.parametrize("T,E,top", [(16, 1024, 32), (16, 64, 4), (1, 256, 8), (9, 33, 15), (5, 1024, 1)])
@pytest.mark.parametrize("opt", [dict(), dict(kind="sigmoid", renorm=True, bias=True)], ids=["plain", "bias"])
def test_route_up_to_16_tokens_needs_no_workspace(T, E, top, opt):
    require_gpu()
    announce("route without workspace", T, E, top, opt)
    opt = dict(opt)
    x = draw(T, E, "f32", 11, False)
    if opt.pop("bias", False):
        opt["bias"] = torch.randn(E, generator=torch.Generator().manual_seed(12)).cuda() * 0.2
    i32 = dict(dtype=torch.int32, device="cuda")
    ids, w = torch.full((T, top), 99, **i32), torch.full((T, top), 9.0, device="cuda")
    plan = [torch.full((E + 1,), 99, **i32), torch.full((T * top,), 99, **i32), torch.full((T, top), 99, **i32)]
    handle = g().gemm_create()
    try:
        g().run_route(handle, x.cuda(), ids, w, *plan, scores=opt.get("kind", "softmax"), bias=opt.get("bias"),
                      renormalize=opt.get("renorm", False))
        torch.cuda.synchronize()
    finally:
        g().gemm_destroy(handle)
    check(x, [v.cpu().numpy() for v in (ids, w, *plan)], top, **opt)


@gpu
def test_route_without_plan_without_tokens_and_on_a_stream():
    require_gpu()
    announce("route without plan")
    x = draw(200, 24, "f32", 5, False)
    check(x, run(x.cuda(), 3, plan=False), 3)
    none = run(torch.empty(0, 24, device="cuda"), 3)
    assert (none[2] == 0).all()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        check(x, run(x.cuda(), 3), 3)


@gpu
@pytest.mark.parametrize("T", [13, 700, 5000, 17000])
def test_route_captured(T):
    """Replayed with other logits between, every replay as the eager call."""
    require_gpu()
    announce("route captured", T)
    E, top = 48, 4
    x = torch.empty(T, E, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    out = [torch.zeros(T, top, **i32), torch.zeros(T, top, device="cuda"), torch.zeros(E + 1, **i32),
           torch.zeros(T * top, **i32), torch.zeros(T, top, **i32)]
    ws, h = g().route_workspace(T, E), g().gemm_create()
    try:
        x.copy_(draw(T, E, "f32", 1, False))
        call = lambda: g().run_route(h, x, *out, ws, renormalize=True)
        call()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call()
        for rep in range(4):
            x.copy_(draw(T, E, "f32", 10 + rep, False))
            for o in out:
                o.fill_(7)
            graph.replay()
            torch.cuda.synchronize()
            got = [o.cpu().numpy() for o in out]
            check(x, got, top, renorm=True)
            eager = run(x, top, renorm=True)
            assert all(np.array_equal(a, b) for a, b in zip(got, eager))
    finally:
        g().gemm_destroy(h)


# ---------------------------------------------------------------- gradient
def grad_reference(x, ids, gw, kind, renorm, scale):
    """The gradient by the formulas, and the magnitudes it is a difference of."""
    T, E = x.shape
    live = (ids >= 0) & (ids < E)
    at = np.where(live, ids, 0)
    gw = np.where(live, gw, 0.0)
    s = np.where(live, np.take_along_axis(scores_of(x, kind), at, 1), 0.0)
    q = weights_of(x, np.where(live, ids, -1), kind, renorm, 1.0)
    dx, mag = np.zeros_like(x), np.zeros_like(x)
    xs = np.where(live, np.take_along_axis(x, at, 1), 0.0)
    with np.errstate(over="ignore"):
        rest = 1.0 / (1.0 + np.exp(xs)) if kind == "sigmoid" else 1.0
    mean = (gw * q).sum(1, keepdims=True)
    amean = (np.abs(gw) * q).sum(1, keepdims=True)
    if renorm:
        d, m = q * rest * (gw - mean), q * rest * (np.abs(gw) + amean)
    else:
        d, m = s * rest * gw, s * rest * np.abs(gw)
    rows = np.arange(T)
    for j in range(ids.shape[1]):
        dx[rows, at[:, j]] += np.where(live[:, j], d[:, j], 0.0)
        mag[rows, at[:, j]] += np.where(live[:, j], m[:, j], 0.0)
    if kind == "softmax" and not renorm:
        dx -= scores_of(x, kind) * mean
        mag += scores_of(x, kind) * amean
    return dx * scale, mag * abs(scale)


GRAD_CASES = [(1, 8, 2), (3, 1, 1), (100, 60, 4), (700, 1024, 32), (1025, 256, 8), (4099, 60, 4),
              (1500, 512, 16), (1300, 33, 20), (2000, 700, 6)]


@gpu
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("case", range(len(GRAD_CASES)))
def test_route_grad(case, dtype, kind, renorm):
    require_gpu()
    T, E, top = GRAD_CASES[case]
    announce("route grad", T, E, top, dtype, kind, renorm)
    x = draw(T, E, dtype, case, False)
    x[::5, ::4] = -float("inf")
    x64 = x.double().numpy()
    ids = choose(x64, top, kind)
    if top > 2:
        ids[::3, 1] = -1                       # fewer than top
        ids[1::3, 2] = ids[1::3, 0]            # an expert named twice
        ids[2::3, 1] = E                       # beyond the experts
    gw = torch.randn(T, top, generator=torch.Generator().manual_seed(9))
    wide = torch.full((T, E + 5), 50.0, dtype=TYPES[dtype], device="cuda")
    wide[:, :E].copy_(x)
    out = torch.full((T, E + 1), 77.0, dtype=TYPES[dtype], device="cuda")
    h = g().gemm_create()
    try:
        g().run_route_grad(h, wide[:, :E], torch.from_numpy(ids).cuda(), gw.cuda(), out[:, :E], scores=kind,
                           renormalize=renorm, scale=1.7)
        torch.cuda.synchronize()
    finally:
        g().gemm_destroy(h)
    got = out.double().cpu().numpy()
    assert (got[:, E] == 77.0).all(), "written beyond the row"
    val, mag = grad_reference(x64, ids, gw.double().numpy(), kind, renorm, 1.7)
    m = np.where(x64 > -np.inf, x64, np.nan)
    live = np.where(np.isnan(m).all(1, keepdims=True), 0.0, m)
    D = np.nanmax(live, axis=1, keepdims=True) - np.nanmin(live, axis=1, keepdims=True)
    tol = (96 + 2 * D) * 2.0 ** -24 * mag
    tol = tol + torch.finfo(TYPES[dtype]).eps / 2 * (np.abs(val) + tol)
    err = np.abs(got[:, :E] - val)
    assert (err <= tol).all(), (err / np.maximum(tol, 1e-300)).max()


@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
def test_gradient_formulas_against_differences(kind, renorm):
    """The reference above against central differences of the weights, in 64 bits:
    with steps of 1e-5 they are off by about 1e-10 (the third derivative, below 1,
    times the step's square) and 1e-11 (rounding over the step)."""
    rng = np.random.RandomState(0)
    x, gw = rng.randn(6, 9), rng.randn(6, 3)
    ids = choose(x, 3, kind)
    ids[2, 1] = -1
    val, _ = grad_reference(x, ids, gw, kind, renorm, 1.3)
    eps = 1e-5
    for e in range(9):
        up, dn = x.copy(), x.copy()
        up[:, e] += eps
        dn[:, e] -= eps
        diff = (weights_of(up, ids, kind, renorm, 1.3) - weights_of(dn, ids, kind, renorm, 1.3)) / (2 * eps)
        assert np.abs((gw * diff).sum(1) - val[:, e]).max() < 1e-8


# ---------------------------------------------------------------- refusals
FAKE = 0x100000  # never dereferenced: every call below fails validation first


def call(h, routing=None, **kw):
    import dense_gemm_11_amd as m
    r = dict(experts=16, top=2, scores=0, groups=1, top_groups=1, group_top=1, bias=None, renormalize=0,
             scale=1.0)
    r.update(routing or {})
    ids, weights, offsets, order, position, ws = (FAKE + (i << 36) for i in range(1, 7))
    a = dict(tokens=100, logits=FAKE, ld=16, dtype=0, ids=ids, weights=weights, offsets=offsets, order=order,
             position=position, ws=ws, ws_bytes=1 << 20)
    a.update(kw)
    rt = None if routing == "none" else m.GemmRouting(**r)
    return m.gemm_route(h, a["tokens"], a["logits"], a["ld"], a["dtype"], rt, a["ids"], a["weights"],
                        a["offsets"], a["order"], a["position"], a["ws"], a["ws_bytes"], None)


@pytest.fixture
def h():
    handle = g().gemm_create()
    yield handle
    g().gemm_destroy(handle)


def test_route_refuses_invalid_values(h):
    bad = g().GEMM_ERR_INVALID_VALUE
    assert call(None) == bad
    for kw in (dict(tokens=-1), dict(ld=15), dict(dtype=3), dict(logits=None), dict(ids=None),
               dict(weights=None), dict(offsets=None), dict(order=None), dict(position=None),
               dict(ws=None), dict(ws=FAKE + 8), dict(ws_bytes=16)):
        assert call(h, **kw) == bad, kw
    for r in (dict(experts=0), dict(top=0), dict(top=17), dict(scores=2), dict(groups=-1),
              dict(groups=3), dict(groups=4, top_groups=0), dict(groups=4, top_groups=5),
              dict(groups=4, group_top=3), dict(groups=4, group_top=0),
              dict(groups=8, top_groups=1, top=3), dict(scale=float("nan")), dict(scale=float("inf"))):
        assert call(h, r) == bad, r


def test_route_refuses_outputs_that_overlap(h):
    """100 tokens of 16 experts, 2 each: ids, weights, order and position of 800 bytes."""
    bad = g().GEMM_ERR_INVALID_VALUE
    ids, weights, offsets, order, position, ws = (FAKE + (i << 36) for i in range(1, 7))
    for kw in (dict(ids=FAKE + 6396), dict(weights=ids + 796), dict(offsets=ids - 64), dict(order=offsets),
               dict(position=order + 796), dict(position=ids), dict(ws=FAKE), dict(ws=order + 512),
               dict(order=FAKE)):
        assert call(h, **kw) == bad, kw
    assert call(h, dict(bias=weights + 796)) == bad and call(h, dict(bias=offsets + 64)) == bad
    assert call(h, ids=FAKE, offsets=None, order=None, position=None) == bad


def test_route_refuses_what_it_does_not_support(h):
    no = g().GEMM_ERR_NOT_SUPPORTED
    for r, kw in ((dict(experts=1025), dict(ld=1025)), (dict(experts=64, top=33), dict(ld=64)),
                  (dict(experts=130, groups=65, top_groups=4), dict(ld=130)), ({}, dict(tokens=1 << 26)),
                  (dict(experts=64, top=32), dict(tokens=(1 << 26) - 63, ld=64, ws_bytes=1 << 40)),
                  ({}, dict(logits=FAKE + 2)), ({}, dict(ids=FAKE + 2)), ({}, dict(position=FAKE + 1)),
                  (dict(bias=FAKE + 2), {}), ({}, dict(ld=1 << 31))):
        assert call(h, r, **kw) == no, (r, kw)


def test_route_fails_its_launch_on_request(monkeypatch):
    monkeypatch.setenv("GEMM_DEBUG_FAIL_LAUNCH", "1")
    handle = g().gemm_create()
    assert call(handle) == g().GEMM_ERR_HIP
    assert call(handle, tokens=0, offsets=None, order=None, position=None) == g().GEMM_OK
    g().gemm_destroy(handle)


def test_route_workspace_is_asked_for_beyond_16_tokens_only(monkeypatch):
    """By what the host refuses: the handle fails the launch of what passes."""
    monkeypatch.setenv("GEMM_DEBUG_FAIL_LAUNCH", "1")
    handle = g().gemm_create()
    none = dict(offsets=None, order=None, position=None)
    try:
        for experts, top in ((16, 2), (1024, 32), (1, 1)):
            r = dict(experts=experts, top=top)
            for tokens in (1, 2, 15, 16):
                assert call(handle, r, tokens=tokens, ld=experts, ws=None, ws_bytes=0) == g().GEMM_ERR_HIP
            for tokens in (17, 100, 5000):
                assert call(handle, r, tokens=tokens, ld=experts, ws=None,
                            ws_bytes=0) == g().GEMM_ERR_INVALID_VALUE
                assert call(handle, r, tokens=tokens, ld=experts, ws=None, ws_bytes=0, **none) == g().GEMM_ERR_HIP
    finally:
        g().gemm_destroy(handle)


def test_route_workspace_grows_with_the_tokens():
    sizes = [0, 1, 16, 17, 64, 1024, 1025, 4096, 4097, 16384, 16385, 40000, 1 << 20]
    for experts in (1, 8, 60, 1024):
        need = [g().gemm_route_workspace_bytes(t, experts) for t in sizes]
        assert need == sorted(need) and need[0] == 0
    assert g().gemm_route_workspace_bytes(5, 0) == 0


def test_route_grad_refusals(h):
    import dense_gemm_11_amd as m

    def grad(r=None, **kw):
        a = dict(tokens=100, logits=FAKE, ld=16, dtype=0, ids=FAKE, dw=FAKE, out=FAKE + (1 << 20), ldd=16)
        a.update(kw)
        q = dict(experts=16, top=2, scale=1.0)
        q.update(r or {})
        return m.gemm_route_grad(h, a["tokens"], a["logits"], a["ld"], a["dtype"], m.GemmRouting(**q),
                                 a["ids"], a["dw"], a["out"], a["ldd"], None)
    for kw in (dict(tokens=-1), dict(ld=15), dict(ldd=15), dict(dtype=-1), dict(logits=None), dict(ids=None),
               dict(dw=None), dict(out=None), dict(out=FAKE + 64), dict(ids=FAKE + (1 << 20)),
               dict(dw=FAKE + (1 << 20) + 6396)):
        assert grad(**kw) == m.GEMM_ERR_INVALID_VALUE, kw
    assert grad(dict(top=17)) == m.GEMM_ERR_INVALID_VALUE
    for kw in (dict(out=FAKE + (1 << 20) + 2), dict(dw=FAKE + 2), dict(tokens=1 << 26, ld=16)):
        if kw.get("tokens"):
            kw["out"] = FAKE + (1 << 40)
        assert grad(**kw) == m.GEMM_ERR_NOT_SUPPORTED, kw
    assert grad(tokens=0, logits=None) == m.GEMM_OK


def test_binding_refuses_wrong_tensors(h):
    m = g()
    x = torch.zeros(4, 8)
    ids, w = torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2)
    with pytest.raises(ValueError, match="GPU"):
        m.run_route(h, x, ids, w)
    with pytest.raises(TypeError):
        m.run_route(h, x.half(), ids, w)
    with pytest.raises(ValueError):
        m.run_route(h, x, ids[0], w)
    with pytest.raises(TypeError):
        m.run_route_grad(h, x.double(), ids, w, x)
    with pytest.raises(ValueError):
        m.run_route_grad(h, x, ids, w, x[:, :4])


def test_workspaces_that_are_not_contiguous_are_refused(h):
    """(Their numel is not what lies behind their first byte; seen before the
    tensors' device is, which here is the host.)"""
    m = g()
    x, ids, w = torch.zeros(40, 8), torch.zeros(40, 2, dtype=torch.int32), torch.zeros(40, 2)
    plan = (torch.zeros(9, dtype=torch.int32), torch.zeros(80, dtype=torch.int32), torch.zeros_like(ids))
    for ws in (torch.zeros(256, dtype=torch.uint8).expand(256, 256), torch.zeros(1, dtype=torch.uint8).expand(1 << 20),
               torch.zeros(64, 512, dtype=torch.uint8)[:, :256]):
        with pytest.raises(ValueError, match="contiguous"):
            m.run_route(h, x, ids, w, *plan, workspace=ws)
        with pytest.raises(ValueError, match="contiguous"):
            m.run_grouped_act_grad(h, x, x.clone(), x.clone(), dbias=torch.zeros(1, 8), workspace=ws)
