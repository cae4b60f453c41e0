"""Products with bias, activation, gate and residual (run_grouped_act) and their
gradient (run_grouped_act_grad) against the same formulas in 64 bits.

The bound on Z counts the roundings as for the ragged products: (K + 8) 2^-23 of
the sum of the magnitudes, t.  The activations' slopes are at most 1.13, and their
own error at most 2^-20 |x| (fp32 D; the exponentials, reciprocals and the normal
distribution to a few units of 2^-23) or 2^-19 |x| (bf16 D; formula 7.1.26 of
Abramowitz and Stegun is off by 1.5e-7, the hardware's exponential of a rounded
argument by less).  A gate's product and the residual add a unit each, D's own
rounding half a step.  What D's gradient meets is the stored Z, exactly.
"""
from __future__ import annotations

import math

import pytest
import torch

from .gpu_support import announce, require_gpu
from .test_grouped import TYPES, bounds_of, draw, padded

gpu = pytest.mark.gpu
ACTS = ["none", "relu", "gelu", "silu", "gelu_tanh"]
# every tile: height and number of that height
TILES = [(0, 0), (16, 0), (16, 1), (32, 0), (32, 1), (64, 0), (64, 1), (128, 0), (128, 1), (192, 0), (256, 0)]


def g():
    import dense_gemm_11_amd
    return dense_gemm_11_amd


def act(x, name):
    if name == "relu":
        return x.clamp_min(0.0)
    if name == "gelu":
        return 0.5 * x * torch.erfc(-x / math.sqrt(2.0))
    if name == "silu":
        return x * torch.sigmoid(x)
    if name == "gelu_tanh":
        return 0.5 * x * (1 + torch.tanh(math.sqrt(2 / math.pi) * (x + 0.044715 * x ** 3)))
    return x


def slope(x, name):
    if name == "relu":
        return (x > 0).to(x.dtype)
    if name == "gelu":
        return 0.5 * torch.erfc(-x / math.sqrt(2.0)) + x * torch.exp(-x * x / 2) / math.sqrt(2 * math.pi)
    if name == "silu":
        s = torch.sigmoid(x)
        return s * (1 + x * (1 - s))
    if name == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        th = torch.tanh(c * (x + 0.044715 * x ** 3))
        return 0.5 * (1 + th) + 0.5 * x * (1 - th * th) * c * (1 + 3 * 0.044715 * x * x)
    return torch.ones_like(x)


def own_error(dtype):
    return 2.0 ** -20 if dtype is torch.float32 else 2.0 ** -19


def within(got, val, tol, what):
    got = got.double().cpu()
    tol = tol + torch.finfo(what[0]).eps / 2 * (val.abs() + tol)
    err = (got - val).abs()
    ok = err <= tol
    assert ok.all(), f"{what[1]}: {int((~ok).sum())} off, worst {(err / tol.clamp_min(1e-300)).max():.3g} of the bound"


def reference(A, B, sizes, lead, trans, alpha, scales, bias, gated, name, R, to):
    """(D, its bound), (Z, its bound), rows in groups."""
    M, N = A.shape[0], (B.shape[2] if trans == "N" else B.shape[1])
    z = torch.zeros(M, N, dtype=torch.float64)
    den = torch.zeros_like(z)
    inside = torch.zeros(M, dtype=torch.bool)
    at = bounds_of(sizes, lead)
    for i in range(len(sizes)):
        r = slice(at[i], at[i + 1])
        inside[r] = True
        a, b = A[r].double(), B[i].double()
        b = b if trans == "N" else b.T
        s = alpha * (float(scales[i]) if scales is not None else 1.0)
        z[r] = s * (a @ b)
        den[r] = abs(s) * (a.abs() @ b.abs())
        if bias is not None:
            bi = (bias[i] if bias.dim() == 2 else bias).double()
            z[r] += bi
            den[r] += bi.abs()
    tz = (A.shape[1] + 8) * 2.0 ** -23 * den
    n = N // 2 if gated else N
    a, ta = act(z[:, :n], name), 1.13 * tz[:, :n] + own_error(to) * z[:, :n].abs()
    if gated:
        u, tu = z[:, n:], tz[:, n:]
        d = a * u
        td = ta * u.abs() + a.abs() * tu + ta * tu + 2.0 ** -23 * d.abs()
    else:
        d, td = a, ta
    if R is not None:
        d = d + R.double()
        td = td + 2.0 ** -23 * (d.abs() + R.double().abs())
    return (d, td), (z, tz), inside


CASES = [
    # sizes, rows before / after, K, N
    ([1], 0, 0, 64, 128),
    ([0, 3, 0, 1, 0], 0, 0, 40, 72),
    ([17, 0, 130, 1, 64], 5, 9, 96, 200),
    ([300, 129, 128, 127], 0, 3, 161, 257),
    ([2] * 70 + [0] * 60 + [5] * 10, 0, 0, 33, 65),
    ([70, 1, 40], 2, 0, 1, 300),
    ([90, 40], 0, 0, 515, 1),
    ([33, 31], 1, 1, 130, 34),
]


@pytest.fixture
def h():
    handle = g().gemm_create()
    yield handle
    g().gemm_destroy(handle)


def run_case(h, case, dtype, trans, gated, tile):
    sizes, before, after, K, N = CASES[case]
    ti, to = TYPES[dtype]
    M, G, W = sum(sizes) + before + after, len(sizes), N * (2 if gated else 1)
    A = draw((M, K), 1, ti)
    B = draw((G, K, W) if trans == "N" else (G, W, K), 2, ti)
    B = (B.float() / math.sqrt(K)).to(ti)
    x = case + 2 * TILES.index(tile) + (trans == "T")
    bias = draw((G, W), 3, to) if x % 3 else None
    R = draw((M, N), 4, to) if x % 4 > 1 else None
    keep, in_place = x % 2 == 0, x % 4 == 3
    scales = draw((G,), 5, torch.float32) if x % 5 == 0 else None
    alpha, name, pad = 0.75 if x % 5 == 1 else 1.0, ACTS[x % 5], 3 if case % 2 else 0
    announce("grouped act", sizes[:5], before, after, K, N, dtype, trans, "gated" if gated else "", tile, name)
    assert g().gemm_set_group_tile_nth(h, *tile) == g().GEMM_OK
    Rd = None if R is None else padded(R, pad)
    D = Rd if in_place and R is not None else padded(torch.full((M, N), 7.0, dtype=to), pad)
    was = D.cpu()
    Z = padded(torch.full((M, W), 7.0, dtype=to), pad + 1) if keep else None
    off = torch.tensor(bounds_of(sizes, before), dtype=torch.int32, device="cuda")
    g().run_grouped_act(h, padded(A, pad, pad), padded(B, pad, pad), D, off, activation=name, gated=gated,
                        bias=None if bias is None else padded(bias[None], pad)[0], Z=Z, R=Rd, transB=trans,
                        scales=None if scales is None else scales.cuda(), alpha=alpha)
    torch.cuda.synchronize()
    if tile[0]:
        launch = g().gemm_last_group_launch(h)
        assert launch.rows <= max(tile[0], 128) and launch.launches == 1
    (d, td), (z, tz), inside = reference(A, B, sizes, before, trans, alpha, scales, bias, gated, name, R, to)
    got = D.cpu()
    assert torch.equal(got[~inside], was[~inside]), "a row of no group was written"
    within(got[inside], d[inside], td[inside], (to, "D"))
    if keep:
        gz = Z.cpu()
        assert (gz[~inside] == 7.0).all(), "a row of no group was written in Z"
        within(gz[inside], z[inside], tz[inside], (to, "Z"))


@gpu
@pytest.mark.parametrize("tile", TILES)
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("trans", ["N", "T"])
@pytest.mark.parametrize("dtype", list(TYPES))
def test_grouped_act(h, dtype, trans, gated, tile):
    require_gpu()
    for case in range(len(CASES)):
        run_case(h, case, dtype, trans, gated, tile)


@gpu
@pytest.mark.parametrize("tile", [t for t in TILES if t[0] >= 64])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_every_number_of_steps(h, dtype, gated, tile):
    """Whole steps of K, one to 21 of 32 (a tile may begin anywhere in K), by groups
    of one row of tiles and of several."""
    require_gpu()
    ti, to = TYPES[dtype]
    sizes, N = [40, 0, 64, 5, 260, 1], 600
    M, G, W = sum(sizes), len(sizes), N * (2 if gated else 1)
    assert g().gemm_set_group_tile_nth(h, *tile) == g().GEMM_OK
    off = torch.tensor(bounds_of(sizes, 0), dtype=torch.int32, device="cuda")
    for steps in range(1, 22):
        K = 32 * steps
        announce("steps", dtype, gated, tile, K)
        A, B = draw((M, K), 1, ti), (draw((G, W, K), 2, ti).float() / math.sqrt(K)).to(ti)
        D = torch.empty(M, N, dtype=to, device="cuda")
        g().run_grouped_act(h, A.cuda(), B.cuda(), D, off, activation="silu", gated=gated, transB="T")
        (d, td), _, _ = reference(A, B, sizes, 0, "T", 1.0, None, None, gated, "silu", None, to)
        within(D, d, td, (to, f"D of K {K}"))


@gpu
@pytest.mark.parametrize("name", ACTS)
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("dtype", list(TYPES))
def test_dense_act(h, dtype, gated, name):
    """One matrix and all rows, without offsets, B of two dimensions or three."""
    require_gpu()
    ti, to = TYPES[dtype]
    for M, K, N, trans in ((1, 256, 130, "T"), (37, 100, 64, "N"), (300, 72, 190, "T")):
        announce("dense act", M, K, N, trans, dtype, gated, name)
        W = N * (2 if gated else 1)
        A, B = draw((M, K), 1, ti), draw((K, W) if trans == "N" else (W, K), 2, ti)
        B = (B.float() / math.sqrt(K)).to(ti)
        bias, R = draw((W,), 3, to), draw((M, N), 4, to)
        D, Z = torch.empty(M, N, dtype=to, device="cuda"), torch.empty(M, W, dtype=to, device="cuda")
        g().run_grouped_act(h, A.cuda(), B.cuda() if M > 1 else B[None].cuda(), D, None, activation=name,
                            gated=gated, bias=bias.cuda(), Z=Z, R=R.cuda(), transB=trans)
        (d, td), (z, tz), _ = reference(A, B[None], [M], 0, trans, 1.0, None, bias, gated, name, R, to)
        within(D, d, td, (to, "D"))
        within(Z, z, tz, (to, "Z"))


@gpu
@pytest.mark.parametrize("dtype", list(TYPES))
def test_activations_over_their_range(h, dtype):
    """Through a product with the identity: every activation from -100 to 100,
    where it underflows or saturates among them."""
    require_gpu()
    ti, to = TYPES[dtype]
    x = torch.cat([torch.linspace(-12, 12, 4001), torch.linspace(-100, 100, 95)]).to(ti)
    A = x[:, None].contiguous()
    B = torch.ones(1, 1, dtype=ti)
    for name in ACTS:
        announce("range", dtype, name)
        D = torch.empty(len(x), 1, dtype=to, device="cuda")
        g().run_grouped_act(h, A.cuda(), B.cuda(), D, None, activation=name)
        val = act(x.double()[:, None], name)
        within(D, val, own_error(to) * x.double().abs()[:, None], (to, name))


# tiles of each height (TILES names up to two of them), by the operands' type
HEIGHTS = {"bf16": {256: 1, 192: 1, 128: 2, 64: 2, 32: 2, 16: 2}, "f32": {128: 1, 64: 1, 32: 2, 16: 2}}


def forced_tile(dtype, tile):
    """(rows, nth) of the tile that gemm_set_group_tile_nth(*tile) makes a call take: of
    the tallest height not above, the nth or else its last."""
    table = HEIGHTS["f32" if dtype == "f32" else "bf16"]
    rows = max(r for r in table if r <= tile[0])
    return rows, min(tile[1], table[rows] - 1)


@gpu
@pytest.mark.parametrize("tile", TILES[1:])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("trans", ["N", "T"])
@pytest.mark.parametrize("dtype", list(TYPES))
def test_the_forced_tile_is_the_one_that_runs(h, dtype, trans, gated, tile):
    """As the tests above force them: heights, numbers and columns of what ran, and that
    every one of a type's tiles is among them."""
    require_gpu()
    announce("forced tile", dtype, trans, gated, tile)
    ti, to = TYPES[dtype]
    rows, nth = forced_tile(dtype, tile)
    assert g().gemm_set_group_tile_nth(h, *tile) == g().GEMM_OK
    seen = set()
    for M, N, K in ((300, 600, 160), (5, 34, 33)):
        W = N * (2 if gated else 1)
        A, B = draw((M, K), 1, ti).cuda(), draw((1, K, W) if trans == "N" else (1, W, K), 2, ti).cuda()
        D = torch.empty(M, N, dtype=to, device="cuda")
        off = torch.tensor([0, M], dtype=torch.int32, device="cuda")
        for offsets in (off, None):
            g().run_grouped_act(h, A, B, D, offsets, activation="silu", gated=gated, transB=trans)
            x = g().gemm_last_group_launch(h)
            assert (x.rows, x.nth, x.launches) == (rows, nth, 1) and g().gemm_last_group_tile(h) == rows
            seen.add(x.columns)
    assert len(seen) == 1
    reached = {forced_tile(dtype, t) for t in TILES[1:]}
    table = HEIGHTS["f32" if dtype == "f32" else "bf16"]
    assert reached == {(r, i) for r in table for i in range(table[r])}


@gpu
def test_act_empty_calls_and_empty_groups(h):
    require_gpu()
    announce("empty")
    bias = torch.tensor([[1.0, -2.0, 3.0, 4.0], [5.0, 6.0, -7.0, 8.0]], device="cuda")
    off = torch.tensor([0, 2, 3], dtype=torch.int32, device="cuda")
    want = torch.relu(bias[:, :2]) * bias[:, 2:]
    for A, alpha in ((torch.empty(3, 0, device="cuda"), 1.0), (torch.full((3, 5), float("nan"), device="cuda"), 0.0)):
        B = torch.full((2, A.shape[1], 4), float("nan"), device="cuda")
        D = torch.empty(3, 2, device="cuda")
        g().run_grouped_act(h, A, B, D, off, activation="relu", gated=True, bias=bias, alpha=alpha)
        assert torch.equal(D, want[[0, 0, 1]])
    D = torch.full((0, 2), 1.0, device="cuda")
    g().run_grouped_act(h, torch.empty(0, 5, device="cuda"), torch.ones(2, 5, 2, device="cuda"), D, off)
    assert g().gemm_last_group_tile(h) == 0


@gpu
def test_act_takes_offsets_past_the_rows(h):
    """Offsets outside [0, M] count as the nearest bound."""
    require_gpu()
    announce("offsets past the rows")
    A, B = draw((40, 32), 1, torch.float32), draw((3, 16, 32), 2, torch.float32)
    D = torch.full((40, 16), 7.0, device="cuda")
    off = torch.tensor([-5, 10, 10, 900], dtype=torch.int32, device="cuda")
    g().run_grouped_act(h, A.cuda(), B.cuda(), D, off, transB="T", activation="silu")
    (d, td), _, _ = reference(A, B, [10, 0, 30], 0, "T", 1.0, None, None, False, "silu", None, torch.float32)
    within(D, d, td, (torch.float32, "D"))


# ---------------------------------------------------------------- gradient
GRAD_CASES = [
    # sizes, rows before / after, N
    ([1], 0, 0, 128),
    ([0, 3, 0, 1, 0], 0, 2, 72),
    ([17, 0, 130, 1, 64], 5, 9, 513),
    ([300, 129, 128, 127], 0, 3, 1030),
    ([2] * 70 + [0] * 60 + [5] * 10, 0, 0, 7),
    ([3000], 0, 0, 1),
    (None, 0, 0, 260),                      # no offsets: 200 rows
]


def ulp_fast(dtype):
    # the slopes' own error: as the values', and x^2 of the argument's rounding
    return 2.0 ** -19 if dtype is torch.float32 else 2.0 ** -18


@gpu
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("case", range(len(GRAD_CASES)))
def test_grouped_act_grad(h, case, dtype, gated, in_place):
    require_gpu()
    sizes, before, after, N = GRAD_CASES[case]
    ti, to = TYPES[dtype]
    groups = [200] if sizes is None else sizes
    M, G, W = sum(groups) + before + after, len(groups), N * (2 if gated else 1)
    in_place = in_place and ti is to
    pad, at = case % 3, bounds_of(groups, before)
    off = None if sizes is None else torch.tensor(at, dtype=torch.int32, device="cuda")
    ws = g().act_grad_workspace(M, W, G)
    for x, name in enumerate(ACTS):
        announce("grouped act grad", groups[:5], before, after, N, dtype, gated, in_place, name)
        Z, dD = draw((M, W), 1, to) * 2, draw((M, N), 2, to)
        Zd, dDd = padded(Z, pad, pad), padded(dD, pad)
        dZ = Zd if in_place else padded(torch.full((M, W), 7.0, dtype=ti), pad, 1)
        H = None if x % 2 else dDd if in_place else padded(torch.full((M, N), 7.0, dtype=ti), pad + 1)
        dbias = torch.full((G, W), 9.0, device="cuda") if x != 1 else None
        ws.fill_(255)
        g().run_grouped_act_grad(h, Zd, dDd, dZ, off, activation=name, gated=gated, H=H, dbias=dbias,
                                 workspace=ws if dbias is not None else None)
        torch.cuda.synchronize()
        z, d = Z.double(), dD.double()
        v, s = act(z[:, :N], name), slope(z[:, :N], name)
        e = ulp_fast(ti) * (z[:, :N].abs() + 1)
        if gated:
            u = z[:, N:]
            val = torch.cat([d * u * s, d * v], 1)
            tol = torch.cat([(d * u).abs() * e, d.abs() * e], 1)
            hv, ht = v * u, e * u.abs()
        else:
            val, tol, hv, ht = d * s, d.abs() * e, v, e
        tol = tol + 2.0 ** -22 * val.abs()
        inside = slice(at[0], at[-1])
        out = torch.ones(M, dtype=torch.bool)
        out[inside] = False
        got = dZ.cpu()
        within(got[inside], val[inside], tol[inside], (ti, "dZ " + name))
        assert torch.equal(got[out], Z[out]) if in_place else (got[out] == 7.0).all()
        if H is not None:
            gh = H.cpu()
            within(gh[inside], hv[inside], (ht + 2.0 ** -22 * hv.abs())[inside], (ti, "H " + name))
            assert torch.equal(gh[out], dD[out]) if in_place else (gh[out] == 7.0).all()
        if dbias is not None:
            for i in range(G):
                r = slice(at[i], at[i + 1])
                n = groups[i]
                within(dbias[i], val[r].sum(0), tol[r].sum(0) + n * 2.0 ** -24 * val[r].abs().sum(0),
                       (torch.float32, "dbias " + name))


@gpu
@pytest.mark.parametrize("dtype", list(TYPES))
def test_values_and_slopes_far_out(h, dtype):
    """Finite Z whose square or cube is not: act(x) is x or 0 and act' 1 or 0,
    exactly, from |x| = 2^7 on (the tails are below 2^-180)."""
    require_gpu()
    ti, to = TYPES[dtype]
    x = torch.tensor([2.0 ** e for e in (7, 20, 42, 60, 64, 100, 126, 127)])
    x = torch.cat([x, -x]).to(to)[:, None]
    up = (x > 0).to(ti).cuda()
    for name in ("relu", "gelu", "silu", "gelu_tanh"):
        announce("far out", dtype, name)
        D, Z = (torch.empty(16, 1, dtype=to, device="cuda") for _ in range(2))
        g().run_grouped_act(h, x.to(ti).cuda(), torch.ones(1, 1, dtype=ti, device="cuda"), D, None,
                            activation=name, Z=Z)
        assert torch.equal(Z.cpu(), x) and torch.equal(D.cpu(), x.clamp_min(0.0)), name
        dZ, H = (torch.empty(16, 1, dtype=ti, device="cuda") for _ in range(2))
        g().run_grouped_act_grad(h, Z, torch.ones_like(D), dZ, None, activation=name, H=H)
        assert torch.equal(dZ, up) and torch.equal(H.cpu().to(to), x.clamp_min(0.0)), name


def infinite_products(h, dtype, name, gated):
    """A product of zeros with inf, -inf and NaN as its bias, and its gradient: (D, Z,
    dZ, H) and, by the formulas in 64 bits, what they are."""
    ti, to = TYPES[dtype]
    inf, nan = float("inf"), float("nan")
    z = torch.tensor([inf, -inf, nan, 0.0] * 3 + [inf])
    n = len(z)
    u = torch.tensor([2.0] * 4 + [-2.0] * 4 + [1.0] * 5)
    bias = (torch.cat([z, u]) if gated else z).to(to)
    M, W = 37, len(bias)
    D, Z = torch.empty(M, n, dtype=to, device="cuda"), torch.empty(M, W, dtype=to, device="cuda")
    A, B = torch.zeros(M, 40, dtype=ti, device="cuda"), torch.ones(W, 40, dtype=ti, device="cuda")
    g().run_grouped_act(h, A, B, D, None, activation=name, gated=gated, bias=bias.cuda(), Z=Z, transB="T")
    dZ, H = (torch.empty(M, k, dtype=ti, device="cuda") for k in (W, n))
    g().run_grouped_act_grad(h, Z, torch.ones_like(D), dZ, None, activation=name, gated=gated, H=H)
    v, s = act(z.double(), name), slope(z.double(), name)
    u = u.double() if gated else torch.ones_like(v)
    want = (v * u, bias.double(), torch.cat([s * u, v]) if gated else s, v * u)
    return [x.double().cpu() for x in (D, Z, dZ, H)], [w.expand(M, -1) for w in want]


@gpu
@pytest.mark.parametrize("tile", [(0, 0), (16, 0), (128, 0)])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("name", ["none", "gelu", "silu", "gelu_tanh"])
@pytest.mark.parametrize("dtype", list(TYPES))
def test_infinities_and_nan(h, dtype, name, gated, tile):
    """What the formulas give: act(inf) is inf, act(-inf) NaN (inf times 0), and so
    are the slopes at either, but for no activation."""
    require_gpu()
    announce("infinities", dtype, name, gated, tile)
    assert g().gemm_set_group_tile_nth(h, *tile) == g().GEMM_OK
    for what, got, want in zip(("D", "Z", "dZ", "H"), *infinite_products(h, dtype, name, gated)):
        torch.testing.assert_close(got, want, rtol=0, atol=0, equal_nan=True, msg=lambda m: f"{what}: {m}")


@gpu
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("dtype", list(TYPES))
def test_relu_of_infinities_and_nan(h, dtype, gated):
    """max(x, 0) of a NaN is NaN, of -inf 0; relu' is 1 above 0 and else 0."""
    require_gpu()
    announce("relu of nan", dtype, gated)
    for what, got, want in zip(("D", "Z", "dZ", "H"), *infinite_products(h, dtype, "relu", gated)):
        torch.testing.assert_close(got, want, rtol=0, atol=0, equal_nan=True, msg=lambda m: f"{what}: {m}")


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "bf16_out"])
def test_gelu_keeps_its_relative_accuracy_in_the_tail(h, dtype):
    """gelu and its slope from -12.5 on: D with bf16 outputs, H and dZ of bf16
    operands.  Phi's tail is off by 2^-17 of itself by its formula, by a^2 2^-22 <
    2^-15 for the roundings of the argument of e^(-a^2) with a = |x| / sqrt 2 up to
    8.9, and a few units of 2^-23: 2^-14 in all, beside the output's half step.  The
    slope is a difference of Phi and |x| times the density, off by as much of each
    of them.  (x itself is a bf16 number.)"""
    require_gpu()
    announce("gelu tail", dtype)
    ti, to = TYPES[dtype]
    x = torch.cat([torch.linspace(-12.5, -2, 3001), torch.linspace(-2, 0, 500)]).bfloat16()[:, None]
    D, Z = (torch.empty(len(x), 1, dtype=to, device="cuda") for _ in range(2))
    one = torch.ones(1, 1, dtype=ti, device="cuda")
    g().run_grouped_act(h, x.cuda(), one, D, None, activation="gelu", Z=Z)
    assert torch.equal(Z.cpu(), x.to(to))
    dZ, H = (torch.empty(len(x), 1, dtype=ti, device="cuda") for _ in range(2))
    g().run_grouped_act_grad(h, Z, torch.ones_like(D), dZ, None, activation="gelu", H=H)
    x = x.double()
    val, phi = act(x, "gelu"), 0.5 * torch.erfc(-x / math.sqrt(2.0))
    within(D, val, 2.0 ** -14 * val.abs(), (to, "D"))
    within(H, val, 2.0 ** -14 * val.abs(), (ti, "H"))
    s = slope(x, "gelu")
    within(dZ, s, 2.0 ** -14 * (phi + (s - phi).abs()), (ti, "dZ"))


@gpu
def test_act_grad_stays_inside_with_offsets_that_descend(h):
    """Groups that share rows make more tiles than the workspace has rows: their
    sums are anything, but nothing beyond the rows, the sums and the workspace is
    read or written."""
    require_gpu()
    M, N = 1000, 72
    Z, dD = (draw((M + 8, N), i, torch.float32).cuda() for i in (1, 2))
    for off in ([0, M, 0, M, 0, M, 3], [M, 0, 1 << 30, -5, 40, 7, M], [0] + [M, 0] * 40):
        announce("offsets that descend", off[:6])
        G = len(off) - 1
        need = g().gemm_act_grad_workspace_bytes(M, N, G)
        ws = torch.full((need + 65536,), 255, dtype=torch.uint8, device="cuda")
        dZ, dbias = torch.full((M + 8, N), 7.0, device="cuda"), torch.full((G + 4, N), 7.0, device="cuda")
        g().run_grouped_act_grad(h, Z[:M], dD[:M], dZ[:M], torch.tensor(off, dtype=torch.int32, device="cuda"),
                                 activation="silu", dbias=dbias[:G], workspace=ws[:need])
        torch.cuda.synchronize()
        assert (ws[need:] == 255).all() and (dZ[M:] == 7.0).all() and (dbias[G:] == 7.0).all()


@pytest.mark.parametrize("name", ACTS)
def test_slopes_against_differences(name):
    """The slopes above against central differences in 64 bits: with steps of 1e-5
    off by a third derivative below 3 times the step's square, and 1e-11."""
    x = torch.linspace(-9, 9, 1001, dtype=torch.float64) + 1e-3
    eps = 1e-5
    d = (act(x + eps, name) - act(x - eps, name)) / (2 * eps)
    assert (d - slope(x, name)).abs().max() < 1e-9


# ---------------------------------------------------------------- refusals
FAKE = 0x100000  # never dereferenced: every call below fails validation first


def call(h, act=None, groups=None, **kw):
    m = g()
    q = dict(activation=m.GEMM_ACT_SILU, gated=0, bias=None, stride_bias=0, Z=None, ldz=0, R=None, ldr=0)
    q.update(act or {})
    a = dict(transB=0, M=4, N=6, K=8, alpha=1.0, A=FAKE, lda=8, B=FAKE, ldb=12, strideB=0, D=FAKE, ldd=6,
             dtype=0)
    a.update(kw)
    gr = m.GemmGroups(*(groups or (2, FAKE, None)))
    return m.gemm_run_grouped_act(h, *a.values(), None if groups == () else gr,
                                  None if act == () else m.GemmAct(**q), None)


def test_act_refuses_invalid_values(h):
    bad = g().GEMM_ERR_INVALID_VALUE
    assert call(None) == bad and call(h, act=()) == bad
    for kw in (dict(transB=2), dict(dtype=3), dict(M=-1), dict(N=-1), dict(K=-1), dict(lda=7),
               dict(ldb=5), dict(transB=1, ldb=7), dict(ldd=5), dict(A=None), dict(B=None), dict(D=None),
               dict(strideB=-1)):
        assert call(h, **kw) == bad, kw
    far = FAKE + (1 << 20)
    for q in (dict(activation=5), dict(activation=-1), dict(gated=1, Z=far, ldz=11), dict(Z=far, ldz=5),
              dict(R=far, ldr=5), dict(stride_bias=-1), dict(Z=FAKE + 16, ldz=6), dict(R=FAKE + 16, ldr=6),
              dict(R=FAKE, ldr=7), dict(bias=FAKE + 8), dict(Z=far, ldz=6, R=far + 4, ldr=6),
              dict(Z=far, ldz=6, bias=far + 20)):
        assert call(h, q) == bad, q
    assert call(h, dict(gated=1), ldb=11) == bad
    assert call(h, groups=(-1, FAKE, None)) == bad and call(h, groups=(2, None, None)) == bad


def test_act_refuses_what_it_does_not_support(h):
    no = g().GEMM_ERR_NOT_SUPPORTED
    big = (1 << 31) - 512
    for kw in (dict(M=big), dict(K=big, lda=big), dict(N=1 << 30, ldb=1 << 31, ldd=1 << 30),
               dict(lda=1 << 31), dict(ldd=1 << 31), dict(A=FAKE + 2), dict(B=FAKE + 1), dict(D=FAKE + 2)):
        assert call(h, **kw) == no, kw
    far = FAKE + (1 << 20)
    for q in (dict(Z=far + 2, ldz=6), dict(R=far + 1, ldr=6), dict(bias=far + 2), dict(Z=far, ldz=1 << 31)):
        assert call(h, q) == no, q
    assert call(h, groups=(70000, FAKE, None)) == no and call(h, groups=(2, FAKE + 2, None)) == no
    # gated, both halves of a k-contiguous B within 4 GiB
    assert call(h, dict(gated=1), transB=1, N=1 << 19, K=1 << 10, lda=1 << 10, ldb=1 << 12, ldd=1 << 19,
                D=FAKE + (1 << 40)) == no


def test_act_empty_calls_do_nothing(h):
    assert call(h, M=0, A=None, B=None, D=None) == g().GEMM_OK
    assert call(h, N=0, ldd=1, D=None) == g().GEMM_OK
    assert call(h, groups=(0, None, None)) == g().GEMM_OK


def grad(h, groups=None, **kw):
    m = g()
    far = [FAKE + (i << 30) for i in range(6)]
    a = dict(M=10, N=8, activation=m.GEMM_ACT_GELU, gated=1, Z=far[0], ldz=16, dD=far[1], lddd=8, dZ=far[2],
             lddz=16, H=far[3], ldh=8, dbias=far[4], dtype=2)
    ws = dict(ws=far[5], ws_bytes=1 << 20)
    for k, v in kw.items():
        (ws if k in ws else a)[k] = v
    gr = None if groups == () else m.GemmGroups(*(groups or (2, FAKE, None)))
    return m.gemm_run_grouped_act_grad(h, *a.values(), gr, ws["ws"], ws["ws_bytes"], None)


def test_act_grad_refusals(h):
    m = g()
    bad, no = m.GEMM_ERR_INVALID_VALUE, m.GEMM_ERR_NOT_SUPPORTED
    z, dd, dz, hh = [FAKE + (i << 30) for i in range(4)]
    assert grad(None) == bad
    for kw in (dict(M=-1), dict(N=-1), dict(activation=9), dict(dtype=5), dict(ldz=15), dict(lddd=7),
               dict(lddz=15), dict(ldh=7), dict(Z=None), dict(dD=None), dict(dZ=None), dict(ws=None),
               dict(ws=FAKE + 64), dict(ws_bytes=64), dict(dZ=z + 8), dict(dZ=z, lddz=17),
               dict(dZ=z, dtype=1), dict(dZ=dd), dict(H=z), dict(H=dz), dict(H=dd, ldh=9),
               dict(dbias=z + 312), dict(dbias=dd - 124), dict(dbias=dz), dict(dbias=hh)):
        assert grad(h, **kw) == bad, kw
    assert grad(h, groups=(2, None, None)) == bad and grad(h, groups=(-2, FAKE, None)) == bad
    for kw in (dict(Z=z + 1), dict(dD=dd + 1), dict(dZ=dz + 1), dict(H=hh + 1), dict(dbias=FAKE + (4 << 30) + 2),
               dict(N=1 << 30, ldz=1 << 31, lddd=1 << 30, lddz=1 << 31, ldh=1 << 30),
               dict(lddd=1 << 31, M=1)):
        assert grad(h, **kw) == no, kw
    assert grad(h, groups=(70000, FAKE, None), ws_bytes=1 << 40) == no
    assert grad(h, M=0, Z=None, dbias=None) == m.GEMM_OK


def test_act_grad_refuses_a_workspace_and_offsets_that_overlap(monkeypatch):
    """50 rows, Z of 16 columns, 2 groups: what is written, the workspace's used part and
    dbias among it, lies apart from all else.  (The handle fails the launch of what
    passes.)"""
    monkeypatch.setenv("GEMM_DEBUG_FAIL_LAUNCH", "1")
    m = g()
    bad, passed = m.GEMM_ERR_INVALID_VALUE, m.GEMM_ERR_HIP
    z, dd, dz, hh, db, ws = [FAKE + (i << 30) for i in range(6)]
    far = FAKE + (8 << 30)
    need = m.gemm_act_grad_workspace_bytes(50, 16, 2)
    assert 256 < need < 512 and need % 4 == 0

    def grad_of(**kw):
        return grad(handle, M=50, **kw)

    handle = m.gemm_create()
    try:
        # Z, dZ: 1600 bytes of bf16; dD, H: 800; dbias: 128; offsets: 12
        for at in (z, z + 1536, z - 256, dd, dz, dz + 1536, hh, db - 256, db):
            assert grad_of(ws=at) == bad, hex(at)
        for at in (db, db + 124, db - 8, dz + 1596, hh + 796, dz - 8, ws, ws + need - 4):
            assert grad_of(groups=(2, at, None)) == bad, hex(at)
        # side by side; a larger workspace counts by what is used of it
        assert grad_of(ws=far, dbias=far + need) == passed
        assert grad_of(ws=far, dZ=far - 1600, groups=(2, far + need, None)) == passed
        assert grad_of(ws=far, dZ=far + need) == passed
        assert grad_of(groups=(2, db + 128, None)) == passed
        # without dbias the workspace is not used; without offsets none are read
        assert grad_of(ws=dz, dbias=None) == passed
        assert grad_of(groups=()) == passed
        # in place (the offsets, by default where Z is, elsewhere)
        assert grad_of(dZ=z, H=dd, groups=(2, far, None)) == passed
        assert grad_of(dZ=z, H=dd) == bad
    finally:
        m.gemm_destroy(handle)


def test_act_failed_launches_are_reported(monkeypatch):
    monkeypatch.setenv("GEMM_DEBUG_FAIL_LAUNCH", "1")
    handle = g().gemm_create()
    assert call(handle) == g().GEMM_ERR_HIP and grad(handle) == g().GEMM_ERR_HIP
    assert g().gemm_last_group_tile(handle) == 0
    g().gemm_destroy(handle)


def test_act_binding_refuses_wrong_tensors(h):
    m = g()
    A, B, D = torch.zeros(4, 8), torch.zeros(2, 8, 12), torch.zeros(4, 6)
    off = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="GPU"):
        m.run_grouped_act(h, A, B, D, off, gated=True)
    for kw in (dict(), dict(gated=True, activation="swish"), dict(gated=True, Z=torch.zeros(4, 6)),
               dict(gated=True, R=torch.zeros(4, 12)), dict(gated=True, bias=torch.zeros(2, 6))):
        with pytest.raises(ValueError):
            m.run_grouped_act(h, A, B, D, off, **kw)
    with pytest.raises(ValueError):
        m.run_grouped_act(h, A, B, D, None, gated=True)           # two groups without offsets
    with pytest.raises(TypeError):
        m.run_grouped_act(h, A, B, D, off, gated=True, Z=torch.zeros(4, 12).bfloat16())
    Z, dZ = torch.zeros(4, 12), torch.zeros(4, 12)
    with pytest.raises(ValueError, match="GPU"):
        m.run_grouped_act_grad(h, Z, D, dZ, off, gated=True)
    with pytest.raises(ValueError):
        m.run_grouped_act_grad(h, Z, D, dZ, off)
    with pytest.raises(TypeError):
        m.run_grouped_act_grad(h, Z, D, dZ, off, gated=True, H=D.bfloat16())
