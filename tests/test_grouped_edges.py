"""The ragged and adapted products where a form of theirs ends: ranks that fill
no tile, groups and calls with nothing to multiply, steps of several calls.
References and bounds as in test_grouped.py."""
from __future__ import annotations

import pytest
import torch

from .gpu_support import announce, require_gpu
from .test_grouped import TYPES, bounds_of, check, draw, g, handle, lora_reference
from .test_grouped_tiles import int32

gpu = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")


@gpu
@pytest.mark.parametrize("tile", [0, 16, 64, 128, 192, 256])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "bf16_out"])
@pytest.mark.parametrize("down", ["N", "T"])
@pytest.mark.parametrize("R", [72, 100, 130, 201])
def test_lora_ranks_past_a_tile_of_the_first_product(R, down, dtype, tile):
    """Ranks above 64 that are no multiple of 16, in a workspace of NaN: tiles of
    one adapter, mixed tiles, rows without one."""
    require_gpu()
    announce("rank", R, down, dtype, tile)
    ti, to = TYPES[dtype]
    sizes, ids, K, N = [300, 40, 21, 3, 60], [1, 0, 1, -1, 0], 96, 136
    M = sum(sizes)
    A, B = draw((M, K), 1, ti), draw((N, K), 2, ti)
    dn, up, s = draw((2, R, K), 3, ti), draw((2, N, R), 4, ti), draw((2,), 5, torch.float32)
    flip = down == "N"
    d_, u_ = (x.transpose(1, 2).contiguous() if flip else x for x in (dn, up))
    h = handle(tile)
    try:
        ws = g().lora_workspace(M, R)
        ws.fill_(255)
        D = torch.full((M, N), NAN, dtype=to, device="cuda")
        g().run_lora(h, A.cuda(), B.cuda(), D, int32(bounds_of(sizes)), d_.cuda(), u_.cuda(), ws,
                     ids=int32(ids), scales=s.cuda(), transB="T", transDown=down, transUp=down)
        val, den, low = lora_reference(A, B, None, sizes, 0, ids, dn, up, "T", 1.0, 0.0, s)
        check(D.cpu(), val, den, 2 * K + R, "rank", 2.0 ** -17 if dtype != "f32" else 0.0, low)
    finally:
        g().gemm_destroy(h)


@gpu
@pytest.mark.parametrize("tile", [0, 32, 64, 128, 192, 256])
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("beta", [0.0, 0.5])
def test_wgrad_of_empty_groups_takes_no_factor(beta, dtype, tile):
    """A factor of 1 / rows is infinite for an empty group, whose D_g is beta C_g
    (0 when beta == 0) all the same."""
    require_gpu()
    announce("factors of empty groups", beta, dtype, tile)
    ti, to = TYPES[dtype]
    sizes, M, N = [0, 40, 0, 7, 0], 70, 130
    at = bounds_of(sizes)
    A, B, C = draw((47, M), 1, ti), draw((47, N), 2, ti), draw((5, M, N), 3, to)
    s = torch.tensor([INF, 1 / 40, NAN, 1 / 7, -INF])
    val, den = beta * C.double(), (beta * C.double()).abs()
    for i in (1, 3):
        a, b = A[at[i]:at[i + 1]].double(), B[at[i]:at[i + 1]].double()
        val[i] += float(s[i]) * (a.T @ b)
        den[i] += abs(float(s[i])) * (a.abs().T @ b.abs())
    h = handle(tile)
    try:
        D = torch.full((5, M, N), NAN, dtype=to, device="cuda")
        g().run_grouped_wgrad(h, A.cuda(), B.cuda(), D, int32(at), C=C.cuda() if beta else None,
                              beta=beta, scales=s.cuda())
        check(D.cpu(), val, den, 40, "factors")
    finally:
        g().gemm_destroy(h)


@gpu
@pytest.mark.parametrize("tile", [0, 16, 64, 128, 256])
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("beta", [0.0, 0.5])
def test_calls_without_a_product_take_no_factor(beta, dtype, tile):
    """alpha == 0, K == 0 and no rows leave beta C, whatever the groups' factors and
    alpha hold."""
    require_gpu()
    announce("no product", beta, dtype, tile)
    ti, to = TYPES[dtype]
    sizes, K, N = [9, 0, 30], 24, 72
    M = sum(sizes)
    off, s = int32(bounds_of(sizes)), torch.tensor([INF, 1.0, NAN], device="cuda")
    A, B = draw((M, K), 1, ti).cuda(), draw((3, K, N), 2, ti).cuda()
    Y, C, G = draw((M, N), 3, ti).cuda(), draw((M, N), 4, to), draw((3, K, N), 5, to)
    h = handle(tile)
    try:
        for a, b, alpha in ((A, B, 0.0), (A[:, :0], B[:, :0], 1.0), (A[:, :0], B[:, :0], INF)):
            D = torch.full((M, N), NAN, dtype=to, device="cuda")
            g().run_grouped(h, a, b, D, off, C=C.cuda() if beta else None, scales=s, alpha=alpha,
                            beta=beta)
            check(D.cpu(), beta * C.double(), beta * C.double().abs(), 0, "rows")
        for a, y, alpha in ((A, Y, 0.0), (A[:0], Y[:0], 1.0), (A[:0], Y[:0], INF)):
            D = torch.full((3, K, N), NAN, dtype=to, device="cuda")
            g().run_grouped_wgrad(h, a, y, D, off, C=G.cuda() if beta else None, scales=s,
                                  alpha=alpha, beta=beta)
            check(D.cpu(), beta * G.double(), beta * G.double().abs(), 0, "gradients")
    finally:
        g().gemm_destroy(h)


@gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16", "bf16_f32"])
@pytest.mark.parametrize("rank", [8, 33, 64])
def test_adapters_gradients_round_once(rank, dtype):
    """The timed case's gradients of down and up (T and U by run_grouped, their
    products by run_grouped_wgrad) against 64 bits.  T and U are sums of K or N
    fp32 terms, then two bf16 terms: hi is off by half a step, 2^-8 of the binade,
    and lo by half a step of what is left, 2^-17 at most.  The second sums are
    over an adapter's rows, and the gradients are rounded once.  Short sums, so
    that one bf16 rounding of T or U (2^-8) would pass the bound."""
    require_gpu()
    announce("adapters' gradients", rank, dtype)
    import perf.operators as ops
    case = {"op": "lora_grad", "dtype": dtype, "rows": 40, "segments": 3, "single": 0,
            "adapters": 3, "without": 0, "rank": rank, "k": 16, "n": 24, "trans": "T"}
    was, ops.own = ops.own, True
    try:
        st = ops.prepare(case, 5)
        _, ddown, dup = ops.run(st)
        torch.cuda.synchronize()
    finally:
        ops.own = was
        g().gemm_destroy(st["h"])
    X, dY, down, up, s = (st[k].double().cpu() for k in ("X", "dY", "down", "up", "scales"))
    at, t_rel = st["offsets"].tolist(), 0.0 if dtype == "f32" else 2.0 ** -17
    for a in range(3):
        x, y = X[at[a]:at[a + 1]], dY[at[a]:at[a + 1]]
        terms = 16 + 24 + len(x)
        u, u_abs = s[a] * (y @ up[a]), s[a] * (y.abs() @ up[a].abs())
        check(ddown[a], u.T @ x, u_abs.T @ x.abs(), terms, "down", t_rel, u.abs().T @ x.abs())
        t, t_abs = s[a] * (x @ down[a].T), s[a] * (x.abs() @ down[a].abs().T)
        check(dup[a], y.T @ t, y.abs().T @ t_abs, terms, "up", t_rel, y.abs().T @ t.abs())
