"""The ragged and adapted products where a form of theirs ends: ranks that fill
no tile, groups and calls with nothing to multiply, steps of several calls.
References and bounds as in test_grouped.py."""
from __future__ import annotations

import pytest
import torch

from .gpu_support import announce, require_gpu
from .test_grouped import (TYPES, bounds_of, check, draw, g, handle, lora_reference, raw_grouped, raw_lora,
                           raw_wgrad)
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


# calls of run_lora that no adapter takes part in: keyword changes to a call of
# rank 8 over two adapters
WITHOUT = [dict(R=0), dict(adapters=0), dict(sizes=[], ids=[]), dict(K=0), dict(alpha=0.0)]


@gpu
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("kw", WITHOUT, ids=str)
def test_lora_without_adapters_leaves_the_handle_alone(kw, dtype):
    """The shared product alone, whatever the handle's workspace, stream-K mode and
    forced variant are: the same bits as from a new handle, and the workspace
    untouched."""
    require_gpu()
    announce("without adapters", kw, dtype)
    ti, to = TYPES[dtype]
    a = dict(dict(sizes=[300, 212], ids=[0, 1], adapters=2, R=8, K=4096, alpha=0.5), **kw)
    M, N, K, R = 512, 520, a["K"], a["R"]
    A, B, C = draw((M, K), 1, ti), draw((K, N), 2, ti), draw((M, N), 3, to)
    dn = draw((a["adapters"], R, K), 4, ti).cuda()
    up = draw((a["adapters"], N, R), 5, ti).cuda()
    p, off, ids = g(), int32(bounds_of(a["sizes"])), int32(a["ids"])
    got = []
    for attached in (False, True):
        h = p.gemm_create()
        try:
            if attached:
                ws = p.attach_workspace(h)
                torch.cuda.synchronize()
                before = ws.clone()
                assert p.gemm_set_stream_k(h, 1) == p.GEMM_OK
                # a variant of the other operand type, which gemm_run refuses
                other = next(i for i, _, d, _ in p.variants() if (d == p.GEMM_DTYPE_F32) != (dtype == "f32"))
                assert p.gemm_set_variant(h, other) == p.GEMM_OK
            D = torch.full((M, N), NAN, dtype=to, device="cuda")
            p.run_lora(h, A.cuda(), B.cuda(), D, off, dn, up, p.lora_workspace(M, 8), ids=ids,
                       C=C.cuda(), alpha=a["alpha"], beta=0.25)
            torch.cuda.synchronize()
            assert p.gemm_last_stream_k(h) == 0 and p.gemm_last_variant(h) == -1
            if attached:
                assert torch.equal(ws, before)
            got.append(D.cpu())
        finally:
            p.gemm_destroy(h)
    a64, b64, c64 = A.double(), B.double(), 0.25 * C.double()
    check(got[0], a["alpha"] * (a64 @ b64) + c64,
          abs(a["alpha"]) * (a64.abs() @ b64.abs()) + c64.abs(), K, "without adapters")
    assert torch.equal(*(x.view(torch.int16 if to is torch.bfloat16 else torch.int32) for x in got))


@pytest.mark.parametrize("kw", [dict(rank=0), dict(adapters=0), dict(segments=0)], ids=str)
def test_lora_without_adapters_is_planned_without_the_handle(kw, monkeypatch):
    """A forced variant of the other operand type does not refuse the call, which
    gets as far as its launch (switched off)."""
    p = g()
    monkeypatch.setenv("GEMM_DEBUG_FAIL_LAUNCH", "1")
    h = p.gemm_create()
    p.gemm_set_planning_model(256, [1] * p.gemm_variant_count())
    try:
        bf16 = next(i for i, _, d, _ in p.variants() if d != p.GEMM_DTYPE_F32)
        assert p.gemm_set_variant(h, bf16) == p.GEMM_OK
        assert raw_lora(h, **kw) == p.GEMM_ERR_HIP
    finally:
        p.gemm_set_planning_model(0, None)
        p.gemm_destroy(h)


@gpu
@pytest.mark.parametrize("tile", [0, 16, 32, 64, 128, 192, 256])
@pytest.mark.parametrize("up", ["N", "T"])
@pytest.mark.parametrize("trans", ["N", "T"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_lora_keeps_24_bits_of_t_beside_an_fp32_d(dtype, trans, up, tile):
    """Whole numbers of up to 21 bits in T, each picked out by a 1 in up: every sum is
    exact in fp32, so D has to equal them, on tiles of one adapter and mixed ones."""
    require_gpu()
    announce("bits of T", dtype, trans, up, tile)
    ti, R, K, N = TYPES[dtype][0], 24, 64, 136
    sizes, ids = [300, 5, 70, 30], [1, 0, -1, 0]
    M = sum(sizes)
    gen = torch.Generator().manual_seed(1)
    A = torch.randint(1, 256, (M, K), generator=gen).to(ti)
    dn = torch.randint(1, 256, (2, R, K), generator=gen).to(ti)
    u = torch.zeros(2, N, R, dtype=ti)
    u[:, torch.arange(N), torch.arange(N) % R] = 1
    want, at = torch.zeros(M, N, dtype=torch.float64), bounds_of(sizes)
    for i, a in enumerate(ids):
        if a >= 0:
            want[at[i]:at[i + 1]] = (A[at[i]:at[i + 1]].double() @ dn[a].double().T)[:, torch.arange(N) % R]
    assert want.max() < 2 ** 22 and (want.long() & 1).any()
    h = handle(tile)
    try:
        D = torch.full((M, N), NAN, device="cuda")
        B = torch.zeros(*((K, N) if trans == "N" else (N, K)), dtype=ti, device="cuda")
        ws = g().lora_workspace(M, R)
        ws.fill_(255)
        u_ = u if up == "T" else u.transpose(1, 2).contiguous()
        g().run_lora(h, A.cuda(), B, D, int32(at), dn.cuda(), u_.cuda(), ws, ids=int32(ids), transB=trans,
                     transUp=up)
        assert torch.equal(D.cpu().double(), want)
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


@gpu
@pytest.mark.parametrize("tile", [0, 16, 64, 128, 256])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_offsets_past_the_rows_are_clamped(dtype, tile):
    """The adapted product and the matrices' gradients with offsets below 0 and past
    the rows; with offsets that decrease, nothing outside D is written."""
    require_gpu()
    announce("clamped offsets", dtype, tile)
    ti, to = TYPES[dtype]
    M, K, N, R = 50, 64, 80, 8
    A, B = draw((M, K), 1, ti), draw((K, N), 2, ti)
    dn, up = draw((3, R, K), 3, ti), draw((3, N, R), 4, ti)
    val, den, low = lora_reference(A, B, None, [20, 0, 30], 0, [0, 1, 2], dn, up, "N", 1.0, 0.0, None)
    h = handle(tile)
    try:
        ws = g().lora_workspace(M, R)
        for off in ([-9, 20, 20, 4000], [40, -3, 35, 10]):
            D = torch.full((M + 4, N), 7.0, dtype=to, device="cuda")
            g().run_lora(h, A.cuda(), B.cuda(), D[2:M + 2], int32(off), dn.cuda(), up.cuda(), ws)
            got = D.cpu()
            assert torch.all(got[:2] == 7.0) and torch.all(got[M + 2:] == 7.0)
            if off[0] < 0:
                check(got[2:M + 2], val, den, 2 * K + R, "clamped", 2.0 ** -17, low)
        Y = draw((M, N), 5, ti)
        D = torch.full((5, K, N), 7.0, dtype=to, device="cuda")
        g().run_grouped_wgrad(h, A.cuda(), Y.cuda(), D[1:4], int32([-9, 20, 20, 4000]))
        got = D.cpu()
        assert torch.all(got[0] == 7.0) and torch.all(got[4] == 7.0)
        for i, r in enumerate((slice(0, 20), slice(0, 0), slice(20, 50))):
            a, y = A[r].double(), Y[r].double()
            check(got[1 + i], a.T @ y, a.abs().T @ y.abs(), 30, "gradient")
    finally:
        g().gemm_destroy(h)


# ---------------------------------------------------------------- limits (no GPU)
@pytest.fixture
def unlaunched(monkeypatch):
    """A handle whose calls report GEMM_ERR_HIP where they would launch."""
    monkeypatch.setenv("GEMM_DEBUG_FAIL_LAUNCH", "1")
    p = g()
    h = p.gemm_create()
    p.gemm_set_planning_model(256, [1] * p.gemm_variant_count())
    yield h
    p.gemm_set_planning_model(0, None)
    p.gemm_destroy(h)


def test_extents_that_32_bit_sums_cannot_carry(unlaunched):
    """Row and step numbers up to a tile past the end are formed in 32 bits."""
    p, h, top = g(), unlaunched, 2 ** 31 - 1
    fits = top - 512
    assert raw_grouped(h, M=top) == raw_grouped(h, M=fits + 1) == p.GEMM_ERR_NOT_SUPPORTED
    assert raw_grouped(h, M=fits) == p.GEMM_ERR_HIP
    assert raw_wgrad(h, rows=top) == raw_wgrad(h, rows=fits + 1) == p.GEMM_ERR_NOT_SUPPORTED
    assert raw_wgrad(h, rows=fits) == p.GEMM_ERR_HIP
    big = dict(bytes=1 << 62)
    assert raw_lora(h, M=top, **big) == p.GEMM_ERR_NOT_SUPPORTED
    assert raw_lora(h, M=2 ** 27, **big) == p.GEMM_ERR_HIP   # more are 2^32 threads
    for rank in (top, 2 ** 30):
        assert raw_lora(h, rank=rank, ld_up=top, stride_up=0, **big) == p.GEMM_ERR_NOT_SUPPORTED
    assert raw_lora(h, rank=1 << 20, ld_up=1 << 20, stride_up=0, **big) == p.GEMM_ERR_HIP


def test_grids_of_2_32_threads_are_refused(unlaunched):
    """65536 groups of one row by 2^24 columns are 2^41 threads of the largest tile,
    which no launch takes; a forced height whose grid is too large is refused where
    the automatic choice finds one that fits."""
    p, h = g(), unlaunched
    wide = dict(M=65536, groups=65536, strideB=0, dtype=2)
    assert raw_grouped(h, N=2 ** 24, ldb=2 ** 24, ldd=2 ** 24, **wide) == p.GEMM_ERR_NOT_SUPPORTED
    fits = dict(N=8192, ldb=8192, ldd=8192, **wide)
    assert raw_grouped(h, **fits) == p.GEMM_ERR_HIP
    assert p.gemm_set_group_tile(h, 16) == p.GEMM_OK
    assert raw_grouped(h, **fits) == p.GEMM_ERR_NOT_SUPPORTED
    assert raw_lora(h, M=2 ** 30, N=2 ** 10, ldb=2 ** 10, ldd=2 ** 10, ld_up=3, stride_up=2 ** 12,
                    bytes=1 << 62) == p.GEMM_ERR_NOT_SUPPORTED


def test_host_tensors_are_refused_on_a_given_stream(unlaunched):
    """... as on the current one: no pointer of host memory reaches a launch."""
    h, A, B, D = unlaunched, torch.zeros(4, 6), torch.zeros(2, 6, 5), torch.zeros(4, 5)
    off = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="GPU"):
        g().run_grouped(h, A, B, D, off, stream=0)
    with pytest.raises(ValueError, match="GPU"):
        g().run_grouped_wgrad(h, A, D, torch.zeros(2, 6, 5), off, stream=0)
    ws = torch.zeros(65536, dtype=torch.uint8)
    ws = ws[-ws.data_ptr() % 256:]
    with pytest.raises(ValueError, match="GPU"):
        g().run_lora(h, A, B[0], D, off, torch.zeros(2, 3, 6), torch.zeros(2, 5, 3), ws, stream=0)


@pytest.mark.parametrize("device,on", [(None, "cuda"), (0, 0), ("cuda:1", "cuda:1")])
def test_workspace_is_on_the_device_asked_for(device, on, monkeypatch):
    """Device 0 by its number is not the current device."""
    asked = []
    monkeypatch.setattr(torch, "empty", lambda *a, **kw: asked.append(kw["device"]))
    g().lora_workspace(4, 8, device)
    assert asked == [on]
