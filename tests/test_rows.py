"""Rows to their experts and back (run_gather_rows, run_combine_rows and its
gradient) against the same sums in 64 bits.

A sum of n products in fp32 is off by at most n + 2 units of 2^-24 of the sum of
their magnitudes, whatever its order; each output adds half a step of its type.
"""
from __future__ import annotations

import pytest
import torch

from .gpu_support import announce, require_gpu

gpu = pytest.mark.gpu
TYPES = {"f32": (torch.float32, torch.float32), "bf16": (torch.bfloat16, torch.float32),
         "bf16_out": (torch.bfloat16, torch.bfloat16)}
# tokens, top, cols
CASES = [(1, 1, 1), (1, 2, 2048), (7, 3, 5), (33, 8, 129), (100, 1, 64), (130, 5, 1537), (64, 4, 4097),
         (3, 9, 20000), (300, 2, 8)]


def g():
    import dense_gemm_11_amd
    return dense_gemm_11_amd


def randn(*shape, seed, dtype=torch.float32):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype)


def wide(host, pad, lead, fill=float("nan")):
    """A device view of host with `pad` elements more to a row and `lead` before it."""
    rows, cols = host.shape
    buf = torch.full((lead + rows * (cols + pad) + 8,), fill, dtype=host.dtype, device="cuda")
    view = buf[lead:lead + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]
    view.copy_(host)
    return view


def plan(tokens, top, seed, gaps=True):
    """Assignments in a random order, some in no row, and rows behind the last."""
    gen = torch.Generator().manual_seed(seed)
    live = torch.randperm(tokens * top, generator=gen)
    live = live[:max(1, live.numel() * 4 // 5)] if gaps else live
    rows = live.numel() + (3 if gaps else 0)
    order = torch.full((rows,), -1)
    order[:live.numel()] = live
    position = torch.full((tokens * top,), -1)
    position[live] = torch.arange(live.numel())
    return order.int(), position.int().view(tokens, top), rows


@pytest.fixture
def h():
    handle = g().gemm_create()
    yield handle
    g().gemm_destroy(handle)


def within(got, val, mag, units):
    tol = units * 2.0 ** -24 * mag
    tol = tol + torch.finfo(got.dtype).eps / 2 * (val.abs() + tol)
    err = (got.double().cpu() - val).abs()
    assert (err <= tol).all(), (err / tol.clamp_min(1e-300)).max()


@gpu
@pytest.mark.parametrize("weighted", [False, True])
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("case", range(len(CASES)))
def test_gather(h, case, dtype, weighted):
    require_gpu()
    T, top, cols = CASES[case]
    announce("gather", T, top, cols, dtype, weighted)
    ti, to = TYPES[dtype]
    order, _, rows = plan(T, top, case)
    if rows > 2:
        order[1] = T * top + 5                    # beyond the assignments: left alone
    X, w = randn(T, cols, seed=1, dtype=ti), randn(T, top, seed=2)
    pad, lead = case % 3, case % 2
    D = wide(torch.full((rows, cols), 7.0, dtype=to), pad, lead, 5.0)
    g().run_gather_rows(h, wide(X, pad, lead), D, order.cuda(), top, weights=w.cuda() if weighted else None)
    torch.cuda.synchronize()
    got = D.cpu()
    live = (order >= 0) & (order < T * top)
    assert (got[~live] == 7.0).all(), "a row of no assignment was written"
    a = order[live].long()
    val = X.double()[a // top]
    if weighted:
        val = val * w.double().view(-1)[a][:, None]
        within(got[live], val, val.abs(), 1)
    else:
        assert torch.equal(got[live].double(), val)


@gpu
@pytest.mark.parametrize("weighted", [False, True])
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("case", range(len(CASES)))
def test_combine(h, case, dtype, weighted):
    require_gpu()
    T, top, cols = CASES[case]
    announce("combine", T, top, cols, dtype, weighted)
    ti, to = TYPES[dtype]
    _, position, rows = plan(T, top, case)
    Y, w = randn(rows, cols, seed=1, dtype=ti), randn(T, top, seed=2)
    Y[-3:] = float("nan")                         # rows that no position names
    if T > 2:
        position[1, 0] = rows                     # beyond the rows: no part
    beta = (0.0, -1.5, 1.0)[case % 3]
    C = randn(T, cols, seed=3, dtype=to)
    pad, lead = case % 3, case % 2
    Cd = wide(C, pad, lead) if beta else wide(torch.full_like(C, float("nan")), pad, lead)
    D = Cd if case % 2 else wide(torch.zeros_like(C), pad + 1, lead, 5.0)
    g().run_combine_rows(h, wide(Y, pad, lead), D, position.cuda(), weights=w.cuda() if weighted else None,
                         C=Cd, beta=beta)
    torch.cuda.synchronize()
    val, mag = torch.zeros(T, cols, dtype=torch.float64), torch.zeros(T, cols, dtype=torch.float64)
    for j in range(top):
        at = position[:, j].long()
        in_ = (at >= 0) & (at < rows)
        part = Y.double()[at[in_]] * (w.double()[in_, j, None] if weighted else 1.0)
        val[in_] += part
        mag[in_] += part.abs()
    if beta:
        val += beta * C.double()
        mag += (beta * C.double()).abs()
    within(D.cpu(), val, mag, 2 * top + 4)


@gpu
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("case", range(len(CASES)))
def test_combine_grad(h, case, dtype, in_place):
    require_gpu()
    T, top, cols = CASES[case]
    announce("combine grad", T, top, cols, dtype, in_place)
    ti, to = TYPES[dtype]
    _, position, rows = plan(T, top, case)
    Y, w, dD = randn(rows, cols, seed=1, dtype=ti), randn(T, top, seed=2), randn(T, cols, seed=3, dtype=to)
    pad, lead = case % 3, case % 2
    Yd = wide(Y, pad, lead)
    dY = Yd if in_place else wide(torch.full_like(Y, 7.0), pad + 1, lead, 5.0)
    dw = torch.full((T, top), 9.0, device="cuda")
    g().run_combine_rows_grad(h, Yd, wide(dD, pad, lead), dY, dw, position.cuda(), w.cuda())
    torch.cuda.synchronize()
    got, dw = dY.cpu(), dw.cpu()
    named = torch.zeros(rows, dtype=torch.bool)
    for j in range(top):
        at = position[:, j].long()
        in_ = at >= 0
        named[at[in_]] = True
        val = w.double()[in_, j, None] * dD.double()[in_]
        within(got[at[in_]], val, val.abs(), 1)
        prod = Y.double()[at[in_]] * dD.double()[in_]
        within(dw[in_, j], prod.sum(1), prod.abs().sum(1), cols + 2)
        assert (dw[~in_, j] == 0).all()
    kept = got[~named]
    assert torch.equal(kept, Y[~named]) if in_place else (kept == 7.0).all()


@gpu
def test_without_rows_and_without_columns(h):
    require_gpu()
    announce("no rows")
    position = torch.full((5, 2), -1, dtype=torch.int32, device="cuda")
    w = torch.ones(5, 2, device="cuda")
    none, C = torch.empty(0, 12, device="cuda"), randn(5, 12, seed=1).cuda()
    D = torch.empty(5, 12, device="cuda")
    g().run_combine_rows(h, none, D, position, weights=w, C=C, beta=2.0)
    assert torch.equal(D, 2 * C)
    dw = torch.ones(5, 2, device="cuda")
    g().run_combine_rows_grad(h, none, C, none, dw, position, w)
    assert (dw == 0).all()
    g().run_gather_rows(h, C, none, torch.empty(0, dtype=torch.int32, device="cuda"), 2)
    dw.fill_(1)
    g().run_combine_rows_grad(h, torch.empty(3, 0, device="cuda"), torch.empty(5, 0, device="cuda"),
                              torch.empty(3, 0, device="cuda"), dw, position, w)
    assert (dw == 0).all()


@gpu
def test_rows_past_2_31_elements(h):
    """Rows whose offsets pass 32 bits, in elements and bytes."""
    require_gpu()
    announce("rows past 2^31 elements")
    cols, rows = 4096, (1 << 19) + 70
    Y = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda")
    position = torch.tensor([[rows - 1, 3], [rows - 60, 1 << 19]], dtype=torch.int32, device="cuda")
    at = position.long().view(-1)
    Y[at] = randn(4, cols, seed=4, dtype=torch.bfloat16).cuda()
    D = torch.empty(2, cols, dtype=torch.float32, device="cuda")
    g().run_combine_rows(h, Y, D, position)
    assert torch.equal(D, Y[position.long()].float().sum(1))
    order = torch.full((rows,), -1, dtype=torch.int32, device="cuda")
    order[at] = torch.arange(4, dtype=torch.int32, device="cuda")
    X = randn(2, cols, seed=5, dtype=torch.bfloat16).cuda()
    g().run_gather_rows(h, X, Y, order, 2)
    assert torch.equal(Y[at], X[torch.tensor([0, 0, 1, 1], device="cuda")])


# ---------------------------------------------------------------- refusals
FAKE, FAR = 0x100000, 0x100000 + (1 << 30)


def test_gather_refusals(h):
    m = g()

    def call(hh=h, **kw):
        a = dict(tokens=10, cols=8, top=2, X=FAKE, ldx=8, rows=20, order=FAKE, weights=None, D=FAR, ldd=8,
                 dtype=0)
        a.update(kw)
        return m.gemm_gather_rows(hh, *[a[k] for k in ("tokens", "cols", "top", "X", "ldx", "rows", "order",
                                                       "weights", "D", "ldd", "dtype")], None)
    assert call(None) == m.GEMM_ERR_INVALID_VALUE
    for kw in (dict(tokens=-1), dict(cols=-1), dict(rows=-1), dict(top=0), dict(ldx=7), dict(ldd=7),
               dict(X=None), dict(order=None), dict(D=None), dict(D=FAKE + 32), dict(dtype=3),
               dict(order=FAR + 632), dict(weights=FAR - 76)):
        assert call(**kw) == m.GEMM_ERR_INVALID_VALUE, kw
    for kw in (dict(tokens=1 << 24), dict(rows=1 << 24, D=FAKE + (1 << 40)), dict(top=1 << 30),
               dict(cols=1 << 27, ldx=1 << 27, ldd=1 << 27, D=FAKE + (1 << 40)), dict(X=FAKE + 2),
               dict(D=FAR + 1), dict(order=FAKE + 2), dict(weights=FAKE + 3), dict(ldx=1 << 31, D=FAKE + (1 << 50))):
        assert call(**kw) == m.GEMM_ERR_NOT_SUPPORTED, kw
    assert call(rows=0, D=None) == m.GEMM_OK and call(cols=0, X=None) == m.GEMM_OK


def test_combine_refusals(h):
    m = g()

    def call(**kw):
        a = dict(tokens=10, cols=8, top=2, Y=FAKE, ldy=8, rows=20, position=FAKE, weights=None, beta=0.0,
                 C=None, ldc=8, D=FAR, ldd=8, dtype=0)
        a.update(kw)
        return m.gemm_combine_rows(h, *[a[k] for k in ("tokens", "cols", "top", "Y", "ldy", "rows", "position",
                                                       "weights", "beta", "C", "ldc", "D", "ldd", "dtype")], None)
    for kw in (dict(tokens=-1), dict(top=-1), dict(ldy=7), dict(ldd=7), dict(Y=None), dict(position=None),
               dict(D=None), dict(D=FAKE + 32), dict(beta=1.0), dict(beta=1.0, C=FAR, ldc=7),
               dict(beta=1.0, C=FAR, ldc=9), dict(beta=1.0, C=FAR + 32), dict(dtype=-1),
               dict(position=FAR + 316), dict(weights=FAR)):
        assert call(**kw) == m.GEMM_ERR_INVALID_VALUE, kw
    for kw in (dict(tokens=1 << 24, D=FAKE + (1 << 40)), dict(Y=FAKE + 1), dict(position=FAKE + 1),
               dict(beta=1.0, C=FAR + (1 << 20) + 2), dict(weights=FAKE + 2)):
        assert call(**kw) == m.GEMM_ERR_NOT_SUPPORTED, kw
    assert call(tokens=0, D=None) == m.GEMM_OK


def test_combine_grad_refusals(h):
    m = g()

    def call(**kw):
        a = dict(tokens=10, cols=8, top=2, Y=FAKE, ldy=8, rows=20, position=FAKE, weights=FAKE, dD=FAKE,
                 lddd=8, dY=FAR, lddy=8, dw=FAR + (1 << 20), dtype=0)
        a.update(kw)
        return m.gemm_combine_rows_grad(h, *[a[k] for k in ("tokens", "cols", "top", "Y", "ldy", "rows",
                                                            "position", "weights", "dD", "lddd", "dY", "lddy",
                                                            "dw", "dtype")], None)
    for kw in (dict(rows=-1), dict(lddd=7), dict(lddy=7), dict(Y=None), dict(weights=None), dict(dw=None),
               dict(dD=None), dict(dY=None), dict(dY=FAKE + 32), dict(dY=FAKE, lddy=9), dict(dD=FAR),
               dict(dtype=7), dict(dw=FAKE), dict(dw=FAR + 636), dict(position=FAR), dict(weights=FAR + 4),
               dict(weights=FAR + (1 << 20) + 76)):
        assert call(**kw) == m.GEMM_ERR_INVALID_VALUE, kw
    for kw in (dict(tokens=1 << 24, dY=FAKE + (1 << 40)), dict(dD=FAKE + 2), dict(dw=FAR + (1 << 20) + 2)):
        assert call(**kw) == m.GEMM_ERR_NOT_SUPPORTED, kw
    assert call(tokens=0, dD=None) == m.GEMM_OK


def test_failed_launches_are_reported(monkeypatch):
    m = g()
    monkeypatch.setenv("GEMM_DEBUG_FAIL_LAUNCH", "1")
    hh = m.gemm_create()
    assert m.gemm_gather_rows(hh, 10, 8, 2, FAKE, 8, 20, FAKE, None, FAR, 8, 0, None) == m.GEMM_ERR_HIP
    assert m.gemm_combine_rows(hh, 10, 8, 2, FAKE, 8, 20, FAKE, None, 0.0, None, 8, FAR, 8, 0,
                               None) == m.GEMM_ERR_HIP
    assert m.gemm_combine_rows_grad(hh, 10, 8, 2, FAKE, 8, 20, FAKE, FAKE, FAKE, 8, FAR, 8, FAR + 4096, 0,
                                    None) == m.GEMM_ERR_HIP
    m.gemm_destroy(hh)


def test_binding_refuses_wrong_tensors(h):
    m = g()
    X, D = torch.zeros(4, 8), torch.zeros(8, 8)
    order, position, w = torch.zeros(8, dtype=torch.int32), torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2)
    with pytest.raises(ValueError, match="GPU"):
        m.run_gather_rows(h, X, D, order, 2)
    with pytest.raises(ValueError):
        m.run_gather_rows(h, X[:, :7], D, order, 2)
    with pytest.raises(TypeError):
        m.run_gather_rows(h, X.half(), D, order, 2)
    with pytest.raises(ValueError, match="GPU"):
        m.run_combine_rows(h, D, X, position, w)
    with pytest.raises(ValueError):
        m.run_combine_rows(h, D, X, position, w, C=X[:3], beta=1.0)
    with pytest.raises(TypeError):
        m.run_combine_rows_grad(h, D, X, D.bfloat16(), w, position, w)
    with pytest.raises(ValueError, match="GPU"):
        m.run_combine_rows_grad(h, D, X, D.clone(), w, position, w)
