"""Products over ragged groups of rows (run_grouped, run_grouped_wgrad,
run_lora) against the same formulas in 64 bits.

The bound on an element counts the roundings: every partial sum in fp32 is off
by at most one unit in its last place (2^-23, whatever the matrix
instructions' rounding) of the sum of the terms' magnitudes `den`, K terms
and a few more for alpha, beta and the low-rank sum; D's own rounding is half
a step of its type.  The low-rank path as bf16 operands carries T as two
terms, whose own rounding is 2^-18 of T.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

from .gpu_support import announce, require_gpu

TYPES = {"f32": (torch.float32, torch.float32), "bf16": (torch.bfloat16, torch.float32),
         "bf16_out": (torch.bfloat16, torch.bfloat16)}
gpu = pytest.mark.gpu


def g():
    import dense_gemm_11_amd
    return dense_gemm_11_amd


def bounds_of(sizes, lead=0):
    out = [lead]
    for s in sizes:
        out.append(out[-1] + s)
    return out


def draw(shape, seed, dtype):
    gen = torch.Generator().manual_seed(seed)
    return torch.randn(*shape, generator=gen).to(dtype)


def padded(host, pad=0, lead=0, fill=float("nan")):
    """A device view of `host` with `pad` more elements per row and `lead`
    elements before it; what lies outside the view is NaN."""
    *batch, rows, cols = host.shape
    buf = torch.full((lead + int(np.prod(batch or [1])) * rows * (cols + pad) + 8,), fill,
                     dtype=host.dtype, device="cuda")
    n = buf.numel() - 8 - lead
    view = buf[lead:lead + n].view(*batch, rows, cols + pad)[..., :cols]
    view.copy_(host.to("cuda"))
    return view


def check(got, val, den, terms, what, t_rel=0.0, low=None):
    """|got - val| within the bound of the module's docstring."""
    got64 = got.double().cpu()
    tol = (terms + 8) * 2.0 ** -23 * den
    if low is not None:
        tol = tol + t_rel * low
    tol = tol + torch.finfo(got.dtype).eps / 2 * (val.abs() + tol)
    bad = ~((got64 - val).abs() <= tol)
    worst = ((got64 - val).abs() / tol.clamp_min(1e-300)).max().item() if got.numel() else 0.0
    assert not bad.any(), f"{what}: {int(bad.sum())} elements off, worst {worst:.3g} of the bound"


def handle(tile=0):
    h = g().gemm_create()
    assert g().gemm_set_group_tile(h, tile) == g().GEMM_OK
    return h


# ---------------------------------------------------------------- rows
def grouped_reference(A, B, C, sizes, lead, trans, alpha, beta, scales):
    M, N = A.shape[0], (B.shape[2] if trans == "N" else B.shape[1])
    val = torch.full((M, N), float("nan"), dtype=torch.float64)
    den = torch.zeros(M, N, dtype=torch.float64)
    at = bounds_of(sizes, lead)
    for i in range(len(sizes)):
        r = slice(at[i], at[i + 1])
        a, b = A[r].double(), B[i].double()
        b = b if trans == "N" else b.T
        s = alpha * (float(scales[i]) if scales is not None else 1.0)
        val[r] = s * (a @ b)
        den[r] = abs(s) * (a.abs() @ b.abs())
        if beta != 0.0:
            val[r] += beta * C[r].double()
            den[r] += (beta * C[r].double()).abs()
    return val, den


ROW_CASES = [
    # sizes, rows before / after, K, N
    ([1], 0, 0, 64, 128),
    ([0, 3, 0, 1, 0], 0, 0, 40, 72),
    ([17, 0, 130, 1, 64], 5, 9, 96, 200),
    ([300, 129, 128, 127], 0, 3, 161, 257),
    ([2] * 70 + [0] * 60 + [5] * 10, 0, 0, 33, 65),
    ([513, 1, 256], 2, 0, 1, 300),
    ([90, 40], 0, 0, 515, 1),
]


@gpu
@pytest.mark.parametrize("tile", [0, 16, 64, 128, 256])
@pytest.mark.parametrize("trans", ["N", "T"])
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("case", range(len(ROW_CASES)))
def test_grouped(case, dtype, trans, tile):
    require_gpu()
    sizes, before, after, K, N = ROW_CASES[case]
    announce("grouped", sizes[:6], before, after, K, N, dtype, trans, tile)
    ti, to = TYPES[dtype]
    M, G = sum(sizes) + before + after, len(sizes)
    A = draw((M, K), 1, ti)
    B = draw((G, K, N) if trans == "N" else (G, N, K), 2, ti)
    C = draw((M, N), 3, to)
    # odd strides on every second case, beta and factors on every third
    pad = 3 if case % 2 else 0
    alpha, beta = (1.0, 0.0) if case % 3 else (0.75, -1.5)
    scales = None if case % 3 else draw((G,), 4, torch.float32)
    h = handle(tile)
    try:
        D = padded(torch.full((M, N), 7.0, dtype=to), pad)
        off = torch.tensor(bounds_of(sizes, before), dtype=torch.int32, device="cuda")
        g().run_grouped(h, padded(A, pad, pad), padded(B, pad, pad), D, off,
                        C=padded(C, pad) if beta else None, transB=trans, alpha=alpha, beta=beta,
                        scales=None if scales is None else scales.cuda())
        torch.cuda.synchronize()
        if tile:
            assert g().gemm_last_group_tile(h) <= max(tile, 128)
        val, den = grouped_reference(A, B, C, sizes, before, trans, alpha, beta, scales)
        inside = ~torch.isnan(val).any(dim=1)
        got = D.cpu()
        assert torch.all(got[~inside] == 7.0), "a row of no group was written"
        check(got[inside], val[inside], den[inside], K, "grouped")
    finally:
        g().gemm_destroy(h)


@gpu
@pytest.mark.parametrize("dtype", ["bf16_out", "f32"])
def test_grouped_in_place_and_shared_matrix(dtype):
    """C == D, one matrix for every group (stride 0), K == 0 and alpha == 0."""
    require_gpu()
    ti, to = TYPES[dtype]
    sizes, K, N = [5, 0, 40], 48, 96
    M = sum(sizes)
    A, B, C = draw((M, K), 1, ti), draw((1, K, N), 2, ti), draw((M, N), 3, to)
    off = torch.tensor(bounds_of(sizes), dtype=torch.int32, device="cuda")
    h = handle()
    try:
        announce("in place", dtype)
        D = C.cuda()
        g().run_grouped(h, A.cuda(), B.cuda().expand(3, K, N), D, off, C=D, beta=2.0)
        val, den = grouped_reference(A, B.expand(3, K, N), C, sizes, 0, "N", 1.0, 2.0, None)
        check(D.cpu(), val, den, K, "in place")
        for kw in (dict(alpha=0.0), dict()):
            a, b = (A.cuda(), B.cuda()) if kw else (A[:, :0].cuda(), B[:, :0].cuda())
            D = torch.empty(M, N, dtype=to, device="cuda")
            g().run_grouped(h, a, b.expand(3, *b.shape[1:]), D, off, C=C.cuda(), beta=0.5, **kw)
            check(D.cpu(), 0.5 * C.double(), (0.5 * C.double()).abs(), 0, "beta C")
    finally:
        g().gemm_destroy(h)


@gpu
@pytest.mark.parametrize("tile", [0, 16, 128])
def test_grouped_offsets_out_of_range_stay_inside(tile):
    """Offsets below 0, past M and decreasing are clamped: what the valid groups
    hold is right and nothing outside D is written."""
    require_gpu()
    M, K, N = 50, 64, 80
    A, B = draw((M, K), 1, torch.bfloat16), draw((4, K, N), 2, torch.bfloat16)
    off = torch.tensor([-9, 20, 12, 30, 4000], dtype=torch.int32, device="cuda")
    spans = [(0, 20), (20, 20), (12, 30), (30, 50)]   # clamped; 12..20 held twice
    h = handle(tile)
    try:
        announce("offsets out of range", tile)
        D = padded(torch.full((M + 4, N), 7.0), 5)
        g().run_grouped(h, A.cuda(), B.cuda(), D[:M], off)
        torch.cuda.synchronize()
        got = D.cpu()
        assert torch.all(got[M:] == 7.0)
        for i, (a, b) in enumerate(spans):
            lo, hi = (a, 12) if i == 0 else (20, b) if i == 2 else (a, b)
            val = A[lo:hi].double() @ B[i].double()
            den = A[lo:hi].double().abs() @ B[i].double().abs()
            check(got[lo:hi], val, den, K, f"group {i}")
    finally:
        g().gemm_destroy(h)


@gpu
@pytest.mark.parametrize("tile", [0, 16, 128, 256])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_grouped_infinities_stay_in_their_rows_and_groups(dtype, tile):
    """An infinity in one row, and a NaN matrix of one group, reach no other row."""
    require_gpu()
    ti, to = TYPES[dtype]
    sizes, K, N = [20, 7, 33], 70, 90
    M = sum(sizes)
    A, B = draw((M, K), 1, ti), draw((3, N, K), 2, ti)
    A[3, K - 1] = float("inf")
    A[40, 0] = float("nan")
    B[1].fill_(float("nan"))
    off = torch.tensor(bounds_of(sizes), dtype=torch.int32, device="cuda")
    h = handle(tile)
    try:
        announce("infinities", dtype, tile)
        D = torch.empty(M, N, dtype=to, device="cuda")
        g().run_grouped(h, padded(A, 1), padded(B, 1), D, off, transB="T")
        got = D.cpu()
        val, den = grouped_reference(A, B, None, sizes, 0, "T", 1.0, 0.0, None)
        clean = torch.ones(M, dtype=torch.bool)
        clean[[3, 40]] = False
        clean[20:27] = False
        check(got[clean], val[clean], den[clean], K, "clean rows")
        assert torch.equal(got[3].double(), val[3])          # infinities by the weights' signs
        assert torch.isnan(got[40]).all() and torch.isnan(got[20:27]).all()
    finally:
        g().gemm_destroy(h)


# ---------------------------------------------------------------- along K
K_CASES = [
    ([1], 0, 64, 128), ([0, 0], 0, 16, 24), ([31, 0, 32, 33, 1], 4, 130, 72),
    ([200, 64, 0, 95], 0, 257, 129), ([3] * 66, 1, 40, 33), ([700], 3, 1, 300), ([65, 66], 0, 300, 7),
]


@gpu
@pytest.mark.parametrize("tile", [0, 128, 256])
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("case", range(len(K_CASES)))
def test_grouped_wgrad(case, dtype, tile):
    require_gpu()
    sizes, lead, M, N = K_CASES[case]
    announce("wgrad", sizes[:6], lead, M, N, dtype, tile)
    ti, to = TYPES[dtype]
    rows, G = sum(sizes) + lead + 2, len(sizes)
    A, B, C = draw((rows, M), 1, ti), draw((rows, N), 2, ti), draw((G, M, N), 3, to)
    pad = 3 if case % 2 else 0
    alpha, beta = (1.0, 0.0) if case % 3 == 1 else (0.5, 1.0)
    scales = draw((G,), 4, torch.float32) if case % 3 == 2 else None
    at = bounds_of(sizes, lead)
    val = torch.zeros(G, M, N, dtype=torch.float64)
    den = torch.zeros_like(val)
    for i in range(G):
        a, b = A[at[i]:at[i + 1]].double(), B[at[i]:at[i + 1]].double()
        s = alpha * (float(scales[i]) if scales is not None else 1.0)
        val[i] = s * (a.T @ b) + beta * C[i].double()
        den[i] = abs(s) * (a.abs().T @ b.abs()) + (beta * C[i].double()).abs()
    h = handle(tile)
    try:
        off = torch.tensor(at, dtype=torch.int32, device="cuda")
        D = padded(torch.full((G, M, N), float("nan"), dtype=to), pad)
        Cd = padded(C, pad) if beta else None
        if case == 2:                      # gradients added in place
            D.copy_(C.cuda())
            Cd = D
        g().run_grouped_wgrad(h, padded(A, pad, pad), padded(B, pad, pad), D, off, C=Cd,
                              alpha=alpha, beta=beta,
                              scales=None if scales is None else scales.cuda())
        check(D.cpu(), val, den, max(sizes), "wgrad")
    finally:
        g().gemm_destroy(h)


@gpu
@pytest.mark.parametrize("tile", [128, 256])
def test_grouped_wgrad_leaves_other_groups_alone(tile):
    """NaN rows of one group reach no other group's gradient."""
    require_gpu()
    sizes, M, N = [33, 20, 45], 70, 130
    at = bounds_of(sizes)
    A, B = draw((98, M), 1, torch.bfloat16), draw((98, N), 2, torch.bfloat16)
    A[33:53] = float("nan")
    h = handle(tile)
    try:
        announce("wgrad nan group", tile)
        D = torch.empty(3, M, N, device="cuda")
        g().run_grouped_wgrad(h, A.cuda(), B.cuda(), D,
                              torch.tensor(at, dtype=torch.int32, device="cuda"))
        got = D.cpu()
        assert torch.isnan(got[1]).all()
        for i in (0, 2):
            a, b = A[at[i]:at[i + 1]].double(), B[at[i]:at[i + 1]].double()
            check(got[i], a.T @ b, a.abs().T @ b.abs(), sizes[i], f"group {i}")
    finally:
        g().gemm_destroy(h)


@gpu
def test_grouped_gradients_against_differences():
    """The two gradient calls against central differences of the forward call
    along random directions (f is linear in each operand, so the difference
    quotient has no truncation error of its own)."""
    require_gpu()
    sizes, K, N = [9, 0, 24, 1], 36, 44
    M = sum(sizes)
    A, B, dY = (draw((M, K), 1, torch.float32).cuda(), draw((4, K, N), 2, torch.float32).cuda(),
                draw((M, N), 3, torch.float32).cuda())
    dirA, dirB = draw((M, K), 4, torch.float32).cuda(), draw((4, K, N), 5, torch.float32).cuda()
    off = torch.tensor(bounds_of(sizes), dtype=torch.int32, device="cuda")
    h = handle()

    def loss(a, b):
        D = torch.empty(M, N, device="cuda")
        g().run_grouped(h, a, b, D, off)
        return float((D.double().cpu() * dY.double().cpu()).sum())

    try:
        announce("differences")
        dA, dB = torch.empty(M, K, device="cuda"), torch.empty(4, K, N, device="cuda")
        g().run_grouped(h, dY, B, dA, off, transB="T")
        g().run_grouped_wgrad(h, A, dY, dB, off)
        eps = 0.5
        for grad, d, f in ((dA, dirA, lambda e: loss(A + e * dirA, B)),
                           (dB, dirB, lambda e: loss(A, B + e * dirB))):
            slope = (f(eps) - f(-eps)) / (2 * eps)
            want = float((grad.double().cpu() * d.double().cpu()).sum())
            # fp32 sums of a few dozen terms, over M*N outputs of magnitude ~10 each
            assert abs(slope - want) <= 1e-4 * M * N
    finally:
        g().gemm_destroy(h)


# ---------------------------------------------------------------- adapters
LORA_CASES = [
    # segment sizes, ids, adapters, rank, K, N
    ([1], [0], 1, 8, 64, 96),
    ([1] * 20, None, 20, 16, 100, 130),
    ([1, 1, 30, 0, 1, 97], [2, -1, 0, 1, 2, 5], 3, 5, 129, 257),
    ([150, 140], [1, 1], 2, 33, 260, 140),
    ([40], [7], 2, 16, 64, 64),
    ([3, 0, 70, 1] * 18, [i % 5 - 1 for i in range(72)], 4, 64, 512, 300),
    ([600], [0], 1, 130, 96, 72),
]


def lora_reference(A, B, C, sizes, lead, ids, down, up, trans, alpha, beta, scales):
    a64, b64 = A.double(), (B if trans == "N" else B.T).double()
    val, den = a64 @ b64, a64.abs() @ b64.abs()
    low = torch.zeros_like(val)
    at = bounds_of(sizes, lead)
    for s in range(len(sizes)):
        i = s if ids is None else ids[s]
        if i < 0 or i >= down.shape[0]:
            continue
        r = slice(at[s], at[s + 1])
        d, u = down[i].double(), up[i].double()       # R x K, N x R
        f = float(scales[i]) if scales is not None else 1.0
        val[r] += f * (a64[r] @ d.T) @ u.T
        low[r] += abs(f) * (a64[r].abs() @ d.abs().T) @ u.abs().T
    val, den, low = alpha * val, abs(alpha) * (den + low), abs(alpha) * low
    if beta != 0.0:
        val, den = val + beta * C.double(), den + (beta * C.double()).abs()
    return val, den, low


@gpu
@pytest.mark.parametrize("tile", [0, 16, 128, 256])
@pytest.mark.parametrize("trans", ["N", "T"])
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("case", range(len(LORA_CASES)))
def test_lora(case, dtype, trans, tile):
    require_gpu()
    sizes, ids, adapters, R, K, N = LORA_CASES[case]
    announce("lora", sizes[:6], adapters, R, K, N, dtype, trans, tile)
    ti, to = TYPES[dtype]
    lead = 3 if case == 2 else 0
    M = sum(sizes) + 2 * lead
    A, B, C = draw((M, K), 1, ti), draw((K, N) if trans == "N" else (N, K), 2, ti), draw((M, N), 3, to)
    down, up = draw((adapters, R, K), 4, ti), draw((adapters, N, R), 5, ti)
    pad = 3 if case % 2 else 0
    alpha, beta = (1.0, 0.0) if case % 3 else (0.5, 1.25)
    scales = draw((adapters,), 6, torch.float32) if case % 2 else None
    flip = case in (2, 5)                       # the adapters in the gradient's layouts
    h = handle(tile)
    try:
        off = torch.tensor(bounds_of(sizes, lead), dtype=torch.int32, device="cuda")
        D = padded(torch.full((M, N), float("nan"), dtype=to), pad)
        d_, u_ = (down.transpose(1, 2).contiguous(), up.transpose(1, 2).contiguous()) if flip \
            else (down, up)
        ws = g().lora_workspace(M, R)
        ws.fill_(255)                            # NaN where nothing is written
        g().run_lora(h, padded(A, pad, pad), padded(B, pad, pad), D, off, padded(d_, pad, pad),
                     padded(u_, pad, pad), ws,
                     ids=None if ids is None else torch.tensor(ids, dtype=torch.int32, device="cuda"),
                     scales=None if scales is None else scales.cuda(),
                     C=padded(C, pad) if beta else None, transB=trans,
                     transDown="N" if flip else "T", transUp="N" if flip else "T", alpha=alpha,
                     beta=beta)
        val, den, low = lora_reference(A, B, C, sizes, lead, ids, down, up, trans, alpha, beta,
                                       scales)
        check(D.cpu(), val, den, 2 * K + R, "lora", 2.0 ** -18 if dtype != "f32" else 0.0, low)
    finally:
        g().gemm_destroy(h)


@gpu
@pytest.mark.parametrize("tile", [0, 16, 128])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_lora_keeps_requests_apart(dtype, tile):
    """An adapter of NaN and infinities, and a NaN row, reach no other request's rows."""
    require_gpu()
    ti, to = TYPES[dtype]
    sizes, ids, R, K, N = [4, 1, 9, 2, 30], [0, 1, 2, -1, 0], 8, 80, 70
    M = sum(sizes)
    A, B = draw((M, K), 1, ti), draw((N, K), 2, ti)
    down, up = draw((3, R, K), 3, ti), draw((3, N, R), 4, ti)
    down[1].fill_(float("nan"))
    up[2].fill_(float("inf"))
    A[20] = float("nan")
    h = handle(tile)
    try:
        announce("requests apart", dtype, tile)
        D = torch.empty(M, N, dtype=to, device="cuda")
        off = torch.tensor(bounds_of(sizes), dtype=torch.int32, device="cuda")
        g().run_lora(h, A.cuda(), B.cuda(), D, off, down.cuda(), up.cuda(),
                     g().lora_workspace(M, R), transB="T",
                     ids=torch.tensor(ids, dtype=torch.int32, device="cuda"))
        got = D.cpu()
        val, den, low = lora_reference(A, B, None, sizes, 0, ids, down, up, "T", 1.0, 0.0, None)
        clean = torch.ones(M, dtype=torch.bool)
        clean[4:14] = False
        clean[20] = False
        check(got[clean], val[clean], den[clean], 2 * K + R, "clean rows", 2.0 ** -18, low[clean])
        assert not torch.isfinite(got[4:14]).any() and torch.isnan(got[20]).all()
    finally:
        g().gemm_destroy(h)


@gpu
def test_lora_input_gradient_is_the_transposed_call():
    """dX of the adapted product by the same call with up and down exchanged."""
    require_gpu()
    sizes, R, K, N = [40, 25], 16, 192, 136
    M = sum(sizes)
    dY, B = draw((M, N), 1, torch.bfloat16), draw((N, K), 2, torch.bfloat16)
    down, up = draw((2, R, K), 3, torch.bfloat16), draw((2, N, R), 4, torch.bfloat16)
    s = torch.tensor([0.5, 2.0])
    h = handle()
    try:
        announce("lora input gradient")
        dX = torch.empty(M, K, device="cuda")
        off = torch.tensor(bounds_of(sizes), dtype=torch.int32, device="cuda")
        g().run_lora(h, dY.cuda(), B.cuda(), dX, off, up.cuda(), down.cuda(),
                     g().lora_workspace(M, R), scales=s.cuda(), transB="N", transDown="N",
                     transUp="N")
        # d/dX of <dY, X B^T + s (X down^T) up^T>
        val, den, low = lora_reference(dY, B, None, sizes, 0, None, up.transpose(1, 2),
                                       down.transpose(1, 2), "N", 1.0, 0.0, s)
        check(dX.cpu(), val, den, 2 * N + R, "dX", 2.0 ** -18, low)
    finally:
        g().gemm_destroy(h)


# ---------------------------------------------------------------- use
@gpu
def test_graph_replays_follow_the_offsets():
    """A captured step of the three calls, replayed after the offsets, ids and
    values change, equals the eager calls bit for bit."""
    require_gpu()
    M, K, N, G, R = 96, 64, 160, 5, 8
    A, B = torch.empty(M, K, dtype=torch.bfloat16, device="cuda"), torch.empty(
        G, N, K, dtype=torch.bfloat16, device="cuda")
    W = draw((N, K), 9, torch.bfloat16).cuda()
    down, up = draw((G, R, K), 10, torch.bfloat16).cuda(), draw((G, N, R), 11, torch.bfloat16).cuda()
    off = torch.empty(G + 1, dtype=torch.int32, device="cuda")
    ids = torch.empty(G, dtype=torch.int32, device="cuda")
    D, E = torch.empty(M, N, device="cuda"), torch.empty(M, N, device="cuda")
    dB = torch.empty(G, N, K, device="cuda")
    ws = g().lora_workspace(M, R)
    h = handle()

    def step():
        g().run_grouped(h, A, B, D, off, transB="T")
        g().run_lora(h, A, W, E, off, down, up, ws, ids=ids, transB="T")
        g().run_grouped_wgrad(h, Dh, A, dB, off)

    Dh = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")

    def fill(rep):
        gen = np.random.RandomState(rep)
        sizes = gen.multinomial(M, np.full(G, 1.0 / G) if rep % 2 else [0.9, 0, 0.1, 0, 0])
        off.copy_(torch.tensor(bounds_of([int(x) for x in sizes]), dtype=torch.int32))
        ids.copy_(torch.tensor(gen.randint(-1, G, G), dtype=torch.int32))
        A.copy_(draw((M, K), 20 + rep, torch.bfloat16))
        B.copy_(draw((G, N, K), 40 + rep, torch.bfloat16))
        Dh.copy_(draw((M, N), 60 + rep, torch.bfloat16))

    try:
        announce("graph")
        fill(0)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            step()
        torch.cuda.current_stream().wait_stream(s)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        for rep in range(4):
            fill(rep)
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            first = [t.clone() for t in (D, E, dB)]
            for t in (D, E, dB):
                t.fill_(float("nan"))
            step()
            torch.cuda.synchronize()
            for a, b in zip(first, (D, E, dB)):
                assert torch.equal(a.view(torch.int32), b.view(torch.int32)), rep
    finally:
        g().gemm_destroy(h)


@gpu
def test_other_stream():
    """A call on a stream of its own, ordered after its inputs by an event."""
    require_gpu()
    sizes, K, N = [100, 28], 256, 128
    A, B = draw((128, K), 1, torch.bfloat16), draw((2, K, N), 2, torch.bfloat16)
    h = handle()
    try:
        announce("stream")
        Ad, Bd, D = A.cuda(), B.cuda(), torch.empty(128, N, device="cuda")
        off = torch.tensor(bounds_of(sizes), dtype=torch.int32, device="cuda")
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        g().run_grouped(h, Ad, Bd, D, off, stream=s.cuda_stream)
        s.synchronize()
        val, den = grouped_reference(A, B, None, sizes, 0, "N", 1.0, 0.0, None)
        check(D.cpu(), val, den, K, "stream")
    finally:
        g().gemm_destroy(h)


# ---------------------------------------------------------------- refusals (no GPU)
FAKE = 0x100000  # never dereferenced: every call fails validation first


@pytest.fixture
def h():
    handle_ = g().gemm_create()
    yield handle_
    g().gemm_destroy(handle_)


def raw_grouped(h, **kw):
    p = g()
    a = dict(transB=0, M=4, N=5, K=6, alpha=1.0, A=FAKE, lda=6, B=FAKE, ldb=5, strideB=30, beta=0.0,
             C=None, ldc=5, D=FAKE, ldd=5, dtype=0, groups=2, offsets=FAKE, scales=None, null=False)
    a.update(kw)
    gr = None if a["null"] else p.GemmGroups(a["groups"], a["offsets"], a["scales"])
    return p.gemm_run_grouped(h, a["transB"], a["M"], a["N"], a["K"], a["alpha"], a["A"], a["lda"],
                              a["B"], a["ldb"], a["strideB"], a["beta"], a["C"], a["ldc"], a["D"],
                              a["ldd"], a["dtype"], gr, None)


@pytest.mark.parametrize("kw", [
    dict(transB=2), dict(dtype=3), dict(M=-1), dict(N=-1), dict(K=-1), dict(lda=5), dict(ldb=4),
    dict(transB=1, ldb=5), dict(ldd=4), dict(strideB=-1), dict(groups=-1), dict(null=True),
    dict(offsets=None), dict(A=None), dict(B=None), dict(D=None), dict(beta=1.0),
    dict(beta=1.0, C=FAKE, ldc=4), dict(beta=1.0, C=FAKE, ldc=6), dict(beta=1.0, C=FAKE + 8),
], ids=str)
def test_grouped_refuses(h, kw):
    assert raw_grouped(h, **kw) == g().GEMM_ERR_INVALID_VALUE
    assert raw_grouped(None) == g().GEMM_ERR_INVALID_VALUE


def test_grouped_limits_and_empty_calls(h):
    p = g()
    assert raw_grouped(h, M=2 ** 31) == p.GEMM_ERR_NOT_SUPPORTED
    assert raw_grouped(h, groups=65537) == p.GEMM_ERR_NOT_SUPPORTED
    assert raw_grouped(h, A=FAKE + 2) == p.GEMM_ERR_NOT_SUPPORTED            # not element-aligned
    assert raw_grouped(h, lda=2 ** 30) == p.GEMM_ERR_NOT_SUPPORTED           # panel past 4 GiB
    for kw in (dict(M=0), dict(N=0), dict(groups=0)):
        assert raw_grouped(h, A=None, B=None, D=None, offsets=None, **kw) == p.GEMM_OK
    assert p.gemm_last_group_tile(h) == 0 and p.gemm_last_group_tile(None) == -1
    assert p.gemm_set_group_tile(h, -1) == p.GEMM_ERR_INVALID_VALUE
    assert p.gemm_set_group_tile(None, 0) == p.GEMM_ERR_INVALID_VALUE


def raw_wgrad(h, **kw):
    p = g()
    a = dict(M=4, N=5, rows=6, alpha=1.0, A=FAKE, lda=4, B=FAKE, ldb=5, beta=0.0, C=None, ldc=5,
             strideC=20, D=FAKE, ldd=5, strideD=20, dtype=0, groups=2, offsets=FAKE)
    a.update(kw)
    return p.gemm_run_grouped_wgrad(
        h, a["M"], a["N"], a["rows"], a["alpha"], a["A"], a["lda"], a["B"], a["ldb"], a["beta"],
        a["C"], a["ldc"], a["strideC"], a["D"], a["ldd"], a["strideD"], a["dtype"],
        p.GemmGroups(a["groups"], a["offsets"], None), None)


@pytest.mark.parametrize("kw", [
    dict(dtype=-1), dict(M=-1), dict(N=-1), dict(rows=-1), dict(lda=3), dict(ldb=4), dict(ldd=4),
    dict(offsets=None), dict(A=None), dict(B=None), dict(D=None), dict(strideD=19), dict(strideD=0),
    dict(beta=1.0), dict(beta=1.0, C=FAKE, ldc=4), dict(beta=1.0, C=FAKE, strideC=21),
    dict(beta=1.0, C=FAKE + 64), dict(beta=1.0, C=4 * FAKE, strideC=-1), dict(groups=-1),
], ids=str)
def test_wgrad_refuses(h, kw):
    assert raw_wgrad(h, **kw) == g().GEMM_ERR_INVALID_VALUE
    assert raw_wgrad(None) == g().GEMM_ERR_INVALID_VALUE


def test_wgrad_empty_calls(h):
    for kw in (dict(M=0), dict(N=0), dict(groups=0)):
        assert raw_wgrad(h, A=None, B=None, D=None, offsets=None, **kw) == g().GEMM_OK
    assert raw_wgrad(h, rows=2 ** 31) == g().GEMM_ERR_NOT_SUPPORTED


def raw_lora(h, **kw):
    p = g()
    a = dict(transB=0, M=4, N=5, K=6, alpha=1.0, A=FAKE, lda=6, B=FAKE, ldb=5, beta=0.0, C=None,
             ldc=5, D=FAKE, ldd=5, dtype=0, segments=2, offsets=FAKE, ids=None, adapters=2, rank=3,
             trans_down=1, down=FAKE, ld_down=6, stride_down=18, trans_up=1, up=FAKE, ld_up=3,
             stride_up=15, ws=FAKE, bytes=1 << 20)
    a.update(kw)
    lo = p.GemmLora(a["segments"], a["offsets"], a["ids"], a["adapters"], a["rank"], None,
                    a["trans_down"], a["down"], a["ld_down"], a["stride_down"], a["trans_up"],
                    a["up"], a["ld_up"], a["stride_up"])
    return p.gemm_run_lora(h, a["transB"], a["M"], a["N"], a["K"], a["alpha"], a["A"], a["lda"],
                           a["B"], a["ldb"], a["beta"], a["C"], a["ldc"], a["D"], a["ldd"],
                           a["dtype"], lo, a["ws"], a["bytes"], None)


@pytest.mark.parametrize("kw", [
    dict(transB=3), dict(dtype=9), dict(M=-1), dict(segments=-1), dict(adapters=-1), dict(rank=-1),
    dict(trans_down=2), dict(trans_up=-1), dict(ld_down=5), dict(trans_down=0, ld_down=2),
    dict(ld_up=2), dict(trans_up=0, ld_up=4), dict(stride_down=-1), dict(stride_up=-1),
    dict(offsets=None), dict(down=None), dict(up=None), dict(A=None), dict(B=None), dict(D=None),
    dict(ws=None), dict(ws=FAKE + 16), dict(bytes=64), dict(beta=1.0), dict(beta=1.0, C=FAKE + 4),
    dict(lda=5), dict(ldb=4), dict(ldd=4),
], ids=str)
def test_lora_refuses(h, kw):
    assert raw_lora(h, **kw) == g().GEMM_ERR_INVALID_VALUE
    assert raw_lora(None) == g().GEMM_ERR_INVALID_VALUE


def test_lora_limits_and_empty_calls(h):
    p = g()
    assert raw_lora(h, M=0, A=None, D=None, ws=None) == p.GEMM_OK
    assert raw_lora(h, up=FAKE + 2) == p.GEMM_ERR_NOT_SUPPORTED
    assert raw_lora(h, segments=65537) == p.GEMM_ERR_NOT_SUPPORTED
    assert p.gemm_lora_workspace_bytes(0, 8) == p.gemm_lora_workspace_bytes(8, 0) == 0
    sizes = [p.gemm_lora_workspace_bytes(m, 17) for m in (1, 2, 511, 512, 513, 4097, 8191, 9000, 20000)]
    assert sizes == sorted(sizes)                # serves every smaller call too


def test_tensor_calls_check_their_arguments(h):
    p = g()
    A, B, D = torch.zeros(4, 6), torch.zeros(2, 6, 5), torch.zeros(4, 5)
    off = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError):
        p.run_grouped(h, A, B, D, off.long())
    with pytest.raises(ValueError):
        p.run_grouped(h, A, B, D, off[:2])
    with pytest.raises(ValueError):
        p.run_grouped(h, A, B, D, off, transB="T")
    with pytest.raises(ValueError):
        p.run_grouped(h, A.t(), B, D, off)
    with pytest.raises(TypeError):
        p.run_grouped(h, A.bfloat16(), B, D, off)
    with pytest.raises(TypeError):
        p.run_grouped(h, A, B, D.bfloat16(), off)
    with pytest.raises(ValueError):
        p.run_grouped_wgrad(h, A, D, torch.zeros(2, 5, 6), off)
    with pytest.raises(ValueError):
        p.run_lora(h, A, B[0], D, off, torch.zeros(2, 3, 6), torch.zeros(2, 4, 3),
                   torch.zeros(4096, dtype=torch.uint8))
    with pytest.raises(TypeError):
        p.run_lora(h, A, B[0], D, off, torch.zeros(2, 3, 6).bfloat16(), torch.zeros(2, 5, 3),
                   torch.zeros(4096, dtype=torch.uint8))
