"""The ragged and adapted products at the sizes where their kernels change
course: several batches of K per wave, more tiles than one round over the
XCDs, tiles of one adapter, one launch for few rows.  References and bounds as
in test_grouped.py."""
from __future__ import annotations

import pytest
import torch

from .gpu_support import announce, require_gpu
from .test_grouped import (TYPES, bounds_of, check, draw, g, grouped_reference, handle, lora_reference,
                           padded)

gpu = pytest.mark.gpu


def int32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@gpu
@pytest.mark.parametrize("tile", [0, 16, 32, 64])
@pytest.mark.parametrize("trans", ["N", "T"])
@pytest.mark.parametrize("dtype", ["f32", "bf16_out"])
@pytest.mark.parametrize("K,N", [(4129, 70), (4224, 8), (2048, 3), (1300, 131), (1152, 64)])
def test_streaming_tiles_over_a_long_k(K, N, dtype, trans, tile):
    """Zero to five batches of K per wave, and a remainder of whole and ragged
    steps; columns that end inside a tile or fill none."""
    require_gpu()
    announce("long k", K, N, dtype, trans, tile)
    ti, to = TYPES[dtype]
    sizes = [33, 0, 5, 16]
    M = sum(sizes)
    A = draw((M, K), 1, ti)
    B = draw((4, K, N) if trans == "N" else (4, N, K), 2, ti)
    h = handle(tile)
    try:
        D = padded(torch.full((M, N), float("nan"), dtype=to), 1)
        g().run_grouped(h, A.cuda(), B.cuda(), D, int32(bounds_of(sizes)), transB=trans)
        val, den = grouped_reference(A, B, None, sizes, 0, trans, 1.0, 0.0, None)
        check(D.cpu(), val, den, K, "long k")
    finally:
        g().gemm_destroy(h)


@gpu
@pytest.mark.parametrize("tile", [16, 32, 64, 128, 192, 256])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_more_tiles_than_a_round_of_blocks(dtype, tile):
    """Several hundred tiles, in place with beta: each is written once."""
    require_gpu()
    announce("many tiles", dtype, tile)
    ti, to = TYPES[dtype]
    sizes, K, N = [200, 1, 0, 130, 257, 90], 40, 6000
    M = sum(sizes)
    A, B, C = draw((M, K), 1, ti), draw((6, K, N), 2, ti), draw((M, N), 3, to)
    h = handle(tile)
    try:
        D = C.cuda()
        g().run_grouped(h, A.cuda(), B.cuda(), D, int32(bounds_of(sizes)), C=D, beta=1.0)
        val, den = grouped_reference(A, B, C, sizes, 0, "N", 1.0, 1.0, None)
        check(D.cpu(), val, den, K, "many tiles")
    finally:
        g().gemm_destroy(h)


@gpu
@pytest.mark.parametrize("tile", [0, 64, 128, 192, 256])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "bf16_out"])
@pytest.mark.parametrize("sizes,M,N", [([0, 70, 300, 1], 520, 1100), ([0, 70, 300, 1], 520, 1152),
                                       ([600, 5, 0], 601, 899), ([2, 0, 1, 1], 100, 4000)])
def test_wgrad_deals_every_tile(sizes, M, N, dtype, tile):
    """Slices, ranges and single tiles per XCD, odd and even extents, rows of D on
    and off 128-byte lines; added to what is there."""
    require_gpu()
    announce("wgrad deal", sizes, M, N, dtype, tile)
    ti, to = TYPES[dtype]
    at = bounds_of(sizes, 1)
    G, rows = len(sizes), at[-1] + 1
    A, B, C = draw((rows, M), 1, ti), draw((rows, N), 2, ti), draw((G, M, N), 3, to)
    val = C.double()
    den = C.double().abs()
    for i in range(G):
        a, b = A[at[i]:at[i + 1]].double(), B[at[i]:at[i + 1]].double()
        val[i] += a.T @ b
        den[i] += a.abs().T @ b.abs()
    h = handle(tile)
    try:
        D = C.cuda()
        g().run_grouped_wgrad(h, A.cuda(), B.cuda(), D, int32(at), C=D, beta=1.0)
        check(D.cpu(), val, den, max(sizes), "wgrad deal")
    finally:
        g().gemm_destroy(h)


@gpu
@pytest.mark.parametrize("tile", [0, 32, 64])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "bf16_out"])
@pytest.mark.parametrize("M,N", [(8, 200), (3, 70), (65, 33), (64, 130), (1, 1)])
def test_wgrad_of_many_rows_and_few_columns(M, N, dtype, tile):
    """Several batches of rows per wave, a remainder, extents below and off a
    tile, factors and gradients added to."""
    require_gpu()
    announce("wgrad long", M, N, dtype, tile)
    ti, to = TYPES[dtype]
    sizes = [3000, 1, 0, 1153]
    at = bounds_of(sizes)
    A, B, C = draw((at[-1], M), 1, ti), draw((at[-1], N), 2, ti), draw((4, M, N), 3, to)
    s = draw((4,), 4, torch.float32)
    val = 0.5 * C.double()
    den = val.abs()
    for i in range(4):
        a, b = A[at[i]:at[i + 1]].double(), B[at[i]:at[i + 1]].double()
        val[i] += float(s[i]) * (a.T @ b)
        den[i] += abs(float(s[i])) * (a.abs().T @ b.abs())
    h = handle(tile)
    try:
        D = padded(torch.full((4, M, N), float("nan"), dtype=to), 1)
        g().run_grouped_wgrad(h, padded(A, 1, 1), padded(B, 3, 1), D, int32(at), C=C.cuda(), beta=0.5,
                              scales=s.cuda())
        check(D.cpu(), val, den, max(sizes), "wgrad long")
    finally:
        g().gemm_destroy(h)


@gpu
@pytest.mark.parametrize("tile", [64, 128, 192, 256])
@pytest.mark.parametrize("up", ["N", "T"])
@pytest.mark.parametrize("trans", ["N", "T"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("R", [8, 30, 64])
def test_lora_tiles_of_one_adapter(R, dtype, trans, up, tile):
    """Segments longer than a tile (with a boundary inside one, a segment without
    an adapter, rows of no segment), in every pairing of B's and up's layouts."""
    require_gpu()
    announce("one adapter", R, dtype, trans, up, tile)
    ti, to = TYPES[dtype]
    sizes, ids, K, N = [400, 300, 290], [2, -1, 0], 200, 272
    M = sum(sizes) + 50
    A, B = draw((M, K), 1, ti), draw((K, N) if trans == "N" else (N, K), 2, ti)
    dn, u = draw((3, R, K), 3, ti), draw((3, N, R), 4, ti)
    s = draw((3,), 5, torch.float32)
    h = handle(tile)
    try:
        D = torch.full((M, N), float("nan"), dtype=to, device="cuda")
        ws = g().lora_workspace(M, R)
        ws.fill_(255)
        u_ = u if up == "T" else u.transpose(1, 2).contiguous()
        g().run_lora(h, A.cuda(), B.cuda(), D, int32(bounds_of(sizes)), dn.cuda(), u_.cuda(), ws,
                     ids=int32(ids), scales=s.cuda(), transB=trans, transUp=up)
        val, den, low = lora_reference(A, B, None, sizes, 0, ids, dn, u, trans, 1.0, 0.0, s)
        check(D.cpu(), val, den, 2 * K + R, "one adapter", 2.0 ** -18 if dtype != "f32" else 0.0, low)
    finally:
        g().gemm_destroy(h)


@gpu
@pytest.mark.parametrize("tile", [0, 16])
@pytest.mark.parametrize("trans", ["N", "T"])
@pytest.mark.parametrize("dtype", ["f32", "bf16_out"])
@pytest.mark.parametrize("sizes,ids,R,K,N", [
    ([1], [1], 8, 2048, 100), ([16], [0], 32, 1545, 64), ([3, 9], [2, 0], 16, 700, 130),
    ([5, 4], [1, 1], 7, 1024, 33), ([2, 1], [-1, 1], 12, 96, 200), ([7, 2], [-1, 9], 5, 300, 16),
    ([0, 11], [0, 2], 3, 31, 6)])
def test_lora_of_few_rows_in_one_launch(sizes, ids, R, K, N, dtype, trans, tile):
    require_gpu()
    announce("one launch", sizes, ids, R, K, N, dtype, trans, tile)
    ti, to = TYPES[dtype]
    M = sum(sizes) + 1                               # the last row in no segment
    A, B = draw((M, K), 1, ti), draw((K, N) if trans == "N" else (N, K), 2, ti)
    dn, u, C = draw((3, R, K), 3, ti), draw((3, N, R), 4, ti), draw((M, N), 6, to)
    s = draw((3,), 5, torch.float32)
    h = handle(tile)
    try:
        D = padded(torch.full((M, N), float("nan"), dtype=to), 3)
        ws = g().lora_workspace(M, R)
        ws.fill_(255)
        g().run_lora(h, padded(A, 1), padded(B, 1), D, int32(bounds_of(sizes)), padded(dn, 1),
                     padded(u, 1), ws, ids=int32(ids), scales=s.cuda(), C=C.cuda(), beta=0.5,
                     transB=trans)
        val, den, low = lora_reference(A, B, C, sizes, 0, ids, dn, u, trans, 1.0, 0.5, s)
        check(D.cpu(), val, den, 2 * K + R, "one launch", 2.0 ** -18 if dtype != "f32" else 0.0, low)
    finally:
        g().gemm_destroy(h)


@gpu
@pytest.mark.parametrize("tile", [0, 16])
def test_lora_of_few_rows_keeps_requests_apart(tile):
    """Adapters of NaN and infinities reach their own request's rows only."""
    require_gpu()
    announce("few rows apart", tile)
    sizes, K, N, R = [4, 3], 640, 96, 8
    A, B = draw((7, K), 1, torch.bfloat16), draw((N, K), 2, torch.bfloat16)
    dn, u = draw((2, R, K), 3, torch.bfloat16), draw((2, N, R), 4, torch.bfloat16)
    h = handle(tile)
    try:
        for bad in (0, 1):
            d2, u2 = dn.clone(), u.clone()
            d2[bad, 0, 0] = float("nan")
            u2[bad, :, 1] = float("inf")
            D = torch.empty(7, N, device="cuda")
            g().run_lora(h, A.cuda(), B.cuda(), D, int32([0, 4, 7]), d2.cuda(), u2.cuda(),
                         g().lora_workspace(7, R), transB="T")
            got = D.cpu()
            val, den, low = lora_reference(A, B, None, sizes, 0, None, dn, u, "T", 1.0, 0.0, None)
            good = slice(4, 7) if bad == 0 else slice(0, 4)
            check(got[good], val[good], den[good], 2 * K + R, "clean rows", 2.0 ** -18, low[good])
            assert torch.isnan(got[0:4] if bad == 0 else got[4:7]).all()
    finally:
        g().gemm_destroy(h)


@gpu
@pytest.mark.parametrize("tile", [0, 16, 32, 64, 128, 192, 256])
def test_rows_past_32_bits(tile):
    """Groups whose rows lie 2^31 elements and 2^32 bytes into A, and
    matrices 1 GiB apart: the three calls on the last rows."""
    require_gpu()
    announce("past 32 bits", tile)
    bf16 = torch.bfloat16
    M, K, N, R, tail = 264000, 8192, 24, 8, 70
    sizes = [M - tail, 0, 41, 29]
    off = int32(bounds_of(sizes))
    A = torch.zeros(M, K, dtype=bf16, device="cuda")
    last = draw((tail, K), 1, bf16)
    A[M - tail:] = last.cuda()
    far = torch.zeros(4, 2 ** 30 // 2, dtype=bf16, device="cuda")   # matrices 2^30 bytes apart
    B = far.as_strided((4, N, K), (far.stride(0), K, 1))
    b = draw((4, N, K), 2, bf16)
    B.copy_(b.cuda())
    val, den = (torch.cat(x) for x in zip(*(
        (last[lo:hi].double() @ b[i].double().T, last[lo:hi].double().abs() @ b[i].double().abs().T)
        for i, lo, hi in ((2, 0, 41), (3, 41, 70)))))
    h = handle(tile)
    try:
        D = torch.full((M, N), 7.0, device="cuda")
        g().run_grouped(h, A, B, D, off, transB="T")
        check(D[M - tail:].cpu(), val, den, K, "rows")
        assert not D[:M - tail].any()
        dn, u = draw((4, R, K), 3, bf16), draw((4, N, R), 4, bf16)
        g().run_lora(h, A, B[0], D, off, dn.cuda(), u.cuda(), g().lora_workspace(M, R), transB="T")
        ref = lora_reference(last, b[0], None, [0, 0, 41, 29], 0, None, dn, u, "T", 1.0, 0.0, None)
        check(D[M - tail:].cpu(), ref[0], ref[1], 2 * K + R, "adapters", 2.0 ** -18, ref[2])
        assert not D[:M - tail].any()
        Y = torch.zeros(M, 8, dtype=bf16, device="cuda")
        y = draw((tail, 8), 5, bf16)
        Y[M - tail:] = y.cuda()
        dB = torch.empty(4, 8, K, device="cuda")
        g().run_grouped_wgrad(h, Y, A, dB, off)
        got = dB.cpu()
        assert not got[:2].any()
        for i, lo, hi in ((2, 0, 41), (3, 41, 70)):
            p, q = y[lo:hi].double(), last[lo:hi].double()
            check(got[i], p.T @ q, p.abs().T @ q.abs(), hi - lo, f"gradient {i}")
    finally:
        g().gemm_destroy(h)


def test_host_tensors_are_refused():
    """Nothing is launched on pointers of host memory."""
    h = g().gemm_create()
    A, B, D = torch.zeros(4, 6), torch.zeros(2, 6, 5), torch.zeros(4, 5)
    off = torch.zeros(3, dtype=torch.int32)
    try:
        with pytest.raises(ValueError, match="GPU"):
            g().run_grouped(h, A, B, D, off)
        with pytest.raises(ValueError, match="GPU"):
            g().run_grouped_wgrad(h, A, D, torch.zeros(2, 6, 5), off)
        with pytest.raises(ValueError, match="GPU"):
            g().run_lora(h, A, B[0], D, off, torch.zeros(2, 3, 6), torch.zeros(2, 5, 3),
                         torch.zeros(4096, dtype=torch.uint8))
    finally:
        g().gemm_destroy(h)
