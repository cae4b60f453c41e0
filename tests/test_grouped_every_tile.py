"""Every tile of the ragged and adapted products, forced one by one and checked
to be the one that ran, on sizes that end inside tiles and on sizes that fill
them.  References and bounds as in test_grouped.py, but a T of two bf16 terms
counts 2^-17: hi is off by half a step, 2^-8 of its binade, lo by half a step of
what is left."""
from __future__ import annotations

import pytest
import torch

from .gpu_support import announce, require_gpu
from .test_grouped import (TYPES, bounds_of, check, draw, g, grouped_reference, lora_reference, padded)
from .test_grouped_tiles import int32

gpu = pytest.mark.gpu

# (rows, columns with B stored K x N, with B stored N x K) of each call's tiles, by
# operand type, in the order of the numbers within a height
NARROW = {"bf16": (32, 16), "f32": (16, 16)}
STREAM = {t: [(32, 64, 64), (32, *n), (16, 64, 64), (16, *n)] for t, n in NARROW.items()}
ROWS = {"bf16": [(256, 256, 256), (192, 256, 256), (128, 256, 256), (128, 128, 128), (64, 128, 128),
                 (64, *NARROW["bf16"])] + STREAM["bf16"],
        "f32": [(128, 128, 128), (64, 128, 128)] + STREAM["f32"]}
LORA = {"bf16": [(256, 256, 256), (192, 256, 256), (128, 128, 128), (64, 128, 128),
                 (64, *NARROW["bf16"])] + STREAM["bf16"],
        "f32": [(128, 128, 128), (64, 128, 128)] + STREAM["f32"]}
ALONG_K = {"bf16": [(256, 256), (192, 256), (128, 256), (128, 128), (128, 128), (64, 64), (32, 32)],
           "f32": [(128, 128), (64, 128), (64, 64), (32, 32)]}


def operand(dtype):
    return "f32" if dtype == "f32" else "bf16"


def tiles(table):
    """(type, rows, nth, tile) of every entry for every output type."""
    out = []
    for dtype in TYPES:
        seen = {}
        for t in table[operand(dtype)]:
            nth = seen.setdefault(t[0], 0)
            seen[t[0]] += 1
            out.append((dtype, t[0], nth, t))
    return out


def forced(rows, nth):
    h = g().gemm_create()
    assert g().gemm_set_group_tile_nth(h, rows, nth) == g().GEMM_OK
    return h


def ran(h, rows, columns, nth, launches=1):
    x = g().gemm_last_group_launch(h)
    assert (x.rows, x.columns, x.nth, x.launches) == (rows, columns, nth, launches)
    assert g().gemm_last_group_tile(h) == rows
    return x


def ids(v):
    return "%s-%d.%d" % v[:3]


@gpu
@pytest.mark.parametrize("trans", ["N", "T"])
@pytest.mark.parametrize("K,N,pad", [(161, 515, 3), (1056, 512, 0)])
@pytest.mark.parametrize("tile", tiles(ROWS), ids=ids)
def test_rows(tile, K, N, pad, trans):
    require_gpu()
    dtype, rows, nth, cols = tile
    announce("rows tile", tile, K, N, trans)
    ti, to = TYPES[dtype]
    sizes = [0, 300, 1, 0, 257, 64, 17]
    M, G = sum(sizes) + 5, len(sizes)
    A, B, C = draw((M, K), 1, ti), draw((G, K, N) if trans == "N" else (G, N, K), 2, ti), draw((M, N), 3, to)
    s = draw((G,), 4, torch.float32)
    h = forced(rows, nth)
    try:
        D = padded(torch.full((M, N), 7.0, dtype=to), pad)
        g().run_grouped(h, padded(A, pad, pad), padded(B, pad, pad), D, int32(bounds_of(sizes, 2)),
                        C=padded(C, pad), transB=trans, alpha=0.5, beta=-1.0, scales=s.cuda())
        ran(h, rows, cols[1 + (trans == "T")], nth)
        val, den = grouped_reference(A, B, C, sizes, 2, trans, 0.5, -1.0, s)
        got, inside = D.cpu(), ~torch.isnan(val).any(dim=1)
        assert torch.all(got[~inside] == 7.0)
        check(got[inside], val[inside], den[inside], K, "rows")
    finally:
        g().gemm_destroy(h)


@gpu
@pytest.mark.parametrize("M,N,pad", [(261, 515, 3), (512, 384, 0), (40, 96, 0)])
@pytest.mark.parametrize("tile", tiles(ALONG_K), ids=ids)
def test_along_k(tile, M, N, pad):
    """Added in place to fp32 or bf16 gradients, and (pad 0) from alpha alone."""
    require_gpu()
    dtype, rows, nth, cols = tile
    announce("tile along k", tile, M, N)
    ti, to = TYPES[dtype]
    sizes = [0, 300, 1, 1290, 33]
    at, G = bounds_of(sizes, 1), len(sizes)
    A, B, C = draw((at[-1] + 2, M), 1, ti), draw((at[-1] + 2, N), 2, ti), draw((G, M, N), 3, to)
    s, beta = draw((G,), 4, torch.float32), 1.0 if pad else 0.0
    val, den = beta * C.double(), (beta * C.double()).abs()
    for i in range(G):
        a, b, f = A[at[i]:at[i + 1]].double(), B[at[i]:at[i + 1]].double(), 0.5 * float(s[i])
        val[i] += f * (a.T @ b)
        den[i] += abs(f) * (a.abs().T @ b.abs())
    h = forced(rows, nth)
    try:
        D = padded(C if beta else torch.full((G, M, N), float("nan"), dtype=to), pad)
        g().run_grouped_wgrad(h, padded(A, pad, pad), padded(B, pad, pad), D, int32(at),
                              C=D if beta else None, alpha=0.5, beta=beta, scales=s.cuda())
        ran(h, rows, cols[1], nth)
        check(D.cpu(), val, den, max(sizes), "along k")
    finally:
        g().gemm_destroy(h)


def adapted(h, dtype, trans, sizes, of, adapters, R, K, N, pad, down="T", up="T", ws_rows=None):
    """One call of run_lora in a workspace of NaN, checked; rows before and after
    the segments have no adapter."""
    ti, to = TYPES[dtype]
    M = sum(sizes) + 2
    A, B, C = draw((M, K), 1, ti), draw((K, N) if trans == "N" else (N, K), 2, ti), draw((M, N), 3, to)
    dn, u, s = draw((adapters, R, K), 4, ti), draw((adapters, N, R), 5, ti), draw((adapters,), 6, torch.float32)
    D = padded(torch.full((M, N), float("nan"), dtype=to), pad)
    ws = g().lora_workspace(M, R)
    ws.fill_(255)
    d_ = dn if down == "T" else dn.transpose(1, 2).contiguous()
    u_ = u if up == "T" else u.transpose(1, 2).contiguous()
    g().run_lora(h, padded(A, pad, pad), padded(B, pad, pad), D, int32(bounds_of(sizes, 1)),
                 padded(d_, pad, pad), padded(u_, pad, pad), ws, ids=int32(of), scales=s.cuda(),
                 C=padded(C, pad), transB=trans, transDown=down, transUp=up, alpha=0.5, beta=0.25)
    val, den, low = lora_reference(A, B, C, sizes, 1, of, dn, u, trans, 0.5, 0.25, s)
    check(D.cpu(), val, den, 2 * K + R, "adapted", 2.0 ** -17 if dtype != "f32" else 0.0, low)


@gpu
@pytest.mark.parametrize("trans", ["N", "T"])
@pytest.mark.parametrize("K,N,pad,layout", [(161, 515, 3, "T"), (1056, 512, 0, "N")])
@pytest.mark.parametrize("tile", tiles(LORA), ids=ids)
def test_adapted(tile, K, N, pad, layout, trans):
    require_gpu()
    dtype, rows, nth, cols = tile
    announce("adapted tile", tile, K, N, trans)
    h = forced(rows, nth)
    try:
        adapted(h, dtype, trans, [300, 1, 20, 0, 530, 64], [1, -1, 0, 1, 2, 0], 3, 24, K, N, pad, layout,
                layout)
        ran(h, rows, cols[1 + (trans == "T")], nth, 2)
    finally:
        g().gemm_destroy(h)


@gpu
@pytest.mark.parametrize("call", ["rows", "along k", "adapted"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_there_is_no_other_tile(dtype, call):
    """The lists above are whole: past a height's last tile the last is taken."""
    require_gpu()
    announce("no other tile", call, dtype)
    ti, to = TYPES[dtype]
    table = {"rows": ROWS, "along k": ALONG_K, "adapted": LORA}[call][dtype]
    A, B, D = (torch.zeros(40, 40, dtype=t, device="cuda") for t in (ti, ti, to))
    off = int32([0, 40])
    for height in sorted({t[0] for t in table}):
        above = min([t[0] for t in table if t[0] > height], default=1 << 20)
        for asked in (height, above - 1):            # and no height lies between
            h = forced(asked, 99)
            try:
                if call == "rows":
                    g().run_grouped(h, A, B[None], D, off)
                elif call == "along k":
                    g().run_grouped_wgrad(h, A, B, D[None], off)
                else:
                    g().run_lora(h, A, B, D, off, A[None, :20], A[None, :, :20], g().lora_workspace(40, 20))
                x = g().gemm_last_group_launch(h)
                assert (x.rows, x.nth) == (height, sum(t[0] == height for t in table) - 1)
            finally:
                g().gemm_destroy(h)


@gpu
@pytest.mark.parametrize("down", ["N", "T"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows", [16, 32])
@pytest.mark.parametrize("R", [5, 16, 24, 32, 40, 64, 90])
def test_first_product_of_the_adapters(R, rows, dtype, down):
    """Each of its tiles: 32 rows where the call has 16 rows per compute unit (4096),
    as wide as the rank needs."""
    require_gpu()
    announce("first product", R, rows, dtype, down)
    if torch.cuda.get_device_properties(0).multi_processor_count != 256:
        pytest.skip("sizes are for 256 compute units")
    sizes = [2500, 0, 1700, 60] if rows == 32 else [200, 0, 31, 60]
    widths = (16, 32, 64) if down == "T" or dtype == "f32" else (32, 32, 64)
    h = g().gemm_create()
    try:
        adapted(h, dtype, "T", sizes, [1, 0, 0, 2], 3, R, 300, 72, 1, down)
        x = g().gemm_last_group_launch(h)
        assert x.launches == 2 and (x.first_rows, x.first_columns) == (
            rows, next((w for w in widths if w >= R), 64))
    finally:
        g().gemm_destroy(h)


@gpu
@pytest.mark.parametrize("nth", [0, 1])
@pytest.mark.parametrize("trans", ["N", "T"])
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("sizes,of,R,down,launches", [
    ([7, 6], [0, 2], 16, "T", 1), ([14], [1], 32, "T", 1), ([1], [2], 5, "T", 1), ([9, 0], [-1, 0], 8, "T", 1),
    ([7, 6], [0, 2], 17, "T", 2), ([14], [1], 33, "T", 2), ([1], [2], 5, "N", 2), ([5, 5, 4], [0, 1, 2], 8, "T", 2)])
def test_few_rows_take_one_launch_or_two(sizes, of, R, down, launches, dtype, trans, nth):
    """Up to 16 rows in one launch where the adapters make two blocks of 16 ranks at
    most and down is stored by rank; wide and narrow tiles, K of several batches."""
    require_gpu()
    announce("one launch", sizes, of, R, down, dtype, trans, nth)
    h = forced(16, nth)
    try:
        adapted(h, dtype, trans, sizes, of, 3, R, 1413, 131, 1, down)
        ran(h, 16, STREAM[operand(dtype)][2 + nth][1 + (trans == "T")], nth, launches)
    finally:
        g().gemm_destroy(h)


@gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("sizes,of,R,K,launches", [
    ([14], [1], 32, 4096, 1), ([14], [1], 32, 4100, 2), ([7, 7], [1, 0], 8, 4096, 1),
    ([7, 7], [1, 0], 8, 8192, 2), ([14], [1], 16, 8192, 1), ([14], [1], 16, 8200, 2)])
def test_one_launch_by_the_length_of_down(sizes, of, R, K, launches, dtype):
    """Two blocks of ranks up to K = 4096, one up to 8192."""
    require_gpu()
    announce("length of down", sizes, R, K, dtype)
    h = forced(16, 0)
    try:
        adapted(h, dtype, "T", sizes, of, 2, R, K, 70, 0)
        ran(h, 16, 64, 0, launches)
    finally:
        g().gemm_destroy(h)


def test_forced_tiles_are_checked():
    p = g()
    h = p.gemm_create()
    try:
        assert p.gemm_set_group_tile_nth(h, 64, -1) == p.GEMM_ERR_INVALID_VALUE
        assert p.gemm_set_group_tile_nth(h, -1, 0) == p.GEMM_ERR_INVALID_VALUE
        assert p.gemm_set_group_tile_nth(None, 0, 0) == p.GEMM_ERR_INVALID_VALUE
        assert p.gemm_set_group_tile_nth(h, 64, 1) == p.GEMM_OK
        x = p.gemm_last_group_launch(h)
        assert (x.rows, x.columns, x.nth, x.launches, x.first_rows) == (0, 0, 0, 0, 0)
        assert p.lib.gemm_last_group_launch(h, None) == p.GEMM_ERR_INVALID_VALUE
        with pytest.raises(p.GemmError):
            p.gemm_last_group_launch(None)
    finally:
        p.gemm_destroy(h)
