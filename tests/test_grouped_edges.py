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
