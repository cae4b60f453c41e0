"""The example of the ragged products: its layer's gradients against the same
layer in 64 bits, and a short run of the whole."""
from __future__ import annotations

import importlib.util
import os

import pytest
import torch

from .gpu_support import announce, require_gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def example():
    spec = importlib.util.spec_from_file_location(
        "experts_and_adapters", os.path.join(ROOT, "examples", "experts_and_adapters.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def test_route_sorts_rows_by_expert():
    gen = torch.Generator().manual_seed(0)
    scores = torch.randn(50, 6, generator=gen)
    scores[:, 4] = -100.0                             # an expert that no token takes
    token, gate, offsets = example().route(scores, 2)
    expert = torch.topk(torch.softmax(scores, 1), 2, dim=1).indices
    at = offsets.tolist()
    assert at[0] == 0 and at[-1] == 100 and at[4] == at[5] and len(token) == 100
    for e in range(6):
        rows = token[at[e]:at[e + 1]].tolist()
        assert rows == [t for t in range(50) if e in expert[t].tolist()]
    assert torch.equal(offsets, torch.tensor(at, dtype=torch.int32))


@pytest.mark.gpu
def test_expert_layer_gradients():
    """fp32 operands, against autograd of the plain layer in 64 bits.  Each value
    is a sum of at most a few hundred products of order 1, so fp32 sums are off
    by under 512 * 2^-23 of the sums' magnitude, about 1e-4 of the largest."""
    require_gpu()
    announce("expert layer")
    ex = example()
    layer = ex.Experts(5, 48, 72, dtype=torch.float32)
    try:
        gen = torch.Generator(device="cuda").manual_seed(3)
        X = torch.randn(60, 48, generator=gen, device="cuda")
        scores = torch.randn(60, 5, generator=gen, device="cuda")
        dY = torch.randn(60, 48, generator=gen, device="cuda")
        Y, saved = layer.forward(X, scores, 2)
        got = [t.double().cpu() for t in (Y, *layer.backward(dY, saved))]
        x, w1, w2 = (t.double().cpu().requires_grad_() for t in (X, layer.w_in, layer.w_out))
        gate, expert = torch.topk(torch.softmax(scores.float(), 1), 2, dim=1)
        rows = [sum(float(gate[t, k]) * (torch.relu(x[t] @ w1[e].T) @ w2[e].T)
                    for k, e in enumerate(expert[t].tolist())) for t in range(60)]
        y = torch.stack(rows)
        y.backward(dY.double().cpu())
        for a, b in zip(got, (y.detach(), x.grad, w1.grad, w2.grad)):
            assert (a - b).abs().max() <= 1e-4 * b.abs().max()
    finally:
        layer.close()


@pytest.mark.gpu
def test_example_runs(capsys):
    require_gpu()
    announce("example")
    losses = example().main(["--tokens", "200", "--experts", "6", "--width", "256", "--hidden", "128",
                             "--steps", "3", "--requests", "9", "--adapters", "3"])
    assert losses[-1] < losses[0]
    assert "finite: True" in capsys.readouterr().out
