"""A layer of gated experts made of the library's calls, both directions (the
example's layer), against autograd of the same layer in 64 bits; captured and
replayed; and two layers on two streams at once."""
from __future__ import annotations

import importlib.util
import os

import pytest
import torch

from .gpu_support import announce, require_gpu

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    require_gpu()
    spec = importlib.util.spec_from_file_location("gated_experts",
                                                  os.path.join(ROOT, "examples", "gated_experts.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def randn(*shape, seed, dtype=torch.float32):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype)


def plain(x, wr, wi, wo, ids, kind, renorm, scale):
    """The layer for given choices, token by token, in x's type."""
    hidden = wo.shape[2]
    logits = x @ wr.T
    s = torch.softmax(logits, 1) if kind == "softmax" else torch.sigmoid(logits)
    out = []
    for t in range(x.shape[0]):
        chosen = [e for e in ids[t].tolist() if e >= 0]
        w = [s[t, e] for e in chosen]
        total = sum(w) if renorm and w else 1.0
        y = x[t]
        for e, v in zip(chosen, w):
            z = wi[e] @ x[t]
            y = y + scale * v / total * (wo[e] @ (torch.nn.functional.silu(z[:hidden]) * z[hidden:]))
        out.append(y)
    return torch.stack(out)


@pytest.mark.parametrize("kind,renorm,scale", [("softmax", True, 1.0), ("softmax", False, 2.0),
                                               ("sigmoid", True, 2.5), ("sigmoid", False, 1.0)])
def test_layer_gradients(example, kind, renorm, scale):
    """fp32 throughout.  Every value is a chain of sums of at most a few hundred
    products, each off by under 512 units of 2^-23 of its magnitude: 1e-4 of the
    largest, as for the layer without gates."""
    announce("gated layer", kind, renorm, scale)
    T, E, top, width, hidden = 60, 6, 2, 48, 72
    layer = example.GatedExperts(T, E, top, width, hidden, dtype=torch.float32, scores=kind,
                                 renormalize=renorm, scale=scale)
    try:
        X, dY = randn(T, width, seed=3), randn(T, width, seed=4)
        mask = torch.zeros(T, 1)
        mask[50:] = -float("inf")
        Y = layer.forward(X.cuda(), mask.cuda())
        got = [Y] + list(layer.backward(X.cuda(), dY.cuda()))
        torch.cuda.synchronize()
        ids = layer.ids.cpu()
        assert (ids[50:] == -1).all() and (ids[:50] >= 0).all()
        leaves = [v.double().cpu().requires_grad_() for v in (X, layer.w_router, layer.w_in, layer.w_out)]
        y = plain(*leaves, ids, kind, renorm, scale)
        y.backward(dY.double())
        assert torch.equal(got[0].cpu()[50:], X[50:])
        for a, b in zip(got, (y.detach(), *(v.grad for v in leaves))):
            assert torch.isfinite(a).all()
            assert (a.double().cpu() - b).abs().max() <= 1e-4 * b.abs().max()
    finally:
        layer.close()


@pytest.mark.parametrize("tokens", [9, 200])
def test_layer_captured(example, tokens):
    """Forward and backward in one graph, replayed on other tokens with eager work
    between: every replay equals the eager calls bit for bit."""
    announce("gated layer captured", tokens)
    layer = example.GatedExperts(tokens, 8, 2, 128, 96)
    X, dY = torch.empty(tokens, 128, dtype=torch.bfloat16, device="cuda"), None
    dY = torch.empty_like(X)

    def step():
        Y = layer.forward(X)
        return (Y, *layer.backward(X, dY))

    def fill(seed):
        X.copy_(randn(tokens, 128, seed=seed, dtype=torch.bfloat16))
        dY.copy_(randn(tokens, 128, seed=seed + 1, dtype=torch.bfloat16))

    try:
        fill(1)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs = step()
        for rep in range(4):
            fill(10 + 2 * rep)
            graph.replay()
            torch.cuda.synchronize()
            got = [o.clone() for o in outs]
            for a, b in zip(got, step()):
                assert torch.equal(a, b)
    finally:
        layer.close()


def test_two_layers_on_two_streams(example):
    announce("two layers")
    layers = [example.GatedExperts(300, 12, 3, 256, 128, seed=s) for s in (1, 2)]
    xs = [randn(300, 256, seed=s, dtype=torch.bfloat16).cuda() for s in (5, 6)]
    try:
        want = [l.forward(x).clone() for l, x in zip(layers, xs)]
        torch.cuda.synchronize()
        streams, got = [torch.cuda.Stream(), torch.cuda.Stream()], [[], []]
        for _ in range(5):
            for i in (0, 1):
                with torch.cuda.stream(streams[i]):
                    got[i].append(layers[i].forward(xs[i]))
        torch.cuda.synchronize()
        for i in (0, 1):
            assert all(torch.equal(y, want[i]) for y in got[i])
    finally:
        for l in layers:
            l.close()


def test_example_runs(example, capsys):
    announce("gated example")
    losses = example.main(["--tokens", "200", "--experts", "6", "--width", "256", "--hidden", "128",
                           "--steps", "3", "--decode", "12"])
    assert len(losses) == 3 and all(x == x for x in losses)
    assert "finite: True" in capsys.readouterr().out
