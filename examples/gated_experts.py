"""A layer of gated experts with its router, trained and then served: the
products, the routing and the moving of rows as a program uses them together.

    python examples/gated_experts.py [--tokens 4096 --experts 16 ...]

Forward, for tokens X with the residual stream X itself:
    logits = X W_r^T                                  run_tensors
    ids, w, plan = route(logits)                      run_route
    rows = X[the rows' tokens]                        run_gather_rows
    H = silu(rows W_in[e][:, :F]) * (... [:, F:])     run_grouped_act (keeps Z)
    R = H W_out[e]                                    run_grouped
    Y = X + sum_j w_j R[row of choice j]              run_combine_rows
Backward, all of it:
    dR, dw from dY                                    run_combine_rows_grad
    dH = dR W_out^T; dW_out                           run_grouped, run_grouped_wgrad
    dZ, H again                                       run_grouped_act_grad
    drows = dZ W_in^T; dW_in                          run_grouped, run_grouped_wgrad
    dlogits                                           run_route_grad
    dX = dY + sum_j drows[row of choice j] + dlogits W_r; dW_r
                                                      run_combine_rows, run_tensors
Nothing waits for the GPU, so both directions can be captured.  Tokens of a padded
batch are masked by logits of -inf: they take no expert and Y is X there.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
import dense_gemm_11_amd as g  # noqa: E402


class GatedExperts:
    """Router (experts x width) and experts (width -> 2 x hidden -> width), weights
    out x in, with the buffers of up to one batch of `tokens` tokens."""

    def __init__(self, tokens, experts, top, width, hidden, device="cuda", dtype=torch.bfloat16, seed=0,
                 **routing):
        gen = torch.Generator(device=device).manual_seed(seed)

        def randn(*shape, std):
            return torch.randn(*shape, generator=gen, device=device).mul_(std).to(dtype)

        def empty(*shape, dtype=dtype):
            return torch.empty(*shape, dtype=dtype, device=device)

        self.w_router = randn(experts, width, std=width ** -0.5)
        self.w_in = randn(experts, 2 * hidden, width, std=width ** -0.5)
        self.w_out = randn(experts, width, hidden, std=hidden ** -0.5)
        self.top, self.routing = top, dict(scores="softmax", renormalize=True, scale=1.0) | routing
        rows, f32, i32 = tokens * top, torch.float32, torch.int32
        self.logits = empty(tokens, experts, dtype=f32)
        self.ids, self.weights = empty(tokens, top, dtype=i32), empty(tokens, top, dtype=f32)
        self.offsets, self.order = empty(experts + 1, dtype=i32), empty(rows, dtype=i32)
        self.position = empty(tokens, top, dtype=i32)
        self.ws = g.route_workspace(tokens, experts, device)
        # zeroed, since rows behind the last expert's are never written
        self.rows, self.Z, self.H, self.R = (torch.zeros(rows, n, dtype=dtype, device=device)
                                             for n in (width, 2 * hidden, hidden, width))
        self.h = g.gemm_create()

    def close(self):
        g.gemm_destroy(self.h)

    def forward(self, X, mask=None):
        """Y of every token; mask: tokens x 1, -inf for padding and 0 else."""
        Y = torch.empty_like(X)
        g.run_tensors(self.h, X, self.w_router, self.logits, transB="T")
        if mask is not None:
            self.logits += mask
        g.run_route(self.h, self.logits, self.ids, self.weights, self.offsets, self.order, self.position,
                    self.ws, **self.routing)
        g.run_gather_rows(self.h, X, self.rows, self.order, self.top)
        g.run_grouped_act(self.h, self.rows, self.w_in, self.H, self.offsets, activation="silu", gated=True,
                          Z=self.Z, transB="T")
        g.run_grouped(self.h, self.H, self.w_out, self.R, self.offsets, transB="T")
        g.run_combine_rows(self.h, self.R, Y, self.position, weights=self.weights, C=X, beta=1.0)
        return Y

    def backward(self, X, dY):
        """After forward(X): dX and the gradients of w_router, w_in and w_out (fp32)."""
        dR, dH, drows = torch.zeros_like(self.R), torch.zeros_like(self.H), torch.zeros_like(self.rows)
        dw, dlogits = torch.empty_like(self.weights), torch.empty_like(self.logits)
        dw_router, dw_in, dw_out = (torch.empty(w.shape, dtype=torch.float32, device=X.device)
                                    for w in (self.w_router, self.w_in, self.w_out))
        keys = ("scores", "renormalize", "scale")
        g.run_combine_rows_grad(self.h, self.R, dY, dR, dw, self.position, self.weights)
        g.run_grouped(self.h, dR, self.w_out, dH, self.offsets, transB="N")
        g.run_grouped_wgrad(self.h, dR, self.H, dw_out, self.offsets)
        dZ = self.Z                                   # its place is free from here
        g.run_grouped_act_grad(self.h, self.Z, dH, dZ, self.offsets, activation="silu", gated=True)
        g.run_grouped(self.h, dZ, self.w_in, drows, self.offsets, transB="N")
        g.run_grouped_wgrad(self.h, dZ, self.rows, dw_in, self.offsets)
        g.run_route_grad(self.h, self.logits, self.ids, dw, dlogits,
                         **{k: self.routing[k] for k in keys})
        dl = dlogits.to(X.dtype)
        dX = torch.empty_like(X)
        g.run_combine_rows(self.h, drows, dX, self.position, C=dY, beta=1.0)
        g.run_tensors(self.h, dl, self.w_router, dX, C=dX, beta=1.0)
        g.run_tensors(self.h, dl, X, dw_router, transA="T")
        return dX, dw_router, dw_in, dw_out


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    for name, default in (("tokens", 4096), ("experts", 16), ("top", 2), ("width", 2048),
                          ("hidden", 1408), ("steps", 5), ("decode", 32)):
        ap.add_argument("--" + name, type=int, default=default)
    a = ap.parse_args(argv)
    gen = torch.Generator(device="cuda").manual_seed(1)

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device="cuda").bfloat16()

    layer = GatedExperts(a.tokens, a.experts, a.top, a.width, a.hidden)
    X, target = randn(a.tokens, a.width), randn(a.tokens, a.width)
    weights = (layer.w_router, layer.w_in, layer.w_out)
    master = [w.float() for w in weights]
    losses = []
    for _ in range(a.steps):
        diff = layer.forward(X).float() - target.float()
        losses.append((diff * diff).mean())
        grads = layer.backward(X, (2.0 / a.width * diff).bfloat16())[1:]
        for w, m, d in zip(weights, master, grads):
            m -= 0.5 * d / a.tokens * a.experts
            w.copy_(m)
    losses = [float(x) for x in losses]
    print("loss per step:", " ".join("%.4f" % x for x in losses))

    # a decode batch of `decode` tokens, the last quarter of them padding, in a graph
    serve = GatedExperts(a.decode, a.experts, a.top, a.width, a.hidden)
    for name in ("w_router", "w_in", "w_out"):
        setattr(serve, name, getattr(layer, name))
    tokens, mask = randn(a.decode, a.width), torch.zeros(a.decode, 1, device="cuda")
    mask[a.decode - a.decode // 4:] = -float("inf")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        serve.forward(tokens, mask)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = serve.forward(tokens, mask)
    for _ in range(a.steps):                    # each request's next token
        graph.replay()
        tokens.copy_(torch.tanh(out.float()))
    print("decoded", tuple(out.shape), "finite:", bool(torch.isfinite(out.float()).all()))
    layer.close()
    serve.close()
    return losses


if __name__ == "__main__":
    main()
