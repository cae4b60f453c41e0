"""A layer of experts trained one step, then served with adapters: the products
over ragged groups of rows as a program uses them together.

    python examples/experts_and_adapters.py [--tokens 4096 --experts 16 ...]

Training.  A router sends each token to its top experts.  The tokens' rows are
sorted by expert, the offsets are the running sum of the experts' counts (on
the GPU throughout: nothing here waits for it), and the layer is
    H = relu(X W_in[e]),  Y = H W_out[e]           run_grouped, twice
with the gradients
    dH = dY W_out[e]^T, dX = dH' W_in[e]^T          run_grouped, the other transB
    dW_out[e] = H^T dY, dW_in[e] = X^T dH'          run_grouped_wgrad
(dH' is dH where H > 0).

Serving.  Requests of one projection with a low-rank adapter each decode
together: run_lora, one segment of rows per request.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
import dense_gemm_11_amd as g  # noqa: E402


def route(scores, top):
    """Rows sorted by expert: (token of each row, its gate, offsets)."""
    experts = scores.shape[1]
    gate, expert = torch.topk(torch.softmax(scores.float(), 1), top, dim=1)
    order = torch.argsort(expert.reshape(-1), stable=True)
    counts = torch.zeros(experts, dtype=torch.int32, device=scores.device)
    counts.scatter_add_(0, expert.reshape(-1), torch.ones_like(order, dtype=torch.int32))
    offsets = torch.zeros(experts + 1, dtype=torch.int32, device=scores.device)
    torch.cumsum(counts, 0, dtype=torch.int32, out=offsets[1:])
    return order // top, gate.reshape(-1)[order], offsets


class Experts:
    """experts x (width -> hidden -> width), relu between, weights out x in."""

    def __init__(self, experts, width, hidden, device="cuda", dtype=torch.bfloat16, seed=0):
        gen = torch.Generator(device=device).manual_seed(seed)
        self.w_in = torch.randn(experts, hidden, width, generator=gen, device=device).mul_(
            width ** -0.5).to(dtype)
        self.w_out = torch.randn(experts, width, hidden, generator=gen, device=device).mul_(
            hidden ** -0.5).to(dtype)
        self.h = g.gemm_create()

    def close(self):
        g.gemm_destroy(self.h)

    def forward(self, X, scores, top):
        """Y of every token, and what the backward pass needs."""
        token, gate, offsets = route(scores, top)
        rows = X[token]
        H = torch.empty(len(token), self.w_in.shape[1], dtype=X.dtype, device=X.device)
        R = torch.empty_like(rows)
        g.run_grouped(self.h, rows, self.w_in, H, offsets, transB="T")
        torch.relu_(H)
        g.run_grouped(self.h, H, self.w_out, R, offsets, transB="T")
        Y = torch.zeros(X.shape, dtype=torch.float32, device=X.device)
        Y.index_add_(0, token, R.float() * gate[:, None])
        return Y, (token, gate, offsets, rows, H)

    def backward(self, dY, saved):
        """dX and the gradients of w_in and w_out (fp32; the gate's is left out)."""
        token, gate, offsets, rows, H = saved
        dR = (dY[token].float() * gate[:, None]).to(rows.dtype)
        dH, d_rows = torch.empty_like(H), torch.empty_like(rows)
        dw_in = torch.empty(self.w_in.shape, dtype=torch.float32, device=rows.device)
        dw_out = torch.empty(self.w_out.shape, dtype=torch.float32, device=rows.device)
        g.run_grouped(self.h, dR, self.w_out, dH, offsets, transB="N")
        g.run_grouped_wgrad(self.h, dR, H, dw_out, offsets)
        dH *= H > 0
        g.run_grouped(self.h, dH, self.w_in, d_rows, offsets, transB="N")
        g.run_grouped_wgrad(self.h, dH, rows, dw_in, offsets)
        dX = torch.zeros(dY.shape, dtype=torch.float32, device=rows.device)
        dX.index_add_(0, token, d_rows.float())
        return dX, dw_in, dw_out


class AdaptedProjection:
    """A projection (out x in) shared by requests that bring an adapter each."""

    def __init__(self, weight, down, up, scales, max_rows):
        self.weight, self.down, self.up, self.scales = weight, down, up, scales
        self.ws = g.lora_workspace(max_rows, down.shape[1], weight.device)
        self.h = g.gemm_create()

    def close(self):
        g.gemm_destroy(self.h)

    def forward(self, X, offsets, ids):
        """offsets: the requests' rows; ids: their adapters (-1: none)."""
        Y = torch.empty(X.shape[0], self.weight.shape[0], dtype=X.dtype, device=X.device)
        g.run_lora(self.h, X, self.weight, Y, offsets, self.down, self.up, self.ws, ids=ids,
                   scales=self.scales, transB="T")
        return Y


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    for name, default in (("tokens", 4096), ("experts", 16), ("top", 2), ("width", 2048),
                          ("hidden", 1408), ("steps", 5), ("requests", 32), ("adapters", 8),
                          ("rank", 16)):
        ap.add_argument("--" + name, type=int, default=default)
    a = ap.parse_args(argv)
    gen = torch.Generator(device="cuda").manual_seed(1)

    def randn(*shape, std=1.0):
        return torch.randn(*shape, generator=gen, device="cuda").mul_(std).bfloat16()

    layer = Experts(a.experts, a.width, a.hidden)
    X, target, scores = randn(a.tokens, a.width), randn(a.tokens, a.width), randn(a.tokens, a.experts)
    master = [layer.w_in.float(), layer.w_out.float()]
    losses = []
    for _ in range(a.steps):
        Y, saved = layer.forward(X, scores, a.top)
        diff = Y - target.float()
        losses.append((diff * diff).mean())
        _, *grads = layer.backward((2.0 / a.width * diff).bfloat16(), saved)
        for w, m, d in zip((layer.w_in, layer.w_out), master, grads):
            m -= 0.5 * d / a.tokens * a.experts
            w.copy_(m)
    layer.close()
    losses = [float(x) for x in losses]
    print("loss per step:", " ".join("%.4f" % x for x in losses))

    proj = AdaptedProjection(randn(a.width, a.width, std=a.width ** -0.5),
                             randn(a.adapters, a.rank, a.width, std=a.width ** -0.5),
                             randn(a.adapters, a.width, a.rank, std=a.rank ** -0.5),
                             torch.ones(a.adapters, device="cuda"), a.requests)
    offsets = torch.arange(a.requests + 1, dtype=torch.int32, device="cuda")
    ids = torch.randint(-1, a.adapters, (a.requests,), generator=gen, device="cuda").int()
    tokens = randn(a.requests, a.width)
    for _ in range(a.steps):                    # each request's next token
        tokens = torch.tanh(proj.forward(tokens, offsets, ids))
    print("decoded", tuple(tokens.shape), "finite:", bool(torch.isfinite(tokens.float()).all()))
    proj.close()
    return losses


if __name__ == "__main__":
    main()
