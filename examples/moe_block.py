"""A mixture-of-experts block around its FP8 products, decoded and trained.

    python examples/moe_block.py [--tokens 16] [--layers 4] [--steps 32]

decode(): layers of residual + RMS norm into FP8, router, and the experts of a
few tokens, captured into one HIP graph and replayed.  gradients(): one training
step of a norm with a dense FP8 projection and a router behind it: the
projection's gradients by the FP8 GEMMs, the router's and the norm's by their
own calls.  Random weights and activations; both say how far they are from the
same computation in float64 without quantization.
"""

import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import fp8_block_scaled_04_amd as fb  # noqa: E402


class MoeBlock:
    """out = experts(norm(x + residual)); the sum goes on to the next block."""

    def __init__(self, hidden, inner, experts, topk, gen):
        draw = lambda *n: torch.randn(*n, generator=gen, device="cuda") * n[-1] ** -0.5  # noqa: E731
        self.topk = topk
        self.weight = 1 + 0.1 * torch.randn(hidden, generator=gen, device="cuda")
        self.router = draw(experts, hidden)
        self.dense = draw(experts, 2 * inner, hidden).to(torch.bfloat16), draw(experts, hidden, inner).to(torch.bfloat16)
        self.w13, self.s13 = fb.quantize_128x128(self.dense[0])
        self.w2, self.s2 = fb.quantize_128x128(self.dense[1])

    def forward(self, x, residual):
        """BF16 [T][hidden] both -> (out, sum), BF16; (ids, weights) stay in self.route."""
        q, s, total, _, y = fb.rms_norm_quantize(x, self.weight, residual=residual, return_y=True)
        self.route = fb.moe_route(y.float() @ self.router.t(), self.topk)
        return fb.moe_experts(q, s, *self.route, self.w13, self.s13, self.w2, self.s2), total

    def exact(self, x, residual):
        """The same in float64 from the unquantized weights, with the last forward's route."""
        h = x + residual
        y = h * torch.rsqrt(h.square().mean(1, keepdim=True) + 1e-6) * self.weight.double()
        out = torch.zeros_like(h)
        ids, weights = self.route
        for t in range(x.shape[0]):
            for e, w in zip(ids[t].tolist(), weights[t].tolist()):
                g, u = (self.dense[0][e].double() @ y[t]).chunk(2)
                out[t] += w * (self.dense[1][e].double() @ (g * torch.sigmoid(g) * u))
        return out, h


def decode(tokens=16, layers=4, steps=32, hidden=512, inner=256, experts=8, topk=2, seed=0):
    """-> (seconds per step, relative error of each layer on its own inputs)."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    blocks = [MoeBlock(hidden, inner, experts, topk, gen) for _ in range(layers)]
    x = torch.randn(tokens, hidden, generator=gen, device="cuda").to(torch.bfloat16)
    residual = torch.randn(tokens, hidden, generator=gen, device="cuda").to(torch.bfloat16)

    def step():
        out, total = x, residual
        for b in blocks:
            out, total = b.forward(out, total)
        return out, total

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    graph.replay()
    torch.cuda.synchronize()
    began = time.perf_counter()
    for _ in range(steps):
        graph.replay()
    torch.cuda.synchronize()
    took = (time.perf_counter() - began) / steps
    eager = step()
    same = all(torch.equal(a, b) for a, b in zip(got, eager))
    errors, out, total = [], x, residual
    for b in blocks:
        mine = b.forward(out, total)
        want = b.exact(out.double(), total.double())
        errors.append(max(float((m.double() - w).norm() / w.norm()) for m, w in zip(mine, want)))
        out, total = mine
    return took, errors, same


def gradients(tokens=256, hidden=512, width=256, experts=8, topk=2, seed=0):
    """One step of: y = norm(x + residual); out = y W^T; router weights w of y.
    -> {name: (gradient, the float64 one)} for L = <out, a> + <w, b>."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *n: torch.randn(*n, generator=gen, device="cuda")  # noqa: E731
    x, residual = rand(tokens, hidden).to(torch.bfloat16), rand(tokens, hidden).to(torch.bfloat16)
    norm_weight = 1 + 0.1 * rand(hidden)
    w = (rand(width, hidden) * hidden ** -0.5).to(torch.bfloat16)
    router = rand(experts, hidden) * hidden ** -0.5
    a, b = rand(tokens, width).to(torch.bfloat16), rand(tokens, topk)
    dh = rand(tokens, hidden).to(torch.bfloat16)         # what reaches the sum from later layers

    q, s, total, rstd, y = fb.rms_norm_quantize(x, norm_weight, residual=residual, return_y=True)
    wq, ws = fb.quantize_128x128(w)
    fb.gemm(q, s, wq, ws)
    logits = y.float() @ router.t()
    ids, _ = fb.moe_route(logits, topk)

    aq, as_, aqt, ast = fb.quantize_dual(a)
    dy = fb.gemm(aq, as_, *fb.transpose_128x128(wq, ws), out_dtype=torch.float32)
    dw = fb.gemm_wgrad(aqt, ast, *fb.quantize_transpose_128x1(q, s))
    dlogits = fb.moe_route_backward(logits, ids, b)
    drouter = dlogits.t() @ y.float()
    dy = (dy + dlogits @ router).to(torch.bfloat16)
    dx, dnorm = fb.rms_norm_backward(dy, total, rstd, norm_weight, dh=dh)

    leaf = [t.double().detach().requires_grad_() for t in (total, norm_weight, w, router)]
    h64, n64, w64, r64 = leaf
    y64 = h64 * torch.rsqrt(h64.square().mean(1, keepdim=True) + 1e-6) * n64
    weights = torch.softmax((y64 @ r64.t()).gather(1, ids.long()), 1)
    loss = (y64 @ w64.t() * a.double()).sum() + (weights * b.double()).sum() + (h64 * dh.double()).sum()
    loss.backward()
    return {n: (g, t.grad) for n, g, t in zip(("dx", "dnorm", "dw", "drouter"), (dx, dnorm, dw, drouter), leaf)}


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--tokens", type=int, default=16)
    ap.add_argument("--layers", type=int, default=4)
    ap.add_argument("--steps", type=int, default=32)
    a = ap.parse_args()
    took, errors, same = decode(a.tokens, a.layers, a.steps)
    print(f"decode: {took * 1e6:.0f} us per step of {a.tokens} tokens through {a.layers} blocks (graph replay"
          f"{'' if same else ', DIFFERENT from eager'}); relative error per block {max(errors):.3f}")
    for n, (g, want) in gradients().items():
        print(f"{n}: relative error {float((g.double() - want).norm() / want.norm()):.4f}")


if __name__ == "__main__":
    main()
