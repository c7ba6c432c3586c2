"""A mixture-of-experts feed-forward layer on the library's operators: trained, then served in 4 bits.

    python examples/moe_layer.py [--tokens 2048] [--experts 8] [--choices 2] [--hidden 512] [--ffn 1024] [--steps 30]

Training: a router picks `choices` of `experts` for every token; the tokens' rows go to expert
order, through two products with a ReLU between them, and back, weighted.  The backward pass uses
the same operators: combine's gradient, the products with the transposed weights, the weights'
gradients, and combine without weights as the gradient of gather.  Row counts stay on the device.

Serving: the trained weights in 4-bit codes with a scale and a zero point per group of 64, and a
step of a few tokens through moe_gemm_w4.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import dense_gemm_19_amd as dg   # noqa: E402

BF16, I32, U8 = torch.bfloat16, torch.int32, torch.uint8
GROUP = 64


class Route:
    """The tables of one routing of T tokens: rows in expert order and back."""

    def __init__(self, ids: torch.Tensor, E: int):
        T, k = ids.shape
        self.k, self.n = k, T * k
        new = lambda *s: torch.empty(*s, dtype=I32, device=ids.device)   # noqa: E731
        self.offsets, self.order, self.pos = dg.moe_sort(ids, E, new(E + 1), new(T * k), new(T, k))


def gates(x, router, k):
    """The k largest experts of every token, their ids and their softmax weights."""
    top = (x.float() @ router).topk(k, dim=1)
    return top.indices, top.values.softmax(dim=1)


def forward(x, route, w, W1, W2):
    """y = sum over a token's experts of w * W2 relu(W1 x), and what the backward pass needs."""
    new = lambda rows, like: torch.empty(rows, like, dtype=BF16, device=x.device)   # noqa: E731
    xs = dg.moe_gather(x, route.order, route.k, new(route.n, x.shape[1]))
    h = dg.moe_gemm(xs, route.offsets, W1, new(route.n, W1.shape[2]), dg.DG_ACT_RELU)
    ys = dg.moe_gemm(h, route.offsets, W2, new(route.n, W2.shape[2]))
    y = dg.moe_combine(ys, route.pos, torch.empty_like(x), w)
    return y, (xs, h, ys)


def backward(dy, route, w, W1, W2, saved):
    """Gradients of the layer's input, gate weights and experts' weights (these in FP32)."""
    xs, h, ys = saved
    dys, dw = dg.moe_combine_grad(dy, ys, route.pos, w, torch.empty_like(ys), torch.empty_like(w))
    dW2 = dg.moe_gemm_wgrad(h, dys, route.offsets, torch.empty(W2.shape, device=dy.device))
    dh = dg.moe_gemm(dys, route.offsets, W2.transpose(1, 2), torch.empty_like(h))
    dh = torch.where(h > 0, dh, torch.zeros_like(dh))
    dW1 = dg.moe_gemm_wgrad(xs, dh, route.offsets, torch.empty(W1.shape, device=dy.device))
    dxs = dg.moe_gemm(dh, route.offsets, W1.transpose(1, 2), torch.empty_like(xs))
    dx = dg.moe_combine(dxs, route.pos, torch.empty_like(dy))
    return dx, dw, dW1, dW2


def quantize4(W):
    """4-bit codes [E, N, K/2], scales and zero points [E, N, K/GROUP] of weights [E, K, N]."""
    g = W.transpose(1, 2).float().unflatten(2, (-1, GROUP))
    lo, hi = g.amin(-1).clamp(max=0), g.amax(-1).clamp(min=0)
    S = ((hi - lo) / 15).clamp(min=1e-8).to(BF16)
    Z = (-lo / S.float()).round().clamp(0, 15)
    q = (g / S.float()[..., None] + Z[..., None]).round().clamp(0, 15).to(U8).flatten(2)
    return (q[..., 0::2] | q[..., 1::2] << 4).contiguous(), S, Z.to(U8)


def serve(x, router, k, E, q1, q2):
    """A decoding step on 4-bit weights."""
    ids, w = gates(x, router, k)
    route = Route(ids, E)
    new = lambda cols: torch.empty(route.n, cols, dtype=BF16, device=x.device)   # noqa: E731
    xs = dg.moe_gather(x, route.order, k, new(x.shape[1]))
    h = dg.moe_gemm_w4(xs, route.offsets, q1[0], q1[1], new(q1[0].shape[1]), GROUP, q1[2], dg.DG_ACT_RELU)
    ys = dg.moe_gemm_w4(h, route.offsets, q2[0], q2[1], new(q2[0].shape[1]), GROUP, q2[2])
    return dg.moe_combine(ys, route.pos, torch.empty_like(x), w)


def main(argv=None):
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    for name, value in (("tokens", 2048), ("experts", 8), ("choices", 2), ("hidden", 512), ("ffn", 1024), ("steps", 30)):
        p.add_argument("--" + name, type=int, default=value)
    a = p.parse_args(argv)
    torch.manual_seed(0)
    E, k, H, F = a.experts, a.choices, a.hidden, a.ffn
    normal = lambda *s: torch.randn(*s, device="cuda")   # noqa: E731
    router = normal(H, E) * H ** -0.5
    master = [normal(E, H, F) * H ** -0.5, normal(E, F, H) * F ** -0.5]
    x = normal(a.tokens, H).to(BF16)
    target = torch.tanh(x.float() @ (normal(H, H) * H ** -0.5))
    losses = []
    for step in range(a.steps):
        W1, W2 = (m.to(BF16) for m in master)
        ids, w = gates(x, router, k)
        route = Route(ids, E)
        y, saved = forward(x, route, w, W1, W2)
        diff = y.float() - target
        losses.append(float((diff * diff).mean()))
        _, _, dW1, dW2 = backward((diff * (2.0 / a.tokens)).to(BF16), route, w, W1, W2, saved)
        for m, d in zip(master, (dW1, dW2)):
            m.sub_(d, alpha=0.05)
        if step % 10 == 0 or step == a.steps - 1:
            print(f"step {step:3d}  loss {losses[-1]:.4f}", flush=True)
    W1, W2 = (m.to(BF16) for m in master)
    few = x[:8]
    ids, w = gates(few, router, k)
    full, _ = forward(few, Route(ids, E), w, W1, W2)
    four = serve(few, router, k, E, quantize4(W1), quantize4(W2))
    err = float((four.float() - full.float()).norm() / full.float().norm())
    print(f"4-bit weights: relative difference {err:.3f}", flush=True)
    return losses, err


if __name__ == "__main__":
    main()
