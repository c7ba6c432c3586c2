"""GPU test of examples/moe_layer.py: the layer's gradients against 64-bit autograd, a training run, 4-bit serving."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def ex():
    spec = importlib.util.spec_from_file_location("moe_layer", os.path.join(HERE, "..", "examples", "moe_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_gradients_against_autograd(ex):
    # Inputs small enough for BF16's 2^-8 roundings to be the whole error: each gradient passes at most
    # four of them (ys or h, dys, dh, the result), so 8 * 2^-8 of the gradient's norm is twice their sum.
    g = torch.Generator().manual_seed(3)
    T, E, k, H, F = 96, 4, 2, 64, 128
    rnd = lambda *s, scale=1.0: (torch.randn(*s, generator=g) * scale).to(torch.bfloat16)   # noqa: E731
    x, W1, W2, dy = rnd(T, H), rnd(E, H, F, scale=H ** -0.5), rnd(E, F, H, scale=F ** -0.5), rnd(T, H)
    ids = torch.rand(T, E, generator=g).argsort(1)[:, :k]
    w = torch.rand(T, k, generator=g)
    dev = [t.cuda() for t in (x, W1, W2, dy, w)]
    route = ex.Route(ids.cuda(), E)
    y, saved = ex.forward(dev[0], route, dev[4], dev[1], dev[2])
    got = (y,) + ex.backward(dev[3], route, dev[4], dev[1], dev[2], saved)
    leaves = [t.double().requires_grad_() for t in (x, w, W1, W2)]
    out = torch.zeros(T, H, dtype=torch.float64)
    for e in range(E):
        h = torch.relu(leaves[0] @ leaves[2][e]) @ leaves[3][e]
        out = out + (h[:, None] * (leaves[1] * (ids == e))[..., None]).sum(1)
    want = (out.detach(),) + torch.autograd.grad(out, leaves, dy.double())
    for name, a, b in zip(("y", "dx", "dw", "dW1", "dW2"), got, want):
        rel = float((a.cpu().double() - b).norm() / b.norm())
        print(name, rel, flush=True)
        assert rel <= 8 * 2.0 ** -8, (name, rel)


def test_training_and_serving(ex):
    losses, err = ex.main(["--tokens", "512", "--hidden", "128", "--ffn", "256", "--steps", "12"])
    assert losses[-1] < 0.9 * losses[0]
    # codes are off by at most half a step of (max - min) / 15, about 5 sigma / 15: a uniform error of 0.1 sigma
    # per product, two products; three times their root sum
    assert err < 0.45
