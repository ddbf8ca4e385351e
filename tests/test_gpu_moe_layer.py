"""The operators together: the layer of examples/moe_layer.py against automatic differentiation of the same
layer in 64 bits, and its training and serving run."""
from __future__ import annotations

import importlib.util
import pathlib

import pytest
import torch

from gpu_harness import require_cuda

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def example():
    require_cuda()
    path = pathlib.Path(__file__).resolve().parents[1] / "examples" / "moe_layer.py"
    spec = importlib.util.spec_from_file_location("moe_layer_example", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def reference(layer, x, d_out):
    """The layer's output and gradients in 64 bits, with the choice of experts that the layer made."""
    w = {n: t.double().requires_grad_() for n, t in layer.w.items()}
    x = x.double().requires_grad_()
    idx = layer.b.topk_idx.long()
    p = torch.softmax(x @ w["router"].T, -1).gather(1, idx)
    p = p / p.sum(-1, keepdim=True)
    out = torch.zeros_like(x)
    for e in range(layer.cfg.E):
        y = torch.nn.functional.silu(x @ w["w_gate"][e].T) * (x @ w["w_up"][e].T) @ w["w_down"][e].T
        out = out + y * (p * (idx == e)).sum(-1, keepdim=True)
    out.backward(d_out.double())
    return out.detach(), x.grad, {n: t.grad for n, t in w.items()}


@pytest.mark.parametrize("T,H,I,E,k", [(40, 64, 32, 4, 2), (700, 256, 136, 16, 4), (1, 128, 64, 8, 8)])
def test_layer_against_automatic_differentiation(example, T, H, I, E, k):
    """In norm: h, g, u, y, d_y, d_g, d_u, the rows' gradients and the results are rounded to bf16 once each on
    the longest way, and a rounding is off by at most 2^-8 and independent of the others: 10 of them stay within
    sqrt(10) 2^-8. d_out is 8-bit exact; a router's gradient is a difference of nearly equal terms, which can
    magnify the error of y by their size over the difference's, here below 10."""
    layer = example.MoeLayer(T, H, I, E, k, seed=T)
    gen = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn((T, H), generator=gen, device="cuda").to(BF16)
    d_out = torch.randn((T, H), generator=gen, device="cuda").to(BF16)
    out = layer.forward(x).clone()
    d_x = layer.backward(d_out)
    want, want_x, grads = reference(layer, x, d_out)
    tol = 10**0.5 * 2.0**-8
    near = lambda a, b, t: ((a.double() - b).norm() <= t * b.norm()).item()  # noqa: E731
    assert near(out, want, tol)
    for n in ("w_gate", "w_up", "w_down"):
        assert near(layer.grad[n], grads[n], tol), n
    assert near(d_x, want_x, 2 * tol)
    if k > 1:
        assert near(layer.grad["router"], grads["router"], 10 * tol)


def test_training_and_serving(example):
    r = example.main(["--steps", "20", "--tokens", "300"])
    assert r["losses"][-1] < 0.8 * r["losses"][0]
    assert all(n > 0 for n in r["norms"])
    # 4 bits: a value is off by up to 1/14 of its group's largest, in norm about 10% a product, three products
    assert r["off"] < 0.35
