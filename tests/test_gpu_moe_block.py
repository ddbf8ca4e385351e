"""The operators around the layer together: the block of examples/moe_layer.py against automatic differentiation of the
same block in 64 bits, and its training."""
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
    spec = importlib.util.spec_from_file_location("moe_layer_example_block", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def reference(block, x, d_n, d_out):
    """Output, stream and gradients in 64 bits, with the choice of experts that the block made."""
    layer = block.layer
    w = {n: t.double().requires_grad_() for n, t in {**layer.w, **block.w}.items()}
    x = x.double().requires_grad_()
    norm = lambda v, g: g * v * (v.square().mean(-1, keepdim=True) + 1e-6).rsqrt()  # noqa: E731
    n_in = norm(x, w["w_in"])
    idx = layer.b.topk_idx.long()
    logits = n_in @ w["router"].T
    p_all = torch.softmax(logits, -1)
    p = p_all.gather(1, idx)
    p = p / p.sum(-1, keepdim=True)
    y = torch.zeros_like(x)
    for e in range(layer.cfg.E):
        h = torch.nn.functional.silu(n_in @ w["w_gate"][e].T) * (n_in @ w["w_up"][e].T)
        y = y + h @ w["w_down"][e].T * (p * (idx == e)).sum(-1, keepdim=True)
    out = x + w["gate"] * norm(y, w["w_post"])
    n = norm(out, w["w_next"])
    load = torch.bincount(idx.flatten(), minlength=layer.cfg.E).double() / idx.numel()
    losses = torch.stack([layer.cfg.E * (load * p_all.mean(0)).sum(), torch.logsumexp(logits, -1).square().mean()])
    total = (n * d_n.double()).sum() + (block.d_loss[0].double() * losses).sum()
    if d_out is not None:
        total = total + (out * d_out.double()).sum()
    total.backward()
    return n.detach(), out.detach(), losses.detach(), x.grad, {k: t.grad for k, t in w.items()}


@pytest.mark.parametrize("T,H,I,E,k,stream", [(48, 64, 32, 4, 2, True), (600, 256, 136, 16, 4, False), (3, 128, 64, 8, 8, True)])
def test_block_against_automatic_differentiation(example, T, H, I, E, k, stream):
    """In norm, as for the layer alone (test_gpu_moe_layer.py): on the longest way n_in, h, g, u, y, d_y, d_g, d_u, the
    rows' gradients, the layer's d_x and d_n_in are rounded to bf16 once each, 12 independent roundings with the results
    stay within sqrt(12) 2^-8. The post norm's gradient takes a row's component along y out of d_y, and the
    router's is a difference of nearly equal terms: both can magnify what goes in, the latter by less than 10."""
    block = example.MoeBlock(T, H, I, E, k, seed=T)
    gen = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn((T, H), generator=gen, device="cuda")
    d_n = torch.randn((T, H), generator=gen, device="cuda").to(BF16)
    d_out = torch.randn((T, H), generator=gen, device="cuda") if stream else None
    n = block.forward(x).clone()
    d_x = block.backward(d_n, d_out)
    want_n, want_out, losses, want_x, grads = reference(block, x, d_n, d_out)
    tol = 12**0.5 * 2.0**-8
    near = lambda a, b, t: ((a.double() - b).norm() <= t * b.norm()).item()  # noqa: E731
    assert near(n, want_n, tol) and near(block.out, want_out, tol)
    # of logits that are products of bf16 values with fp32 sums: the norm's rounding, 2^-8, through a softmax
    assert near(block.loss[0], losses, 2.0**-6)
    for name in ("w_post", "w_next", "gate", "w_in"):
        assert near(block.grad[name], grads[name], 2 * tol), name
    for name in ("w_gate", "w_up", "w_down"):
        assert near(block.layer.grad[name], grads[name], 2 * tol), name
    assert near(d_x, want_x, 2 * tol)
    if k < E or k > 1:
        assert near(block.layer.grad["router"], grads["router"], 10 * tol)


def test_step_moves_the_experts_by_orthogonal_updates(example):
    """Every expert's update has singular values of about lr 0.2 sqrt(max(1, N / K)), whatever its gradient's size."""
    block = example.MoeBlock(400, 128, 64, 4, 2, seed=1)
    gen = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randn((400, 128), generator=gen, device="cuda")
    before = {n: m.clone() for n, m in block.layer.master.items()}
    block.forward(x)
    block.backward(torch.randn((400, 128), generator=gen, device="cuda").to(BF16) * 1e-3)
    block.step(0.1, max_norm=1.0)
    for n in block.experts:
        N, K = before[n].shape[1:]
        size = 0.1 * 0.2 * max(1.0, N / K) ** 0.5
        s = torch.linalg.svdvals((before[n] - block.layer.master[n]).double()) / size
        # the steps leave singular values between 0.66 and 1.21, small ones of the gradient may not have come that far
        assert s.max() < 1.25 and s.median() > 0.6, n
    assert not torch.equal(before["router"], block.layer.master["router"])


def test_block_trains(example):
    r = example.main(["--block", "--steps", "8", "--tokens", "300"])
    assert all(v > 0 and v < float("inf") for v in r["losses"] + r["balance"] + r["norms"])
