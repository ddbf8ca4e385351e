"""ep_combine_backward and ep_route_backward against their formulas in 64 bits, and against differences."""
from __future__ import annotations

import pytest
import torch

import experts_ref as ref
from gpu_harness import require_cuda

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
U24 = 2.0**-24


@pytest.fixture(scope="module")
def ep():
    require_cuda()
    import combine_router_softmax_gb300 as m

    return m


def layer(ep, T, H, E, k, renorm, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    cfg = ep.EpConfig.make(T=T, H=H, E=E, R=1, k=k, renormalize=renorm, num_workers=8)
    b = ep.LayerBuffers.allocate(cfg)
    b.logits.copy_(torch.randn((T, E), generator=gen, device="cuda"))
    b.x.copy_(torch.randn((T, H), generator=gen, device="cuda"))
    b.y.copy_(torch.randn((T * k, H), generator=gen, device="cuda"))
    b.route()
    b.layout()
    d_out = (torch.randn((T, H), generator=gen, device="cuda") * 0.3).to(BF16)
    return cfg, b, d_out


SHAPES = [(1, 8, 1, 1), (1, 7168, 256, 8), (3, 72, 5, 2), (64, 4096, 128, 8), (17, 264, 40, 7), (130, 1000, 33, 9),
          (5, 64, 64, 32), (2, 16384, 16, 16), (700, 520, 300, 4), (9, 2048, 1024, 3)]


@pytest.mark.parametrize("T,H,E,k", SHAPES)
def test_combine_backward(ep, T, H, E, k):
    cfg, b, d_out = layer(ep, T, H, E, k, 1, seed=T + H)
    d_y = torch.full((T * k, H), 7.0, dtype=BF16, device="cuda")
    d_w = torch.full((T, k), 7.0, device="cuda")
    ep.ep_combine_backward(cfg, d_out, b.y, b.slot, b.topk_w, d_y, d_w)
    w, slot = b.topk_w.double(), b.slot.long()
    want = w[..., None] * d_out.double()[:, None]
    got = d_y[slot.view(-1)].view(T, k, H)
    # the product in fp32 and its rounding to bf16
    ref.check(got, want, (ref.U16 + 2 * U24) * want.abs(), "d_y")
    pairs = b.y[slot].double() * d_out.double()[:, None]
    ref.check(d_w, pairs.sum(-1), H * ref.U32 * pairs.abs().sum(-1) + 1e-30, "d_topk_w")


def test_combine_backward_skips_slots_outside(ep):
    cfg, b, d_out = layer(ep, 6, 136, 8, 3, 1)
    slot = b.slot.clone()
    slot[2, 1], slot[4, 0] = -1, 18
    missing = [b.slot[2, 1].item(), b.slot[4, 0].item()]
    d_y = torch.full((18, 136), 7.0, dtype=BF16, device="cuda")
    d_w = torch.full((6, 3), 7.0, device="cuda")
    ep.ep_combine_backward(cfg, d_out, b.y, slot, b.topk_w, d_y, d_w)
    assert d_w[2, 1] == 0 and d_w[4, 0] == 0
    assert (d_y[missing] == 7.0).all()
    others = [i for i in range(18) if i not in missing]
    assert (d_y[others] != 7.0).any(1).all()


def test_combine_backward_with_a_nan_row(ep):
    """A row of y that holds NaN makes the product it is part of NaN, and nothing else."""
    cfg, b, d_out = layer(ep, 5, 64, 8, 2, 1)
    b.y[b.slot[3, 1].long()] = float("nan")
    d_y, d_w = torch.zeros((10, 64), dtype=BF16, device="cuda"), torch.zeros((5, 2), device="cuda")
    ep.ep_combine_backward(cfg, d_out, b.y, b.slot, b.topk_w, d_y, d_w)
    nan = torch.isnan(d_w)
    assert nan[3, 1] and nan.sum() == 1 and torch.isfinite(d_y).all()


def route_reference(logits, idx, w, dw, renorm):
    """Values and bounds. inner is a sum of k <= 32 products taken as a tree: off by 8 half steps of their
    magnitudes; the softmax by 2^-19 for logits within +-20."""
    p = torch.zeros_like(logits).scatter_(1, idx, w) if renorm else torch.softmax(logits, -1)
    d = torch.zeros_like(logits).scatter_(1, idx, dw)
    inner = (w * dw).sum(-1, keepdim=True)
    off = 8 * U24 * (w * dw).abs().sum(-1, keepdim=True)
    want = p * (d - inner)
    size = d.abs() + inner.abs()
    return want, ref.SLACK * (p * (off + 2 * U24 * size) + (0 if renorm else 2.0**-19) * p * size + 2 * U24 * want.abs())


@pytest.mark.parametrize("renorm", [0, 1])
@pytest.mark.parametrize("T,H,E,k", SHAPES)
def test_route_backward(ep, T, H, E, k, renorm):
    cfg, b, _ = layer(ep, T, 8, E, k, renorm, seed=E)
    dw = torch.randn((T, k), device="cuda", generator=torch.Generator(device="cuda").manual_seed(k))
    d_l = torch.full((T, E), 7.0, device="cuda")
    ep.ep_route_backward(cfg, None if renorm else b.logits, b.topk_idx, b.topk_w, dw, d_l)
    want, tol = route_reference(b.logits.double(), b.topk_idx.long(), b.topk_w.double(), dw.double(), renorm)
    off = (d_l.double() - want).abs()
    assert (off <= tol + 1e-37).all(), (off - tol).max().item()
    if renorm:
        chosen = torch.zeros((T, E), dtype=torch.bool, device="cuda").scatter_(1, b.topk_idx.long(), True)
        assert (d_l[~chosen] == 0).all()


@pytest.mark.parametrize("renorm", [0, 1])
def test_route_backward_ignores_ids_outside(ep, renorm):
    cfg, b, _ = layer(ep, 3, 8, 8, 2, renorm)
    dw = torch.ones((3, 2), device="cuda")
    idx = b.topk_idx.clone()
    idx[1, 0], idx[2, 1] = -1, 8
    d_l = torch.full((3, 8), 7.0, device="cuda")
    ep.ep_route_backward(cfg, b.logits, idx, b.topk_w, dw, d_l)
    assert torch.isfinite(d_l).all() and (d_l != 7.0).all()


@pytest.mark.parametrize("renorm,k", [(0, 3), (1, 3), (0, 1), (1, 1)])
def test_layer_gradients_against_differences(ep, renorm, k):
    """out = sum_j w_j(logits) y[slot_j] and L = <out, d_out>: its differences in 64 bits along a direction of
    the logits (the choice held fixed) and of y are what the two calls give."""
    T, H, E = 12, 72, 10
    cfg, b, d_out = layer(ep, T, H, E, k, renorm, seed=4)
    d_y, d_w, d_l = torch.empty_like(b.y), torch.empty((T, k), device="cuda"), torch.empty((T, E), device="cuda")
    ep.ep_combine_backward(cfg, d_out, b.y, b.slot, b.topk_w, d_y, d_w)
    ep.ep_route_backward(cfg, b.logits, b.topk_idx, b.topk_w, d_w, d_l)
    idx, slot = b.topk_idx.long(), b.slot.long()

    def loss(logits, y):
        w = torch.softmax(logits, -1).gather(1, idx)
        if renorm:
            w = w / w.sum(-1, keepdim=True)
        return ((w[..., None] * y[slot]).sum(1) * d_out.double()).sum().item()

    logits, y = b.logits.double(), b.y.double()
    gen = torch.Generator(device="cuda").manual_seed(9)
    v = torch.randn((T, E), generator=gen, device="cuda", dtype=torch.float64)
    u = torch.randn(y.shape, generator=gen, device="cuda", dtype=torch.float64)
    scale = (d_w.double().abs().sum() + 1e-3).item()
    for got, at, bound in (
            ((d_l.double() * v).sum().item(), lambda e: loss(logits + e * v, y), 1e-5 * scale * v.abs().max().item()),
            ((d_y.double() * u).sum().item(), lambda e: loss(logits, y + e * u), ref.U16 * 1.01 * (d_y.double() * u).abs().sum().item())):
        d1, d2 = ((at(e) - at(-e)) / (2 * e) for e in (1e-4, 5e-5))
        assert abs(got - (4 * d2 - d1) / 3) <= bound + 2 * abs(d1 - d2) + 1e-9 * scale


def test_dispatch_backward_is_combine_with_ones(ep):
    cfg, b, _ = layer(ep, 30, 136, 16, 4, 1)
    g = torch.randn((120, 136), device="cuda", generator=torch.Generator(device="cuda").manual_seed(3)).to(BF16)
    dx = torch.empty((30, 136), dtype=BF16, device="cuda")
    ep.ep_combine(cfg, g, b.slot, torch.ones((30, 4), device="cuda"), dx)
    terms = g[b.slot.long()].double()
    ref.check(dx, terms.sum(1), ref.U16 * terms.sum(1).abs() + 4 * ref.U32 * terms.abs().sum(1), "d_x")


def test_graph(ep):
    cfg, b, d_out = layer(ep, 40, 264, 24, 6, 0)
    d_y, d_w, d_l = torch.empty_like(b.y), torch.empty((40, 6), device="cuda"), torch.empty((40, 24), device="cuda")

    def both():
        ep.ep_combine_backward(cfg, d_out, b.y, b.slot, b.topk_w, d_y, d_w)
        ep.ep_route_backward(cfg, b.logits, b.topk_idx, b.topk_w, d_w, d_l)

    both()
    want = [t.clone() for t in (d_y, d_w, d_l)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        both()
    for t in (d_y, d_w, d_l):
        t.zero_()
    g.replay()
    assert all(torch.equal(a, c) for a, c in zip(want, (d_y, d_w, d_l)))
