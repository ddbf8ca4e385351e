"""The gradient norm over the whole range of fp32: sums of squares that leave it, and squares that vanish."""
from __future__ import annotations

import math

import pytest
import torch

from gpu_harness import require_cuda
from test_gpu_grad_clip import HALF_STEP, NORM_TOL, exact_norm, make

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module")
def ep():
    require_cuda()
    import combine_router_softmax_gb300 as m

    return m


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("scale", [1e-36, 1e-30, 1e-24, 1e-21, 1e-19, 1e-17, 1e15, 1e17, 1e20, 1e30, 1e34])
@pytest.mark.parametrize("sizes", [[5], [4099, 70], [3000001, 1, 0, 40000]])
def test_norm_at_any_scale(ep, sizes, scale, dtype):
    grads = make(sizes, [dtype], seed=len(sizes), scale=scale)
    before = [g.clone() for g in grads]
    n = exact_norm(before)
    norm = torch.full((1,), -1.0, device="cuda")
    ep.GradList(grads).norm(norm)
    assert abs(norm.item() - n) <= NORM_TOL * n
    if n < 1e-6:  # the factor is max_norm / (norm + 1e-6), which a norm as small does not move
        return
    ep.GradList(grads).clip(0.25 * n, norm)
    assert abs(norm.item() - n) <= NORM_TOL * n
    for g, b in zip(grads, before):
        want = b.double() * 0.25
        assert ((g.double() - want).abs() <= want.abs() * (HALF_STEP[dtype] + NORM_TOL + 4 * 2.0**-24) + 1e-38).all()


def test_scales_mixed(ep):
    """Tensors, and values of one tensor, of very different sizes: what is small next to the rest counts for
    nothing, and what is alone in its chunk is not lost."""
    norm = torch.zeros((1,), device="cuda")
    for scales in ([1e-30, 1e-36], [1e25, 1e-25], [1e30, 1.0], [1e-28, 1e28, 1.0], [0.0, 1e-30], [0.0, 1e30]):
        grads = [t for i, s in enumerate(scales) for t in make([50001, 33], [F32], seed=i, scale=s)]
        grads.append(torch.zeros(5000, device="cuda"))
        n = exact_norm(grads)
        ep.GradList(grads).norm(norm)
        assert abs(norm.item() - n) <= NORM_TOL * n, scales
    one = torch.zeros(300007, device="cuda")
    for at, v in ((0, 1e-37), (299999, 3e38), (131072, -1e-25)):
        one.zero_()
        one[at] = v
        ep.GradList([one]).norm(norm)
        assert abs(norm.item() - abs(one[at].item())) <= 2.0**-23 * abs(v), v


def test_a_norm_beyond_fp32(ep):
    g = torch.full((1000,), 3e38, device="cuda")
    norm = torch.zeros((1,), device="cuda")
    ep.GradList([g]).clip(1.0, norm)
    assert math.isinf(norm.item()) and (g == 0).all()
