"""ep_orthogonalize of matrices that have fewer singular vectors than rows, against the steps in 64 bits.

The bound is the figure that include/ep_layer.h gives, with the last rounding to bf16, taken from the exact result
itself: the two are independent, so their squares add. N rounding errors, each anywhere within half a step, have a sum of squares
within 9 / sqrt(N) of its mean in ten standard deviations, the root within half of that.
Figure: 0.0012 after five steps and 0.002 after up to ten for 64 rows and more, 0.002 and 0.005 for 16; and
2^-21 a^steps / sqrt(rank) for what fp32 leaves in directions that the matrix has nothing in (sums of up to 2048 terms by
turns, eight times 2^-24, grown by a = 3.4445 a step; X has the norm sqrt(rank) in the end)."""
from __future__ import annotations

import ctypes

import pytest
import torch

from gpu_harness import require_cuda

BF16, F32 = torch.bfloat16, torch.float32
A, B, C = 3.4445, -4.7750, 2.0315


def load():
    import __graft_entry__

    __graft_entry__._cuda_build_module().build()
    import combine_router_softmax_gb300 as m

    return m


@pytest.fixture(scope="module")
def ep():
    require_cuda()
    return load()


def exact(m, steps, eps=1e-7):
    tall = m.shape[1] > m.shape[2]
    x = m.double().transpose(1, 2) if tall else m.double()
    x = x / (x.square().sum((1, 2), keepdim=True).sqrt() + eps)
    for a, b, c in steps:
        g = x @ x.transpose(1, 2)
        x = a * x + (b * g + c * g @ g) @ x
    return x.transpose(1, 2) if tall else x


def run(ep, m, steps):
    cfg = ep.EpOrthoConfig.make(B=m.shape[0], N=m.shape[1], K=m.shape[2], dtype=m.dtype, steps=len(steps))
    out = torch.full(m.shape, float("nan"), dtype=BF16, device="cuda")
    ws = torch.full((ep.ep_orthogonalize_workspace_size(cfg),), 255, dtype=torch.uint8, device="cuda")
    ep.ep_orthogonalize(cfg, m, out, ws, coefficients=steps)
    assert ep.ep_device_error() == 0
    return out


def of_rank(count, N, K, rank, seed, dtype=F32):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=gen, device="cuda", dtype=torch.float64)  # noqa: E731
    return (n(count, N, rank) @ n(count, rank, K) * 0.01).to(dtype)


def off(got, want):
    return (got.double() - want).flatten(1).norm(dim=1) / want.flatten(1).norm(dim=1)


def figure(few, rank, steps):
    grown = 2.0**-21 / rank**0.5
    for a, _, _ in steps:
        grown *= abs(a)
    return (0.0012 if few >= 64 else 0.002) * (1 if len(steps) <= 5 else 5 / 3 if few >= 64 else 2.5) + grown


def check(ep, m, rank, steps):
    e = exact(m, steps)
    got, own = off(run(ep, m, steps), e), off(e.to(BF16), e)
    bound = (own**2 + figure(min(m.shape[1:]), rank, steps) ** 2).sqrt() * (1 + 4.5 / (m.shape[1] * m.shape[2]) ** 0.5)
    assert (got <= bound).all(), f"{got.max().item():g} off, the bound is {bound.min().item():g}"


# by one cluster, several CTAs of it, and by products of single CTAs and of pairs; wide and tall
@pytest.mark.gpu
@pytest.mark.parametrize("count,N,K", [(8, 16, 24), (4, 16, 400), (4, 64, 64), (3, 250, 64), (2, 128, 1000), (1, 128, 4096), (2, 256, 384),
                                       (7, 1000, 360), (1, 256, 7168), (1, 1024, 1024), (6, 1100, 1200)])
@pytest.mark.parametrize("steps", [5, 8, 10])
@pytest.mark.parametrize("share", [0, 1 / 16, 1 / 2])
def test_of_low_rank(ep, count, N, K, steps, share):
    rank = max(1, int(min(N, K) * share))
    check(ep, of_rank(count, N, K, rank, seed=N + steps), rank, [(A, B, C)] * steps)


@pytest.mark.gpu
@pytest.mark.parametrize("count,N,K", [(4, 64, 96), (3, 300, 400), (2, 1000, 130)])
@pytest.mark.parametrize("steps", [5, 8])
def test_of_full_rank_keeps_its_figure(ep, count, N, K, steps):
    few = min(N, K)
    check(ep, of_rank(count, N, K, 2 * few, seed=3), few, [(A, B, C)] * steps)


@pytest.mark.gpu
@pytest.mark.parametrize("N,K", [(48, 200), (200, 330)])
@pytest.mark.parametrize("steps", [[(1.5, -0.5, 0.0)] * 12, [(A, B, C)] * 4 + [(1.875, -1.25, 0.375)] * 3, [(1.9, -0.9, 0.0)] + [(A, B, C)] * 6])
def test_of_low_rank_by_other_coefficients(ep, N, K, steps):
    for rank in (1, 5, N // 2):
        check(ep, of_rank(3, N, K, rank, seed=4), rank, steps)


@pytest.mark.gpu
def test_an_update_of_few_tokens(ep):
    """What an expert's weights get from eight tokens, kept in bf16, whose own rounding has all directions."""
    for N, K in ((96, 320), (512, 640)):
        m = of_rank(2, N, K, 8, seed=5, dtype=BF16)
        for steps in (5, 8):
            check(ep, m, 8, [(A, B, C)] * steps)


def forms(steps, rows):
    """What each step takes of X's lower half: 0 the diagonal of B, 1 nothing, 2 all of B."""
    flat = [v for s in steps for v in s]
    out = (ctypes.c_uint8 * len(steps))()
    f = getattr(load()._lib, "_ZN2ep11ortho_stepsEPKfiiPNS_9OrthoFormE")  # ep::ortho_steps
    f.restype = ctypes.c_bool
    assert f((ctypes.c_float * len(flat))(*flat), len(steps), rows, out)
    return list(out)


def test_what_a_step_takes():
    """Behind the last two default steps nothing grows tenfold; before them B is small beside a as long as 1 / sqrt(rows), grown, is."""
    for rows, want in ((1, [2, 2, 2, 0, 0]), (16, [1, 2, 2, 0, 0]), (256, [1, 1, 2, 0, 0]), (2048, [1, 1, 1, 0, 0])):
        assert forms([(A, B, C)] * 5, rows) == want
    assert forms([(A, B, C)] * 8, 256) == [1, 1, 2, 2, 2, 2, 0, 0]
    assert forms([(2.0, 0.0, 0.0)], 8) == [0]
    assert forms([(1.5, -0.5, 0.0)] * 3, 64) == [0, 0, 0]
