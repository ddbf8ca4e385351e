"""ep_grad_norm and ep_grad_clip against 64 bits."""
from __future__ import annotations

import math

import pytest
import torch

from gpu_harness import require_cuda

pytestmark = pytest.mark.gpu
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
HALF_STEP = {F32: 2.0**-24, BF16: 2.0**-8, F16: 2.0**-11}
# squares in fp32, chains of at most 2^20 / 512 / 4 of them in fp32 (each step half an ulp), then 64 bits; the
# root halves the relative error, and its own rounding to fp32 adds one
NORM_TOL = 0.5 * 600 * 2.0**-24 + 2.0**-23


@pytest.fixture(scope="module")
def ep():
    require_cuda()
    import combine_router_softmax_gb300 as m

    return m


def make(sizes, types, seed=0, scale=0.02):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return [(torch.randn((n,), generator=gen, device="cuda") * scale).to(types[i % len(types)]) for i, n in enumerate(sizes)]


def exact_norm(ts):
    return math.sqrt(sum((t.double() ** 2).sum().item() for t in ts))


def check_clip(out, before, max_norm, norm):
    n = exact_norm(before)
    assert abs(norm.item() - n) <= NORM_TOL * n
    coef = min(1.0, max_norm / (n + 1e-6))
    for o, b in zip(out, before):
        want = b.double() * coef
        # the factor carries the norm's error and its own roundings; below fp16's normal range a step is 2^-24
        tol = want.abs() * (HALF_STEP[b.dtype] + NORM_TOL + 4 * 2.0**-24) + (2.0**-25 if b.dtype == F16 else 1e-38)
        assert ((o.double() - want).abs() <= tol).all()


LISTS = [
    ([1], [F32]), ([7], [BF16]), ([8], [F16]), ([4096], [BF16]), ([4097, 1, 0, 31], [F32, BF16]),
    ([0, 0], [F32]), ([3, 4095, 65537, 12], [F16, F32, BF16]), ([1 << 20, 5], [BF16]), ([17] * 900, [F32, BF16, F16]),
    ([1] * 2000, [BF16]), ([300007, 1000003], [F32]),
]


@pytest.mark.parametrize("factor", [0.3, 2.0])
@pytest.mark.parametrize("sizes,types", LISTS)
def test_clip(ep, sizes, types, factor):
    grads = make(sizes, types, seed=len(sizes))
    before = [g.clone() for g in grads]
    max_norm = factor * max(exact_norm(before), 1e-3)
    norm = torch.full((1,), -1.0, device="cuda")
    ep.GradList(grads).norm(norm)
    n = exact_norm(before)
    assert abs(norm.item() - n) <= NORM_TOL * n
    assert all(torch.equal(g, b) for g, b in zip(grads, before))
    out = [torch.full_like(g, 7.0) for g in grads]
    ep.GradList(grads, out).clip(max_norm, norm)
    check_clip(out, before, max_norm, norm)
    assert all(torch.equal(g, b) for g, b in zip(grads, before))
    ep.GradList(grads).clip(max_norm, norm)
    assert all(torch.equal(g, o) for g, o in zip(grads, out))
    if factor > 1:
        assert all(torch.equal(g, b) for g, b in zip(grads, before))


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_any_alignment(ep, dtype):
    """Views that start anywhere, and outputs that lie differently to the 16-byte boundary than their inputs."""
    base = make([40000], [dtype], seed=3)[0]
    to = torch.full((40000,), 7.0, dtype=dtype, device="cuda")
    cuts = [(1, 5000), (5003, 1), (5007, 17), (6001, 8191), (20000, 15000)]
    grads = [base[a:a + n] for a, n in cuts]
    out = [to[a - 1 if i % 2 else a:][:n] for i, (a, n) in enumerate(cuts)]
    before = [g.clone() for g in grads]
    norm = torch.zeros((1,), device="cuda")
    ep.GradList(grads, out).clip(0.01, norm)
    check_clip(out, before, 0.01, norm)
    used = torch.zeros(40000, dtype=torch.bool, device="cuda")
    for i, (a, n) in enumerate(cuts):
        used[a - (i % 2):a - (i % 2) + n] = True
    assert (to[~used] == 7.0).all()


def test_empty_list(ep):
    norm = torch.full((1,), -1.0, device="cuda")
    ep.GradList([]).clip(1.0, norm)
    assert norm.item() == 0
    norm.fill_(-1.0)
    ep.GradList([]).norm(norm)
    assert norm.item() == 0


def test_zero_gradients_and_zero_limit(ep):
    norm = torch.full((1,), -1.0, device="cuda")
    z = [torch.zeros((100,), device="cuda")]
    ep.GradList(z).clip(1.0, norm)
    assert norm.item() == 0 and (z[0] == 0).all()
    g = make([100], [F32])
    ep.GradList(g).clip(0.0, norm)
    assert (g[0] == 0).all()


def test_nan_and_infinity(ep):
    norm = torch.zeros((1,), device="cuda")
    for bad in (float("nan"), float("inf")):
        g = make([5000, 70], [BF16, F32])
        g[1][3] = bad
        ep.GradList(g).clip(1.0, norm)
        if math.isnan(bad):
            assert torch.isnan(norm).all() and all(torch.isnan(t).all() for t in g)
        else:
            assert torch.isinf(norm).all() and (g[0] == 0).all() and torch.isnan(g[1][3])
            assert (g[1][4:] == 0).all()


def test_repeats_bit_by_bit_and_in_a_graph(ep):
    g = make([100003, 77, 1 << 18], [BF16, F32])
    out = [torch.empty_like(t) for t in g]
    lst, norm = ep.GradList(g, out), torch.zeros((1,), device="cuda")
    lst.clip(0.5, norm)
    first, n = [o.clone() for o in out], norm.item()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lst.clip(0.5, norm)
    for o in out:
        o.zero_()
    graph.replay()
    assert norm.item() == n and all(torch.equal(a, b) for a, b in zip(first, out))
