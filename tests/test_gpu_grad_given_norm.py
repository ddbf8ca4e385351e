"""ep_grad_clip_with_norm: gradients spread over several lists, as over processes, clipped by the norm of all."""
from __future__ import annotations

import math

import pytest
import torch

from gpu_harness import require_cuda
from test_gpu_grad_clip import BF16, F16, F32, NORM_TOL, check_clip, exact_norm, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ep():
    require_cuda()
    import combine_router_softmax_gb300 as m

    return m


@pytest.mark.parametrize("factor", [0.3, 2.0])
@pytest.mark.parametrize("parts", [([1], [5]), ([4097, 1, 0], [300007]), ([17] * 900, [1 << 20, 3]), ([], [70])])
def test_two_lists_by_one_norm(ep, parts, factor):
    lists = [make(p, [F32, BF16, F16], seed=i) for i, p in enumerate(parts)]
    before = [[g.clone() for g in ts] for ts in lists]
    n = exact_norm(before[0] + before[1])
    squares = torch.zeros(1, dtype=torch.float64, device="cuda")
    for ts in lists:
        own = torch.full((1,), -1.0, device="cuda")
        ep.GradList(ts).norm(own)
        squares += own.double() ** 2
    norm = squares.sqrt().float()
    assert abs(norm.item() - n) <= NORM_TOL * n
    kept = norm.clone()
    for ts in lists:
        ep.GradList(ts).clip_with_norm(factor * n, norm)
    assert torch.equal(norm, kept)
    # check_clip's factor is made of the norm of the tensors that it gets: all of them
    check_clip([g for ts in lists for g in ts], [g for ts in before for g in ts], factor * n, norm)


def test_the_same_as_clip_for_its_own_norm(ep):
    grads = make([5000, 77, 300003], [BF16, F32, F16])
    out = [[torch.full_like(g, 7.0) for g in grads] for _ in range(2)]
    norm = torch.zeros((1,), device="cuda")
    ep.GradList(grads, out[0]).clip(0.25, norm)
    ep.GradList(grads, out[1]).clip_with_norm(0.25, norm)
    assert all(torch.equal(a, b) for a, b in zip(*out))


def test_what_the_norm_says_passes_to_the_values(ep):
    for value, check in ((float("nan"), torch.isnan), (float("inf"), lambda t: t == 0)):
        g = make([5000, 70], [BF16, F32])
        ep.GradList(g).clip_with_norm(1.0, torch.full((1,), value, device="cuda"))
        assert all(check(t).all() for t in g)
    g = make([100], [F32])
    before = g[0].clone()
    ep.GradList(g).clip_with_norm(1.0, torch.zeros((1,), device="cuda"))
    assert torch.equal(g[0], before)
    ep.GradList([]).clip_with_norm(1.0, torch.ones((1,), device="cuda"))


def test_other_stream_and_graph(ep):
    """The norm is read when the stream gets there: a graph replays on what it holds by then."""
    g = make([9000, 41], [F32, BF16])
    out = [torch.empty_like(t) for t in g]
    lst, norm = ep.GradList(g, out), torch.full((1,), 4.0, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    lst.clip_with_norm(1.0, norm, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lst.clip_with_norm(1.0, norm)
    for value in (8.0, 2.0):
        norm.fill_(value)
        graph.replay()
        for o, t in zip(out, g):
            want = (t.double() / (value + 1e-6)).to(t.dtype)
            assert torch.allclose(o.float(), want.float(), rtol=2.0**-7, atol=0), value
    assert math.isfinite(norm.item())
