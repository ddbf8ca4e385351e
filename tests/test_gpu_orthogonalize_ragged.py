"""ep_orthogonalize of matrices whose result's rows lie on no 16-byte boundary: it goes out of an epilogue's buffers value by
value, and the next pieces are copied into the same buffers. Many pieces a CTA, wide and tall; and what else is in a batch."""
from __future__ import annotations

import pytest
import torch

from gpu_harness import require_cuda

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ep():
    require_cuda()
    import combine_router_softmax_gb300 as m

    return m


def call(ep, m, out, ws):
    cfg = ep.EpOrthoConfig.make(B=m.shape[0], N=m.shape[1], K=m.shape[2], dtype=m.dtype)
    ep.ep_orthogonalize(cfg, m, out, ws)


def setup(ep, B, N, K, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    m = torch.randn((B, N, K), generator=gen, device="cuda").to(torch.bfloat16)
    cfg = ep.EpOrthoConfig.make(B=B, N=N, K=K)
    return m, torch.empty((ep.ep_orthogonalize_workspace_size(cfg),), dtype=torch.uint8, device="cuda")


# narrow and wide tiles of single CTAs, and pairs
@pytest.mark.parametrize("B,N,K", [(1, 300, 515), (7, 333, 1001), (9, 1001, 333), (6, 1100, 1203), (6, 1203, 1099)])
def test_the_same_every_time(ep, B, N, K):
    """Bit by bit in twenty calls, and where the matrix lies in a wider one with zeros behind it, whose result goes out by copies:
    there within two roundings to bf16, 2^-8 of a value each, and the sums' order, a tenth of that of the matrix' rms."""
    m, ws = setup(ep, B, N, K, seed=N)
    want = torch.empty_like(m)
    call(ep, m, want, ws)
    got = torch.empty_like(m)
    for _ in range(20):
        got.fill_(float("nan"))
        call(ep, m, got, ws)
        assert torch.equal(got, want)
    n, k = (N + 7) // 8 * 8, (K + 7) // 8 * 8
    wide, ws2 = setup(ep, B, n, k, seed=0)
    wide.zero_()
    wide[:, :N, :K] = m
    filled = torch.empty_like(wide)
    call(ep, wide, filled, ws2)
    w, f = want.double(), filled[:, :N, :K].double()
    rms = w.square().mean().sqrt()
    assert ((w - f).abs() <= 2.0**-7 * w.abs() + 2.0**-8 * rms).all()


@pytest.mark.parametrize("B,N,K", [(5, 256, 300), (12, 100, 200), (6, 1100, 1200)])
def test_whatever_else_is_in_the_batch(ep, B, N, K):
    m, ws = setup(ep, B, N, K, seed=2)
    want = torch.empty_like(m)
    call(ep, m, want, ws)
    other, _ = setup(ep, B, N, K, seed=3)
    other[1], other[B - 1] = m[1], m[B - 1]
    got = torch.empty_like(m)
    call(ep, other, got, ws)
    assert torch.equal(got[1], want[1]) and torch.equal(got[B - 1], want[B - 1])
