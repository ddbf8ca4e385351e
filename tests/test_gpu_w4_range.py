"""4-bit products where activations differ much in size: a large one that meets a weight of zero leaves nothing
behind, and infinities give what the values give, however many rows an expert has."""
from __future__ import annotations

import math

import pytest
import torch

import experts_ref as ref
from gpu_harness import require_cuda
from test_gpu_expert_w4 import normal, pack_plain, packed

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def ep():
    require_cuda()
    import combine_router_softmax_gb300 as m

    return m


def linear(ep, x, q, scale, N, K, group):
    rows = x.shape[0]
    off = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
    y = torch.full((rows, N), 7.0, dtype=BF16, device="cuda")
    ep.ep_w4_linear(ep.EpW4Config.make(rows=rows, N=N, K=K, E=1, group=group), x, off, q, scale, y)
    return y


@pytest.mark.parametrize("rows", [1, 8, 9, 16, 40])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("size", [1e3, 1e5, 1e30])
def test_large_activations_at_zero_weights(ep, rows, group, size):
    """One activation in every 40 is `size`, where every weight is 0: the sums are those of the others."""
    N, K = 72, 1032
    gen = torch.Generator(device="cuda").manual_seed(rows + group)
    w = normal(gen, 1, N, K, s=1 / math.sqrt(K))
    x = normal(gen, rows, K)
    w[:, :, ::40] = 0
    x[:, ::40] = size
    q, scale = packed(ep, w, group)
    _, _, values = pack_plain(w, group)
    want = x.double() @ values[0].T
    # as for any product: K products and K / group scalings in fp32, one rounding of the result
    tol = ref.SLACK * ((K + K // group + 16) * ref.U32 * (x.double().abs() @ values[0].abs().T) + ref.U16 * want.abs())
    ref.check(linear(ep, x, q, scale, N, K, group), want, tol, "y")


@pytest.mark.parametrize("rows", [1, 8, 9, 40])
def test_infinite_activations(ep, rows):
    """An infinity times a weight has the weight's sign, and is no number where the weight is 0."""
    N, K = 64, 256
    gen = torch.Generator(device="cuda").manual_seed(rows)
    w = normal(gen, 1, N, K, s=1 / math.sqrt(K))
    w[0, ::5, 17] = 0
    x = normal(gen, rows, K)
    x[-1, 17] = float("inf")
    q, scale = packed(ep, w, 64)
    _, _, values = pack_plain(w, 64)
    y = linear(ep, x, q, scale, N, K, 64)
    at = values[0, :, 17]
    assert torch.equal(torch.isnan(y[-1]), at == 0)
    assert (y[-1][at > 0] == float("inf")).all() and (y[-1][at < 0] == -float("inf")).all()
    assert torch.isfinite(y[:-1]).all()
