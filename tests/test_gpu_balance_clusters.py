"""ep_balance where the CTAs of a cluster hand their parts of a loss to its first one, which may start last."""
from __future__ import annotations

import pytest
import torch

from gpu_harness import require_cuda

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("E,k,T,first", [(256, 8, 4096, None), (256, 8, 20000, [0, 9000, 20000]), (96, 4, 30000, [0, 30000])])
def test_the_same_loss_while_the_sms_are_taken(E, k, T, first):
    """Products on another stream come and go on the SMs, so that a cluster's CTAs find their place one by one: every call gives
    the loss that it gives alone, bit by bit, and that is within 2^-14 of the loss in 64 bits (sums of fewer than 2^10 terms
    a chain)."""
    require_cuda()
    import combine_router_softmax_gb300 as ep

    gen = torch.Generator(device="cuda").manual_seed(1)
    S = 1 if first is None else len(first) - 1
    cfg = ep.EpConfig.make(T=T, H=8, E=E, R=1, k=k)
    logits = torch.randn((T, E), generator=gen, device="cuda")
    idx = torch.topk(logits, k, dim=-1)[1].to(torch.int32)
    bounds = None if first is None else torch.tensor(first, dtype=torch.int32, device="cuda")
    ws = torch.empty((ep.ep_balance_workspace_size(cfg, S),), dtype=torch.uint8, device="cuda")
    count = torch.empty((S, E), dtype=torch.int32, device="cuda")
    load, prob = torch.empty((S, E), device="cuda"), torch.empty((S, E), device="cuda")

    def call(loss):
        ep.ep_balance(cfg, logits, idx, bounds, None, count, load, prob, loss, ws)

    want = torch.full((S, 2), float("nan"), device="cuda")
    call(want)
    for s, (a, b) in enumerate(zip(first or [0], (first or [0, T])[1:])):
        l = logits[a:b].double()
        f = torch.bincount(idx[a:b].long().flatten(), minlength=E).double() / (k * (b - a))
        exact = torch.stack([E * (f * torch.softmax(l, -1).mean(0)).sum(), torch.logsumexp(l, -1).square().mean()])
        assert ((want[s].double() - exact).abs() <= 2.0**-14 * exact).all()
    other, a = torch.cuda.Stream(), torch.randn((2048, 2048), device="cuda")
    other.wait_stream(torch.cuda.current_stream())
    got = torch.full((200, S, 2), float("nan"), device="cuda")
    torch.cuda.synchronize()
    for i in range(200):
        if i % 4 == 0:
            with torch.cuda.stream(other):
                a @ a
        call(got[i])
    torch.cuda.synchronize()
    assert torch.equal(got, want.expand(200, S, 2))
