"""ep_balance and its gradient at the most rows that there can be, with sequences that begin just before the last one: a
warp's first row would lie beyond 2^31."""
from __future__ import annotations

import pytest
import torch

from gpu_harness import require_cuda

pytestmark = pytest.mark.gpu


def test_a_short_sequence_behind_nearly_2_31_rows():
    require_cuda()
    import combine_router_softmax_gb300 as ep

    T, S = 2**31 - 1, 3
    first = [0, T - 150, T - 3, T]
    cfg = ep.EpConfig.make(T=T, H=8, E=1, R=1, k=1)
    logits = torch.full((T, 1), 0.5, device="cuda")
    logits[T - 150:T - 3] = 2.0
    logits[T - 3:] = -3.0
    idx = torch.zeros((T, 1), dtype=torch.int32, device="cuda")
    bounds = torch.tensor(first, dtype=torch.int32, device="cuda")
    count = torch.full((S, 1), -1, dtype=torch.int32, device="cuda")
    load, prob = torch.full((S, 1), -1.0, device="cuda"), torch.full((S, 1), -1.0, device="cuda")
    loss = torch.full((S, 2), -1.0, device="cuda")
    ws = torch.empty((ep.ep_balance_workspace_size(cfg, S),), dtype=torch.uint8, device="cuda")
    ep.ep_balance(cfg, logits, idx, bounds, None, count, load, prob, loss, ws)
    rows = [b - a for a, b in zip(first, first[1:])]
    assert count[:, 0].tolist() == rows
    # one expert: its probability is 1, the logarithm its logit; chains of sums are shorter than 2^17 terms
    want = torch.tensor([[1.0, 0.25], [1.0, 4.0], [1.0, 9.0]], device="cuda")
    assert ((load - 1).abs() <= 2.0**-22).all() and ((prob - 1).abs() <= 2.0**-7).all()
    assert ((loss - want).abs() <= 2.0**-7 * want).all()
    assert ((prob[1:] - 1).abs() <= 2.0**-20).all() and ((loss[1:] - want[1:]).abs() <= 2.0**-20 * want[1:]).all()
    del idx
    d_loss = torch.tensor([[1.0, 3.0]], device="cuda").expand(S, 2).contiguous()
    d = torch.full((T, 1), float("nan"), device="cuda")
    ep.ep_balance_backward(cfg, logits, bounds, None, load, d_loss, None, d)
    for s, (at, l) in enumerate(((0, 0.5), (T - 150, 2.0), (T - 3, -3.0))):
        w = 6.0 * l / rows[s]
        slope = d[at:first[s + 1], 0]
        assert ((slope[-150:].double() - w).abs() <= 2.0**-19 * abs(w)).all() and ((slope[:150].double() - w).abs() <= 2.0**-19 * abs(w)).all()
