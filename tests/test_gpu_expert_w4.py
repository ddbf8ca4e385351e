"""4-bit weights: ep_w4_pack bit by bit, ep_w4_linear and ep_expert_ffn_w4 against 64 bits."""
from __future__ import annotations

import math

import pytest
import torch

import experts_ref as ref
from gpu_harness import require_cuda

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def ep():
    require_cuda()
    import combine_router_softmax_gb300 as m

    return m


def pack_plain(w, group):
    """The packed form by its definition, with the quotients taken in 64 bits."""
    E, N, K = w.shape
    Kp = (K + 127) // 128 * 128
    full = torch.zeros((E, N, Kp), dtype=torch.float64, device=w.device)
    full[:, :, :K] = w.double()
    groups = full.view(E, N, Kp // group, group)
    scale = (groups.abs().amax(-1) / 7).to(BF16)
    s = scale.double()[..., None]
    q = torch.where(s > 0, (groups / s.clamp(min=1e-300)).round().clamp(-8, 7), 0.0) + 8
    q = q.view(E, N, Kp).long()
    words = torch.zeros((E, N, Kp // 8), dtype=torch.int64, device=w.device)
    for c in range(Kp // 128):
        for t in range(4):
            for j in range(4):
                for i in range(8):
                    k = 128 * c + 32 * j + 8 * t + 2 * (i % 4) + i // 4
                    words[:, :, 16 * c + 4 * t + j] |= q[:, :, k] << (4 * i)
    by = torch.stack([(words >> (8 * b)) & 255 for b in range(4)], -1).view(E, N, Kp // 2)
    values = (q.double() - 8).view(E, N, Kp // group, group) * s
    return by.to(torch.uint8), scale, values.view(E, N, Kp)[:, :, :K]


def packed(ep, w, group):
    E, N, K = w.shape
    cfg = ep.EpW4Config.make(N=N, K=K, E=E, group=group)
    Kp = (K + 127) // 128 * 128
    q = torch.full((E, N, Kp // 2), 0xAA, dtype=torch.uint8, device="cuda")
    scale = torch.full((E, N, Kp // group), 9.0, dtype=BF16, device="cuda")
    assert ep.ep_w4_sizes(cfg) == (q.numel(), 2 * scale.numel())
    ep.ep_w4_pack(cfg, w, q, scale)
    return q, scale


def normal(gen, *shape, s=1.0):
    return (torch.randn(shape, generator=gen, device="cuda") * s).to(BF16)


def offsets(counts, before=0):
    b = [before]
    for c in counts:
        b.append(b[-1] + c)
    return b, torch.tensor(b, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("E,N,K", [(1, 1, 8), (2, 5, 128), (3, 7, 200), (1, 64, 1032), (4, 33, 120)])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_pack(ep, E, N, K, group):
    w = normal(torch.Generator(device="cuda").manual_seed(K), E, N, K, s=0.05)
    w[0, 0, :8] = 0  # a run of zeros, and with K = 8 a group of nothing else
    w[-1, -1] *= 1e-3
    q, scale = packed(ep, w, group)
    want_q, want_s, _ = pack_plain(w, group)
    assert torch.equal(scale.view(torch.int16), want_s.view(torch.int16))
    assert torch.equal(q, want_q)


def test_pack_rounds_halves_to_even(ep):
    """Quotients of exactly n + 1/2: scale 1 (the largest value is 7), values at the halves."""
    w = torch.zeros((1, 1, 128), dtype=BF16, device="cuda")
    w[0, 0, :15] = torch.arange(-7.0, 8.0, device="cuda") + 0.0
    w[0, 0, 16:30] = torch.arange(-6.5, 7.5, device="cuda")
    q, scale = packed(ep, w, 128)
    want_q, want_s, _ = pack_plain(w, 128)
    assert scale.item() == 1.0 and torch.equal(q, want_q) and torch.equal(scale, want_s)


LINEAR = [
    ([1], 1, 8, 0, 0), ([1], 64, 128, 0, 0), ([3], 65, 136, 0, 0), ([8], 130, 1000, 2, 1), ([9], 63, 256, 0, 0),
    ([16], 200, 2056, 0, 0), ([17, 0, 5, 40], 72, 392, 3, 2), ([0, 0, 1], 321, 1024, 0, 0), ([2] * 150, 40, 128, 0, 0),
]


@pytest.mark.parametrize("counts,N,K,before,after", LINEAR)
@pytest.mark.parametrize("group", [32, 64, 128])
def test_linear(ep, counts, N, K, before, after, group):
    gen = torch.Generator(device="cuda").manual_seed(N + K)
    E, S = len(counts), before + sum(counts) + after
    w = normal(gen, E, N, K, s=1 / math.sqrt(K))
    x = normal(gen, S, K)
    q, scale = packed(ep, w, group)
    _, _, values = pack_plain(w, group)
    b, off = offsets(counts, before)
    y = torch.full((S, N), 7.0, dtype=BF16, device="cuda")
    ep.ep_w4_linear(ep.EpW4Config.make(rows=S, N=N, K=K, E=E, group=group), x, off, q, scale, y)
    for e in range(E):
        s = slice(b[e], b[e + 1])
        if s.stop == s.start:
            continue
        xe = x[s].double()
        want = xe @ values[e].T
        # K products and K / group scalings in fp32, one rounding of the result
        tol = ref.SLACK * ((K + K // group + 16) * ref.U32 * (xe.abs() @ values[e].abs().T) + ref.U16 * want.abs())
        ref.check(y[s], want, tol, f"expert {e}")
    assert (y[:before] == 7.0).all() and (y[b[-1]:] == 7.0).all()


@pytest.mark.parametrize("counts,H,I,group", [
    ([1], 128, 64, 128), ([1, 0, 2], 264, 136, 32), ([8, 9, 3], 1000, 360, 64), ([30, 1], 512, 1032, 128),
    ([1] * 8 + [0] * 56, 768, 256, 128),
])
def test_block(ep, counts, H, I, group):
    gen = torch.Generator(device="cuda").manual_seed(H)
    E, S = len(counts), sum(counts)
    x = normal(gen, S, H)
    ws = [normal(gen, E, I, H, s=1 / math.sqrt(H)), normal(gen, E, I, H, s=1 / math.sqrt(H)),
          normal(gen, E, H, I, s=1 / math.sqrt(I))]
    parts = [packed(ep, w, group) for w in ws]
    values = [pack_plain(w, group)[2] for w in ws]
    b, off = offsets(counts)
    h = torch.full((S, I), 7.0, dtype=BF16, device="cuda")
    y = torch.full((S, H), 7.0, dtype=BF16, device="cuda")
    ep.ep_expert_ffn_w4(ep.EpFfnConfig.make(rows=S, H=H, I=I, E=E), group, x, off, *parts[0], *parts[1], *parts[2], h, y)
    for e in range(E):
        s = slice(b[e], b[e + 1])
        if s.stop > s.start:
            # the sums are K + K / group long, where forward() counts K: 2 K covers them
            f = ref.forward(x[s].double(), *(v[e] for v in values))
            ref.check(h[s], f["h"], 2 * f["tol_h"], f"h of expert {e}")
            ref.check(y[s], f["y"], 2 * f["tol_y"], f"y of expert {e}")


def test_graph_and_stream(ep):
    gen = torch.Generator(device="cuda").manual_seed(1)
    w = normal(gen, 4, 96, 264)
    q, scale = packed(ep, w, 64)
    x, y = normal(gen, 12, 264), torch.zeros((12, 96), dtype=BF16, device="cuda")
    _, off = offsets([4, 0, 7, 1])
    cfg = ep.EpW4Config.make(rows=12, N=96, K=264, E=4, group=64)
    ep.ep_w4_linear(cfg, x, off, q, scale, y)
    want = y.clone()
    y.zero_()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    ep.ep_w4_linear(cfg, x, off, q, scale, y, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(y, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ep.ep_w4_linear(cfg, x, off, q, scale, y)
    y.zero_()
    g.replay()
    assert torch.equal(y, want)


def test_nan_row_stays_a_row(ep):
    gen = torch.Generator(device="cuda").manual_seed(2)
    q, scale = packed(ep, normal(gen, 2, 64, 256), 128)
    x = normal(gen, 6, 256)
    _, off = offsets([4, 2])
    y, z = (torch.zeros((6, 64), dtype=BF16, device="cuda") for _ in range(2))
    cfg = ep.EpW4Config.make(rows=6, N=64, K=256, E=2, group=128)
    ep.ep_w4_linear(cfg, x, off, q, scale, y)
    x[1] = float("nan")
    ep.ep_w4_linear(cfg, x, off, q, scale, z)
    keep = [0, 2, 3, 4, 5]
    assert torch.equal(y[keep], z[keep]) and torch.isnan(z[1]).all()
