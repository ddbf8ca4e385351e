"""What ep_expert_ffn keeps for the backward pass (g and u), over the whole range of finite values."""
from __future__ import annotations

import math

import pytest
import torch

import experts_ref as ref
from gpu_harness import require_cuda

pytestmark = pytest.mark.gpu
BF16, F16 = torch.bfloat16, torch.float16
HALF_MAX = 65504.0
GRADS = ("d_rows", "d_w_gate", "d_w_up", "d_w_down")


@pytest.fixture(scope="module")
def ep():
    require_cuda()
    import combine_router_softmax_gb300 as m

    return m


def run(ep, counts, H, I, x_scale, seed, dtype=F16, dy_scale=0.1, **cfg):
    """One forward and backward call: inputs and outputs by name, and the experts' bounds."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    S, E = sum(counts), len(counts)
    n = lambda *shape, s=1.0: (torch.randn(shape, generator=gen, device="cuda") * s).to(BF16)  # noqa: E731
    o = {"x": n(S, H, s=x_scale), "d_y": n(S, H, s=dy_scale),
         "w": [n(E, I, H, s=1 / math.sqrt(H)), n(E, I, H, s=1 / math.sqrt(H)), n(E, H, I, s=1 / math.sqrt(I))]}
    full = lambda *shape, dtype=BF16: torch.full(shape, 7.0, dtype=dtype, device="cuda")  # noqa: E731
    for k in ("g", "u"):
        o[k] = full(S, I, dtype=dtype)
    for k in ("h", "d_g", "d_u"):
        o[k] = full(S, I)
    for k in ("y", "d_rows"):
        o[k] = full(S, H)
    for k, w in zip(("d_w_gate", "d_w_up", "d_w_down"), o["w"]):
        o[k] = torch.full_like(w, 7.0)
    bounds = [0]
    for c in counts:
        bounds.append(bounds[-1] + c)
    off = torch.tensor(bounds, dtype=torch.int32, device="cuda")
    cfg = ep.EpFfnConfig.make(rows=S, H=H, I=I, E=E, **cfg)
    ep.ep_expert_ffn(cfg, o["x"], off, *o["w"], o["h"], o["y"], g=o["g"], u=o["u"])
    ep.ep_expert_ffn_backward(cfg, o["x"], off, *o["w"], o["g"], o["u"], o["h"], o["d_y"], o["d_g"], o["d_u"],
                              *(o[k] for k in GRADS))
    torch.cuda.synchronize()
    assert ep.ep_device_error() == 0
    return o, bounds


def reference(x, w, d_y, half_step, limit):
    """One expert in 64 bits. g and u as they are kept: off by half_step of the value and by the fp32 sums' error,
    and no larger than `limit`, which silu has reached its limits by."""
    f = ref.forward(x, *w)
    for k, m in (("g", w[0]), ("u", w[1])):
        sums = x.shape[1] * ref.U32 * (x.abs() @ m.abs().T)
        f["tol_" + k] = ref.SLACK * (half_step * f[k].abs() + sums)
    kept = {**f, "g": f["g"].clamp(-limit, limit), "u": f["u"].clamp(-limit, limit)}
    return f, kept, ref.backward(x, *w, d_y, kept)


def check(o, bounds, half_step, limit):
    for e, (a, b) in enumerate(zip(bounds, bounds[1:])):
        s = slice(a, b)
        f, kept, r = reference(o["x"][s].double(), [w[e].double() for w in o["w"]], o["d_y"][s].double(), half_step, limit)
        for k, want in (("g", kept["g"]), ("u", kept["u"]), ("h", f["h"]), ("y", f["y"])):
            ref.check(o[k][s], want, f["tol_" + k], f"{k} of expert {e}")
        for k in ("d_g", "d_u", "d_rows"):
            ref.check(o[k][s], r[k], r["tol_" + k], f"{k} of expert {e}")
        for k in ("d_w_gate", "d_w_up", "d_w_down"):
            ref.check(o[k][e], r[k], r["tol_" + k], f"{k} of expert {e}")


@pytest.mark.parametrize("counts,H,I", [([40], 64, 64), ([5, 300], 264, 136)])
def test_halves_beyond_their_range(ep, counts, H, I):
    """g and u of both signs beyond 65504: kept as 65504, at which silu is at its limit, and every gradient is
    finite and what that value gives."""
    o, bounds = run(ep, counts, H, I, 1e5, seed=H)
    for k in ("g", "u"):
        assert torch.isfinite(o[k]).all() and (o[k] == HALF_MAX).any() and (o[k] == -HALF_MAX).any()
    check(o, bounds, ref.U11, HALF_MAX)


@pytest.mark.parametrize("counts,H,I", [([40], 64, 64), ([5, 300], 264, 136)])
@pytest.mark.parametrize("x_scale", [1e-12, 1e-6, 1.0, 1e5, 1e15])
def test_bfloat16_at_any_scale(ep, counts, H, I, x_scale):
    """Kept as bf16, g and u of any size give gradients within the roundings' bounds."""
    o, bounds = run(ep, counts, H, I, x_scale, seed=I, dtype=BF16, saved_bf16=1)
    check(o, bounds, ref.U16, math.inf)


def test_bfloat16_at_the_end_of_fp32(ep):
    """Sums between the largest bf16 and the largest fp32 value stay finite, and silu is at its limits."""
    n = 64
    x = torch.zeros((3, n), dtype=BF16, device="cuda")
    x[0, 0], x[1, 0], x[2, 0] = 2.0**127, -2.0**127, 1.0
    x[:, 1] = x[:, 0]
    x[0, 2], x[1, 2] = 1.0, -1.0
    w = torch.zeros((1, n, n), dtype=BF16, device="cuda")
    w[0, :, 0], w[0, :, 1] = 2 - 2.0**-7, 2.0**-8  # x0 (w0 + w1) = 2^127 (2 - 2^-8): bf16 would round it up
    up, down = torch.zeros_like(w), torch.zeros_like(w)
    up[0, :, 2], down[0] = 1.0, 1.0
    g, u, h, d_g, d_u = (torch.full((3, n), 7.0, dtype=BF16, device="cuda") for _ in range(5))
    y, d_y = torch.zeros((3, n), dtype=BF16, device="cuda"), torch.ones((3, n), dtype=BF16, device="cuda")
    off = torch.tensor([0, 3], dtype=torch.int32, device="cuda")
    cfg = ep.EpFfnConfig.make(rows=3, H=n, I=n, E=1, saved_bf16=1)
    ep.ep_expert_ffn(cfg, x, off, w, up, down, h, y, g=g, u=u)
    ep.ep_expert_ffn_backward(cfg, x, off, w, up, down, g, u, h, d_y, d_g, d_u)
    top = torch.finfo(BF16).max
    assert (g[0] == top).all() and (g[1] == -top).all()
    assert (u[0] == 1).all() and (u[1] == -1).all()
    # dh = 64: d_g = dh u silu'(g) with silu' = 1 and 0, d_u = dh silu(g), which is infinite and 0
    assert (d_g[0] == 64).all() and (d_g[1] == 0).all() and (d_u[1] == 0).all()


@pytest.mark.parametrize("kept", [F16, BF16])
def test_an_infinite_row_stays_infinite(ep, kept):
    """What the forward pass cannot represent is not made finite: a row with an infinity has no gradient."""
    gen = torch.Generator(device="cuda").manual_seed(0)
    x = torch.randn((9, 64), generator=gen, device="cuda").to(BF16)
    x[4, 7] = float("inf")
    x[6, 3] = float("nan")
    w = [(torch.randn((1, 64, 64), generator=gen, device="cuda") / 8).to(BF16) for _ in range(3)]
    h, y = (torch.empty((9, 64), dtype=BF16, device="cuda") for _ in range(2))
    g, u = (torch.empty((9, 64), dtype=kept, device="cuda") for _ in range(2))
    off = torch.tensor([0, 9], dtype=torch.int32, device="cuda")
    ep.ep_expert_ffn(ep.EpFfnConfig.make(rows=9, H=64, I=64, E=1, saved_bf16=int(kept is BF16)), x, off, *w, h, y, g=g, u=u)
    for t in (g, u):
        assert torch.isinf(t[4]).all() and torch.isnan(t[6]).all()
        assert torch.isfinite(t[[0, 1, 2, 3, 5, 7, 8]]).all()
