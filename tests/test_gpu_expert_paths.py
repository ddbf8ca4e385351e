"""Paths of the experts' kernels that sizes decide on: bands of tiles in the weights' gradients, the streamed kernel
with as many experts as it takes, 4-bit products of several passes, weights of more than 2^31 values."""
from __future__ import annotations

import math

import pytest
import torch

import experts_ref as ref
from gpu_harness import require_cuda
from test_gpu_expert_ffn import Block
from test_gpu_expert_w4 import normal, offsets, pack_plain, packed

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def ep():
    require_cuda()
    import combine_router_softmax_gb300 as m

    return m


@pytest.mark.parametrize("counts,H,I", [
    ([2100, 700], 2312, 264),        # by CTA pairs: ten row tiles of d_w_down, bands of eight
    ([2100] + [0] * 6 + [1], 2312, 264),  # single CTAs: nineteen, bands of sixteen
    ([2049, 3], 264, 4104),          # the bands in d_w_gate and d_w_up
])
def test_weight_gradients_in_bands(ep, counts, H, I):
    """More than 2048 rows of an expert, output rows that are no whole number of bands."""
    b = Block(ep, counts, H, I, seed=H)
    b.forward(ep)
    b.backward(ep)
    b.check(ep)


def check_few_rows(ep, b):
    b.forward(ep, save=False)
    torch.cuda.synchronize()
    assert ep.ep_device_error() == 0
    for e, s, f, _ in b.experts():
        if s.stop > s.start:
            ref.check(b.o["h"][s], f["h"], f["tol_h"], f"h of expert {e}")
            ref.check(b.o["y"][s], f["y"], f["tol_y"], f"y of expert {e}")
    outside = list(range(b.bounds[0])) + list(range(b.bounds[-1], b.cfg.rows))
    assert (b.o["y"][outside] == 7.0).all() and (b.o["h"][outside] == 7.0).all()


@pytest.mark.parametrize("counts,H,I", [
    ([1, 0, 0, 0] * 16, 1032, 520),           # as many experts as rows fit
    ([0, 1] * 16, 2312, 4104),                # many blocks of columns an expert, work for every CTA
    ([0] * 100 + [1] * 8 + [0] * 400 + [8], 264, 136),
    ([16], 4104, 2056),                       # a whole pass of one expert
    ([2, 0, 7, 0, 6], 120, 8200),
])
def test_streamed_rows(ep, counts, H, I):
    """Up to 16 rows, g and u not wanted: the kernel that streams the weights."""
    assert sum(counts) <= 16
    check_few_rows(ep, Block(ep, counts, H, I, seed=I))


@pytest.mark.parametrize("counts,N,K", [([100, 33, 0, 257], 136, 520), ([48], 72, 1032), ([49, 1, 64], 321, 128)])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_4_bit_products_of_several_passes(ep, counts, N, K, group):
    gen = torch.Generator(device="cuda").manual_seed(N + K)
    E, S = len(counts), sum(counts)
    w, x = normal(gen, E, N, K, s=1 / math.sqrt(K)), normal(gen, S, K)
    q, scale = packed(ep, w, group)
    _, _, values = pack_plain(w, group)
    b, off = offsets(counts)
    y = torch.full((S, N), 7.0, dtype=BF16, device="cuda")
    ep.ep_w4_linear(ep.EpW4Config.make(rows=S, N=N, K=K, E=E, group=group), x, off, q, scale, y)
    for e in range(E):
        s = slice(b[e], b[e + 1])
        if s.stop > s.start:
            xe = x[s].double()
            want = xe @ values[e].T
            # K products and K / group scalings in fp32, one rounding of the result
            tol = ref.SLACK * ((K + K // group + 16) * ref.U32 * (xe.abs() @ values[e].abs().T) + ref.U16 * want.abs())
            ref.check(y[s], want, tol, f"expert {e}")


def free(least_gb):
    if torch.cuda.mem_get_info()[0] < least_gb << 30:
        pytest.skip(f"needs {least_gb} GB of device memory")


@pytest.mark.parametrize("save", [True, False])
def test_weights_beyond_2_31_values(ep, save):
    """The last expert's weights start beyond 2^31 values, their gradients as well; the others have no rows, and
    their gradients are zero."""
    free(80)
    E, I, H, rows = 9, 16392, 16384, 5
    assert (E - 1) * I * H > 2**31
    gen = torch.Generator(device="cuda").manual_seed(1)
    w = [torch.empty((E, *s), dtype=BF16, device="cuda") for s in ((I, H), (I, H), (H, I))]
    for t in w:
        t[-1] = normal(gen, *t.shape[1:], s=1 / math.sqrt(t.shape[-1]))
    x, d_y = normal(gen, rows, H), normal(gen, rows, H, s=0.1)
    off = torch.tensor([0] * E + [rows], dtype=torch.int32, device="cuda")
    cfg = ep.EpFfnConfig.make(rows=rows, H=H, I=I, E=E)
    h, d_g, d_u = (torch.full((rows, I), 7.0, dtype=BF16, device="cuda") for _ in range(3))
    g, u = (torch.full((rows, I), 7.0, dtype=torch.float16, device="cuda") for _ in range(2))
    y, d_rows = (torch.full((rows, H), 7.0, dtype=BF16, device="cuda") for _ in range(2))
    ep.ep_expert_ffn(cfg, x, off, *w, h, y, g=g if save else None, u=u if save else None)
    last = [t[-1].double() for t in w]
    f = ref.forward(x.double(), *last)
    ref.check(h, f["h"], f["tol_h"], "h")
    ref.check(y, f["y"], f["tol_y"], "y")
    if not save:
        return
    grads = [torch.full_like(t, 7.0) for t in w]
    ep.ep_expert_ffn_backward(cfg, x, off, *w, g, u, h, d_y, d_g, d_u, d_rows, *grads)
    r = ref.backward(x.double(), *last, d_y.double(), f)
    for k, got in (("d_g", d_g), ("d_u", d_u), ("d_rows", d_rows), ("d_w_gate", grads[0][-1]), ("d_w_up", grads[1][-1]),
                   ("d_w_down", grads[2][-1])):
        ref.check(got, r[k], r["tol_" + k], k)
    for t in grads:
        assert all(not t[e].any() for e in range(E - 1))
    assert ep.ep_device_error() == 0


def test_4_bit_weights_beyond_2_31_bytes(ep):
    free(40)
    E, N, K, rows = 5, 32776, 32768, 3
    assert (E - 1) * N * K // 2 > 2**31
    gen = torch.Generator(device="cuda").manual_seed(2)
    w = normal(gen, 1, N, K, s=1 / math.sqrt(K))
    q = torch.empty((E, N, K // 2), dtype=torch.uint8, device="cuda")
    scale = torch.empty((E, N, K // 64), dtype=BF16, device="cuda")
    one = ep.EpW4Config.make(N=N, K=K, E=1, group=64)
    ep.ep_w4_pack(one, w, q[-1:], scale[-1:])
    x, y = normal(gen, rows, K), torch.full((rows, N), 7.0, dtype=BF16, device="cuda")
    off = torch.tensor([0] * E + [rows], dtype=torch.int32, device="cuda")
    ep.ep_w4_linear(ep.EpW4Config.make(rows=rows, N=N, K=K, E=E, group=64), x, off, q, scale, y)
    some = torch.cat([torch.arange(0, 64), torch.arange(N - 64, N)]).cuda()
    values = pack_plain(w[:, some].contiguous(), 64)[2][0]
    want = x.double() @ values.T
    tol = ref.SLACK * ((K + K // 64 + 16) * ref.U32 * (x.double().abs() @ values.abs().T) + ref.U16 * want.abs())
    ref.check(y[:, some], want, tol, "y")
