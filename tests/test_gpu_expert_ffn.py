"""ep_expert_ffn and ep_expert_ffn_backward against the block in 64 bits (experts_ref)."""
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


class Block:
    """Inputs and sentinel-filled outputs of one call; `before` / `after` rows belong to no expert."""

    def __init__(self, ep, counts, H, I, before=0, after=0, seed=0, scale=1.0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        S, E = before + sum(counts) + after, len(counts)
        n = lambda *shape, s=1.0: (torch.randn(shape, generator=gen, device="cuda") * s).to(BF16)  # noqa: E731
        self.cfg = ep.EpFfnConfig.make(rows=S, H=H, I=I, E=E)
        bounds = [before]
        for c in counts:
            bounds.append(bounds[-1] + c)
        self.bounds = bounds
        self.offset = torch.tensor(bounds, dtype=torch.int32, device="cuda")
        self.x, self.dy = n(S, H, s=scale), n(S, H, s=0.1)
        self.w = [n(E, I, H, s=1 / math.sqrt(H)), n(E, I, H, s=1 / math.sqrt(H)), n(E, H, I, s=1 / math.sqrt(I))]
        full = lambda *shape: torch.full(shape, 7.0, dtype=BF16, device="cuda")  # noqa: E731
        self.o = {**{k: full(S, I) for k in ("h", "d_g", "d_u")}, "g": full(S, I).half(), "u": full(S, I).half(), "y": full(S, H), "d_rows": full(S, H),
                  "d_w_gate": full(E, I, H), "d_w_up": full(E, I, H), "d_w_down": full(E, H, I)}

    def forward(self, ep, save=True, **kw):
        o = self.o
        ep.ep_expert_ffn(self.cfg, self.x, self.offset, *self.w, o["h"], o["y"], g=o["g"] if save else None,
                         u=o["u"] if save else None, **kw)

    def backward(self, ep, want=("d_rows", "d_w_gate", "d_w_up", "d_w_down"), **kw):
        o = self.o
        ep.ep_expert_ffn_backward(self.cfg, self.x, self.offset, *self.w, o["g"], o["u"], o["h"], self.dy, o["d_g"],
                                  o["d_u"], **{k: o[k] for k in want}, **kw)

    def experts(self):
        """Per expert: its rows' slice and the reference values with their bounds."""
        for e, (a, b) in enumerate(zip(self.bounds, self.bounds[1:])):
            w = [t[e].double() for t in self.w]
            x, dy = self.x[a:b].double(), self.dy[a:b].double()
            f = ref.forward(x, *w)
            yield e, slice(a, b), f, ref.backward(x, *w, dy, f)

    def check(self, ep, backward=True):
        torch.cuda.synchronize()
        assert ep.ep_device_error() == 0
        for e, s, f, r in self.experts():
            if s.stop > s.start:
                for k in ("g", "u", "h", "y"):
                    ref.check(self.o[k][s], f[k], f["tol_" + k], f"{k} of expert {e}")
            if not backward:
                continue
            if s.stop > s.start:
                for k in ("d_g", "d_u", "d_rows"):
                    ref.check(self.o[k][s], r[k], r["tol_" + k], f"{k} of expert {e}")
            for k in ("d_w_gate", "d_w_up", "d_w_down"):
                ref.check(self.o[k][e], r[k], r["tol_" + k], f"{k} of expert {e}")
        outside = list(range(self.bounds[0])) + list(range(self.bounds[-1], self.cfg.rows))
        for k in ("g", "u", "h", "y") + (("d_g", "d_u", "d_rows") if backward else ()):
            assert (self.o[k][outside] == 7.0).all(), f"{k}: a row of no expert was written"


CASES = [
    ([1], 64, 64, 0, 0),                          # one token, one expert, one stage
    ([8], 8, 8, 0, 0),                            # the narrowest block
    ([128], 256, 256, 0, 0),                      # a full tile
    ([3, 0, 1], 72, 40, 2, 5),                    # widths inside one box, rows of no expert around
    ([128, 1, 127, 129], 264, 200, 0, 3),         # tiles that end at, before and after 128 rows
    ([15, 16, 17, 96, 97, 0, 64, 65], 520, 392, 1, 0),
    ([255, 256, 257, 513], 320, 1032, 0, 0),      # several row tiles, ragged column tiles
    ([0, 0, 300], 1000, 360, 0, 0),               # leading experts without rows
    ([700, 0, 11], 2056, 136, 7, 130),            # long contraction, one wide and one narrow expert
    ([2] * 200, 128, 64, 0, 0),                   # more experts than SMs
    ([513, 576, 577, 639, 640, 641], 1536, 1544, 0, 1),  # CTA pairs: last tiles of 1 to 129 rows
]


@pytest.mark.parametrize("counts,H,I,before,after", CASES)
def test_forward_and_backward(ep, counts, H, I, before, after):
    b = Block(ep, counts, H, I, before, after, seed=len(counts) + H)
    b.forward(ep)
    b.backward(ep)
    b.check(ep)


@pytest.mark.parametrize("rows,E,H,I", [(6000, 3, 1024, 768), (9000, 40, 512, 264), (40, 64, 768, 512), (1, 1, 7168, 2048)])
def test_larger_shapes(ep, rows, E, H, I):
    gen = torch.Generator().manual_seed(rows)
    cut = torch.sort(torch.randint(0, rows + 1, (E - 1,), generator=gen)).values.tolist()
    counts = [b - a for a, b in zip([0] + cut, cut + [rows])]
    b = Block(ep, counts, H, I, seed=rows)
    b.forward(ep)
    b.backward(ep)
    b.check(ep)


def test_forward_without_saved_halves_is_the_same(ep):
    b = Block(ep, [5, 200, 33], 264, 136)
    b.forward(ep)
    h, y = b.o["h"].clone(), b.o["y"].clone()
    for k in ("h", "y", "g", "u"):
        b.o[k].fill_(7.0)
    b.forward(ep, save=False)
    assert torch.equal(b.o["h"], h) and torch.equal(b.o["y"], y)
    assert (b.o["g"] == 7.0).all() and (b.o["u"] == 7.0).all()


@pytest.mark.parametrize("want", [("d_rows",), ("d_w_down",), ("d_w_up", "d_w_gate"), ()])
def test_backward_writes_what_is_asked_for(ep, want):
    b = Block(ep, [40, 0, 90], 136, 72)
    b.forward(ep)
    b.backward(ep)
    all_of = {k: t.clone() for k, t in b.o.items()}
    names = ("d_rows", "d_w_gate", "d_w_up", "d_w_down")
    for k in names:
        b.o[k].fill_(7.0)
    b.backward(ep, want=want)
    for k in names:
        assert torch.equal(b.o[k], all_of[k]) if k in want else bool((b.o[k] == 7.0).all()), k


def test_repeated_calls_give_the_same_bits(ep):
    b = Block(ep, [300, 2, 77], 520, 264)
    b.forward(ep)
    b.backward(ep)
    first = {k: t.clone() for k, t in b.o.items()}
    b.forward(ep)
    b.backward(ep)
    assert all(torch.equal(first[k].view(torch.int16), b.o[k].view(torch.int16)) for k in first)


def test_nan_rows_stay_with_their_expert(ep):
    """Rows next to an expert's in the buffer, another expert's or nobody's, may hold NaN or infinities."""
    b = Block(ep, [70, 90, 5, 130], 136, 200, before=3, after=4)
    clean = Block(ep, [70, 90, 5, 130], 136, 200, before=3, after=4)
    for t in (b.x, b.dy):
        t[:3] = float("nan")
        t[3 + 70:3 + 160] = float("nan")  # expert 1
        t[-4:] = float("inf")
    for c in (b, clean):
        c.forward(ep)
        c.backward(ep)
    keep = list(range(3, 73)) + list(range(163, 298))
    for k in ("g", "u", "h", "y", "d_g", "d_u", "d_rows"):
        assert torch.equal(b.o[k][keep], clean.o[k][keep]), k
    for k in ("d_w_gate", "d_w_up", "d_w_down"):
        for e in (0, 2, 3):
            assert torch.equal(b.o[k][e], clean.o[k][e]), (k, e)
        assert torch.isnan(b.o[k][1]).all()


def test_large_gates_saturate(ep):
    """exp(-g) overflows for g below -88: silu goes to 0 there and to g at the other end."""
    b = Block(ep, [50], 64, 64, scale=60.0)
    b.forward(ep)
    b.backward(ep)
    assert (b.o["g"].float().abs().max() > 90).item()
    b.check(ep)


def test_part_of_the_experts(ep):
    """A rank's share: expert_offset + e0 and the weights from e0 on, over the whole row buffer."""
    b = Block(ep, [40, 7, 0, 150, 3, 20], 136, 72)
    whole = Block(ep, [40, 7, 0, 150, 3, 20], 136, 72)
    whole.forward(ep)
    whole.backward(ep)
    cfg = ep.EpFfnConfig.make(rows=b.cfg.rows, H=136, I=72, E=3)
    part = [w[2:5] for w in b.w]
    o, off = b.o, b.offset[2:6]
    ep.ep_expert_ffn(cfg, b.x, off, *part, o["h"], o["y"], g=o["g"], u=o["u"])
    ep.ep_expert_ffn_backward(cfg, b.x, off, *part, o["g"], o["u"], o["h"], b.dy, o["d_g"], o["d_u"], o["d_rows"],
                              o["d_w_gate"][2:5], o["d_w_up"][2:5], o["d_w_down"][2:5])
    inside = slice(47, 200)
    for k in ("g", "u", "h", "y", "d_g", "d_u", "d_rows"):
        assert torch.equal(o[k][inside], whole.o[k][inside]), k
        assert (o[k][:47] == 7.0).all() and (o[k][200:] == 7.0).all(), k
    for k in ("d_w_gate", "d_w_up", "d_w_down"):
        assert torch.equal(o[k][2:5], whole.o[k][2:5]), k
        assert (o[k][:2] == 7.0).all() and (o[k][5:] == 7.0).all(), k


def test_offsets_outside_the_buffer_are_clamped(ep):
    b = Block(ep, [30, 30, 30], 72, 72)
    b.forward(ep)
    y = b.o["y"].clone()
    b.o["y"].fill_(7.0)
    b.offset.copy_(torch.tensor([-5, 30, 60, 1000], dtype=torch.int32))
    b.forward(ep)
    assert torch.equal(b.o["y"], y)
    # decreasing bounds own nothing
    b.o["y"].fill_(7.0)
    b.offset.copy_(torch.tensor([90, 60, 30, 0], dtype=torch.int32))
    b.forward(ep)
    torch.cuda.synchronize()
    assert (b.o["y"] == 7.0).all() and ep.ep_device_error() == 0


def test_saved_halves_in_bfloat16_storage(ep):
    """g and u may be bfloat16 tensors, as storage: the bits are the same."""
    b, c = (Block(ep, [5, 70], 136, 72) for _ in range(2))
    for k in ("g", "u"):
        c.o[k] = torch.empty_like(c.o["h"])
    for t in (b, c):
        t.forward(ep)
        t.backward(ep)
    for k in b.o:
        assert torch.equal(b.o[k].view(torch.int16), c.o[k].view(torch.int16)), k


def test_no_rows(ep):
    b = Block(ep, [0, 0], 64, 64)
    b.forward(ep)
    b.backward(ep)
    for k in ("d_w_gate", "d_w_up", "d_w_down"):
        assert (b.o[k] == 0).all()


def test_other_stream_and_graph(ep):
    """The call runs on the stream it is given, and captures into a graph that replays on new contents."""
    b = Block(ep, [60, 3, 140], 264, 136)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    b.forward(ep, stream=s)
    b.backward(ep, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    b.check(ep)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.forward(ep)
        b.backward(ep)
    other = Block(ep, [100, 90, 13], 264, 136, seed=5)
    b.x.copy_(other.x)
    b.dy.copy_(other.dy)
    b.offset.copy_(other.offset)
    b.bounds = other.bounds
    graph.replay()
    b.check(ep)


def test_gradients_against_differences(ep):
    """Along a direction v, (L(a + eps v) - L(a - eps v)) / 2 eps in 64 bits, L = <y, dy>, is what the kernels'
    gradients give, up to those gradients' bounds and the differences' own error of order eps^2."""
    b = Block(ep, [37], 72, 56, seed=3)
    b.forward(ep)
    b.backward(ep)
    (_, s, f, r), = b.experts()
    args = [b.x.double()] + [w[0].double() for w in b.w]
    dy = b.dy.double()
    gen = torch.Generator(device="cuda").manual_seed(11)
    loss = lambda a: (ref.forward(*a)["y"] * dy).sum().item()  # noqa: E731
    for i, k in enumerate(("d_rows", "d_w_gate", "d_w_up", "d_w_down")):
        v = torch.randn(args[i].shape, generator=gen, device="cuda", dtype=torch.float64)
        at = lambda eps: loss([a + eps * v if j == i else a for j, a in enumerate(args)])  # noqa: E731
        d1, d2 = ((at(e) - at(-e)) / (2 * e) for e in (1e-4, 5e-5))
        exact = (4 * d2 - d1) / 3
        got = b.o[k].double().reshape(v.shape)
        bound = (r["tol_" + k] * v.abs()).sum().item() + 1e-6 * abs(exact) + 2 * abs(d1 - d2)
        assert abs((got * v).sum().item() - exact) <= bound, k


@pytest.mark.parametrize("counts,H,I,before,after", [
    ([1], 8, 8, 0, 0), ([1, 0, 2, 0, 0, 1], 72, 40, 1, 2), ([16], 264, 200, 0, 0), ([9, 7], 1000, 360, 0, 0),
    ([1] * 7 + [0] * 25, 4096, 1024, 0, 0), ([0] * 9 + [33] + [0] * 10, 520, 136, 0, 3), ([3] * 170, 128, 64, 0, 0),
])
def test_few_rows(ep, counts, H, I, before, after):
    """Forward calls with few rows an expert, saved halves not wanted: more rows than one pass takes,
    experts without rows, widths that end inside a stage."""
    b = Block(ep, counts, H, I, before, after, seed=H)
    b.forward(ep, save=False)
    torch.cuda.synchronize()
    assert ep.ep_device_error() == 0
    for e, s, f, _ in b.experts():
        if s.stop > s.start:
            ref.check(b.o["h"][s], f["h"], f["tol_h"], f"h of expert {e}")
            ref.check(b.o["y"][s], f["y"], f["tol_y"], f"y of expert {e}")
    outside = list(range(b.bounds[0])) + list(range(b.bounds[-1], b.cfg.rows))
    assert (b.o["y"][outside] == 7.0).all() and (b.o["h"][outside] == 7.0).all()


def test_few_rows_with_nan_neighbours(ep):
    b, clean = (Block(ep, [2, 0, 3, 1], 136, 72, before=1, after=1) for _ in range(2))
    b.x[0] = float("nan")
    b.x[1 + 2:1 + 4] = float("nan")  # two of expert 2's three rows
    b.x[-1] = float("inf")
    for c in (b, clean):
        c.forward(ep, save=False)
    keep = [1, 2, 5, 6]
    assert torch.equal(b.o["y"][keep], clean.o["y"][keep]) and torch.isnan(b.o["y"][3:5]).all()
