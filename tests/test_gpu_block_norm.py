"""ep_block_norm and ep_block_norm_backward against the same in 64 bits.

Bounds count roundings. A value that is stored as bf16 is off by at most 2^-8 of itself, as float 2^-24.
Before that everything is fp32: a mean square adds up H values in chains of at most 64 steps and a tree
of ten (74 2^-24 of it, half of that in its root), the root itself is within 2^-22, a gate's sigmoid within
2^-19 for |gate| <= 8 (the argument of its exponential is rounded), sums over rows are chains of fewer than
200 steps. A result is a sum of terms each of which has at most three factors of r, one of the gate and eight
more roundings: 3 (37 2^-24 + 2^-22) + 2^-19 + 8 2^-24 + 200 2^-24 < 2^-15 of the terms' magnitudes."""
from __future__ import annotations

import itertools

import pytest
import torch

from gpu_harness import require_cuda

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
E32 = 2.0**-15
KINDS = ("none", "channel", "token", "element")


@pytest.fixture(scope="module")
def ep():
    require_cuda()
    import combine_router_softmax_gb300 as m

    return m


def step(dtype):
    return 2.0**-8 if dtype is BF16 else 2.0**-24


class Problem:
    def __init__(self, ep, T, H, post=True, gate="none", sigmoid=False, f32=False, scale=1.0, offset=0.0, eps=1e-6, block=True,
                 next=True, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        row = F32 if f32 else BF16
        normal = lambda *s, dtype=BF16, scale=1.0: (torch.randn(s, generator=gen, device="cuda") * scale).to(dtype)  # noqa: E731
        self.ep, self.T, self.H, self.kind, self.sigmoid, self.row = ep, T, H, gate, sigmoid, row
        self.scale, self.offset, self.eps = scale, offset, eps
        self.x = normal(T, H, dtype=row, scale=2.0)
        self.y = normal(T, H) if block else None
        self.w_post = normal(H, scale=0.5) if post and block else None
        self.w_next = normal(H, scale=0.5) if next else None
        shape = {"none": None, "channel": (H,), "token": (T,), "element": (T, H)}[gate]
        self.gate = None if shape is None else normal(*shape, dtype=F32 if gate == "token" else BF16).clamp_(-8, 8)
        self.d_out = normal(T, H, dtype=row)
        self.d_n = normal(T, H) if next else None
        self.cfg = ep.EpNormConfig.make(T=T, H=H, gate=KINDS.index(gate), gate_sigmoid=int(sigmoid), residual_f32=int(f32),
                                        eps=eps, scale=scale, weight_offset=offset)

    def empty(self, *shape, dtype=BF16):
        return torch.full(shape, float("nan"), dtype=dtype, device="cuda")

    def forward(self, **over):
        T, H = self.T, self.H
        o = dict(out=self.empty(T, H, dtype=self.row) if self.y is not None else None,
                 n=self.empty(T, H) if self.w_next is not None else None,
                 rstd_post=self.empty(T, dtype=F32) if self.w_post is not None else None,
                 rstd_next=self.empty(T, dtype=F32) if self.w_next is not None else None)
        o.update(over)
        self.ep.ep_block_norm(self.cfg, self.x, self.y, self.w_post, self.gate, self.w_next, o["out"], o["n"], o["rstd_post"],
                              o["rstd_next"])
        return o

    def backward(self, f, d_out="given", **over):
        T, H = self.T, self.H
        o = dict(d_x=self.empty(T, H, dtype=self.row), d_y=self.empty(T, H) if self.y is not None else None,
                 d_w_post=self.empty(H, dtype=F32) if self.w_post is not None else None,
                 d_w_next=self.empty(H, dtype=F32) if self.w_next is not None else None,
                 d_gate=None if self.gate is None else self.empty(*self.gate.shape, dtype=BF16 if self.kind == "element" else F32))
        o.update(over)
        ws = torch.empty((self.ep.ep_block_norm_workspace_size(self.cfg),), dtype=torch.uint8, device="cuda")
        self.ep.ep_block_norm_backward(self.cfg, self.x, self.y, self.w_post, self.gate, self.w_next, f["rstd_post"], f["rstd_next"],
                                       self.d_out if d_out == "given" else d_out, self.d_n, o["d_x"], o["d_y"], o["d_w_post"],
                                       o["d_gate"], o["d_w_next"], ws)
        return o

    def reference(self, d_out="given"):
        """{name: (value, bound)}, by the formulas in 64 bits."""
        d = lambda t: None if t is None else t.double()  # noqa: E731
        x, y, wp, wn, g = (d(t) for t in (self.x, self.y, self.w_post, self.w_next, self.gate))
        r, s = {}, self.scale
        z = torch.zeros_like(x)
        f = slope = torch.ones((), dtype=torch.float64, device="cuda")
        if y is not None:
            z = y
            if wp is not None:
                wp = wp + self.offset
                ry = (y.square().mean(-1, keepdim=True) + self.eps).rsqrt()
                z = wp * y * ry
                r["rstd_post"] = ry[:, 0], E32 * ry[:, 0]
            if g is not None:
                g = g[:, None] if self.kind == "token" else g
                f = torch.sigmoid(g) if self.sigmoid else g
                slope = f * (1 - f) if self.sigmoid else slope
        out = x + s * f * z
        mag = x.abs() + (s * f * z).abs()  # of the terms
        if y is not None:
            r["out"] = out, step(self.row) * out.abs() + E32 * mag
        if wn is not None:
            wn = wn + self.offset
            rr = (out.square().mean(-1, keepdim=True) + self.eps).rsqrt()
            # out's error also reaches r: relative to the row's norm, at most that of the terms
            off_r = E32 * (1 + mag.norm(dim=-1, keepdim=True) / out.norm(dim=-1, keepdim=True).clamp(min=1e-30))
            r["rstd_next"] = rr[:, 0], (off_r * rr)[:, 0]
            n = wn * out * rr
            r["n"] = n, 2.0**-8 * n.abs() + (wn * rr).abs() * E32 * mag + off_r * n.abs()
        do = torch.zeros_like(x) if d_out is None else self.d_out.double()
        D, magD = do, do.abs()
        if wn is not None:
            gn = wn * self.d_n.double()
            D = do + rr * gn - out * rr**3 * (gn * out).mean(-1, keepdim=True)
            magD = do.abs() + (rr * gn).abs() + mag * rr**3 * (gn.abs() * mag).mean(-1, keepdim=True)
            magD = magD * (off_r / E32)
            r["d_w_next"] = ((self.d_n.double() * out * rr).sum(0),
                             (E32 * (off_r / E32) * self.d_n.double().abs() * mag * rr).sum(0))
        r["d_x"] = D, step(self.row) * D.abs() + E32 * magD
        if y is None:
            return r
        e, mag_e = s * f * D, (s * f).abs() * magD
        if wp is not None:
            ew = wp * e
            dy = ry * ew - y * ry**3 * (ew * y).mean(-1, keepdim=True)
            mag_dy = ry * wp.abs() * mag_e + y.abs() * ry**3 * (wp.abs() * mag_e * y.abs()).mean(-1, keepdim=True)
            r["d_w_post"] = (e * y * ry).sum(0), E32 * (mag_e * y.abs() * ry).sum(0)
        else:
            dy, mag_dy = e, mag_e
        r["d_y"] = dy, 2.0**-8 * dy.abs() + E32 * mag_dy
        if g is not None:
            dg, mag_g = s * D * z * slope, (s * z * slope).abs() * magD
            if self.kind == "element":
                r["d_gate"] = dg, 2.0**-8 * dg.abs() + E32 * mag_g
            else:
                axis = 0 if self.kind == "channel" else 1
                r["d_gate"] = dg.sum(axis), E32 * mag_g.sum(axis)
        return r


def check(got, want):
    for name, (value, tol) in want.items():
        t = got[name].double()
        assert torch.isfinite(t).all(), f"{name}: not finite"
        off = (t - value).abs() - tol - 1e-30
        assert off.max().item() <= 0, f"{name}: {int((off > 0).sum())} of {off.numel()} beyond their bound, worst by {off.max().item():g}"


# every path of the row's length (a warp with 1, 2, 4 vectors a lane, a CTA with 1 and 2 a thread), whole and ragged
@pytest.mark.parametrize("T,H", [(1, 8), (9, 64), (33, 256), (7, 264), (20, 512), (17, 1000), (300, 1024), (5, 1032), (40, 4096),
                                 (3, 4104), (13, 7168), (2, 8200), (4, 16384)])
@pytest.mark.parametrize("f32", [False, True])
def test_against_64_bits(ep, T, H, f32):
    p = Problem(ep, T, H, f32=f32, gate="channel", sigmoid=True, scale=0.7, offset=1.0, seed=H)
    f = p.forward()
    check({**f, **p.backward(f)}, p.reference())


@pytest.mark.parametrize("gate,sigmoid,post,next", list(itertools.product(KINDS, (False, True), (False, True), (False, True))))
@pytest.mark.parametrize("H", [200, 1400])
def test_every_form(ep, gate, sigmoid, post, next, H):
    p = Problem(ep, 37, H, gate=gate, sigmoid=sigmoid, post=post, next=next, f32=sigmoid != post, scale=-0.3, seed=3)
    f = p.forward()
    check({**f, **p.backward(f)}, p.reference())


@pytest.mark.parametrize("H", [96, 2048])
@pytest.mark.parametrize("f32", [False, True])
def test_norm_alone(ep, H, f32):
    """Before the first block: no y."""
    p = Problem(ep, 50, H, block=False, f32=f32, seed=4)
    f = p.forward()
    check({**f, **p.backward(f)}, p.reference())
    if not f32:  # n may be x
        n = p.x.clone()
        p2 = Problem(ep, 50, H, block=False, f32=f32, seed=4)
        p2.x = n
        p2.forward(n=n)
        assert torch.equal(n, f["n"])


def test_without_d_out(ep):
    p = Problem(ep, 21, 1200, gate="element", seed=5)
    f = p.forward()
    check(p.backward(f, d_out=None), {k: v for k, v in p.reference(d_out=None).items() if k.startswith("d_")})


@pytest.mark.parametrize("T", [1000, 2500])
@pytest.mark.parametrize("H", [128, 1536])
def test_many_rows(ep, T, H):
    """More rows than CTAs: every one walks several, and partial sums are joined."""
    p = Problem(ep, T, H, gate="channel", seed=6)
    f = p.forward()
    a = p.backward(f)
    check({**f, **a}, p.reference())
    b = p.backward(f)
    assert all(torch.equal(a[k], b[k]) for k in a)


@pytest.mark.parametrize("T,H", [(1216, 2056), (1300, 4104), (1217, 8200), (2500, 7168)])
@pytest.mark.parametrize("gate", KINDS)
@pytest.mark.parametrize("f32", [False, True])
def test_many_rows_of_a_normed_block(ep, T, H, gate, f32):
    """Rows whose first sum is made with the second one of the row before; then in place."""
    p = Problem(ep, T, H, gate=gate, sigmoid=gate != "channel", f32=f32, seed=T)
    f = p.forward()
    check({**f, **p.backward(f)}, p.reference())
    q = Problem(ep, T, H, gate=gate, sigmoid=gate != "channel", f32=f32, seed=T)
    h = q.forward(out=q.x, n=q.y)
    assert all(torch.equal(h[k], f[k]) for k in f)


@pytest.mark.parametrize("post,gate", [(True, "none"), (True, "channel"), (True, "element"), (False, "token"), (False, "element")])
@pytest.mark.parametrize("H", [4096, 4104, 5120, 5128])
@pytest.mark.parametrize("f32", [False, True])
def test_rows_of_two_ctas_an_sm(ep, post, gate, H, f32):
    p = Problem(ep, 620, H, post=post, gate=gate, f32=f32, seed=H)
    f = p.forward()
    check({**f, **p.backward(f)}, p.reference())


@pytest.mark.parametrize("T,H", [(5, 72), (400, 1000), (300, 7168)])
def test_float_stream_on_16_bytes(ep, T, H):
    """Aligned to 16 bytes, as is asked for, and not to 32."""
    p = Problem(ep, T, H, gate="channel", f32=True, seed=9)
    f = p.forward()
    a = p.backward(f)
    off = lambda: torch.full((T * H + 4,), float("nan"), device="cuda")[4:].view(T, H)  # noqa: E731
    assert off().data_ptr() % 32 == 16
    for name in ("x", "d_out"):
        setattr(p, name, off().copy_(getattr(p, name)))
    g = p.forward(out=off())
    b = p.backward(g, d_x=off())
    assert all(torch.equal(g[k], f[k]) for k in f) and all(torch.equal(b[k], a[k]) for k in a)


@pytest.mark.parametrize("T", [152, 153, 304, 305, 608, 609, 1217])
@pytest.mark.parametrize("H", [264, 1000, 2048, 4096])
def test_as_many_rows_as_run_at_once(ep, T, H):
    """And one more: a CTA for each of them, or rows in turns."""
    p = Problem(ep, T, H, gate="channel", f32=T % 2 == 0, seed=T)
    f = p.forward()
    r = p.reference()
    check(f, {k: r[k] for k in f})


@pytest.mark.parametrize("T", [300, 1300])
@pytest.mark.parametrize("H", [1000, 4096, 7168])
def test_joined_without_a_next_norm(ep, T, H):
    p = Problem(ep, T, H, gate="token", sigmoid=True, f32=True, next=False, seed=H)
    f = p.forward(rstd_post=None)
    assert torch.equal(f["out"], p.forward()["out"])
    check({"out": f["out"]}, {"out": p.reference()["out"]})


def test_the_most_rows(ep):
    """2^31 - 1 rows, of 8: the first and the last ones as in a call of their own."""
    T, H = 2**31 - 1, 8
    if torch.cuda.mem_get_info()[0] < 90 * 2**30:
        pytest.skip("not enough memory")
    x, w = torch.ones((T, H), dtype=BF16, device="cuda"), torch.full((H,), 0.5, dtype=BF16, device="cuda")
    rows = torch.randn((2, 1000, H), device="cuda", generator=torch.Generator(device="cuda").manual_seed(5)).to(BF16)
    x[:1000], x[-1000:] = rows[0], rows[1]
    n = torch.full((T, H), float("nan"), dtype=BF16, device="cuda")
    ep.ep_block_norm(ep.EpNormConfig.make(T=T, H=H), x, w_next=w, n=n)
    want = torch.empty_like(rows)
    ep.ep_block_norm(ep.EpNormConfig.make(T=2000, H=H), rows.view(2000, H), w_next=w, n=want.view(2000, H))
    assert torch.equal(n[:1000], want[0]) and torch.equal(n[-1000:], want[1])
    assert torch.equal(n[T // 2 : T // 2 + 1000], torch.full((1000, H), 0.5, dtype=BF16, device="cuda"))


def test_in_place(ep):
    for H in (256, 2992):
        p = Problem(ep, 65, H, gate="token", sigmoid=True, seed=7)
        f = p.forward()
        g = p.backward(f)
        q = Problem(ep, 65, H, gate="token", sigmoid=True, seed=7)
        x, y = q.x.clone(), q.y.clone()
        q.x, q.y = x, y
        h = q.forward(out=x, n=y)
        assert torch.equal(x, f["out"]) and torch.equal(y, f["n"])
        q = Problem(ep, 65, H, gate="token", sigmoid=True, seed=7)
        k = q.backward(f, d_x=q.d_out, d_y=q.d_n)
        assert all(torch.equal(k[n], g[n]) for n in g)
        assert torch.equal(h["rstd_next"], f["rstd_next"])


def test_rows_of_zeros_and_large_ones(ep):
    """eps alone keeps a row of zeros finite; values of 1e15 square within fp32's range."""
    p = Problem(ep, 4, 512, gate="channel", eps=1e-5, seed=8)
    p.x[0] = 0
    p.y[0] = 0
    p.y[1] = 0
    p.x[2] *= 1e15
    p.y[3] *= 1e15
    f = p.forward()
    want = p.reference()
    check({**f, **p.backward(f)}, want)
    assert (f["n"][0] == 0).all()


def test_nan_stays_in_its_row(ep):
    p = Problem(ep, 12, 640, gate="element", seed=9)
    f0 = p.forward()
    b0 = p.backward(f0)
    p.y[5, 17] = float("nan")
    f = p.forward()
    b = p.backward(f)
    keep = torch.arange(12, device="cuda") != 5
    for n, a, c in (("out", f0, f), ("n", f0, f), ("d_x", b0, b), ("d_y", b0, b), ("d_gate", b0, b)):
        assert torch.equal(a[n][keep], c[n][keep]), n
    assert torch.isnan(f["n"][5]).all()


def test_no_rows(ep):
    p = Problem(ep, 0, 64, gate="channel")
    f = p.forward()
    b = p.backward(f)
    for n in ("d_w_post", "d_w_next", "d_gate"):
        assert (b[n] == 0).all(), n


@pytest.mark.parametrize("gate", KINDS)
def test_against_differences(ep, gate):
    """The gradients along random directions against central differences of the 64-bit forward pass: truncation
    is of order h^2 = 1e-8 relative, the gradients' own roundings 2^-8 each, independent, so small against
    4 2^-8 of the directions' length times the gradients' norm."""
    p = Problem(ep, 6, 264, gate=gate, sigmoid=True, scale=0.5, seed=10)
    f = p.forward()
    b = p.backward(f)
    names = [n for n in ("x", "y", "w_post", "w_next", "gate") if getattr(p, n) is not None]
    base = {n: getattr(p, n).double() for n in names}
    gen = torch.Generator(device="cuda").manual_seed(11)
    for n in names:
        direction = torch.randn(base[n].shape, generator=gen, device="cuda", dtype=torch.float64)

        def loss(h):
            q = Problem.__new__(Problem)
            q.__dict__.update(p.__dict__)
            setattr(q, n, base[n] + h * direction)
            r = q.reference()
            return (r["out"][0] * p.d_out.double()).sum() + (r["n"][0] * p.d_n.double()).sum()

        slope = (loss(1e-4) - loss(-1e-4)) / 2e-4
        grad = b["d_" + n].double()
        assert abs((grad * direction).sum() - slope) <= 4 * 2.0**-8 * grad.norm() * direction.norm(), n


def test_captured(ep):
    """Forward and backward in a graph, replayed on new inputs."""
    p = Problem(ep, 70, 2048, gate="channel", seed=12)
    f, o = p.forward(), {}
    ws = torch.empty((ep.ep_block_norm_workspace_size(p.cfg),), dtype=torch.uint8, device="cuda")
    o = p.backward(f)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ep.ep_block_norm(p.cfg, p.x, p.y, p.w_post, p.gate, p.w_next, f["out"], f["n"], f["rstd_post"], f["rstd_next"])
        ep.ep_block_norm_backward(p.cfg, p.x, p.y, p.w_post, p.gate, p.w_next, f["rstd_post"], f["rstd_next"], p.d_out, p.d_n,
                                  o["d_x"], o["d_y"], o["d_w_post"], o["d_gate"], o["d_w_next"], ws)
    q = Problem(ep, 70, 2048, gate="channel", seed=13)
    for n in ("x", "y", "w_post", "w_next", "gate", "d_out", "d_n"):
        getattr(p, n).copy_(getattr(q, n))
    g.replay()
    torch.cuda.synchronize()
    check({**f, **o}, q.reference())


def test_on_another_stream(ep):
    p = Problem(ep, 128, 1024, seed=14)
    want = p.forward()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = p.forward()
    s.synchronize()
    assert all(torch.equal(got[n], want[n]) for n in ("out", "n"))
