"""ep_balance and ep_balance_backward against the same in 64 bits.

Bounds count roundings. An exponential is off by 2^-21 and by its argument's rounding, |l - top| 1.5 2^-24; the
sums of a row are trees of at most 37 steps, those over rows chains of fewer than 2^10 (2^-14 of the terms'
magnitudes, all of one sign for the probabilities); quotients and products add a few 2^-24."""
from __future__ import annotations

import pytest
import torch

from gpu_harness import require_cuda

pytestmark = pytest.mark.gpu
F32, I32 = torch.float32, torch.int32


@pytest.fixture(scope="module")
def ep():
    require_cuda()
    import combine_router_softmax_gb300 as m

    return m


class Problem:
    def __init__(self, ep, T, E, k, first=None, length=None, seed=0, size=2.0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.ep, self.T, self.E, self.k = ep, T, E, k
        self.S = 1 if first is None else len(first) - 1
        self.cfg = ep.EpConfig.make(T=T, H=8, E=E, R=1, k=k)
        self.logits = torch.randn((T, E), generator=gen, device="cuda") * size
        self.idx = torch.topk(self.logits, k, dim=-1)[1].to(I32)
        self.first = None if first is None else torch.tensor(first, dtype=I32, device="cuda")
        self.length = None if length is None else torch.tensor(length, dtype=I32, device="cuda")
        self.d_loss = torch.randn((self.S, 2), generator=gen, device="cuda")
        self.d_in = torch.randn((T, E), generator=gen, device="cuda") * 1e-3

    def forward(self):
        o = dict(count=torch.full((self.S, self.E), -7, dtype=I32, device="cuda"))
        for n, w in (("load", self.E), ("prob", self.E), ("loss", 2)):
            o[n] = torch.full((self.S, w), float("nan"), device="cuda")
        ws = torch.empty((self.ep.ep_balance_workspace_size(self.cfg, self.S),), dtype=torch.uint8, device="cuda")
        ws.fill_(255)  # needs no initialisation: all NaN
        self.ep.ep_balance(self.cfg, self.logits, self.idx, self.first, self.length, o["count"], o["load"], o["prob"], o["loss"], ws)
        return o

    def backward(self, load, d_in=True, out=None):
        out = torch.full((self.T, self.E), float("nan"), device="cuda") if out is None else out
        self.ep.ep_balance_backward(self.cfg, self.logits, self.first, self.length, load, self.d_loss, self.d_in if d_in else None, out)
        return out

    def rows(self, s):
        if self.first is None:
            return 0, self.T
        a, b = (min(max(int(self.first[s + i]), 0), self.T) for i in (0, 1))
        b = max(a, b)
        return a, b if self.length is None else min(b, a + max(int(self.length[s]), 0))

    def reference(self, load=None, d_in=True):
        r = {n: [] for n in ("count", "load", "prob", "loss", "tol_prob", "tol_loss")}
        d = self.d_in.double().clone() if d_in else torch.zeros((self.T, self.E), dtype=torch.float64, device="cuda")
        tol = 2.0**-23 * d.abs()
        for s in range(self.S):
            a, b = self.rows(s)
            n = max(b - a, 1)
            l = self.logits[a:b].double()
            dead = (l == -torch.inf).all(-1, keepdim=True)
            p = torch.where(dead, 0.0, torch.softmax(l, -1))
            lse = torch.where(dead, 0.0, torch.logsumexp(l, -1, keepdim=True))
            top = l.amax(-1, keepdim=True)
            # of a probability, relative: its exponential, and the sum that it is divided by
            far = torch.where(p > 0, (top - l).nan_to_num(0, 0, 0), 0.0)
            rel = 2.0**-20 + far * 2.0**-23 + (far * p).sum(-1, keepdim=True) * 2.0**-23
            chosen = self.idx[a:b].long()
            c = torch.bincount(chosen[(chosen >= 0) & (chosen < self.E)], minlength=self.E)
            f = c.double() / (self.k * n)
            prob = p.sum(0) / n
            tol_prob = ((p * rel).sum(0) + 2.0**-14 * p.sum(0)) / n
            off_lse = (2.0**-20 + 2.0**-22 * lse.abs() + 2.0**-22 * top.nan_to_num(0, 0, 0).abs())
            z = lse.square().sum() / n
            tol_z = ((2 * lse.abs() * off_lse).sum() + 2.0**-14 * lse.square().sum()) / n
            r["count"].append(c)
            r["load"].append(f)
            r["prob"].append(prob)
            r["tol_prob"].append(tol_prob)
            r["loss"].append(torch.stack([self.E * (f * prob).sum(), z]))
            r["tol_loss"].append(torch.stack([self.E * (f * (tol_prob + 2.0**-20 * prob)).sum(), tol_z]))
            w = f if load is None else load[s].double()
            c0, c1 = self.d_loss[s, 0].double() * self.E / n, 2 * self.d_loss[s, 1].double() / n
            mean = (w * p).sum(-1, keepdim=True)
            d[a:b] += p * (c0 * (w - mean) + c1 * lse)
            mag = c0.abs() * (w + mean) + (c1 * lse).abs()
            off = c0.abs() * ((w * p * rel).sum(-1, keepdim=True) + 2.0**-19 * (w + mean)) + c1.abs() * (off_lse + 2.0**-20 * lse.abs())
            tol[a:b] += p * (rel * mag + off) + 2.0**-23 * (p * mag)
        r = {n: torch.stack(v) for n, v in r.items()}
        r["d_logits"], r["tol_d_logits"] = d, 1.01 * tol
        return r


def check(p, o, r):
    assert torch.equal(o["count"].long(), r["count"])
    assert ((o["load"].double() - r["load"]).abs() <= 2.0**-22 * r["load"]).all()
    for n in ("prob", "loss", "d_logits"):
        if n in o:
            # what no float can hold is infinite: a row of the lowest value has a squared log-sum-exp of 1e77
            beyond = r[n].abs() > torch.finfo(F32).max
            assert torch.equal(o[n][beyond], r[n][beyond].float())
            off = ((o[n].double() - r[n]).abs() - r["tol_" + n] - 1e-30)[~beyond]
            assert off.max().item() <= 0, f"{n}: {int((off > 0).sum())} beyond their bound, worst by {off.max().item():g}"


def run(p, d_in=True):
    o = p.forward()
    o["d_logits"] = p.backward(o["load"], d_in)
    check(p, o, p.reference(o["load"], d_in))
    return o


# every number of logits a lane, whole and ragged, rows from one to several tiles
@pytest.mark.parametrize("E,k", [(1, 1), (5, 2), (32, 8), (33, 32), (100, 6), (128, 8), (200, 3), (256, 8), (257, 1), (1024, 32)])
@pytest.mark.parametrize("T", [1, 50, 1111])
def test_against_64_bits(ep, E, k, T):
    run(Problem(ep, T, E, k, seed=E + T), d_in=T != 50)


@pytest.mark.parametrize("E,k", [(3, 1), (37, 6), (150, 8), (203, 2), (511, 8), (1001, 4)])
def test_rows_on_no_boundary(ep, E, k):
    """Rows of no multiple of four logits, by tiles of many and with ends of sequences inside, gradients added in place."""
    run(Problem(ep, 20001, E, k, first=[0, 7000, 7013, 20001], seed=E))


@pytest.mark.parametrize("T,first,length", [
    (100, [0, 100], None),
    (100, [0, 0, 0, 37, 38, 38, 100, 100], None),           # empty ones, one of a single row
    (5000, [0, 3, 700, 701, 2600, 5000], None),
    (1000, [10, 200, 900], None),                            # rows before the first and behind the last
    (700, [0, 100, 200, 300, 400, 500, 600, 700], [100, 0, 1, 57, 99, 100, 30]),  # padded
    (64, list(range(65)), None),                             # a sequence a row
    (300, [0, 150, 300], [200, 1000]),                       # longer than the place they have
    (300, [-5, 100, 5000], [20, -3]),                        # out of range: clamped
])
def test_sequences(ep, T, first, length):
    p = Problem(ep, T, 60, 4, first, length, seed=T)
    own = torch.zeros(T, dtype=torch.bool)
    for s in range(p.S):
        own[slice(*p.rows(s))] = True
    p.logits[~own.cuda()] = float("nan")  # rows of no sequence are not read
    o = run(p)
    assert torch.equal(o["d_logits"][~own.cuda()], p.d_in[~own.cuda()])
    for s in range(p.S):
        a, b = p.rows(s)
        if a == b:
            assert not o["count"][s].any() and not o["load"][s].any() and not o["prob"][s].any() and not o["loss"][s].any()


def test_sequences_are_separate(ep):
    """Every sequence as it would be alone, whatever tiles its rows fall into."""
    first = [0, 313, 1900, 1901, 4000]
    p = Problem(ep, 4000, 128, 8, first, seed=1)
    o = p.forward()
    for s, (a, b) in enumerate(zip(first, first[1:])):
        q = Problem(ep, b - a, 128, 8)
        q.logits, q.idx = p.logits[a:b].contiguous(), p.idx[a:b].contiguous()
        w = q.forward()
        assert torch.equal(w["count"][0], o["count"][s])
        assert ((w["prob"][0] - o["prob"][s]).abs() <= 2.0**-14 * w["prob"][0]).all()


def test_masked_experts(ep):
    """-infinity: no probability and no gradient; a row of nothing else has none at all."""
    p = Problem(ep, 200, 40, 2, [0, 90, 200], seed=2)
    p.logits[:, 7] = -torch.inf
    p.logits[30:60] = -torch.inf
    p.logits[100, 1:] = -torch.inf
    p.logits[101] = torch.finfo(F32).min  # a mask of the type's lowest value
    o = run(p)
    # row 101 is even over all 40, expert 7 among them: 1/40 of one of the 110 rows
    assert o["prob"][0, 7] == 0 and abs(o["prob"][1, 7].item() * 110 * 40 - 1) < 2.0**-20
    others = torch.arange(200, device="cuda") != 101
    assert torch.equal(o["d_logits"][others, 7], p.d_in[others, 7]) and torch.equal(o["d_logits"][30:60], p.d_in[30:60])


def test_large_logits(ep):
    run(Problem(ep, 333, 77, 5, seed=3, size=60.0))


def test_ids_outside_are_not_counted(ep):
    p = Problem(ep, 130, 16, 3, seed=4)
    p.idx[::3, 1] = -1
    p.idx[::4, 2] = 16
    p.idx[5] = 9  # the same id three times counts three times
    run(p)


def test_nan_stays_in_its_sequence(ep):
    p = Problem(ep, 600, 64, 4, [0, 200, 400, 600], seed=5)
    want = p.forward()
    p.logits[300, 3] = float("nan")
    o = p.forward()
    for n in ("prob", "loss"):
        assert torch.equal(o[n][[0, 2]], want[n][[0, 2]]) and torch.isnan(o[n][1]).any()
    d = p.backward(want["load"])
    rows = torch.arange(600, device="cuda") != 300
    assert torch.isfinite(d[rows]).all()


def test_in_place_other_load_and_repeats(ep):
    p = Problem(ep, 3000, 96, 8, [0, 1500, 3000], seed=6)
    o = p.forward()
    again = p.forward()
    assert all(torch.equal(o[n], again[n]) for n in o)
    load = o["load"].mean(0, keepdim=True).expand(2, 96).contiguous()  # that of all processes, say
    r = p.reference(load)
    d = p.backward(load)
    check(p, {**o, "d_logits": d}, {**p.reference(), "d_logits": r["d_logits"], "tol_d_logits": r["tol_d_logits"]})
    buf = p.d_in.clone()
    p.backward(load, out=buf)  # d_in itself is still p.d_in
    q = p.d_in.clone()
    p.ep.ep_balance_backward(p.cfg, p.logits, p.first, p.length, load, p.d_loss, q, q)
    assert torch.equal(q, d) and torch.equal(buf, d)


def test_no_rows(ep):
    p = Problem(ep, 0, 12, 2)
    o = p.forward()
    assert not any(o[n].any() for n in o)
    p.backward(o["load"])


def test_against_differences(ep):
    """Along random directions, the losses in 64 bits with the choice of experts kept: h^2 = 1e-8 of truncation, and
    2^-14 of the gradient's magnitude for its own roundings (the bound of the tests above)."""
    p = Problem(ep, 64, 24, 3, [0, 20, 64], seed=7)
    o = p.forward()
    grad = p.backward(o["load"], d_in=False).double()
    base = p.logits.double()
    gen = torch.Generator(device="cuda").manual_seed(8)
    for _ in range(4):
        direction = torch.randn(base.shape, generator=gen, device="cuda", dtype=torch.float64)

        def loss(h):
            total = 0.0
            for s in range(2):
                a, b = p.rows(s)
                l = (base + h * direction)[a:b]
                prob, z = torch.softmax(l, -1).mean(0), torch.logsumexp(l, -1).square().mean()
                total = total + p.d_loss[s, 0].double() * 24 * (o["load"][s].double() * prob).sum() + p.d_loss[s, 1].double() * z
            return total

        slope = (loss(1e-4) - loss(-1e-4)) / 2e-4
        assert abs((grad * direction).sum() - slope) <= 2.0**-13 * grad.norm() * direction.norm()


def test_captured(ep):
    p = Problem(ep, 900, 64, 4, [0, 300, 900], seed=9)
    o = p.forward()
    d = p.backward(o["load"])
    ws = torch.empty((ep.ep_balance_workspace_size(p.cfg, 2),), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ep.ep_balance(p.cfg, p.logits, p.idx, p.first, None, o["count"], o["load"], o["prob"], o["loss"], ws)
        ep.ep_balance_backward(p.cfg, p.logits, p.first, None, o["load"], p.d_loss, p.d_in, d)
    q = Problem(ep, 900, 64, 4, [0, 450, 800], seed=10)
    for n in ("logits", "idx", "first", "d_loss", "d_in"):
        getattr(p, n).copy_(getattr(q, n))
    g.replay()
    torch.cuda.synchronize()
    check(q, {**o, "d_logits": d}, q.reference(o["load"]))


def test_after_the_router(ep):
    """The router's gradient and the losses', one after the other into one buffer."""
    T, E, k = 500, 64, 6
    p = Problem(ep, T, E, k, seed=11)
    w = torch.empty((T, k), device="cuda")
    ep.ep_route(p.cfg, p.logits, p.idx, w)
    d_w = torch.randn((T, k), device="cuda")
    ep.ep_route_backward(p.cfg, None, p.idx, w, d_w, p.d_in)
    router = p.d_in.clone()
    o = p.forward()
    ep.ep_balance_backward(p.cfg, p.logits, None, None, o["load"], p.d_loss, p.d_in, p.d_in)
    got = p.d_in.clone()
    p.d_in = router
    check(p, {**o, "d_logits": got}, p.reference(o["load"]))
