"""ep_block_norm and its gradients against automatic differentiation in 64 bits of the definition, and the longest rows in
numbers that are taken in turns.

Stored as bf16 a value is off by 2^-8 of itself at most, so a tensor by 2^-8 of its norm; before that all is fp32, within 2^-15 of the
magnitude of the terms that make a value up (as test_gpu_block_norm.py counts), of which there are a few here and none beyond
thirty times the tensor's rms: 2^-10 of it. Sums over 40 rows: of terms with signs, whose magnitudes add up to about sqrt(40)
times the sum's, 2^-15 sqrt(40) < 2^-12 of the norm."""
from __future__ import annotations

import itertools

import pytest
import torch

from gpu_harness import require_cuda
from test_gpu_block_norm import KINDS, Problem, check

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def ep():
    require_cuda()
    import combine_router_softmax_gb300 as m

    return m


def differentiate(p, use_out, use_n):
    v = {n: None if getattr(p, n) is None else getattr(p, n).double().requires_grad_() for n in ("x", "y", "w_post", "w_next", "gate")}

    def norm(rows, w):
        return (p.offset + w) * rows / torch.sqrt((rows * rows).mean(1, keepdim=True) + p.eps)

    out = v["x"]
    if v["y"] is not None:
        z = v["y"] if v["w_post"] is None else norm(v["y"], v["w_post"])
        if v["gate"] is not None:
            g = v["gate"].unsqueeze(1) if p.kind == "token" else v["gate"]
            z = z * (1 / (1 + torch.exp(-g)) if p.sigmoid else g)
        out = out + p.scale * z
    total = (out * p.d_out.double()).sum() if use_out else 0.0
    got = {}
    if v["w_next"] is not None:
        n = norm(out, v["w_next"])
        got["n"] = n.detach()
        total = total + (n * p.d_n.double()).sum() if use_n else total
    if v["y"] is not None:
        got["out"] = out.detach()
    total.backward()
    got.update({"d_" + k: t.grad for k, t in v.items() if t is not None})
    return got


def compare(got, want):
    for name, w in want.items():
        g = got[name]
        half_step = torch.finfo(g.dtype).eps / 2
        off = g.double() - w
        assert off.norm() <= (half_step + 2.0**-12) * w.norm(), f"{name}: {(off.norm() / w.norm()).item():g} off"
        rms = w.square().mean().sqrt()
        assert (off.abs() <= half_step * w.abs() + 2.0**-10 * rms).all(), name


@pytest.mark.parametrize("gate,sigmoid", [("none", False), *itertools.product(KINDS[1:], (False, True))])
@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("H", [192, 1160, 8296])
def test_gradients(ep, gate, sigmoid, post, f32, H):
    p = Problem(ep, 40, H, gate=gate, sigmoid=sigmoid, post=post, f32=f32, scale=0.6, offset=0.5, seed=H + post)
    f = p.forward()
    compare({**f, **p.backward(f)}, differentiate(p, True, True))


@pytest.mark.parametrize("gate", KINDS)
def test_gradients_of_one_of_the_two(ep, gate):
    p = Problem(ep, 40, 1160, gate=gate, sigmoid=True, seed=3)
    f = p.forward()
    compare({**f, **p.backward(f, d_out=None)}, differentiate(p, False, True))
    q = Problem(ep, 40, 1160, gate=gate, sigmoid=True, next=False, seed=4)
    f = q.forward()
    compare({**{k: v for k, v in f.items() if v is not None}, **q.backward(f)}, differentiate(q, True, False))


@pytest.mark.parametrize("H", [192, 1160, 8296])
@pytest.mark.parametrize("f32", [False, True])
def test_gradients_of_a_norm_alone(ep, H, f32):
    p = Problem(ep, 40, H, block=False, f32=f32, offset=1.0, seed=5)
    f = p.forward()
    compare({**f, **p.backward(f)}, differentiate(p, True, True))


@pytest.mark.parametrize("T,H", [(1300, 16384), (1220, 12808), (1216, 8200)])
@pytest.mark.parametrize("gate,post", [("element", True), ("element", False), ("channel", True), ("none", False)])
@pytest.mark.parametrize("f32", [False, True])
def test_the_longest_rows_in_turns(ep, T, H, gate, post, f32):
    """More of them than run at once, by as many bytes in flight as one row has at most: with fp32 and a gate of elements a CTA
    has one row in flight from 12808 columns on."""
    p = Problem(ep, T, H, gate=gate, sigmoid=post, post=post, f32=f32, seed=T)
    f = p.forward()
    check({**f, **p.backward(f)}, p.reference())
    del p, f
    torch.cuda.empty_cache()
