"""Operators around an MoE layer in training, as cases to be measured.

Three operators: the norms before and after a block fused with its gate and residual
scale (forward, and forward with backward), the balance loss of the router with
per-expert counts and gradients, and the orthogonalisation of weight updates by
Newton-Schulz products. ``run`` computes each in plain torch operations in 32 bits, or
(``own``) through the package.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
_TYPES = {"bf16": BF16, "f16": F16, "f32": F32}
_COEFFICIENTS = (3.4445, -4.7750, 2.0315)  # of the quintic that draws singular values towards one


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def listed() -> list[dict]:
    return [
        # one token between two blocks of a wide model: latency of a decode step
        dict(name="norm-decode-1", op="norm", train=False, T=1, H=7168, post=False, gate="none", sigmoid=False,
             f32=False, scale=1.0, offset=0.0),
        # a prompt of 4096 tokens, norms on either side of the block and a learned scale of every channel
        dict(name="norm-prefill", op="norm", train=False, T=4096, H=7168, post=True, gate="channel", sigmoid=False,
             f32=False, scale=1.0, offset=0.0),
        # a training step with few rows of an odd width, the residual stream in 32 bits, a sigmoid gate for each token
        dict(name="norm-train-odd", op="norm", train=True, T=777, H=1000, post=True, gate="token", sigmoid=True,
             f32=True, scale=0.22, offset=1.0),
        # a training step of 16384 tokens, norm, residual and the next block's norm
        dict(name="norm-train", op="norm", train=True, T=16384, H=4096, post=False, gate="none", sigmoid=False,
             f32=False, scale=1.0, offset=0.0),
        # a microbatch of a small layer: latency
        dict(name="balance-tiny", op="balance", T=128, E=8, k=2, seqs=1, padded=False, zipf=0.0, through=True),
        # a padded batch of seven sequences of different lengths, an odd number of experts
        dict(name="balance-padded", op="balance", T=4095, E=100, k=6, seqs=7, padded=True, zipf=0.5, through=True),
        # a batch of 32768 tokens over 256 experts, unevenly chosen
        dict(name="balance-32768", op="balance", T=32768, E=256, k=8, seqs=1, padded=False, zipf=1.2, through=True),
        # 64 packed sequences, each balanced by itself
        dict(name="balance-sequences", op="balance", T=131072, E=128, k=8, seqs=64, padded=False, zipf=0.5, through=False),
        # the updates of a small layer's 64 experts: many matrices that each fit one tile
        dict(name="ortho-small", op="ortho", B=64, N=128, K=256, type="bf16", spread=0.5),
        # the update of a wide layer's router
        dict(name="ortho-router", op="ortho", B=1, N=256, K=7168, type="f32", spread=0.5),
        # the updates of seven experts of odd sizes, taller than wide
        dict(name="ortho-odd", op="ortho", B=7, N=1000, K=360, type="bf16", spread=1.0),
        # the updates of 16 experts' up projections
        dict(name="ortho-experts", op="ortho", B=16, N=2048, K=4096, type="bf16", spread=0.5),
    ]


def _between(rng, low, high, step=1):
    """A size between low and high, spread over its logarithm, a multiple of step."""
    v = int(round(math.exp(rng.uniform(math.log(low), math.log(high))) / step))
    return max(math.ceil(low / step), min(high // step, v)) * step


def draw(rng) -> dict:
    op = rng.choice(["norm", "norm", "balance", "balance", "ortho", "ortho"])
    if op == "norm":
        return dict(op="norm", train=rng.random() < 0.6, T=_between(rng, 1, 8192), H=_between(rng, 64, 8192, 8),
                    post=rng.random() < 0.5, gate=rng.choice(["none", "channel", "token", "element"]),
                    sigmoid=rng.random() < 0.5, f32=rng.random() < 0.4, scale=rng.choice([1.0, 0.22]),
                    offset=rng.choice([0.0, 1.0]))
    if op == "balance":
        T, E = _between(rng, 1, 65536), _between(rng, 2, 256)
        return dict(op="balance", T=T, E=E, k=rng.randint(1, min(8, E)), seqs=min(T, _between(rng, 1, 100)),
                    padded=rng.random() < 0.4, zipf=rng.choice([0.0, 0.5, 1.2]), through=rng.random() < 0.5)
    return dict(op="ortho", B=_between(rng, 1, 16), N=_between(rng, 1, 2048), K=_between(rng, 1, 4096),
                type=rng.choice(["bf16", "f16", "f32"]), spread=rng.choice([0.0, 0.5, 1.0]))


def work(case) -> dict:
    if case["op"] == "norm":
        T, H, r = case["T"], case["H"], 4 if case["f32"] else 2
        gate = {"none": 0, "channel": 2 * H, "token": 4 * T, "element": 2 * T * H}[case["gate"]]
        weights = 2 * H * (2 if case["post"] else 1)
        b = T * H * (2 * r + 4) + gate + weights  # x, y -> out, n
        f = T * H * 10
        if case["train"]:  # and d_out, d_n -> d_x, d_y, with the gradients of gate and weights
            b += T * H * (2 * r + 4) + 2 * weights + (gate if case["gate"] in ("token", "element") else 2 * gate)
            f += T * H * 30
        return {"bytes": b, "flops": f}
    if case["op"] == "balance":
        T, E, k, S = case["T"], case["E"], case["k"], case["seqs"]
        return {"bytes": 4 * T * E * (3 if case["through"] else 2) + 4 * T * k + 12 * S * E, "flops": 12 * T * E}
    B, m, n = case["B"], min(case["N"], case["K"]), max(case["N"], case["K"])
    size = 4 if case["type"] == "f32" else 2
    # X X^T and A A are symmetric: half of each
    return {"bytes": B * m * n * (size + 2), "flops": 5 * B * (3 * m * m * n + m * m * m)}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _normal(gen, shape, scale=1.0, dtype=BF16):
    return torch.randn(shape, generator=gen, device="cuda").mul_(scale).to(dtype)


def _bounds(case, seed) -> tuple[np.ndarray, np.ndarray]:
    """First row of every sequence, with the end of the last, and the sequences' lengths."""
    r = np.random.default_rng([seed, 29])
    T, S = case["T"], case["seqs"]
    if case["padded"]:  # as many rows for each, of which some are used
        row = T // S
        return np.arange(S + 1) * row, r.integers(0, row + 1, S)
    cuts = np.sort(r.integers(0, T + 1, S - 1))
    first = np.concatenate([[0], cuts, [T]])
    return first, np.diff(first)


def prepare(case, seed) -> dict:
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    st = dict(case=dict(case))
    if case["op"] == "norm":
        T, H, row = case["T"], case["H"], F32 if case["f32"] else BF16
        st["x"], st["y"] = _normal(gen, (T, H), 2.0, row), _normal(gen, (T, H), 0.7)
        st["w_post"] = _normal(gen, (H,), 0.1).add_(1.0 - case["offset"]) if case["post"] else None
        st["w_next"] = _normal(gen, (H,), 0.1).add_(1.0 - case["offset"])
        shape = {"none": None, "channel": (H,), "token": (T,), "element": (T, H)}[case["gate"]]
        st["gate"] = None if shape is None else _normal(gen, shape, 1.0, F32 if case["gate"] == "token" else BF16)
        new = lambda *s, dtype: torch.empty(s, dtype=dtype, device="cuda")  # noqa: E731
        st["out"], st["n"] = new(T, H, dtype=row), new(T, H, dtype=BF16)
        if case["train"]:
            st["d_out"], st["d_n"] = _normal(gen, (T, H), 0.02, row), _normal(gen, (T, H), 0.02)
            st["d_x"], st["d_y"] = new(T, H, dtype=row), new(T, H, dtype=BF16)
            st["d_w_next"] = new(H, dtype=F32)
            st["d_w_post"] = new(H, dtype=F32) if case["post"] else None
            st["d_gate"] = None if shape is None else new(*shape, dtype=BF16 if case["gate"] == "element" else F32)
            st["rstd_post"] = new(T, dtype=F32) if case["post"] else None
            st["rstd_next"] = new(T, dtype=F32)
    elif case["op"] == "balance":
        T, E, k, S = case["T"], case["E"], case["k"], case["seqs"]
        popular = -case["zipf"] * torch.log(1.0 + torch.randperm(E, generator=gen, device="cuda").float())
        st["logits"] = _normal(gen, (T, E), 1.0, F32) + popular
        st["topk_idx"] = torch.topk(st["logits"], k, dim=-1)[1].to(torch.int32)
        first, length = _bounds(case, seed)
        st["first"] = torch.from_numpy(first.astype(np.int32)).cuda()
        st["length"] = torch.from_numpy(length.astype(np.int32)).cuda()
        st["d_loss"] = torch.tensor([[0.01, 0.001]], device="cuda").expand(S, 2).contiguous() / S
        st["d_in"] = _normal(gen, (T, E), 1e-4 / T, F32) if case["through"] else None
        st["count"] = torch.empty((S, E), dtype=torch.int32, device="cuda")
        for n, shape in (("load", (S, E)), ("prob", (S, E)), ("loss", (S, 2)), ("d_logits", (T, E))):
            st[n] = torch.empty(shape, dtype=F32, device="cuda")
    else:
        # a gradient: outer products of activations and their gradients, whose channels differ in size
        B, N, K = case["B"], case["N"], case["K"]
        m = torch.randn((B, N, K), generator=gen, device="cuda")
        m *= torch.exp(case["spread"] * torch.randn((B, 1, K), generator=gen, device="cuda"))
        m += torch.randn((B, N, 1), generator=gen, device="cuda") * torch.randn((B, 1, K), generator=gen, device="cuda")
        st["m"] = m.mul_(1e-3).to(_TYPES[case["type"]])
        st["out"] = torch.empty((B, N, K), dtype=BF16, device="cuda")
    return st


# ---------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------

_EPS_NORM, _EPS_ORTHO = 1e-6, 1e-7


def _plain_norm(st):
    c = st["case"]
    x, y, o, s = st["x"].float(), st["y"].float(), c["offset"], c["scale"]
    r = r_y = None
    z = y
    if c["post"]:
        r_y = torch.rsqrt((y * y).mean(-1, keepdim=True) + _EPS_NORM)
        w_post = o + st["w_post"].float()
        z = w_post * (y * r_y)
    act = 1.0
    if c["gate"] != "none":
        g = st["gate"].float()
        g = g[:, None] if c["gate"] == "token" else g
        act = torch.sigmoid(g) if c["sigmoid"] else g
    out = x + s * act * z
    r = torch.rsqrt((out * out).mean(-1, keepdim=True) + _EPS_NORM)
    w_next = o + st["w_next"].float()
    got = {"out": out.to(st["x"].dtype), "n": (w_next * (out * r)).to(BF16)}
    if not c["train"]:
        return got
    d_n = st["d_n"].float()
    gn = w_next * d_n
    d = st["d_out"].float() + r * (gn - out * r * r * (gn * out).mean(-1, keepdim=True))
    e = s * act * d
    got["d_x"], got["d_w_next"] = d.to(st["x"].dtype), (d_n * (out * r)).sum(0)
    if c["post"]:
        ew = w_post * e
        got["d_y"] = (r_y * (ew - y * r_y * r_y * (ew * y).mean(-1, keepdim=True))).to(BF16)
        got["d_w_post"] = (e * (y * r_y)).sum(0)
    else:
        got["d_y"] = e.to(BF16)
    if c["gate"] != "none":
        dg = s * d * z
        dg = dg * act * (1 - act) if c["sigmoid"] else dg
        got["d_gate"] = {"channel": lambda: dg.sum(0), "token": lambda: dg.sum(1), "element": lambda: dg.to(BF16)}[c["gate"]]()
    return got


def _plain_balance(st):
    c = st["case"]
    T, E, k, S = c["T"], c["E"], c["k"], c["seqs"]
    logits = st["logits"]
    row = torch.arange(T, device="cuda", dtype=torch.int32)
    s = (torch.searchsorted(st["first"], row, right=True) - 1).clamp(0, S - 1)
    inside = (row - st["first"][s] < st["length"][s]) & (row < st["first"][-1])
    n = st["length"].float().clamp(min=1.0)
    top = logits.amax(-1, keepdim=True)
    e = torch.exp(logits - top)
    total = e.sum(-1, keepdim=True)
    p, lse = e / total, (top + torch.log(total))[:, 0]
    chosen = torch.zeros((T, E), device="cuda").scatter_add_(1, st["topk_idx"].long(), torch.ones((T, k), device="cuda"))
    # sums over a sequence's rows, in 64 bits: they are long
    member = torch.zeros((S, E), dtype=torch.float64, device="cuda")
    count = member.index_add(0, s, (chosen * inside[:, None]).double())
    prob = member.index_add(0, s, (p * inside[:, None]).double()) / n[:, None]
    z = torch.zeros(S, dtype=torch.float64, device="cuda").index_add(0, s, (lse * lse * inside).double()) / n
    load = count / (k * n[:, None])
    loss = torch.stack([E * (load * prob).sum(-1), z], -1)
    f = load.float()[s]
    c0, c1 = st["d_loss"][s, 0] * E / n[s], 2.0 * st["d_loss"][s, 1] / n[s]
    d = p * (c0[:, None] * (f - (f * p).sum(-1, keepdim=True)) + (c1 * lse)[:, None]) * inside[:, None]
    if c["through"]:
        d = d + st["d_in"]
    return {"count": count.to(torch.int32), "load": load.float(), "prob": prob.float(), "loss": loss.float(), "d_logits": d}


def _plain_ortho(st):
    x = st["m"].float()
    tall = x.shape[1] > x.shape[2]
    if tall:
        x = x.transpose(1, 2)
    x = x / ((x * x).sum((1, 2), keepdim=True).sqrt() + _EPS_ORTHO)
    a, b, c = _COEFFICIENTS
    for _ in range(5):
        g = x @ x.transpose(1, 2)
        x = a * x + (b * g + c * (g @ g)) @ x
    return {"out": (x.transpose(1, 2) if tall else x).to(BF16)}


# ---------------------------------------------------------------------------
# The package's calls
# ---------------------------------------------------------------------------

def _own(st):
    import combine_router_softmax_gb300 as ep

    c = st["case"]
    if c["op"] == "norm":
        gate = {"none": ep.EP_GATE_NONE, "channel": ep.EP_GATE_CHANNEL, "token": ep.EP_GATE_TOKEN,
                "element": ep.EP_GATE_ELEMENT}[c["gate"]]
        cfg = ep.EpNormConfig.make(T=c["T"], H=c["H"], gate=gate, gate_sigmoid=int(c["sigmoid"]),
                                   residual_f32=int(c["f32"]), eps=_EPS_NORM, scale=c["scale"], weight_offset=c["offset"])
        if not c["train"]:
            ep.ep_block_norm(cfg, st["x"], st["y"], st["w_post"], st["gate"], st["w_next"], st["out"], st["n"])
            return {"out": st["out"], "n": st["n"]}
        if "workspace" not in st:
            st["workspace"] = torch.empty((ep.ep_block_norm_workspace_size(cfg),), dtype=torch.uint8, device="cuda")
        ep.ep_block_norm(cfg, st["x"], st["y"], st["w_post"], st["gate"], st["w_next"], st["out"], st["n"],
                         rstd_post=st["rstd_post"], rstd_next=st["rstd_next"])
        ep.ep_block_norm_backward(cfg, st["x"], st["y"], st["w_post"], st["gate"], st["w_next"], st["rstd_post"],
                                  st["rstd_next"], st["d_out"], st["d_n"], st["d_x"], st["d_y"],
                                  d_w_post=st["d_w_post"], d_gate=st["d_gate"], d_w_next=st["d_w_next"],
                                  workspace=st["workspace"])
        got = {n: st[n] for n in ("out", "n", "d_x", "d_w_next", "d_y")}
        if c["post"]:
            got["d_w_post"] = st["d_w_post"]
        if c["gate"] != "none":
            got["d_gate"] = st["d_gate"]
        return got
    if c["op"] == "balance":
        cfg = ep.EpConfig.make(T=c["T"], H=8, E=c["E"], R=1, k=c["k"])
        if "workspace" not in st:
            st["workspace"] = torch.empty((ep.ep_balance_workspace_size(cfg, c["seqs"]),), dtype=torch.uint8, device="cuda")
        length = st["length"] if c["padded"] else None
        ep.ep_balance(cfg, st["logits"], st["topk_idx"], st["first"], length, st["count"], st["load"], st["prob"],
                      st["loss"], st["workspace"])
        ep.ep_balance_backward(cfg, st["logits"], st["first"], length, st["load"], st["d_loss"], st["d_in"], st["d_logits"])
        return {n: st[n] for n in ("count", "load", "prob", "loss", "d_logits")}
    cfg = ep.EpOrthoConfig.make(B=c["B"], N=c["N"], K=c["K"], dtype=st["m"].dtype, steps=5, eps=_EPS_ORTHO)
    if "workspace" not in st:
        st["workspace"] = torch.empty((ep.ep_orthogonalize_workspace_size(cfg),), dtype=torch.uint8, device="cuda")
    ep.ep_orthogonalize(cfg, st["m"], st["out"], st["workspace"])
    return {"out": st["out"]}


_PLAIN = {"norm": _plain_norm, "balance": _plain_balance, "ortho": _plain_ortho}


def run(state):
    if own:
        return _own(state)
    return _PLAIN[state["case"]["op"]](state)


# ---------------------------------------------------------------------------
# The same from the definitions, in 64 bits
# ---------------------------------------------------------------------------

def _exact_norm(case, st):
    """Forward by the definitions, backward by automatic differentiation."""
    names = ("x", "y", "w_post", "w_next", "gate")
    v = {n: None if st[n] is None else st[n].double().requires_grad_(case["train"]) for n in names}

    def normed(rows, w):
        return (case["offset"] + w) * rows / torch.sqrt(rows.square().mean(1) + _EPS_NORM).unsqueeze(1)

    z = normed(v["y"], v["w_post"]) if case["post"] else v["y"]
    if v["gate"] is not None:
        g = v["gate"] if case["gate"] != "token" else v["gate"].unsqueeze(1)
        z = z * (1 / (1 + torch.exp(-g)) if case["sigmoid"] else g)
    out = v["x"] + case["scale"] * z
    n = normed(out, v["w_next"])
    got = {"out": out.detach(), "n": n.detach()}
    if case["train"]:
        ((out * st["d_out"].double()).sum() + (n * st["d_n"].double()).sum()).backward()
        got.update({"d_" + k: t.grad for k, t in v.items() if t is not None})
    return got


def _exact_balance(case, st):
    """Sequence by sequence; the gradient by automatic differentiation, with the loads as they are."""
    E, k = case["E"], case["k"]
    logits = st["logits"].double().requires_grad_()
    d_loss = st["d_loss"].double()
    count, load, prob, loss = [], [], [], []
    total = torch.zeros((), dtype=torch.float64, device="cuda")
    for s, (first, n) in enumerate(zip(st["first"].tolist(), st["length"].tolist())):
        rows = logits[first:first + n]
        chosen = st["topk_idx"][first:first + n].reshape(-1).long()
        count.append(torch.bincount(chosen, minlength=E))
        load.append(count[-1].double() / (k * max(n, 1)))
        prob.append(torch.softmax(rows, 1).sum(0) / max(n, 1))
        z = torch.logsumexp(rows, 1).square().sum() / max(n, 1)
        balance = E * torch.dot(load[-1], prob[-1])
        loss.append(torch.stack([balance, z]))
        total = total + d_loss[s, 0] * balance + d_loss[s, 1] * z
    total.backward()
    d = logits.grad if st["d_in"] is None else logits.grad + st["d_in"].double()
    return {"count": torch.stack(count).to(torch.int32), "load": torch.stack(load), "prob": torch.stack(prob).detach(),
            "loss": torch.stack(loss).detach(), "d_logits": d}


def _exact_ortho(case, st):
    """Matrix by matrix, the polynomial taken as it stands."""
    out = torch.empty(st["m"].shape, dtype=torch.float64, device="cuda")
    a, b, c = _COEFFICIENTS
    for i in range(case["B"]):
        x = st["m"][i].double()
        x = x / (torch.linalg.vector_norm(x) + _EPS_ORTHO)
        for _ in range(5):
            if case["N"] <= case["K"]:
                g = x @ x.T
                y = g @ x
                x = a * x + b * y + c * (g @ y)
            else:
                g = x.T @ x
                y = x @ g
                x = a * x + b * y + c * (y @ g)
        out[i] = x
    return {"out": out}


def exact(case, seed):
    if case["op"] == "ortho" and work(case)["flops"] > 5e12:
        return None
    st = prepare(case, seed)
    return {"norm": _exact_norm, "balance": _exact_balance, "ortho": _exact_ortho}[case["op"]](case, st)
