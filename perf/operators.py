"""Operators of an MoE layer around dispatch and combine, as cases to be measured.

Four operators: the experts' gated feed-forward block (forward, and forward with
backward), products with 4-bit weights and group scales, the backward pass of
combine and router, and the global gradient norm with clipping. ``run`` computes
each in plain torch operations in 32 bits, or (``own``) through the package.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def listed() -> list[dict]:
    return [
        # one token's eight experts out of the 32 of a small layer: latency of a single decode step
        dict(name="ffn-decode-1", op="ffn", train=False, rows=8, E=32, H=4096, I=1024, zipf=0.0),
        # a decode batch of 64 tokens, top-8, on a device that holds 64 wide experts: the weights are the traffic
        dict(name="ffn-decode-64", op="ffn", train=False, rows=512, E=64, H=7168, I=2048, zipf=0.0),
        # a prompt of 2048 tokens, top-8, unevenly spread over 16 wide experts
        dict(name="ffn-prefill", op="ffn", train=False, rows=16384, E=16, H=7168, I=2048, zipf=0.6),
        # a training step of a small layer with odd widths and few rows, some experts without any
        dict(name="ffn-train-odd", op="ffn", train=True, rows=777, E=7, H=1000, I=360, zipf=1.2),
        # a training step of 2048 tokens, top-8, over 16 experts
        dict(name="ffn-train", op="ffn", train=True, rows=16384, E=16, H=4096, I=2048, zipf=0.3),
        # one token through eight of 64 wide experts with 4-bit weights: a single decode step
        dict(name="w4-decode-1", op="w4_ffn", rows=8, E=64, H=7168, I=2048, group=128, zipf=0.0),
        # a decode batch of 64 tokens, top-8, over 64 experts with 4-bit weights
        dict(name="w4-decode-64", op="w4_ffn", rows=512, E=64, H=4096, I=1024, group=64, zipf=0.0),
        # one dense layer with 4-bit weights in small groups, a few tokens, odd sizes
        dict(name="w4-linear-odd", op="w4_linear", rows=3, E=1, H=5000, I=4321, group=32, zipf=0.0),
        # the way back through combine and router for a short sequence: latency
        dict(name="combine-bwd-64", op="combine_bwd", T=64, H=4096, E=128, k=8, renorm=False),
        # the same for a prompt-sized batch
        dict(name="combine-bwd-4096", op="combine_bwd", T=4096, H=7168, E=256, k=8, renorm=True),
        # the many small tensors of a model's norms, biases and routers, types mixed
        dict(name="clip-many", op="clip", tensors=300, numel=9001, mixed=True, factor=0.4),
        # the weight gradients of one layer's experts: three stacked tensors
        dict(name="clip-experts", op="clip", tensors=3, numel=16 * 4096 * 2048, mixed=False, factor=0.3),
    ]


def _between(rng, low, high, step=1):
    """A size between low and high, spread over its logarithm, a multiple of step."""
    v = int(round(math.exp(rng.uniform(math.log(low), math.log(high))) / step))
    return max(math.ceil(low / step), min(high // step, v)) * step


def draw(rng) -> dict:
    op = rng.choice(["ffn", "ffn", "ffn_train", "w4_ffn", "w4_linear", "combine_bwd", "clip"])
    if op in ("ffn", "ffn_train"):
        return dict(op="ffn", train=op == "ffn_train", rows=_between(rng, 1, 16384), E=_between(rng, 1, 24),
                    H=_between(rng, 64, 5000, 8), I=_between(rng, 64, 2048, 8), zipf=rng.choice([0.0, 0.5, 1.2]))
    if op == "w4_ffn":
        return dict(op="w4_ffn", rows=_between(rng, 1, 600), E=_between(rng, 1, 64), H=_between(rng, 64, 5000, 8),
                    I=_between(rng, 64, 2048, 8), group=rng.choice([32, 64, 128]), zipf=rng.choice([0.0, 1.0]))
    if op == "w4_linear":
        return dict(op="w4_linear", rows=_between(rng, 1, 100), E=_between(rng, 1, 8), H=_between(rng, 64, 8000, 8),
                    I=_between(rng, 1, 8000), group=rng.choice([32, 64, 128]), zipf=0.0)
    if op == "combine_bwd":
        E = _between(rng, 8, 300)
        return dict(op="combine_bwd", T=_between(rng, 1, 4096), H=_between(rng, 64, 7168, 8), E=E,
                    k=rng.randint(1, 8), renorm=rng.random() < 0.5)
    return dict(op="clip", tensors=_between(rng, 1, 300), numel=_between(rng, 1, 300000), mixed=rng.random() < 0.5,
                factor=rng.choice([0.1, 0.7, 1.5]))


def _counts(case, seed) -> np.ndarray:
    """Rows of each expert: drawn for every row alone, with popularities that fall as 1 / rank^zipf."""
    r = np.random.default_rng([seed, 17])
    p = 1.0 / np.arange(1, case["E"] + 1, dtype=np.float64) ** case["zipf"]
    r.shuffle(p)
    return r.multinomial(case["rows"], p / p.sum())


def _expected_experts(case) -> float:
    """Experts that have rows, in the mean over draws of _counts."""
    p = 1.0 / np.arange(1, case["E"] + 1, dtype=np.float64) ** case["zipf"]
    p /= p.sum()
    return float(np.sum(1.0 - (1.0 - p) ** case["rows"]))


def _clip_sizes(case) -> list[tuple[int, torch.dtype]]:
    """Sizes and types of the gradient tensors: about numel values each, odd ones among them."""
    out = []
    for i in range(case["tensors"]):
        n = case["numel"] if case["tensors"] <= 3 else max(1, case["numel"] * (1 + i % 7) // 4 + i % 5)
        out.append((n, (F32, BF16, F16)[i % 3] if case["mixed"] else BF16))
    return out


def work(case) -> dict:
    if case["op"] == "ffn":
        S, H, I, hit = case["rows"], case["H"], case["I"], _expected_experts(case)
        forward = hit * 6 * H * I + 4 * S * H
        if not case["train"]:
            return {"bytes": forward, "flops": 6 * S * H * I}
        # the weights once, the rows, y, dy and d_rows once, and every expert's weight gradients written once
        return {"bytes": forward + 4 * S * H + case["E"] * 6 * H * I, "flops": 18 * S * H * I}
    if case["op"] == "w4_ffn":
        S, H, I, G, hit = case["rows"], case["H"], case["I"], case["group"], _expected_experts(case)
        return {"bytes": hit * 3 * H * I * (0.5 + 2 / G) + 4 * S * H, "flops": 6 * S * H * I}
    if case["op"] == "w4_linear":
        S, K, N, G, hit = case["rows"], case["H"], case["I"], case["group"], _expected_experts(case)
        return {"bytes": hit * N * K * (0.5 + 2 / G) + 2 * S * (K + N), "flops": 2 * S * N * K}
    if case["op"] == "combine_bwd":
        T, H, E, k = case["T"], case["H"], case["E"], case["k"]
        gate = T * E * (4 if case["renorm"] else 8)
        return {"bytes": 2 * T * H + 4 * T * k * H + 20 * T * k + gate, "flops": 3 * T * k * H}
    sizes = _clip_sizes(case)
    b = sum(2 * n * torch.empty((), dtype=t).element_size() for n, t in sizes)
    return {"bytes": b, "flops": 3 * sum(n for n, _ in sizes)}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _normal(gen, shape, scale, dtype=BF16):
    return torch.randn(shape, generator=gen, device="cuda", dtype=dtype if dtype != F16 else F32).mul_(scale).to(dtype)


def _padded(k: int) -> int:
    return (k + 127) // 128 * 128


def _w4_weight(gen, E, N, K, group):
    """A packed 4-bit weight [E, N, Kp / 2] and its bf16 scales [E, N, Kp / group]; values 8 (zero) past K."""
    Kp = _padded(K)
    q = torch.randint(0, 256, (E, N, Kp // 2), generator=gen, device="cuda", dtype=torch.uint8)
    if Kp != K:
        used = (torch.arange(Kp, device="cuda") < K)[_w4_order(Kp)].to(torch.uint8).view(-1, 2)
        low, high = q & 15, q >> 4
        low = torch.where(used[:, 0] > 0, low, torch.full_like(low, 8))
        high = torch.where(used[:, 1] > 0, high, torch.full_like(high, 8))
        q = low | (high << 4)
    scale = torch.rand((E, N, Kp // group), generator=gen, device="cuda").add_(0.5).mul_(0.22 / math.sqrt(K)).to(BF16)
    return q, scale


def _w4_order(Kp: int) -> torch.Tensor:
    """The k that the i-th nibble of a packed row holds. A 32-bit word holds k0 .. k0 + 7, its nibble n the one at
    offset 2 (n mod 4) + n / 4; word (c, t, j) of a row, in this order, starts at k0 = 128 c + 32 j + 8 t."""
    c = torch.arange(Kp // 128, device="cuda").view(-1, 1, 1, 1) * 128
    t = torch.arange(4, device="cuda").view(1, -1, 1, 1) * 8
    j = torch.arange(4, device="cuda").view(1, 1, -1, 1) * 32
    n = torch.arange(8, device="cuda").view(1, 1, 1, -1)
    return (c + t + j + 2 * (n % 4) + n // 4).reshape(-1)


def _rows_and_experts(case, seed, gen):
    counts = _counts(case, seed)
    offset = torch.from_numpy(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)).cuda()
    hit = torch.from_numpy(np.nonzero(counts)[0]).cuda()
    x = _normal(gen, (case["rows"], case["H"]), 1.0)
    return dict(rows=x, expert_offset=offset, hit=hit, most=int(counts.max()))


def prepare(case, seed) -> dict:
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    st = dict(case=dict(case))
    if case["op"] == "ffn":
        S, E, H, I = case["rows"], case["E"], case["H"], case["I"]
        st.update(_rows_and_experts(case, seed, gen))
        st["w_gate"] = _normal(gen, (E, I, H), 1 / math.sqrt(H))
        st["w_up"] = _normal(gen, (E, I, H), 1 / math.sqrt(H))
        st["w_down"] = _normal(gen, (E, H, I), 1 / math.sqrt(I))
        st["h"] = torch.empty((S, I), dtype=BF16, device="cuda")
        st["y"] = torch.empty((S, H), dtype=BF16, device="cuda")
        if case["train"]:
            st["d_y"] = _normal(gen, (S, H), 0.1)
            for n in ("g", "u", "d_g", "d_u"):
                st[n] = torch.empty((S, I), dtype=BF16, device="cuda")
            st["d_rows"] = torch.empty((S, H), dtype=BF16, device="cuda")
            for n in ("w_gate", "w_up", "w_down"):
                st["d_" + n] = torch.empty_like(st[n])
    elif case["op"] == "w4_ffn":
        S, E, H, I, G = case["rows"], case["E"], case["H"], case["I"], case["group"]
        st.update(_rows_and_experts(case, seed, gen))
        for n, (N, K) in (("gate", (I, H)), ("up", (I, H)), ("down", (H, I))):
            st["q_" + n], st["s_" + n] = _w4_weight(gen, E, N, K, G)
        st["h"] = torch.empty((S, I), dtype=BF16, device="cuda")
        st["y"] = torch.empty((S, H), dtype=BF16, device="cuda")
    elif case["op"] == "w4_linear":
        st.update(_rows_and_experts(case, seed, gen))
        st["q"], st["s"] = _w4_weight(gen, case["E"], case["I"], case["H"], case["group"])
        st["y"] = torch.empty((case["rows"], case["I"]), dtype=BF16, device="cuda")
    elif case["op"] == "combine_bwd":
        T, H, E, k = case["T"], case["H"], case["E"], case["k"]
        st["logits"] = _normal(gen, (T, E), 1.0, F32)
        p = torch.softmax(st["logits"], -1)
        w, idx = torch.topk(p, k, dim=-1)
        st["topk_w"] = (w / w.sum(-1, keepdim=True) if case["renorm"] else w).contiguous()
        st["topk_idx"] = idx.to(torch.int32)
        # rows are ordered by expert, then by token
        order = torch.argsort(idx.reshape(-1), stable=True)
        slot = torch.empty_like(order)
        slot[order] = torch.arange(T * k, device="cuda")
        st["slot"] = slot.view(T, k).to(torch.int32)
        st["y"] = _normal(gen, (T * k, H), 1.0)
        st["d_out"] = _normal(gen, (T, H), 0.1)
        st["d_y"] = torch.empty_like(st["y"])
        st["d_topk_w"] = torch.empty_like(st["topk_w"])
        st["d_logits"] = torch.empty_like(st["logits"])
    else:
        # the tensors lie one after another in one buffer of each type, so most start off a 16-byte boundary
        sizes = _clip_sizes(case)
        types = [t for t in (F32, BF16, F16) if any(u == t for _, u in sizes)]
        st["flat"] = {t: _normal(gen, (sum(n for n, u in sizes if u == t),), 0.01, t) for t in types}
        st["flat_clipped"] = {t: torch.empty_like(f) for t, f in st["flat"].items()}
        for name in ("flat", "flat_clipped"):
            parts = {t: list(f.split([n for n, u in sizes if u == t])) for t, f in st[name].items()}
            st[name.replace("flat", "grads")] = [parts[t].pop(0) for _, t in sizes]
        # about the norm that these gradients have, times factor: above one nothing is to be scaled
        st["max_norm"] = case["factor"] * 0.01 * math.sqrt(sum(n for n, _ in _clip_sizes(case)))
        st["norm"] = torch.empty((1,), dtype=F32, device="cuda")
    return st


# ---------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------

def _by_expert(st, rows):
    """[experts with rows, most rows of one, n] in 32 bits, zero past an expert's rows."""
    first, end = st["expert_offset"][st["hit"]], st["expert_offset"][st["hit"] + 1]
    i = first[:, None] + torch.arange(st["most"], device="cuda")
    inside = i < end[:, None]
    return rows[torch.where(inside, i, 0)].float() * inside[..., None]


def _by_row(st, padded):
    """The rows of _by_expert's form in their own order."""
    row = torch.arange(st["rows"].shape[0], device="cuda", dtype=torch.int32)
    p = torch.searchsorted(st["expert_offset"][st["hit"]], row, right=True) - 1
    return padded[p, row - st["expert_offset"][st["hit"]][p]]


def _every_expert(st, of_hit, E):
    """[E, ...] with the experts that have rows filled in and zeros for the others."""
    out = torch.zeros((E,) + tuple(of_hit.shape[1:]), dtype=BF16, device="cuda")
    out[st["hit"]] = of_hit.to(BF16)
    return out


def _plain_ffn(st):
    x = _by_expert(st, st["rows"])
    wg, wu, wd = (st[n][st["hit"]].float() for n in ("w_gate", "w_up", "w_down"))
    g, u = x @ wg.transpose(1, 2), x @ wu.transpose(1, 2)
    s = torch.sigmoid(g)
    h = g * s * u
    y = _by_row(st, h @ wd.transpose(1, 2)).to(BF16)
    if not st["case"]["train"]:
        return {"y": y}
    dy = _by_expert(st, st["d_y"])
    dh = dy @ wd
    du = dh * g * s
    dg = dh * u * s * (1 + g * (1 - s))
    E = st["case"]["E"]
    return {"y": y, "d_rows": _by_row(st, dg @ wg + du @ wu).to(BF16),
            "d_w_gate": _every_expert(st, dg.transpose(1, 2) @ x, E),
            "d_w_up": _every_expert(st, du.transpose(1, 2) @ x, E),
            "d_w_down": _every_expert(st, dy.transpose(1, 2) @ h, E)}


def _plain_w4_matrix(st, q, scale, K, group):
    """The experts that have rows, [hit, N, K] in 32 bits."""
    q, scale = q[st["hit"]], scale[st["hit"]].float()
    E, N, Kp = q.shape[0], q.shape[1], 2 * q.shape[2]
    values = torch.stack((q & 15, q >> 4), -1).view(E, N, Kp).float() - 8
    w = torch.empty_like(values)
    w[:, :, _w4_order(Kp)] = values
    return (w.view(E, N, Kp // group, group) * scale[..., None]).view(E, N, Kp)[:, :, :K]


def _plain_w4_ffn(st):
    c = st["case"]
    x = _by_expert(st, st["rows"])
    g = x @ _plain_w4_matrix(st, st["q_gate"], st["s_gate"], c["H"], c["group"]).transpose(1, 2)
    u = x @ _plain_w4_matrix(st, st["q_up"], st["s_up"], c["H"], c["group"]).transpose(1, 2)
    h = g * torch.sigmoid(g) * u
    y = h @ _plain_w4_matrix(st, st["q_down"], st["s_down"], c["I"], c["group"]).transpose(1, 2)
    return {"y": _by_row(st, y).to(BF16)}


def _plain_w4_linear(st):
    c = st["case"]
    y = _by_expert(st, st["rows"]) @ _plain_w4_matrix(st, st["q"], st["s"], c["H"], c["group"]).transpose(1, 2)
    return {"y": _by_row(st, y).to(BF16)}


def _plain_combine_bwd(st):
    c = st["case"]
    slot, idx, w = st["slot"].long(), st["topk_idx"].long(), st["topk_w"]
    d_out = st["d_out"].float()
    d_y = torch.empty_like(st["y"])
    d_y[slot.view(-1)] = (w[..., None] * d_out[:, None, :]).to(BF16).view(-1, c["H"])
    d_w = (st["y"][slot].float() * d_out[:, None, :]).sum(-1)
    mean = (w * d_w).sum(-1, keepdim=True)
    if c["renorm"]:
        d_l = torch.zeros_like(st["logits"]).scatter_(1, idx, w * (d_w - mean))
    else:
        l = st["logits"]
        p = torch.exp(l - l.amax(-1, keepdim=True))
        p = p / p.sum(-1, keepdim=True)
        d_l = p * (torch.zeros_like(l).scatter_(1, idx, d_w) - mean)
    return {"d_y": d_y, "d_topk_w": d_w, "d_logits": d_l}


def _plain_clip(st):
    norm = torch.stack([(f.float() ** 2).sum() for f in st["flat"].values()]).sum().sqrt()
    coef = (st["max_norm"] / (norm + 1e-6)).clamp(max=1.0)
    return {"norm": norm.view(1), "clipped": [(f.float() * coef).to(t) for t, f in st["flat"].items()]}


# ---------------------------------------------------------------------------
# The package's calls
# ---------------------------------------------------------------------------

def _own(st):
    import combine_router_softmax_gb300 as ep

    c = st["case"]
    if c["op"] == "ffn":
        cfg = ep.EpFfnConfig.make(rows=c["rows"], H=c["H"], I=c["I"], E=c["E"])
        weights = (st["w_gate"], st["w_up"], st["w_down"])
        if not c["train"]:
            ep.ep_expert_ffn(cfg, st["rows"], st["expert_offset"], *weights, st["h"], st["y"])
            return {"y": st["y"]}
        ep.ep_expert_ffn(cfg, st["rows"], st["expert_offset"], *weights, st["h"], st["y"], g=st["g"], u=st["u"])
        ep.ep_expert_ffn_backward(cfg, st["rows"], st["expert_offset"], *weights, st["g"], st["u"], st["h"], st["d_y"],
                                  st["d_g"], st["d_u"], st["d_rows"], st["d_w_gate"], st["d_w_up"], st["d_w_down"])
        return {n: st[n] for n in ("y", "d_rows", "d_w_gate", "d_w_up", "d_w_down")}
    if c["op"] == "w4_ffn":
        cfg = ep.EpFfnConfig.make(rows=c["rows"], H=c["H"], I=c["I"], E=c["E"])
        ep.ep_expert_ffn_w4(cfg, c["group"], st["rows"], st["expert_offset"], st["q_gate"], st["s_gate"], st["q_up"],
                            st["s_up"], st["q_down"], st["s_down"], st["h"], st["y"])
        return {"y": st["y"]}
    if c["op"] == "w4_linear":
        cfg = ep.EpW4Config.make(rows=c["rows"], N=c["I"], K=c["H"], E=c["E"], group=c["group"])
        ep.ep_w4_linear(cfg, st["rows"], st["expert_offset"], st["q"], st["s"], st["y"])
        return {"y": st["y"]}
    if c["op"] == "combine_bwd":
        cfg = ep.EpConfig.make(T=c["T"], H=c["H"], E=c["E"], R=1, k=c["k"], renormalize=int(c["renorm"]))
        ep.ep_combine_backward(cfg, st["d_out"], st["y"], st["slot"], st["topk_w"], st["d_y"], st["d_topk_w"])
        ep.ep_route_backward(cfg, st["logits"], st["topk_idx"], st["topk_w"], st["d_topk_w"], st["d_logits"])
        return {n: st[n] for n in ("d_y", "d_topk_w", "d_logits")}
    if "plan" not in st:
        st["plan"] = ep.GradList(st["grads"], st["grads_clipped"])
    st["plan"].clip(st["max_norm"], st["norm"])
    return {"norm": st["norm"], "clipped": list(st["flat_clipped"].values())}


_PLAIN = {"ffn": _plain_ffn, "w4_ffn": _plain_w4_ffn, "w4_linear": _plain_w4_linear,
          "combine_bwd": _plain_combine_bwd, "clip": _plain_clip}


def run(state):
    if own:
        return _own(state)
    return _PLAIN[state["case"]["op"]](state)


# ---------------------------------------------------------------------------
# The same from the definitions, in 64 bits
# ---------------------------------------------------------------------------

def _exact_w4(q, scale, K, group):
    """One expert's matrix [N, K] in 64 bits, word by word as the packed form is defined."""
    N, words = q.shape[0], q.shape[1] // 4
    bits = q.view(N, words, 4).long()
    word = bits[..., 0] | bits[..., 1] << 8 | bits[..., 2] << 16 | bits[..., 3] << 24
    w = torch.zeros((N, 8 * words), dtype=torch.float64, device="cuda")
    at = torch.arange(words, device="cuda")
    first = at // 16 * 128 + at % 4 * 32 + at % 16 // 4 * 8
    for n in range(8):
        k = first + 2 * (n % 4) + n // 4
        w[:, k] = ((word >> (4 * n)) & 15).double() - 8
    return (w * scale.double().repeat_interleave(group, 1))[:, :K]


def exact(case, seed):
    if case["op"] in ("ffn", "w4_ffn", "w4_linear") and work(case)["flops"] > 4e12:
        return None
    st = prepare(case, seed)
    if case["op"] in ("ffn", "w4_ffn", "w4_linear"):
        bounds = st["expert_offset"].tolist()
        train = case.get("train", False)
        S, H, I, E = case["rows"], case["H"], case["I"], case["E"]
        f64 = dict(dtype=torch.float64, device="cuda")
        y = torch.zeros((S, I if case["op"] == "w4_linear" else H), **f64)
        if train:
            d_x = torch.zeros((S, H), **f64)
            d_g, d_u, d_d = torch.zeros((E, I, H), **f64), torch.zeros((E, I, H), **f64), torch.zeros((E, H, I), **f64)
        for e in range(E):
            a, b = bounds[e], bounds[e + 1]
            if a == b:
                continue
            x = st["rows"][a:b].double()
            if case["op"] == "w4_linear":
                y[a:b] = x @ _exact_w4(st["q"][e], st["s"][e], H, case["group"]).T
                continue
            if case["op"] == "ffn":
                wg, wu, wd = st["w_gate"][e].double(), st["w_up"][e].double(), st["w_down"][e].double()
            else:
                wg, wu = (_exact_w4(st["q_" + n][e], st["s_" + n][e], H, case["group"]) for n in ("gate", "up"))
                wd = _exact_w4(st["q_down"][e], st["s_down"][e], I, case["group"])
            g, u = x @ wg.T, x @ wu.T
            h = g / (1 + torch.exp(-g)) * u
            y[a:b] = h @ wd.T
            if train:
                dy = st["d_y"][a:b].double()
                dh = dy @ wd
                s = 1 / (1 + torch.exp(-g))
                dg, du = dh * u * (s + g * s * (1 - s)), dh * g * s
                d_x[a:b] = dg @ wg + du @ wu
                d_g[e], d_u[e], d_d[e] = dg.T @ x, du.T @ x, dy.T @ h
        if train:
            return {"y": y, "d_rows": d_x, "d_w_gate": d_g, "d_w_up": d_u, "d_w_down": d_d}
        return {"y": y}
    if case["op"] == "combine_bwd":
        T, k = case["T"], case["k"]
        w, d_out = st["topk_w"].double(), st["d_out"].double()
        d_y = torch.zeros(st["y"].shape, dtype=torch.float64, device="cuda")
        d_w = torch.zeros((T, k), dtype=torch.float64, device="cuda")
        for j in range(k):
            at = st["slot"][:, j].long()
            d_y[at] = w[:, j:j + 1] * d_out
            d_w[:, j] = torch.einsum("th,th->t", d_out, st["y"][at].double())
        # the weights that the layer used are inputs; the softmax over all experts is the logits'
        d_p = torch.zeros(st["logits"].shape, dtype=torch.float64, device="cuda")
        d_p.scatter_(1, st["topk_idx"].long(), d_w)
        if case["renorm"]:
            p = torch.zeros_like(d_p).scatter_(1, st["topk_idx"].long(), w)
        else:
            p = torch.softmax(st["logits"].double(), -1)
        inner = torch.einsum("tk,tk->t", w, d_w)
        return {"d_y": d_y, "d_topk_w": d_w, "d_logits": p * (d_p - inner[:, None])}
    flats = list(st["flat"].values())
    square = sum(float(torch.dot(f.double(), f.double())) for f in flats)
    norm = math.sqrt(square)
    coef = min(1.0, st["max_norm"] / (norm + 1e-6))
    return {"norm": torch.tensor([norm], dtype=torch.float64, device="cuda"),
            "clipped": [f.double() * coef for f in flats]}
