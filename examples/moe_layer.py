"""One MoE layer trained and then served on one GPU, every step of it through the library.

Training: router -> dispatch -> experts -> combine, the way back through all of them, clipping of the
gradients by their global norm, and a plain gradient step. The layer learns to imitate a fixed map of
its input. Serving: the trained experts' weights are packed to 4 bits and a few tokens are run through
the layer with them.

    python examples/moe_layer.py [--steps 30] [--tokens 512]
"""
from __future__ import annotations

import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import combine_router_softmax_gb300 as ep  # noqa: E402

BF16 = torch.bfloat16


class MoeLayer:
    """Router, experts and every buffer of one layer for T tokens, allocated once."""

    def __init__(self, T: int, H: int, I: int, E: int, k: int, seed: int = 0):
        self.cfg = ep.EpConfig.make(T=T, H=H, E=E, R=1, k=k)
        self.ffn = ep.EpFfnConfig.make(rows=T * k, H=H, I=I, E=E)
        gen = torch.Generator(device="cuda").manual_seed(seed)
        normal = lambda *s, scale: (torch.randn(s, generator=gen, device="cuda") * scale)  # noqa: E731
        # fp32 masters and the bf16 copies that the kernels read
        self.master = {"router": normal(E, H, scale=1 / math.sqrt(H)), "w_gate": normal(E, I, H, scale=1 / math.sqrt(H)),
                       "w_up": normal(E, I, H, scale=1 / math.sqrt(H)), "w_down": normal(E, H, I, scale=1 / math.sqrt(I))}
        self.w = {n: m.to(BF16) for n, m in self.master.items()}
        self.b = ep.LayerBuffers.allocate(self.cfg)
        new = lambda *s, dtype=BF16: torch.empty(s, dtype=dtype, device="cuda")  # noqa: E731
        S = T * k
        self.g, self.u = (new(S, I, dtype=torch.float16) for _ in range(2))
        self.h, self.d_g, self.d_u = (new(S, I) for _ in range(3))
        self.d_send, self.d_y = new(S, H), new(S, H)
        self.d_x = new(T, H)
        self.d_topk_w, self.d_logits = new(T, k, dtype=torch.float32), new(T, E, dtype=torch.float32)
        self.ones = torch.ones((T, k), device="cuda")
        self.grad = {n: torch.empty_like(w) for n, w in self.w.items()}
        self.clip = ep.GradList(self.grad.values())
        self.norm = new(1, dtype=torch.float32)

    @property
    def experts(self):
        return self.w["w_gate"], self.w["w_up"], self.w["w_down"]

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        b = self.b
        b.x.copy_(x)
        b.logits.copy_(x.float() @ self.w["router"].float().T)
        b.dispatch_fused()
        ep.ep_expert_ffn(self.ffn, b.send, b.expert_offset, *self.experts, self.h, b.y, g=self.g, u=self.u)
        b.combine()
        return b.out

    def backward(self, d_out: torch.Tensor) -> torch.Tensor:
        """Gradients of every weight into self.grad, that of the input returned."""
        b = self.b
        ep.ep_combine_backward(self.cfg, d_out, b.y, b.slot, b.topk_w, self.d_y, self.d_topk_w)
        ep.ep_route_backward(self.cfg, None, b.topk_idx, b.topk_w, self.d_topk_w, self.d_logits)
        ep.ep_expert_ffn_backward(self.ffn, b.send, b.expert_offset, *self.experts, self.g, self.u, self.h, self.d_y,
                                  self.d_g, self.d_u, self.d_send, self.grad["w_gate"], self.grad["w_up"],
                                  self.grad["w_down"])
        ep.ep_combine(self.cfg, self.d_send, b.slot, self.ones, self.d_x)  # dispatch backward: the sum over a token's rows
        self.grad["router"].copy_(self.d_logits.T @ b.x.float())
        return self.d_x.float() + self.d_logits @ self.w["router"].float()

    def step(self, lr: float, max_norm: float) -> None:
        self.clip.clip(max_norm, self.norm)
        for n, m in self.master.items():
            m.sub_(self.grad[n].float(), alpha=lr)
            self.w[n].copy_(m)

    def pack(self, group: int) -> dict:
        """The experts' weights in 4 bits."""
        out = {}
        for n in ("w_gate", "w_up", "w_down"):
            E, N, K = self.w[n].shape
            c = ep.EpW4Config.make(N=N, K=K, E=E, group=group)
            q_bytes, s_bytes = ep.ep_w4_sizes(c)
            q = torch.empty((E, N, q_bytes // (E * N)), dtype=torch.uint8, device="cuda")
            s = torch.empty((E, N, s_bytes // (2 * E * N)), dtype=BF16, device="cuda")
            ep.ep_w4_pack(c, self.w[n], q, s)
            out[n] = (q, s)
        return out


def serve(layer: MoeLayer, packed: dict, group: int, x: torch.Tensor) -> torch.Tensor:
    """A few tokens through the layer, its experts in 4 bits."""
    T, E = x.shape[0], layer.cfg.E
    cfg = ep.EpConfig.make(T=T, H=layer.cfg.H, E=E, R=1, k=layer.cfg.k)
    b = ep.LayerBuffers.allocate(cfg)
    b.x.copy_(x)
    b.logits.copy_(x.float() @ layer.w["router"].float().T)
    b.dispatch_fused()
    ffn = ep.EpFfnConfig.make(rows=T * cfg.k, H=cfg.H, I=layer.ffn.I, E=E)
    h = torch.empty((T * cfg.k, layer.ffn.I), dtype=BF16, device="cuda")
    ep.ep_expert_ffn_w4(ffn, group, b.send, b.expert_offset, *packed["w_gate"], *packed["w_up"], *packed["w_down"], h, b.y)
    b.combine()
    return b.out


def main(argv=None) -> dict:
    a = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    a.add_argument("--steps", type=int, default=30)
    a.add_argument("--tokens", type=int, default=512)
    a.add_argument("--hidden", type=int, default=256)
    a.add_argument("--width", type=int, default=128)
    a.add_argument("--experts", type=int, default=16)
    a.add_argument("--k", type=int, default=4)
    a.add_argument("--lr", type=float, default=0.5)
    a = a.parse_args(argv)
    layer = MoeLayer(a.tokens, a.hidden, a.width, a.experts, a.k)
    gen = torch.Generator(device="cuda").manual_seed(1)
    teach = torch.randn((a.hidden, a.hidden), generator=gen, device="cuda") / math.sqrt(a.hidden)
    x = torch.randn((a.tokens, a.hidden), generator=gen, device="cuda").to(BF16)
    target = torch.tanh(x.float() @ teach.T)
    losses, norms = [], []
    for _ in range(a.steps):
        off = layer.forward(x).float() - target
        losses.append(off.square().mean().item())
        layer.backward((off * (2 / off.shape[0])).to(BF16))  # of the squared error, summed over H, mean over the tokens
        layer.step(a.lr, max_norm=1.0)
        norms.append(layer.norm.item())
    out = layer.forward(x[:a.tokens]).float()[:4].clone()
    served = serve(layer, layer.pack(32), 32, x[:4]).float()
    off = ((served - out).norm() / out.norm()).item()
    print(f"loss {losses[0]:.4f} -> {losses[-1]:.4f} over {a.steps} steps, last gradient norm {norms[-1]:.4f}")
    print(f"4 tokens with 4-bit experts: {100 * off:.1f}% off the bf16 layer")
    assert ep.ep_device_error() == 0
    return {"losses": losses, "norms": norms, "off": off}


if __name__ == "__main__":
    main()
