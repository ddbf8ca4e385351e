"""Binding of ``include/ep_experts.h``: the experts between dispatch and combine, and the way back.

Like the rest of the binding this only marshals arguments: every function has
the name of its C entry point, checks dtype, shape and device of each tensor,
passes the current CUDA stream and raises :class:`EpError` on a non-zero
status. The package re-exports everything here.
"""
from __future__ import annotations

import ctypes

import numpy as np
import torch

from . import EpConfig, _check, _device, _lib, _ptr, _stream

EXPORTS = ("ep_expert_ffn", "ep_expert_ffn_backward", "ep_w4_sizes", "ep_w4_pack", "ep_w4_linear", "ep_expert_ffn_w4",
           "ep_combine_backward", "ep_route_backward", "ep_grad_workspace_size", "ep_grad_norm", "ep_grad_clip",
           "ep_grad_clip_with_norm")
__all__ = [*EXPORTS, "EpFfnConfig", "EpW4Config", "EpGradTensor", "GradList"]


class EpFfnConfig(ctypes.Structure):
    """``ep_ffn_config`` of include/ep_experts.h.

    ``saved_bf16``: what ep_expert_ffn keeps for the backward pass (g and u) is float16 (0), finer for values
    between 6.1e-5 and 65504, or bfloat16 (1), for values of any size."""
    _fields_ = [(n, ctypes.c_int32) for n in ("rows", "H", "I", "E", "saved_bf16")]

    @classmethod
    def make(cls, *, rows, H, I, E, saved_bf16=0) -> "EpFfnConfig":
        return cls(rows, H, I, E, saved_bf16)


class EpW4Config(ctypes.Structure):
    """``ep_w4_config`` of include/ep_experts.h."""
    _fields_ = [(n, ctypes.c_int32) for n in ("rows", "N", "K", "E", "group")]

    @classmethod
    def make(cls, *, rows=0, N, K, E=1, group=128) -> "EpW4Config":
        return cls(rows, N, K, E, group)


class EpGradTensor(ctypes.Structure):
    """``ep_grad_tensor`` of include/ep_experts.h."""
    _fields_ = [("data", ctypes.c_void_p), ("out", ctypes.c_void_p), ("numel", ctypes.c_int64),
                ("dtype", ctypes.c_int32), ("reserved", ctypes.c_int32)]


def _declare() -> None:
    P, vp, i32, size = ctypes.POINTER, ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
    ffn, w4, layer, grads = P(EpFfnConfig), P(EpW4Config), P(EpConfig), P(EpGradTensor)
    _lib.ep_w4_sizes.argtypes = [w4, P(size), P(size)]
    _lib.ep_w4_pack.argtypes = [w4] + [vp] * 4
    _lib.ep_w4_linear.argtypes = [w4] + [vp] * 6
    _lib.ep_expert_ffn_w4.argtypes = [ffn, i32] + [vp] * 11
    _lib.ep_combine_backward.argtypes = [layer] + [vp] * 7
    _lib.ep_route_backward.argtypes = [layer] + [vp] * 6
    _lib.ep_grad_workspace_size.argtypes = [i32, P(size)]
    _lib.ep_grad_norm.argtypes = [grads, i32, vp, vp, size, vp]
    _lib.ep_grad_clip.argtypes = [grads, i32, ctypes.c_float, vp, vp, size, vp]
    _lib.ep_grad_clip_with_norm.argtypes = [grads, i32, ctypes.c_float, vp, vp]
    _lib.ep_expert_ffn.argtypes = [ffn] + [vp] * 10
    _lib.ep_expert_ffn_backward.argtypes = [ffn] + [vp] * 16
    for name in EXPORTS:
        getattr(_lib, name).restype = ctypes.c_int


_declare()


def _bf16(t, shape, name, device=None):
    return _ptr(t, torch.bfloat16, shape, name, device)


def _saved(cfg, t, shape, name, device=None):
    """g or u: a bfloat16 tensor where cfg.saved_bf16 is 1; else a float16 one, or a bfloat16 one as mere memory for
    the halves, of which nobody reads the values."""
    bf16 = cfg.saved_bf16 == 1 or t is not None and t.dtype is torch.bfloat16
    return _ptr(t, torch.bfloat16 if bf16 else torch.float16, shape, name, device)


def ep_expert_ffn(cfg: EpFfnConfig, rows, expert_offset, w_gate, w_up, w_down, h, y, g=None, u=None,
                  stream=None) -> None:
    """y = (silu(rows Wg^T) * (rows Wu^T)) Wd^T with each row's own expert; h is the product before Wd.

    rows, y bf16 [rows, H]; h bf16 [rows, I]; w_gate, w_up bf16 [E, I, H]; w_down bf16 [E, H, I]; expert_offset
    int32 [E + 1]. g and u ([rows, I], both or neither) are what ep_expert_ffn_backward needs besides h: bfloat16
    where cfg.saved_bf16 is 1, else float16. Without it they are written as halves into bfloat16 tensors too, which
    are then storage only: their values mean nothing."""
    S, H, I, E = cfg.rows, cfg.H, cfg.I, cfg.E
    dev = _device()
    _check(_lib.ep_expert_ffn(ctypes.byref(cfg), _bf16(rows, (S, H), "rows", dev),
                              _ptr(expert_offset, torch.int32, (E + 1,), "expert_offset", dev),
                              _bf16(w_gate, (E, I, H), "w_gate", dev), _bf16(w_up, (E, I, H), "w_up", dev),
                              _bf16(w_down, (E, H, I), "w_down", dev), _saved(cfg, g, (S, I), "g", dev), _saved(cfg, u, (S, I), "u", dev),
                              _bf16(h, (S, I), "h", dev), _bf16(y, (S, H), "y", dev), _stream(stream)), "ep_expert_ffn")


def ep_expert_ffn_backward(cfg: EpFfnConfig, rows, expert_offset, w_gate, w_up, w_down, g, u, h, d_y, d_g, d_u,
                           d_rows=None, d_w_gate=None, d_w_up=None, d_w_down=None, stream=None) -> None:
    """Gradients of ep_expert_ffn for d_y, the gradient of y, from the g, u and h that it wrote with the same cfg. d_g
    and d_u bf16 [rows, I] are written on the way; d_rows and the weights' gradients (overwritten) are written
    where they are given."""
    S, H, I, E = cfg.rows, cfg.H, cfg.I, cfg.E
    dev = _device()
    _check(_lib.ep_expert_ffn_backward(
        ctypes.byref(cfg), _bf16(rows, (S, H), "rows", dev), _ptr(expert_offset, torch.int32, (E + 1,), "expert_offset", dev),
        _bf16(w_gate, (E, I, H), "w_gate", dev), _bf16(w_up, (E, I, H), "w_up", dev), _bf16(w_down, (E, H, I), "w_down", dev),
        _saved(cfg, g, (S, I), "g", dev), _saved(cfg, u, (S, I), "u", dev), _bf16(h, (S, I), "h", dev), _bf16(d_y, (S, H), "d_y", dev),
        _bf16(d_g, (S, I), "d_g", dev), _bf16(d_u, (S, I), "d_u", dev), _bf16(d_rows, (S, H), "d_rows", dev),
        _bf16(d_w_gate, (E, I, H), "d_w_gate", dev), _bf16(d_w_up, (E, I, H), "d_w_up", dev),
        _bf16(d_w_down, (E, H, I), "d_w_down", dev), _stream(stream)), "ep_expert_ffn_backward")


def ep_w4_sizes(cfg: EpW4Config) -> tuple[int, int]:
    """Bytes of a packed weight's q and scale."""
    q, s = ctypes.c_size_t(0), ctypes.c_size_t(0)
    _check(_lib.ep_w4_sizes(ctypes.byref(cfg), ctypes.byref(q), ctypes.byref(s)), "ep_w4_sizes")
    return q.value, s.value


def _packed(cfg: EpW4Config, q, scale, name, device=None):
    """Pointers of a packed weight: q uint8 [E, N, Kp / 2], scale bf16 [E, N, Kp / group]."""
    Kp = (cfg.K + 127) // 128 * 128
    return (_ptr(q, torch.uint8, (cfg.E, cfg.N, Kp // 2), "q" + name, device),
            _bf16(scale, (cfg.E, cfg.N, Kp // max(cfg.group, 1)), "scale" + name, device))


def ep_w4_pack(cfg: EpW4Config, w, q, scale, stream=None) -> None:
    """w bf16 [E, N, K] -> q uint8 [E, N, Kp / 2], scale bf16 [E, N, Kp / group]; Kp is K filled up to 128."""
    _check(_lib.ep_w4_pack(ctypes.byref(cfg), _bf16(w, (cfg.E, cfg.N, cfg.K), "w"), *_packed(cfg, q, scale, ""),
                           _stream(stream)), "ep_w4_pack")


def ep_w4_linear(cfg: EpW4Config, x, expert_offset, q, scale, y, stream=None) -> None:
    """y[s] = W[e(s)] x[s] with packed 4-bit weights; x bf16 [rows, K], y bf16 [rows, N]."""
    dev = _device()
    _check(_lib.ep_w4_linear(ctypes.byref(cfg), _bf16(x, (cfg.rows, cfg.K), "x", dev),
                             _ptr(expert_offset, torch.int32, (cfg.E + 1,), "expert_offset", dev),
                             *_packed(cfg, q, scale, "", dev), _bf16(y, (cfg.rows, cfg.N), "y", dev), _stream(stream)),
           "ep_w4_linear")


def ep_expert_ffn_w4(cfg: EpFfnConfig, group: int, rows, expert_offset, q_gate, s_gate, q_up, s_up, q_down, s_down, h,
                     y, stream=None) -> None:
    """ep_expert_ffn's forward pass with packed 4-bit weights."""
    S, H, I, E = cfg.rows, cfg.H, cfg.I, cfg.E
    wide = EpW4Config.make(N=I, K=H, E=E, group=group)
    down = EpW4Config.make(N=H, K=I, E=E, group=group)
    dev = _device()
    _check(_lib.ep_expert_ffn_w4(ctypes.byref(cfg), ctypes.c_int32(group), _bf16(rows, (S, H), "rows", dev),
                                 _ptr(expert_offset, torch.int32, (E + 1,), "expert_offset", dev),
                                 *_packed(wide, q_gate, s_gate, "_gate", dev), *_packed(wide, q_up, s_up, "_up", dev),
                                 *_packed(down, q_down, s_down, "_down", dev), _bf16(h, (S, I), "h", dev),
                                 _bf16(y, (S, H), "y", dev), _stream(stream)), "ep_expert_ffn_w4")


def ep_combine_backward(cfg: EpConfig, d_out, y, slot, topk_w, d_y, d_topk_w, stream=None) -> None:
    """d_out bf16 [T, H], y bf16 [T*k, H] -> d_y bf16 [T*k, H] (slot order), d_topk_w fp32 [T, k]."""
    T, H, k = cfg.T, cfg.H, cfg.k
    dev = _device()
    _check(_lib.ep_combine_backward(ctypes.byref(cfg), _bf16(d_out, (T, H), "d_out", dev), _bf16(y, (T * k, H), "y", dev),
                                    _ptr(slot, torch.int32, (T, k), "slot", dev),
                                    _ptr(topk_w, torch.float32, (T, k), "topk_w", dev), _bf16(d_y, (T * k, H), "d_y", dev),
                                    _ptr(d_topk_w, torch.float32, (T, k), "d_topk_w", dev), _stream(stream)),
           "ep_combine_backward")


def ep_route_backward(cfg: EpConfig, logits, topk_idx, topk_w, d_topk_w, d_logits, stream=None) -> None:
    """d_topk_w fp32 [T, k] -> d_logits fp32 [T, E]; logits may be None where cfg.renormalize is 1."""
    T, E, k = cfg.T, cfg.E, cfg.k
    dev = _device()
    _check(_lib.ep_route_backward(ctypes.byref(cfg), _ptr(logits, torch.float32, (T, E), "logits", dev),
                                  _ptr(topk_idx, torch.int32, (T, k), "topk_idx", dev),
                                  _ptr(topk_w, torch.float32, (T, k), "topk_w", dev),
                                  _ptr(d_topk_w, torch.float32, (T, k), "d_topk_w", dev),
                                  _ptr(d_logits, torch.float32, (T, E), "d_logits", dev), _stream(stream)),
           "ep_route_backward")


_GRAD_TYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
_GRAD_RECORD = np.dtype([("data", np.uint64), ("out", np.uint64), ("numel", np.int64), ("dtype", np.int32),
                         ("reserved", np.int32)])  # EpGradTensor


def _address(ptr) -> int:
    """What _ptr gave, as a number."""
    return (ptr.value if isinstance(ptr, ctypes.c_void_p) else ptr) or 0


def ep_grad_workspace_size(n: int) -> int:
    b = ctypes.c_size_t(0)
    _check(_lib.ep_grad_workspace_size(n, ctypes.byref(b)), "ep_grad_workspace_size")
    return b.value


class GradList:
    """A list of gradient tensors with its C records and workspace.

    ``out``: where the clipped values go (same shapes and types); the tensors themselves if None.

    A list names the memory that its tensors have when it is made, and keeps that memory alive. It serves every
    step that writes the gradients in place. Where they come in new memory (``zero_grad(set_to_none=True)``,
    ``p.grad = ...``, ``p.grad.data = ...``) make a new list every step: an old one goes on naming the old memory.
    Making one takes 0.5 us a tensor on the host (1 with ``out``), before the calls below. The calls of one list share its
    workspace: they must not run at the same time, on two streams for instance."""

    def __init__(self, grads, out=None):
        grads = list(grads)
        out = grads if out is None else list(out)
        if len(out) != len(grads):
            raise ValueError(f"out: {len(out)} tensors for {len(grads)} gradients")
        self.n = len(grads)
        self.records = (EpGradTensor * max(self.n, 1))()
        table = np.frombuffer(self.records, dtype=_GRAD_RECORD)[:self.n]
        device = torch.cuda.current_device() if torch.cuda.is_initialized() else -2  # -1: the CPU
        usual = lambda ts: (set(map(type, ts)) <= {torch.Tensor} and set(map(torch.Tensor.get_device, ts)) <= {device}  # noqa: E731
                            and all(map(torch.Tensor.is_contiguous, ts)))
        fast = usual(grads) and (out is grads or usual(out))
        types = [g.dtype for g in grads] if fast else []
        if fast and set(types) <= _GRAD_TYPES.keys() and (out is grads or [o.dtype for o in out] == types
                                                          and all(g.shape == o.shape for g, o in zip(grads, out))):
            table["data"] = list(map(torch.Tensor.data_ptr, grads))
            table["out"] = table["data"] if out is grads else list(map(torch.Tensor.data_ptr, out))
        else:  # says which tensor is wrong
            for i, (g, o) in enumerate(zip(grads, out)):
                if not isinstance(g, torch.Tensor) or g.dtype not in _GRAD_TYPES:
                    raise TypeError(f"grads[{i}]: expected a float32, bfloat16 or float16 tensor")
                table["data"][i] = _address(_ptr(g, g.dtype, None, f"grads[{i}]"))
                table["out"][i] = _address(_ptr(o, g.dtype, tuple(g.shape), f"out[{i}]"))
        # of a tensor itself `.data = ...` would free the memory that the record names
        self._keep = list(map(torch.Tensor.untyped_storage, grads if out is grads else grads + out))
        table["numel"] = list(map(torch.Tensor.numel, grads))
        table["dtype"] = [_GRAD_TYPES[g.dtype] for g in grads]
        self.workspace = torch.empty((ep_grad_workspace_size(self.n),), dtype=torch.uint8, device="cuda")

    def norm(self, norm, stream=None) -> None:
        ep_grad_norm(self, norm, stream)

    def clip(self, max_norm: float, norm, stream=None) -> None:
        ep_grad_clip(self, max_norm, norm, stream)

    def clip_with_norm(self, max_norm: float, norm, stream=None) -> None:
        ep_grad_clip_with_norm(self, max_norm, norm, stream)


def ep_grad_norm(grads: GradList, norm, stream=None) -> None:
    """norm fp32 [1]: the 2-norm over all values of all tensors of the list."""
    ws = grads.workspace
    _check(_lib.ep_grad_norm(grads.records, grads.n, _ptr(norm, torch.float32, (1,), "norm"),
                             _ptr(ws, torch.uint8, None, "workspace"), ws.numel(), _stream(stream)), "ep_grad_norm")


def ep_grad_clip(grads: GradList, max_norm: float, norm, stream=None) -> None:
    """The norm, and every tensor times min(1, max_norm / (norm + 1e-6)) to its ``out``."""
    ws = grads.workspace
    _check(_lib.ep_grad_clip(grads.records, grads.n, float(max_norm), _ptr(norm, torch.float32, (1,), "norm"),
                             _ptr(ws, torch.uint8, None, "workspace"), ws.numel(), _stream(stream)), "ep_grad_clip")


def ep_grad_clip_with_norm(grads: GradList, max_norm: float, norm, stream=None) -> None:
    """Every tensor times min(1, max_norm / (norm + 1e-6)) to its ``out``, norm fp32 [1] given: that of all processes'
    gradients, for instance (``exchange.reduce_grad_norm``)."""
    _check(_lib.ep_grad_clip_with_norm(grads.records, grads.n, float(max_norm), _ptr(norm, torch.float32, (1,), "norm"),
                                       _stream(stream)), "ep_grad_clip_with_norm")
