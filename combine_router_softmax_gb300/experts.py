"""Binding of ``include/ep_experts.h``: the experts between dispatch and combine, and the way back.

Like the rest of the binding this only marshals arguments: every function has
the name of its C entry point, checks dtype, shape and device of each tensor,
passes the current CUDA stream and raises :class:`EpError` on a non-zero
status. The package re-exports everything here.
"""
from __future__ import annotations

import ctypes
from dataclasses import dataclass

import torch

from . import _check, _lib, _ptr, _stream

__all__ = ["EpFfnConfig", "ep_expert_ffn", "ep_expert_ffn_backward"]

EXPORTS = ("ep_expert_ffn", "ep_expert_ffn_backward")


class EpFfnConfig(ctypes.Structure):
    """``ep_ffn_config`` of include/ep_experts.h."""
    _fields_ = [(n, ctypes.c_int32) for n in ("rows", "H", "I", "E")]

    @classmethod
    def make(cls, *, rows, H, I, E) -> "EpFfnConfig":
        return cls(rows, H, I, E)


def _declare() -> None:
    P, vp = ctypes.POINTER, ctypes.c_void_p
    ffn = P(EpFfnConfig)
    _lib.ep_expert_ffn.argtypes = [ffn] + [vp] * 10
    _lib.ep_expert_ffn_backward.argtypes = [ffn] + [vp] * 16
    for name in EXPORTS:
        getattr(_lib, name).restype = ctypes.c_int


_declare()


def _bf16(t, shape, name):
    return _ptr(t, torch.bfloat16, shape, name)


def ep_expert_ffn(cfg: EpFfnConfig, rows, expert_offset, w_gate, w_up, w_down, h, y, g=None, u=None,
                  stream=None) -> None:
    """y = (silu(rows Wg^T) * (rows Wu^T)) Wd^T with each row's own expert; h is the product before Wd.

    rows, y bf16 [rows, H]; h, g, u bf16 [rows, I]; w_gate, w_up bf16 [E, I, H]; w_down bf16 [E, H, I];
    expert_offset int32 [E + 1]. g and u (both or neither) are what ep_expert_ffn_backward needs besides h."""
    S, H, I, E = cfg.rows, cfg.H, cfg.I, cfg.E
    _check(_lib.ep_expert_ffn(ctypes.byref(cfg), _bf16(rows, (S, H), "rows"),
                              _ptr(expert_offset, torch.int32, (E + 1,), "expert_offset"),
                              _bf16(w_gate, (E, I, H), "w_gate"), _bf16(w_up, (E, I, H), "w_up"),
                              _bf16(w_down, (E, H, I), "w_down"), _bf16(g, (S, I), "g"), _bf16(u, (S, I), "u"),
                              _bf16(h, (S, I), "h"), _bf16(y, (S, H), "y"), _stream(stream)), "ep_expert_ffn")


def ep_expert_ffn_backward(cfg: EpFfnConfig, rows, expert_offset, w_gate, w_up, w_down, g, u, h, d_y, d_g, d_u,
                           d_rows=None, d_w_gate=None, d_w_up=None, d_w_down=None, stream=None) -> None:
    """Gradients of ep_expert_ffn for d_y, the gradient of y. d_g and d_u bf16 [rows, I] are written on the
    way; d_rows and the weights' gradients (overwritten) are written where they are given."""
    S, H, I, E = cfg.rows, cfg.H, cfg.I, cfg.E
    _check(_lib.ep_expert_ffn_backward(
        ctypes.byref(cfg), _bf16(rows, (S, H), "rows"), _ptr(expert_offset, torch.int32, (E + 1,), "expert_offset"),
        _bf16(w_gate, (E, I, H), "w_gate"), _bf16(w_up, (E, I, H), "w_up"), _bf16(w_down, (E, H, I), "w_down"),
        _bf16(g, (S, I), "g"), _bf16(u, (S, I), "u"), _bf16(h, (S, I), "h"), _bf16(d_y, (S, H), "d_y"),
        _bf16(d_g, (S, I), "d_g"), _bf16(d_u, (S, I), "d_u"), _bf16(d_rows, (S, H), "d_rows"),
        _bf16(d_w_gate, (E, I, H), "d_w_gate"), _bf16(d_w_up, (E, I, H), "d_w_up"),
        _bf16(d_w_down, (E, H, I), "d_w_down"), _stream(stream)), "ep_expert_ffn_backward")
