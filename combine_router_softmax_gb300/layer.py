"""Binding of ``include/ep_layer.h``: what surrounds an MoE layer in a model and its training.

Like the rest of the binding this only marshals arguments: every function has
the name of its C entry point, checks dtype, shape and device of each tensor,
passes the current CUDA stream and raises :class:`EpError` on a non-zero
status. The package re-exports everything here.
"""
from __future__ import annotations

import ctypes

import torch

from . import EpConfig, _check, _device, _lib, _ptr, _stream

EXPORTS = ("ep_block_norm", "ep_block_norm_workspace_size", "ep_block_norm_backward", "ep_balance_workspace_size",
           "ep_balance", "ep_balance_backward", "ep_orthogonalize_workspace_size", "ep_orthogonalize")
__all__ = [*EXPORTS, "EpNormConfig", "EpOrthoConfig", "EP_GATE_NONE", "EP_GATE_CHANNEL", "EP_GATE_TOKEN", "EP_GATE_ELEMENT"]

EP_GATE_NONE, EP_GATE_CHANNEL, EP_GATE_TOKEN, EP_GATE_ELEMENT = range(4)


class EpNormConfig(ctypes.Structure):
    """``ep_norm_config`` of include/ep_layer.h."""
    _fields_ = [*((n, ctypes.c_int32) for n in ("T", "H", "gate", "gate_sigmoid", "residual_f32")),
                *((n, ctypes.c_float) for n in ("eps", "scale", "weight_offset"))]

    @classmethod
    def make(cls, *, T, H, gate=EP_GATE_NONE, gate_sigmoid=0, residual_f32=0, eps=1e-6, scale=1.0,
             weight_offset=0.0) -> "EpNormConfig":
        return cls(T, H, gate, gate_sigmoid, residual_f32, eps, scale, weight_offset)


_ORTHO_TYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}


class EpOrthoConfig(ctypes.Structure):
    """``ep_ortho_config`` of include/ep_layer.h; ``dtype`` of make(): torch.float32, bfloat16 or float16."""
    _fields_ = [*((n, ctypes.c_int32) for n in ("B", "N", "K", "dtype", "steps")), ("eps", ctypes.c_float)]

    @classmethod
    def make(cls, *, B=1, N, K, dtype=torch.bfloat16, steps=5, eps=1e-7) -> "EpOrthoConfig":
        if dtype not in _ORTHO_TYPES:
            raise TypeError(f"dtype {dtype}: expected float32, bfloat16 or float16")
        return cls(B, N, K, _ORTHO_TYPES[dtype], steps, eps)


def _declare() -> None:
    P, vp, size = ctypes.POINTER, ctypes.c_void_p, ctypes.c_size_t
    norm = P(EpNormConfig)
    _lib.ep_block_norm.argtypes = [norm] + [vp] * 10
    _lib.ep_block_norm_workspace_size.argtypes = [norm, P(size)]
    _lib.ep_block_norm_backward.argtypes = [norm] + [vp] * 15 + [size, vp]
    layer, i32 = P(EpConfig), ctypes.c_int32
    _lib.ep_balance_workspace_size.argtypes = [layer, i32, P(size)]
    _lib.ep_balance.argtypes = [layer, i32] + [vp] * 9 + [size, vp]
    _lib.ep_balance_backward.argtypes = [layer, i32] + [vp] * 8
    ortho = P(EpOrthoConfig)
    _lib.ep_orthogonalize_workspace_size.argtypes = [ortho, P(size)]
    _lib.ep_orthogonalize.argtypes = [ortho, P(ctypes.c_float), vp, vp, vp, size, vp]
    for name in EXPORTS:
        getattr(_lib, name).restype = ctypes.c_int


_declare()

_BF16, _F32, _I32 = torch.bfloat16, torch.float32, torch.int32


def _gate(cfg, t, name, device, gradient=False):
    """Pointer of a gate, or of its gradient."""
    if t is None:
        return None
    T, H = cfg.T, cfg.H
    kinds = {EP_GATE_CHANNEL: (_F32 if gradient else _BF16, (H,)), EP_GATE_TOKEN: (_F32, (T,)), EP_GATE_ELEMENT: (_BF16, (T, H))}
    if cfg.gate not in kinds:
        raise ValueError(f"{name}: cfg.gate is {cfg.gate}")
    return _ptr(t, *kinds[cfg.gate], name, device)


def _workspace(ws, device):
    return (None, 0) if ws is None else (_ptr(ws, torch.uint8, None, "workspace", device), ws.numel())


def ep_block_norm(cfg: EpNormConfig, x, y=None, w_post=None, gate=None, w_next=None, out=None, n=None, rstd_post=None,
                  rstd_next=None, stream=None) -> None:
    """out = x + scale act(gate) norm(y, w_post), n = norm(out, w_next); without y: n = norm(x, w_next).

    x, out bf16 or (cfg.residual_f32) float32 [T, H], out may be x; y, n bf16 [T, H]; w_post, w_next bf16 [H], None for no
    norm; gate bf16 [H], float32 [T] or bf16 [T, H] by cfg.gate; rstd_post, rstd_next float32 [T], optional, for the
    backward pass."""
    T, H = cfg.T, cfg.H
    dev = _device()
    row = _F32 if cfg.residual_f32 == 1 else _BF16
    _check(_lib.ep_block_norm(ctypes.byref(cfg), _ptr(x, row, (T, H), "x", dev), _ptr(y, _BF16, (T, H), "y", dev),
                              _ptr(w_post, _BF16, (H,), "w_post", dev), _gate(cfg, gate, "gate", dev),
                              _ptr(w_next, _BF16, (H,), "w_next", dev), _ptr(out, row, (T, H), "out", dev),
                              _ptr(n, _BF16, (T, H), "n", dev), _ptr(rstd_post, _F32, (T,), "rstd_post", dev),
                              _ptr(rstd_next, _F32, (T,), "rstd_next", dev), _stream(stream)), "ep_block_norm")


def ep_block_norm_workspace_size(cfg: EpNormConfig) -> int:
    """Bytes of the workspace of ep_block_norm_backward."""
    b = ctypes.c_size_t(0)
    _check(_lib.ep_block_norm_workspace_size(ctypes.byref(cfg), ctypes.byref(b)), "ep_block_norm_workspace_size")
    return b.value


def ep_block_norm_backward(cfg: EpNormConfig, x, y, w_post, gate, w_next, rstd_post, rstd_next, d_out, d_n, d_x, d_y=None,
                           d_w_post=None, d_gate=None, d_w_next=None, workspace=None, stream=None) -> None:
    """Gradients of ep_block_norm for d_out and d_n (either may be None), from its inputs and the rstd_* that it wrote.

    d_x like x, may be d_out; d_y bf16 [T, H] with y; d_w_post, d_w_next float32 [H], overwritten, and d_gate (float32
    [H] or [T], bf16 [T, H]) where they are given; workspace uint8, for the sums over rows."""
    T, H = cfg.T, cfg.H
    dev = _device()
    row = _F32 if cfg.residual_f32 == 1 else _BF16
    _check(_lib.ep_block_norm_backward(
        ctypes.byref(cfg), _ptr(x, row, (T, H), "x", dev), _ptr(y, _BF16, (T, H), "y", dev),
        _ptr(w_post, _BF16, (H,), "w_post", dev), _gate(cfg, gate, "gate", dev), _ptr(w_next, _BF16, (H,), "w_next", dev),
        _ptr(rstd_post, _F32, (T,), "rstd_post", dev), _ptr(rstd_next, _F32, (T,), "rstd_next", dev),
        _ptr(d_out, row, (T, H), "d_out", dev), _ptr(d_n, _BF16, (T, H), "d_n", dev), _ptr(d_x, row, (T, H), "d_x", dev),
        _ptr(d_y, _BF16, (T, H), "d_y", dev), _ptr(d_w_post, _F32, (H,), "d_w_post", dev),
        _gate(cfg, d_gate, "d_gate", dev, gradient=True), _ptr(d_w_next, _F32, (H,), "d_w_next", dev),
        *_workspace(workspace, dev), _stream(stream)), "ep_block_norm_backward")


def ep_balance_workspace_size(cfg: EpConfig, n_seq: int = 1) -> int:
    """Bytes of the workspace of ep_balance."""
    b = ctypes.c_size_t(0)
    _check(_lib.ep_balance_workspace_size(ctypes.byref(cfg), n_seq, ctypes.byref(b)), "ep_balance_workspace_size")
    return b.value


def ep_balance(cfg: EpConfig, logits, topk_idx, seq_first, seq_len, count, load, prob, loss, workspace, stream=None) -> None:
    """Counts, loads, mean probabilities and the two losses (balance, z) of every sequence.

    logits float32 [T, E], topk_idx int32 [T, k]; seq_first int32 [S + 1] (None: one sequence of all T rows), seq_len
    int32 [S] or None; count int32 [S, E], load and prob float32 [S, E], loss float32 [S, 2]."""
    T, E, k = cfg.T, cfg.E, cfg.k
    S = count.shape[0]
    dev = _device()
    _check(_lib.ep_balance(ctypes.byref(cfg), S, _ptr(logits, _F32, (T, E), "logits", dev),
                           _ptr(topk_idx, _I32, (T, k), "topk_idx", dev), _ptr(seq_first, _I32, (S + 1,), "seq_first", dev),
                           _ptr(seq_len, _I32, (S,), "seq_len", dev), _ptr(count, _I32, (S, E), "count", dev),
                           _ptr(load, _F32, (S, E), "load", dev), _ptr(prob, _F32, (S, E), "prob", dev),
                           _ptr(loss, _F32, (S, 2), "loss", dev), *_workspace(workspace, dev), _stream(stream)),
           "ep_balance")


def ep_balance_backward(cfg: EpConfig, logits, seq_first, seq_len, load, d_loss, d_in, d_logits, stream=None) -> None:
    """d_logits = d_in (None: 0) + the gradient of the losses' sum with the weights d_loss float32 [S, 2]; d_logits may be d_in."""
    T, E = cfg.T, cfg.E
    S = load.shape[0]
    dev = _device()
    _check(_lib.ep_balance_backward(ctypes.byref(cfg), S, _ptr(logits, _F32, (T, E), "logits", dev),
                                    _ptr(seq_first, _I32, (S + 1,), "seq_first", dev), _ptr(seq_len, _I32, (S,), "seq_len", dev),
                                    _ptr(load, _F32, (S, E), "load", dev), _ptr(d_loss, _F32, (S, 2), "d_loss", dev),
                                    _ptr(d_in, _F32, (T, E), "d_in", dev), _ptr(d_logits, _F32, (T, E), "d_logits", dev),
                                    _stream(stream)), "ep_balance_backward")


def ep_orthogonalize_workspace_size(cfg: EpOrthoConfig) -> int:
    """Bytes of the workspace of ep_orthogonalize."""
    b = ctypes.c_size_t(0)
    _check(_lib.ep_orthogonalize_workspace_size(ctypes.byref(cfg), ctypes.byref(b)), "ep_orthogonalize_workspace_size")
    return b.value


def ep_orthogonalize(cfg: EpOrthoConfig, m, out, workspace, coefficients=None, stream=None) -> None:
    """out = each matrix of m with its singular values drawn towards one, by cfg.steps Newton-Schulz steps.

    m [B, N, K] (float32, bfloat16 or float16, as cfg says), out bf16 [B, N, K], may be m where that is of 16 bits; coefficients: a sequence of
    cfg.steps triples (a, b, c), None for the default."""
    shape = (cfg.B, cfg.N, cfg.K)
    dev = _device()
    types = {v: t for t, v in _ORTHO_TYPES.items()}
    k = None
    if coefficients is not None:
        flat = [float(v) for step in coefficients for v in step]
        if len(flat) != 3 * cfg.steps:
            raise ValueError(f"coefficients: {len(flat)} values, expected {cfg.steps} triples")
        k = (ctypes.c_float * max(len(flat), 1))(*flat)
    _check(_lib.ep_orthogonalize(ctypes.byref(cfg), k, _ptr(m, types.get(cfg.dtype, _F32), shape, "m", dev),
                                 _ptr(out, _BF16, shape, "out", dev), *_workspace(workspace, dev), _stream(stream)),
           "ep_orthogonalize")
