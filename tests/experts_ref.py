"""The experts' block in 64 bits, and how far a bf16 kernel with fp32 sums may be from it.

Every bound is a worst case that counts roundings: 2^-8 for one rounding to bf16,
2^-11 (and 2^-25 below the normal range) for one to fp16, which g and u are kept in, and for a sum of n terms in fp32, n 2^-23 of the sum of their magnitudes
(products of bf16 values are exact in fp32; an accumulation step is off by at most
one unit in the last place, whichever way it rounds). silu' stays within 1.1 and
silu'' within 0.5 in magnitude; the sigmoid itself is within 2^-20. Terms of
second order are covered by the factor SLACK."""
from __future__ import annotations

import torch

U16, U11, U32, SIG, SLACK = 2.0**-8, 2.0**-11, 2.0**-23, 2.0**-20, 1.05


def silu_parts(g):
    s = 1 / (1 + torch.exp(-g))
    return s, g * s, s * (1 + g * (1 - s))


def forward(x, wg, wu, wd):
    """One expert, float64: dict of values, and 'tol_' + name their bounds."""
    r = {"g": x @ wg.T, "u": x @ wu.T}
    H, I = wg.shape[1], wg.shape[0]
    eg, eu = H * U32 * (x.abs() @ wg.abs().T), H * U32 * (x.abs() @ wu.abs().T)
    _, silu, _ = silu_parts(r["g"])
    r["h"] = silu * r["u"]
    r["y"] = r["h"] @ wd.T
    r["tol_g"], r["tol_u"] = (SLACK * (U11 * r[k].abs() + e) + 2.0**-25 for k, e in (("g", eg), ("u", eu)))
    r["tol_h"] = SLACK * ((U16 + SIG) * r["h"].abs() + 1.1 * r["u"].abs() * eg + silu.abs() * eu)
    r["tol_y"] = SLACK * (r["tol_h"] @ wd.abs().T + I * U32 * (r["h"].abs() @ wd.abs().T) + U16 * r["y"].abs())
    return r


def backward(x, wg, wu, wd, dy, f):
    """The gradients for dy, from forward()'s values and the bounds they already have."""
    H, I, n = wg.shape[1], wg.shape[0], x.shape[0]
    dh = dy @ wd
    edh = H * U32 * (dy.abs() @ wd.abs())
    s, silu, d = silu_parts(f["g"])
    r = {"d_u": dh * silu, "d_g": dh * f["u"] * d}
    r["tol_d_u"] = SLACK * (silu.abs() * edh + 1.1 * dh.abs() * f["tol_g"] + (U16 + SIG) * r["d_u"].abs())
    r["tol_d_g"] = SLACK * ((f["u"] * d).abs() * edh + (dh * d).abs() * f["tol_u"]
                            + 0.5 * (dh * f["u"]).abs() * f["tol_g"] + U16 * r["d_g"].abs()
                            + SIG * (dh * f["u"]).abs() * (1 + f["g"].abs()))
    r["d_rows"] = r["d_g"] @ wg + r["d_u"] @ wu
    r["tol_d_rows"] = SLACK * (r["tol_d_g"] @ wg.abs() + r["tol_d_u"] @ wu.abs() + U16 * r["d_rows"].abs()
                               + 2 * I * U32 * (r["d_g"].abs() @ wg.abs() + r["d_u"].abs() @ wu.abs()))
    for name, a, ta, b, tb in (("d_w_gate", r["d_g"], r["tol_d_g"], x, None),
                               ("d_w_up", r["d_u"], r["tol_d_u"], x, None),
                               ("d_w_down", dy, None, f["h"], f["tol_h"])):
        r[name] = a.T @ b
        off = ta.T @ b.abs() if ta is not None else a.abs().T @ tb
        r["tol_" + name] = SLACK * (off + n * U32 * (a.abs().T @ b.abs()) + U16 * r[name].abs())
    return r


def check(got, want, tol, what):
    got = got.double()
    assert torch.isfinite(got).all(), f"{what}: not finite"
    off = (got - want).abs()
    worst = (off - tol).max().item()
    assert worst <= 0, f"{what}: {int((off > tol).sum())} of {off.numel()} values beyond their bound, worst by {worst:g}"
    # in the mean: one rounding of the result and at most one of what went into it
    if want.numel() >= 4096:
        assert (off.norm() <= 2.0**-7 * want.norm()).item(), f"{what}: off by {(off.norm() / want.norm()).item():g} in norm"
