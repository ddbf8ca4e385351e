"""The entry points of include/ep_layer.h reject bad arguments on the host, with nothing
enqueued. CPU only: no call here reaches a kernel launch."""
import ctypes

import pytest
import torch

F = ctypes.c_void_p(0x10000)  # 16-byte aligned, never dereferenced: every call below fails its checks first
ODD8, ODD2 = ctypes.c_void_p(0x10008), ctypes.c_void_p(0x10002)
BIG = 1 << 40


@pytest.fixture(scope="module")
def ep():
    import __graft_entry__

    __graft_entry__._cuda_build_module().build()
    import combine_router_softmax_gb300 as m

    return m


def expected(ep, kind):
    return {"INVALID": ep.EP_ERR_INVALID_ARG, "UNSUPPORTED": ep.EP_ERR_UNSUPPORTED, "CAPACITY": ep.EP_ERR_CAPACITY}[kind]


# Norms ------------------------------------------------------------------------

FORWARD = dict(x=F, y=F, w_post=F, gate=None, w_next=F, out=F, n=F, rstd_post=F, rstd_next=F)
BACKWARD = dict(x=F, y=F, w_post=F, gate=None, w_next=F, rstd_post=F, rstd_next=F, d_out=F, d_n=F, d_x=F, d_y=F, d_w_post=F,
                d_gate=None, d_w_next=F, workspace=F)


def norm_cfg(ep, **kw):
    return ep.EpNormConfig.make(**{**dict(T=5, H=64), **kw})


def forward(ep, cfg, **kw):
    return ep._lib.ep_block_norm(None if cfg is None else ctypes.byref(cfg), *{**FORWARD, **kw}.values(), None)


def backward(ep, cfg, nbytes=BIG, **kw):
    return ep._lib.ep_block_norm_backward(None if cfg is None else ctypes.byref(cfg), *{**BACKWARD, **kw}.values(), nbytes, None)


@pytest.mark.parametrize("bad,expect", [
    (dict(T=-1), "INVALID"), (dict(H=0), "INVALID"), (dict(H=-8), "INVALID"), (dict(gate=4), "INVALID"),
    (dict(gate=-1), "INVALID"), (dict(gate_sigmoid=2), "INVALID"), (dict(residual_f32=-1), "INVALID"),
    (dict(eps=-1e-6), "INVALID"), (dict(eps=float("nan")), "INVALID"), (dict(eps=float("inf")), "INVALID"),
    (dict(scale=float("nan")), "INVALID"), (dict(weight_offset=float("inf")), "INVALID"),
    (dict(H=12), "UNSUPPORTED"), (dict(H=16392), "UNSUPPORTED"),
])
def test_norm_shapes(ep, bad, expect):
    want = expected(ep, expect)
    cfg = norm_cfg(ep, **bad)
    assert forward(ep, cfg) == want and backward(ep, cfg) == want
    assert ep._lib.ep_block_norm_workspace_size(ctypes.byref(cfg), ctypes.byref(ctypes.c_size_t(0))) == want


def test_norm_pointers(ep):
    bad = ep.EP_ERR_INVALID_ARG
    cfg = norm_cfg(ep)
    assert forward(ep, None) == bad and backward(ep, None) == bad
    assert ep._lib.ep_block_norm_workspace_size(ctypes.byref(cfg), None) == bad
    for k, v in FORWARD.items():
        if v is not None:
            assert forward(ep, cfg, **{k: ODD2 if k.startswith("rstd") else ODD8}) == bad, k
    for k, v in BACKWARD.items():
        if v is not None:
            assert backward(ep, cfg, **{k: ODD2 if k.startswith("rstd") else ODD8}) == bad, k
    # what has to come together
    for miss in ("x", "y", "out", "n", "w_next"):
        assert forward(ep, cfg, **{miss: None}) == bad, miss
    assert forward(ep, cfg, w_post=None) == bad                       # rstd_post of no norm
    assert forward(ep, cfg, n=None, w_next=None) == bad               # rstd_next of no norm
    alone = dict(y=None, w_post=None, out=None, rstd_post=None)
    assert forward(ep, cfg, **alone, n=None, w_next=None, rstd_next=None) == bad  # nothing to do
    for more in (dict(w_post=F), dict(out=F), dict(gate=F)):
        assert forward(ep, cfg, **{**alone, **more}) == bad
    for miss in ("x", "y", "w_post", "w_next", "rstd_post", "rstd_next", "d_n", "d_x", "d_y", "workspace"):
        assert backward(ep, cfg, **{miss: None}) == bad, miss
    no_next = dict(w_next=None, rstd_next=None, d_n=None, d_w_next=None)
    assert backward(ep, cfg, **no_next, d_out=None) == bad            # no gradient at all
    assert backward(ep, cfg, **{**no_next, "d_w_next": F}) == bad     # of no weight
    assert backward(ep, cfg, w_post=None, rstd_post=None) == bad      # d_w_post of no weight
    assert backward(ep, cfg, nbytes=ep.ep_block_norm_workspace_size(cfg) - 1) == ep.EP_ERR_CAPACITY


@pytest.mark.parametrize("kind", [1, 2, 3])
def test_norm_gates(ep, kind):
    bad = ep.EP_ERR_INVALID_ARG
    cfg = norm_cfg(ep, gate=kind)
    assert forward(ep, cfg) == bad and backward(ep, cfg) == bad       # without one
    off = ODD2 if kind == 2 else ODD8
    assert forward(ep, cfg, gate=off) == bad and backward(ep, cfg, gate=off) == bad
    assert backward(ep, cfg, gate=F, d_gate=off) == bad
    assert forward(ep, cfg, y=None, w_post=None, out=None, rstd_post=None) == bad  # of nothing
    plain = norm_cfg(ep)
    assert forward(ep, plain, gate=F) == bad and backward(ep, plain, gate=F) == bad
    assert backward(ep, plain, d_gate=F) == bad


def test_norm_without_rows_needs_nothing(ep):
    cfg = norm_cfg(ep, T=0)
    assert forward(ep, cfg, **dict.fromkeys(FORWARD)) == ep.EP_OK
    assert backward(ep, cfg, 0, **dict.fromkeys(BACKWARD)) == ep.EP_OK


def test_norm_workspace(ep):
    for T, H in ((0, 8), (1, 64), (100, 7168), (100000, 16384)):
        n = ep.ep_block_norm_workspace_size(norm_cfg(ep, T=T, H=H))
        assert 0 <= n <= 2 * 4 * H * min(T, 1216) and (n > 0) == (T > 0)


def test_norm_binding_checks_tensors(ep):
    cfg = norm_cfg(ep)
    x, w = torch.zeros((5, 64), dtype=torch.bfloat16), torch.zeros(64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        ep.ep_block_norm(cfg, x, x, w, None, w, x, x)  # on the CPU
    with pytest.raises(TypeError):
        ep.ep_block_norm(cfg, x.float(), x, w, None, w, x, x)
    with pytest.raises(ValueError):
        ep.ep_block_norm(cfg, x, x, w, w, w, x, x)  # a gate where the configuration has none


# Balance ----------------------------------------------------------------------

BAL = dict(logits=F, topk_idx=F, seq_first=F, seq_len=F, count=F, load=F, prob=F, loss=F, workspace=F)
BAL_BWD = dict(logits=F, seq_first=F, seq_len=F, load=F, d_loss=F, d_in=F, d_logits=F)


def layer_cfg(ep, **kw):
    return ep.EpConfig.make(**{**dict(T=40, H=8, E=8, R=1, k=2), **kw})


def balance(ep, cfg, n_seq=3, nbytes=BIG, **kw):
    return ep._lib.ep_balance(None if cfg is None else ctypes.byref(cfg), n_seq, *{**BAL, **kw}.values(), nbytes, None)


def balance_backward(ep, cfg, n_seq=3, **kw):
    return ep._lib.ep_balance_backward(None if cfg is None else ctypes.byref(cfg), n_seq, *{**BAL_BWD, **kw}.values(), None)


@pytest.mark.parametrize("bad,expect", [
    (dict(T=-1), "INVALID"), (dict(E=0), "INVALID"), (dict(k=0), "INVALID"), (dict(k=9), "INVALID"),
    (dict(T=2**30, k=4), "INVALID"), (dict(E=1025), "UNSUPPORTED"), (dict(E=64, k=33), "UNSUPPORTED"),
])
def test_balance_shapes(ep, bad, expect):
    want = expected(ep, expect)
    cfg = layer_cfg(ep, **bad)
    assert balance(ep, cfg) == want and balance_backward(ep, cfg) == want
    assert ep._lib.ep_balance_workspace_size(ctypes.byref(cfg), 1, ctypes.byref(ctypes.c_size_t(0))) == want


def test_balance_pointers(ep):
    bad, cfg = ep.EP_ERR_INVALID_ARG, layer_cfg(ep)
    assert balance(ep, None) == bad and balance_backward(ep, None) == bad
    for n in (0, -1):
        assert balance(ep, cfg, n) == bad and balance_backward(ep, cfg, n) == bad
        assert ep._lib.ep_balance_workspace_size(ctypes.byref(cfg), n, ctypes.byref(ctypes.c_size_t(0))) == bad
    assert ep._lib.ep_balance_workspace_size(ctypes.byref(cfg), 1, None) == bad
    for k in BAL:
        assert balance(ep, cfg, **{k: ODD8 if k == "workspace" else ODD2}) == bad, k
        if k != "seq_len":
            assert balance(ep, cfg, **{k: None}) == bad, k
    for k in BAL_BWD:
        assert balance_backward(ep, cfg, **{k: ODD2}) == bad, k
        if k not in ("seq_len", "d_in"):
            assert balance_backward(ep, cfg, **{k: None}) == bad, k
    # lengths of sequences that have no bounds
    assert balance(ep, cfg, 1, seq_first=None) == bad and balance_backward(ep, cfg, 1, seq_first=None) == bad
    assert balance(ep, cfg, nbytes=ep.ep_balance_workspace_size(cfg, 3) - 1) == ep.EP_ERR_CAPACITY
    assert balance_backward(ep, layer_cfg(ep, T=0), **{k: None for k in BAL_BWD if not k.startswith("seq")}) == ep.EP_OK


def test_balance_binding_checks_tensors(ep):
    cfg = layer_cfg(ep)
    l, idx = torch.zeros((40, 8)), torch.zeros((40, 2), dtype=torch.int32)
    c, f = torch.zeros((1, 8), dtype=torch.int32), torch.zeros((1, 8))
    with pytest.raises(ValueError):
        ep.ep_balance(cfg, l, idx, None, None, c, f, f, torch.zeros((1, 2)), None)  # on the CPU
    with pytest.raises(TypeError):
        ep.ep_balance(cfg, l.double(), idx, None, None, c, f, f, torch.zeros((1, 2)), None)


def test_balance_workspace_of_the_most_rows(ep):
    """Rows of partial sums: one of every tile, 304 at most, and one for every sequence, of 2 E + 1 values."""
    for T in (2**31 - 1, 2**31 - 2**20, 2**30):
        n = ep.ep_balance_workspace_size(layer_cfg(ep, T=T, E=2, k=1), 1)
        assert 300 * 5 * 4 < n <= 305 * 5 * 4, T


# Orthogonalised updates --------------------------------------------------------

def ortho_cfg(ep, **kw):
    base = dict(B=2, N=16, K=24, dtype=1, steps=5, eps=1e-7)
    base.update(kw)
    return ep.EpOrthoConfig(*(base[k] for k in ("B", "N", "K", "dtype", "steps", "eps")))


def ortho(ep, cfg, k=None, m=F, out=F, ws=F, nbytes=BIG):
    return ep._lib.ep_orthogonalize(None if cfg is None else ctypes.byref(cfg), k, m, out, ws, nbytes, None)


@pytest.mark.parametrize("bad,expect", [
    (dict(B=-1), "INVALID"), (dict(N=0), "INVALID"), (dict(K=-3), "INVALID"), (dict(dtype=3), "INVALID"), (dict(dtype=-1), "INVALID"),
    (dict(steps=0), "INVALID"), (dict(eps=-1.0), "INVALID"), (dict(eps=float("nan")), "INVALID"), (dict(eps=float("inf")), "INVALID"),
    (dict(N=65537), "UNSUPPORTED"), (dict(K=65537), "UNSUPPORTED"), (dict(B=65537), "UNSUPPORTED"), (dict(steps=65), "UNSUPPORTED"),
])
def test_ortho_shapes(ep, bad, expect):
    want = expected(ep, expect)
    cfg = ortho_cfg(ep, **bad)
    assert ortho(ep, cfg) == want
    assert ep._lib.ep_orthogonalize_workspace_size(ctypes.byref(cfg), ctypes.byref(ctypes.c_size_t(0))) == want


def test_ortho_pointers(ep):
    bad, cfg = ep.EP_ERR_INVALID_ARG, ortho_cfg(ep)
    assert ortho(ep, None) == bad
    assert ep._lib.ep_orthogonalize_workspace_size(ctypes.byref(cfg), None) == bad
    for k in ("m", "out", "ws"):
        assert ortho(ep, cfg, **{k: None}) == bad, k
    assert ortho(ep, cfg, m=ctypes.c_void_p(0x10001)) == bad and ortho(ep, ortho_cfg(ep, dtype=0), m=ODD2) == bad
    assert ortho(ep, cfg, out=ODD8) == bad and ortho(ep, cfg, ws=ctypes.c_void_p(0x10080)) == bad
    assert ortho(ep, cfg, nbytes=ep.ep_orthogonalize_workspace_size(cfg) - 1) == ep.EP_ERR_CAPACITY
    assert ortho(ep, ortho_cfg(ep, B=0), m=None, out=None, ws=None, nbytes=0) == ep.EP_OK


def test_ortho_in_place_takes_16_bits(ep):
    """The results of floats are half as long: the second one would lie in the first matrix."""
    cfg = ortho_cfg(ep, dtype=0)
    assert ortho(ep, cfg, nbytes=0) == ep.EP_ERR_INVALID_ARG
    assert ortho(ep, cfg, out=ctypes.c_void_p(0x20000), nbytes=0) == ep.EP_ERR_CAPACITY
    assert ortho(ep, ortho_cfg(ep), nbytes=0) == ep.EP_ERR_CAPACITY


@pytest.mark.parametrize("k,fits", [
    ((3.4445, -4.7750, 2.0315), True), ((1.5, -0.5, 0.0), True), ((3.9, 0.0, 0.0), True), ((4.1, 0.0, 0.0), False),
    ((1.0, 31.5, -31.5), False), ((1.0, -32.0, 0.5), False), ((float("nan"), 0.0, 0.0), False), ((1.0, float("inf"), 0.0), False),
    ((0.0, 8.0, -8.0), True), ((3.0, 3.0, 3.0), False),
])
def test_ortho_coefficients(ep, k, fits):
    """Refused where X or B could leave the halves' range: |X| < 4, |b u + c u^2| < 31 for u up to X's square.
    s + 31.5 s^3 (1 - s^2) is 6.6 at s = 0.78; 8 s^3 (1 - s^2) is 1.5 there."""
    want = ep.EP_OK if fits else ep.EP_ERR_UNSUPPORTED
    cfg = ortho_cfg(ep, B=0, steps=1)  # nothing is enqueued
    assert ortho(ep, cfg, (ctypes.c_float * 3)(*k)) == want


def test_ortho_coefficients_step_by_step(ep):
    """1.9 a step: 1.9, 3.6, 6.9."""
    for steps, want in ((2, ep.EP_OK), (3, ep.EP_ERR_UNSUPPORTED)):
        k = (ctypes.c_float * (3 * steps))(*([1.9, 0.0, 0.0] * steps))
        assert ortho(ep, ortho_cfg(ep, B=0, steps=steps), k) == want


def test_ortho_binding_checks_tensors(ep):
    cfg = ep.EpOrthoConfig.make(B=1, N=8, K=8)
    m = torch.zeros((1, 8, 8), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        ep.ep_orthogonalize(cfg, m, m, None)  # on the CPU
    with pytest.raises(TypeError):
        ep.ep_orthogonalize(cfg, m.float(), m, None)
    with pytest.raises(ValueError):
        ep.ep_orthogonalize(cfg, m, m, None, coefficients=[(1.0, 0.0, 0.0)])  # one step of five
    with pytest.raises(TypeError):
        ep.EpOrthoConfig.make(N=8, K=8, dtype=torch.float64)
