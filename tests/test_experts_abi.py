"""The entry points of include/ep_experts.h reject bad arguments on the host, with nothing
enqueued. CPU only: no call here reaches a kernel launch."""
import ctypes

import pytest
import torch

F = ctypes.c_void_p(0x10000)  # 16-byte aligned, never dereferenced: every call below fails its checks first
ODD = ctypes.c_void_p(0x10008)


@pytest.fixture(scope="module")
def ep():
    import __graft_entry__

    __graft_entry__._cuda_build_module().build()
    import combine_router_softmax_gb300 as m

    return m


def ffn_cfg(ep, **kw):
    return ep.EpFfnConfig.make(**{**dict(rows=10, H=64, I=32, E=4), **kw})


FFN_ARGS = dict(rows=F, expert_offset=F, w_gate=F, w_up=F, w_down=F, g=None, u=None, h=F, y=F)
BWD_ARGS = dict(rows=F, expert_offset=F, w_gate=F, w_up=F, w_down=F, g=F, u=F, h=F, d_y=F, d_g=F, d_u=F, d_rows=F,
                d_w_gate=F, d_w_up=F, d_w_down=F)


def calls(ep):
    return (("ep_expert_ffn", FFN_ARGS), ("ep_expert_ffn_backward", BWD_ARGS))


@pytest.mark.parametrize("bad,expect", [
    (dict(rows=-1), "INVALID"), (dict(H=0), "INVALID"), (dict(I=-8), "INVALID"), (dict(E=0), "INVALID"),
    (dict(H=12), "UNSUPPORTED"), (dict(I=20), "UNSUPPORTED"), (dict(E=1025), "UNSUPPORTED"),
])
def test_ffn_shapes(ep, bad, expect):
    want = ep.EP_ERR_INVALID_ARG if expect == "INVALID" else ep.EP_ERR_UNSUPPORTED
    for name, args in calls(ep):
        assert getattr(ep._lib, name)(ctypes.byref(ffn_cfg(ep, **bad)), *args.values(), None) == want, name


def test_ffn_pointers(ep):
    for name, args in calls(ep):
        f = getattr(ep._lib, name)
        assert f(None, *args.values(), None) == ep.EP_ERR_INVALID_ARG
        for k, v in args.items():
            optional = v is None or k in ("d_rows", "d_w_gate", "d_w_up", "d_w_down")
            if not optional:
                assert f(ctypes.byref(ffn_cfg(ep)), *{**args, k: None}.values(), None) == ep.EP_ERR_INVALID_ARG, k
            if k != "expert_offset":
                more = {"g": ODD, "u": ODD} if v is None else {k: ODD}
                assert f(ctypes.byref(ffn_cfg(ep)), *{**args, **more}.values(), None) == ep.EP_ERR_INVALID_ARG, k
    # g without u
    assert ep._lib.ep_expert_ffn(ctypes.byref(ffn_cfg(ep)), *{**FFN_ARGS, "g": F}.values(), None) == ep.EP_ERR_INVALID_ARG


def test_ffn_without_rows_needs_nothing(ep):
    cfg = ffn_cfg(ep, rows=0)
    assert ep._lib.ep_expert_ffn(ctypes.byref(cfg), *[None] * 9, None) == ep.EP_OK
    assert ep._lib.ep_expert_ffn_backward(ctypes.byref(cfg), *[None] * 15, None) == ep.EP_OK


def test_ffn_binding_checks_tensors(ep):
    cfg = ffn_cfg(ep)
    x = torch.zeros((10, 64), dtype=torch.bfloat16)
    off = torch.zeros(5, dtype=torch.int32)
    w, d, h = (torch.zeros(s, dtype=torch.bfloat16) for s in ((4, 32, 64), (4, 64, 32), (10, 32)))
    with pytest.raises(ValueError):
        ep.ep_expert_ffn(cfg, x, off, w, w, d, h, x)
    with pytest.raises(TypeError):
        ep.ep_expert_ffn(cfg, x.float(), off, w, w, d, h, x)


# 4-bit weights ---------------------------------------------------------------

def w4_cfg(ep, **kw):
    return ep.EpW4Config.make(**{**dict(rows=4, N=16, K=64, E=2, group=32), **kw})


@pytest.mark.parametrize("bad,expect", [
    (dict(rows=-1), "INVALID"), (dict(N=0), "INVALID"), (dict(K=0), "INVALID"), (dict(E=0), "INVALID"),
    (dict(K=12), "UNSUPPORTED"), (dict(group=16), "UNSUPPORTED"), (dict(group=256), "UNSUPPORTED"),
    (dict(E=1025), "UNSUPPORTED"),
])
def test_w4_shapes(ep, bad, expect):
    want = ep.EP_ERR_INVALID_ARG if expect == "INVALID" else ep.EP_ERR_UNSUPPORTED
    c = ctypes.byref(w4_cfg(ep, **bad))
    a, b = ctypes.c_size_t(0), ctypes.c_size_t(0)
    assert ep._lib.ep_w4_sizes(c, ctypes.byref(a), ctypes.byref(b)) == want
    assert ep._lib.ep_w4_pack(c, F, F, F, None) == want
    assert ep._lib.ep_w4_linear(c, F, F, F, F, F, None) == want


def test_w4_sizes(ep):
    for K, kp in ((8, 128), (128, 128), (136, 256), (1000, 1024)):
        for group in (32, 64, 128):
            assert ep.ep_w4_sizes(w4_cfg(ep, K=K, group=group)) == (2 * 16 * kp // 2, 2 * 16 * (kp // group) * 2)


def test_w4_pointers(ep):
    L, c = ep._lib, ctypes.byref(w4_cfg(ep))
    assert L.ep_w4_sizes(c, None, None) == ep.EP_ERR_INVALID_ARG
    for i in range(3):
        for bad in (None, ODD):
            assert L.ep_w4_pack(c, *[bad if j == i else F for j in range(3)], None) == ep.EP_ERR_INVALID_ARG
    for i in range(5):
        for bad in (None, ODD) if i != 1 else (None,):
            assert L.ep_w4_linear(c, *[bad if j == i else F for j in range(5)], None) == ep.EP_ERR_INVALID_ARG
    f = ctypes.byref(ffn_cfg(ep))
    for i in range(10):
        for bad in (None, ODD) if i != 1 else (None,):
            assert L.ep_expert_ffn_w4(f, 64, *[bad if j == i else F for j in range(10)], None) == ep.EP_ERR_INVALID_ARG
    assert L.ep_expert_ffn_w4(f, 48, *[F] * 10, None) == ep.EP_ERR_UNSUPPORTED
    assert L.ep_expert_ffn_w4(ctypes.byref(ffn_cfg(ep, rows=0)), 64, *[None] * 10, None) == ep.EP_OK
    assert L.ep_w4_linear(ctypes.byref(w4_cfg(ep, rows=0)), *[None] * 5, None) == ep.EP_OK


# Backward of combine and router ----------------------------------------------

def layer_cfg(ep, **kw):
    return ep.EpConfig.make(**{**dict(T=4, H=64, E=8, R=1, k=2), **kw})


@pytest.mark.parametrize("bad,expect", [
    (dict(T=-1), "INVALID"), (dict(k=9), "INVALID"), (dict(k=0), "INVALID"), (dict(E=0), "INVALID"),
    (dict(renormalize=2), "INVALID"), (dict(T=2**30, k=4), "INVALID"), (dict(E=2000), "UNSUPPORTED"),
    (dict(E=64, k=33), "UNSUPPORTED"), (dict(H=0), "rows INVALID"), (dict(H=20), "rows UNSUPPORTED"),
])
def test_gate_backward_shapes(ep, bad, expect):
    want = ep.EP_ERR_INVALID_ARG if "INVALID" in expect else ep.EP_ERR_UNSUPPORTED
    c = ctypes.byref(layer_cfg(ep, **bad))
    assert ep._lib.ep_combine_backward(c, F, F, F, F, F, F, None) == want
    if "rows" not in expect:
        assert ep._lib.ep_route_backward(c, F, F, F, F, F, None) == want


def test_gate_backward_pointers(ep):
    L, c = ep._lib, ctypes.byref(layer_cfg(ep))
    assert L.ep_combine_backward(None, *[F] * 6, None) == ep.EP_ERR_INVALID_ARG
    for i in range(6):
        assert L.ep_combine_backward(c, *[None if j == i else F for j in range(6)], None) == ep.EP_ERR_INVALID_ARG
        if i in (0, 1, 4):
            assert L.ep_combine_backward(c, *[ODD if j == i else F for j in range(6)], None) == ep.EP_ERR_INVALID_ARG
    raw = ctypes.byref(layer_cfg(ep, renormalize=0))
    for i in range(5):
        assert L.ep_route_backward(raw, *[None if j == i else F for j in range(5)], None) == ep.EP_ERR_INVALID_ARG
    none = ctypes.byref(layer_cfg(ep, T=0))
    assert L.ep_combine_backward(none, *[None] * 6, None) == ep.EP_OK
    assert L.ep_route_backward(none, *[None] * 5, None) == ep.EP_OK


# Gradient norm and clipping ---------------------------------------------------

def test_grad_refusals(ep):
    L = ep._lib
    size = ep.ep_grad_workspace_size(2)
    assert size % 8 == 0 and ep.ep_grad_workspace_size(0) > 0
    assert L.ep_grad_workspace_size(-1, ctypes.byref(ctypes.c_size_t(0))) == ep.EP_ERR_INVALID_ARG

    def clip(max_norm=1.0, n=2, norm=F, ws=F, nbytes=size, **kw):
        rec = (ep.EpGradTensor * 2)(*[ep.EpGradTensor(0x10000, 0x20000, 10, 0, 0)] * 2)
        for k, v in kw.items():
            setattr(rec[1], k, v)
        return L.ep_grad_clip(rec, n, max_norm, norm, ws, nbytes, None), L.ep_grad_norm(rec, n, norm, ws, nbytes, None)

    bad = ep.EP_ERR_INVALID_ARG
    assert clip(n=-1) == (bad, bad)
    assert clip(norm=None) == (bad, bad) and clip(ws=None) == (bad, bad)
    assert clip(ws=ctypes.c_void_p(0x10004)) == (bad, bad)
    assert clip(nbytes=size - 1) == (ep.EP_ERR_CAPACITY, ep.EP_ERR_CAPACITY)
    assert clip(dtype=3) == (bad, bad) and clip(numel=-1) == (bad, bad) and clip(reserved=1) == (bad, bad)
    assert clip(data=0) == (bad, bad) and clip(data=0x10002) == (bad, bad)
    assert L.ep_grad_clip(None, 1, 1.0, F, F, size, None) == bad
    for m in (-1.0, float("nan")):
        assert L.ep_grad_clip(None, 0, m, F, F, size, None) == bad
    rec = (ep.EpGradTensor * 1)(ep.EpGradTensor(0x10000, 0, 10, 0, 0))  # out is clip's alone
    assert L.ep_grad_clip(rec, 1, 1.0, F, F, size, None) == bad


def test_grad_list_checks_tensors(ep):
    with pytest.raises(TypeError):
        ep.GradList([torch.zeros(3, dtype=torch.float64)])
    with pytest.raises(ValueError):
        ep.GradList([torch.zeros(3)])  # on the CPU
    with pytest.raises(ValueError):
        ep.GradList([], out=[torch.zeros(3)])
