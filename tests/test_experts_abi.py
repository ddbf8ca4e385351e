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
