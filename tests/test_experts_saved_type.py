"""The type that g and u are kept in: refusals, on the CPU."""
import ctypes

import pytest
import torch

from test_experts_abi import BWD_ARGS, FFN_ARGS, F, ep  # noqa: F401


def test_struct_layout(ep):  # noqa: F811
    assert ctypes.sizeof(ep.EpFfnConfig) == 5 * 4
    assert ep.EpFfnConfig.make(rows=1, H=8, I=8, E=1).saved_bf16 == 0


@pytest.mark.parametrize("value", [-1, 2])
def test_unknown_type(ep, value):  # noqa: F811
    cfg = ep.EpFfnConfig.make(rows=10, H=64, I=32, E=4, saved_bf16=value)
    bad = ep.EP_ERR_INVALID_ARG
    assert ep._lib.ep_expert_ffn(ctypes.byref(cfg), *FFN_ARGS.values(), None) == bad
    assert ep._lib.ep_expert_ffn_backward(ctypes.byref(cfg), *BWD_ARGS.values(), None) == bad
    assert ep._lib.ep_expert_ffn_w4(ctypes.byref(cfg), 64, *[F] * 10, None) == bad


def test_halves_are_not_taken_for_bfloat16(ep):  # noqa: F811
    cfg = ep.EpFfnConfig.make(rows=10, H=64, I=32, E=4, saved_bf16=1)
    g = torch.zeros((10, 32), dtype=torch.float16)
    with pytest.raises(TypeError):
        ep.experts._saved(cfg, g, (10, 32), "g")
    with pytest.raises(ValueError):  # the type is right; a CPU tensor
        ep.experts._saved(cfg, g.bfloat16(), (10, 32), "g")
    with pytest.raises(TypeError):
        ep.experts._saved(ep.EpFfnConfig.make(rows=10, H=64, I=32, E=4), g.float(), (10, 32), "g")
