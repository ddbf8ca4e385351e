"""The bounded waits of the expert kernels (tcgen05.cuh): a warp's lanes agree on a failure, a wait for what never
comes ends, and ep_device_error reports it."""
from __future__ import annotations

import ctypes
import subprocess

import pytest
import torch

from gpu_harness import require_cuda


@pytest.fixture(scope="module")
def waits(tmp_path_factory):
    import __graft_entry__

    b = __graft_entry__._cuda_build_module()
    lib = tmp_path_factory.mktemp("waits") / "expert_waits.so"
    cmd = [b.nvcc_path(), *b.ARCH, "-O3", "-std=c++17", "--expt-relaxed-constexpr", "-Xcompiler", "-fPIC", "-shared",
           f"-I{b.ROOT / 'include'}", f"-I{b.CSRC}", str(b.ROOT / "tests" / "expert_waits.cu"), "-o", str(lib)]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    return lib


def test_helpers_build(waits):
    assert ctypes.CDLL(str(waits)).run_agreement


@pytest.mark.gpu
def test_a_warp_agrees_on_a_failure(waits):
    require_cuda()
    rounds = 400
    out = torch.full((3,), -1, dtype=torch.int32, device="cuda")
    assert ctypes.CDLL(str(waits)).run_agreement(rounds, ctypes.c_void_p(out.data_ptr())) == 0
    differ, good, bad = out.tolist()
    assert differ == 0 and good + bad == rounds
    assert good >= rounds // 2 and bad >= rounds // 4  # every other round has no failure, every fourth no arrival


@pytest.mark.gpu
@pytest.mark.parametrize("fills", [1, 2, 4, 6, 9])
def test_copies_under_way_are_waited_for(waits, fills):
    """Two producers take a ring's fills in turn: each waits for its own, and says so when the last one does not
    come in time."""
    require_cuda()
    out = torch.full((2,), -1, dtype=torch.int32, device="cuda")
    assert ctypes.CDLL(str(waits)).run_fills(fills, ctypes.c_void_p(out.data_ptr())) == 0
    late = (fills - 1) % 2  # the producer of the last fill
    assert out.tolist() == [3, 3 - (1 << late)]


@pytest.mark.gpu
def test_a_wait_that_runs_out_is_reported(waits):
    require_cuda()
    import combine_router_softmax_gb300 as ep

    assert ep.ep_device_error() == 0
    word = ctypes.c_void_p()
    symbol = getattr(ep._lib, "_ZN2ep17expert_error_wordEPPi")  # ep::expert_error_word
    assert symbol(ctypes.byref(word)) == 0
    out = torch.full((4,), -1, dtype=torch.int32, device="cuda")
    assert ctypes.CDLL(str(waits)).run_give_up(ctypes.c_void_p(out.data_ptr()), word) == 0
    assert out.tolist() == [0, 1, 0, 32]
    assert ep.ep_device_error() == 16  # an expert product gave up
    assert ep.ep_device_error() == 0   # read and cleared
