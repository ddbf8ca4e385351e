"""Layers of different sizes called from several threads at a time, each on a stream of its own."""
from __future__ import annotations

import ctypes
import pathlib
import subprocess
import threading

import pytest
import torch

from gpu_harness import require_cuda

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def ep():
    require_cuda()
    import combine_router_softmax_gb300 as m

    return m


@pytest.fixture(scope="module")
def caller(tmp_path_factory):
    lib = tmp_path_factory.mktemp("threads") / "expert_threads.so"
    source = pathlib.Path(__file__).with_name("expert_threads.c")
    subprocess.run(["gcc", "-O1", "-shared", "-fPIC", str(source), "-o", str(lib)], check=True)
    return ctypes.CDLL(str(lib))


@pytest.mark.parametrize("rows", [8, 40])
def test_layers_of_many_and_of_few_experts(ep, caller, rows):
    """The tables that a kernel keeps of the experts take more shared memory with 1024 of them than with 2: what
    one thread's call sets must not be too little for another's."""
    errors, H, I = [], 8, 8
    start = threading.Barrier(4)

    def work(E):
        torch.cuda.set_device(0)
        cfg = ep.EpFfnConfig.make(rows=rows, H=H, I=I, E=E)
        off = torch.arange(E + 1, dtype=torch.int32, device="cuda").clamp_(max=rows)
        x, y = (torch.zeros((rows, H), dtype=BF16, device="cuda") for _ in range(2))
        w, d = (torch.zeros((E, a, b), dtype=BF16, device="cuda") for a, b in ((I, H), (H, I)))
        h = torch.zeros((rows, I), dtype=BF16, device="cuda")
        stream = torch.cuda.Stream()
        ep.ep_expert_ffn(cfg, x, off, w, w, d, h, y, stream=stream)
        torch.cuda.synchronize()
        at = ctypes.c_int(-1)
        vp = lambda t: ctypes.c_void_p(t.data_ptr())  # noqa: E731
        start.wait()
        status = caller.call_often(ep._lib.ep_expert_ffn, 20000, ctypes.byref(at), ctypes.byref(cfg), vp(x), vp(off),
                                   vp(w), vp(d), vp(h), vp(y), ctypes.c_void_p(stream.cuda_stream))
        stream.synchronize()
        if status:
            errors.append((E, status, at.value))

    threads = [threading.Thread(target=work, args=(E,)) for E in (1024, 2, 1024, 2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors, errors
    assert ep.ep_device_error() == 0
