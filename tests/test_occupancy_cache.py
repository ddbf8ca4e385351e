"""The host asks the runtime once how many CTAs of a kernel an SM holds, whatever number of kernels and shapes a process comes to use."""
from __future__ import annotations

import ctypes
import subprocess
import threading

import pytest


@pytest.fixture
def cache(tmp_path):
    import __graft_entry__

    b = __graft_entry__._cuda_build_module()
    lib = tmp_path / "occupancy_cache.so"
    cmd = [b.nvcc_path(), *b.ARCH, "-O2", "-std=c++17", "--expt-relaxed-constexpr", "-Xcompiler", "-fPIC", "-shared",
           f"-I{b.ROOT / 'include'}", f"-I{b.CSRC}", str(b.ROOT / "tests" / "occupancy_cache.cu"), "-o", str(lib)]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    f = ctypes.CDLL(str(lib))
    f.occupancy_of.argtypes = [ctypes.c_int, ctypes.c_int, ctypes.c_size_t]
    return f


def blocks(threads, smem, device=0):
    return 1 + (threads + smem + 7 * device) % 31


def test_asked_once(cache):
    shapes = [(kernel, 32 * (1 + i % 32), 16 * i) for kernel in range(7) for i in range(300)]
    for _ in range(3):
        for kernel, threads, smem in shapes:
            assert cache.occupancy_of(kernel, threads, smem) == blocks(threads, smem)
        assert cache.occupancy_questions() == len(shapes)
    cache.use_device(3)
    assert cache.occupancy_of(*shapes[5]) == blocks(*shapes[5][1:], device=3)
    cache.use_device(0)
    assert cache.occupancy_of(*shapes[5]) == blocks(*shapes[5][1:])
    assert cache.occupancy_questions() == len(shapes) + 1


def test_from_several_threads(cache):
    wrong = []

    def ask(seed):
        for i in range(2000):
            j = (i * 7 + seed) % 500
            if cache.occupancy_of(j % 5, 32 + j, j) != blocks(32 + j, j):
                wrong.append(j)

    threads = [threading.Thread(target=ask, args=(s,)) for s in range(8)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong and 500 <= cache.occupancy_questions() <= 500 * 8


def test_a_failure_is_not_kept(cache):
    cache.fail(1)
    assert cache.occupancy_of(0, 64, 10) == 1  # a launch of one CTA an SM is right for any kernel
    cache.fail(0)
    assert cache.occupancy_of(0, 64, 10) == blocks(64, 10)
