"""Matrices that a cluster of more than eight CTAs keeps on the chip, on a device that has no place for one: the library is
linked a second time with a runtime that says so, and takes the products of their own instead."""
from __future__ import annotations

import ctypes
import subprocess

import pytest
import torch

from gpu_harness import require_cuda

FAKE = """#include <cuda_runtime.h>
namespace {
template <typename T>
cudaError_t no_place(int *n, T *, const cudaLaunchConfig_t *) {
    *n = 0;
    return FAIL ? cudaErrorInvalidConfiguration : cudaSuccess;
}
}
#define cudaOccupancyMaxActiveClusters no_place
#include "ortho_fused.cu"
"""


@pytest.fixture(scope="module", params=[0, 1])
def without(request, tmp_path_factory):
    import __graft_entry__

    b = __graft_entry__._cuda_build_module()
    b.build()
    path = tmp_path_factory.mktemp("places")
    (path / "fake.cu").write_text(FAKE)
    objects = [b.BUILD / (s.stem + ".o") for s in b.sources() if s.stem != "ortho_fused"]
    if not all(o.exists() for o in objects):
        b.build(force=True)
    cmd = [b.nvcc_path(), *b.ARCH, "-O3", "-std=c++17", "--expt-relaxed-constexpr", "-Xcompiler", "-fPIC", "-shared", f"-DFAIL={request.param}",
           "-Xlinker", "-Bsymbolic", f"-I{b.ROOT / 'include'}", f"-I{b.CSRC}", str(path / "fake.cu"), *map(str, objects), "-o", str(path / "without.so")]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    return ctypes.CDLL(str(path / "without.so"))


@pytest.mark.gpu
@pytest.mark.parametrize("count,N,K", [(1, 128, 4096), (3, 2500, 64), (2, 70, 2300), (2, 128, 2048)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_products_where_no_cluster_fits(without, count, N, K, dtype):
    """Both ways round alike: within the sum of the figure that the header gives for each, 0.0012, and of their roundings to bf16, 0.0017 each."""
    require_cuda()
    import combine_router_softmax_gb300 as ep

    gen = torch.Generator(device="cuda").manual_seed(N)
    m = torch.randn((count, N, K), generator=gen, device="cuda").to(dtype)
    cfg = ep.EpOrthoConfig.make(B=count, N=N, K=K, dtype=dtype)
    ws = torch.full((ep.ep_orthogonalize_workspace_size(cfg),), 255, dtype=torch.uint8, device="cuda")
    want, got = (torch.full(m.shape, float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    ep.ep_orthogonalize(cfg, m, want, ws)
    p = lambda t: ctypes.c_void_p(t.data_ptr())  # noqa: E731
    stream = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    for _ in range(2):  # the answer is kept
        assert without.ep_orthogonalize(ctypes.byref(cfg), None, p(m), p(got), p(ws), ctypes.c_size_t(ws.numel()), stream) == 0
    w, g = want.double(), got.double()
    assert torch.isfinite(g).all() and (g - w).norm() <= (2 * 0.0012 + 2 * 0.0017) * w.norm()


def test_workspace_of_what_not_every_device_keeps_on_the_chip():
    import __graft_entry__

    __graft_entry__._cuda_build_module().build()
    import combine_router_softmax_gb300 as ep

    size = lambda N, K: ep.ep_orthogonalize_workspace_size(ep.EpOrthoConfig.make(B=3, N=N, K=K))  # noqa: E731
    assert size(128, 2048) == size(2048, 5) == 256
    for N, K in ((128, 2049), (4096, 16), (1, 4096)):
        assert size(N, K) >= 8 * 3 * N * K
