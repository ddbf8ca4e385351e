"""The gradient norm across processes (exchange.reduce_grad_norm), gloo on the CPU, and the refusals of the call that
clips by it."""
import ctypes
import math
import os
import socket

import pytest
import torch
import torch.multiprocessing as mp

from test_experts_abi import F, ep  # noqa: F401

# what each of two processes' gradients are made of
PARTS = {"usual": ([0.3, -2.0, 5e-3], [1.5, 0.25]), "one has none": ([], [3.0, 4.0]),
         "large": ([3e30, 1e29], [4e30]), "small": ([3e-30], [4e-30, 1e-38]), "far apart": ([1e38], [1e-38]),
         "infinite": ([1.0], [float("inf")]), "nan": ([float("nan")], [1.0])}


def _free_port():
    with socket.socket() as s:
        s.bind(("127.0.0.1", 0))
        return s.getsockname()[1]


def _norm(values):
    return math.sqrt(sum(v * v for v in values))


def _worker(rank, world, port, out_dir):
    os.environ.update(MASTER_ADDR="127.0.0.1", MASTER_PORT=str(port), RANK=str(rank), WORLD_SIZE=str(world),
                      LOCAL_RANK=str(rank))
    import torch.distributed as dist

    from combine_router_softmax_gb300.exchange import reduce_grad_norm

    dist.init_process_group("gloo", rank=rank, world_size=world)
    got = {}
    for name, parts in PARTS.items():
        norm = torch.tensor([_norm(parts[rank])], dtype=torch.float32)
        same = reduce_grad_norm(norm)
        assert same.data_ptr() == norm.data_ptr() and norm.dtype is torch.float32
        # the factor that either process clips its own gradients by
        got[name] = (norm.item(), torch.clamp(0.5 / (norm + 1e-6), max=1.0).item())
    torch.save(got, os.path.join(out_dir, f"n{rank}.pt"))
    dist.destroy_process_group()


def test_two_processes_clip_by_one_norm(ep, tmp_path):  # noqa: F811
    mp.start_processes(_worker, args=(2, _free_port(), str(tmp_path)), nprocs=2, start_method="spawn")
    first, second = (torch.load(tmp_path / f"n{r}.pt") for r in range(2))
    for name, (a, b) in PARTS.items():
        want = _norm(a + b)
        for norm, factor in (first[name], second[name]):
            if math.isnan(want):
                assert math.isnan(norm) and math.isnan(factor)
            elif math.isinf(want):
                assert math.isinf(norm) and factor == 0
            else:  # each process's norm and the result are rounded to fp32
                assert abs(norm - want) <= 2 * 2.0**-24 * want, name
        assert math.isnan(want) or first[name] == second[name]


def test_clip_with_norm_refusals(ep):  # noqa: F811
    bad = ep.EP_ERR_INVALID_ARG

    def call(max_norm=1.0, n=2, norm=F, **kw):
        rec = (ep.EpGradTensor * 2)(*[ep.EpGradTensor(0x10000, 0x20000, 10, 0, 0)] * 2)
        for k, v in kw.items():
            setattr(rec[1], k, v)
        return ep._lib.ep_grad_clip_with_norm(rec, n, max_norm, norm, None)

    assert call(n=-1) == bad and call(norm=None) == bad and call(norm=ctypes.c_void_p(0x10002)) == bad
    assert call(max_norm=-1.0) == bad and call(max_norm=float("nan")) == bad
    assert call(dtype=3) == bad and call(numel=-1) == bad and call(reserved=1) == bad
    assert call(data=0) == bad and call(data=0x10002) == bad and call(out=0) == bad
    assert ep._lib.ep_grad_clip_with_norm(None, 1, 1.0, F, None) == bad
    assert ep._lib.ep_grad_clip_with_norm(None, 0, 1.0, F, None) == ep.EP_OK  # nothing to scale


def test_binding_checks_the_norm(ep):  # noqa: F811
    class Empty:
        records, n = (ep.EpGradTensor * 1)(), 0

    with pytest.raises(TypeError):
        ep.ep_grad_clip_with_norm(Empty, 1.0, torch.zeros(1, dtype=torch.float64))
    with pytest.raises(ValueError):
        ep.ep_grad_clip_with_norm(Empty, 1.0, torch.zeros(1))  # on the CPU
