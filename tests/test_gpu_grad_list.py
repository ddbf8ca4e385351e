"""GradList and the memory of its tensors."""
from __future__ import annotations

import pytest
import torch

from gpu_harness import require_cuda

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ep():
    require_cuda()
    import combine_router_softmax_gb300 as m

    return m


def test_a_list_keeps_the_memory_it_names(ep):
    """A tensor that is given other memory (`.data = ...`) leaves the list with the memory that it had when the
    list was made: nobody else gets it while the list lives."""
    n = 1 << 20
    p, out = torch.ones(n, device="cuda"), torch.ones(n, device="cuda")
    lst = ep.GradList([p], [out])
    named = {lst.records[0].data, lst.records[0].out}
    assert named == {p.data_ptr(), out.data_ptr()}
    p.data = torch.zeros(n, device="cuda")
    out.data = torch.zeros(n, device="cuda")
    others = [torch.empty(n, device="cuda") for _ in range(8)]
    assert not named & {t.data_ptr() for t in others}
    del lst
    others += [torch.empty(n, device="cuda") for _ in range(8)]
    assert named <= {t.data_ptr() for t in others}  # given back with the list
