"""The paged-cache calls allocate no device memory, in the library or through torch, when a caller
passes what they write to."""

import pytest
import torch

import kv_cache_eviction_scores_b200 as dk
from test_gpu_cache_calls import CASES, DEV, attend, problem

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,fmt,qt", CASES)
def test_the_cache_calls_allocate_nothing(T, fmt, qt):
    s = problem(T, fmt, qt)
    out, lse = torch.empty_like(s["q"]), torch.empty(s["q"].shape[:3], device=DEV)
    ws = dk.cache_attention_workspace(s["q"], s["k"], s["table"])
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    back = torch.empty_like(s["kn"]), torch.empty_like(s["vn"])

    def step():
        dk.dropkv_cache_write(s["kn"], s["vn"], s["k"], s["v"], s["table"], start=s["lens"],
                              status=status, **s["sc"])
        attend(s, out=out, lse=lse, workspace=ws, status=status)
        dk.dropkv_cache_read(s["k"], s["v"], s["table"], T, start=s["lens"], out=back,
                             status=status, **s["sc"])

    step()  # the modules are loaded
    torch.cuda.synchronize()
    made = torch.cuda.memory_stats()["allocation.all.allocated"]

    def stable():
        free = torch.cuda.mem_get_info()[0]
        for _ in range(20):
            step()
        torch.cuda.synchronize()
        return torch.cuda.mem_get_info()[0] == free

    assert any(stable() for _ in range(3))  # the device may have other users for a moment
    assert torch.cuda.memory_stats()["allocation.all.allocated"] == made
