"""The paged-cache calls on the GPU: what they refuse before any work, and how they are used
beside the rest of the library."""

import pytest
import torch

import kv_cache_eviction_scores_b200 as dk
from cache_ref import BF16, E4M3, F32

pytestmark = pytest.mark.gpu
DEV = "cuda"


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def test_evict_to_cache_refuses_before_any_work(monkeypatch):
    B, Hq, Hkv, n, d, w = 2, 4, 2, 40, 16, 2
    q, k = torch.zeros(B, Hq, w, d, device=DEV), torch.zeros(B, Hkv, n, d, device=DEV)
    pages = torch.zeros(8, Hkv, 8, d, device=DEV)
    table = torch.arange(8, dtype=torch.int32, device=DEV).view(B, 4)

    def work(*a, **kw):
        raise AssertionError("the prompt was scored before the refusal")

    monkeypatch.setattr(dk, "evict", work)
    monkeypatch.setattr(dk, "dropkv_scores_select", work)

    def call(q=q, k=k, v=k, pages=pages, table=table, keep=(9, 9)):
        dk.evict_to_cache(q, k, v, w, 1, list(keep), pages, pages.clone(), table)

    with pytest.raises(AssertionError):
        call()                                                     # what is right goes to work
    for kw in (dict(table=table[:1].contiguous()),                 # sequences
               dict(pages=torch.zeros(8, Hkv + 1, 8, d, device=DEV)),  # heads
               dict(pages=torch.zeros(8, Hkv, 8, d + 1, device=DEV)),  # head dim
               dict(v=k[:, :, :-1].contiguous()), dict(k=k[0], v=k[0]), dict(keep=(33, 9)),
               dict(k=k.transpose(1, 2), v=k.transpose(1, 2))):
        with pytest.raises(ValueError):
            call(**kw)
    for kw in (dict(v=k.bfloat16()), dict(q=q.bfloat16()), dict(k=k.half(), v=k.half(), q=q.half()),
               dict(q=q.cpu()), dict(k=k.cpu(), v=k.cpu())):
        with pytest.raises(TypeError):
            call(**kw)
