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


def problem(T, fmt, qt=BF16, B=2, Hq=8, Hkv=2, d=128, L=200, seed=1):
    """Pages with room for 40 slots more, and a chunk of T tokens."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    page, per = 16, -(-(L + 40) // 16)
    shape = (B * per, Hkv, page, d)
    s = {x: (torch.randn(shape, generator=g, device=DEV) * (48 if fmt == E4M3 else 1)).to(fmt) for x in "kv"}
    s["sc"] = dict.fromkeys(("k_scale", "v_scale"))
    if fmt == E4M3:
        s["sc"] = {x: torch.randint(119, 124, shape[:3], generator=g, device=DEV, dtype=torch.uint8)
                   for x in s["sc"]}
    s["table"] = torch.randperm(B * per, generator=g, device=DEV).to(torch.int32).view(B, per)
    s["lens"] = i32([L - 13 * b for b in range(B)])
    s["q"], s["kn"], s["vn"] = (torch.randn(B, H, T, d, generator=g, device=DEV).to(qt)
                                for H in (Hq, Hkv, Hkv))
    return s


def attend(s, **kw):
    return dk.dropkv_cache_attention(s["q"], s["k"], s["v"], s["table"], s["lens"], **s["sc"], **kw)


CASES = [(1, BF16, BF16), (1, E4M3, BF16), (4, BF16, BF16), (4, E4M3, BF16), (20, BF16, BF16),
         (20, E4M3, BF16), (100, BF16, BF16), (100, E4M3, BF16), (3, F32, F32), (60, F32, F32)]


@pytest.mark.parametrize("T,fmt,qt", CASES)
def test_a_captured_call_with_a_workspace_of_its_size(T, fmt, qt):
    s = problem(T, fmt, qt)
    want = attend(s)
    out, ws = torch.zeros_like(want), dk.cache_attention_workspace(s["q"], s["k"], s["table"])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        made = torch.cuda.memory_stats()["allocation.all.allocated"]
        attend(s, out=out, workspace=ws)
        assert torch.cuda.memory_stats()["allocation.all.allocated"] == made
    for _ in range(2):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_pages_without_heads_are_refused():
    z, q = torch.zeros(2, 0, 4, 16, device=DEV), torch.zeros(1, 4, 1, 16, device=DEV)
    with pytest.raises(ValueError):
        dk.dropkv_cache_attention(q, z, z, i32([[0, 1]]), i32([3]))
