"""Cache attention's waits run out without a fault: the tcgen05 kernel with one hand-over
withheld and a short limit reports DROPKV_ERR_TIMEOUT, leaves no wait behind, and the next calls
are right."""

import time

import pytest
import torch

import kv_cache_eviction_scores_b200 as dk

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("limit_ms", [5.0, 50.0])
@pytest.mark.parametrize("T", [9, 60, 64, 65, 300])  # both kernels, with and without idle rows
@pytest.mark.parametrize("e4m3,d", [(False, 128), (True, 128), (False, 64), (True, 64)])
@pytest.mark.parametrize("B", [2, 200])                # a piece of a unit a CTA, and many units
def test_expired_waits_are_reported(B, T, e4m3, d, limit_ms):
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    assert dk.selftest_cache_attention_timeout(T, e4m3, d, B, limit_ms) == dk.ERR_TIMEOUT
    dt = (time.perf_counter() - t0) * 1e3
    assert dt >= 0.9 * limit_ms  # a wait held for its limit before giving up
    # nor did the waits run out one after the other, or at the default of two seconds
    assert dt <= 10 * limit_ms + 1000


@pytest.mark.parametrize("T", [60, 300])
def test_calls_after_an_expired_wait_are_right(T):
    g = torch.Generator(device=DEV).manual_seed(T)
    k, v = (torch.randn(16, 2, 32, 128, generator=g, device=DEV).bfloat16() for _ in range(2))
    q = torch.randn(1, 4, T, 128, generator=g, device=DEV).bfloat16()
    table = torch.arange(16, dtype=torch.int32, device=DEV)[None]
    lens = torch.tensor([500], dtype=torch.int32, device=DEV)
    want = dk.dropkv_cache_attention(q, k, v, table, lens, sync=True)
    assert dk.selftest_cache_attention_timeout(T, limit_ms=5.0) == dk.ERR_TIMEOUT
    assert torch.equal(dk.dropkv_cache_attention(q, k, v, table, lens, sync=True), want)


def test_calls_without_such_waits_are_refused():
    with pytest.raises(dk.DropKVError) as e:
        dk.selftest_cache_attention_timeout(4)  # eight rows per KV head
    assert e.value.status == dk.ERR_UNSUPPORTED
    for limit_ms in (0.0, 1001.0):
        with pytest.raises(dk.DropKVError) as e:
            dk.selftest_cache_attention_timeout(60, limit_ms=limit_ms)
        assert e.value.status == dk.ERR_ARG
