"""What the paged-cache entry points refuse at the edges of their ranges, on the host (no GPU
needed: only calls that fail validation are made)."""

import ctypes

import pytest
import torch

import kv_cache_eviction_scores_b200 as dk
from test_cache_host import FAKE, _attend, _attn, _cache, _call, _rows


@pytest.mark.parametrize("scale", [1e-46, 1e39, 0.0, -1.0, float("nan"), float("inf")])
def test_scales_that_fp32_does_not_hold_are_refused(scale):
    # 1e-46 is 0 in fp32, which means the default to the library
    pages, x = torch.zeros(4, 2, 16, 8), torch.zeros(1, 2, 5, 8)
    table, n = torch.zeros(1, 4, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="scale"):
        dk.dropkv_cache_attention(x, pages, pages, table, n, scale=scale)


def test_a_scale_that_overflows_in_units_of_log2_is_refused():
    assert _attend(_cache(), _attn(scale=2.5e38)) == dk.ERR_ARG
    if not torch.cuda.is_available():
        for fine in (2.3e38, 1e-45):
            assert _attend(_cache(), _attn(scale=fine)) == dk.ERR_UNSUPPORTED


@pytest.mark.parametrize("name", ["dropkv_cache_write", "dropkv_cache_read"])
@pytest.mark.parametrize("listed", [None, FAKE])
def test_more_rows_than_the_kernel_counts_are_refused(name, listed):
    # a block's items past the last one would pass 2^31 and be looked up in front of the list
    fn, top = getattr(dk.lib(), name), 2 ** 31 - 1
    for m in (top, 0x7FFF0001):
        assert _call(fn, _cache(), _rows(n=top, m=m, rows=listed)) == dk.ERR_ARG
    if not torch.cuda.is_available():
        assert _call(fn, _cache(), _rows(n=top, m=0x7FFF0000, rows=listed)) == dk.ERR_UNSUPPORTED


def test_the_timeout_self_test_refuses_bad_arguments():
    fn, c, a = dk.lib().dropkv_selftest_cache_attention_timeout, _cache(), _attn(T=40)

    def call(attn=a, status=FAKE, limit=1000, nbytes=1 << 40):
        return fn(ctypes.byref(c), ctypes.byref(attn), FAKE, nbytes, status, limit, None)

    assert call(status=None) == call(limit=0) == call(limit=10 ** 9 + 1) == dk.ERR_ARG
    assert call(status=FAKE + 2) == call(_attn(T=40, q=None)) == dk.ERR_ARG
    assert call(_attn(T=8)) == call(_attn(T=40, path=dk.PATH_SIMT)) == dk.ERR_UNSUPPORTED
    assert call(nbytes=16) == dk.ERR_WORKSPACE


@pytest.mark.parametrize("T", [1, 4, 40, 200])
@pytest.mark.parametrize("dtype,code", [(torch.bfloat16, dk.BF16), (torch.float8_e4m3fn, dk.E4M3)])
@pytest.mark.parametrize("path", ["auto", "simt", "tensor"])
def test_a_workspace_from_the_calls_own_tensors(T, dtype, code, path):
    q = torch.zeros(2, 8, T, 128, dtype=torch.bfloat16)
    pages = torch.zeros(64, 4, 16, 128).to(dtype)
    table = torch.zeros(2, 8, dtype=torch.int32)
    ws = dk.cache_attention_workspace(q, pages, table, path=path)
    assert ws.dtype == torch.uint8 and ws.numel() == dk.cache_attention_workspace_bytes(
        _cache(dtype=code), _attn(T=T, path=dk._PATHS[path]))
    for bad in (q[..., :64], q[:1]):
        with pytest.raises(ValueError):
            dk.cache_attention_workspace(bad, pages, table)
    with pytest.raises(TypeError):
        dk.cache_attention_workspace(q.half(), pages, table)
    with pytest.raises(dk.DropKVError):
        dk.cache_attention_workspace(q[:, :7], pages, table)


def test_an_empty_chunk_needs_no_workspace():
    pages, table = torch.zeros(64, 4, 16, 128), torch.zeros(2, 8, dtype=torch.int32)
    assert dk.cache_attention_workspace(torch.zeros(2, 8, 0, 128), pages, table).numel() == 0


def test_rows_that_lie_close_are_no_overlap():
    # the last row of a head ends where the next head begins, with a gap behind the others
    pages, table = torch.zeros(4, 2, 16, 8), torch.zeros(1, 4, dtype=torch.int32)
    for strides in ((88, 44, 9, 1), (0, 44, 9, 1), (1, 8, 16, 1)):
        out = torch.zeros(100).as_strided((1, 2, 5, 8), strides)
        with pytest.raises(TypeError, match="no CPU path"):  # past the check of out
            dk.dropkv_cache_read(pages, pages, table, 5, out=(out, out))
    for strides in ((88, 43, 9, 1), (88, 44, 7, 1), (88, 0, 9, 1), (88, 4, 9, 1)):
        out = torch.zeros(100).as_strided((1, 2, 5, 8), strides)
        with pytest.raises(ValueError, match="overlap"):
            dk.dropkv_cache_read(pages, pages, table, 5, out=(out, out))


def test_what_is_no_tensor_or_has_another_rank_is_refused_by_name():
    pages, table = torch.zeros(4, 2, 16, 8), torch.zeros(1, 4, dtype=torch.int32)
    x = torch.zeros(1, 2, 5, 8)
    for k in (None, x[0], x[0, 0], [1.0]):
        with pytest.raises(ValueError, match="k must"):
            dk.dropkv_cache_write(k, x, pages, pages, table)
    for rows in ([1], torch.tensor(5), torch.zeros(5, dtype=torch.int32)):
        with pytest.raises(ValueError, match="rows must"):
            dk.dropkv_cache_read(pages, pages, table, 5, rows=rows)
    for p, t in ((None, table), (pages[0], table), (pages, None), (pages, table[0])):
        with pytest.raises(ValueError, match="pages must"):
            dk.dropkv_cache_read(p, pages, t, 5)
    with pytest.raises(ValueError, match="negative"):
        dk.dropkv_cache_read(pages, pages, table, -1)
    with pytest.raises(TypeError, match="out k"):
        dk.dropkv_cache_read(pages, pages, table, 5, out=(None, None))
    with pytest.raises(TypeError, match="out v must"):
        dk.dropkv_cache_read(pages, pages, table, 5, out=(x, [x]))
