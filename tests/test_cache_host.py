"""The paged-cache entry points refuse bad arguments on the host, before any
device work (no GPU needed: only calls that fail validation are made)."""

import ctypes

import pytest
import torch

import cache_ref as R
import kv_cache_eviction_scores_b200 as dk

FAKE = 0x100000


def _cache(**kw):
    f = dict(B=2, Hkv=4, d=128, n_pages=64, page_size=16, max_pages=8, dtype=dk.BF16, reserved=0,
             k_pages=FAKE, v_pages=FAKE, k_scale=None, v_scale=None, page_table=FAKE)
    f.update(kw)
    return dk.Cache(*f.values())


def _rows(**kw):
    s = (ctypes.c_int64 * 3)(4 * 10 * 128, 10 * 128, 128)
    f = dict(k=FAKE, v=FAKE, k_stride=s, v_stride=s, dtype=dk.BF16, n=10, m=10, reserved=0,
             rows=None, start=None, counts=None)
    f.update(kw)
    return dk.CacheRows(*f.values())


def _attn(**kw):
    s = (ctypes.c_int64 * 3)(8 * 5 * 128, 5 * 128, 128)
    f = dict(q=FAKE, out=FAKE, lse=None, q_stride=s, out_stride=s, dtype=dk.BF16, Hq=8, T=5,
             causal=1, scale=0.0, path=dk.PATH_AUTO, lengths=FAKE, q_lengths=None)
    f.update(kw)
    return dk.CacheAttn(*f.values())


NEG = (ctypes.c_int64 * 3)(-1, 1, 1)
BAD_CACHE = [dict(B=0), dict(Hkv=0), dict(d=0), dict(d=257), dict(n_pages=0), dict(page_size=0),
             dict(page_size=1025), dict(max_pages=0), dict(dtype=3), dict(dtype=-1),
             dict(reserved=1), dict(max_pages=1 << 30), dict(k_pages=None), dict(v_pages=None),
             dict(k_pages=FAKE + 8), dict(v_pages=FAKE + 4), dict(page_table=None),
             dict(page_table=FAKE + 2), dict(dtype=dk.E4M3), dict(k_scale=FAKE),
             dict(dtype=dk.E4M3, k_scale=FAKE), dict(v_scale=FAKE)]
BAD_ROWS = [dict(k=None), dict(v=None), dict(k=FAKE + 1), dict(dtype=dk.E4M3), dict(dtype=5),
            dict(n=0), dict(m=0), dict(m=11), dict(reserved=3), dict(rows=FAKE + 1),
            dict(start=FAKE + 2), dict(counts=FAKE + 3), dict(k_stride=NEG), dict(v_stride=NEG)]
BAD_ATTN = [dict(q=None), dict(out=None), dict(q=FAKE + 1), dict(out=FAKE + 1), dict(lse=FAKE + 2),
            dict(dtype=dk.E4M3), dict(Hq=0), dict(Hq=6), dict(T=0), dict(causal=2),
            dict(scale=-1.0), dict(scale=float("inf")), dict(scale=float("nan")), dict(path=3),
            dict(lengths=None), dict(lengths=FAKE + 1), dict(q_lengths=FAKE + 2),
            dict(q_stride=NEG), dict(out_stride=NEG), dict(T=1 << 30)]


def _call(fn, *structs, status=None):
    return fn(*[None if s is None else ctypes.byref(s) for s in structs], status, None)


@pytest.mark.parametrize("name", ["dropkv_cache_write", "dropkv_cache_read"])
def test_rows_calls_refuse_bad_arguments(name):
    fn = getattr(dk.lib(), name)
    for bad in BAD_CACHE:
        assert _call(fn, _cache(**bad), _rows()) == dk.ERR_ARG, bad
    for bad in BAD_ROWS:
        assert _call(fn, _cache(), _rows(**bad)) == dk.ERR_ARG, bad
    assert _call(fn, None, _rows()) == dk.ERR_ARG
    assert _call(fn, _cache(), None) == dk.ERR_ARG
    if not torch.cuda.is_available():
        assert _call(fn, _cache(), _rows()) == dk.ERR_UNSUPPORTED  # no CPU fallback


def test_a_list_may_be_longer_than_the_rows_of_a_write_only():
    if torch.cuda.is_available():
        pytest.skip("the accepted call would run")
    L = dk.lib()
    assert _call(L.dropkv_cache_write, _cache(), _rows(rows=FAKE, m=11)) == dk.ERR_UNSUPPORTED
    assert _call(L.dropkv_cache_read, _cache(), _rows(rows=FAKE, m=11)) == dk.ERR_ARG


def _attend(c, a, ws=FAKE, nbytes=1 << 40, status=None):
    return dk.lib().dropkv_cache_attention(None if c is None else ctypes.byref(c),
                                           None if a is None else ctypes.byref(a), ws, nbytes,
                                           status, None)


def test_attention_refuses_bad_arguments():
    for bad in BAD_CACHE:
        assert _attend(_cache(**bad), _attn()) == dk.ERR_ARG, bad
    for bad in BAD_ATTN:
        assert _attend(_cache(), _attn(**bad)) == dk.ERR_ARG, bad
    assert _attend(None, _attn()) == dk.ERR_ARG
    assert _attend(_cache(), None) == dk.ERR_ARG
    assert _attend(_cache(), _attn(), status=FAKE + 2) == dk.ERR_ARG
    need = dk.cache_attention_workspace_bytes(_cache(), _attn())
    assert need > 0
    assert _attend(_cache(), _attn(), nbytes=need - 1) == dk.ERR_WORKSPACE
    assert _attend(_cache(), _attn(), ws=None) == dk.ERR_WORKSPACE
    assert _attend(_cache(), _attn(), ws=FAKE + 8) == dk.ERR_WORKSPACE
    if not torch.cuda.is_available():
        assert _attend(_cache(), _attn(), nbytes=need) == dk.ERR_UNSUPPORTED


def test_workspace_and_path_need_no_pointers():
    empty = dict(k_pages=None, v_pages=None, page_table=None)
    a = _attn(q=None, out=None, lengths=None)
    assert dk.cache_attention_workspace_bytes(_cache(**empty), a) > 0
    assert dk.cache_attention_workspace_bytes(_cache(d=0), a) == 0
    assert dk.cache_attention_workspace_bytes(_cache(**empty), _attn(Hq=7)) == 0
    f32 = dict(dtype=dk.F32)
    assert dk.cache_attention_path(_cache(**f32), _attn(**f32)) == dk.PATH_SIMT
    assert dk.cache_attention_path(_cache(d=0), a) == -1


def test_python_calls_refuse_what_the_library_cannot_take():
    pages = torch.zeros(4, 2, 16, 8)
    table = torch.zeros(1, 4, dtype=torch.int32)
    x = torch.zeros(1, 2, 5, 8)
    n = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(TypeError, match="no CPU path"):
        dk.dropkv_cache_write(x, x, pages, pages, table)
    with pytest.raises(TypeError, match="no CPU path"):
        dk.dropkv_cache_read(pages, pages, table, 5)
    with pytest.raises(TypeError, match="no CPU path"):
        dk.dropkv_cache_attention(x, pages, pages, table, n)
    with pytest.raises(TypeError, match="no CPU path"):
        dk.evict_to_cache(x, x, x, 2, 1, [3], pages, pages, table)
    with pytest.raises(ValueError, match="overlap"):
        dk.dropkv_cache_read(pages, pages, table, 5, out=(x[:, :1].expand(1, 2, 5, 8), x))


def test_the_reference_grid_is_the_stored_format():
    grid = R.e4m3_grid()
    assert torch.equal(grid, torch.arange(127, dtype=torch.uint8).view(R.E4M3).double())


def test_the_reference_rounds_as_the_stored_format_does():
    g = torch.Generator().manual_seed(3)
    x = (torch.randn(64, 40, generator=g) * torch.exp2(torch.randint(-12, 12, (64, 1), generator=g)
                                                       .float())).bfloat16()
    v, byte = R.quantise(x.double())
    y = x.double() * torch.exp2(127 - byte.double())[:, None]
    assert (y.abs().amax(1) <= 448).all() and (y.abs().amax(1) > 224).all()
    assert torch.equal(v, y.float().to(R.E4M3).double())  # y is exact in fp32
