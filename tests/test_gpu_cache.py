"""The paged cache on the GPU: write, read and attend against plain fp64 forms."""

import math

import pytest
import torch

import cache_ref as R
import kv_cache_eviction_scores_b200 as dk
from cache_ref import BF16, E4M3, F32

pytestmark = pytest.mark.gpu
DEV = "cuda"


def pools(n_pages, Hkv, page, d, dtype, gen, fill=None):
    """(k_pages, v_pages, k_scale, v_scale) on the CPU, N(0, 1) or a constant."""
    out = []
    for _ in range(2):
        x = torch.randn(n_pages, Hkv, page, d, generator=gen) if fill is None else \
            torch.full((n_pages, Hkv, page, d), fill)
        out.append((x * (48 if dtype == E4M3 else 1)).to(dtype))
    if dtype != E4M3:
        return (*out, None, None)
    for _ in range(2):
        out.append(torch.randint(119, 124, (n_pages, Hkv, page), generator=gen, dtype=torch.uint8))
    return tuple(out)


def on(x):
    return None if x is None else x.to(DEV)


def i32(x):
    return torch.tensor(x, dtype=torch.int32)


def bits(x):
    return x.view({1: torch.uint8, 2: torch.int16, 4: torch.int32}[x.element_size()])


# ---- write --------------------------------------------------------------------

def ref_write(k, v, kp, vp, ks, vs, table, rows, start, counts):
    """The pools after a write, in plain loops."""
    kp, vp = kp.clone(), vp.clone()
    ks, vs = (x if x is None else x.clone() for x in (ks, vs))
    B, Hkv, n, d = k.shape
    page = kp.shape[2]
    for b in range(B):
        for h in range(Hkv):
            for i in range(int(counts[b])):
                r = i if rows is None else int(rows[b, h, i])
                if r == -1:
                    continue
                slot = int(start[b]) + i
                p, o = int(table[b, slot // page]), slot % page
                for x, pool, sc in ((k, kp, ks), (v, vp, vs)):
                    if sc is None:
                        pool[p, h, o] = x[b, h, r].to(pool.dtype)
                    else:
                        val, byte = R.quantise(x[b, h, r].double()[None])
                        pool[p, h, o] = val[0].float().to(E4M3)
                        sc[p, h, o] = byte[0]
    return kp, vp, ks, vs


@pytest.mark.parametrize("src", [BF16, F32])
@pytest.mark.parametrize("dtype", [BF16, F32, E4M3])
@pytest.mark.parametrize("d,page,Hkv", [(128, 16, 2), (8, 1, 3), (33, 24, 1), (80, 7, 2),
                                        (256, 5, 1), (1, 64, 2)])
@pytest.mark.parametrize("listed", [False, True])
def test_write_bits(src, dtype, d, page, Hkv, listed):
    g = torch.Generator().manual_seed(d * 100 + page)
    B, n = 3, 21
    k, v = (torch.randn(B, Hkv, n, d, generator=g).to(src) for _ in range(2))
    counts, start = i32([21, 0, 13]), i32([0, 4, 9])
    rows = None
    if listed:
        rows = torch.stack([torch.randperm(n, generator=g) for _ in range(B * Hkv)])
        rows = rows.view(B, Hkv, n).to(torch.int32)
        rows[:, :, 11] = -1
    table, n_pages = R.table_for([21, 4, 22], page, g)
    kp, vp, ks, vs = pools(n_pages, Hkv, page, d, dtype, g)
    want = ref_write(k, v, kp, vp, ks, vs, table, rows, start, counts)
    got = [on(x) for x in (kp, vp, ks, vs)]
    dk.dropkv_cache_write(on(k), on(v), got[0], got[1], on(table), rows=on(rows), start=on(start),
                          counts=on(counts), k_scale=got[2], v_scale=got[3], sync=True)
    for a, b in zip(got, want):
        if b is not None:
            assert torch.equal(bits(a.cpu()), bits(b))


def test_write_from_token_major_rows():
    g = torch.Generator().manual_seed(1)
    k, v = (torch.randn(2, 9, 3, 64, generator=g).to(BF16) for _ in range(2))  # [B, n, Hkv, d]
    table, n_pages = R.table_for([9, 9], 4, g)
    kp, vp, _, _ = pools(n_pages, 3, 4, 64, BF16, g)
    want = ref_write(k.transpose(1, 2), v.transpose(1, 2), kp, vp, None, None, table, None,
                     [0, 0], [9, 9])
    kd, vd = on(kp), on(vp)
    dk.dropkv_cache_write(on(k).transpose(1, 2), on(v).transpose(1, 2), kd, vd, on(table),
                          sync=True)
    assert torch.equal(kd.cpu(), want[0]) and torch.equal(vd.cpu(), want[1])


@pytest.mark.parametrize("d", [64, 33])
def test_write_e4m3_special_rows(d):
    x = torch.zeros(1, 1, 12, d)
    x[0, 0, 1, 0] = 448.0                       # the border of a scale, and just over it
    x[0, 0, 2, 0] = 448.0 * (1 + 2 ** -23)
    x[0, 0, 3] = -torch.tensor([3.0, 5.0, 7.0, 9.0, 1.0625, 17.0, 19.0, 0.0]).repeat(d)[:d]
    x[0, 0, 3, 1] = 448.0                       # ties of the grid
    x[0, 0, 4, d - 1] = math.inf
    x[0, 0, 5, 3] = math.nan
    x[0, 0, 6, 2] = 3e38                        # the largest scales
    x[0, 0, 7, 2] = 1e-38                       # the smallest, and subnormals below it
    x[0, 0, 8, 2] = 1e-44
    x[0, 0, 9, :2] = torch.tensor([1.0, 2.0 ** -17])  # far below the row's maximum
    x[0, 0, 10] = -0.0
    x[0, 0, 11] = 2.0 ** -126
    want, byte = R.quantise(x.double())
    kp = torch.zeros(1, 1, 12, d).to(E4M3).to(DEV)
    vp, ks, vs = kp.clone(), *(torch.full((1, 1, 12), 9, dtype=torch.uint8, device=DEV)
                               for _ in range(2))
    table = torch.zeros(1, 1, dtype=torch.int32, device=DEV)
    dk.dropkv_cache_write(on(x), on(-x), kp, vp, table, k_scale=ks, v_scale=vs, sync=True)
    assert torch.equal(ks.cpu(), byte) and torch.equal(vs.cpu(), byte)
    assert torch.equal(kp.cpu().double().nan_to_num(9999.0), want.nan_to_num(9999.0))
    back, _ = dk.dropkv_cache_read(kp, vp, table, 12, k_scale=ks, v_scale=vs, dtype=F32)
    ref = (want * torch.exp2(byte.double() - 127)[..., None]).float()
    bad = byte == 255
    assert torch.isnan(back.cpu()[bad]).all()
    assert torch.equal(back.cpu()[~bad], ref[~bad])


# ---- read -----------------------------------------------------------------------

@pytest.mark.parametrize("dst", [BF16, F32])
@pytest.mark.parametrize("dtype", [BF16, F32, E4M3])
@pytest.mark.parametrize("d,page,Hkv", [(128, 16, 2), (8, 1, 3), (33, 24, 1), (80, 7, 2),
                                        (256, 5, 1)])
@pytest.mark.parametrize("listed", [False, True])
def test_read_values(dst, dtype, d, page, Hkv, listed):
    g = torch.Generator().manual_seed(d + page)
    B, n, slots = 3, 17, 40
    table, n_pages = R.table_for([slots] * B, page, g)
    kp, vp, ks, vs = pools(n_pages, Hkv, page, d, dtype, g)
    counts, start = i32([17, 0, 5]), i32([3, 0, 22])
    rows = None
    if listed:
        rows = torch.randint(0, 18, (B, Hkv, n), generator=g, dtype=torch.int32)
        rows[:, :, 2] = -1
    out = [torch.full((B, n, Hkv, d), 0.25, dtype=dst, device=DEV).transpose(1, 2)
           for _ in range(2)]  # token-major
    got = dk.dropkv_cache_read(on(kp), on(vp), on(table), n, rows=on(rows), start=on(start),
                               counts=on(counts), k_scale=on(ks), v_scale=on(vs), out=tuple(out),
                               sync=True)
    assert got[0] is out[0] and got[1] is out[1]
    for x, pool, sc in ((got[0], kp, ks), (got[1], vp, vs)):
        want = torch.full((B, Hkv, n, d), 0.25, dtype=torch.float64)
        for b in range(B):
            for h in range(Hkv):
                line = R.held(pool, sc, table, b, h, slots)
                for i in range(int(counts[b])):
                    at = i if rows is None else int(rows[b, h, i])
                    if at != -1:
                        want[b, h, i] = line[int(start[b]) + at]
        assert torch.equal(x.cpu().double(), want.to(dst).double())


def test_rows_out_of_range_are_left_out_and_reported():
    g = torch.Generator().manual_seed(5)
    B, Hkv, n, d, page = 2, 2, 8, 16, 4
    k = torch.randn(B, Hkv, n, d, generator=g)
    table = i32([[0, 1], [2, 3]])

    def run(rows=None, start=None, counts=None, tab=table):
        kp = torch.full((4, Hkv, page, d), 5.0, device=DEV)
        vp = kp.clone()
        status = torch.full((1,), 77, dtype=torch.int32, device=DEV)
        dk.dropkv_cache_write(on(k), on(k), kp, vp, on(tab), rows=on(rows),
                              start=on(start), counts=on(counts), status=status)
        out = torch.full((B, Hkv, n, d), 5.0, device=DEV)
        st2 = torch.full((1,), 77, dtype=torch.int32, device=DEV)
        dk.dropkv_cache_read(kp, vp, on(tab), n, rows=on(rows), start=on(start),
                             counts=on(counts), out=(out, out.clone()), status=st2)
        return int(status), int(st2), kp.cpu(), out.cpu()

    assert run()[:2] == (dk.OK, dk.OK)
    # the second sequence's last page does not exist: its slots are left out
    for bad in (4, -1, 2 ** 31 - 1):
        tab = table.clone()
        tab[1, 1] = bad
        s, r, kp, out = run(tab=tab)
        assert s == dk.ERR_ARG and r == dk.ERR_ARG
        assert (kp[3] == 5).all() and torch.equal(out[0], k[0]) and torch.equal(out[1, :, :4],
                                                                                 k[1, :, :4])
        assert (out[1, :, 4:] == 5).all()
    # slots behind the table's last page, and before the first
    for s0 in (1, 8, 2 ** 31 - 1, -1):
        s, r, kp, out = run(start=i32([0, s0]))
        assert s == dk.ERR_ARG and r == dk.ERR_ARG and torch.equal(out[0], k[0])
    # rows that the tensors do not have
    rows = torch.arange(n, dtype=torch.int32).repeat(B, Hkv, 1)
    rows[0, 1, 3] = 8
    rows[1, 0, 0] = -2
    s, r, kp, out = run(rows=rows)
    assert s == dk.ERR_ARG and r == dk.ERR_ARG
    assert (kp[0, 1, 3] == 5).all() and (kp[2, 0, 0] == 5).all() and (kp[0, 0] == k[0, 0, :4]).all()
    # counts are clamped
    s, r, kp, out = run(counts=i32([9, -3]))
    assert s == dk.ERR_ARG and r == dk.ERR_ARG
    assert torch.equal(out[0], k[0]) and (out[1] == 5).all() and (kp[2:] == 5).all()
    with pytest.raises(dk.DropKVError):
        dk.dropkv_cache_write(on(k), on(k), torch.zeros(4, Hkv, page, d, device=DEV),
                              torch.zeros(4, Hkv, page, d, device=DEV), on(table),
                              start=on(i32([0, 1])), sync=True)


def test_read_and_write_past_32_bit_offsets():
    # pools of more than 2^32 elements; the pages used are at both ends
    Hkv, page, d = 1, 1024, 256
    n_pages = (1 << 32) // (Hkv * page * d) + 8
    kp, vp = (torch.empty(n_pages, Hkv, page, d, dtype=torch.uint8, device=DEV).view(E4M3)
              for _ in range(2))
    ks, vs = (torch.zeros(n_pages, Hkv, page, dtype=torch.uint8, device=DEV) for _ in range(2))
    table = i32([[n_pages - 1, 0, n_pages - 2]])
    g = torch.Generator().manual_seed(2)
    x = torch.randn(1, Hkv, 3 * page, d, generator=g).to(BF16)
    sc = dict(k_scale=ks, v_scale=vs)
    dk.dropkv_cache_write(on(x), on(x), kp, vp, on(table), sync=True, **sc)
    k, v = dk.dropkv_cache_read(kp, vp, on(table), 3 * page, sync=True, **sc)
    val, byte = R.quantise(x.double())
    want = (val * torch.exp2(byte.double() - 127)[..., None]).to(BF16)
    assert torch.equal(k.cpu(), want) and torch.equal(v.cpu(), want)
    q = torch.randn(1, 4, 3, d, generator=g).to(BF16)
    L = i32([2 * page + 5])
    out, lse = dk.dropkv_cache_attention(on(q), kp, vp, on(table), on(L), return_lse=True,
                                         sync=True, **sc)
    small = [on(torch.stack([p[n_pages - 1].cpu().view(torch.uint8), p[0].cpu().view(torch.uint8),
                             p[n_pages - 2].cpu().view(torch.uint8)])) for p in (kp, vp)]
    near = [p.view(E4M3) for p in small]
    nsc = [torch.stack([s[n_pages - 1], s[0], s[n_pages - 2]]) for s in (ks, vs)]
    out2, lse2 = dk.dropkv_cache_attention(on(q), *near, on(i32([[0, 1, 2]])), on(L),
                                           k_scale=nsc[0], v_scale=nsc[1], return_lse=True)
    assert torch.equal(out, out2) and torch.equal(lse, lse2)


# ---- attend -----------------------------------------------------------------------

def check_attend(q, kp, vp, ks, vs, table, lengths, q_lengths, causal=True, scale=None, path="auto",
                 n_max=None):
    B, Hq, T, d = q.shape
    out = torch.full((B, Hq, T, d), 3.0, dtype=q.dtype, device=DEV)
    lse = torch.full((B, Hq, T), 3.0, device=DEV)
    dk.dropkv_cache_attention(on(q), on(kp), on(vp), on(table), on(i32(lengths)),
                              q_lengths=on(i32(q_lengths)), causal=causal, scale=scale, path=path,
                              k_scale=on(ks), v_scale=on(vs), out=out, lse=lse, sync=True)
    s = scale if scale is not None else 1.0 / math.sqrt(d)
    ref = R.attend(q, kp, vp, table, lengths, q_lengths, s, causal, ks, vs)
    compare(out, lse, ref, q_lengths, d, max(lengths), q.dtype, path != "simt" and q.dtype == BF16)
    return out, lse


def compare(out, lse, ref, q_lengths, d, n, dtype, low_p):
    tol, ltol = R.bounds(*ref, d, n, dtype, low_p)
    got, glse = out.cpu().double(), lse.cpu().double()
    for b in range(out.shape[0]):
        c = int(q_lengths[b])
        if c < out.shape[2]:  # rows behind the chunk stay as they were
            assert (got[b, :, c:] == 3).all() and (glse[b, :, c:] == 3).all()
        err = (got[b, :, :c] - ref[0][b, :, :c]).abs()
        assert torch.isfinite(got[b, :, :c]).all()
        assert bool((err <= tol[b, :, :c]).all()), float((err / tol[b, :, :c]).max())
        w, x = ref[1][b, :, :c], glse[b, :, :c]
        assert torch.equal(torch.isinf(w), torch.isinf(x))
        fin = torch.isfinite(w)
        lerr = (x - w).abs()[fin]
        assert (x[~fin] == -math.inf).all()
        assert bool((lerr <= ltol[b, :, :c][fin]).all()), float((lerr / ltol[b, :, :c][fin]).max())


TYPES = [(BF16, BF16, "auto"), (BF16, E4M3, "auto"), (BF16, BF16, "simt"), (BF16, E4M3, "simt"),
         (BF16, F32, "auto"), (F32, F32, "auto"), (F32, E4M3, "auto"), (F32, BF16, "auto")]


@pytest.mark.parametrize("qt,pt,path", TYPES)
@pytest.mark.parametrize("Hq,Hkv,d,page,T,lengths,q_lengths,causal", [
    (4, 2, 128, 16, 1, [1, 2, 17, 300], [1, 1, 1, 1], True),
    (8, 2, 128, 64, 1, [515, 64, 128], [1, 0, 1], True),
    (7, 1, 128, 24, 3, [200, 3, 131], [3, 3, 2], True),
    (8, 1, 64, 16, 5, [129, 70], [5, 4], True),
    (4, 4, 64, 7, 2, [90, 31], [2, 1], False),
    (32, 8, 128, 32, 4, [150], [4], True),
    (6, 2, 128, 128, 37, [333, 40], [37, 5], True),
    (4, 1, 128, 16, 70, [70, 200], [70, 33], False),
    (6, 2, 80, 24, 9, [100, 45], [9, 2], True),
    (4, 2, 8, 3, 6, [22, 9], [6, 1], True),
    (2, 1, 256, 16, 3, [67, 5], [3, 3], True),
    (3, 3, 1, 1, 4, [33, 7], [4, 4], True),
])
def test_attend_values(qt, pt, path, Hq, Hkv, d, page, T, lengths, q_lengths, causal):
    g = torch.Generator().manual_seed(Hq * d + T)
    table, n_pages = R.table_for(lengths, page, g)
    kp, vp, ks, vs = pools(n_pages, Hkv, page, d, pt, g)
    q = torch.randn(len(lengths), Hq, T, d, generator=g).to(qt)
    check_attend(q, kp, vp, ks, vs, table, lengths, q_lengths, causal, path=path)


@pytest.mark.parametrize("pt", [BF16, E4M3, F32])
@pytest.mark.parametrize("d", [128, 64, 40])
def test_attend_rows_that_see_nothing(pt, d):
    # no slots, no tokens, more tokens than slots
    g = torch.Generator().manual_seed(d)
    lengths, q_lengths = [0, 5, 3, 40], [2, 0, 6, 6]
    table, n_pages = R.table_for(lengths, 16, g)
    kp, vp, ks, vs = pools(n_pages, 2, 16, d, pt, g)
    q = torch.randn(4, 8, 6, d, generator=g).to(F32 if pt == F32 else BF16)
    for causal in (True, False):
        check_attend(q, kp, vp, ks, vs, table, lengths, q_lengths, causal)


def test_attend_nothing_at_all():
    g = torch.Generator().manual_seed(1)
    kp, vp, _, _ = pools(2, 2, 16, 128, BF16, g)
    q = torch.randn(3, 4, 2, 128, generator=g).to(BF16)
    table = torch.full((3, 1), -1, dtype=torch.int32)
    check_attend(q, kp, vp, None, None, table, [0, 0, 0], [0, 0, 0])
    check_attend(q, kp, vp, None, None, table, [0, 0, 0], [2, 1, 0])


@pytest.mark.parametrize("pt", [BF16, E4M3, F32])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("T", [4, 50])
def test_attend_ignores_whatever_a_row_does_not_see(pt, bad, T):
    g = torch.Generator().manual_seed(T)
    page, d, Hkv, Hq = 16, 128, 2, 8
    lengths, q_lengths = [150, 77], [T, T - 3]
    table, n_pages = R.table_for([160, 90], page, g)
    kp, vp, ks, vs = pools(n_pages, Hkv, page, d, pt, g)
    q = torch.randn(2, Hq, T, d, generator=g).to(F32 if pt == F32 else BF16)
    if pt == E4M3 and not math.isnan(bad):
        bad = math.nan  # the format has no infinities
    # everything behind the last slot, and the last token's own slot: only the
    # last row sees the latter
    for b, L in enumerate(lengths):
        for j in range(L - 1, [160, 90][b]):
            p, o = int(table[b, j // page]), j % page
            kp[p, :, o] = torch.tensor(bad).to(pt)
            vp[p, :, o] = torch.tensor(bad).to(pt)
            if ks is not None:
                ks[p, :, o] = vs[p, :, o] = 255
    clean = [L - 1 for L in lengths]
    n1 = [n - 1 for n in q_lengths]
    out = torch.full((2, Hq, T, d), 3.0, dtype=q.dtype, device=DEV)
    lse = torch.full((2, Hq, T), 3.0, device=DEV)
    dk.dropkv_cache_attention(on(q), on(kp), on(vp), on(table), on(i32(lengths)),
                              q_lengths=on(i32(q_lengths)), k_scale=on(ks), v_scale=on(vs),
                              out=out, lse=lse, sync=True)
    ref = R.attend(q, kp, vp, table, clean, n1, 1.0 / math.sqrt(d), True, ks, vs)
    for b in range(2):
        if bad != -math.inf or pt == E4M3:  # -inf logits of either sign: no claim
            assert torch.isnan(out[b, :, n1[b]].float()).all()
        out[b, :, n1[b]:] = 3.0
        lse[b, :, n1[b]:] = 3.0
    compare(out, lse, ref, n1, d, max(clean), q.dtype, q.dtype == BF16)


@pytest.mark.parametrize("path", ["auto", "simt"])
@pytest.mark.parametrize("T", [1, 40])
def test_attend_leaves_bad_pages_out_and_reports_them(path, T):
    g = torch.Generator().manual_seed(9)
    d, page, L = 128, 16, 100
    table, n_pages = R.table_for([L, L], page, g)
    kp, vp, _, _ = pools(n_pages, 2, page, d, BF16, g)
    q = torch.randn(2, 4, T, d, generator=g).to(BF16)
    full = dk.dropkv_cache_attention(on(q), on(kp), on(vp), on(table), on(i32([L, L])), path=path)
    for bad in (-1, n_pages, 2 ** 31 - 1):
        tab = table.clone()
        tab[1, 2] = bad
        status = torch.zeros(1, dtype=torch.int32, device=DEV)
        out = dk.dropkv_cache_attention(on(q), on(kp), on(vp), on(tab), on(i32([L, L])), path=path,
                                        status=status, causal=False)
        assert int(status) == dk.ERR_ARG
        assert torch.isfinite(out.float()).all()
        # without the page: the slots before and after it
        keep = [j for j in range(L) if j // page != 2]
        K, V = (torch.stack([R.held(p, None, table, 1, h, L)[keep] for h in range(2)])
                for p in (kp, vp))
        S = torch.einsum("hgtd,hjd->hgtj", q[1].double().view(2, 2, T, d), K) / math.sqrt(d)
        ref = torch.einsum("hgtj,hjd->hgtd", S.softmax(-1), V).reshape(4, T, d)
        # two roundings to bf16, as above
        A = torch.einsum("hgtj,hjd->hgtd", S.softmax(-1), V.abs()).reshape(4, T, d)
        assert bool(((out[1].cpu().double() - ref).abs() <= 2 ** -8 * 1.02 * (A + ref.abs())).all())
    # lengths and chunk lengths outside their ranges are clamped
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    lens, ql = on(i32([L, -5])), on(i32([T + 1, T]))
    out = dk.dropkv_cache_attention(on(q), on(kp), on(vp), on(table), lens, q_lengths=ql,
                                    status=status, path=path)
    assert int(status) == dk.ERR_ARG
    assert torch.equal(out[0], full[0]) and (out[1] == 0).all()
    with pytest.raises(dk.DropKVError):
        dk.dropkv_cache_attention(on(q), on(kp), on(vp), on(table), lens, path=path, sync=True)


@pytest.mark.parametrize("pt", [BF16, E4M3, F32])
@pytest.mark.parametrize("T", [1, 33])
def test_attend_strided_and_unaligned(pt, T):
    g = torch.Generator().manual_seed(T)
    B, Hq, Hkv, d, page = 2, 8, 2, 128, 16
    lengths, ql = [200, 93], [T, max(1, T - 5)]
    table, n_pages = R.table_for(lengths, page, g)
    kp, vp, ks, vs = pools(n_pages, Hkv, page, d, pt, g)
    qt = F32 if pt == F32 else BF16
    q = torch.randn(B, T, Hq, d, generator=g).to(qt)
    args = (on(kp), on(vp), on(table), on(i32(lengths)))
    kw = dict(q_lengths=on(i32(ql)), k_scale=on(ks), v_scale=on(vs))
    want = dk.dropkv_cache_attention(on(q).transpose(1, 2).contiguous(), *args, **kw)
    out = torch.zeros(B, T, Hq, d, dtype=qt, device=DEV)
    dk.dropkv_cache_attention(on(q).transpose(1, 2), *args, out=out.transpose(1, 2), **kw)
    assert torch.equal(out.transpose(1, 2), want)
    # rows of 129 values: no 16-byte alignment (the CUDA-core path)
    wide = torch.zeros(B, Hq, T, d + 1, dtype=qt, device=DEV)
    wide[..., 1:] = on(q).transpose(1, 2)
    got = torch.zeros(B, Hq, T, d + 1, dtype=qt, device=DEV)
    dk.dropkv_cache_attention(wide[..., 1:], *args, out=got[..., :d], **kw)
    ref = R.attend(q.transpose(1, 2), kp, vp, table, lengths, ql, 1 / math.sqrt(d), True, ks, vs)
    tol, _ = R.bounds(*ref, d, 200, qt, False)
    for b in range(B):
        err = (got[b, :, :ql[b], :d].cpu().double() - ref[0][b, :, :ql[b]]).abs()
        assert (err <= tol[b, :, :ql[b]]).all()
    assert (got[..., d] == 0).all()


@pytest.mark.parametrize("qt,pt", [(BF16, BF16), (BF16, E4M3), (F32, F32)])
def test_attend_peaked_and_shifted_logits(qt, pt):
    # growing logits move the running maximum at every slot; a scale of 4 peaks them
    g = torch.Generator().manual_seed(4)
    d, page, L = 128, 16, 400
    table, n_pages = R.table_for([L], page, g)
    kp, vp, ks, vs = pools(n_pages, 1, page, d, pt, g)
    q = torch.randn(1, 4, 3, d, generator=g).to(qt)
    for order in (1, -1):
        for j in range(L):
            p, o = int(table[0, j // page]), j % page
            up = (j if order == 1 else L - j) / L
            kp[p, 0, o] = (q[0, 0, 0].float() * up * (24 if pt == E4M3 else 1)).to(pt)
        check_attend(q, kp, vp, ks, vs, table, [L], [3])
        check_attend(q, kp, vp, ks, vs, table, [L], [3], scale=0.5)


@pytest.mark.parametrize("T", [1, 2, 130])
def test_attend_splits_agree_with_one_piece(T):
    # a batch in which this sequence's tiles are cut differently gives the same
    # values up to rounding, and repeated calls the same bits
    g = torch.Generator().manual_seed(T)
    d, page, L, Hq, Hkv = 128, 64, 4000, 8, 2
    table, n_pages = R.table_for([L, 1000, 17], page, g)
    kp, vp, ks, vs = (on(x) for x in pools(n_pages, Hkv, page, d, E4M3, g))
    q = on(torch.randn(3, Hq, T, d, generator=g).to(BF16))
    lens, tab = on(i32([L, 1000, 17])), on(table)
    sc = dict(k_scale=ks, v_scale=vs)
    a, la = dk.dropkv_cache_attention(q, kp, vp, tab, lens, return_lse=True, **sc)
    b, lb = dk.dropkv_cache_attention(q, kp, vp, tab, lens, return_lse=True, **sc)
    assert torch.equal(a, b) and torch.equal(la, lb)
    # A = sum_j p_j |v_j|: each result is within 2^-8 (A + |out|) of the exact one (the roundings
    # of P and of the output); A itself comes out rounded once more, hence the 1.02
    vabs = (vp.view(torch.uint8) & 0x7F).view(E4M3)
    A = dk.dropkv_cache_attention(q, kp, vabs, tab, lens, path="simt", **sc).float()
    tol = 2 * 2 ** -8 * 1.02 * (A + a.float().abs()) + 1e-6
    for i in range(3):
        x, lx = dk.dropkv_cache_attention(q[i:i + 1], kp, vp, tab[i:i + 1].contiguous(),
                                          lens[i:i + 1].contiguous(), return_lse=True, **sc)
        fin = torch.isfinite(lx[0])
        assert bool(((x[0].float() - a[i].float()).abs() <= tol[i]).all())
        assert ((lx[0] - la[i]).abs()[fin] < 1e-4).all()


# ---- together, on streams, in graphs ------------------------------------------------

def test_streams_and_two_calls_at_once():
    g = torch.Generator().manual_seed(8)
    d, page, Hq, Hkv = 128, 16, 8, 2
    table, n_pages = R.table_for([900, 700], page, g)
    kp, vp, _, _ = (on(x) for x in pools(n_pages, Hkv, page, d, BF16, g))
    tab, lens = on(table), on(i32([900, 700]))
    qs = [on(torch.randn(2, Hq, T, d, generator=g).to(BF16)) for T in (1, 40)]
    want = [dk.dropkv_cache_attention(q, kp, vp, tab, lens) for q in qs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in qs]
    got = [[], []]
    for _ in range(5):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i].append(dk.dropkv_cache_attention(qs[i], kp, vp, tab, lens))
    torch.cuda.synchronize()
    for w, xs in zip(want, got):
        assert all(torch.equal(w, x) for x in xs)


@pytest.mark.parametrize("pt", [BF16, E4M3])
def test_a_decoding_step_replayed_from_a_graph(pt):
    # append one token, count it, attend: captured once, replayed over growing caches
    g = torch.Generator().manual_seed(6)
    B, Hq, Hkv, d, page, steps = 3, 8, 2, 128, 16, 6
    first = [30, 0, 15]
    table, n_pages = R.table_for([n + steps for n in first], page, g)
    kp, vp, ks, vs = pools(n_pages, Hkv, page, d, pt, g)
    kd, vd, ksd, vsd, tab = (on(x) for x in (kp, vp, ks, vs, table))
    lens = on(i32(first))
    new = [[torch.randn(B, H, 1, d, generator=g).to(BF16) for H in (Hq, Hkv, Hkv)]
           for _ in range(steps)]
    q, k, v = (x.to(DEV) for x in new[0])
    sc = dict(k_scale=ksd, v_scale=vsd)
    out, lse = torch.zeros_like(q), torch.zeros(B, Hq, 1, device=DEV)
    ws = torch.empty(64 << 20, dtype=torch.uint8, device=DEV)

    def step():
        dk.dropkv_cache_write(k, v, kd, vd, tab, start=lens, **sc)
        lens.add_(1)
        dk.dropkv_cache_attention(q, kd, vd, tab, lens, out=out, lse=lse, workspace=ws, **sc)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    keep = [x.clone() for x in (kd, vd, lens)]
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    kd.copy_(keep[0]), vd.copy_(keep[1]), lens.copy_(keep[2])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    n = list(first)
    for s in range(steps):
        for x, y in zip((q, k, v), new[s]):
            x.copy_(y)
        graph.replay()
        torch.cuda.synchronize()
        kp, vp, ks, vs = ref_write(new[s][1], new[s][2], kp, vp, ks, vs, table, None, n, [1] * B)
        n = [x + 1 for x in n]
        ref = R.attend(new[s][0], kp, vp, table, n, [1] * B, 1 / math.sqrt(d), True, ks, vs)
        compare(out, lse, ref, [1] * B, d, max(n), BF16, True)
    assert lens.tolist() == n


@pytest.mark.parametrize("pt", [BF16, E4M3, F32])
def test_evict_write_decode_read_and_score_again(pt):
    g = torch.Generator().manual_seed(12)
    B, Hq, Hkv, d, w, n, page = 2, 8, 2, 128, 16, 400, 16
    lengths, keep = [400, 333], [100, 61]
    dt = F32 if pt == F32 else BF16
    q, k, v = (torch.randn(B, H, m, d, generator=g).to(dt) for H, m in ((Hq, w), (Hkv, n), (Hkv, n)))
    T = 5
    table, n_pages = R.table_for([x + T for x in keep], page, g)
    kp, vp, ks, vs = pools(n_pages, Hkv, page, d, pt, g)
    kd, vd, ksd, vsd, tab = (on(x) for x in (kp, vp, ks, vs, table))
    sc = dict(k_scale=ksd, v_scale=vsd)
    counts, scores, keep_idx, evict_idx = dk.evict_to_cache(
        on(q), on(k), on(v), w, 7, keep, kd, vd, tab, lengths, **sc)
    s2, k2, e2 = dk.evict(on(q), on(k), on(v), w, 7, keep, lengths)
    assert torch.equal(keep_idx, k2) and torch.equal(evict_idx, e2)
    assert torch.equal(scores.nan_to_num(-1.0), s2.nan_to_num(-1.0)) and counts.tolist() == keep
    kp, vp, ks, vs = ref_write(k, v, kp, vp, ks, vs, table, keep_idx.cpu(), [0, 0], keep)
    # five new tokens: written, then attended in one chunk
    qn, kn, vn = (torch.randn(B, H, T, d, generator=g).to(dt) for H in (Hq, Hkv, Hkv))
    dk.dropkv_cache_write(on(kn), on(vn), kd, vd, tab, start=counts, **sc)
    lens = counts + T
    out, lse = dk.dropkv_cache_attention(on(qn), kd, vd, tab, lens, return_lse=True, **sc)
    kp, vp, ks, vs = ref_write(kn, vn, kp, vp, ks, vs, table, None, keep, [T, T])
    now = [x + T for x in keep]
    ref = R.attend(qn, kp, vp, table, now, [T, T], 1 / math.sqrt(d), True, ks, vs)
    compare(out, lse, ref, [T, T], d, max(now), dt, dt == BF16)
    # one token at a time gives the chunk's rows
    for t in range(T):
        at = counts + t + 1
        o, l1 = dk.dropkv_cache_attention(on(qn[:, :, t:t + 1].contiguous()), kd, vd, tab,
                                          at.to(torch.int32), return_lse=True, **sc)
        sub = tuple(x[:, :, t:t + 1] for x in ref)
        compare(o, l1, sub, [1, 1], d, max(now), dt, dt == BF16)
    # back to dense rows, and scored again with the new tokens as the window
    kb, vb = dk.dropkv_cache_read(kd, vd, tab, max(now), counts=lens.to(torch.int32), dtype=dt,
                                  sync=True, **sc)
    for b in range(B):
        for h in range(Hkv):
            want = R.held(kp, ks, table, b, h, now[b])
            assert torch.equal(kb[b, h, :now[b]].cpu().double(), want.to(dt).double())
    again = dk.dropkv_scores(on(qn), kb, vb, T, 7, now)
    direct = torch.zeros(B, Hkv, max(now), d, dtype=dt), torch.zeros(B, Hkv, max(now), d, dtype=dt)
    for b in range(B):
        for h in range(Hkv):
            direct[0][b, h, :now[b]] = R.held(kp, ks, table, b, h, now[b]).to(dt)
            direct[1][b, h, :now[b]] = R.held(vp, vs, table, b, h, now[b]).to(dt)
    other = dk.dropkv_scores(on(qn), on(direct[0]), on(direct[1]), T, 7, now)
    assert torch.equal(again.nan_to_num(-1.0), other.nan_to_num(-1.0))


def test_empty_calls_change_nothing():
    g = torch.Generator().manual_seed(1)
    kp, vp, _, _ = (on(x) for x in pools(2, 2, 4, 16, F32, g))
    a = kp.clone()
    table = on(i32([[0]]))
    z = torch.zeros(1, 2, 0, 16, device=DEV)
    dk.dropkv_cache_write(z, z, kp, vp, table, sync=True)
    assert dk.dropkv_cache_read(kp, vp, table, 0)[0].shape == (1, 2, 0, 16)
    assert dk.dropkv_cache_attention(torch.zeros(1, 4, 0, 16, device=DEV), kp, vp, table,
                                     on(i32([3]))).shape == (1, 4, 0, 16)
    assert torch.equal(a, kp)


def test_refusals_on_the_gpu():
    g = torch.Generator().manual_seed(1)
    kp, vp, _, _ = (on(x) for x in pools(2, 2, 4, 16, F32, g))
    table, L = on(i32([[0, 1]])), on(i32([3]))
    q = torch.zeros(1, 4, 1, 16, device=DEV)
    call = dk.dropkv_cache_attention
    for bad in (lambda: call(q[:, :3], kp, vp, table, L), lambda: call(q, kp, vp[:1], table, L),
                lambda: call(q, kp, vp, table, None), lambda: call(q, kp, vp, table, L, scale=-1.0),
                lambda: call(q, kp, vp, table, L, scale=0.0),
                lambda: call(q, kp, vp, table[0], L),
                lambda: call(q, kp, vp, table, L, lse=torch.zeros(1, 4, device=DEV)),
                lambda: call(q, kp, vp, table, L, out=q.expand(1, 4, 1, 16)[:, :1].expand(1, 4, 1, 16)),
                lambda: call(q, kp, vp, table, on(i32([3, 4]))),
                lambda: call(q, kp.transpose(2, 3), vp.transpose(2, 3), table, L),
                lambda: call(q, kp.to(E4M3), vp.to(E4M3), table, L)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: call(q.half(), kp, vp, table, L), lambda: call(q, kp, vp, table.long(), L),
                lambda: call(q, kp, vp, table, L.float()), lambda: call(q.cpu(), kp, vp, table, L),
                lambda: call(q, kp, vp, table, L, status=torch.zeros(1, device=DEV)),
                lambda: call(q, kp.half(), vp.half(), table, L)):
        with pytest.raises(TypeError):
            bad()
    with pytest.raises(dk.DropKVError):  # fp32 has no tensor path
        call(q, kp, vp, table, L, path="tensor")
    with pytest.raises(ValueError):
        dk.evict_to_cache(torch.zeros(1, 4, 2, 16, device=DEV), torch.zeros(1, 2, 20, 16, device=DEV),
                          torch.zeros(1, 2, 20, 16, device=DEV), 2, 1, [9], kp, vp, table)
