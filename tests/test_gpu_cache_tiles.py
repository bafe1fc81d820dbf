"""Cache attention at the borders of its kernels (8, 16 and 128 query rows per KV head
on the tensor path, 128 on the CUDA-core path), over the formats' scales, and in
graphs, against a plain fp64 form on the GPU."""

import math

import pytest
import torch

import cache_ref as R
import kv_cache_eviction_scores_b200 as dk
from cache_ref import BF16, E4M3, F32

pytestmark = pytest.mark.gpu
DEV = "cuda"


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def make(lengths, Hq, Hkv, T, d, page, qt, pt, seed, k_bytes=(119, 124), v_bytes=(119, 124), q_scale=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    table, n_pages = R.table_for(lengths, page, torch.Generator().manual_seed(seed))
    s = {"table": table.to(DEV)}
    for x in "kv":
        val = torch.randn(n_pages, Hkv, page, d, generator=g, device=DEV)
        s[x] = (val * 48).to(pt) if pt == E4M3 else val.to(pt)
        lo, hi = k_bytes if x == "k" else v_bytes
        s[x + "s"] = torch.randint(lo, hi, (n_pages, Hkv, page), generator=g, device=DEV,
                                   dtype=torch.uint8) if pt == E4M3 else None
    s["q"] = (torch.randn(len(lengths), Hq, T, d, generator=g, device=DEV) * q_scale).to(qt)
    return s


def dense(pages, scale, table, L):
    """The first L slots of a sequence [Hkv, L, d] in fp64."""
    page = pages.shape[2]
    n = -(-L // page)
    x = pages[table[:n].long()].double()
    if scale is not None:
        x = x * torch.exp2(scale[table[:n].long()].double() - 127)[..., None]
    return x.permute(1, 0, 2, 3).reshape(pages.shape[1], n * page, pages.shape[3])[:, :L]


def check(s, lengths, q_lengths, causal=True, path="auto", scale=None, low_p=None):
    q = s["q"]
    B, Hq, T, d = q.shape
    Hkv = s["k"].shape[1]
    out = torch.full_like(q, 3.0)
    lse = torch.full((B, Hq, T), 3.0, device=DEV)
    dk.dropkv_cache_attention(q, s["k"], s["v"], s["table"], i32(lengths), q_lengths=i32(q_lengths),
                              causal=causal, path=path, k_scale=s["ks"], v_scale=s["vs"], out=out,
                              lse=lse, scale=scale, sync=True)
    sc = scale or 1.0 / math.sqrt(d)
    if low_p is None:
        low_p = path != "simt" and q.dtype == BF16
    for b, (L, n) in enumerate(zip(lengths, q_lengths)):
        assert (out[b, :, n:] == 3).all() and (lse[b, :, n:] == 3).all()
        if n == 0:
            continue
        K, V = dense(s["k"], s["ks"], s["table"][b], L), dense(s["v"], s["vs"], s["table"][b], L)
        j, t = torch.arange(L, device=DEV), torch.arange(n, device=DEV)
        seen = j <= (L - n + t if causal else torch.full_like(t, L - 1))[:, None]
        for h in range(Hkv):
            G = Hq // Hkv
            x = q[b, h * G:(h + 1) * G, :n].double()
            y = (x @ K[h].T) * sc if L else torch.zeros(G, n, 0, dtype=torch.float64, device=DEV)
            y = y.masked_fill(~seen, -math.inf)
            w = torch.logsumexp(y, 2) if L else torch.full((G, n), -math.inf, device=DEV).double()
            p = torch.exp(y - w[..., None]).nan_to_num(0.0)
            o, A = p @ V[h], p @ V[h].abs()
            S = (x.abs() @ K[h].abs().T * sc).masked_fill(~seen, 0.0)
            S = S.amax(2) if L else torch.zeros_like(w)
            Y = y.abs().masked_fill(~seen, 0.0)
            Y = Y.amax(2) if L else torch.zeros_like(w)
            tol, ltol = R.bounds(o, w, A, S, Y, d, L, q.dtype, low_p)
            got, glse = out[b, h * G:(h + 1) * G, :n].double(), lse[b, h * G:(h + 1) * G, :n].double()
            assert torch.isfinite(got).all()
            err = (got - o).abs()
            assert bool((err <= tol).all()), (b, h, float((err / tol).max()))
            fin = torch.isfinite(w)
            assert torch.equal(fin, torch.isfinite(glse)) and (glse[~fin] == -math.inf).all()
            lerr = (glse - w).abs()[fin]
            assert bool((lerr <= ltol[fin]).all()), (b, h, float((lerr / ltol[fin]).max()))
    return out, lse


# rows per KV head (G, T) on both sides of each border
@pytest.mark.parametrize("pt", [BF16, E4M3])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G,T", [(1, 1), (7, 1), (8, 1), (1, 8), (3, 2), (9, 1), (3, 3), (16, 1), (1, 16),
                                 (17, 1), (1, 17), (5, 25), (4, 32), (1, 128), (43, 3), (1, 129),
                                 (4, 64), (257, 1), (1, 257), (7, 40)])
def test_rows_of_every_kernel(pt, d, G, T):
    lengths = [max(T, 1) + x for x in (0, 1, 126, 700, 2113)]
    n = [T, max(1, T - 1), T, (T + 1) // 2, T]
    s = make(lengths, 2 * G, 2, T, d, 16, BF16, pt, G * 1000 + T)
    check(s, lengths, n)
    check(s, lengths, n, causal=False)


@pytest.mark.parametrize("pt", [BF16, E4M3])
@pytest.mark.parametrize("page", [1, 7, 24, 129, 1024])
@pytest.mark.parametrize("T", [1, 20, 200])
def test_pages_of_any_size(pt, page, T):
    lengths = [1500, 200, 1024]
    s = make(lengths, 4, 2, T, 128, page, BF16, pt, page + T)
    check(s, lengths, [T, T, max(1, T - 3)])


@pytest.mark.parametrize("pt,d", [(BF16, 128), (E4M3, 128), (E4M3, 64)])
@pytest.mark.parametrize("T", [1, 3, 40])
def test_more_sequences_than_threads(pt, d, T):
    B = 700
    lengths = [(i * 37) % 90 for i in range(B)]
    n = [(i * 5) % (T + 1) for i in range(B)]
    s = make(lengths, 8, 2, T, d, 16, BF16, pt, T)
    check(s, lengths, n)


@pytest.mark.parametrize("pt", [BF16, E4M3])
@pytest.mark.parametrize("G,T", [(1, 20), (4, 100), (1, 300)])
def test_more_tokens_than_slots(pt, G, T):
    lengths = [T // 3, 0, T, 1]
    s = make(lengths, 2 * G, 2, T, 128, 16, BF16, pt, T)
    check(s, lengths, [T, T, T, T])
    check(s, lengths, [T, T, T, T], causal=False)


@pytest.mark.parametrize("G,T", [(4, 1), (4, 4), (4, 30), (4, 80)])
@pytest.mark.parametrize("k_bytes,q_scale", [((118, 123), 1.0), ((133, 137), 2.0 ** -14),
                                             ((200, 204), 2.0 ** -80), ((20, 24), 2.0 ** 98)])
@pytest.mark.parametrize("v_bytes", [(119, 124), (133, 137), (100, 160), (196, 200), (12, 30)])
def test_scales_of_the_whole_range(G, T, k_bytes, q_scale, v_bytes):
    # Where v's scales are small, so is everything: A and the tolerance scale with them
    lengths = [300, 171]
    s = make(lengths, 2 * G, 2, T, 128, 16, BF16, E4M3, T, k_bytes, v_bytes, q_scale)
    check(s, lengths, [T, max(1, T - 2)])


@pytest.mark.parametrize("pt", [BF16, E4M3])
@pytest.mark.parametrize("G,T", [(2, 4), (2, 8), (4, 20), (4, 70)])
@pytest.mark.parametrize("d", [64, 128])
def test_what_a_row_does_not_see_and_what_it_does(pt, G, T, d):
    # NaN in the K of the tokens a row does not see, infinities and NaN in their V: nothing
    # of them; in the V of one that some rows see: in those rows' value, and nowhere else
    L, page = 333, 16
    s = make([L], 2 * G, 2, T, d, page, BF16, pt, T)
    base, lbase = check(s, [L], [T])
    at = L - 2                                  # seen by the last two tokens
    p, o = int(s["table"][0, at // page]), at % page
    if pt == E4M3:
        s["vs"][p, :, o] = 255
    else:
        s["v"][p, :, o, 3] = math.inf
        s["v"][p, :, o, 5] = math.nan
    got, lse = torch.zeros_like(base), torch.zeros_like(lbase)
    dk.dropkv_cache_attention(s["q"], s["k"], s["v"], s["table"], i32([L]), k_scale=s["ks"],
                              v_scale=s["vs"], out=got, lse=lse)
    assert torch.equal(got[:, :, :T - 2], base[:, :, :T - 2]) and torch.equal(lse, lbase)
    tail = got[:, :, T - 2:].float()
    if pt == E4M3:
        assert torch.isnan(tail).all()
    else:
        assert (tail[..., 3] == math.inf).all() and torch.isnan(tail[..., 5]).all()
        rest = [i for i in range(d) if i not in (3, 5)]
        want = base[:, :, T - 2:].float()
        # the same products and sums but for the scalar order of one tile: fp32 sums of at most L
        # terms, and the rounding to bf16 on top
        assert ((tail[..., rest] - want[..., rest]).abs() <= 2.0 ** -7 * want[..., rest].abs() + 2e-3).all()
    # and a key that only the last token sees
    at = L - 1
    p, o = int(s["table"][0, at // page]), at % page
    if pt == E4M3:
        s["ks"][p, :, o] = 255
    else:
        s["k"][p, :, o] = math.nan
    dk.dropkv_cache_attention(s["q"], s["k"], s["v"], s["table"], i32([L]), k_scale=s["ks"],
                              v_scale=s["vs"], out=got, lse=lse)
    assert torch.equal(got[:, :, :T - 2], base[:, :, :T - 2])
    assert torch.equal(lse[:, :, :T - 1], lbase[:, :, :T - 1])
    assert torch.isnan(got[:, :, T - 1].float()).all() and torch.isnan(lse[:, :, T - 1]).all()


@pytest.mark.parametrize("qt,pt", [(F32, F32), (F32, E4M3), (F32, BF16), (BF16, F32)])
@pytest.mark.parametrize("d", [8, 33, 64, 80, 128, 200, 256])
@pytest.mark.parametrize("G,T", [(1, 128), (1, 129), (4, 50), (3, 1)])
def test_cuda_core_rows(qt, pt, d, G, T):
    lengths = [max(T, 1) + x for x in (0, 31, 500)]
    s = make(lengths, 2 * G, 2, T, d, 24, qt, pt, d + T)
    n = [T, T, max(1, T - 7)]
    check(s, lengths, n, path="simt")
    check(s, lengths, n, causal=False, path="simt")


@pytest.mark.parametrize("pt", [F32, E4M3])
def test_cuda_core_rows_ignore_what_they_do_not_see(pt):
    L, T, page, d = 200, 70, 16, 40
    s = make([L], 4, 2, T, d, page, F32, pt, 1)
    base, _ = check(s, [L], [T], path="simt")
    p, o = int(s["table"][0, (L - 1) // page]), (L - 1) % page
    for x in "kv":
        if pt == E4M3:
            s[x + "s"][p, :, o] = 255
        else:
            s[x][p, :, o] = math.nan
    got = dk.dropkv_cache_attention(s["q"], s["k"], s["v"], s["table"], i32([L]), k_scale=s["ks"],
                                    v_scale=s["vs"], path="simt")
    assert torch.equal(got[:, :, :T - 1], base[:, :, :T - 1]) and torch.isnan(got[:, :, T - 1]).all()


@pytest.mark.parametrize("pt", [BF16, E4M3])
def test_a_long_cache_split_over_all_ctas(pt):
    # every unit cut into many pieces, and the same bits from call to call
    for G, T, L in ((4, 1, 40000), (4, 4, 30000), (1, 100, 20000), (2, 300, 9000)):
        s = make([L], G, 1, T, 128, 64, BF16, pt, L)
        a = check(s, [L], [T])
        b = check(s, [L], [T])
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("T", [1, 3, 24, 90])
def test_two_graphs_with_a_workspace_each(T):
    lengths = [700, 93]
    a = make(lengths, 8, 2, T, 128, 16, BF16, BF16, 1)
    b = make(lengths, 8, 2, T, 128, 16, BF16, E4M3, 2)
    graphs, outs, want = [], [], []
    lens = i32(lengths)
    for s in (a, b):
        want.append(dk.dropkv_cache_attention(s["q"], s["k"], s["v"], s["table"], lens,
                                              k_scale=s["ks"], v_scale=s["vs"]))
        out, ws = torch.zeros_like(s["q"]), torch.empty(96 << 20, dtype=torch.uint8, device=DEV)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            dk.dropkv_cache_attention(s["q"], s["k"], s["v"], s["table"], lens, k_scale=s["ks"],
                                      v_scale=s["vs"], out=out, workspace=ws)
        graphs.append((g, ws))
        outs.append(out)
    side = torch.cuda.Stream()
    for _ in range(3):
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        graphs[0][0].replay()
        with torch.cuda.stream(side):
            graphs[1][0].replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1])


def test_workspaces_of_the_wrong_kind_are_refused():
    s = make([30], 4, 2, 1, 128, 16, BF16, BF16, 1)
    for ws in (torch.empty(64 << 20, dtype=torch.uint8), [1, 2],
               torch.empty(64 << 20, 2, dtype=torch.uint8, device=DEV)[:, 0]):
        with pytest.raises(TypeError):
            dk.dropkv_cache_attention(s["q"], s["k"], s["v"], s["table"], i32([30]), workspace=ws)


@pytest.mark.parametrize("src", [BF16, F32])
def test_written_bits_over_all_magnitudes(src):
    # rows whose values span forty binades around a random power of two
    g = torch.Generator().manual_seed(3)
    n, d = 512, 128
    e = torch.randint(-120, 100, (1, 1, n, 1), generator=g).float()
    x = torch.randn(1, 1, n, d, generator=g) * torch.exp2(e - torch.randint(0, 40, (1, 1, n, d), generator=g))
    x = x.to(src)
    want, byte = R.quantise(x.double())
    kp = torch.zeros(8, 1, 64, d).to(E4M3).to(DEV)
    vp, ks, vs = kp.clone(), *(torch.zeros(8, 1, 64, dtype=torch.uint8, device=DEV) for _ in range(2))
    table = torch.arange(8, dtype=torch.int32, device=DEV)[None]
    dk.dropkv_cache_write(x.to(DEV), -x.to(DEV), kp, vp, table, k_scale=ks, v_scale=vs, sync=True)
    assert torch.equal(ks.cpu().view(1, 1, n), byte) and torch.equal(vs, ks)
    assert torch.equal(kp.cpu().double().view(1, 1, n, d), want)
    assert torch.equal(vp.cpu().double().view(1, 1, n, d), -want)


@pytest.mark.parametrize("T", [1, 3, 24, 90])
def test_a_graph_that_reports_its_status(T):
    s = make([200, 130], 8, 2, T, 128, 16, BF16, BF16, T)
    lens = i32([200, 130])
    want = dk.dropkv_cache_attention(s["q"], s["k"], s["v"], s["table"], lens)
    out, status = torch.zeros_like(s["q"]), torch.full((1,), 9, dtype=torch.int32, device=DEV)
    ws = torch.empty(96 << 20, dtype=torch.uint8, device=DEV)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        dk.dropkv_cache_attention(s["q"], s["k"], s["v"], s["table"], lens, out=out, workspace=ws,
                                  status=status)
    for length, code in ((200, dk.OK), (10 ** 6, dk.ERR_ARG), (200, dk.OK)):
        lens[0] = length
        g.replay()
        torch.cuda.synchronize()
        assert int(status) == code
        if code == dk.OK:
            assert torch.equal(out, want)


@pytest.mark.parametrize("G,T", [(4, 1), (4, 4), (4, 20), (4, 60)])
def test_calls_back_to_back_see_what_came_between(G, T):
    # each call may be launched while its predecessor ends: lengths, queries and pages that a
    # kernel between two calls changes are the second call's
    s = make([900], G, 1, T, 128, 16, BF16, BF16, T)
    lens = i32([300])
    want = []
    for L in (300, 301, 700):
        lens.fill_(L)
        torch.cuda.synchronize()
        want.append(dk.dropkv_cache_attention(s["q"], s["k"], s["v"], s["table"], lens))
        torch.cuda.synchronize()
    for _ in range(20):
        lens.fill_(300)
        got = [dk.dropkv_cache_attention(s["q"], s["k"], s["v"], s["table"], lens)]
        lens.add_(1)
        got.append(dk.dropkv_cache_attention(s["q"], s["k"], s["v"], s["table"], lens))
        lens.add_(399)
        got.append(dk.dropkv_cache_attention(s["q"], s["k"], s["v"], s["table"], lens))
        assert all(torch.equal(a, b) for a, b in zip(got, want))
