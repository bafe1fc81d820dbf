"""Cache attention's precision on the GPU against fp64: the weights that meet V, and
sums over long ranges of slots."""

import math

import pytest
import torch

import cache_ref as R
import kv_cache_eviction_scores_b200 as dk
from cache_ref import BF16, E4M3, F32
from test_gpu_cache_tiles import dense, make

pytestmark = pytest.mark.gpu
DEV = "cuda"


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def line(L, Hkv, d, dtype, gen, byte=121):
    """One sequence's pages of 64 slots: (pages, scale, table, dense fp64 [Hkv, L, d])."""
    n = -(-L // 64)
    x = torch.randn(n, Hkv, 64, d, generator=gen, device=DEV)
    x = (x * 48).to(E4M3) if dtype == E4M3 else x.to(dtype)
    scale = torch.full((n, Hkv, 64), byte, dtype=torch.uint8, device=DEV) if dtype == E4M3 else None
    dense = x.double() * (1.0 if scale is None else 2.0 ** (byte - 127))
    return x, scale, dense.permute(1, 0, 2, 3).reshape(Hkv, n * 64, d)[:, :L]


# rows per KV head of each of the tensor path's kernels
@pytest.mark.parametrize("pt", [BF16, E4M3])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G,T", [(4, 1), (4, 4), (4, 20), (4, 100)])
def test_the_weights_that_meet_v_keep_fifteen_bits(pt, d, G, T):
    # Two bf16 parts of a weight leave 2^-15 of it (the lower part, at most 2^-7 of the weight, is
    # rounded by 2^-8 of itself at most), and the factor 1 + 2^-20 that keeps the lower part above
    # zero adds its own.  Everything else is R.bounds' fp32 arithmetic and the output's rounding.
    # One bf16 part would be off by 2^-8 of a weight, which shows wherever V's values cancel.
    g = torch.Generator(device=DEV).manual_seed(G * T + d)
    Hkv, L = 2, T + 100
    k, ks, K = line(L, Hkv, d, pt, g)
    v, vs, V = line(L, Hkv, d, pt, g)
    q = torch.randn(1, G * Hkv, T, d, generator=g, device=DEV).to(BF16)
    table = torch.arange(k.shape[0], dtype=torch.int32, device=DEV)[None]
    out, lse = dk.dropkv_cache_attention(q, k, v, table, i32([L]), k_scale=ks, v_scale=vs,
                                         return_lse=True, sync=True)
    x = q[0].double().view(Hkv, G, T, d)
    y = torch.einsum("hgtd,hjd->hgtj", x, K) / math.sqrt(d)
    seen = torch.arange(L, device=DEV) <= (L - T + torch.arange(T, device=DEV))[:, None]
    p = y.masked_fill(~seen, -math.inf).softmax(-1)
    o, A = torch.einsum("hgtj,hjd->hgtd", p, V), torch.einsum("hgtj,hjd->hgtd", p, V.abs())
    S = (torch.einsum("hgtd,hjd->hgtj", x.abs(), K.abs()) / math.sqrt(d)).masked_fill(~seen, 0).amax(-1)
    Y = y.abs().masked_fill(~seen, 0).amax(-1)
    lw = torch.logsumexp(y.masked_fill(~seen, -math.inf), -1)
    tol, _ = R.bounds(o, lw, A, S, Y, d, L, BF16, False)
    tol = tol + A * (2.0 ** -15 + 2.0 ** -20)
    err = (out[0].double().view(Hkv, G, T, d) - o).abs()
    assert bool((err <= tol).all()), float((err / tol).max())


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G,T", [(4, 1), (4, 4), (4, 20), (4, 100)])
def test_infinities_that_a_row_sees_reach_it(d, G, T):
    # equal weights of a power of two: their lower parts would be 0, and 0 * inf is NaN
    g = torch.Generator(device=DEV).manual_seed(G * T + d)
    Hkv, L = 2, T + 300
    k, _, _ = line(L, Hkv, d, BF16, g)
    v, _, V = line(L, Hkv, d, BF16, g)
    k.zero_()
    v[0, :, 9, 3], v[1, :, 4, 5], v[0, :, 20, d - 1] = math.inf, -math.inf, math.nan
    q = torch.randn(1, G * Hkv, T, d, generator=g, device=DEV).to(BF16)
    table = torch.arange(k.shape[0], dtype=torch.int32, device=DEV)[None]
    out = dk.dropkv_cache_attention(q, k, v, table, i32([L]), sync=True)[0]
    assert (out[..., 3] == math.inf).all() and (out[..., 5] == -math.inf).all()
    assert torch.isnan(out[..., d - 1]).all()
    rest = [i for i in range(d) if i not in (3, 5, d - 1)]
    assert torch.isfinite(out[..., rest]).all()


@pytest.mark.parametrize("pt", [BF16, E4M3, F32])
@pytest.mark.parametrize("rows", [(1, 128), (1, 512)])
@pytest.mark.parametrize("c", [0.34375, 0.5625, 0.625])
def test_sums_over_a_long_range_that_no_split_shortens(pt, rows, c):
    # The first 128 slots' logits are c and set the reference; all others are 0, so that every
    # weight behind them is exp(-c) and the sums' roundings all go one way.  With units to fill
    # the CTAs, one CTA sums all slots of a row.  A tile's slots (128 on the tensor path, 32 on
    # CUDA cores) are summed by themselves, in at most 128 additions of 2^-24 each, and then added
    # to the total: n / 128 or n / 32 additions more.  The weights' own errors are ex2's 2^-22 and
    # the exponent's rounding, 2^-24 of c.
    G, T = rows
    d, Hkv = 64, 8
    L, B, tile = (65536, 12, 32) if pt == F32 else (131072, 20, 128)
    n = L // 64
    k = torch.zeros(n, Hkv, 64, d, device=DEV)
    k[:2, :, :, 0] = c
    k = k.to(pt)
    v = torch.full_like(k.float(), 3.0).to(pt)
    sc = torch.full((n, Hkv, 64), 127, dtype=torch.uint8, device=DEV) if pt == E4M3 else None
    # one set of pages for all sequences
    table = torch.arange(n, dtype=torch.int32, device=DEV)[None].repeat(B, 1)
    q = torch.zeros(B, Hkv * G, T, d, dtype=F32 if pt == F32 else BF16, device=DEV)
    q[..., 0] = 8.0                                  # times the default scale of 1 / 8
    out, lse = dk.dropkv_cache_attention(q, k, v, table, i32([L] * B), causal=False, k_scale=sc,
                                         v_scale=sc, return_lse=True, sync=True)
    rel = (128 + L / tile) * 2.0 ** -24 + 2.0 ** -21
    want = math.log(128 * math.exp(c) + L - 128)
    err = float((lse.double() - want).abs().max())
    assert err <= rel + want * 2.0 ** -22, err
    tol = 3.0 * (2 * rel + 2.0 ** -22 + (2.0 ** -8 if pt != F32 else 0.0))
    err = float((out.double() - 3.0).abs().max())
    assert err <= tol, err


@pytest.mark.parametrize("G,T", [(4, 1), (4, 4), (4, 30), (4, 80)])
@pytest.mark.parametrize("path", ["auto", "simt"])
def test_small_scales_of_v_keep_their_precision(G, T, path):
    # V's scales are 2^-115 to 2^-98, so outputs are some 2^-100.  Tensor path: a weight times such a
    # scale can lie among bf16's subnormals, whose step of 2^-133 its two parts resolve to 2^-134;
    # with V's own values (at most 448) over n slots, and a sum of weights of at least 1 (the
    # reference is some slot's logit): 448 n 2^-134.  CUDA cores: V times its scale is exact in fp32.
    # Nothing else depends on the scale.
    lengths, n = [300, 171], [T, max(1, T - 2)]
    s = make(lengths, 2 * G, 2, T, 128, 16, BF16, E4M3, T, (118, 123), (12, 30))
    out = dk.dropkv_cache_attention(s["q"], s["k"], s["v"], s["table"], i32(lengths),
                                    q_lengths=i32(n), k_scale=s["ks"], v_scale=s["vs"], path=path,
                                    sync=True)
    for b, (L, c) in enumerate(zip(lengths, n)):
        K, V = (dense(s[x], s[x + "s"], s["table"][b], L) for x in "kv")
        x = s["q"][b, :, :c].double().view(2, G, c, 128)
        y = torch.einsum("hgtd,hjd->hgtj", x, K) / math.sqrt(128)
        seen = torch.arange(L, device=DEV) <= (L - c + torch.arange(c, device=DEV))[:, None]
        w = torch.logsumexp(y.masked_fill(~seen, -math.inf), -1)
        p = torch.exp(y.masked_fill(~seen, -math.inf) - w[..., None])
        o, A = torch.einsum("hgtj,hjd->hgtd", p, V), torch.einsum("hgtj,hjd->hgtd", p, V.abs())
        S = torch.einsum("hgtd,hjd->hgtj", x.abs(), K.abs()) / math.sqrt(128)
        S, Y = S.masked_fill(~seen, 0).amax(-1), y.abs().masked_fill(~seen, 0).amax(-1)
        tol = R.bounds(o, w, A, S, Y, 128, L, BF16, False)[0] - 1e-30
        if path == "auto":
            tol = tol + A * (2.0 ** -15 + 2.0 ** -20) + 448 * L * 2.0 ** -134
        err = (out[b, :, :c].double().view(2, G, c, 128) - o).abs()
        assert bool((err <= tol).all()), float((err / tol).max())


@pytest.mark.parametrize("qt,T", [(BF16, 1), (BF16, 9), (BF16, 20), (BF16, 129), (F32, 1), (F32, 129)])
def test_the_logarithm_of_exact_sums(qt, T):
    # logits of 0: a row over L slots sums L weights of 1 exactly, so its lse is logf(L), off by one
    # unit in the last place at most
    most, B = 2048, 2048 if T == 1 else 300
    L = torch.arange(1, B + 1) if B == most else torch.unique((most ** (torch.arange(B) / (B - 1.0))).round().int())
    B = len(L)
    k = torch.zeros(most // 64, 1, 64, 64, dtype=qt, device=DEV)
    table = torch.arange(most // 64, dtype=torch.int32, device=DEV).repeat(B, 1)
    q = torch.zeros(B, 1, T, 64, dtype=qt, device=DEV)
    _, lse = dk.dropkv_cache_attention(q, k, k, table, i32(L.tolist()), causal=False, return_lse=True,
                                       sync=True)
    want = L.double().log().to(DEV)[:, None, None]
    err = (lse.double() - want).abs()
    assert bool((err <= torch.exp2(torch.floor(torch.log2(want.clamp(min=1e-30))) - 23)).all()), float(err.max())


@pytest.mark.parametrize("qt,T", [(BF16, 1), (BF16, 64), (F32, 1), (F32, 129)])
def test_lse_is_as_close_as_the_plain_form(qt, T):
    # The plain form in fp32 (maximum, exponentials, sum, log) rounds a logit's sum and scaling, the
    # logarithm and the last sum; this one's roundings are as many.  The two kinds of errors are
    # independent and differ in size from draw to draw, so the norm over 512 sequences is compared
    # with room for a fifth.
    g = torch.Generator(device=DEV).manual_seed(1)
    B, n = 512, 25
    L = (torch.arange(B) * 3 + 1).int().to(DEV)
    k = torch.randn(n, 1, 64, 64, generator=g, device=DEV).to(qt)
    table = torch.arange(n, dtype=torch.int32, device=DEV).repeat(B, 1)
    q = torch.randn(B, 1, T, 64, generator=g, device=DEV).to(qt)
    _, lse = dk.dropkv_cache_attention(q, k, k, table, L, causal=False, return_lse=True, sync=True)
    K = k.reshape(-1, 64)
    hidden = torch.arange(len(K), device=DEV)[None, None] >= L[:, None, None]
    exact = (q[:, 0].double() @ K.double().T / 8).masked_fill(hidden, -math.inf).logsumexp(-1)
    y = (q[:, 0].float() @ K.float().T * 0.125).masked_fill(hidden, -math.inf)
    top = y.amax(-1, keepdim=True)
    plain = top[..., 0] + torch.log(torch.exp(y - top).sum(-1))
    ours, theirs = ((x.double() - exact).norm() for x in (lse[:, 0], plain))
    assert float(ours) <= 1.2 * float(theirs), (float(ours), float(theirs))


@pytest.mark.parametrize("pt", [BF16, E4M3])
@pytest.mark.parametrize("G,T", [(4, 1), (4, 4), (4, 16), (4, 512)])
def test_outputs_over_a_long_range_that_no_split_shortens(pt, G, T):
    # V of one sign and weights that are no powers of two, so that nothing is exact and every sum
    # that a matrix product cuts off errs downwards.  How much an instruction cuts off is documented
    # nowhere: one unit of the total's last place, 2^-23, where it is cut once, and 2^-22 is allowed.
    # One instruction takes 16 slots and one of a weight's two parts.  Up to 16 rows, eight warps
    # share the slots: n / 64 instructions each.  Above, O leaves the tensor core every 128 tiles of
    # 128 slots: 2048 instructions, and n / 16384 sums of 2^-24.  Besides: a weight's two parts (2^-15
    # and 2^-20), ex2 and the exponent's rounding (2^-21) in the weight and in l, whose sums are of
    # 128 + n / 128 terms; the output's own rounding, 2^-8.
    d, Hkv, L = 128, 8, 131072
    B = 37 if T < 512 else 3                        # with units to fill the CTAs
    n = L // 128
    g = torch.Generator(device=DEV).manual_seed(T)
    off = 1 + torch.arange(Hkv * d, device=DEV).view(1, Hkv, 1, d) / (Hkv * d)
    v = off + 0.3 * torch.rand(n, Hkv, 128, d, generator=g, device=DEV)
    k = torch.zeros(n, Hkv, 128, d, device=DEV)
    k[1:, :, :, 0] = 1                              # the first 128 slots set the reference
    k, v = k.to(pt), (v * 64).to(pt)
    sc = torch.full((n, Hkv, 128), 127, dtype=torch.uint8, device=DEV) if pt == E4M3 else None
    table = torch.arange(n, dtype=torch.int32, device=DEV).repeat(B, 1)
    q = torch.zeros(B, Hkv * G, T, d, device=DEV, dtype=BF16)
    q[..., 0] = 9.625
    w = torch.full((L,), math.exp(9.625 / math.sqrt(d)), dtype=torch.float64, device=DEV)
    w[:128] = 1
    want = torch.einsum("nhsd,ns->hd", v.double(), w.view(n, 128)) / w.sum()
    out = dk.dropkv_cache_attention(q, k, v, table, i32([L] * B), causal=False, k_scale=sc, v_scale=sc,
                                    sync=True)
    chain = L / 64 if G * T <= 16 else 2048 + L / 16384
    rel = chain * 2.0 ** -22 + 2.0 ** -15 + 2.0 ** -20 + 2 * 2.0 ** -21 + (128 + L / 128) * 2.0 ** -24
    err = (out.double().view(B, Hkv, G * T, d) / want[None, :, None] - 1).abs().max()
    assert float(err) <= 2.0 ** -8 + rel, (float(err), rel)


@pytest.mark.parametrize("pt", [BF16, E4M3])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G,T", [(4, 30), (4, 80), (3, 43)])
def test_references_that_move_between_parts_of_a_long_sum(pt, d, G, T):
    # logits that grow along the slots, ragged and causal, whole units and cut ones (with units to
    # fill the CTAs, many of them have over 256 tiles to themselves); infinities and a NaN early on
    B, Hkv, page = 21, 8, 64
    L = [40000 - 1042 * b for b in range(B)]
    n = -(-L[0] // page)
    g = torch.Generator(device=DEV).manual_seed(T + d)
    k, v = (torch.randn(n, Hkv, page, d, generator=g, device=DEV) for _ in range(2))
    k *= (0.5 + 1.5 * torch.arange(n, device=DEV) / n)[:, None, None, None]
    sc = None
    if pt == E4M3:
        k, v = k * 32, v * 32
        sc = torch.full((n, Hkv, page), 122, dtype=torch.uint8, device=DEV)
    k, v = k.to(pt), v.to(pt)
    odd = () if pt == E4M3 else (3, 5, 9)
    if odd:
        v[10, :, 7, 3], v[90, :, 7, 5], v[2, :, 0, 9] = math.inf, -math.inf, math.nan
    table = torch.arange(n, dtype=torch.int32, device=DEV).repeat(B, 1)
    q = torch.randn(B, Hkv * G, T, d, generator=g, device=DEV).to(BF16)
    out, lse = dk.dropkv_cache_attention(q, k, v, table, i32(L), k_scale=sc, v_scale=sc,
                                         return_lse=True, sync=True)
    if odd:
        assert (out[..., 3] == math.inf).all() and (out[..., 5] == -math.inf).all()
        assert torch.isnan(out[..., 9]).all()
    rest = [i for i in range(d) if i not in odd]
    K, V = (x.double().permute(1, 0, 2, 3).reshape(Hkv, n * page, d) * (1 if sc is None else 2.0 ** -5)
            for x in (k, v))
    V = V[..., rest]
    for b in (0, 1, 10, 20):
        x, c = q[b].double().view(Hkv, G * T, d), L[b]
        seen = (torch.arange(c, device=DEV) <= (c - T + torch.arange(T, device=DEV))[:, None]).repeat(G, 1)
        for h in range(Hkv):
            y = (x[h] @ K[h, :c].T / math.sqrt(d)).masked_fill(~seen, -math.inf)
            w = torch.logsumexp(y, -1)
            p = torch.exp(y - w[:, None])
            o, A = p @ V[h, :c], p @ V[h, :c].abs()
            S = (x[h].abs() @ K[h, :c].abs().T / math.sqrt(d)).masked_fill(~seen, 0).amax(-1)
            Y = y.masked_fill(~seen, 0).abs().amax(-1)
            tol, ltol = R.bounds(o, w, A, S, Y, d, c, BF16, False)
            tol = tol + A * (2.0 ** -15 + 2.0 ** -20)
            err = (out[b].view(Hkv, G * T, d)[h][:, rest].double() - o).abs()
            assert bool((err <= tol).all()), float((err / tol).max())
            err = (lse[b].view(Hkv, G * T)[h].double() - w).abs()
            assert bool((err <= ltol).all()), float((err / ltol).max())
