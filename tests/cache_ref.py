"""Plain fp64 forms of the paged-cache operators, for the tests, and the bounds
their kernels' results are held to."""

import math

import torch

BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


def e4m3_grid():
    """The non-negative finite e4m3 values, from the format's definition."""
    vals = [m * 2.0 ** -9 for m in range(8)]
    for e in range(1, 16):
        vals += [(8 + m) * 2.0 ** (e - 10) for m in range(8) if not (e == 15 and m == 7)]
    return torch.tensor(vals, dtype=torch.float64)


def quantise(x):
    """(values x 2^-e rounded to the e4m3 grid, ties to even, as fp64; scale bytes) of fp64
    rows [..., d]: by search in the grid.  Rows with an inf or a NaN: (NaN, 255)."""
    grid = e4m3_grid()
    top = x.abs().amax(dim=-1)
    bad = ~torch.isfinite(x).all(dim=-1)
    e = torch.full(top.shape, -127, dtype=torch.float64)
    for k in range(-127, 121):  # the least e that takes the row into [-448, 448]
        e = torch.where(top > 448.0 * 2.0 ** k, torch.full_like(e, k + 1), e)
    y = torch.where(bad[..., None], torch.zeros_like(x), x * torch.exp2(-e)[..., None])
    a = y.abs()
    hi = torch.searchsorted(grid, a.contiguous()).clamp(max=len(grid) - 1)
    lo = (hi - 1).clamp(min=0)
    d_hi, d_lo = grid[hi] - a, a - grid[lo]
    up = (d_hi < d_lo) | ((d_hi == d_lo) & (hi % 2 == 0))  # grid index parity = mantissa parity
    v = torch.copysign(torch.where(up, grid[hi], grid[lo]), y)
    v = torch.where(bad[..., None], torch.full_like(v, math.nan), v)
    return v, torch.where(bad, torch.full_like(e, 255.0), e + 127).to(torch.uint8)


def table_for(slots, page, gen, spare=2, width=None):
    """A shuffled page table for slots[b] slots of each sequence: (table, pages in the pools).
    Entries no slot needs are -7."""
    per = [-(-n // page) for n in slots]
    total = sum(per) + spare
    order = torch.randperm(total, generator=gen)
    t = torch.full((len(per), max(max(per), 1) if width is None else width), -7, dtype=torch.int32)
    at = 0
    for b, n in enumerate(per):
        t[b, :n] = order[at:at + n].to(torch.int32)
        at += n
    return t, total


def held(pages, scale, table, b, h, count):
    """The first `count` slots of (b, h) as fp64 rows."""
    page = pages.shape[2]
    rows = []
    for j in range(0, count, page):
        p = int(table[b, j // page])
        x = pages[p, h].double()
        if scale is not None:
            x = x * torch.exp2(scale[p, h].double() - 127)[:, None]
        rows.append(x)
    return torch.cat(rows)[:count] if rows else torch.zeros(0, pages.shape[3], dtype=torch.float64)


def attend(q, k_pages, v_pages, table, lengths, q_lengths, scale, causal, k_scale=None,
           v_scale=None):
    """fp64 (out, lse, A, S, Y) with A = sum_j p_j |v_j|, and per row S = max_j sum_i |q_i k_ij|
    times the scale and Y = max_j |logit|; rows behind the chunk are NaN."""
    B, Hq, T, d = q.shape
    Hkv = k_pages.shape[1]
    out = torch.full((B, Hq, T, d), math.nan, dtype=torch.float64)
    A, lse = out.clone(), torch.full((B, Hq, T), math.nan, dtype=torch.float64)
    S, Y = lse.clone(), lse.clone()
    for b in range(B):
        L, n = int(lengths[b]), int(q_lengths[b])
        for h in range(Hkv):
            K = held(k_pages, k_scale, table, b, h, L)
            V = held(v_pages, v_scale, table, b, h, L)
            for g in range(h * (Hq // Hkv), (h + 1) * (Hq // Hkv)):
                for t in range(n):
                    c = max(0, L - n + t + 1) if causal else L
                    if c == 0:
                        out[b, g, t], A[b, g, t], lse[b, g, t], S[b, g, t], Y[b, g, t] = \
                            0, 0, -math.inf, 0, 0
                        continue
                    x = q[b, g, t].double()
                    y = (K[:c] @ x) * scale
                    lse[b, g, t] = torch.logsumexp(y, 0)
                    p = torch.exp(y - lse[b, g, t])
                    out[b, g, t], A[b, g, t] = p @ V[:c], p @ V[:c].abs()
                    S[b, g, t] = (K[:c].abs() @ x.abs()).max() * scale
                    Y[b, g, t] = y.abs().max()
    return out, lse, A, S, Y


def bounds(out, lse, A, S, Y, d, n, dtype, low_p):
    """Tolerances of (out, lse).  A logit is off by at most d 2^-24 S (an fp32 sum of d products)
    plus its scaling and the exponent's rounding, 8 2^-24 Y; ex2 by 2^-22 relative, and log the
    same; sums of n terms by n 2^-24.  A weight's error enters once through the numerator and once
    through the sum.  low_p: the weights that meet V are rounded to bf16 (at most 2^-8 each).  The
    output's own rounding: 2^-8 for bf16, 2^-24 for fp32."""
    e = d * 2.0 ** -24 * S + 8 * 2.0 ** -24 * Y
    rel = 2 * (e + 2.0 ** -21 + (n + 64) * 2.0 ** -24)
    step = 2.0 ** -8 if dtype == BF16 else 2.0 ** -24
    tol = A * ((rel + (2.0 ** -8 if low_p else 0.0))[..., None]) + out.abs() * step + 1e-30
    return tol, e + 2.0 ** -20 + (n + 64) * 2.0 ** -24 + lse.abs().nan_to_num(0, 0, 0) * 2.0 ** -22
