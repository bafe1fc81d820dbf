"""The paged-cache operators: what is measured, in plain form and through the library.

Three operators work on a paged K/V cache that holds what an eviction kept and
the tokens that came after it:

* write: rows of dense K/V (all of them, or the kept positions of a list) go to
  consecutive slots of each sequence, as they are or quantised to e4m3 with one
  power-of-two scale per row;
* read: slots come back as dense K/V rows;
* attend: a chunk of T new tokens (T = 1 is decoding) attends over its
  sequence's slots, causally, with grouped heads; the output and the log of
  each row's softmax sum.

Where ``own`` is false, ``run`` computes them with elementary torch operations
in fp32; where it is true, it calls the package.
"""

import math

import torch

own = False

FLOAT = {"bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}
BYTES = {"bf16": 2, "f32": 4, "e4m3": 1}
GOLDEN = 0.6180339887498949


def listed():
    # heads and lengths: the benchmark's 32/8 x 128 and 28/4 x 128 shapes and
    # its 4K to 128K caches with budgets of 5 to 20 %; the other sizes are generic
    return [
        # one decoded token for each of 16 sequences: the smallest write
        dict(name="write_token_e4m3", op="write", B=16, Hkv=8, d=128, src="bf16", fmt="e4m3",
             page=64, n=1, count=1, count_min=1, start=8191, start_min=1000, rows=False),
        # the 5 % of a 128K prompt that an eviction keeps, gathered into pages
        dict(name="write_kept_bf16", op="write", B=1, Hkv=8, d=128, src="bf16", fmt="bf16",
             page=64, n=131072, count=6553, count_min=6553, start=0, start_min=0, rows=True),
        # four long prompts of unequal length stored whole in 8 bits: the largest write
        dict(name="write_fill_e4m3", op="write", B=4, Hkv=4, d=128, src="bf16", fmt="e4m3",
             page=128, n=65536, count=65536, count_min=49152, start=0, start_min=0, rows=False),
        # a 32K cache read back whole, to be scored again
        dict(name="read_all_e4m3", op="read", B=1, Hkv=8, d=128, dst="bf16", fmt="e4m3",
             page=64, slots=32768, count=32768, count_min=32768, start=0, start_min=0, rows=False),
        # listed slots of an fp32 cache, odd head size and page
        dict(name="read_rows_f32", op="read", B=3, Hkv=5, d=80, dst="f32", fmt="f32",
             page=24, slots=4099, count=1001, count_min=700, start=0, start_min=0, rows=True),
        # one token after the eviction of a 128K prompt: the smallest attention
        dict(name="attend_kept_token", op="attend", B=1, Hq=32, Hkv=8, d=128, q="bf16", fmt="bf16",
             page=64, T=1, T_min=1, L=6554, L_min=6554, causal=True),
        # a serving batch of 64 sequences, one token each, 8-bit cache
        dict(name="attend_batch_e4m3", op="attend", B=64, Hq=28, Hkv=4, d=128, q="bf16", fmt="e4m3",
             page=64, T=1, T_min=1, L=16384, L_min=2048, causal=True),
        # four whole 128K caches, one token each: the largest read of a cache
        dict(name="attend_long_bf16", op="attend", B=4, Hq=32, Hkv=8, d=128, q="bf16", fmt="bf16",
             page=128, T=1, T_min=1, L=131072, L_min=131072, causal=True),
        # sixteen drafted tokens checked at once, ragged 8-bit caches, small pages
        dict(name="attend_draft_e4m3", op="attend", B=8, Hq=32, Hkv=8, d=128, q="bf16", fmt="e4m3",
             page=16, T=16, T_min=9, L=32768, L_min=5000, causal=True),
        # a chunk of a long prompt over what came before it
        dict(name="attend_chunk_bf16", op="attend", B=1, Hq=32, Hkv=8, d=128, q="bf16", fmt="bf16",
             page=64, T=512, T_min=512, L=32768, L_min=32768, causal=True),
        # large chunks of unequal length in one batch: the most arithmetic
        dict(name="attend_prefill_e4m3", op="attend", B=4, Hq=28, Hkv=4, d=128, q="bf16",
             fmt="e4m3", page=128, T=2048, T_min=1001, L=8192, L_min=3001, causal=True),
        # fp32, odd head size, page and lengths
        dict(name="attend_odd_f32", op="attend", B=2, Hq=6, Hkv=2, d=80, q="f32", fmt="f32",
             page=24, T=37, T_min=5, L=1501, L_min=333, causal=True),
    ]


def _between(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["write", "read", "attend", "attend"])
    B = _between(rng, 1, 64)
    page = rng.choice([16, 24, 32, 64, 128])
    Hq, Hkv = rng.choice([(32, 8), (28, 4), (4, 2), (8, 8), (6, 2), (5, 5), (16, 1)])
    if op != "attend":
        wide = rng.choice(["bf16", "bf16", "f32"])
        fmt = rng.choice([wide, "e4m3"])
        d = rng.choice([128, 128, 64, 80, 8, 256, 33])
        # values moved: at most those of the largest listed write
        most = (100_000_000 if wide == "bf16" else 50_000_000) // (B * Hkv * d)
        n = _between(rng, 1, max(1, min(131072, most)))
        rows = rng.random() < 0.5
        count = _between(rng, 1, n) if rows else n
        case = dict(op=op, B=B, Hkv=Hkv, d=d, fmt=fmt, page=page, count=count,
                    count_min=rng.randint((count + 1) // 2, count), rows=rows)
        if op == "write":
            start = rng.randint(0, 5000) if rng.random() < 0.5 and B * Hkv * d < 200_000 else 0
            return dict(case, src=wide, n=n, start=start, start_min=start // 2)
        start = 0 if rows else rng.randint(0, n - count)
        return dict(case, dst=wide, slots=n, start=start, start_min=start // 2)
    causal = rng.random() < 0.9
    if rng.random() < 0.75:
        wide, d = "bf16", rng.choice([128, 128, 128, 64])
        elems, pairs = 250_000_000, 1.2e9 / (d / 64)
    else:
        wide, d = "f32", rng.choice([128, 64, 80, 8, 33])
        elems, pairs = 20_000_000, 3e7
    fmt = rng.choice([wide, "e4m3"])
    L = _between(rng, 1, max(1, min(131072, elems // (B * Hkv * d))))
    T = 1 if rng.random() < 0.4 else _between(rng, 1, int(max(1, min(2048, L, pairs / (B * Hq * L)))))
    return dict(op=op, B=B, Hq=Hq, Hkv=Hkv, d=d, q=wide, fmt=fmt, page=page, T=T,
                T_min=rng.randint((T + 1) // 2, T), L=L, L_min=rng.randint((L + 1) // 2, L),
                causal=causal)


def _ragged(B, lo, hi):
    """B whole numbers of [lo, hi], the first one hi, the others spread over it."""
    return [hi if i == 0 else lo + int((i * GOLDEN % 1.0) * (hi - lo + 1)) for i in range(B)]


def _pages(case, slots, gen):
    """Pages for `slots[b]` slots of every sequence, in a shuffled order."""
    per = [max(1, -(-n // case["page"])) for n in slots]
    total = sum(per)
    order = torch.randperm(total + 1, generator=gen, device="cuda").to(torch.int32)
    table = torch.zeros(len(per), max(per), dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(per):
        table[b, :n] = order[at:at + n]
        at += n
    return table, total + 1


def _values(shape, dtype, gen):
    """N(0, 1) values in a storage type."""
    return torch.randn(shape, generator=gen, device="cuda").to(FLOAT[dtype])


def _int32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    B, Hkv, d, page, fmt = case["B"], case["Hkv"], case["d"], case["page"], case["fmt"]
    s = dict(op=case["op"])
    if case["op"] == "write":
        counts = _ragged(B, case["count_min"], case["count"])
        starts = _ragged(B, case["start_min"], case["start"])
        s["table"], pages = _pages(case, [a + c for a, c in zip(starts, counts)], gen)
        shape = (pages, Hkv, page, d)
        s["k_pages"] = torch.zeros(shape, device="cuda").to(FLOAT[fmt])
        s["v_pages"] = s["k_pages"].clone()
        s["k"] = _values((B, Hkv, case["n"], d), case["src"], gen)
        s["v"] = _values((B, Hkv, case["n"], d), case["src"], gen)
        # a few large channels of K, as trained models have them
        s["k"][..., :: max(1, d // 4)] *= 8
        of = case["n"]
    else:
        if case["op"] == "read":
            counts, starts = _ragged(B, case["count_min"], case["count"]), \
                _ragged(B, case["start_min"], case["start"])
            slots, of = [case["slots"]] * B, case["slots"]
            s["n"], s["dst"] = case["count"], FLOAT[case["dst"]]
            for x in "kv":  # rows past a sequence's count stay as they are
                s[x + "_out"] = torch.full((B, Hkv, case["count"], d), 2.0 ** -9, dtype=s["dst"],
                                           device="cuda")
        else:
            slots = _ragged(B, case["L_min"], case["L"])
            counts = starts = None
        s["table"], pages = _pages(case, slots, gen)
        shape = (pages, Hkv, page, d)
        s["k_pages"] = _values(shape, "f32" if fmt == "f32" else "bf16", gen)
        s["v_pages"] = _values(shape, "f32" if fmt == "f32" else "bf16", gen)
        if fmt == "e4m3":  # values of up to a few hundred, scaled to N(0, 1) by the rows' scales
            for x in "kv":
                s[x + "_pages"] = (s[x + "_pages"] * 48).to(FLOAT[fmt])
    if fmt == "e4m3":
        lo, hi = (0, 1) if case["op"] == "write" else (120, 123)  # bytes: 2^(byte - 127)
        for x in "kv":
            s[x + "_scale"] = torch.randint(lo, hi, shape[:3], generator=gen, device="cuda",
                                            dtype=torch.uint8)
    else:
        s["k_scale"] = s["v_scale"] = None
    if case["op"] == "attend":
        T = case["T"]
        s["q"] = _values((B, case["Hq"], T, d), case["q"], gen)
        s["q_lengths"] = _int32(_ragged(B, case["T_min"], T))
        s["lengths"] = _int32(slots)
        s["causal"] = case["causal"]
        # rows past a sequence's chunk stay as they are
        s["out"] = torch.full_like(s["q"], 2.0 ** -9)
        s["lse"] = torch.full((B, case["Hq"], T), 0.5, device="cuda")
        return s
    s["start"], s["counts"] = _int32(starts), _int32(counts)
    s["rows"] = None
    if case["rows"]:  # ascending positions per head, as a selection lists them; -1 behind the last
        rank = torch.rand(B, Hkv, of, generator=gen, device="cuda").argsort(dim=2)
        rows = rank[..., : case["count"]].to(torch.int32)
        past = torch.arange(case["count"], device="cuda") >= s["counts"][:, None, None]
        rows = rows.masked_fill(past, of).sort(dim=2).values
        s["rows"] = rows.masked_fill(past, -1).contiguous()
    return s


# ---- plain forms -------------------------------------------------------------

def _factor(scale):
    """2^(byte - 127) in fp32."""
    bits = scale.to(torch.int32)
    return torch.where(bits > 0, bits << 23, torch.full_like(bits, 1 << 22)).view(torch.float32)


def _places(s, H):
    """For every (sequence, head, i): the dense row, page and offset in the page.  An i past
    the sequence's count repeats its last one."""
    B, P = s["table"].shape
    page = s["k_pages"].shape[2]
    n = s["rows"].shape[2] if s["rows"] is not None else int(s["n"] if "n" in s else s["k"].shape[2])
    i = torch.arange(n, device="cuda")[None, :]
    i = torch.minimum(i, s["counts"][:, None].long() - 1)          # [B, n]
    first = s["start"][:, None].long()
    if s["rows"] is not None:
        rows = s["rows"].long().gather(2, i[:, None, :].expand(B, H, n))
    else:
        rows = i[:, None, :].expand(B, H, n)
    return i, first, rows, page


def _plain_write(s):
    B, H, _, d = s["k"].shape
    i, first, rows, page = _places(s, H)
    slot = first + i
    at = s["table"].long().gather(1, slot // page)[:, None, :]     # [B, 1, n]
    off = (slot % page)[:, None, :]
    head = torch.arange(H, device="cuda")[None, :, None]
    seq = torch.arange(B, device="cuda")[:, None, None]
    for x in "kv":
        val = s[x][seq, head, rows].float()
        if s[x + "_scale"] is not None:
            big = val.abs().amax(dim=3)
            part, exp = torch.frexp(big)
            byte = (exp - 9 + (part > 0.875).to(exp.dtype) + 127).clamp(0, 254)
            byte = torch.where(big > 0, byte, torch.zeros_like(byte)).to(torch.uint8)
            s[x + "_scale"][at, head, off] = byte
            val = val / _factor(byte)[..., None]
        s[x + "_pages"][at, head, off] = val.to(s[x + "_pages"].dtype)
    return _written(s)


def _written(s):
    got = dict(k=s["k_pages"], v=s["v_pages"])
    if s["k_scale"] is not None:
        got.update(k_scale=s["k_scale"], v_scale=s["v_scale"])
    return got


def _plain_read(s):
    H = s["k_pages"].shape[1]
    B, _, n, d = s["k_out"].shape
    i, first, rows, page = _places(s, H)
    slot = (rows if s["rows"] is not None else first[:, None, :] + rows)
    at = s["table"].long()[:, None, :].expand(B, H, -1).gather(2, slot // page)
    off = slot % page
    head = torch.arange(H, device="cuda")[None, :, None]
    live = (torch.arange(n, device="cuda")[None, :] < s["counts"][:, None])[:, None, :, None]
    for x in "kv":
        val = s[x + "_pages"][at, head, off].float()
        if s[x + "_scale"] is not None:
            val = val * _factor(s[x + "_scale"][at, head, off])[..., None]
        s[x + "_out"].copy_(torch.where(live, val.to(s["dst"]), s[x + "_out"]))
    return s["k_out"], s["v_out"]


def _dense(pages, scale, table):
    """The slots of every sequence as fp32 rows [B, Hkv, slots, d]."""
    B, P = table.shape
    _, H, page, d = pages.shape
    val = pages[table.long()].float()                                # [B, P, H, page, d]
    if scale is not None:
        val = val * _factor(scale[table.long()])[..., None]
    return val.permute(0, 2, 1, 3, 4).reshape(B, H, P * page, d)


def _visible(s, n):
    """Which slots a row sees [B, T, n], and which rows there are [B, T]."""
    T = s["q"].shape[2]
    L, Q = s["lengths"].long()[:, None], s["q_lengths"].long()[:, None]
    t, j = torch.arange(T, device="cuda"), torch.arange(n, device="cuda")
    last = (L - Q + t if s["causal"] else (L - 1).expand(-1, T))[..., None]
    return (j <= last) & (j < L[..., None]), t < Q


def _plain_attend(s):
    q = s["q"]
    B, Hq, T, d = q.shape
    K = _dense(s["k_pages"], s["k_scale"], s["table"])
    H, n = K.shape[1], K.shape[2]
    G = Hq // H
    seen, live = _visible(s, n)
    S = q.float().reshape(B, H, G * T, d) @ K.transpose(2, 3)
    del K
    S = S.reshape(B, H, G, T, n).mul_(1.0 / math.sqrt(d))
    S.masked_fill_(~seen[:, None, None], -math.inf)
    m = S.amax(dim=4, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    P = S.sub_(m).exp_()
    l = P.sum(dim=4, keepdim=True)
    V = _dense(s["v_pages"], s["v_scale"], s["table"])
    O = (P.reshape(B, H, G * T, n) @ V).reshape(B, H, G, T, d)
    O = torch.where(l > 0, O / l, torch.zeros_like(O)).reshape(B, Hq, T, d)
    lse = (m + l.log()).reshape(B, Hq, T)
    live = live[:, None]
    s["out"].copy_(torch.where(live[..., None], O.to(q.dtype), s["out"]))
    s["lse"].copy_(torch.where(live, lse, s["lse"]))
    return s["out"], s["lse"]


# ---- the library's calls -------------------------------------------------------

def _own(s):
    import kv_cache_eviction_scores_b200 as dk

    scales = dict(k_scale=s["k_scale"], v_scale=s["v_scale"])
    if s["op"] == "write":
        dk.dropkv_cache_write(s["k"], s["v"], s["k_pages"], s["v_pages"], s["table"],
                              rows=s["rows"], start=s["start"], counts=s["counts"], **scales)
        return _written(s)
    if s["op"] == "read":
        return dk.dropkv_cache_read(s["k_pages"], s["v_pages"], s["table"], s["n"], rows=s["rows"],
                                    start=s["start"], counts=s["counts"], dtype=s["dst"],
                                    out=(s["k_out"], s["v_out"]), **scales)
    return dk.dropkv_cache_attention(s["q"], s["k_pages"], s["v_pages"], s["table"], s["lengths"],
                                     q_lengths=s["q_lengths"], causal=s["causal"], out=s["out"],
                                     lse=s["lse"], **scales)


def run(state):
    if own:
        return _own(state)
    if state["op"] == "write":
        return _plain_write(state)
    if state["op"] == "read":
        return _plain_read(state)
    return _plain_attend(state)


def work(case):
    B, Hkv, d = case["B"], case["Hkv"], case["d"]
    held = d * BYTES[case["fmt"]] + (1 if case["fmt"] == "e4m3" else 0)  # a row in the cache
    if case["op"] != "attend":
        moved = sum(_ragged(B, case["count_min"], case["count"])) * Hkv
        dense = d * BYTES[case["src" if case["op"] == "write" else "dst"]]
        return {"bytes": moved * (2 * (held + dense) + (4 if case["rows"] else 0)), "flops": 0}
    G = case["Hq"] // Hkv
    pairs = slots = tokens = 0
    for L, T in zip(_ragged(B, case["L_min"], case["L"]), _ragged(B, case["T_min"], case["T"])):
        tokens, slots = tokens + T, slots + L
        if case["causal"]:  # row t sees L - T + t + 1 slots
            pairs += sum(range(max(0, L - T + 1), L + 1))
        else:
            pairs += T * L
    io = tokens * case["Hq"] * (2 * d * BYTES[case["q"]] + 4)
    return {"bytes": 2 * slots * Hkv * held + io, "flops": 4 * pairs * G * Hkv * d}


# ---- in 64 bits ------------------------------------------------------------------

def _e4m3_round(x):
    """fp64 values of at most 448 rounded to the nearest of the e4m3 grid, ties to even."""
    step = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -9))).clamp(min=-6.0) - 3.0
    # one binade is eight steps, so a log2 that is off by rounding at a power of two is undone here
    step = torch.where(x.abs() >= torch.exp2(step + 4.0), step + 1.0, step)
    step = torch.where((x.abs() < torch.exp2(step + 3.0)) & (step > -9.0), step - 1.0, step)
    return torch.round(x / torch.exp2(step)) * torch.exp2(step)


def exact(case, seed):
    s = prepare(case, seed)
    B, page = case["B"], case["page"]
    table = s["table"].tolist()
    if case["op"] == "attend":
        return _exact_attend(case, s, table)
    counts, starts = s["counts"].tolist(), s["start"].tolist()
    if case["op"] == "read":
        got = []
        for x in "kv":
            pages, out = s[x + "_pages"], s[x + "_out"].double()
            for b in range(B):
                order = torch.tensor(table[b], device="cuda")
                for h in range(case["Hkv"]):
                    line = pages[order, h].double()
                    if s[x + "_scale"] is not None:
                        line = torch.ldexp(line, s[x + "_scale"][order, h].double()[..., None] - 127)
                    line = line.reshape(-1, case["d"])
                    c = counts[b]
                    if s["rows"] is not None:
                        out[b, h, :c] = line[s["rows"][b, h, :c].long()]
                    else:
                        out[b, h, :c] = line[starts[b]:starts[b] + c]
            got.append(out)
        return tuple(got)
    got = {}
    for x in "kv":
        pages = s[x + "_pages"].double()
        scale = s[x + "_scale"]
        for b in range(B):
            slot = torch.arange(starts[b], starts[b] + counts[b], device="cuda")
            where = torch.tensor(table[b], device="cuda")[slot // page]
            for h in range(case["Hkv"]):
                c = counts[b]
                val = s[x][b, h, s["rows"][b, h, :c].long() if s["rows"] is not None else slice(0, c)]
                val = val.double()
                if scale is not None:
                    # the least power of two that takes the row into [-448, 448]
                    big = val.abs().amax(dim=1)
                    e = torch.ceil(torch.log2((big / 448).clamp(min=2.0 ** -127)))
                    e = torch.where(torch.exp2(e - 1) * 448 >= big, e - 1, e)
                    e = torch.where(torch.exp2(e) * 448 < big, e + 1, e).clamp(min=-127)
                    scale[where, h, slot % page] = (e + 127).to(torch.uint8)
                    val = _e4m3_round(val * torch.exp2(-e)[:, None])
                pages[where, h, slot % page] = val
        got[x] = pages
        if scale is not None:
            got[x + "_scale"] = scale
    return got


def _exact_attend(case, s, table):
    out, lse = s["out"].double(), s["lse"].double()
    G, d = case["Hq"] // case["Hkv"], case["d"]
    for b, (L, T) in enumerate(zip(s["lengths"].tolist(), s["q_lengths"].tolist())):
        order = torch.tensor(table[b][: -(-L // case["page"])], device="cuda")
        hidden = None
        if case["causal"]:
            hidden = torch.ones(T, L, dtype=torch.bool, device="cuda").triu(L - T + 1)
        for h in range(case["Hkv"]):
            K, V = (s[x + "_pages"][order, h].double() for x in "kv")
            if s["k_scale"] is not None:
                K, V = (torch.ldexp(val, s[x + "_scale"][order, h].double()[..., None] - 127)
                        for x, val in (("k", K), ("v", V)))
            K, V = K.reshape(-1, d)[:L], V.reshape(-1, d)[:L]
            for g in range(h * G, (h + 1) * G):
                S = torch.einsum("td,jd->tj", s["q"][b, g, :T].double(), K) / math.sqrt(d)
                if hidden is not None:
                    S = S.masked_fill(hidden, -math.inf)
                lse[b, g, :T] = torch.logsumexp(S, dim=1)
                weight = torch.exp(S - lse[b, g, :T, None]).nan_to_num(0.0)
                out[b, g, :T] = weight @ V
    return out, lse
