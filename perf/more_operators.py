"""Operators around a paged key/value cache as they are measured: attention over
a cache that holds 4-bit values, appending keys and values with the position
rotation applied on the way (queries too), and reading tokens back.

A cache holds K and V as pools of pages and three integer tensors: page_table
[seqs][max_pages] (-1: no page), seq_lens [seqs], ref_counts [pages].  A pool of
bf16 or float32 values is [pages][heads][page_size][d] (``layout`` "token": token
by token).  A pool of 4-bit values holds for each page and head page_size * d / 2
bytes of codes (slot by slot, two columns to a byte, the even one in the low
half) and then page_size * d / 16 bytes of scales, one to 16 columns.  A code is
sign, two exponent bits and a fraction bit (0, 0.5, 1, 1.5, 2, 3, 4, 6); a scale
has five exponent bits and three fraction bits: a float16's bits 14 .. 7.

``run`` takes one pass through one operator, in its plain form with elementary
torch operations, or through the library where ``own`` is true.
"""
import math
import random

import torch

own = False

BF16 = torch.bfloat16
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32, "e2m1": torch.bfloat16}   # of the rows that go in and out
SCALE_TOP = 10240.0


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _attend(name, seqs, ctx_lo, ctx_hi, new_lo, new_hi, heads, group, d, page, causal=True, ragged=1):
    c = dict(kind="attend", store="e2m1", layout="head", seqs=seqs, ctx_lo=ctx_lo, ctx_hi=ctx_hi, new_lo=new_lo,
             new_hi=new_hi, heads=heads, group=group, d=d, page=page, causal=causal, ragged=ragged)
    return dict(c, name=name) if name else c


def _append(name, store, seqs, ctx_lo, ctx_hi, new_lo, new_hi, heads, group, d, page, rot, pairs="halves", placed=False,
            layout="head", ragged=1):
    c = dict(kind="append", store=store, layout=layout, seqs=seqs, ctx_lo=ctx_lo, ctx_hi=ctx_hi, new_lo=new_lo,
             new_hi=new_hi, heads=heads, group=group, d=d, page=page, rot=rot, pairs=pairs, placed=placed, ragged=ragged)
    return dict(c, name=name) if name else c


def _step(name, seqs, ctx_lo, ctx_hi, heads, group, d, page, rot, ragged=1):
    c = dict(kind="step", store="e2m1", layout="head", seqs=seqs, ctx_lo=ctx_lo, ctx_hi=ctx_hi, new_lo=1, new_hi=1,
             heads=heads, group=group, d=d, page=page, rot=rot, pairs="halves", placed=False, causal=True, ragged=ragged)
    return dict(c, name=name) if name else c


def _read(name, store, seqs, len_lo, len_hi, heads, d, page, layout="head", ragged=1):
    c = dict(kind="read", store=store, layout=layout, seqs=seqs, ctx_lo=0, ctx_hi=0, new_lo=len_lo, new_hi=len_hi,
             heads=heads, d=d, page=page, ragged=ragged)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one decode step of a few short conversations: latency counts
        _attend("attend4_decode_4x1k", 4, 300, 1000, 1, 1, 8, 4, 128, 16, ragged=2),
        # one decode step of a full server: a stream over every cached key and value
        _attend("attend4_decode_64x8k", 64, 2048, 8191, 1, 1, 8, 4, 128, 64, ragged=3),
        # five drafted tokens a sequence checked at once
        _attend("attend4_verify_16x4k", 16, 1000, 4096, 5, 5, 2, 8, 128, 32, ragged=4),
        # chunks of long prompts: matrix work
        _attend("attend4_chunk_4x1k_8k", 4, 4000, 8192, 511, 1024, 8, 4, 128, 64, ragged=5),
        # a short chunk behind one very long context: few query rows, a long axis to split
        _attend("attend4_long_1x128_131k", 1, 130907, 130907, 128, 128, 4, 4, 64, 16, ragged=6),
        # a layer's decode step over the 4-bit cache: the new token rotated and appended, then attended
        _step("step4_32x4k", 32, 1000, 4095, 8, 4, 128, 16, 128, ragged=7),
        # the new tokens of a decode step, into a bf16 cache: latency counts
        _append("rotate_decode_64", "bf16", 64, 500, 4000, 1, 1, 8, 4, 128, 16, 128, ragged=8),
        # prompt chunks into a bf16 cache with pages in token order
        _append("rotate_prompt_4x2k", "bf16", 4, 1000, 4000, 1500, 2048, 8, 4, 128, 64, 128, layout="token", ragged=9),
        # float32, neighbouring columns rotated, three quarters of them, odd lengths
        _append("rotate_f32_3x700", "f32", 3, 0, 300, 333, 701, 4, 2, 64, 16, 48, pairs="neighbours", placed=True, ragged=10),
        # prompts into a 4-bit cache, and what it holds of them read back (to hand them on)
        _append("store4_prompt_4x2k", "e2m1", 4, 0, 500, 1500, 2048, 8, 4, 128, 64, 128, ragged=11),
        # whole sequences of a 4-bit cache read back
        _read("read4_16x4k", "e2m1", 16, 1000, 4096, 8, 128, 16, ragged=12),
        # a few sequences of a bf16 cache
        _read("read_bf16_3x900", "bf16", 3, 100, 901, 4, 96, 32, layout="token", ragged=13),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    ragged = rng.randrange(1, 1 << 20)
    kind = rng.choice(["attend", "attend", "attend", "append", "append", "step", "read"])
    d = rng.choice([32, 64, 64, 96, 128, 128, 128])
    page = rng.choice([16, 32, 64, 128, 256])
    heads = rng.choice([1, 2, 3, 4, 8])
    group = rng.choice([1, 2, 3, 4, 5, 8, 16])
    if kind == "attend":
        seqs = _log_int(rng, 1, 48)
        new_hi = 1 if rng.random() < 0.35 else _log_int(rng, 1, 1024)
        # bounded so that no drawn case is dearer than the largest listed one
        ctx_hi = _log_int(rng, 64, 65536)
        ctx_hi = max(16, min(ctx_hi, int(3.0e9 / (seqs * heads * d * 8)), int(5.0e10 / (seqs * heads * group * d * new_hi)),
                             int(6.0e8 / (seqs * heads * group * new_hi))))
        return _attend(None, seqs, rng.randint(0, ctx_hi), ctx_hi, rng.randint(1, new_hi), new_hi, heads, group, d, page,
                       rng.random() < 0.75, ragged)
    rot = rng.choice([d, d, d // 2, d // 4, 3 * d // 4])
    if kind == "step":
        seqs = _log_int(rng, 1, 48)
        ctx_hi = max(16, min(_log_int(rng, 64, 16384), int(2.0e9 / (seqs * heads * d * 8)),
                             int(6.0e8 / (seqs * heads * group))))
        return _step(None, seqs, rng.randint(0, ctx_hi), ctx_hi, heads, group, d, page, rot, ragged)
    store = rng.choice(["e2m1", "e2m1", "bf16", "bf16", "f32"])
    layout = "head" if store == "e2m1" else rng.choice(["head", "token"])
    if kind == "read":
        seqs = _log_int(rng, 1, 48)
        hi = max(16, min(_log_int(rng, 16, 8192), int(6.0e7 / (seqs * heads * d))))
        return _read(None, store, seqs, rng.randint(1, hi), hi, heads, d, page, layout, ragged)
    seqs = _log_int(rng, 1, 64)
    new_hi = max(1, min(_log_int(rng, 1, 2048), int(4.0e7 / (seqs * heads * (2 + group) * d))))
    ctx_hi = max(16, min(_log_int(rng, 16, 8192), int(2.0e8 / (seqs * heads * d))))
    return _append(None, store, seqs, rng.randint(0, ctx_hi), ctx_hi, rng.randint(1, new_hi), new_hi, heads, group, d, page, rot,
                   rng.choice(["halves", "halves", "neighbours"]), rng.random() < 0.3, layout, ragged)


# ---------------------------------------------------------------------------
# lengths (of the case alone, so that work() knows them)
# ---------------------------------------------------------------------------
def _spread(rng, lo, hi, n):
    v = [rng.randint(lo, hi) for _ in range(n)]
    v[0] = hi
    return v


def _lens(case):
    """(tokens held before, new tokens) of every sequence."""
    rng = random.Random(case["ragged"])
    return _spread(rng, case["ctx_lo"], case["ctx_hi"], case["seqs"]), _spread(rng, case["new_lo"], case["new_hi"], case["seqs"])


def _ceil(a, b):
    return -(-a // b)


# ---------------------------------------------------------------------------
# the 4-bit format
# ---------------------------------------------------------------------------
def _quantize(x):
    """float32 [..., d] to codes [..., d / 2] and scales [..., d / 16], bytes."""
    g = x.unflatten(-1, (-1, 16))
    top = g.abs().amax(-1)
    t = top / torch.full_like(top, 6.0)   # (a division by a number would multiply by its rounded reciprocal)
    exponent = torch.frexp(t).exponent.clamp(min=-13)
    step = torch.ldexp(torch.ones_like(t), exponent - 4)   # four significant bits, 2^-17 at least
    s = (torch.round(t / step) * step).clamp(max=SCALE_TOP)
    a = torch.where(s[..., None] > 0, g.abs() / s[..., None], 0.0)
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    code = torch.where(torch.signbit(g) & (s[..., None] > 0), code + 8, code).flatten(-2)
    scales = (s.half().view(torch.int16) >> 7).to(torch.uint8)
    return code[..., 0::2] | (code[..., 1::2] << 4), scales


def _values(codes, scales):
    """What bytes stand for, float32."""
    byte = torch.arange(256, device=codes.device)
    steps = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0], device=codes.device)
    pairs = torch.stack([steps[byte & 15], steps[byte >> 4]], 1)
    s = (scales.to(torch.int16) << 7).view(torch.float16).float()
    return (pairs[codes.int()].flatten(-2).unflatten(-1, (-1, 16)) * s[..., None]).flatten(-2)


def _split(pool, page, d):
    """Codes [pages, heads, page, d / 2] and scales [pages, heads, page, d / 16] of a pool, as views of it."""
    flat = pool.flatten(-2)
    return flat[..., :page * d // 2].unflatten(-1, (page, d // 2)), flat[..., page * d // 2:].unflatten(-1, (page, d // 16))


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _randn(shape, dtype, gen):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(dtype)


def _pool(case, pages, gen):
    H, S, d = case["heads"], case["page"], case["d"]
    if case["store"] == "e2m1":
        pool = torch.empty((pages, H, S, 9 * d // 16), device="cuda", dtype=torch.uint8)
        codes, scales = _quantize(_randn((pages, H, S, d), torch.float32, gen))
        for part, values in zip(_split(pool, S, d), (codes, scales)):
            part.copy_(values)
        return pool
    t = torch.empty((pages, H, S, d) if case["layout"] == "head" else (pages, S, H, d), device="cuda", dtype=DTYPES[case["store"]])
    t.normal_(generator=gen)
    return t if case["layout"] == "head" else t.transpose(1, 2)


def _tables(lens, rows, max_pages, pages, page, seed):
    """Sequences of the given lengths in rows of the table, on random pages."""
    rng = random.Random(seed)
    free = list(range(pages))
    rng.shuffle(free)
    table = torch.full((rows, max_pages), -1, dtype=torch.int32)
    refs = torch.zeros(pages, dtype=torch.int32)
    seq_lens = torch.zeros(rows, dtype=torch.int32)
    at = 0
    for r, n in enumerate(lens):
        k = _ceil(n, page)
        ids = torch.tensor(free[at:at + k], dtype=torch.int32)
        at += k
        table[r, :k] = ids
        refs[ids.long()] = 1
        seq_lens[r] = n
    return table.cuda(), seq_lens.cuda(), refs.cuda()


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    ctx, new = _lens(case)
    H, S, d, kind = case["heads"], case["page"], case["d"], case["kind"]
    dtype = DTYPES[case["store"]]
    st = {"case": case}
    lens = [a + b for a, b in zip(ctx, new)]
    pages, rows = sum(_ceil(n, S) for n in lens) + 3, case["seqs"] + 1
    max_pages = max(_ceil(n, S) for n in lens) + 2
    T = sum(new)
    st["seqs"] = torch.randperm(case["seqs"], generator=gen, device="cuda").int()
    by_row = [0] * case["seqs"]      # table row r belongs to list entry order[r]
    for i, r in enumerate(st["seqs"].tolist()):
        by_row[r] = lens[i]
    st["page_table"], st["seq_lens"], st["ref_counts"] = _tables(by_row, rows, max_pages, pages, S, seed)
    starts = [0]
    for n in new:
        starts.append(starts[-1] + n)
    st["q_start"], st["T"], st["max_q"], st["keys"] = _ints(starts), T, max(new), max(lens)
    # what the plain forms pad and gather with
    st["entry"] = torch.repeat_interleave(torch.arange(len(new)), torch.tensor(new)).cuda()
    st["offset"] = torch.cat([torch.arange(n) for n in new]).cuda()
    st["k"], st["v"] = _pool(case, pages, gen), _pool(case, pages, gen)
    if kind == "attend":
        st["q"] = _randn((T, H * case["group"], d), dtype, gen) * 2
    if kind in ("append", "step"):
        # the rows of one projection: queries, keys and values of a token side by side
        qkv = _randn((T, H * (case["group"] + 2), d), dtype, gen)
        st["q"], st["k_new"], st["v_new"] = qkv.split([H * case["group"], H, H], 1)
        st["positions"] = None
        top = max(lens)
        if case["placed"]:     # tokens that stand further along than their index (the sequence's beginning was dropped)
            moved = random.Random(seed).randrange(1, 2000)
            top += moved
            st["positions"] = _ints([c + moved + t for c, n in zip(ctx, new) for t in range(n)])
        half = case["rot"] // 2
        turn = torch.arange(top, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(half, dtype=torch.float64) / half)
        st["table"] = torch.cat([turn.cos(), turn.sin()], 1).float().cuda()
    if own:
        # the handle a program keeps beside its cache (it holds the tensors' addresses and sizes)
        import exact_tiled_attention_17_gb300 as eta
        st["eta"] = eta
        st["cache"] = eta.PagedCache(st["k"][None], st["v"][None], st["page_table"], st["seq_lens"], st["ref_counts"])
    return st


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _gathered(st, pool, pages):
    """The pages of a pool as float32, [..., heads, page, d]."""
    case = st["case"]
    if case["store"] != "e2m1":
        return pool[pages].float()
    codes, scales = _split(pool, case["page"], case["d"])
    return _values(codes[pages], scales[pages])


def _attention(st, q):
    case = st["case"]
    S, Hk, g, d = case["page"], case["heads"], case["group"], case["d"]
    seqs = st["seqs"].long()
    n = seqs.numel()
    lens = st["seq_lens"][seqs].long()
    nq = (st["q_start"][1:] - st["q_start"][:-1]).long()
    cols = _ceil(st["keys"], S)
    pages = st["page_table"][seqs, :cols].long().clamp(min=0)
    key = torch.arange(cols * S, device="cuda")
    held = key[None] < lens[:, None]
    k = _gathered(st, st["k"], pages).transpose(1, 2).reshape(n, Hk, cols * S, d)
    v = _gathered(st, st["v"], pages).transpose(1, 2).reshape(n, Hk, cols * S, d)
    v = torch.where(held[:, None, :, None], v, 0.0)
    row = torch.arange(st["max_q"], device="cuda")
    at = (st["q_start"][:-1].long()[:, None] + row).clamp(max=q.shape[0] - 1)
    x = q[at].float().reshape(n, -1, Hk, g, d).permute(0, 2, 1, 3, 4).reshape(n, Hk, -1, d)
    s = torch.matmul(x, k.transpose(2, 3)) * (1.0 / math.sqrt(d))
    seen = held[:, None, :].expand(n, row.numel(), key.numel())
    if case["causal"]:
        seen = seen & (key <= (lens - nq)[:, None, None] + row[:, None])
    seen = seen.repeat_interleave(g, dim=1)[:, None]
    s = torch.where(seen, s, -math.inf)
    m = s.amax(dim=3, keepdim=True)
    p = torch.exp(s - torch.where(torch.isinf(m), 0.0, m))
    total = p.sum(dim=3, keepdim=True)
    o = torch.matmul(p, v) / torch.where(total > 0, total, 1.0)
    lse = (m + torch.log(total)).squeeze(3)
    o = o.reshape(n, Hk, -1, g, d).permute(0, 2, 1, 3, 4).reshape(n, -1, Hk * g, d)
    lse = lse.reshape(n, Hk, -1, g).permute(0, 2, 1, 3).reshape(n, -1, Hk * g)
    return o[st["entry"], st["offset"]].to(q.dtype), lse[st["entry"], st["offset"]]


def _places(st):
    """Page, slot and index in its sequence of every new token."""
    S = st["case"]["page"]
    seq = st["seqs"].long()[st["entry"]]
    new = (st["q_start"][1:] - st["q_start"][:-1]).long()
    index = st["seq_lens"].long()[seq] - new[st["entry"]] + st["offset"]
    return st["page_table"][seq, index // S].long(), index % S, index


def _rotated(st, x, at):
    """Rows [T, heads, d] turned by the table's row at[t], float32."""
    rot = st["case"]["rot"]
    cos, sin = st["table"][at][:, None].chunk(2, -1)
    turned, rest = x[..., :rot].float(), x[..., rot:].float()
    if st["case"]["pairs"] == "halves":
        a, b = turned.chunk(2, -1)
        return torch.cat([a * cos - b * sin, b * cos + a * sin, rest], -1)
    a, b = turned[..., 0::2], turned[..., 1::2]
    return torch.cat([torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2), rest], -1)


def _plain_store(st):
    """The new tokens' rows into the pools; returns the rotated queries and where the tokens lie."""
    case = st["case"]
    page, slot, index = _places(st)
    at = index if st["positions"] is None else st["positions"].long()
    k, v = _rotated(st, st["k_new"], at), st["v_new"].float()
    if case["store"] == "e2m1":
        (kc, ks), (vc, vs) = _split(st["k"], case["page"], case["d"]), _split(st["v"], case["page"], case["d"])
        for_k, for_v = _quantize(k), _quantize(v)
        kc.transpose(1, 2)[page, slot], ks.transpose(1, 2)[page, slot] = for_k
        vc.transpose(1, 2)[page, slot], vs.transpose(1, 2)[page, slot] = for_v
    else:
        st["k"].transpose(1, 2)[page, slot] = k.to(st["k"].dtype)
        st["v"].transpose(1, 2)[page, slot] = v.to(st["v"].dtype)
    return _rotated(st, st["q"], at).to(st["q"].dtype), page, slot


def _plain_rows(st, pool, page, slot):
    """The rows that a pool holds at the given places, [T, heads, d]."""
    case = st["case"]
    if case["store"] != "e2m1":
        return pool.transpose(1, 2)[page, slot]
    codes, scales = _split(pool, case["page"], case["d"])
    return _values(codes.transpose(1, 2)[page, slot], scales.transpose(1, 2)[page, slot]).to(BF16)


def _plain(st):
    kind = st["case"]["kind"]
    if kind == "attend":
        o, lse = _attention(st, st["q"])
        return {"o": o, "lse": lse}
    if kind == "read":
        page, slot, _ = _places(st)
        return {"k": _plain_rows(st, st["k"], page, slot), "v": _plain_rows(st, st["v"], page, slot)}
    q, page, slot = _plain_store(st)
    if kind == "step":
        o, lse = _attention(st, q)
        return {"q": q, "o": o, "lse": lse}
    if st["case"]["store"] != "e2m1":
        return {"q": q, "k": st["k"], "v": st["v"]}
    # what the cache now holds of the new tokens, as values
    return {"q": q, "k": _plain_rows(st, st["k"], page, slot), "v": _plain_rows(st, st["v"], page, slot)}


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def _own(st):
    eta, cache, case = st["eta"], st["cache"], st["case"]
    kind, seqs, q_start = case["kind"], st["seqs"], st["q_start"]
    if kind == "attend":
        o, lse = eta.attn_paged_fwd(st["q"], cache, 0, seqs, q_start, max_q=st["max_q"], causal=case["causal"])
        return {"o": o, "lse": lse}
    if kind == "read":
        k, v = eta.attn_cache_read(cache, 0, seqs, q_start, st["T"])
        return {"k": k, "v": v}
    q = eta.attn_cache_append_rotated(cache, 0, st["k_new"], st["v_new"], seqs, q_start, st["table"], q=st["q"],
                                      neighbours=case["pairs"] == "neighbours", positions=st["positions"])
    if kind == "step":
        o, lse = eta.attn_paged_fwd(q, cache, 0, seqs, q_start, max_q=st["max_q"], causal=case["causal"])
        return {"q": q, "o": o, "lse": lse}
    if case["store"] != "e2m1":
        return {"q": q, "k": st["k"], "v": st["v"]}
    k, v = eta.attn_cache_read(cache, 0, seqs, q_start, st["T"])
    return {"q": q, "k": k, "v": v}


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    ctx, new = _lens(case)
    H, S, d, T = case["heads"], case["page"], case["d"], sum(new)
    lens = [a + b for a, b in zip(ctx, new)]
    es = 4 if case["store"] == "f32" else 2                                # of a value that goes in or out
    row = 9 * d // 16 if case["store"] == "e2m1" else d * es               # of a row in the cache
    total = {"bytes": sum(_ceil(n, S) for n in lens) * 4, "flops": 0}
    if case["kind"] in ("attend", "step"):
        Hq = H * case["group"]
        pairs = sum(b * a + b * (b + 1) // 2 if case["causal"] else b * (a + b) for a, b in zip(ctx, new))
        total["bytes"] += 2 * sum(lens) * H * row + 2 * T * Hq * d * es + T * Hq * 4
        total["flops"] += 4 * pairs * Hq * d
    if case["kind"] in ("append", "step"):
        rows = T * H * (2 + case["group"])
        total["bytes"] += rows * d * es + T * H * case["group"] * d * es + 2 * T * H * row + T * case["rot"] * 4
        total["flops"] += 3 * T * H * (1 + case["group"]) * case["rot"]
    if case["kind"] == "read" or (case["kind"] == "append" and case["store"] == "e2m1"):
        total["bytes"] += 2 * T * H * (row + d * es)
    return total


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------
def _exact_turn(st, x, at):
    """Rotation as a product of complex numbers."""
    rot, half = st["case"]["rot"], st["case"]["rot"] // 2
    row = st["table"][at].double()
    z = torch.complex(row[:, :half], row[:, half:])[:, None]
    x = x.double()
    first = torch.arange(half, device="cuda") * (1 if st["case"]["pairs"] == "halves" else 2)
    second = first + (half if st["case"]["pairs"] == "halves" else 1)
    w = torch.complex(x[..., first], x[..., second]) * z
    out = x.clone()
    out[..., first], out[..., second] = w.real, w.imag
    return out


def _exact_held(x):
    """What a 4-bit cache holds of rows, by nearness: of all scales the nearest, of all codes the nearest."""
    g = x.reshape(*x.shape[:-1], -1, 16)
    bits = torch.arange(0xE2 + 1, dtype=torch.int16, device="cuda")     # up to 10240
    scales = (bits << 7).view(torch.float16).double()
    top = g.abs().amax(-1)
    want = (top / torch.full_like(top, 6)).clamp(max=float(scales[-1]))
    above = torch.searchsorted(scales, want).clamp(1, scales.numel() - 1)
    lo, hi = scales[above - 1], scales[above]
    near_hi = (hi - want < want - lo) | ((hi - want == want - lo) & (above % 2 == 0))
    s = torch.where(near_hi, hi, lo)[..., None]
    steps = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64, device="cuda")
    a = torch.where(s > 0, g.abs() / s, 0.0)
    above = torch.searchsorted(steps, a).clamp(1, 7)
    lo, hi = steps[above - 1], steps[above]
    near_hi = (hi - a < a - lo) | ((hi - a == a - lo) & (above % 2 == 0))
    return (torch.where(near_hi, hi, lo) * s * torch.sign(g)).reshape(x.shape)


def _exact_cached(st, which, ids, n):
    """K or V of a sequence on the given pages, [heads, n, d]."""
    case = st["case"]
    H, S, d = case["heads"], case["page"], case["d"]
    flat = st[which][ids].reshape(len(ids), H, -1).long()
    codes = flat[..., :S * d // 2]
    sign, size = torch.tensor([1.0, -1.0], device="cuda").double(), torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device="cuda").double()
    nibbles = torch.stack([codes % 16, codes // 16], -1).reshape(len(ids), H, S, d)
    scale = flat[..., S * d // 2:].reshape(len(ids), H, S, d // 16)
    scale = torch.where(scale < 8, scale / 2.0 ** 17, (8 + scale % 8).double() * 2.0 ** (scale // 8 - 18).double())
    x = sign[nibbles // 8] * size[nibbles % 8] * scale.repeat_interleave(16, -1)
    return x.transpose(0, 1).reshape(H, -1, d)[:, :n]


def _exact_attention(st, q, fresh=None):
    """Attention by its definition, sequence by sequence and head by head.
    fresh: (k, v) of the new tokens where the cache does not hold them yet."""
    case = st["case"]
    S, Hk, g, d = case["page"], case["heads"], case["group"], case["d"]
    starts, table = st["q_start"].tolist(), st["page_table"].tolist()
    outs, lses = [], []
    for i, row in enumerate(st["seqs"].tolist()):
        n = int(st["seq_lens"][row])
        a, b = starts[i], starts[i + 1]
        ids = torch.tensor(table[row][:_ceil(n, S)], device="cuda")
        k, v = _exact_cached(st, "k", ids, n), _exact_cached(st, "v", ids, n)
        if fresh is not None:
            k[:, n - (b - a):], v[:, n - (b - a):] = fresh[0][a:b].transpose(0, 1), fresh[1][a:b].transpose(0, 1)
        heads_o, heads_l = [], []
        for h in range(Hk):
            for j in range(g):
                s = q[a:b, h * g + j].double() @ k[h].T / d ** 0.5
                if case["causal"]:
                    last = torch.arange(n - (b - a), n, device="cuda")
                    s.masked_fill_(torch.arange(n, device="cuda")[None] > last[:, None], -math.inf)
                w = torch.logsumexp(s, dim=1)
                heads_o.append(torch.exp(s - w[:, None]) @ v[h])
                heads_l.append(w)
        outs.append(torch.stack(heads_o, 1))
        lses.append(torch.stack(heads_l, 1))
    return torch.cat(outs), torch.cat(lses)


def exact(case, seed):
    """The definitions in float64.  What only moves values (reading, V on its way
    into a cache of its own type) has none."""
    if case["kind"] == "read":
        return None
    st = prepare(case, seed)
    if case["kind"] == "attend":
        o, lse = _exact_attention(st, st["q"])
        return {"o": o, "lse": lse}
    starts, lens = st["q_start"].tolist(), st["seq_lens"].tolist()
    at = st["positions"]
    if at is None:
        at = torch.cat([torch.arange(lens[r] - (b - a), lens[r], device="cuda")
                        for r, a, b in zip(st["seqs"].tolist(), starts, starts[1:])])
    q, k = _exact_turn(st, st["q"], at.long()), _exact_turn(st, st["k_new"], at.long())
    if case["store"] != "e2m1":
        table, S = st["page_table"].tolist(), case["page"]
        held = st["k"].double()
        for r, a, b in zip(st["seqs"].tolist(), starts, starts[1:]):
            index = torch.arange(lens[r] - (b - a), lens[r], device="cuda")
            ids = torch.tensor(table[r], device="cuda")[index // S]
            held[ids, :, index % S] = k[a:b]
        return {"q": q, "k": held, "v": None}
    k, v = _exact_held(k), _exact_held(st["v_new"].double())
    if case["kind"] == "append":
        return {"q": q, "k": k, "v": v}
    o, lse = _exact_attention(st, q.to(BF16), (k, v))
    return {"q": q, "o": o, "lse": lse}
