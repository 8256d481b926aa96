"""The paged key/value cache operators as they are measured: attention of new
tokens over a paged cache, the growth of a batch by new tokens (free to a kept
length, reserve, append), forking sequences and compacting the page pool.

A cache holds K and V as pools of pages, [layers][pages][heads][page_size][d]
(``layout`` says how a page lies in memory: head by head or token by token),
and three integer tensors: page_table [seqs][max_pages] (-1: no page), seq_lens
[seqs] and ref_counts [pages] (table entries that name the page, 0 = free).

``run`` takes one pass through one operator, in its plain form with elementary
torch operations, or through the library where ``own`` is true.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _attend(name, seqs, ctx_lo, ctx_hi, new_lo, new_hi, heads, group, d, page, dtype="bf16", causal=True, layout="head",
            ragged=1):
    c = dict(kind="attend", seqs=seqs, ctx_lo=ctx_lo, ctx_hi=ctx_hi, new_lo=new_lo, new_hi=new_hi, heads=heads,
             group=group, d=d, page=page, dtype=dtype, causal=causal, layout=layout, ragged=ragged)
    return dict(c, name=name) if name else c


def _grow(name, seqs, ctx_lo, ctx_hi, new_lo, new_hi, layers, heads, d, page, dtype="bf16", layout="head", ragged=1):
    c = dict(kind="grow", seqs=seqs, ctx_lo=ctx_lo, ctx_hi=ctx_hi, new_lo=new_lo, new_hi=new_hi, layers=layers,
             heads=heads, d=d, page=page, dtype=dtype, layout=layout, ragged=ragged)
    return dict(c, name=name) if name else c


def _fork(name, parents, forks, ctx_lo, ctx_hi, copy, layers, heads, d, page, dtype="bf16", layout="head", ragged=1):
    c = dict(kind="fork", parents=parents, forks=forks, ctx_lo=ctx_lo, ctx_hi=ctx_hi, copy=copy, layers=layers,
             heads=heads, d=d, page=page, dtype=dtype, layout=layout, ragged=ragged)
    return dict(c, name=name) if name else c


def _compact(name, seqs, ctx_lo, ctx_hi, spare, layers, heads, d, page, dtype="bf16", layout="head", ragged=1):
    c = dict(kind="compact", seqs=seqs, ctx_lo=ctx_lo, ctx_hi=ctx_hi, spare=spare, layers=layers, heads=heads, d=d,
             page=page, dtype=dtype, layout=layout, ragged=ragged)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one decode step of a few short conversations: latency counts
        _attend("attend_decode_4x1k", 4, 300, 1000, 1, 1, 8, 4, 128, 16, ragged=2),
        # one decode step of a full server: a stream over every cached key and value
        _attend("attend_decode_64x8k", 64, 2048, 8191, 1, 1, 8, 4, 128, 64, ragged=3),
        # five drafted tokens a sequence checked at once, odd lengths, pages in token order
        _attend("attend_verify_16x4k", 16, 1000, 4096, 5, 5, 2, 8, 128, 32, layout="token", ragged=4),
        # chunks of long prompts: matrix work
        _attend("attend_chunk_4x1k_8k", 4, 4000, 8192, 511, 1024, 8, 4, 128, 64, ragged=5),
        # a short chunk behind one very long context: few query rows, a long axis to split
        _attend("attend_long_1x128_131k", 1, 130907, 130907, 128, 128, 4, 4, 64, 16, ragged=6),
        # float32, every query sees every key (a cached encoder output)
        _attend("attend_f32_3x200", 3, 700, 1500, 77, 200, 4, 2, 64, 16, dtype="f32", causal=False, ragged=7),
        # the cache of a decode step: two rejected drafts go, one to three tokens come
        _grow("grow_decode_64", 64, 500, 4000, 1, 3, 2, 8, 128, 16, ragged=8),
        # the cache of a prompt chunk
        _grow("grow_prompt_4x2k", 4, 1000, 4000, 1500, 2048, 2, 8, 128, 64, layout="token", ragged=9),
        # a beam-search step: losing beams are freed, the winners forked
        _fork("fork_beams_32", 8, 32, 500, 1500, False, 4, 8, 128, 16, ragged=10),
        # whole sequences copied to pages of their own
        _fork("fork_copies_4x8k", 4, 4, 6000, 8192, True, 2, 8, 128, 64, ragged=11),
        # a small pool after many sequences have left
        _compact("compact_1k_pages", 24, 100, 500, 1.0, 2, 8, 64, 16, ragged=12),
        # a large pool, a third of it holes
        _compact("compact_8k_pages", 64, 3000, 8191, 0.5, 1, 8, 128, 64, layout="token", ragged=13),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    ragged = rng.randrange(1, 1 << 20)
    kind = rng.choice(["attend", "attend", "attend", "grow", "fork", "compact"])
    d = rng.choice([32, 64, 64, 96, 128, 128, 128])
    page = rng.choice([16, 32, 64, 128])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    layout = rng.choice(["head", "token"])
    heads = rng.choice([1, 2, 3, 4, 8])
    if kind == "attend":
        group = rng.choice([1, 2, 3, 4, 5, 8, 16])
        seqs = _log_int(rng, 1, 48)
        new_hi = 1 if rng.random() < 0.35 else _log_int(rng, 1, 1024 if dtype == "bf16" else 256)
        # bounded so that no drawn case is dearer than the largest listed one
        ctx_hi = _log_int(rng, 64, 65536)
        ctx_hi = max(16, min(ctx_hi, int(3.0e9 / (seqs * heads * d * 8)), int(5.0e10 / (seqs * heads * group * d * new_hi)),
                             int(6.0e8 / (seqs * heads * group * new_hi))))
        if dtype == "f32":
            ctx_hi = max(16, min(ctx_hi, int(2.0e9 / (seqs * heads * group * d * new_hi))))
        ctx_lo = rng.randint(0, ctx_hi)
        return _attend(None, seqs, ctx_lo, ctx_hi, rng.randint(1, new_hi), new_hi, heads, group, d, page, dtype,
                       rng.random() < 0.75, layout, ragged)
    layers = rng.randint(1, 4)
    per_token = layers * heads * d * 8
    if kind == "grow":
        seqs = _log_int(rng, 1, 64)
        new_hi = max(1, min(_log_int(rng, 1, 2048), int(2.0e8 / (seqs * per_token))))
        ctx_hi = max(16, min(_log_int(rng, 16, 8192), int(1.0e9 / (seqs * per_token))))
        return _grow(None, seqs, rng.randint(1, ctx_hi), ctx_hi, rng.randint(1, new_hi), new_hi, layers, heads, d, page,
                     dtype, layout, ragged)
    if kind == "fork":
        parents = rng.randint(1, 8)
        forks = _log_int(rng, 1, 32)
        copy = rng.random() < 0.4
        ctx_hi = max(16, min(_log_int(rng, 16, 8192), int(2.5e8 / ((forks if copy else 1) * per_token)),
                             int(1.0e9 / (parents * per_token))))
        return _fork(None, parents, forks, rng.randint(1, ctx_hi), ctx_hi, copy, layers, heads, d, page, dtype, layout,
                     ragged)
    seqs = _log_int(rng, 1, 64)
    ctx_hi = max(16, min(_log_int(rng, 16, 8192), int(8.0e8 / (seqs * per_token))))
    return _compact(None, seqs, rng.randint(1, ctx_hi), ctx_hi, round(rng.uniform(0.1, 1.0), 3), layers, heads, d, page,
                    dtype, layout, ragged)


# ---------------------------------------------------------------------------
# lengths (of the case alone, so that work() knows them)
# ---------------------------------------------------------------------------
def _spread(rng, lo, hi, n):
    v = [rng.randint(lo, hi) for _ in range(n)]
    v[0] = hi
    return v


def _lens(case):
    """(tokens held before, new tokens) of every sequence that takes part."""
    rng = random.Random(case["ragged"])
    n = case["parents"] if case["kind"] == "fork" else case["seqs"]
    ctx = _spread(rng, case["ctx_lo"], case["ctx_hi"], n)
    new = _spread(rng, case["new_lo"], case["new_hi"], n) if "new_lo" in case else [0] * n
    return ctx, new


def _ceil(a, b):
    return -(-a // b)


def _cut(case):
    """grow: how many tokens each sequence gives back first (rejected drafts)."""
    ctx, _ = _lens(case)
    rng = random.Random(case["ragged"] + 1)
    return [rng.randint(0, min(2, c)) for c in ctx]


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _randn(shape, dtype, gen):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(dtype)


def _pool(case, layers, pages, gen):
    H, S, d = case["heads"], case["page"], case["d"]
    order = (layers, pages, H, S, d) if case["layout"] == "head" else (layers, pages, S, H, d)
    t = torch.empty(order, device="cuda", dtype=DTYPES[case["dtype"]])
    t.normal_(generator=gen)
    return t if case["layout"] == "head" else t.transpose(2, 3)


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
    dtype = DTYPES[case["dtype"]]
    st = {"case": case}
    if kind == "attend":
        lens = [a + b for a, b in zip(ctx, new)]
        used = sum(_ceil(n, S) for n in lens)
        pages, rows = used + 3, case["seqs"] + 1
        max_pages = max(_ceil(n, S) for n in lens) + 2
        layers = 1
        T = sum(new)
        st["q"] = _randn((T, H * case["group"], d), dtype, gen) * 2
        st["seqs"] = torch.randperm(case["seqs"], generator=gen, device="cuda").int()
        # table row r belongs to list entry order[r]
        order = st["seqs"].tolist()
        by_row = [0] * case["seqs"]
        for i, r in enumerate(order):
            by_row[r] = lens[i]
        st["page_table"], st["seq_lens"], st["ref_counts"] = _tables(by_row, rows, max_pages, pages, S, seed)
        starts = [0]
        for n in new:
            starts.append(starts[-1] + n)
        st["q_start"] = _ints(starts)
        st["max_q"] = max(new)
        # what the plain form pads and gathers with
        st["keys"] = max(lens)
        st["entry"] = torch.repeat_interleave(torch.arange(len(new)), torch.tensor(new)).cuda()
        st["offset"] = torch.cat([torch.arange(n) for n in new]).cuda()
    elif kind == "grow":
        cut = _cut(case)
        lens = [a + b for a, b in zip(ctx, new)]
        used = sum(_ceil(n, S) for n in ctx)
        more = sum(_ceil(n, S) for n in lens)
        pages, rows = max(used, more) + 8, case["seqs"] + 2
        max_pages = max(_ceil(n, S) for n in lens) + 1
        layers = case["layers"]
        st["page_table"], st["seq_lens"], st["ref_counts"] = _tables(ctx, rows, max_pages, pages, S, seed)
        st["seqs"] = _ints(range(len(ctx)))
        # the pass starts from what it leaves behind: ctx tokens a sequence, of
        # which the last (drafts and the pass's own tokens) go first
        st["keep"] = _ints([c - x for c, x in zip(ctx, cut)])
        st["n_new"] = _ints(new)
        starts = [0]
        for n in new:
            starts.append(starts[-1] + n)
        st["q_start"] = _ints(starts)
        st["k_new"] = _randn((layers, starts[-1], H, d), dtype, gen)
        st["v_new"] = _randn((layers, starts[-1], H, d), dtype, gen)
        st["entry"] = torch.repeat_interleave(torch.arange(len(new)), torch.tensor(new)).cuda()
        st["offset"] = torch.cat([torch.arange(n) for n in new]).cuda()
    elif kind == "fork":
        rng = random.Random(case["ragged"] + 2)
        layers, forks = case["layers"], case["forks"]
        which = [rng.randrange(case["parents"]) for _ in range(forks)]
        old = [rng.randint(1, 2 * S) for _ in range(forks)]   # what the losing beams hold
        lens = ctx + old
        fresh = sum(_ceil(ctx[w], S) if case["copy"] else 1 for w in which)
        pages = sum(_ceil(n, S) for n in lens) + fresh + 4
        max_pages = max(_ceil(n, S) for n in lens) + 2
        st["page_table"], st["seq_lens"], st["ref_counts"] = _tables(lens, len(lens), max_pages, pages, S, seed)
        st["parents"] = _ints(which)
        st["children"] = _ints(range(case["parents"], case["parents"] + forks))
    else:
        layers = case["layers"]
        used = sum(_ceil(n, S) for n in ctx)
        pages = used + max(1, int(used * case["spare"]))
        max_pages = max(_ceil(n, S) for n in ctx) + 1
        st["page_table"], st["seq_lens"], st["ref_counts"] = _tables(ctx, len(ctx), max_pages, pages, S, seed)
    st["k"] = _pool(case, layers, pages, gen)
    st["v"] = _pool(case, layers, pages, gen)
    if own:
        # the handle a program keeps beside its cache (it holds the tensors' addresses and sizes)
        import exact_tiled_attention_17_gb300 as eta
        st["eta"] = eta
        st["cache"] = eta.PagedCache(st["k"], st["v"], st["page_table"], st["seq_lens"], st["ref_counts"])
    return st


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _plain_attend(st):
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
    k = st["k"][0][pages].transpose(1, 2).reshape(n, Hk, cols * S, d).float()
    v = st["v"][0][pages].transpose(1, 2).reshape(n, Hk, cols * S, d).float()
    v = torch.where(held[:, None, :, None], v, 0.0)
    row = torch.arange(st["max_q"], device="cuda")
    at = (st["q_start"][:-1].long()[:, None] + row).clamp(max=st["q"].shape[0] - 1)
    q = st["q"][at].float().reshape(n, -1, Hk, g, d).permute(0, 2, 1, 3, 4).reshape(n, Hk, -1, d)
    s = torch.matmul(q, k.transpose(2, 3)) * (1.0 / math.sqrt(d))
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
    return {"o": o[st["entry"], st["offset"]].to(st["q"].dtype), "lse": lse[st["entry"], st["offset"]]}


def _plain_free(st, seqs, keep):
    S = st["case"]["page"]
    seqs = seqs.long()
    table, refs, lens = st["page_table"], st["ref_counts"], st["seq_lens"]
    keep = torch.minimum(keep, lens[seqs])
    rows = table[seqs]
    col = torch.arange(table.shape[1], device="cuda")
    gone = (col >= ((keep + S - 1) // S)[:, None]) & (rows >= 0)
    refs.index_add_(0, rows.clamp(min=0).reshape(-1).long(), -gone.reshape(-1).int())
    table[seqs] = torch.where(gone, -1, rows)
    lens[seqs] = keep


def _plain_take(st, have, need):
    """Free pages, lowest first, for entries that hold `have` and need `need`: (granted, page of every column)."""
    refs, cols = st["ref_counts"], st["page_table"].shape[1]
    used = refs > 0
    order = torch.sort(used.int(), stable=True).indices
    total = torch.cumsum(need, 0)
    granted = (have + need <= cols) & (total <= (~used).sum())
    col = torch.arange(cols, device="cuda")
    mine = (col >= have[:, None]) & (col < (have + need)[:, None]) & granted[:, None]
    at = ((total - need)[:, None] + col - have[:, None]).clamp(0, refs.numel() - 1)
    return granted, torch.where(mine, order[at].int(), -1)


def _plain_grow(st):
    case, S = st["case"], st["case"]["page"]
    table, refs, lens = st["page_table"], st["ref_counts"], st["seq_lens"]
    _plain_free(st, st["seqs"], st["keep"])
    seqs = st["seqs"].long()
    have = (lens[seqs] + S - 1) // S
    need = (lens[seqs] + st["n_new"] + S - 1) // S - have
    granted, ids = _plain_take(st, have, need)
    refs.index_add_(0, ids.clamp(min=0).reshape(-1).long(), (ids >= 0).reshape(-1).int())
    table[seqs] = torch.where(ids >= 0, ids, table[seqs])
    lens[seqs] += torch.where(granted, st["n_new"], 0)
    seq = seqs[st["entry"]]
    pos = (lens[seq] - st["n_new"][st["entry"]]).long() + st["offset"]
    page, slot = table[seq, pos // S].long(), pos % S
    st["k"].permute(1, 3, 0, 2, 4)[page, slot] = st["k_new"].permute(1, 0, 2, 3)
    st["v"].permute(1, 3, 0, 2, 4)[page, slot] = st["v_new"].permute(1, 0, 2, 3)
    return {"granted": granted.int(), "page_table": table, "seq_lens": lens, "ref_counts": refs, "k": st["k"], "v": st["v"]}


def _plain_fork(st):
    case, S = st["case"], st["case"]["page"]
    table, refs, lens = st["page_table"], st["ref_counts"], st["seq_lens"]
    _plain_free(st, st["children"], torch.zeros_like(st["children"]))
    par, kid = st["parents"].long(), st["children"].long()
    n = lens[par]
    full, held = n // S, (n + S - 1) // S
    shared = torch.zeros_like(full) if case["copy"] else full   # pages the child shares; the rest it gets copies of
    granted, ids = _plain_take(st, shared, held - shared)
    col = torch.arange(table.shape[1], device="cuda")
    rows = torch.where((col < shared[:, None]) & granted[:, None], table[par], ids)
    refs.index_add_(0, rows.clamp(min=0).reshape(-1).long(), (rows >= 0).reshape(-1).int())
    table[kid] = rows
    lens[kid] = torch.where(granted, n, 0)
    # copied: the slots that hold a token of the parent
    pos = col[:, None] * S + torch.arange(S, device="cuda")
    i, c, slot = torch.nonzero((ids >= 0)[:, :, None] & (pos < n[:, None, None]), as_tuple=True)
    src, dst = table[par[i], c].long(), ids[i, c].long()
    for_k, for_v = st["k"].permute(1, 3, 0, 2, 4), st["v"].permute(1, 3, 0, 2, 4)
    for_k[dst, slot] = for_k[src, slot]
    for_v[dst, slot] = for_v[src, slot]
    return {"granted": granted.int(), "page_table": table, "seq_lens": lens, "ref_counts": refs, "k": st["k"], "v": st["v"]}


def _plain_compact(st):
    table, refs = st["page_table"], st["ref_counts"]
    live = refs > 0
    n_live = live.sum()
    page = torch.arange(refs.numel(), device="cuda")
    holes, strays = page[~live & (page < n_live)], page[live & (page >= n_live)]
    to = page.clone()
    to[strays] = holes
    st["k"][:, holes] = st["k"][:, strays]
    st["v"][:, holes] = st["v"][:, strays]
    out = torch.where(table >= 0, to[table.clamp(min=0).long()].int(), -1)
    new_refs = torch.zeros_like(refs)
    new_refs[to[live]] = refs[live]
    return {"page_table": out, "ref_counts": new_refs, "n_live": n_live.int().reshape(1), "k": st["k"], "v": st["v"]}


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def _own_attend(st):
    o, lse = st["eta"].attn_paged_fwd(st["q"], st["cache"], 0, st["seqs"], st["q_start"], max_q=st["max_q"],
                                      causal=st["case"]["causal"])
    return {"o": o, "lse": lse}


def _own_grow(st):
    eta, cache = st["eta"], st["cache"]
    eta.attn_cache_free(cache, st["seqs"], st["keep"])
    granted = eta.attn_cache_reserve(cache, st["seqs"], st["n_new"])
    for layer in range(st["case"]["layers"]):
        eta.attn_cache_append(cache, layer, st["k_new"][layer], st["v_new"][layer], st["seqs"], st["q_start"])
    return {"granted": granted, "page_table": st["page_table"], "seq_lens": st["seq_lens"],
            "ref_counts": st["ref_counts"], "k": st["k"], "v": st["v"]}


def _own_fork(st):
    eta, cache = st["eta"], st["cache"]
    eta.attn_cache_free(cache, st["children"])
    granted = eta.attn_cache_fork(cache, st["parents"], st["children"], copy=st["case"]["copy"])
    return {"granted": granted, "page_table": st["page_table"], "seq_lens": st["seq_lens"],
            "ref_counts": st["ref_counts"], "k": st["k"], "v": st["v"]}


def _own_compact(st):
    # new tables: a step in flight may go on reading the old ones, whose pages keep their contents
    table, refs, n_live = st["eta"].attn_cache_compact(st["cache"], inplace=False)
    return {"page_table": table, "ref_counts": refs, "n_live": n_live, "k": st["k"], "v": st["v"]}


def run(state):
    kind = state["case"]["kind"]
    if own:
        return {"attend": _own_attend, "grow": _own_grow, "fork": _own_fork, "compact": _own_compact}[kind](state)
    return {"attend": _plain_attend, "grow": _plain_grow, "fork": _plain_fork, "compact": _plain_compact}[kind](state)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    ctx, new = _lens(case)
    H, S, d = case["heads"], case["page"], case["d"]
    es = 2 if case["dtype"] == "bf16" else 4
    if case["kind"] == "attend":
        g = case["group"]
        lens = [a + b for a, b in zip(ctx, new)]
        pairs = sum(b * a + b * (b + 1) // 2 if case["causal"] else b * (a + b) for a, b in zip(ctx, new))
        rows = sum(new) * H * g
        byts = 2 * sum(lens) * H * d * es + 2 * rows * d * es + rows * 4 + sum(_ceil(n, S) for n in lens) * 4
        return {"bytes": byts, "flops": 4 * pairs * H * g * d}
    token = 2 * case["layers"] * H * d * es      # K and V of one token in every layer
    if case["kind"] == "grow":
        cut = _cut(case)
        pages = sum(_ceil(c - x + b, S) - _ceil(c - x, S) for c, x, b in zip(ctx, cut, new))
        return {"bytes": 2 * sum(new) * token + 3 * 4 * pages + 6 * 4 * len(ctx), "flops": 0}
    if case["kind"] == "fork":
        rng = random.Random(case["ragged"] + 2)
        which = [rng.randrange(case["parents"]) for _ in range(case["forks"])]
        moved = sum(ctx[w] if case["copy"] else ctx[w] % S for w in which)
        entries = sum(_ceil(ctx[w], S) for w in which)
        return {"bytes": 2 * moved * token + 4 * 4 * entries, "flops": 0}
    used = sum(_ceil(n, S) for n in ctx)
    pages = used + max(1, int(used * case["spare"]))
    # on average a live page lies past the last place that is kept with this probability
    moved = int(used * (pages - used) / pages)
    return {"bytes": 2 * moved * S * token + 2 * 4 * pages + 2 * 4 * used, "flops": 0}


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    """Attention by its definition, sequence by sequence and head by head, in
    float64.  The other operators only move values, so they have no computed
    numbers."""
    if case["kind"] != "attend":
        return None
    st = prepare(case, seed)
    S, Hk, g, d = case["page"], case["heads"], case["group"], case["d"]
    starts, table = st["q_start"].tolist(), st["page_table"].tolist()
    outs, lses = [], []
    for i, row in enumerate(st["seqs"].tolist()):
        n = int(st["seq_lens"][row])
        a, b = starts[i], starts[i + 1]
        ids = torch.tensor(table[row][:_ceil(n, S)], device="cuda")
        heads_o, heads_l = [], []
        for h in range(Hk):
            k = st["k"][0, ids, h].reshape(-1, d)[:n].double()
            v = st["v"][0, ids, h].reshape(-1, d)[:n].double()
            for j in range(g):
                s = st["q"][a:b, h * g + j].double() @ k.T / d ** 0.5
                if case["causal"]:
                    last = torch.arange(n - (b - a), n, device="cuda")
                    s.masked_fill_(torch.arange(n, device="cuda")[None] > last[:, None], -math.inf)
                w = torch.logsumexp(s, dim=1)
                heads_o.append(torch.exp(s - w[:, None]) @ v)
                heads_l.append(w)
        outs.append(torch.stack(heads_o, 1))
        lses.append(torch.stack(heads_l, 1))
    return {"o": torch.cat(outs), "lse": torch.cat(lses)}
