"""Plain references for the cache of 4-bit values and the rotated append (not
collected by pytest).  Everything on the CPU, in float64 unless said otherwise."""
import math
import random
from types import SimpleNamespace

import torch

from paged_ref import attention, gather

STEPS = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)
# every finite scale that is written, by its byte: bits 14 .. 7 of a float16, up to 10240
SCALES = (torch.arange(0xE3, dtype=torch.int16) << 7).view(torch.float16).double()


def _nearest(x, grid):
    """Index of the nearest value of an increasing grid, the even one of two at the same distance."""
    hi = torch.searchsorted(grid, x).clamp(1, grid.numel() - 1)
    a, b = x - grid[hi - 1], grid[hi] - x
    return torch.where((b < a) | ((b == a) & (hi % 2 == 0)), hi, hi - 1)


def quantize(x):
    """Rows [..., d] (exact numbers) to codes [..., d / 2] and scales [..., d / 16], uint8.

    float64 decides every case right: amax / 6 and x / scale are quotients of
    float32 numbers by numbers of few bits, so one that is not on a border is at
    least 2^-26 of itself away from it, and one that is on it is exact."""
    g = x.double().unflatten(-1, (-1, 16))
    bad = ~torch.isfinite(g).all(-1)
    top = torch.where(bad, 0.0, g.abs().nan_to_num(0, 0, 0).amax(-1))
    s = _nearest(torch.minimum(top / torch.full_like(top, 6), SCALES[-1]), SCALES)
    scale = SCALES[s][..., None]
    a = torch.where((scale > 0) & ~bad[..., None], g.abs() / scale, 0.0).clamp(max=6.0)
    code = _nearest(a, STEPS)
    code = torch.where(torch.signbit(g) & (scale > 0) & ~bad[..., None], code + 8, code).flatten(-2).to(torch.uint8)
    return code[..., 0::2] | (code[..., 1::2] << 4), torch.where(bad, 255, s).to(torch.uint8)


def values(codes, scales):
    """What codes and scales stand for, float64 (exact)."""
    n = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).long()
    x = torch.where(n >= 8, -STEPS[n & 7], STEPS[n & 7])
    s = (scales.to(torch.int16) << 7).view(torch.float16).double()
    return (x.unflatten(-1, (-1, 16)) * s[..., None]).flatten(-2)


def turned(x, table, pos, neighbours):
    """Rows [T, heads, d] turned, in float32 step by step (the definition), float32."""
    dims = table.shape[1]
    row = table.cpu()[pos.cpu().long()][:, None]
    c, s = row[..., :dims // 2], row[..., dims // 2:]
    x = x.cpu().float().clone()
    if neighbours:
        a, b = x[..., 0:dims:2].clone(), x[..., 1:dims:2].clone()
        x[..., 0:dims:2], x[..., 1:dims:2] = a * c - b * s, b * c + a * s
    else:
        a, b = x[..., :dims // 2].clone(), x[..., dims // 2:dims].clone()
        x[..., :dims // 2], x[..., dims // 2:dims] = a * c - b * s, b * c + a * s
    return x


def angles(rows, dims, seed=0):
    """A table of cosines and sines of the usual angles."""
    t = torch.arange(rows, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(dims // 2, dtype=torch.float64) / (dims // 2))
    return torch.cat([t.cos(), t.sin()], 1).float().cuda()


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def starts(new, before=0):
    v = [before]
    for n in new:
        v.append(v[-1] + n)
    return v


def place(lens, page, spare, seed, max_pages=None):
    """Sequences on random pages: (table, refs, pages)."""
    rng = random.Random(seed)
    need = [-(-n // page) for n in lens]
    pages = sum(need) + spare
    order = list(range(pages))
    rng.shuffle(order)
    table = torch.full((len(lens), max_pages or max(need + [1]) + 1), -1, dtype=torch.int32)
    refs = torch.zeros(pages, dtype=torch.int32)
    for r in range(len(lens)):
        for c in range(need[r]):
            table[r, c] = order.pop()
            refs[table[r, c]] = 1
    return table, refs, pages


def build4(eta, lens, heads, page, d, layers=1, spare=3, seed=0, size=1.0, max_pages=None, pool=None):
    """A cache of 4-bit values with sequences of the given lengths; every byte
    that holds no token is 255 (a NaN).  Returns it with `held`: what
    paged_ref looks at, the values as numbers."""
    g = torch.Generator().manual_seed(seed)
    table, refs, pages = place(lens, page, spare, seed, max_pages)
    k = torch.full((layers, pages, heads, page, 9 * d // 16), 255, dtype=torch.uint8)
    v = torch.full_like(k, 255)
    held = SimpleNamespace(heads=heads, d=d, page_size=page, pages=pages)
    for name, p in (("k", k), ("v", v)):
        flat = p.flatten(3)
        codes, scales = flat[..., :page * d // 2].unflatten(3, (page, d // 2)), flat[..., page * d // 2:].unflatten(3, (page, d // 16))
        x = torch.full((layers, pages, heads, page, d), math.nan, dtype=torch.float64)
        for r, n in enumerate(lens):
            for c in range(-(-n // page)):
                m = min(page, n - c * page)
                cs, ss = quantize((size * torch.randn((layers, heads, m, d), generator=g)).float())
                id_ = int(table[r, c])
                codes[:, id_, :, :m], scales[:, id_, :, :m] = cs, ss
                x[:, id_, :, :m] = values(cs, ss)
        setattr(held, name, x)
    if pool is not None:
        k, v = pool(k), pool(v)
    else:
        k, v = k.cuda(), v.cuda()
    cache = eta.PagedCache(k, v, table.cuda(), ints(lens), refs.cuda())
    held.page_table, held.seq_lens = table, torch.tensor(lens, dtype=torch.int32)
    return cache, held


def rows_of(cache, layer, row, first, n):
    """K and V of tokens of a sequence of a 4-bit cache as numbers, float64 [n, heads, d]."""
    out = []
    table = cache.page_table[row].cpu().long()
    for pool in (cache.k, cache.v):
        codes, scales = (t[layer].cpu() for t in cache.parts(pool))
        t = torch.arange(first, first + n)
        id_, slot = table[t // cache.page_size], t % cache.page_size
        out.append(values(codes[id_, :, slot], scales[id_, :, slot]))
    return out


def check_attention4(q, held, layer, seqs, q_start, causal, scale, o, lse, untouched):
    """Every row of the list against the definition; the others as `untouched` says.

    The bounds are paged_ref's (a weight rounded once to bf16; here it is float16,
    eight times finer), and one more term: float16 has no numbers below 2^-24.  A
    weight is rounded as p = 2^(s - m + 7), where the reference m is at most the
    row's largest score (it is a maximum of scores, and only ever grows to another),
    so below 2^-14 it is off by 2^-25 at most, while the sum of weights is at least
    2^7 (the largest score's own): O is off by 2^-32 sum |v| more, over the keys that
    are there.  (In a part of the keys the same holds against the part's largest
    score, and parts are joined with weights of at most 1.)  It shows where the
    largest weight's key has a 0 in a column: of 16 values one or two are."""
    ref = attention(q, held, layer, seqs, q_start, causal, scale)
    og, lg = o.cpu().double(), lse.cpu().double()
    rows = seqs.tolist() if seqs is not None else range(q_start.numel() - 1)
    g = q.shape[1] // held.heads
    mass = {}
    for i, row in enumerate(rows):
        _, v, there = gather(held, layer, row, int(held.seq_lens[row]))
        for t in range(int(q_start[i]), int(q_start[i + 1])):
            mass[t] = v[:, there].abs().sum(1).repeat_interleave(g, 0)
    for r in range(q.shape[0]):
        if r not in ref:
            assert torch.equal(og[r], untouched[0][r].cpu().double()), f"row {r} was written"
            assert torch.equal(lg[r], untouched[1][r].cpu().double()), f"LSE of row {r} was written"
            continue
        ro, rl, to, tl = ref[r]
        to = to + 2.0 ** -32 * mass[r] * 1.01
        assert not torch.isnan(og[r]).any() and not torch.isnan(lg[r]).any(), f"NaN in row {r}"
        err = (og[r] - ro).abs()
        assert (err <= to).all(), f"row {r}: off by {(err / to).max():.3g} of the bound"
        inf = torch.isinf(rl)
        assert torch.equal(torch.isinf(lg[r]) & (lg[r] < 0), inf), f"LSE of row {r}"
        assert (og[r][inf] == 0).all()
        assert ((lg[r] - rl).abs()[~inf] <= tl[~inf]).all(), f"LSE of row {r}: {(lg[r] - rl).abs()[~inf].max():.3g}"
