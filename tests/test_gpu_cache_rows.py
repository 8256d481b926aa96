"""Rows in and out of a paged cache on the GPU: the rotated append, appending to
a cache of 4-bit values, and reading back.  Results are compared bit by bit: the
rotation with its definition in float32 (every product and sum rounded once, as
the CPU does it), the 4-bit format with its definition in exact numbers."""
import math
import random

import pytest
import torch

from e2m1_ref import angles, build4, ints, quantize, rows_of, starts, turned, values
from test_gpu_paged import build

pytestmark = pytest.mark.gpu
BF16, F32, E2M1 = torch.bfloat16, torch.float32, torch.float4_e2m1fn_x2


@pytest.fixture(scope="module")
def eta():
    import exact_tiled_attention_17_gb300 as m
    return m


def cache_of(eta, store, lens, heads, page, d, layout="head", layers=1, seed=0):
    if store == E2M1:
        return build4(eta, lens, heads, page, d, layers, seed=seed)[0]
    return build(eta, lens, heads, page, d, store, layout, layers, seed=seed)


def rows(T, heads, d, dtype, seed, size=1.0):
    g = torch.Generator().manual_seed(seed)
    return (size * torch.randn((T, heads, d), generator=g)).to(dtype).cuda()


def held(cache, layer, row, first, n):
    """Rows of the cache as they lie there: [n, heads, d], or (4-bit) codes and scales."""
    table = cache.page_table[row].cpu().long()
    t = torch.arange(first, first + n)
    id_, slot = table[t // cache.page_size], t % cache.page_size
    if cache.k.dtype == torch.uint8:
        return [tuple(p[layer].cpu()[id_, :, slot] for p in cache.parts(pool)) for pool in (cache.k, cache.v)]
    return [pool[layer].cpu()[id_, :, slot] for pool in (cache.k, cache.v)]


def same(got, want, what):
    """Equal bit by bit (NaN and the sign of zero included)."""
    assert got.dtype == want.dtype and got.shape == want.shape, what
    n = {1: torch.uint8, 2: torch.int16, 4: torch.int32}[got.element_size()]
    assert torch.equal(got.contiguous().view(n), want.contiguous().view(n)), f"{what}: {(got != want).sum()} of {got.numel()} differ"


def check_append(eta, cache, lens, new, seqs, dims, neighbours, Hq, layer=0, before=0, behind=0, positions=None, top=None, seed=0,
                 fused=False, in_place=False, size=1.0):
    """Appends the sequences' last tokens and looks at every row of the cache and of q."""
    T = sum(new) + before + behind
    H, d, dt = cache.heads, cache.d, cache.dtype
    if fused:      # the rows of one projection
        x = rows(T, Hq + 2 * H, d, dt, seed + 1, size)
        q, k, v = x.split([Hq, H, H], 1) if Hq else (None, *x.split([H, H], 1))
    else:
        q, k, v = rows(T, max(Hq, 1), d, dt, seed + 1, size) if Hq else None, rows(T, H, d, dt, seed + 2, size), rows(T, H, d, dt, seed + 3, size)
    table = angles(top or max(lens) + 1, dims)
    qs = ints(starts(new, before))
    first = {}
    pos = torch.zeros(T, dtype=torch.long)
    for i, r in enumerate(seqs):
        a = int(qs[i])
        pos[a:a + new[i]] = torch.arange(lens[r] - new[i], lens[r])
        first[r] = a
    if positions is not None:
        pos = positions.cpu().long()
    q_in = None if q is None else q.clone()
    pools = cache.k.clone(), cache.v.clone()
    out = q if in_place else (None if q is None else torch.full_like(q.contiguous(), 7.0))
    got = eta.attn_cache_append_rotated(cache, layer, k, v, ints(seqs), qs, table, q=q, q_out=out, neighbours=neighbours,
                                        positions=positions)
    torch.cuda.synchronize()
    assert eta.attn_status() == eta.ATTN_OK
    tk, tv = turned(k, table, pos, neighbours), v.cpu().float()
    untouched = torch.zeros(cache.pages, cache.page_size, dtype=torch.bool)
    for i, r in enumerate(seqs):
        a, n = int(qs[i]), new[i]
        for name, x, g in zip("kv", (tk, tv), held(cache, layer, r, lens[r] - n, n)):
            if cache.k.dtype == torch.uint8:
                for part, w, s in zip(g, quantize(x[a:a + n]), ("codes", "scales")):
                    same(part, w, f"{s} of {name}, entry {i}")
            else:
                same(g, x[a:a + n].to(dt), f"{name}, entry {i}")
        table_r = cache.page_table[r].cpu().long()
        t = torch.arange(lens[r] - n, lens[r])
        untouched[table_r[t // cache.page_size], t % cache.page_size] = True
    # nothing else was written
    for pool, was in zip((cache.k, cache.v), pools):
        if cache.k.dtype == torch.uint8:
            for a, b in zip(cache.parts(pool), cache.parts(was)):
                a, b = a.clone(), b.clone()
                for x in (a, b):
                    x.transpose(2, 3)[layer][untouched.cuda()] = 0
                assert torch.equal(a, b), "other slots were written"
        else:
            a, b = pool.clone(), was.clone()
            for x in (a, b):
                x.transpose(2, 3)[layer][untouched.cuda()] = 0
            same(a.cpu(), b.cpu(), "other slots")
    if q is None:
        assert got is None
        return
    want = turned(q_in, table, pos, neighbours).to(dt)
    here = torch.zeros(T, dtype=torch.bool)
    for i in range(len(seqs)):
        here[int(qs[i]):int(qs[i + 1])] = True
    same(got.cpu()[here], want[here], "q")
    rest = q_in.cpu() if in_place else torch.full_like(q_in, 7.0).cpu()
    same(got.cpu()[~here], rest[~here], "rows of q of no entry")


@pytest.mark.parametrize("neighbours", [False, True])
@pytest.mark.parametrize("store,heads,Hq,d,dims,page,layout", [
    (BF16, 2, 8, 128, 128, 16, "head"), (BF16, 1, 3, 64, 32, 32, "token"), (BF16, 3, 3, 96, 72, 64, "head"),
    (BF16, 2, 2, 32, 8, 128, "token"), (BF16, 1, 1, 128, 2, 256, "side"), (BF16, 2, 10, 64, 48, 16, "layers"),
    (BF16, 5, 0, 96, 96, 16, "head"), (F32, 2, 4, 128, 128, 16, "head"), (F32, 1, 5, 64, 16, 32, "token"),
    (F32, 3, 6, 96, 24, 64, "side"), (F32, 1, 0, 32, 32, 128, "layers"), (F32, 4, 4, 64, 30, 16, "head"),
    (E2M1, 2, 8, 128, 128, 16, "head"), (E2M1, 1, 3, 64, 64, 32, "head"), (E2M1, 3, 3, 96, 96, 64, "head"),
    (E2M1, 2, 2, 32, 32, 128, "head"), (E2M1, 1, 4, 128, 96, 256, "head"), (E2M1, 2, 0, 64, 16, 16, "head"),
    (E2M1, 8, 1, 96, 72, 32, "head"), (E2M1, 1, 7, 128, 6, 16, "head"), (E2M1, 3, 6, 32, 24, 64, "head"),
])
def test_rotated_append(eta, neighbours, store, heads, Hq, d, dims, page, layout):
    lens, new, seqs = [40, 1, 200, 129, 7, 16], [17, 1, 0, 129, 3], [0, 1, 2, 3, 4]
    cache = cache_of(eta, store, lens, heads, page, d, layout, layers=2, seed=d + dims)
    check_append(eta, cache, lens, new, seqs, dims, neighbours, Hq, layer=1, before=1, behind=2, seed=d, fused=True)


@pytest.mark.parametrize("store", [BF16, F32, E2M1])
@pytest.mark.parametrize("d", [32, 64, 96, 128])
def test_every_width_of_halves(eta, store, d):
    """Halves of an odd number of 8 columns meet inside a group of 16 that shares a scale."""
    lens, new, seqs = [40, 700, 650], [20, 640, 3], [0, 1, 2]
    for dims in range(16, d + 1, 16):
        cache = cache_of(eta, store, lens, 2, 32, d, "head", seed=dims)
        check_append(eta, cache, lens, new, seqs, dims, False, 3, seed=d + dims, fused=True)
        check_append(eta, cache, lens, new, seqs, dims, False, 3, seed=d + dims + 1, in_place=True)


@pytest.mark.parametrize("store", [BF16, F32, E2M1])
@pytest.mark.parametrize("dims,neighbours", [(64, False), (48, False), (64, True), (20, True), (26, False)])
def test_in_place_and_placed(eta, store, dims, neighbours):
    """Queries turned in place, positions of their own (far ones, one twice), a table row order of entries."""
    lens, new, seqs = [33, 90, 5], [5, 40, 2], [2, 0, 1]
    lens2 = [lens[r] for r in range(3)]
    new = [2, 20, 40]
    cache = cache_of(eta, store, lens2, 2, 16, 64, seed=dims)
    T = sum(new)
    g = torch.Generator().manual_seed(dims)
    positions = torch.randint(0, 100000, (T,), generator=g).int().cuda()
    positions[1] = positions[0]
    check_append(eta, cache, lens2, new, seqs, dims, neighbours, 4, positions=positions, top=100000, seed=3, in_place=True)
    check_append(eta, cache, lens2, new, seqs, dims, neighbours, 4, positions=positions, top=100000, seed=4, in_place=True, fused=True)


@pytest.mark.parametrize("store", [BF16, E2M1])
@pytest.mark.parametrize("n", [1, 64, 4100])
def test_many_tokens_and_entries(eta, store, n):
    """One token each of many sequences, and more tokens than the few-token variant takes."""
    rng = random.Random(n)
    if n < 4000:
        lens = [rng.randint(1, 50) for _ in range(n)]
        new, seqs = [1] * n, rng.sample(range(n), n)
    else:
        lens, new, seqs = [n - 600, 600, 7], [n - 700, 600, 0], [0, 1, 2]
    cache = cache_of(eta, store, lens, 2, 16, 64, seed=n)
    check_append(eta, cache, lens, new, seqs, 64, False, 2, seed=n)


@pytest.mark.parametrize("size", [1e-6, 1e-4, 1.0, 300.0, 2e4, 1e30])
def test_format_over_the_range(eta, size):
    """Small numbers (scales below 2^-14, groups that become 0), ordinary, and ones that are cut to 61440."""
    cache = build4(eta, [64], 2, 16, 128)[0]
    check_append(eta, cache, [64], [64], [0], 128, False, 0, seed=int(math.log10(size)) + 9, size=size)
    k = rows(64, 2, 128, BF16, 5, size)
    eta.attn_cache_append(cache, 0, k, k, None, ints([0, 64]))
    for g in held(cache, 0, 0, 0, 64):
        for part, want in zip(g, quantize(k.cpu().float())):
            same(part, want, "plain append")


def test_borders_zeros_and_nan(eta):
    """Every border between two codes (ties to even), zeros of both signs, groups with a NaN or an infinity, the
    largest bfloat16: through the append without a rotation."""
    d = 64
    steps = torch.tensor([0, .25, .5, .75, 1, 1.25, 1.5, 1.75, 2, 2.5, 3, 3.5, 4, 5, 5.5, 6])
    x = torch.zeros(16, 1, d)
    for i in range(16):
        s = 2.0 ** (i - 8) * (1 + i % 8 / 8)
        x[i, 0, :16] = steps * s
        x[i, 0, 16:32] = -steps * s
        x[i, 0, 32:48] = steps.flip(0) * s * 1.0078125
    x[3, 0, 48] = math.nan
    x[4, 0, 50] = math.inf
    x[5, 0, 51] = -math.inf
    x[6, 0, 48:] = 3.3895313892515355e38
    x[7, 0, 48:] = -0.0
    x[8, 0, 48:] = torch.tensor([2.0 ** -18 * 6, 2.0 ** -18 * 3] + [0.0] * 14)
    x[9, 0, 48:] = torch.tensor([2.0 ** -18 * 6.0625, 2.0 ** -18 * -3] + [1e-40] * 14)
    k = x.bfloat16().cuda()
    cache = build4(eta, [16], 1, 16, d)[0]
    eta.attn_cache_append(cache, 0, k, k.flip(2).contiguous(), None, ints([0, 16]))
    torch.cuda.synchronize()
    for g, w in zip(held(cache, 0, 0, 0, 16), (k, k.flip(2))):
        for part, want in zip(g, quantize(w.cpu().float())):
            same(part, want, "codes or scales")
    rk, rv = eta.attn_cache_read(cache, 0, None, ints([0, 16]), 16)
    for got, (c, s) in zip((rk, rv), held(cache, 0, 0, 0, 16)):
        want = values(c, s)
        assert torch.equal(torch.isnan(got).cpu(), torch.isnan(want)) and torch.isnan(want).any()
        assert torch.equal(got.cpu().double().nan_to_num(1), want.nan_to_num(1))
    # what the header promises of a value
    g = k.cpu().double().unflatten(-1, (-1, 16))
    fine = torch.isfinite(g).all(-1)
    top = g.abs().amax(-1)
    off = (rk.cpu().double().unflatten(-1, (-1, 16)) - g).abs().amax(-1)
    small = fine & (top <= 61440)
    assert (off[small] <= 0.18 * top[small] + 2.0 ** -15).all()


@pytest.mark.parametrize("store,layout", [(BF16, "head"), (BF16, "token"), (BF16, "side"), (F32, "layers"), (F32, "token"), (E2M1, "head")])
@pytest.mark.parametrize("d,page", [(32, 16), (64, 256), (96, 32), (128, 64)])
def test_read(eta, store, layout, d, page):
    """Last tokens, given ranges, a sequence twice, empty entries, rows of no entry; strided outputs."""
    lens = [70, 1, 300, 33]
    cache = cache_of(eta, store, lens, 3, page, d, layout, layers=2, seed=d)
    cases = [([0, 1, 2, 3], [70, 1, 300, 33], None), ([2, 2, 0], [5, 300, 0], None), ([3, 2, 2, 0], [33, 7, 1, 4], [0, 290, 299, 60])]
    for seqs, new, first in cases:
        T = sum(new) + 3
        q_start = starts(new, 2)
        big = torch.full((T, 2, 5, d), 7.0, dtype=cache.dtype, device="cuda")
        k, v = big[:, 0, 1:4], big[:, 1, 1:4]
        f = None if first is None else ints(first)
        got = eta.attn_cache_read(cache, 1, ints(seqs), ints(q_start), k_out=k, v_out=v, first=f)
        torch.cuda.synchronize()
        assert eta.attn_status() == eta.ATTN_OK and got[0] is k
        rest = torch.full((T, 2, 5, d), 7.0, dtype=cache.dtype)
        for i, r in enumerate(seqs):
            a = lens[r] - new[i] if first is None else first[i]
            if store == E2M1:
                want = rows_of(cache, 1, r, a, new[i])
            else:
                want = held(cache, 1, r, a, new[i])
            for j, w in enumerate(want):
                rest[q_start[i]:q_start[i + 1], j, 1:4] = w.to(cache.dtype)
        assert torch.equal(big.cpu(), rest)
        if first is None:
            k2, v2 = eta.attn_cache_read(cache, 1, ints(seqs), ints(q_start), T)
            here = slice(q_start[0], q_start[-1])
            assert torch.equal(k2.cpu()[here], rest[here, 0, 1:4]) and torch.equal(v2.cpu()[here], rest[here, 1, 1:4])


@pytest.mark.parametrize("store", [BF16, F32, E2M1])
def test_what_is_left_out(eta, store):
    """Rows that go nowhere: bad rows of the table, bad ranges, sequences named twice, no room, shared pages, positions
    outside the table, more new tokens than the sequence has.  Nothing of theirs is written, q included."""
    lens = [40, 20, 33, 16, 5]
    heads, d, page = 2, 64, 16
    g = torch.Generator().manual_seed(1)

    def run(seqs, q_start, T, expect, granted=None, positions=None, break_=None, rows_of_table=64, status=None):
        cache = cache_of(eta, store, lens, heads, page, d, seed=7)
        if break_:
            break_(cache)
        x = torch.randn((T, 6, d), generator=g).to(cache.dtype).cuda()
        q, k, v = x[:, :2], x[:, 2:4], x[:, 4:6]
        table = angles(rows_of_table, 64)
        was = cache.k.clone(), cache.v.clone()
        out = torch.full((T, 2, d), 7.0, dtype=cache.dtype, device="cuda")
        eta.attn_status()
        eta.attn_cache_append_rotated(cache, 0, k, v, ints(seqs), ints(q_start), table, q=q, q_out=out, positions=positions,
                                      granted=None if granted is None else ints(granted))
        rc = eta.attn_status()
        assert rc == (eta.ATTN_ERR_ARG if status is None else status)
        written = torch.zeros(T, dtype=torch.bool)
        written[expect] = True
        assert torch.equal((out != 7.0).flatten(1).any(1).cpu(), written)
        n_slots = 0
        for pool, w in zip((cache.k, cache.v), was):
            n = {1: torch.uint8, 2: torch.int16, 4: torch.int32}[pool.element_size()]
            if pool.dtype == torch.uint8:
                diff = [(a != b).any(-1) for a, b in zip(cache.parts(pool), cache.parts(w))]
                diff = (diff[0] | diff[1])
            else:
                diff = (pool.view(n) != w.view(n)).any(-1)
            n_slots += int(diff.any(2).sum())
        assert n_slots == 2 * len(expect)

    run([0, 9, 1], [0, 2, 4, 6], 6, [0, 1, 4, 5])                    # no such sequence
    run([0, -1], [0, 2, 4], 4, [0, 1])
    run([0, 1, 0], [0, 2, 4, 6], 6, [0, 1, 2, 3])                    # named twice: the first counts
    run([0, 1], [0, 2, 9], 4, [0, 1])                                # a range past the rows
    run([4, 1], [0, 7, 9], 9, [2, 3, 4, 5, 6, 7, 8])                 # more tokens than the sequence has
    run([0, 1], [0, 2, 4], 4, [2, 3], granted=[0, 1], status=0)      # no room, and said so
    run([0, 1], [0, 2, 4], 4, [0, 1], positions=ints([3, 63, 64, -1]))   # positions outside the table
    run([0, 1], [0, 3, 4], 4, [3], rows_of_table=37)                 # tokens past the table's rows

    def share(c):
        c.ref_counts[c.page_table[0, 2]] = 2
    run([0, 1], [0, 2, 4], 4, [2, 3], break_=share)

    def lose(c):
        c.page_table[0, 2] = c.pages
    run([0, 1], [0, 2, 4], 4, [2, 3], break_=lose)

    # reading: what is not there stays
    cache = cache_of(eta, store, lens, heads, page, d, seed=7)
    cache.page_table[0, 1] = -1
    k, v = (torch.full((20, heads, d), 7.0, dtype=cache.dtype, device="cuda") for _ in range(2))
    eta.attn_status()
    eta.attn_cache_read(cache, 0, ints([0, 9, 1, 4, 3]), ints([0, 4, 6, 10, 14, 16]), first=ints([14, 0, 17, -1, 0]), k_out=k, v_out=v)
    assert eta.attn_status() == eta.ATTN_ERR_ARG
    written = [bool((k[t] != 7.0).any()) for t in range(20)]
    # 14, 15 of sequence 0 and not 16, 17 (page missing); 17 .. 19 of 1 and not 20; none from -1; 0, 1 of 3
    assert written == [True, True, False, False] + [False] * 2 + [True] * 3 + [False] + [False] * 4 + [True] * 2 + [False] * 4


@pytest.mark.parametrize("store", [BF16, E2M1])
def test_streams_graphs_and_empty_calls(eta, store):
    """A call on a stream of its own, a captured one replayed after the lengths changed, and calls without work."""
    lens = [20, 33]
    cache = cache_of(eta, store, lens, 2, 16, 64, seed=2)
    table = angles(64, 64)
    k, v, q = rows(2, 2, 64, BF16, 1), rows(2, 2, 64, BF16, 2), rows(2, 4, 64, BF16, 3)
    qs, seqs = ints([0, 1, 2]), ints([0, 1])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    a = eta.attn_cache_append_rotated(cache, 0, k, v, seqs, qs, table, q=q, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    want = turned(q, table, torch.tensor([19, 32]), False).bfloat16()
    same(a.cpu(), want, "side stream")
    graph = torch.cuda.CUDAGraph()
    out, rk, rv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    with torch.cuda.graph(graph):
        eta.attn_cache_append_rotated(cache, 0, k, v, seqs, qs, table, q=q, q_out=out)
        eta.attn_cache_read(cache, 0, seqs, qs, k_out=rk, v_out=rv)
    cache.seq_lens.copy_(ints([18, 30]))
    graph.replay()
    torch.cuda.synchronize()
    same(out.cpu(), turned(q, table, torch.tensor([17, 29]), False).bfloat16(), "replayed")
    back = turned(k, table, torch.tensor([17, 29]), False)
    want = values(*quantize(back)).bfloat16() if store == E2M1 else back.bfloat16()
    same(rk.cpu(), want, "read back")
    empty = torch.empty((0, 2, 64), dtype=BF16, device="cuda")
    eta.attn_cache_append_rotated(cache, 0, empty, empty, None, ints([0]), table)
    kr, _ = eta.attn_cache_read(cache, 0, None, ints([0]), 0)
    assert kr.shape == (0, 2, 64)
    torch.cuda.synchronize()
    assert eta.attn_status() == eta.ATTN_OK


def test_python_refusals(eta):
    cache = cache_of(eta, E2M1, [20], 2, 16, 64)
    k = rows(2, 2, 64, BF16, 1)
    q = rows(2, 4, 64, BF16, 1)
    table, qs = angles(32, 64), ints([0, 2])
    call = eta.attn_cache_append_rotated
    for bad in (dict(table=table.double()), dict(table=table[:, ::2]), dict(table=table[0]), dict(table=table.cpu()), dict(q=q.float()),
                dict(q=q[:1]), dict(q=q[..., :32]), dict(q=q, q_out=q[:, :2]), dict(q_out=q), dict(positions=ints([1])),
                dict(positions=torch.zeros(2, device="cuda")), dict(granted=ints([1, 1])), dict(k_new=k.float(), v_new=k.float()),
                dict(k_new=k[:, :1], v_new=k[:, :1])):
        a = dict(k_new=k, v_new=k, seqs=None, q_start=qs, table=table)
        a.update(bad)
        with pytest.raises(ValueError):
            call(cache, 0, **a)
    with pytest.raises(eta.AttnError):
        call(cache, 0, k, k, None, qs, angles(32, 66)[:, :66].contiguous())     # more columns than a row has
    with pytest.raises(eta.AttnError):
        call(cache, 1, k, k, None, qs, table)                                   # no such layer
    with pytest.raises(eta.AttnError):
        call(cache, 0, k, k, None, qs, table, q=q, q_out=q.expand(2, 4, 64)[:, :1].expand(2, 4, 64))   # rows that overlap
    with pytest.raises(ValueError):
        eta.attn_cache_read(cache, 0, None, qs)
    with pytest.raises(ValueError):
        eta.attn_cache_read(cache, 0, None, qs, 3, k_out=k, v_out=k)
    with pytest.raises(ValueError):
        eta.attn_cache_read(cache, 0, None, qs, 2, k_out=k)
    with pytest.raises(eta.AttnError):
        eta.attn_cache_read(cache, 0, None, qs, k_out=k, v_out=k)               # one memory for both
    with pytest.raises(ValueError):
        eta.PagedCache(cache.k[..., :-1], cache.v[..., :-1], cache.page_table, cache.seq_lens, cache.ref_counts)
    with pytest.raises(ValueError):
        eta.PagedCache.empty(1, 4, 2, 16, 64, 2, 4, dtype=E2M1, token_major=True)
    with pytest.raises(ValueError):
        cache_of(eta, BF16, [20], 2, 16, 64).parts(cache.k)
    assert eta.attn_status() == eta.ATTN_OK


@pytest.mark.parametrize("store", [BF16, F32, E2M1])
def test_more_entries_than_few(eta, store):
    """More tokens than the few-token variants take, one or two to an entry, entries in another order than the table."""
    rng = random.Random(5)
    n, heads, d = 1100, 2, 64
    lens = [rng.randint(2, 20) for _ in range(n)]
    seqs, new = rng.sample(range(n), n), [rng.randint(0, 2) for _ in range(n)]
    cache = cache_of(eta, store, lens, heads, 16, d, seed=3)
    T, at = sum(new), starts(new)
    q, k, v = (rows(T, h, d, cache.dtype, 7 + h) for h in (4, heads, heads))
    table = angles(32, d)
    pos = torch.cat([torch.arange(lens[r] - m, lens[r]) for r, m in zip(seqs, new)])
    out = eta.attn_cache_append_rotated(cache, 0, k, v, ints(seqs), ints(at), table, q=q)
    rk, rv = eta.attn_cache_read(cache, 0, ints(seqs), ints(at), T)
    torch.cuda.synchronize()
    assert eta.attn_status() == eta.ATTN_OK
    same(out.cpu(), turned(q, table, pos, False).to(cache.dtype), "q")
    for got, x in ((rk, turned(k, table, pos, False)), (rv, v.cpu().float())):
        same(got.cpu(), (values(*quantize(x)) if store == E2M1 else x).to(cache.dtype), "read back")


def test_far_into_a_large_pool(eta):
    """Pages that lie more than 2^32 bytes into their pool: written, read and attended to."""
    heads, page, d = 8, 64, 128
    pages = 120000     # 4.4 GB a pool
    cache = eta.PagedCache.empty(1, pages, heads, page, d, 2, 4, dtype=E2M1)
    ids = [pages - 1, 3, pages - 2]
    cache.page_table[1, :3] = ints(ids)
    cache.ref_counts[ids] = 1
    cache.seq_lens[1] = 150
    for pool in (cache.k, cache.v):
        for i in ids:
            pool[0, i].fill_(255)
    k, v, q = rows(150, heads, d, BF16, 1), rows(150, heads, d, BF16, 2), rows(150, heads, d, BF16, 3)
    table = angles(150, d)
    qs = ints([0, 150])
    qr = eta.attn_cache_append_rotated(cache, 0, k, v, ints([1]), qs, table, q=q)
    rk, rv = eta.attn_cache_read(cache, 0, ints([1]), qs, 150)
    pos = torch.arange(150)
    want_k, want_v = values(*quantize(turned(k, table, pos, False))), values(*quantize(v.cpu().float()))
    same(rk.cpu(), want_k.bfloat16(), "k")
    same(rv.cpu(), want_v.bfloat16(), "v")
    for n, max_q in ((150, 150), (1, 1)):
        o, _ = eta.attn_paged_fwd(qr[150 - n:].contiguous(), cache, 0, ints([1]), ints([0, n]), max_q=max_q)
        s = torch.einsum("hd,nhd->hn", qr[149].cpu().double(), want_k) / math.sqrt(d)
        w = torch.softmax(s, 1)
        want, size = torch.einsum("hn,nhd->hd", w, want_v), torch.einsum("hn,nhd->hd", w, want_v.abs())
        assert ((o[-1].cpu().double() - want).abs() <= 2.0 ** -8 * (want.abs() + size) * 1.05).all()
    assert eta.attn_status() == eta.ATTN_OK


def test_threads_share_a_cache(eta):
    """Two threads that append to and read different sequences of one cache, each on a stream of its own."""
    import threading
    lens = [400, 400]
    cache = cache_of(eta, E2M1, lens, 2, 16, 64, seed=9)
    table = angles(400, 64)
    failed = []

    def work(r):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                k, v, q = (rows(400, h, 64, BF16, 10 * r + h) for h in (2, 2, 4))
                v = v + r
                for i in range(30):
                    got = eta.attn_cache_append_rotated(cache, 0, k, v, ints([r]), ints([0, 400]), table, q=q)
                    rk, rv = eta.attn_cache_read(cache, 0, ints([r]), ints([0, 400]), 400)
                    stream.synchronize()
                    want = turned(k, table, torch.arange(400), False)
                    same(rk.cpu(), values(*quantize(want)).bfloat16(), "k")
                    same(rv.cpu(), values(*quantize(v.cpu().float())).bfloat16(), "v")
                    same(got.cpu(), turned(q, table, torch.arange(400), False).bfloat16(), "q")
        except Exception as e:   # noqa: BLE001 (told to the test below)
            failed.append(e)
    threads = [threading.Thread(target=work, args=(r,)) for r in (0, 1)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed[0]
    assert eta.attn_status() == eta.ATTN_OK
