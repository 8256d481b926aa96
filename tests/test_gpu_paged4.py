"""Attention over a paged cache of 4-bit values on the GPU, against the
definition in float64 on the values that the cache holds (bounds derived in
e2m1_ref.py and paged_ref.py), and the page operators on such a cache."""
import math
import random

import pytest
import torch

from e2m1_ref import angles, build4, check_attention4, ints, quantize, rows_of, starts, turned, values
from paged_ref import Pages

pytestmark = pytest.mark.gpu
BF16, E2M1 = torch.bfloat16, torch.float4_e2m1fn_x2


@pytest.fixture(scope="module")
def eta():
    import exact_tiled_attention_17_gb300 as m
    return m


def queries(T, Hq, d, seed=0, size=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed + 99)
    return (size * torch.randn((T, Hq, d), generator=g, device="cuda")).to(BF16)


def attend(eta, cache, held, new, g, seqs=None, causal=True, layer=0, seed=0, before=0, behind=0, size=1.0, max_q=None,
           scale=None, q=None, out=None, status=0, **kw):
    T = sum(new) + before + behind
    Hq = cache.heads * g
    q = queries(T, Hq, cache.d, seed, size) if q is None else q
    o = torch.full((T, Hq, cache.d), 7.0, dtype=BF16, device="cuda") if out is None else out
    lse = torch.full((T, Hq), 7.0, device="cuda")
    was = (o.clone(), lse.clone())
    qs = ints(starts(new, before))
    sq = None if seqs is None else ints(seqs)
    eta.attn_paged_fwd(q, cache, layer, sq, qs, max_q=max_q or max(max(new), 1), causal=causal, scale=scale, out=o, lse=lse, **kw)
    torch.cuda.synchronize()
    assert eta.attn_status() == status
    check_attention4(q, held, layer, sq, qs, causal, scale if scale is not None else 1 / math.sqrt(cache.d), o, lse, was)
    return o, lse


BATCHES = {
    "one": ([1], [1]),
    "decode": ([1, 15, 16, 17, 63, 64, 65, 129, 300], [1] * 9),
    "few": ([5, 200, 33, 64, 7], [5, 3, 2, 1, 4]),
    "chunk": ([40, 200, 129, 90], [40, 77, 129, 1]),
    "empty": ([0, 70, 0, 3, 20], [0, 0, 2, 5, 0]),       # no tokens; more new tokens than the sequence holds
}


@pytest.mark.parametrize("batch", BATCHES)
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("heads,g,d,page", [
    (2, 4, 128, 16), (1, 1, 64, 32), (3, 3, 96, 64), (2, 8, 32, 128), (1, 16, 128, 256), (2, 5, 64, 16), (1, 64, 64, 16),
    (4, 2, 128, 64), (2, 1, 96, 16), (1, 7, 32, 16),
])
def test_attention(eta, batch, causal, heads, g, d, page):
    lens, new = BATCHES[batch]
    cache, held = build4(eta, lens, heads, page, d, layers=2, seed=len(lens))
    attend(eta, cache, held, new, g, causal=causal, layer=1, before=1, behind=2)


@pytest.mark.parametrize("n,new", [(5000, 1), (5000, 4), (4097, 33), (2000, 500), (1023, 1023), (9000, 129)])
def test_long_and_split(eta, n, new):
    """Long axes, which several CTAs share, beside short sequences; large scores."""
    cache, held = build4(eta, [n, 3, n // 3], 2, 16, 64, seed=n)
    attend(eta, cache, held, [new, 1, min(new, n // 3)], 4, seed=n)
    cache, held = build4(eta, [n], 1, 64, 128, seed=n + 1, size=4.0)
    attend(eta, cache, held, [new], 2, seed=n, size=4.0)


@pytest.mark.parametrize("d", [32, 64, 96, 128])
@pytest.mark.parametrize("g,new", [(1, 1), (3, 1), (2, 2), (8, 1), (1, 7), (5, 2), (4, 4), (3, 9), (8, 4), (17, 1), (16, 2), (11, 3),
                                   (6, 5), (9, 3), (13, 2)])
def test_few_rows(eta, d, g, new):
    """Every size of the units for few rows: short lengths, ends inside a tile, entries with less than the most tokens."""
    lens = [1, 700, 2, 15, 33, 0, 64, 65, 5, 1291]
    cache, held = build4(eta, lens, 2, 16 if g < 4 else 128, d, seed=d + g)
    some = [min(n, 1 + (new * i) % (new + 1)) for i, n in enumerate(lens)]
    some[1] = new
    attend(eta, cache, held, some, g, causal=new != 2, before=1, behind=1, seed=g)


@pytest.mark.parametrize("new,g", [(1, 4), (3, 5), (40, 4)])
def test_strides_order_and_granted(eta, new, g):
    """q and o as slices of wider tensors, entries in another order than the table, entries that got no room."""
    lens = [100, 64, 37, 200]
    cache, held = build4(eta, lens, 2, 16, 64, seed=new, max_pages=40)
    T, Hq, d = 3 * new, 2 * g, 64
    wide = queries(T, Hq + 4, d, 5)
    big = torch.full((T, Hq + 3, d), 7.0, dtype=BF16, device="cuda")
    attend(eta, cache, held, [new] * 3, g, seqs=[3, 0, 2], q=wide[:, 2:2 + Hq], out=big[:, 1:1 + Hq])
    assert (big[:, 0] == 7).all() and (big[:, Hq + 1:] == 7).all()
    # heads outside, tokens inside
    q, o = queries(Hq, T, d, 6).transpose(0, 1), torch.full((Hq, T, d), 7.0, dtype=BF16, device="cuda").transpose(0, 1)
    attend(eta, cache, held, [new] * 3, g, seqs=[3, 0, 2], q=q, out=o)
    q = queries(T, Hq, d, 7)
    o, lse = (torch.full(s, 7.0, dtype=t, device="cuda") for s, t in (((T, Hq, d), BF16), ((T, Hq), torch.float32)))
    eta.attn_paged_fwd(q, cache, 0, ints([3, 0, 2]), ints([0, new, 2 * new, T]), max_q=new, granted=ints([1, 0, 1]), out=o, lse=lse)
    torch.cuda.synchronize()
    assert eta.attn_status() == 0
    assert (o[new:2 * new] == 7).all() and (lse[new:2 * new] == 7).all()
    o2, _ = eta.attn_paged_fwd(q, cache, 0, ints([3, 0, 2]), ints([0, new, 2 * new, T]), max_q=new)
    assert torch.equal(o[:new], o2[:new]) and torch.equal(o[2 * new:], o2[2 * new:])


@pytest.mark.parametrize("new", [1, 6, 40])
def test_missing_pages_and_nan(eta, new):
    """A page that the table does not name counts as keys that no row sees; a NaN in a query stays with its row; an
    infinite key or value that the cache holds as a NaN reaches the rows that see it and no other sequence's."""
    lens = [100, 90]
    cache, held = build4(eta, lens, 2, 16, 64, seed=3)
    cache.page_table[0, 2] = -1
    cache.page_table[0, 4] = cache.pages + 5
    held.page_table = cache.page_table.cpu()
    attend(eta, cache, held, [new, new], 4, status=eta.ATTN_ERR_ARG)
    cache, held = build4(eta, lens, 2, 16, 64, seed=4)
    q = queries(2 * new, 8, 64, 1)
    clean, _ = eta.attn_paged_fwd(q, cache, 0, None, ints([0, new, 2 * new]), max_q=new)
    q[0, 3, 7] = math.nan
    o, lse = eta.attn_paged_fwd(q, cache, 0, None, ints([0, new, 2 * new]), max_q=new)
    assert torch.isnan(o[0, 3]).all() and torch.isnan(lse[0, 3])
    o[0, 3] = clean[0, 3]
    assert torch.equal(o, clean)
    for pool in (cache.k, cache.v):
        scales = cache.parts(pool)[1]
        id_ = int(cache.page_table[0, 1])
        keep = scales[0, id_, 1, 5, 2].clone()
        scales[0, id_, 1, 5, 2] = 255
        o, lse = eta.attn_paged_fwd(queries(2 * new, 8, 64, 1), cache, 0, None, ints([0, new, 2 * new]), max_q=new)
        assert torch.isnan(o[:new, 4:]).any(2).all() and not torch.isnan(o[:new, :4]).any() and not torch.isnan(o[new:]).any()
        scales[0, id_, 1, 5, 2] = keep
    assert eta.attn_status() == 0


@pytest.mark.parametrize("new,g", [(1, 4), (2, 8), (64, 2)])
def test_known_results(eta, new, g):
    """Inputs whose result is known: K = 0, so every weight is 1, and V marks blocks of keys, so O is a share of the keys
    and LSE a logarithm of their number (what rounds: 1 / l, its product with o, O in bf16: 2^-8; log2(l) ln 2)."""
    n, d = 6000, 64
    cache, _ = build4(eta, [n], 1, 64, d, seed=1)
    cache.k.zero_()
    kk = torch.zeros((n, 1, d), dtype=BF16, device="cuda")
    v = (torch.arange(n)[:, None] * d // n == torch.arange(d)).float()
    eta.attn_cache_append(cache, 0, kk, (v * 6).to(BF16).cuda()[:, None].contiguous(), None, ints([0, n]))
    q = queries(new, g, d, 3)
    o, lse = eta.attn_paged_fwd(q, cache, 0, None, ints([0, new]), max_q=new)
    for t in range(new):
        see = n - new + 1 + t
        want = 6 * v[:see].double().sum(0) / see
        assert ((o[t].cpu().double() - want).abs() <= (2.0 ** -22 + 2.0 ** -8) * want).all()
        assert (lse[t].cpu().double() - math.log(see)).abs().max() <= 2.0 ** -18


@pytest.mark.parametrize("new,g", [(1, 4), (40, 2)])
@pytest.mark.parametrize("qs,ks", [(1e-3, 1.0), (1.0, 1e-4), (300.0, 0.02), (1e4, 1e-4), (0.02, 500.0), (2e-30, 1.0), (1e15, 1e-5)])
def test_sizes(eta, new, g, qs, ks):
    """Queries and keys of very different sizes (bf16 has the exponents of float32, float16 has not)."""
    cache, held = build4(eta, [300, 40], 2, 16, 128, seed=1, size=ks)
    scale = 1 / math.sqrt(128) / max(1.0, qs * ks / 4)
    attend(eta, cache, held, [new, new], g, size=qs, scale=scale)


def test_columns_of_very_different_sizes(eta):
    """One row whose columns span 2^40: what is small beside the row's largest column still counts where the keys'
    columns make up for it."""
    d = 64
    cache, held = build4(eta, [200], 1, 16, d, seed=5)
    q = queries(1, 4, d, 2)
    q[..., 0] *= 2.0 ** 20
    q[..., 1] *= 2.0 ** -20
    attend(eta, cache, held, [1], 4, q=q, scale=2.0 ** -18)


@pytest.mark.parametrize("seed", range(4))
def test_a_server(eta, seed):
    """Sequences grow (rotated appends), fork, are cut back, freed and compacted; after each step every sequence's cache
    is what its tokens say, and attention over it is right."""
    rng = random.Random(seed)
    heads, page, d, layers = 2, 16, [64, 128, 32, 96][seed], 2
    cache = eta.PagedCache.empty(layers, 60, heads, page, d, 8, 12, dtype=E2M1)
    for pool in (cache.k, cache.v):
        pool.fill_(255)
    pages = Pages(cache)
    table = angles(256, d)
    have = {}         # row: [(k, v)] of each layer, numbers [n, heads, d]

    def check():
        pages.check(cache)
        for r, per in have.items():
            for layer, (k, v) in enumerate(per):
                gk, gv = rows_of(cache, layer, r, 0, k.shape[0])
                assert torch.equal(gk, k) and torch.equal(gv, v)

    for step in range(25):
        act = rng.choice(["grow", "grow", "grow", "fork", "cut", "drop", "compact"])
        empty = [r for r in range(8) if r not in have]
        if act == "grow":
            seqs = rng.sample(range(8), rng.randint(1, 4))
            new = [rng.choice([1, 1, 3, 20]) for _ in seqs]
            ok = pages.reserve(seqs, new)
            granted = eta.attn_cache_reserve(cache, ints(seqs), ints(new))
            assert granted.tolist() == ok
            T = sum(new)
            for layer in range(layers):
                x = torch.randn((T, heads * 6, d), generator=torch.Generator().manual_seed(1000 * seed + 10 * step + layer)).to(BF16).cuda()
                q, k, v = x.split([heads * 4, heads, heads], 1)
                qr = eta.attn_cache_append_rotated(cache, layer, k, v, ints(seqs), ints(starts(new)), table, q=q, granted=granted)
                at = starts(new)
                pos = torch.zeros(T, dtype=torch.long)
                for i, r in enumerate(seqs):
                    if ok[i]:
                        pos[at[i]:at[i + 1]] = torch.arange(pages.lens[r] - new[i], pages.lens[r])
                kv = values(*quantize(turned(k, table, pos, False))), values(*quantize(v.cpu().float()))
                for i, r in enumerate(seqs):
                    if not ok[i]:
                        continue
                    old = have.setdefault(r, [(torch.zeros((0, heads, d), dtype=torch.float64),) * 2] * layers)
                    old = list(old)
                    old[layer] = tuple(torch.cat([o, n[at[i]:at[i + 1]]]) for o, n in zip(old[layer], kv))
                    have[r] = old
                o, _ = eta.attn_paged_fwd(qr, cache, layer, ints(seqs), ints(at), max_q=max(new), granted=granted)
                for i, r in enumerate(seqs):
                    if not ok[i]:
                        continue
                    kk, vv = (t.repeat_interleave(4, 1) for t in have[r][layer])
                    for t in range(at[i], at[i + 1]):
                        n = int(pos[t]) + 1
                        s = torch.einsum("hd,nhd->hn", qr[t].cpu().double(), kk[:n]) / math.sqrt(d)
                        w = torch.softmax(s, 1)
                        want = torch.einsum("hn,nhd->hd", w, vv[:n])
                        size = torch.einsum("hn,nhd->hd", w, vv[:n].abs())
                        assert ((o[t].cpu().double() - want).abs() <= 2.0 ** -8 * (size + want.abs()) * 1.05).all()
        elif act == "fork" and empty and have:
            a, b = rng.choice(list(have)), rng.choice(empty)
            copy = rng.random() < 0.5
            ok = pages.fork([a], [b], copy)
            assert eta.attn_cache_fork(cache, ints([a]), ints([b]), copy=copy).tolist() == ok
            if ok[0]:
                have[b] = list(have[a])
        elif act == "cut" and have:
            r = rng.choice(list(have))
            keep = rng.randint(0, have[r][0][0].shape[0])
            if keep % page and pages.refs[pages.table[r][keep // page]] > 1:
                keep = keep // page * page
            pages.free([r], [keep])
            eta.attn_cache_free(cache, ints([r]), ints([keep]))
            have[r] = [(k[:keep], v[:keep]) for k, v in have[r]]
            if keep == 0:
                del have[r]
        elif act == "drop" and have:
            r = rng.choice(list(have))
            pages.free([r])
            eta.attn_cache_free(cache, ints([r]))
            del have[r]
        elif act == "compact":
            live = pages.compact()
            assert int(eta.attn_cache_compact(cache)[2]) == live
        assert eta.attn_status() == 0
        check()


@pytest.mark.parametrize("heads,page,d", [(1, 16, 32), (8, 64, 128), (3, 256, 96)])
def test_pools_side_by_side(eta, heads, page, d):
    """K and V of a page next to each other, layers inside a page: strides that are not those of a contiguous pool."""
    lens, new = [70, 300, 17], [1, 3, 2]
    layers = 2

    def wide(shape):
        return torch.full(shape, 255, dtype=torch.uint8, device="cuda")
    row = 9 * d // 16
    pages = sum(-(-n // page) for n in lens) + 3
    t = wide((pages, layers, 2, heads, page, row))
    pools = [t[:, :, 0].transpose(0, 1), t[:, :, 1].transpose(0, 1)]

    def put(x):
        p = pools.pop(0)
        p.copy_(x)
        return p
    cache, held = build4(eta, lens, heads, page, d, layers=layers, seed=d, pool=put)
    attend(eta, cache, held, new, 4, layer=1)
    attend(eta, cache, held, [40, 40, 17], 4, layer=0)


def test_graph_of_a_step(eta):
    """Reserve, rotated append and attention captured once and replayed: each replay is one more token."""
    heads, g, d, page, B = 2, 4, 64, 16, 3
    cache = eta.PagedCache.empty(1, 40, heads, page, d, B, 10, dtype=E2M1)
    for pool in (cache.k, cache.v):
        pool.fill_(255)
    table = angles(200, d)
    x = torch.zeros((B, heads * (g + 2), d), dtype=BF16, device="cuda")
    q, k, v = x.split([heads * g, heads, heads], 1)
    seqs, ones, qs = ints([2, 0, 1]), ints([1] * B), ints(list(range(B + 1)))
    o, lse, qr = (torch.empty(s, dtype=t, device="cuda") for s, t in
                  (((B, heads * g, d), BF16), ((B, heads * g), torch.float32), ((B, heads * g, d), BF16)))

    def step():
        granted = eta.attn_cache_reserve(cache, seqs, ones)
        eta.attn_cache_append_rotated(cache, 0, k, v, seqs, qs, table, q=q, q_out=qr, granted=granted)
        eta.attn_paged_fwd(qr, cache, 0, seqs, qs, max_q=1, out=o, lse=lse, granted=granted)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    hist = []
    for i in range(40):
        x.copy_(torch.randn(x.shape, generator=torch.Generator().manual_seed(i)).to(BF16))
        graph.replay()
        kv = values(*quantize(turned(k, table, torch.full((B,), i), False))), values(*quantize(v.cpu().float()))
        hist.append(kv)
        qd = qr.cpu().double()
        kk, vv = (torch.stack([h[j] for h in hist], 1).repeat_interleave(g, 2) for j in (0, 1))
        s = torch.einsum("bhd,bnhd->bhn", qd, kk) / math.sqrt(d)
        w = torch.softmax(s, 2)
        want, size = torch.einsum("bhn,bnhd->bhd", w, vv), torch.einsum("bhn,bnhd->bhd", w, vv.abs())
        assert ((o.cpu().double() - want).abs() <= 2.0 ** -8 * (size + want.abs()) * 1.05).all()
        assert ((lse.cpu().double() - torch.logsumexp(s, 2)).abs() <= 1e-4).all()
    assert eta.attn_status() == 0 and cache.seq_lens.tolist() == [40] * B


def fill(cache, lens, gen, size=1.0):
    """Random 4-bit values for whole sequences, through the append."""
    for r, n in enumerate(lens):
        x = (size * torch.randn((n, 2 * cache.heads, cache.d), generator=gen, device="cuda")).to(BF16)
        eta_append(cache, x[:, :cache.heads], x[:, cache.heads:], r, n)


def eta_append(cache, k, v, r, n):
    import exact_tiled_attention_17_gb300 as m
    m.attn_cache_append(cache, 0, k, v, ints([r]), ints([0, n]))


@pytest.mark.parametrize("lens,new,heads,g,d,page", [
    ([5200, 3100, 4500], [640, 511, 300], 8, 4, 128, 64),
    ([5200, 3100, 4500], [640, 511, 300], 8, 4, 64, 16),
    ([4000, 2500], [400, 513], 6, 5, 96, 32),
    ([6000, 100], [300, 100], 4, 8, 32, 256),
    ([30000], [140], 4, 4, 128, 16),
    ([3000 + 61 * i for i in range(32)], [1] * 32, 8, 4, 128, 64),
    ([3000 + 61 * i for i in range(32)], [1] * 32, 8, 2, 64, 16),
    ([2000 + 61 * i for i in range(24)], [4] * 24, 4, 4, 128, 32),
    ([2000 + 61 * i for i in range(24)], [1] * 24, 4, 7, 96, 128),
])
def test_large_batches_again_and_again(eta, lens, new, heads, g, d, page):
    """Many units to a CTA and full pipelines: every output against the definition in float64 (on the GPU), and the same
    bits each time.  Weights are rounded once to float16 (2^-11), O to bf16 (2^-8), a weight is off by 2^-32 of the
    largest at least, and sums of up to 2^15 float32 numbers add 2^-9 at most where all errors have one sign."""
    gen = torch.Generator(device="cuda").manual_seed(d + page)
    cache = eta.PagedCache.empty(1, sum(-(-n // page) for n in lens) + 5, heads, page, d, len(lens), max(lens) // page + 2, dtype=E2M1)
    for pool in (cache.k, cache.v):
        pool.fill_(255)
    assert eta.attn_cache_reserve(cache, ints(list(range(len(lens)))), ints(lens)).tolist() == [1] * len(lens)
    fill(cache, lens, gen)
    T, Hq, at = sum(new), heads * g, starts(new)
    q = (1.5 * torch.randn((T, Hq, d), generator=gen, device="cuda")).to(BF16)
    runs = [eta.attn_paged_fwd(q, cache, 0, None, ints(at), max_q=max(new)) for _ in range(6)]
    torch.cuda.synchronize()
    assert eta.attn_status() == 0
    for o, lse in runs[1:]:
        assert torch.equal(o, runs[0][0]) and torch.equal(lse, runs[0][1])
    o, lse = runs[0]
    for i, n in enumerate(lens):
        k, v = eta.attn_cache_read(cache, 0, ints([i]), ints([0, n]), n)
        a, b = at[i], at[i + 1]
        see = torch.arange(n, device="cuda")[None] <= n - (b - a) + torch.arange(b - a, device="cuda")[:, None]
        for h in range(heads):
            kd, vd = k[:, h].double(), v[:, h].double()
            for j in range(h * g, h * g + g):
                s = (q[a:b, j].double() @ kd.T / math.sqrt(d)).masked_fill(~see, -math.inf)
                w = torch.softmax(s, 1)
                want, size = w @ vd, w @ vd.abs()
                tol = 2.0 ** -8 * want.abs() + (2.0 ** -11 + 2.0 ** -9) * size + 2.0 ** -32 * vd.abs().sum(0)
                err = (o[a:b, j].double() - want).abs()
                assert (err <= tol).all(), f"entry {i}, head {j}: off by {(err / tol).max():.3g} of the bound"
                assert ((lse[a:b, j].double() - torch.logsumexp(s, 1)).abs() <= 1e-4).all()


@pytest.mark.parametrize("new,g", [(1, 4), (40, 2)])
def test_the_largest_scales(eta, new, g):
    """Scores of 0 under the largest scales: weights are equal, not NaN (queries above 2^15 scale it up once more)."""
    n, d = 100, 64
    cache, held = build4(eta, [n], 1, 16, d, seed=2)
    zero = torch.zeros((n, 1, d), dtype=BF16, device="cuda")
    eta.attn_cache_append(cache, 0, zero, (zero + 3), None, ints([0, n]))
    for scale in (1.0, 1e30, 2.3e38):
        for size in (1e-20, 1.0, 1e6, 1e30):
            o, lse = eta.attn_paged_fwd(queries(new, g, d, 1, size), cache, 0, None, ints([0, new]), max_q=new, scale=scale)
            assert (o == 3).all()
            want = torch.log(torch.arange(n - new + 1, n + 1, dtype=torch.float64))[:, None]
            assert ((lse.cpu().double() - want).abs() <= 1e-5).all()
    assert eta.attn_status() == 0


def test_workspaces_and_streams(eta):
    """A workspace of the caller's, calls on two streams at once, and a captured call replayed beside an eager one."""
    cache, held = build4(eta, [900, 40], 2, 16, 64, seed=8)
    q = queries(2, 8, 64, 4)
    qs = ints([0, 1, 2])
    want, want_l = eta.attn_paged_fwd(q, cache, 0, None, qs, max_q=1)
    need = eta.attn_paged_workspace_size(8, 2, 1, 64, E2M1)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    o, _ = eta.attn_paged_fwd(q, cache, 0, None, qs, max_q=1, workspace=ws)
    assert torch.equal(o, want)
    with pytest.raises(eta.AttnError):
        eta.attn_paged_fwd(q, cache, 0, None, qs, max_q=1, workspace=ws[:need - 16])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        og, lg = eta.attn_paged_fwd(q, cache, 0, None, qs, max_q=1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(50):
        graph.replay()
        with torch.cuda.stream(side):
            o, l = eta.attn_paged_fwd(q, cache, 0, None, qs, max_q=1)
    torch.cuda.synchronize()
    for a, b in ((og, want), (o, want), (lg, want_l), (l, want_l)):
        assert torch.equal(a, b)
