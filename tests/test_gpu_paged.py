"""The paged key/value cache on the GPU: attention of new tokens against the
definition in float64 (bounds derived in paged_ref.py), the page operators
against plain integers, and both together as a server uses them."""
import math
import random
import threading

import pytest
import torch

from paged_bounds import close_weights, counts, fine_keys
from paged_ref import Pages, check_attention, gather

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def eta():
    import exact_tiled_attention_17_gb300 as m
    return m


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def pools(layers, pages, heads, page, d, dtype, layout):
    """K and V, all NaN."""
    if layout == "head":
        kv = [torch.full((layers, pages, heads, page, d), math.nan, dtype=dtype, device="cuda") for _ in range(2)]
    elif layout == "token":
        kv = [torch.full((layers, pages, page, heads, d), math.nan, dtype=dtype, device="cuda").transpose(2, 3)
              for _ in range(2)]
    elif layout == "side":      # K and V of a page side by side
        t = torch.full((layers, pages, 2, heads, page, d), math.nan, dtype=dtype, device="cuda")
        kv = [t[:, :, 0], t[:, :, 1]]
    else:                       # layers inside a page
        kv = [torch.full((pages, layers, heads, page, d), math.nan, dtype=dtype, device="cuda").transpose(0, 1)
              for _ in range(2)]
    return kv


def build(eta, lens, heads, page, d, dtype=BF16, layout="head", layers=1, spare=3, seed=0, size=1.0, max_pages=None):
    """A cache whose rows hold sequences of the given lengths on random pages;
    every slot that holds no token is NaN."""
    rng, g = random.Random(seed), torch.Generator(device="cuda").manual_seed(seed)
    need = [-(-n // page) for n in lens]
    pages = sum(need) + spare
    cols = max_pages or max(need + [1]) + 1
    order = list(range(pages))
    rng.shuffle(order)
    table = torch.full((len(lens), cols), -1, dtype=torch.int32)
    refs = torch.zeros(pages, dtype=torch.int32)
    k, v = pools(layers, pages, heads, page, d, dtype, layout)
    for r, n in enumerate(lens):
        for c in range(need[r]):
            p = order.pop()
            table[r, c], refs[p] = p, 1
            m = min(page, n - c * page)
            for t in (k, v):
                t[:, p, :, :m] = (size * torch.randn((layers, heads, m, d), generator=g, device="cuda")).to(dtype)
    return eta.PagedCache(k, v, table.cuda(), ints(lens), refs.cuda())


def queries(T, Hq, d, dtype, seed=0, size=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed + 99)
    return (size * torch.randn((T, Hq, d), generator=g, device="cuda")).to(dtype)


def starts(new):
    v = [0]
    for n in new:
        v.append(v[-1] + n)
    return v


def attend(eta, cache, new, g, seqs=None, causal=True, layer=0, seed=0, before=0, behind=0, size=1.0, max_q=None, scale=None,
           out=None, **kw):
    """Runs attn_paged_fwd over a list, with rows of Q before and behind it, and checks every row."""
    T = sum(new) + before + behind
    Hq = cache.heads * g
    q = queries(T, Hq, cache.d, cache.dtype, seed, size)
    o = out if out is not None else torch.full_like(q, 7.0)
    lse = torch.full((T, Hq), 7.0, device="cuda")
    held = (o.clone(), lse.clone())
    qs = ints([before + x for x in starts(new)])
    sq = None if seqs is None else ints(seqs)
    eta.attn_paged_fwd(q, cache, layer, sq, qs, max_q=max_q or max(max(new), 1), causal=causal, scale=scale, out=o, lse=lse, **kw)
    torch.cuda.synchronize()
    assert eta.attn_status() == eta.ATTN_OK
    check_attention(q, cache, layer, sq, qs, causal, scale if scale is not None else 1 / math.sqrt(cache.d), o, lse, held)


# lengths (with the new tokens) and new tokens of a batch
BATCHES = {
    "one": ([1], [1]),
    "decode": ([1, 15, 16, 17, 63, 64, 65, 129, 300], [1] * 9),
    "few": ([5, 200, 33, 64, 7], [5, 3, 2, 1, 4]),
    "chunk": ([40, 200, 129, 90], [40, 77, 129, 1]),
    "empty": ([0, 70, 0, 3, 20], [0, 0, 2, 5, 0]),       # no tokens; more new tokens than the sequence holds
}


@pytest.mark.parametrize("batch", BATCHES)
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dtype,heads,g,d,page,layout", [
    (BF16, 2, 4, 128, 16, "head"), (BF16, 1, 1, 64, 32, "token"), (BF16, 3, 3, 96, 64, "head"), (BF16, 2, 8, 32, 128, "token"),
    (BF16, 1, 16, 128, 256, "side"), (BF16, 2, 5, 64, 16, "layers"), (BF16, 1, 64, 64, 16, "head"), (BF16, 4, 2, 128, 64, "token"),
    (F32, 2, 4, 128, 16, "head"), (F32, 1, 1, 64, 32, "token"), (F32, 3, 3, 96, 64, "side"), (F32, 1, 7, 32, 128, "layers"),
    (F32, 1, 64, 64, 16, "head"), (F32, 2, 16, 128, 256, "token"),
])
def test_attention(eta, batch, causal, dtype, heads, g, d, page, layout):
    lens, new = BATCHES[batch]
    cache = build(eta, lens, heads, page, d, dtype, layout, layers=2, seed=len(lens))
    attend(eta, cache, new, g, causal=causal, layer=1, before=1, behind=2)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n,new", [(5000, 1), (5000, 4), (4097, 33), (2000, 500), (1023, 1023), (9000, 129)])
def test_long_and_split(eta, dtype, n, new):
    """Long axes, which several CTAs share, beside short sequences; large scores."""
    cache = build(eta, [n, 3, n // 3], 2, 16, 64, dtype, seed=n)
    new2 = [new, 1, min(new, n // 3)]
    attend(eta, cache, new2, 4, seed=n)
    cache = build(eta, [n], 1, 64, 128, dtype, seed=n + 1, size=4.0)
    attend(eta, cache, [new], 2, seed=n, size=4.0)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d", [32, 64, 96, 128])
@pytest.mark.parametrize("g,new", [(1, 1), (3, 1), (2, 2), (8, 1), (1, 7), (5, 2), (4, 4), (3, 9), (8, 4)])
def test_few_rows(eta, dtype, d, g, new):
    """Every size of the units for few rows: short lengths, ends inside a batch of keys, entries with less than the most tokens."""
    lens = [1, 700, 2, 15, 33, 0, 64, 65, 5, 1291]
    cache = build(eta, lens, 2, 16 if g < 4 else 128, d, dtype, ["head", "token"][g % 2], seed=d + g)
    some = [min(n, 1 + (new * i) % (new + 1)) for i, n in enumerate(lens)]
    some[1] = new
    attend(eta, cache, some, g, causal=new != 2, before=1, behind=1, seed=g)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("new", [1, 7, 40])
def test_one_unit_over_all_ctas(eta, dtype, new):
    """More parts to a row than the merge kernel reads at once (one kv head, a long context)."""
    cache = build(eta, [70001], 1, 64, 64, dtype, seed=new)
    attend(eta, cache, [new], 4, seed=new)


def run_known(eta, known, page=64):
    """The known case as a sequence on random pages, beside NaN."""
    (n, d), dtype = known.k.shape, known.q.dtype
    cache = build(eta, [3, n], 1, page, d, dtype, seed=n)
    at = torch.arange(n, device="cuda")
    ids = cache.page_table[1].long()[at // page]
    cache.k[0, ids, 0, at % page] = known.k.cuda()
    cache.v[0, ids, 0, at % page] = known.v.cuda()
    T = known.q.shape[0]
    o, lse = eta.attn_paged_fwd(known.q.cuda(), cache, 0, ints([1]), ints([0, T]), scale=known.scale)
    assert eta.attn_status() == eta.ATTN_OK
    known.check(o, lse)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("new", [1, 2, 7, 40])
def test_every_key_of_a_long_context_counts(eta, dtype, new):
    """One unit over all CTAs, more parts than the merge reads at once: none may be lost."""
    run_known(eta, counts(70001, new, 4, 64, dtype))


@pytest.mark.parametrize("d", [32, 64, 96, 128])
@pytest.mark.parametrize("n,new,g", [(2, 1, 8), (17, 1, 4), (40, 4, 4), (64, 16, 1)])
def test_probabilities_in_two_parts(eta, d, n, new, g):
    """At most 16 rows: one rounding of P to bf16 would be far outside the bound."""
    run_known(eta, close_weights(n, new, g, d), page=16)


@pytest.mark.parametrize("n,new", [(50, 1), (5000, 1), (5000, 2), (5000, 4), (5000, 8), (5000, 40), (70001, 1), (70001, 40)])
def test_float32_keeps_its_bits(eta, n, new):
    """Keys that TF32 does not tell apart, at lengths where a bound by the worst sum would hide it."""
    run_known(eta, fine_keys(n, new, 4))


@pytest.mark.parametrize("dtype,d", [(BF16, 128), (BF16, 64), (F32, 64)])
def test_many_short_chunks(eta, dtype, d):
    """Several list entries to a lane of the planning warp, in the kernels for many rows."""
    lens = [(11 * i) % 150 for i in range(230)]
    new = [(5 * i) % 23 for i in range(230)]
    cache = build(eta, lens, 2, 16, d, dtype, seed=6)
    attend(eta, cache, new, 3, seqs=[(i * 7) % 230 for i in range(230)], before=2, behind=3)


def test_many_sequences(eta):
    """More list entries than a block has threads."""
    lens = [(7 * i) % 90 for i in range(1300)]
    new = [1 + (i % 3) if i % 5 else 0 for i in range(1300)]
    cache = build(eta, lens, 1, 16, 64, BF16, seed=5)
    attend(eta, cache, new, 2, seqs=list(reversed(range(1300))))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("new", [1, 40])
def test_a_sequence_twice_and_rows_in_any_order(eta, dtype, new):
    cache = build(eta, [100, 64, 81, 200], 2, 32, 64, dtype)
    attend(eta, cache, [new] * 5, 4, seqs=[3, 1, 3, 0, 2])


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("new", [1, 100])
def test_strides(eta, dtype, new):
    """Q as a slice of a fused projection, O head by head."""
    lens, nn = [300, 120], [new, 100]
    cache = build(eta, lens, 2, 16, 64, dtype)
    T, Hq, d = sum(nn), 8, 64
    fused = queries(T, Hq + 4, d, dtype)
    q = fused[:, 2:2 + Hq]
    o = torch.full((Hq, T, d), 7.0, dtype=dtype, device="cuda").transpose(0, 1)
    qs = ints(starts(nn))
    o2, lse = eta.attn_paged_fwd(q, cache, 0, None, qs, out=o)
    torch.cuda.synchronize()
    assert o2 is o and eta.attn_status() == eta.ATTN_OK
    check_attention(q, cache, 0, None, qs, True, 0.125, o, lse)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_dimensions_of_one(eta, dtype):
    """One token, one head: whatever strides torch gives these dimensions."""
    cache = build(eta, [21], 1, 16, 64, dtype)
    wide = queries(3, 5, 64, dtype)
    q = wide.as_strided((1, 1, 64), (3, 7, 1))
    o, lse = eta.attn_paged_fwd(q, cache, 0, None, ints([0, 1]))
    torch.cuda.synchronize()
    check_attention(q, cache, 0, None, ints([0, 1]), True, 0.125, o, lse)
    eta.attn_cache_append(cache, 0, q, q, None, ints([0, 1]))
    torch.cuda.synchronize()
    assert torch.equal(cache.k[0, int(cache.page_table[0, 1]), 0, 4], q[0, 0])
    assert eta.attn_status() == eta.ATTN_OK


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("new", [1, 70])
def test_offsets_past_32_bits(eta, dtype, new):
    """Pages further apart than 2^31 elements."""
    page, heads, d = 16, 1, 64
    far = (1 << 31) // (2 if dtype == F32 else 1) + 1024 * 64
    raw = torch.empty(far + 4096, dtype=dtype, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    k = raw.as_strided((1, 2, heads, page, d), (0, far, page * d, d, 1))
    raw[:1024].normal_(generator=g)
    raw[far:far + 1024].normal_(generator=g)
    raw2 = torch.empty(far + 4096, dtype=dtype, device="cuda")
    v2 = raw2.as_strided((1, 2, heads, page, d), (0, far, page * d, d, 1))
    v2.copy_(k.flip(3))
    cache = eta.PagedCache(k, v2, ints([[1, 0]]), ints([27]), ints([1, 1]))
    attend(eta, cache, [min(new, 27)], 4)
    kn = queries(5, heads, d, dtype, 3)
    eta.attn_cache_append(cache, 0, kn, -kn, None, ints([0, 5]))
    torch.cuda.synchronize()
    for t in range(5):
        pos = 22 + t
        assert torch.equal(k[0, [1, 0][pos // 16], :, pos % 16], kn[t])
        assert torch.equal(v2[0, [1, 0][pos // 16], :, pos % 16], -kn[t])


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("new", [1, 60])
def test_pages_that_do_not_exist(eta, dtype, new):
    """A table entry outside the pool counts as keys that no row sees, and is reported."""
    cache = build(eta, [200, 90], 2, 16, 64, dtype)
    cache.page_table[0, 3] = cache.pages
    cache.page_table[0, 12] = -5
    cache.page_table[1, 0] = 2 ** 30
    q = queries(2 * new, 8, 64, dtype)
    qs = ints([0, new, 2 * new])
    o, lse = eta.attn_paged_fwd(q, cache, 0, None, qs)
    assert eta.attn_status() == eta.ATTN_ERR_ARG
    assert eta.attn_status() == eta.ATTN_OK
    check_attention(q, cache, 0, None, qs, True, 0.125, o, lse)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("new", [1, 60])
def test_bad_entries_are_left_out(eta, dtype, new):
    cache = build(eta, [200, 90, 77], 2, 16, 64, dtype)
    q = queries(5 * new, 8, 64, dtype)
    o, lse = torch.full_like(q, 7.0), torch.full((5 * new, 8), 7.0, device="cuda")
    qs = [new * i for i in range(6)]
    eta.attn_paged_fwd(q, cache, 0, ints([0, 9, 1, -1, 2]), ints(qs), max_q=new, out=o, lse=lse)
    assert eta.attn_status() == eta.ATTN_ERR_ARG
    for i, s in enumerate([0, None, 1, None, 2]):
        a, b = qs[i], qs[i + 1]
        if s is None:
            assert (o[a:b] == 7).all() and (lse[a:b] == 7).all()
        else:
            check_attention(q[a:b], cache, 0, ints([s]), ints([0, b - a]), True, 0.125, o[a:b], lse[a:b])


@pytest.mark.parametrize("new", [1, 50])
def test_scores_of_any_size(eta, new):
    """Scores far above 2^8 apart and all equal: the running maximum must follow."""
    cache = build(eta, [400], 1, 16, 64, BF16, size=1.0)
    ids = cache.page_table[0, :25].long()
    ramp = torch.arange(400, device="cuda", dtype=torch.float32).reshape(25, 1, 16, 1) * 0.05
    cache.k[0, ids] = ramp.expand(25, 1, 16, 64).to(BF16)     # every query with a positive sum prefers the last keys
    attend(eta, cache, [new], 2, size=3.0)
    cache.k[0, ids] = -ramp.expand(25, 1, 16, 64).to(BF16)
    attend(eta, cache, [new], 2, size=3.0)
    cache.k[0, ids] = 0.0
    attend(eta, cache, [new], 2)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("new,n", [(1, 100), (1, 5000), (40, 100), (40, 5000)])
def test_nan_reaches_its_own_rows_only(eta, dtype, new, n):
    """A NaN in one query row, or in a key, is seen where it belongs and nowhere else."""
    cache = build(eta, [n, 77], 2, 16, 64, dtype)
    q = queries(new + 3, 8, 64, dtype)
    q[0, 3] = math.nan
    o, lse = eta.attn_paged_fwd(q, cache, 0, None, ints([0, new, new + 3]))
    bad = torch.zeros(new + 3, 8, dtype=torch.bool)
    bad[0, 3] = True
    assert torch.equal(torch.isnan(o).all(2).cpu(), bad) and torch.equal(torch.isnan(o).any(2).cpu(), bad)
    assert torch.equal(torch.isnan(lse).cpu(), bad)
    q[0, 3] = 0.5
    cache.k[0, int(cache.page_table[1, 74 // 16]), 1, 74 % 16, 5] = math.nan   # seen by the second entry's rows, kv head 1
    o, lse = eta.attn_paged_fwd(q, cache, 0, None, ints([0, new, new + 3]))
    bad = torch.zeros(new + 3, 8, dtype=torch.bool)
    bad[new:, 4:] = True
    assert torch.equal(torch.isnan(lse).cpu(), bad)
    assert torch.equal(torch.isnan(o).all(2).cpu(), bad) and torch.equal(torch.isnan(o).any(2).cpu(), bad)
    assert eta.attn_status() == eta.ATTN_OK


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_entries_past_max_q_are_left_out(eta, dtype):
    cache = build(eta, [100, 90], 1, 16, 64, dtype)
    q = queries(30, 4, 64, dtype)
    o, lse = torch.full_like(q, 7.0), torch.full((30, 4), 7.0, device="cuda")
    eta.attn_paged_fwd(q, cache, 0, None, ints([0, 20, 30]), max_q=10, out=o, lse=lse)
    assert eta.attn_status() == eta.ATTN_ERR_ARG
    assert (o[:20] == 7).all() and (lse[:20] == 7).all()
    check_attention(q[20:], cache, 0, ints([1]), ints([0, 10]), True, 0.125, o[20:], lse[20:])


def test_streams_and_graphs(eta):
    """A call on another stream; a captured one replayed after the lengths changed."""
    cache = build(eta, [500, 40, 300], 2, 16, 128, BF16, spare=30, max_pages=40)
    q = queries(3, 8, 128, BF16)
    qs = ints([0, 1, 2, 3])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o, lse = eta.attn_paged_fwd(q, cache, 0, None, qs, max_q=1, stream=side)
    side.synchronize()
    check_attention(q, cache, 0, None, qs, True, 128 ** -0.5, o, lse)
    kn, vn = queries(3, 2, 128, BF16, 1), queries(3, 2, 128, BF16, 2)
    seqs, one = ints([0, 1, 2]), ints([1, 1, 1])
    ref = Pages(cache)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        granted = eta.attn_cache_reserve(cache, seqs, one)
        eta.attn_cache_append(cache, 0, kn, vn, seqs, qs)
        o, lse = eta.attn_paged_fwd(q, cache, 0, seqs, qs, max_q=1)
    for step in range(20):
        kn.normal_()
        vn.normal_()
        q.normal_()
        graph.replay()
        torch.cuda.synchronize()
        assert granted.tolist() == ref.reserve([0, 1, 2], [1, 1, 1]) == [1, 1, 1]
        if step in (0, 7, 19):
            check_attention(q, cache, 0, seqs, qs, True, 128 ** -0.5, o, lse)
    ref.check(cache)
    assert eta.attn_status() == eta.ATTN_OK


def test_workspaces_of_threads(eta):
    """Threads on one stream and on streams of their own: right results, and no workspace outlives its thread."""
    cache = build(eta, [300, 90], 2, 16, 128, BF16)
    q, qs = queries(40, 8, 128, BF16), ints([0, 30, 40])
    want = eta.attn_paged_fwd(q, cache, 0, None, qs)
    torch.cuda.synchronize()
    held, got = torch.cuda.memory_allocated(), []

    def work(stream):
        for _ in range(20):
            o, lse = eta.attn_paged_fwd(q, cache, 0, None, qs, stream=stream)
        torch.cuda.synchronize()
        got.append((o.cpu(), lse.cpu()))

    for _ in range(3):
        threads = [threading.Thread(target=work, args=(s,)) for s in (None, None, torch.cuda.Stream(), torch.cuda.Stream())]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
    assert len(got) == 12
    for o, lse in got:
        assert torch.equal(o, want[0].cpu()) and torch.equal(lse, want[1].cpu())
    assert torch.cuda.memory_allocated() == held
    assert eta.attn_status() == eta.ATTN_OK


@pytest.mark.parametrize("dtype,new", [(BF16, 1), (BF16, 30), (BF16, 300), (F32, 1), (F32, 100)])
def test_repeated_runs_are_bitwise_equal(eta, dtype, new):
    cache = build(eta, [3000, 700], 2, 16, 128, dtype)
    q = queries(2 * new, 8, 128, dtype)
    qs = ints([0, new, 2 * new])
    o, lse = eta.attn_paged_fwd(q, cache, 0, None, qs)
    for _ in range(10):
        a, b = eta.attn_paged_fwd(q, cache, 0, None, qs)
        assert torch.equal(a, o) and torch.equal(b, lse)


def test_refusals(eta):
    cache = build(eta, [20, 20], 2, 16, 64)
    q, qs = queries(2, 4, 64, BF16), ints([0, 1, 2])
    with pytest.raises(ValueError):
        eta.attn_paged_fwd(q.float(), cache, 0, None, qs)
    with pytest.raises(ValueError):
        eta.attn_paged_fwd(q[..., :32], cache, 0, None, qs)
    with pytest.raises(ValueError):
        eta.attn_paged_fwd(q, cache, 0, ints([0]), qs)
    with pytest.raises(ValueError):
        eta.attn_paged_fwd(q, cache, 0, None, qs.long())
    with pytest.raises(ValueError):
        eta.attn_paged_fwd(q, cache, 0, None, qs, out=torch.empty_like(q)[:1])
    with pytest.raises(ValueError):
        eta.attn_cache_append(cache, 0, q, q, None, qs)
    for bad in (dict(layer=1), dict(max_q=3), dict(scale=-1.0), dict(workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))):
        kw = dict(layer=0)
        kw.update(bad)
        layer = kw.pop("layer")
        with pytest.raises(eta.AttnError):
            eta.attn_paged_fwd(q, cache, layer, None, qs, **kw)
    with pytest.raises(ValueError):
        eta.PagedCache(cache.k, cache.v, cache.page_table, cache.seq_lens, ints([0]))
    with pytest.raises(ValueError):
        eta.PagedCache(cache.k, cache.v.float(), cache.page_table, cache.seq_lens, cache.ref_counts)
    o, _ = eta.attn_paged_fwd(q[:0], cache, 0, None, ints([0, 0, 0]))
    assert o.shape == (0, 4, 64)


# ---------------------------------------------------------------------------
# pages
# ---------------------------------------------------------------------------
def new_cache(eta, pages, page, seqs, max_pages, layers=2, heads=2, d=32, dtype=BF16, token_major=False):
    c = eta.PagedCache.empty(layers, pages, heads, page, d, seqs, max_pages, dtype, "cuda", token_major)
    c.k.normal_()
    c.v.normal_()
    return c


def check_copies(cache, before, copies):
    """The pools after a call: the copied slots, and everything else as it was."""
    for now, was in zip((cache.k, cache.v), before):
        want = was.clone()
        for s, t, n in copies:
            want[:, t, :, :n] = was[:, s, :, :n]
        assert torch.equal(now, want)


@pytest.mark.parametrize("seed", range(12))
def test_pages_against_plain_integers(eta, seed):
    """A long run of random operators, each checked: tables, counts, grants, contents."""
    rng = random.Random(seed)
    rows, page = rng.choice([5, 40]), rng.choice([16, 32, 64, 128, 256])
    pages = rng.choice([7, 60, 300])
    cache = new_cache(eta, pages, page, rows, rng.choice([4, 30]), layers=rng.choice([1, 3]), heads=rng.choice([1, 3]),
                      d=rng.choice([32, 64, 96, 128]), dtype=rng.choice([BF16, F32]), token_major=rng.random() < 0.5)
    ref = Pages(cache)
    for _ in range(25):
        n = rng.randint(1, 8)
        some = rng.sample(range(rows), min(n, rows))
        before = (cache.k.clone(), cache.v.clone())
        ref.copies = []
        op = rng.choice(["reserve", "reserve", "free", "fork", "fork", "compact"])
        if op == "reserve":
            add = [rng.choice([0, 1, 5, page, rng.randint(0, 4 * page)]) for _ in some]
            got = eta.attn_cache_reserve(cache, ints(some), ints(add))
            assert got.tolist() == ref.reserve(some, add)
        elif op == "free":
            keep = None if rng.random() < 0.4 else [rng.choice([0, 1, page, rng.randint(0, 4 * page)]) for _ in some]
            eta.attn_cache_free(cache, ints(some), None if keep is None else ints(keep))
            ref.free(some, keep)
        elif op == "fork":
            empty = [r for r in range(rows) if ref.lens[r] == 0]
            kids = rng.sample(empty, min(n, len(empty)))
            if not kids:
                continue
            par, copy = [rng.randrange(rows) for _ in kids], rng.random() < 0.5
            got = eta.attn_cache_fork(cache, ints(par), ints(kids), copy=copy)
            assert got.tolist() == ref.fork(par, kids, copy)
        else:
            if rng.random() < 0.5:
                _, _, live = eta.attn_cache_compact(cache)
                assert live.tolist() == [ref.compact()]
            else:
                was = (cache.page_table.clone(), cache.ref_counts.clone())
                table, refs, live = eta.attn_cache_compact(cache, inplace=False)
                assert torch.equal(cache.page_table, was[0]) and torch.equal(cache.ref_counts, was[1])
                assert live.tolist() == [ref.compact()]
                cache.page_table.copy_(table)
                cache.ref_counts.copy_(refs)
        ref.check(cache)
        ref.consistent()
        check_copies(cache, before, ref.copies)
    assert eta.attn_status() == (eta.ATTN_ERR_ARG if ref.shared else eta.ATTN_OK)


def test_growing_into_a_shared_page(eta):
    """A fork that is cut back into a full page, which its parent reads too: neither grows into it."""
    cache = new_cache(eta, 12, 16, 5, 4)
    ref = Pages(cache)
    assert eta.attn_cache_reserve(cache, ints([0]), ints([32])).tolist() == ref.reserve([0], [32]) == [1]
    assert eta.attn_cache_fork(cache, ints([0, 0]), ints([1, 2])).tolist() == ref.fork([0, 0], [1, 2], False) == [1, 1]
    eta.attn_cache_free(cache, ints([1, 2]), ints([20, 16]))
    ref.free([1, 2], [20, 16])
    assert eta.attn_status() == eta.ATTN_OK
    # sequence 1's next token would go into page 1; sequence 2's starts a page, sequence 0's too
    assert eta.attn_cache_reserve(cache, ints([1, 2, 0]), ints([1, 5, 1])).tolist() == ref.reserve([1, 2, 0], [1, 5, 1]) == [0, 1, 1]
    assert eta.attn_status() == eta.ATTN_ERR_ARG
    ref.check(cache)
    # a fork of it has a copy
    before = (cache.k.clone(), cache.v.clone())
    assert eta.attn_cache_fork(cache, ints([1]), ints([3])).tolist() == ref.fork([1], [3], False) == [1]
    check_copies(cache, before, ref.copies)
    assert eta.attn_cache_reserve(cache, ints([3]), ints([6])).tolist() == ref.reserve([3], [6]) == [1]
    # and once the others have left, the page is its own
    eta.attn_cache_free(cache, ints([0]))
    ref.free([0])
    assert eta.attn_cache_reserve(cache, ints([1]), ints([6])).tolist() == ref.reserve([1], [6]) == [1]
    ref.check(cache)
    ref.consistent()
    assert eta.attn_status() == eta.ATTN_OK


@pytest.mark.parametrize("tokens", [1, 9, 5000])
def test_append_leaves_shared_pages_alone(eta, tokens):
    """Tokens appended although no room was granted for them: none goes into a page that another sequence reads."""
    rows, page = max(2 * tokens, 32) // 16 * 16 + 16, 16
    cache = new_cache(eta, 3 * rows // page, page, 4, 2 * rows // page)
    assert eta.attn_cache_reserve(cache, ints([0]), ints([rows])).tolist() == [1]
    assert eta.attn_cache_fork(cache, ints([0]), ints([1])).tolist() == [1]
    eta.attn_cache_free(cache, ints([1]), ints([rows - 3]))      # cut back into a page that sequence 0 names too
    kn, vn = queries(tokens, 2, 32, BF16, 1), queries(tokens, 2, 32, BF16, 2)
    q = queries(1, 4, 32, BF16)
    qs = ints([0, tokens])
    o, lse = eta.attn_paged_fwd(q, cache, 0, ints([0]), ints([0, 1]))
    held = (cache.k.clone(), cache.v.clone())
    assert eta.attn_cache_reserve(cache, ints([1]), ints([tokens])).tolist() == [0]
    assert eta.attn_status() == eta.ATTN_ERR_ARG
    for row in (0, 1):   # neither of the two may write what both read
        for layer in range(2):
            eta.attn_cache_append(cache, layer, kn, vn, ints([row]), qs)
        assert eta.attn_status() == eta.ATTN_ERR_ARG
    assert torch.equal(cache.k, held[0]) and torch.equal(cache.v, held[1])
    o2, lse2 = eta.attn_paged_fwd(q, cache, 0, ints([0]), ints([0, 1]))
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    # what has room of its own is written all the same, beside a sequence that has none
    assert eta.attn_cache_reserve(cache, ints([2]), ints([1])).tolist() == [1]
    both = queries(tokens + 1, 2, 32, BF16, 3)
    eta.attn_cache_append(cache, 1, both, both, ints([1, 2]), ints([0, tokens, tokens + 1]))
    assert eta.attn_status() == eta.ATTN_ERR_ARG
    want = held[0].clone()
    want[1, int(cache.page_table[2, 0]), :, 0] = both[tokens]
    assert torch.equal(cache.k, want)


@pytest.mark.parametrize("T", [10, 5000])
def test_append_token_ranges(eta, T):
    """Entries whose tokens are not all rows of the call are left out whole and reported, as in the attention."""
    big, lens = 2 ** 31 - 1, [T + 8, 40]
    for qs, ok in (([0, 4, T + 2], [1, 0]), ([-2, 4, 10], [0, 1]), ([0, 4, big], [1, 0]), ([0, T, T + 3], [1, 0]),
                   ([-5, 0, 3], [0, 1]), ([-9, -5, 3], [0, 0]), ([4, 2, 9], [0, 1]), ([T, T + 1, T + 1], [0, 0])):   # (the last: empty, but past the rows)
        cache = build(eta, lens, 2, 16, 64)
        kn = queries(T, 2, 64, BF16)
        want, table = cache.k.clone(), cache.page_table.tolist()
        for i in (0, 1):
            for t in range(qs[i], qs[i + 1] if ok[i] else qs[i]):
                at = lens[i] - qs[i + 1] + t
                want[0, table[i][at // 16], :, at % 16] = kn[t]
        eta.attn_cache_append(cache, 0, kn, kn, None, ints(qs))
        assert eta.attn_status() == eta.ATTN_ERR_ARG, qs
        assert torch.equal(cache.k.nan_to_num(9.0), want.nan_to_num(9.0)), qs
        # an entry that got no room is not looked at
        eta.attn_cache_append(cache, 0, kn, kn, None, ints(qs), granted=ints(ok))
        assert eta.attn_status() == eta.ATTN_OK, qs
        assert torch.equal(cache.k.nan_to_num(9.0), want.nan_to_num(9.0)), qs


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("new", [1, 6, 40])
def test_entries_without_room_are_left_out(eta, dtype, new):
    """The pool runs out inside a list: what was refused keeps its tokens, and its rows stay as they were."""
    lens, page, heads, g = [29, 64, 47, 16], 16, 2, 4
    cache = build(eta, lens, heads, page, 64, dtype, spare=-(-new // page), max_pages=20)
    ref = Pages(cache)
    seqs, add = [1, 3, 0, 2, 2], [new] * 4 + [1]
    T = sum(add)
    room = eta.attn_cache_reserve(cache, ints(seqs), ints(add))
    # (sequence 2's second mention does not count in any case)
    assert room.tolist() == ref.reserve(seqs, add) and 0 < sum(room.tolist()) < 4
    assert eta.attn_status() == eta.ATTN_ERR_ARG
    kn, vn = queries(T, heads, 64, dtype, 1), queries(T, heads, 64, dtype, 2)
    qs = ints(starts(add))
    want, table = [cache.k.clone(), cache.v.clone()], cache.page_table.tolist()
    for i, s in enumerate(seqs):
        for t in range(add[i] if room[i] else 0):
            at = ref.lens[s] - add[i] + t
            for pool, x in zip(want, (kn, vn)):
                pool[0, table[s][at // page], :, at % page] = x[sum(add[:i]) + t]
    eta.attn_cache_append(cache, 0, kn, vn, ints(seqs), qs, granted=room)
    assert eta.attn_status() == eta.ATTN_OK
    for pool, x in zip((cache.k, cache.v), want):
        assert torch.equal(pool.nan_to_num(9.0), x.nan_to_num(9.0))
    q = queries(T, heads * g, 64, dtype)
    o, lse = torch.full_like(q, 7.0), torch.full((T, heads * g), 7.0, device="cuda")
    eta.attn_paged_fwd(q, cache, 0, ints(seqs), qs, max_q=new, out=o, lse=lse, granted=room)
    assert eta.attn_status() == eta.ATTN_OK
    for i, s in enumerate(seqs):
        a, b = sum(add[:i]), sum(add[:i + 1])
        if room[i]:
            check_attention(q[a:b], cache, 0, ints([s]), ints([0, b - a]), True, 0.125, o[a:b], lse[a:b])
        else:
            assert (o[a:b] == 7).all() and (lse[a:b] == 7).all()
    # a refused mention is none: the sequence's next entry is its first
    room2 = ints([0, 1])
    eta.attn_cache_append(cache, 0, kn[:2], vn[:2], ints([1, 1]), ints([0, 1, 2]), granted=room2)
    assert eta.attn_status() == eta.ATTN_OK
    at = ref.lens[1] - 1
    assert torch.equal(cache.k[0, table[1][at // page], :, at % page], kn[1])
    with pytest.raises(ValueError):
        eta.attn_cache_append(cache, 0, kn[:2], vn[:2], ints([1, 1]), ints([0, 1, 2]), granted=room)
    with pytest.raises(ValueError):
        eta.attn_paged_fwd(q, cache, 0, ints(seqs), qs, granted=room.float())


def test_a_captured_step_outlives_its_pool(eta):
    """Reserve, append and attention in one graph, replayed until the pages have run out and beyond."""
    page, heads, g, d = 16, 2, 2, 64
    cache = new_cache(eta, 9, page, 3, 8, layers=1, heads=heads, d=d)
    assert eta.attn_cache_reserve(cache, ints([0, 1, 2]), ints([16, 30, 7])).tolist() == [1, 1, 1]
    ref = Pages(cache)
    seqs, add, qs = ints([2, 0, 1]), ints([3, 5, 2]), ints([0, 3, 8, 10])
    kn, q = queries(10, heads, d, BF16, 1), queries(10, heads * g, d, BF16)
    o, lse = torch.zeros_like(q), torch.zeros((10, heads * g), device="cuda")
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        room = eta.attn_cache_reserve(cache, seqs, add)
        eta.attn_cache_append(cache, 0, kn, kn, seqs, qs, granted=room)
        eta.attn_paged_fwd(q, cache, 0, seqs, qs, max_q=5, out=o, lse=lse, granted=room)
    held = {s: gather(cache, 0, s, ref.lens[s])[0] for s in range(3)}
    refused = 0
    for _ in range(25):
        kn.normal_()
        q.normal_()
        o.fill_(7.0)
        lse.fill_(7.0)
        graph.replay()
        assert room.tolist() == ref.reserve([2, 0, 1], [3, 5, 2])
        refused += 3 - sum(room.tolist())
        ref.check(cache)
        for i, s in enumerate([2, 0, 1]):
            a, b = [0, 3, 8, 10][i:i + 2]
            if room[i]:
                held[s] = torch.cat([held[s], kn[a:b].transpose(0, 1).cpu().double()], 1)
                check_attention(q[a:b], cache, 0, ints([s]), ints([0, b - a]), True, d ** -0.5, o[a:b], lse[a:b])
            else:
                assert (o[a:b] == 7).all() and (lse[a:b] == 7).all()
            assert torch.equal(gather(cache, 0, s, ref.lens[s])[0], held[s])
    assert refused > 20 and eta.attn_status() == eta.ATTN_OK


def test_free_keeps_what_it_is_told(eta):
    """Counts of none, negative ones, all, and more than there is."""
    cache = new_cache(eta, 30, 16, 6, 4)
    ref = Pages(cache)
    everyone, lens = list(range(6)), [33, 16, 1, 64, 20, 0]
    assert eta.attn_cache_reserve(cache, ints(everyone), ints(lens)).tolist() == ref.reserve(everyone, lens)
    keep = [-1, 16, 0, 2 ** 31 - 1, -2 ** 31, 3]
    eta.attn_cache_free(cache, ints(everyone), ints(keep))
    ref.free(everyone, keep)
    assert ref.lens == [0, 16, 0, 64, 0, 0]
    ref.check(cache)
    ref.consistent()
    assert eta.attn_status() == eta.ATTN_OK


@pytest.mark.parametrize("copy", [False, True])
def test_fork_of_a_sequence_that_lacks_pages(eta, copy):
    """A table entry of the parent that names no page: the child has none there either, and no page is lost."""
    cache = build(eta, [200, 53, 0, 0, 64, 0], 2, 16, 64, spare=25)
    cache.k.nan_to_num_(50.0)         # what a handed-out page would bring with it
    cache.v.nan_to_num_(50.0)
    for row, col, id_ in ((0, 3, -1), (0, 12, cache.pages), (1, 3, -7), (1, 0, 2 ** 31 - 1)):
        cache.ref_counts[int(cache.page_table[row, col])] = 0
        cache.page_table[row, col] = id_
    assert eta.attn_cache_fork(cache, ints([0, 1, 4]), ints([2, 3, 5]), copy=copy).tolist() == [1, 1, 1]
    assert eta.attn_status() == eta.ATTN_ERR_ARG
    assert cache.seq_lens.tolist() == [200, 53, 200, 53, 64, 64]
    table = cache.page_table.tolist()
    for parent, child in ((0, 2), (1, 3), (4, 5)):
        assert [0 <= x < cache.pages for x in table[parent]] == [x >= 0 for x in table[child]]
    names = [0] * cache.pages
    for row in table:
        for p in row:
            if 0 <= p < cache.pages:
                names[p] += 1
    assert names == cache.ref_counts.tolist()
    q = queries(3, 4, 64, BF16)
    a = eta.attn_paged_fwd(q, cache, 0, ints([0, 1, 4]), ints([0, 1, 2, 3]), max_q=1)
    b = eta.attn_paged_fwd(q, cache, 0, ints([2, 3, 5]), ints([0, 1, 2, 3]), max_q=1)
    assert eta.attn_status() == eta.ATTN_ERR_ARG
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("pages", [1, 16, 17, 16384, 16385, 70001])
def test_pools_of_any_size(eta, pages):
    """The scan over the reference counts: its steps, its tail, a pool that is used up."""
    rng = random.Random(pages)
    cols = min(pages, 3000)
    cache = eta.PagedCache.empty(1, pages, 1, 16, 32, 40, cols)
    cache.ref_counts.copy_(ints([1 if rng.random() < 0.7 else 0 for _ in range(pages)]))
    ref = Pages(cache)
    seqs = rng.sample(range(40), 30)
    for _ in range(3):
        add = [rng.randint(0, max(16 * pages // 60, 1)) for _ in seqs]
        assert eta.attn_cache_reserve(cache, ints(seqs), ints(add)).tolist() == ref.reserve(seqs, add)
        ref.check(cache)
    eta.attn_cache_free(cache, ints(seqs[:10]))
    ref.free(seqs[:10])
    # pages no table names go, so that compaction's table is whole
    cache.ref_counts.zero_()
    names = cache.page_table[cache.page_table >= 0].long()
    cache.ref_counts[names] = 1
    ref.refs = cache.ref_counts.tolist()
    _, _, live = eta.attn_cache_compact(cache)
    assert live.tolist() == [ref.compact()]
    ref.check(cache)


def test_long_lists(eta):
    """More list entries than the planning block has threads."""
    cache = eta.PagedCache.empty(1, 5000, 1, 16, 32, 2500, 4)
    ref = Pages(cache)
    rng = random.Random(3)
    seqs = rng.sample(range(2500), 2400)
    add = [rng.randint(0, 40) for _ in seqs]
    assert eta.attn_cache_reserve(cache, ints(seqs), ints(add)).tolist() == ref.reserve(seqs, add)
    ref.check(cache)
    eta.attn_cache_free(cache, ints(seqs[:1500]))
    ref.free(seqs[:1500])
    ref.check(cache)
    kids = [r for r in range(2500) if ref.lens[r] == 0][:1300]
    par = [rng.randrange(2500) for _ in kids]
    assert eta.attn_cache_fork(cache, ints(par), ints(kids)).tolist() == ref.fork(par, kids, False)
    ref.check(cache)


def test_needs_past_32_bits(eta):
    """Entries that together ask for more pages than 32 bits count, in rows that could hold them."""
    cols = 1 << 26
    cache = eta.PagedCache.empty(1, 5000, 1, 16, 32, 70, cols)
    seqs = list(range(69, 1, -1))
    add = [40] + [16 * cols] * (len(seqs) - 3) + [0, 5]
    granted = eta.attn_cache_reserve(cache, ints(seqs), ints(add)).tolist()
    assert granted == [1] + [0] * (len(seqs) - 3) + [1, 0]
    assert cache.seq_lens.tolist() == [0] * 69 + [40]
    assert cache.ref_counts.nonzero().flatten().tolist() == [0, 1, 2] and int(cache.ref_counts.sum()) == 3
    assert cache.page_table[69, :5].tolist() == [0, 1, 2, -1, -1]
    assert int((cache.page_table >= 0).sum()) == 3
    # a length at the row's end, and past it: cut to what the row can hold
    cache.seq_lens[5] = 16 * cols
    cache.seq_lens[6] = (1 << 31) - 1
    cache.page_table[5, cols - 1] = 7
    cache.ref_counts[7] = 1
    eta.attn_cache_free(cache, ints([5, 6]), ints([16 * cols - 1, (1 << 31) - 1]))
    assert cache.seq_lens[5:7].tolist() == [16 * cols - 1, 16 * cols]
    assert cache.ref_counts[7] == 1 and cache.page_table[5, cols - 1] == 7
    assert eta.attn_status() == eta.ATTN_OK


def test_refused_entries(eta):
    """Sequences named twice, out of range, too long for their row; children that hold tokens."""
    cache = new_cache(eta, 12, 16, 6, 4)
    ref = Pages(cache)

    def status(code):
        assert eta.attn_status() == code

    assert eta.attn_cache_reserve(cache, ints([0, 1, 0, 7, -1, 2]), ints([20, 65, 5, 5, 5, 64])).tolist() == [1, 0, 0, 0, 0, 1]
    status(eta.ATTN_ERR_ARG)
    ref.reserve([0, 1, 0, 7, -1, 2], [20, 65, 5, 5, 5, 64])
    ref.check(cache)
    assert eta.attn_cache_reserve(cache, ints([3, 4, 5]), ints([64, 64, 0])).tolist() == ref.reserve([3, 4, 5], [64, 64, 0])
    ref.check(cache)
    status(eta.ATTN_OK)
    assert eta.attn_cache_reserve(cache, ints([5]), ints([-3])).tolist() == [0]
    status(eta.ATTN_ERR_ARG)
    # the child holds tokens; the child is named twice; out of range; a child of a child that is empty before the call
    par, kid = [0, 2, 0, 0, 9, 1], [2, 1, 1, 8, 4, 5]
    assert eta.attn_cache_fork(cache, ints(par), ints(kid)).tolist() == ref.fork(par, kid, False)
    status(eta.ATTN_ERR_ARG)
    ref.check(cache)
    assert ref.lens[1] == 64 and ref.lens[5] == 0
    eta.attn_cache_free(cache, ints([1, 1, 77]), ints([3, 0, 0]))
    status(eta.ATTN_ERR_ARG)
    ref.free([1, 1, 77], [3, 0, 0])
    ref.check(cache)
    assert ref.lens[1] == 3
    # an entry that names no page of the pool
    cache.page_table[0, 1] = 12
    eta.attn_cache_free(cache, ints([0]))
    status(eta.ATTN_ERR_ARG)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("layout", ["head", "token", "side", "layers"])
@pytest.mark.parametrize("d,heads", [(32, 1), (64, 5), (96, 2), (128, 3)])
def test_append(eta, dtype, layout, d, heads):
    lens, new = [3, 40, 16, 33, 5, 70], [3, 17, 1, 0, 5, 70]
    cache = build(eta, lens, heads, 16, d, dtype, layout, layers=2)
    T = sum(new) + 3
    kv = queries(T, 2 * heads, d, dtype)
    kn, vn = kv[:, :heads], kv[:, heads:]
    order = [2, 0, 5, 3, 1, 4]
    qs = [1 + x for x in starts([new[r] for r in order])]
    want = [cache.k.clone(), cache.v.clone()]
    table = cache.page_table.tolist()
    for i, r in enumerate(order):
        for t in range(qs[i], qs[i + 1]):
            pos = lens[r] - new[r] + t - qs[i]
            want[0][1, table[r][pos // 16], :, pos % 16] = kn[t]
            want[1][1, table[r][pos // 16], :, pos % 16] = vn[t]
    eta.attn_cache_append(cache, 1, kn, vn, ints(order), ints(qs))
    assert eta.attn_status() == eta.ATTN_OK
    assert torch.equal(cache.k.nan_to_num(9.0), want[0].nan_to_num(9.0))
    assert torch.equal(cache.v.nan_to_num(9.0), want[1].nan_to_num(9.0))


@pytest.mark.parametrize("pad", [2, 1500])
def test_padded_lists(eta, pad):
    """Entries without tokens before and behind the others, of the same sequences."""
    cache = new_cache(eta, 40, 16, 6, 4)
    ref = Pages(cache)
    front, back = [i % 3 for i in range(pad)], [2] * pad
    seqs, add = front + [0, 1, 2] + back, [0] * pad + [20, 5, 33] + [0] * pad
    for _ in range(2):
        add[pad + 2] -= 10
        assert eta.attn_cache_reserve(cache, ints(seqs), ints(add)).tolist() == ref.reserve(seqs, add) == [1] * len(seqs)
        ref.check(cache)
    kn = queries(7, cache.heads, cache.d, cache.dtype)
    want, table = cache.k.clone(), cache.page_table.tolist()
    for i, (s, n) in enumerate([(0, 2), (1, 4), (2, 1)]):
        for t in range(n):
            at = ref.lens[s] - n + t
            want[0, table[s][at // 16], :, at % 16] = kn[[0, 2, 6][i] + t]
    qs = [0] * (pad + 1) + [2, 6] + [7] * (pad + 1)
    eta.attn_cache_append(cache, 0, kn, kn, ints(seqs), ints(qs))
    assert eta.attn_status() == eta.ATTN_OK
    assert torch.equal(cache.k.nan_to_num(9.0), want.nan_to_num(9.0))


def test_append_bad_places(eta):
    """Tokens without a place are dropped and reported; the others are written."""
    cache = build(eta, [20, 4, 30], 2, 16, 64)
    cache.page_table[2, 1] = cache.pages + 1
    kn = queries(30, 2, 64, BF16)
    want = cache.k.clone()
    table = cache.page_table.tolist()
    qs = [0, 2, 8, 10, 14, 16]           # 6 new tokens of a sequence of 4; row 7; row 2's page 1; row 0 again
    for t in range(2):
        want[0, table[0][(18 + t) // 16], :, (18 + t) % 16] = kn[t]
    for t in range(4):
        want[0, table[1][0], :, t] = kn[4 + t]
    eta.attn_cache_append(cache, 0, kn, kn, ints([0, 1, 7, 2, 0]), ints(qs))
    assert eta.attn_status() == eta.ATTN_ERR_ARG
    assert torch.equal(cache.k.nan_to_num(9.0), want.nan_to_num(9.0))


@pytest.mark.parametrize("dtype,token_major", [(BF16, False), (F32, True)])
def test_a_server_for_a_while(eta, dtype, token_major):
    """Prompts in chunks, decoding, forks that go their own ways, rejected
    tokens, sequences that leave, compaction: after every step each sequence's
    attention is that of its own tokens, kept beside the cache."""
    rng = random.Random(11)
    layers, heads, g, d, page = 2, 2, 4, 64, 16
    cache = new_cache(eta, 90, page, 10, 30, layers, heads, d, dtype, token_major)
    book = {}        # row -> per layer (k, v) [tokens, heads, d], what the sequence should hold

    def step(rows, new):
        qs = ints(starts(new))
        got = eta.attn_cache_reserve(cache, ints(rows), ints(new))
        assert got.tolist() == [1] * len(rows)
        for layer in range(layers):
            kn = torch.randn((sum(new), heads, d), device="cuda").to(dtype)
            vn = torch.randn((sum(new), heads, d), device="cuda").to(dtype)
            for i, r in enumerate(rows):
                a, b = sum(new[:i]), sum(new[:i + 1])
                k0, v0 = book.setdefault(r, [(kn[:0], vn[:0])] * layers)[layer]
                book[r] = list(book[r])
                book[r][layer] = (torch.cat([k0, kn[a:b]]), torch.cat([v0, vn[a:b]]))
            eta.attn_cache_append(cache, layer, kn, vn, ints(rows), qs)
            q = torch.randn((sum(new), heads * g, d), device="cuda").to(dtype)
            o, lse = eta.attn_paged_fwd(q, cache, layer, ints(rows), qs, max_q=max(new))
            check_attention(q, cache, layer, ints(rows), qs, True, d ** -0.5, o, lse)

    def check():
        lens = cache.seq_lens.tolist()
        for r in range(10):
            n = len(book[r][0][0]) if r in book else 0
            assert lens[r] == n
            for layer in range(layers if n else 0):
                ids = cache.page_table[r, :-(-n // page)].long()
                for pool, want in zip((cache.k, cache.v), book[r][layer]):
                    assert torch.equal(pool[layer, ids].transpose(1, 2).reshape(-1, heads, d)[:n], want)
        assert eta.attn_status() == eta.ATTN_OK

    step([0, 1, 2], [40, 17, 100])
    step([0, 1, 2], [33, 1, 60])
    check()
    assert eta.attn_cache_fork(cache, ints([0, 0, 2]), ints([3, 4, 5])).tolist() == [1, 1, 1]
    book[3], book[4], book[5] = list(book[0]), list(book[0]), list(book[2])
    check()
    for _ in range(18):
        step([0, 1, 2, 3, 4, 5], [1] * 6)
    check()
    keep = {r: len(book[r][0][0]) - rng.randint(0, 3) for r in (1, 3, 5)}
    eta.attn_cache_free(cache, ints(list(keep)), ints(list(keep.values())))
    for r, n in keep.items():
        book[r] = [(k[:n], v[:n]) for k, v in book[r]]
    step([1, 3, 5, 0], [5, 2, 3, 1])
    check()
    eta.attn_cache_free(cache, ints([0, 2]))
    del book[0], book[2]
    check()
    _, _, live = eta.attn_cache_compact(cache)
    n_live = int(live)
    assert (cache.ref_counts[:n_live] > 0).all() and (cache.ref_counts[n_live:] == 0).all()
    check()
    assert eta.attn_cache_fork(cache, ints([4]), ints([0]), copy=True).tolist() == [1]
    book[0] = list(book[4])
    step([0, 4, 5, 1], [20, 1, 1, 7])
    check()
