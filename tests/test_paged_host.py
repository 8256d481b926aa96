"""The paged cache on the host: argument rejection before any launch, and the
index arithmetic of csrc/paged_index.h (compiled here with the host compiler)
checked exhaustively, bad table entries and token ranges included."""
import bisect
import ctypes
import os
import random
import subprocess

import pytest

from test_abi_host import ROOT, lib  # noqa: F401  (the fixture builds and loads the library)

vp, ci, ll, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_longlong, ctypes.c_size_t


class CacheT(ctypes.Structure):
    _fields_ = [("K", vp), ("V", vp), ("page_table", vp), ("seq_lens", vp), ("ref_counts", vp)] + \
               [(n, ci) for n in ("dtype", "layers", "pages", "heads", "page_size", "d", "seqs", "max_pages")] + \
               [(n, ll) for n in ("layer_stride", "page_stride", "head_stride", "slot_stride")]


def cache(**kw):
    a = dict(K=256, V=512, page_table=256, seq_lens=256, ref_counts=256, dtype=1, layers=2, pages=10, heads=4, page_size=16,
             d=64, seqs=3, max_pages=5)
    a.update(kw)
    block = a["heads"] * a["page_size"] * a["d"]
    a.setdefault("page_stride", block)
    a.setdefault("layer_stride", block * a["pages"])
    a.setdefault("head_stride", a["page_size"] * a["d"])
    a.setdefault("slot_stride", a["d"])
    return CacheT(**a)


BAD_CACHES = [
    (dict(K=None), -1), (dict(V=None), -1), (dict(page_table=None), -1), (dict(seq_lens=None), -1),
    (dict(ref_counts=None), -1), (dict(K=264), -1), (dict(ref_counts=260), -1), (dict(page_table=258), -1),
    (dict(dtype=2), -2), (dict(dtype=9), -1), (dict(layers=0), -1), (dict(pages=-1), -1), (dict(heads=0), -1),
    (dict(seqs=0), -1), (dict(max_pages=0), -1), (dict(d=48), -2), (dict(d=160), -2), (dict(page_size=8), -2),
    (dict(page_size=48), -2), (dict(page_size=512), -2), (dict(max_pages=1 << 28), -1),
    (dict(head_stride=64, slot_stride=64), -1),               # neither head by head nor token by token
    (dict(page_stride=4 * 16 * 64 - 8), -1),                  # pages overlap
    (dict(page_stride=4 * 16 * 64 + 4), -1),                  # not a multiple of 16 bytes
    (dict(layer_stride=4 * 16 * 64 * 9), -1),                 # layers overlap
    (dict(layer_stride=4 * 16 * 64, page_stride=4 * 16 * 64), -1),
    (dict(page_stride=-4 * 16 * 64), -1),
    (dict(max_pages=(1 << 26) + 1), -1),                      # more than 2^30 tokens
    (dict(pages=(1 << 31) - 1, page_stride=1 << 40, layer_stride=1 << 41), -1),   # layers overlap, past 64 bits
]


def test_the_longest_sequence_a_cache_may_hold(lib):  # noqa: F811
    assert paged(lib, ctypes.byref(cache(max_pages=1 << 26)), T=0) == 0
    assert paged(lib, ctypes.byref(cache(max_pages=1 << 22, page_size=256)), T=0) == 0


def test_the_most_tokens_of_a_call(lib):  # noqa: F811
    one, most = ctypes.byref(cache(heads=1)), 1 << 30
    kw = dict(Hq=1, qt=64, ot=64, n=0)
    assert paged(lib, one, T=most, **kw) == 0 and paged(lib, one, T=most + 1, **kw) == -1
    a = lib.attn_cache_append
    assert a(one, ci(0), vp(256), vp(256), ll(64), ll(64), ci(most), None, vp(256), ci(0), None) == 0
    assert a(one, ci(0), vp(256), vp(256), ll(64), ll(64), ci(most + 1), None, vp(256), ci(1), None) == -1
    # rows of O that do not overlap only where 64 bits overflow
    wide = ctypes.byref(cache())
    assert paged(lib, wide, T=(1 << 27) + 1, max_q=1, Hq=8, oh=1 << 36, ot=1 << 37) == -1


@pytest.mark.parametrize("bad,code", BAD_CACHES)
def test_every_entry_rejects_a_bad_cache(lib, bad, code):  # noqa: F811
    c = ctypes.byref(cache(**bad))
    p, big = vp(256), sz(1 << 40)
    assert lib.attn_cache_reserve(c, p, p, ci(1), p, p, big, None) == code
    assert lib.attn_cache_free(c, p, p, ci(1), None) == code
    assert lib.attn_cache_fork(c, p, p, ci(1), ci(0), p, p, big, None) == code
    assert lib.attn_cache_compact(c, p, p, p, p, big, None) == code
    assert lib.attn_cache_append(c, ci(0), p, p, ll(256), ll(64), ci(4), p, p, ci(1), None) == code
    assert paged(lib, c) == code
    assert paged(lib, None) == -1


def paged(lib, c, **kw):  # noqa: F811
    a = dict(layer=0, Q=vp(256), O=vp(256), LSE=None, qt=512, qh=64, ot=512, oh=64, T=4, Hq=8, seqs=None, qs=vp(256), n=1,
             max_q=4, causal=1, scale=0.125, ws=vp(256), ws_bytes=1 << 40)
    a.update(kw)
    f = lib.attn_paged_fwd
    f.restype = ci
    f.argtypes = [vp, ci, vp, vp, vp, ll, ll, ll, ll, ci, ci, vp, vp, ci, ci, ci, ctypes.c_float, vp, sz, vp]
    return f(c, a["layer"], a["Q"], a["O"], a["LSE"], a["qt"], a["qh"], a["ot"], a["oh"], a["T"], a["Hq"], a["seqs"], a["qs"],
             a["n"], a["max_q"], a["causal"], a["scale"], a["ws"], a["ws_bytes"], None)


def test_paged_fwd_rejection(lib):  # noqa: F811
    c = ctypes.byref(cache())
    f = lib.attn_paged_workspace_size
    f.restype, f.argtypes = sz, [ci] * 5
    need = f(8, 4, 4, 64, 1)
    assert need > 0
    for bad in ((0, 4, 4, 64, 1), (8, 0, 4, 64, 1), (8, 3, 4, 64, 1), (8, 4, 0, 64, 1), (8, 4, 4, 48, 1), (8, 4, 4, 64, 2),
                (4 * 65, 4, 4, 64, 1)):
        assert f(*bad) == 0
    assert paged(lib, c, layer=2) == -1 and paged(lib, c, layer=-1) == -1
    assert paged(lib, c, Q=None) == -1 and paged(lib, c, O=None) == -1 and paged(lib, c, qs=None) == -1
    assert paged(lib, c, Q=vp(264)) == -1 and paged(lib, c, LSE=vp(258)) == -1 and paged(lib, c, seqs=vp(257)) == -1
    assert paged(lib, c, Hq=6) == -1 and paged(lib, c, Hq=4 * 65, ot=4 * 65 * 64) == -2
    assert paged(lib, c, T=-1) == -1 and paged(lib, c, n=-1) == -1
    assert paged(lib, c, max_q=0) == -1 and paged(lib, c, max_q=5) == -1
    assert paged(lib, c, causal=2) == -1
    for s in (0.0, -1.0, float("nan"), float("inf")):
        assert paged(lib, c, scale=s) == -1
    assert paged(lib, c, qt=516) == -1 and paged(lib, c, qh=-64) == -1
    assert paged(lib, c, oh=32) == -1 and paged(lib, c, ot=64, oh=64) == -1      # rows of O overlap
    one = ctypes.byref(cache(heads=1))
    assert paged(lib, one, Hq=1, qh=3, oh=5, qt=64, ot=64, T=0) == 0            # strides of a dimension of one: ignored
    assert paged(lib, c, T=0, qt=4) == -1
    assert paged(lib, c, ws=None) == -3 and paged(lib, c, ws_bytes=need - 1) == -3 and paged(lib, c, ws=vp(264)) == -3
    assert paged(lib, c, T=0, max_q=0) == 0 and paged(lib, c, n=0) == 0          # nothing to do


def test_the_largest_scale(lib):  # noqa: F811
    """Scores are kept in powers of two: scale * log2(e) must be finite in float32."""
    c = ctypes.byref(cache())
    for scale, code in ((2.35e38, 0), (2.36e38, -1), (3.4e38, -1), (1e-30, 0)):
        assert paged(lib, c, scale=scale, n=0) == code, scale


def test_cache_entries_rejection(lib):  # noqa: F811
    c = ctypes.byref(cache())
    p, big = vp(256), sz(1 << 40)
    f = lib.attn_cache_workspace_size
    f.restype, f.argtypes = sz, [ci, ci]
    assert f(0, 1) == 0 and f(10, -1) == 0
    need = sz(f(10, 4))
    less = sz(f(10, 4) - 1)
    # the largest lists: a plan holds three integers an entry and one a page, compaction three a page
    assert f(10, 100000) >= (3 * 100000 + 10) * 4 and f(100000, 1) >= 3 * 100000 * 4
    r = lib.attn_cache_reserve
    assert r(c, None, p, ci(4), p, p, need, None) == -1 and r(c, p, None, ci(4), p, p, need, None) == -1
    assert r(c, p, p, ci(4), None, p, need, None) == -1 and r(c, p, p, ci(-1), p, p, need, None) == -1
    assert r(c, p, p, ci(4), p, None, need, None) == -3 and r(c, p, p, ci(4), p, p, less, None) == -3
    assert r(c, p, p, ci(4), p, vp(264), need, None) == -3 and r(c, vp(258), p, ci(4), p, p, need, None) == -1
    assert r(c, p, p, ci(0), p, p, need, None) == 0
    assert lib.attn_cache_free(c, None, None, ci(1), None) == -1
    assert lib.attn_cache_free(c, p, vp(258), ci(1), None) == -1
    assert lib.attn_cache_free(c, p, None, ci(-1), None) == -1
    assert lib.attn_cache_free(c, p, None, ci(0), None) == 0
    k = lib.attn_cache_fork
    assert k(c, None, p, ci(4), ci(0), p, p, big, None) == -1 and k(c, p, None, ci(4), ci(0), p, p, big, None) == -1
    assert k(c, p, p, ci(4), ci(2), p, p, big, None) == -1 and k(c, p, p, ci(4), ci(0), None, p, big, None) == -1
    assert k(c, p, p, ci(4), ci(0), p, p, less, None) == -3 and k(c, p, p, ci(0), ci(1), p, p, big, None) == 0
    m = lib.attn_cache_compact
    assert m(c, None, p, p, p, big, None) == -1 and m(c, p, None, p, p, big, None) == -1 and m(c, p, p, None, p, big, None) == -1
    assert m(c, p, vp(260), p, p, big, None) == -1 and m(c, p, p, p, None, big, None) == -3
    assert m(c, p, p, p, p, sz(f(10, 0) - 1), None) == -3
    a = lib.attn_cache_append
    assert a(c, ci(2), p, p, ll(256), ll(64), ci(4), p, p, ci(1), None) == -1
    assert a(c, ci(0), None, p, ll(256), ll(64), ci(4), p, p, ci(1), None) == -1
    assert a(c, ci(0), p, vp(264), ll(256), ll(64), ci(4), p, p, ci(1), None) == -1
    assert a(c, ci(0), p, p, ll(257), ll(64), ci(4), p, p, ci(1), None) == -1
    assert a(c, ci(0), p, p, ll(256), ll(-64), ci(4), p, p, ci(1), None) == -1
    assert a(c, ci(0), p, p, ll(256), ll(64), ci(-4), p, p, ci(1), None) == -1
    assert a(c, ci(0), p, p, ll(256), ll(64), ci(4), p, None, ci(1), None) == -1
    assert a(c, ci(0), p, p, ll(256), ll(64), ci(0), p, p, ci(1), None) == 0
    assert a(c, ci(0), p, p, ll(256), ll(64), ci(4), p, p, ci(0), None) == 0


def test_the_longest_list(lib):  # noqa: F811
    """Entry numbers, and the ends of blocks of entries that reach past them, stay inside 32 bits."""
    c, p, big = ctypes.byref(cache(max_pages=1)), vp(256), sz(1 << 62)
    f = lib.attn_cache_workspace_size
    f.restype, f.argtypes = sz, [ci, ci]
    assert f(10, 1 << 20) >= (3 << 20) * 4
    for n in ((1 << 20) + 1, 1 << 30, (1 << 31) - 1024, (1 << 31) - 1):
        assert f(10, n) == 0
        assert lib.attn_cache_reserve(c, p, p, ci(n), p, p, big, None) == -1
        assert lib.attn_cache_free(c, p, p, ci(n), None) == -1
        assert lib.attn_cache_fork(c, p, p, ci(n), ci(0), p, p, big, None) == -1
        assert lib.attn_cache_append(c, ci(0), p, p, ll(256), ll(64), ci(0), p, p, ci(n), None) == -1
        assert paged(lib, c, n=n, T=0) == -1
    assert paged(lib, c, n=1 << 20, T=0) == 0


def test_accepted_layouts(lib):  # noqa: F811
    """Layouts the header allows pass the checks (n = 0: nothing is launched)."""
    p = vp(256)
    block = 4 * 16 * 64
    for kw in (dict(), dict(head_stride=64, slot_stride=256),                       # token by token
               dict(page_stride=2 * block, layer_stride=2 * block * 10),            # K and V of a page side by side
               dict(page_stride=2 * block, layer_stride=block),                     # layers inside a page
               dict(heads=1, head_stride=8, slot_stride=64), dict(layers=1, layer_stride=0), dict(pages=1, page_stride=0)):
        assert lib.attn_cache_free(ctypes.byref(cache(**kw)), p, None, ci(0), None) == 0, kw


# ---------------------------------------------------------------------------
# index arithmetic
# ---------------------------------------------------------------------------
SHIM = r"""
#include "paged_index.h"
using namespace eta;
extern "C" {
struct G { const int *table, *lens, *seqs, *qs; int v[15]; };
static PagedGeom geom(const G *g) {
    PagedGeom m;
    m.page_table = g->table; m.seq_lens = g->lens; m.seqs = g->seqs; m.q_start = g->qs;
    const int *v = g->v;
    m.n = v[0]; m.rows = v[1]; m.max_pages = v[2]; m.pages = v[3]; m.page_size = v[4]; m.T = v[5]; m.max_q = v[6];
    m.heads = v[7]; m.g = v[8]; m.causal = v[9]; m.tpu = v[10]; m.tk = v[11]; m.unit_cost = v[12]; m.min_share = v[13];
    paged_derive(m);
    return m;
}
int entry(const G *g, int i, int *out) {
    PagedEntry e; const bool ok = paged_entry(geom(g), i, e);
    out[0] = e.seq; out[1] = e.q0; out[2] = e.nq; out[3] = e.len;
    return ok;
}
int page(const G *g, int seq, int col) { return paged_page(geom(g), seq, col); }
// the shares of `ctas` CTAs, as each finds its own: [c] = i, h, u, tile of its begin
int shares(const G *g, int ctas, int *out) {
    PagedGeom m = geom(g);
    long long W = 0;
    PagedEntry e;
    for (int i = 0; i < m.n; ++i) { paged_entry(m, i, e); W += paged_entry_work(m, e); }
    const int s = paged_shares(m, W, ctas);
    for (int c = 0; c <= ctas; ++c) {
        const long long x = paged_share_begin(W, c, s);
        PagedPos p{m.n, 0, 0, 0};
        long long at = 0;
        for (int i = 0; i < m.n; ++i) {
            paged_entry(m, i, e);
            const long long w = paged_entry_work(m, e);
            if (x >= at && x < at + w) p = paged_locate(m, e, i, x - at);
            at += w;
        }
        out[4 * c] = p.i; out[4 * c + 1] = p.h; out[4 * c + 2] = p.u; out[4 * c + 3] = p.tile;
    }
    return s;
}
// every unit in order: (i, h, u, tiles)
int units(const G *g, int *out, int cap) {
    PagedGeom m = geom(g);
    int k = 0;
    PagedEntry e;
    for (int i = 0; i < m.n; ++i) {
        paged_entry(m, i, e);
        if (e.nq == 0) continue;
        PagedPos p{i, 0, 0, 0};
        while (p.i == i && k < cap) {
            out[4 * k] = p.i; out[4 * k + 1] = p.h; out[4 * k + 2] = p.u; out[4 * k + 3] = paged_tiles(m, e, p.u);
            ++k;
            paged_next_unit(m, e, p);
        }
    }
    return k;
}
int token(const G *g, int r) { return paged_token(geom(g), r); }
int visible(const G *g, int i, int t) { PagedEntry e; paged_entry(geom(g), i, e); return paged_visible(geom(g), e, t); }
}
"""


class G(ctypes.Structure):
    _fields_ = [("table", vp), ("lens", vp), ("seqs", vp), ("qs", vp), ("v", ci * 15)]


@pytest.fixture(scope="module")
def shim(tmp_path_factory):
    d = tmp_path_factory.mktemp("paged_index")
    src, out = d / "shim.cpp", d / "shim.so"
    src.write_text(SHIM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-shared", "-fPIC", "-I",
                    os.path.join(ROOT, "exact_tiled_attention_17_gb300", "csrc"), str(src), "-o", str(out)], check=True)
    return ctypes.CDLL(str(out))


def geom(lens, seqs, qs, T, max_q, heads=2, g=4, causal=1, tpu=4, tk=64, unit_cost=64, min_share=128, max_pages=64, pages=50,
         page_size=16, table=None):
    ints = lambda v: (ci * len(v))(*v)  # noqa: E731
    keep = [ints(lens), ints(seqs), ints(qs), ints(table if table is not None else [0] * (len(lens) * max_pages))]
    a = G(ctypes.cast(keep[3], vp), ctypes.cast(keep[0], vp), ctypes.cast(keep[1], vp), ctypes.cast(keep[2], vp),
          (ci * 15)(len(qs) - 1, len(lens), max_pages, pages, page_size, T, max_q, heads, g, causal, tpu, tk, unit_cost,
                    min_share, 0))
    a.keep = keep
    return a


@pytest.mark.parametrize("seed", range(60))
def test_shares_cover_every_tile_once(shim, seed):
    """Whatever the lengths, the CTAs' shares put together are all tiles of all
    units, each once and in order, and no share holds two parts of which the
    first does not begin its unit (a CTA has one slot for such a part)."""
    rng = random.Random(seed)
    n, rows = rng.randint(1, 9), 12
    lens = [rng.choice([0, 1, 63, 64, 65, rng.randint(0, 1000), 1024]) for _ in range(rows)]
    qs = [0]
    for _ in range(n):
        qs.append(qs[-1] + rng.choice([0, 1, 2, 5, rng.randint(0, 40), 300]))
    seqs = [rng.randrange(-1, rows + 1) if rng.random() < 0.1 else rng.randrange(rows) for _ in range(n)]
    tk, ctas = rng.choice([32, 64, 128]), rng.choice([1, 2, 7, 152, 304, 640])
    a = geom(lens, seqs, qs, qs[-1], max(max(b - c for b, c in zip(qs[1:], qs)), 1), heads=rng.choice([1, 3, 8]), g=3,
             causal=rng.randint(0, 1), tpu=rng.choice([1, 4, 5, 21, 64]), tk=tk, unit_cost=rng.choice([1, 64, 500]),
             min_share=rng.choice([1, tk, 4 * tk]))
    cap = 100000
    u = (ci * (4 * cap))()
    k = shim.units(ctypes.byref(a), u, cap)
    assert k < cap
    line = [(tuple(u[4 * x:4 * x + 3]), t) for x in range(k) for t in range(u[4 * x + 3])]
    out = (ci * (4 * (ctas + 1)))()
    s = shim.shares(ctypes.byref(a), ctas, out)
    assert 1 <= s <= ctas
    # a border may lie before an entry without tokens: it stands for the first tile after it
    marks = [bisect.bisect_left(line, (tuple(out[4 * c:4 * c + 3]), out[4 * c + 3])) for c in range(ctas + 1)]
    for c in range(ctas + 1):
        key, t = tuple(out[4 * c:4 * c + 3]), out[4 * c + 3]
        assert t == 0 or (key, t) in line[marks[c]:marks[c] + 1], (key, t)
    assert marks == sorted(marks)
    if line:
        assert marks[0] == 0
    assert marks[-1] == len(line)
    for c in range(ctas):
        part = line[marks[c]:marks[c + 1]]
        heads = {key for key, t in part if t == 0}
        assert len({key for key, _ in part if key not in heads}) <= 1   # at most one part that does not begin its unit


@pytest.mark.parametrize("causal", [0, 1])
def test_visible_keys(shim, causal):
    for n in (0, 1, 5, 100):
        for nq in (1, 3, 7):
            a = geom([n], [0], [0, nq], nq, nq, causal=causal)
            for t in range(nq):
                want = sum(1 for j in range(n) if j <= n - nq + t) if causal else n
                assert shim.visible(ctypes.byref(a), 0, t) == want


def test_rows_to_tokens(shim):
    for g in range(1, 65):
        a = geom([1], [0], [0, 1], 1, 1, g=g)
        assert [shim.token(ctypes.byref(a), r) for r in range(256)] == [r // g for r in range(256)]


def test_bad_entries_are_left_out(shim):
    out = (ci * 4)()
    lens = [10, -5, 5000, 20]
    for seqs, qs, T, max_q, i, ok, want in [
            ([0], [0, 3], 3, 3, 0, 1, [0, 0, 3, 10]),
            ([4], [0, 3], 3, 3, 0, 0, [0, 0, 0, 0]),        # no such row
            ([-1], [0, 3], 3, 3, 0, 0, [0, 0, 0, 0]),
            ([1], [0, 3], 3, 3, 0, 0, [1, 0, 3, 0]),        # a negative length: no keys
            ([2], [0, 3], 3, 3, 0, 0, [2, 0, 3, 64 * 16]),  # longer than the table row holds
            ([0], [0, 4], 3, 4, 0, 0, [0, 0, 0, 0]),        # past the rows of Q
            ([0], [-1, 2], 3, 3, 0, 0, [0, 0, 0, 0]),
            ([0, 3], [2, 1, 3], 3, 3, 0, 0, [0, 0, 0, 0]),  # decreasing
            ([0], [0, 3], 3, 2, 0, 0, [0, 0, 0, 0]),        # more than max_q
            ([0], [2147483600, 2147483647], 3, 3, 0, 0, [0, 0, 0, 0])]:
        a = geom(lens, seqs, qs, T, max_q)
        assert shim.entry(ctypes.byref(a), i, out) == ok and list(out) == want, (seqs, qs)


def test_granted_lists_are_checked_and_null_is_none(lib):  # noqa: F811
    c = ctypes.byref(cache())
    p = vp(256)
    a, f = lib.attn_cache_append_granted, lib.attn_paged_fwd_granted
    a.argtypes = [vp, ci, vp, vp, ll, ll, ci, vp, vp, vp, ci, vp]
    f.argtypes = [vp, ci, vp, vp, vp, ll, ll, ll, ll, ci, ci, vp, vp, vp, ci, ci, ci, ctypes.c_float, vp, sz, vp]
    for g, T, n, code in ((vp(258), 4, 1, -1), (vp(257), 4, 1, -1), (p, 4, 0, 0), (None, 4, 0, 0), (p, 0, 1, 0)):
        assert a(c, 0, p, p, 256, 64, T, p, p, g, n, None) == code
        assert f(c, 0, p, p, None, 512, 64, 512, 64, T, 8, p, p, g, n, 4, 1, 0.125, p, 1 << 40, None) == code
    assert a(c, 0, None, p, 256, 64, 4, p, p, p, 1, None) == -1
    assert f(c, 0, p, p, None, 512, 64, 512, 64, 4, 8, p, p, p, 1, 4, 1, 0.125, None, 1 << 40, None) == -3


def test_entries_without_room_take_no_part(tmp_path):
    """granted = 0: no tokens, no work, nothing to report, whatever else the entry says."""
    src, out = tmp_path / "granted.cpp", tmp_path / "granted.so"
    src.write_text(r"""
#include "paged_index.h"
using namespace eta;
extern "C" int entry(const int *lens, const int *seqs, const int *qs, const int *granted, int n, int i, int *out) {
    PagedGeom m;
    m.page_table = nullptr; m.seq_lens = lens; m.seqs = seqs; m.q_start = qs; m.granted = granted;
    m.n = n; m.rows = 2; m.max_pages = 4; m.pages = 9; m.page_size = 16; m.T = 20; m.max_q = 9; m.heads = 2; m.g = 3;
    m.causal = 1; m.tpu = 4; m.tk = 64; m.unit_cost = 64; m.min_share = 128;
    paged_derive(m);
    PagedEntry e;
    const bool ok = paged_entry(m, i, e);
    out[0] = e.seq; out[1] = e.q0; out[2] = e.nq; out[3] = e.len; out[4] = paged_entry_work(m, e) > 0;
    return ok;
}
""")
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-shared", "-fPIC", "-I",
                    os.path.join(ROOT, "exact_tiled_attention_17_gb300", "csrc"), str(src), "-o", str(out)], check=True)
    f, got = ctypes.CDLL(str(out)).entry, (ci * 5)()
    ints = lambda v: (ci * len(v))(*v)  # noqa: E731
    lens, seqs, qs = ints([10, 20]), ints([0, 1, 7, 0]), ints([0, 3, 5, 8, 30])
    for granted, i, ok, want in ((None, 0, 1, [0, 0, 3, 10, 1]), ([1, 1, 1, 1], 1, 1, [1, 3, 2, 20, 1]),
                                 ([0, 1, 0, 0], 0, 1, [0, 0, 0, 0, 0]), ([0, 1, 0, 0], 1, 1, [1, 3, 2, 20, 1]),
                                 ([0, 1, 0, 0], 2, 1, [0, 0, 0, 0, 0]), ([1, 1, 1, 1], 2, 0, [0, 0, 0, 0, 0]),
                                 ([0, 1, 0, 0], 3, 1, [0, 0, 0, 0, 0]), ([0, 0, 0, 5], 3, 0, [0, 0, 0, 0, 0])):
        assert f(lens, seqs, qs, ints(granted) if granted else None, 4, i, got) == ok
        assert list(got) == want, (granted, i)


def test_bad_pages_are_not_followed(shim):
    table = [0, 49, 50, -1, -2147483648, 2147483647, 7, 8]
    a = geom([128], [0], [0, 1], 1, 1, max_pages=8, table=table)
    got = [shim.page(ctypes.byref(a), 0, c) for c in range(-1, 9)]
    assert got == [-1, 0, 49, -1, -1, -1, -1, 7, 8, -1]


def test_widest_work_does_not_overflow(shim):
    """A long cache, many heads and entries: the line is longer than 2^32."""
    lens = [2_000_000_000 // 16 * 16] * 64
    qs = [64 * x for x in range(65)]
    a = geom(lens, list(range(64)), qs, qs[-1], 64, heads=64, g=1, causal=1, tpu=1, tk=64, max_pages=(1 << 31) // 16 - 1,
             table=[0])
    out = (ci * (4 * 305))()
    assert shim.shares(ctypes.byref(a), 304, out) == 304
    marks = [tuple(out[4 * c:4 * c + 4]) for c in range(305)]
    assert marks == sorted(marks) and marks[0] == (0, 0, 0, 0) and marks[-1][0] == 64
    # equal shares: every CTA holds 64 * 64 * 64 / 304 units, give or take the rounding
    flat = [(m[0] * 64 + m[1]) * 64 + m[2] for m in marks]
    assert max(b - a_ for a_, b in zip(flat, flat[1:])) - min(b - a_ for a_, b in zip(flat, flat[1:])) <= 2
