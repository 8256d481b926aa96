"""Host side of the 4-bit paged cache, the rotated append and reading back:
arguments are rejected before any launch (no GPU is needed)."""
import ctypes

import pytest

from test_abi_host import lib  # noqa: F401  (the fixture builds and loads the library)
from test_paged_host import CacheT, ci, ll, paged, sz, vp

E2M1 = 3


def cache(**kw):
    a = dict(K=256, V=512, page_table=256, seq_lens=256, ref_counts=256, dtype=E2M1, layers=2, pages=10, heads=4, page_size=16,
             d=64, seqs=3, max_pages=5)
    a.update(kw)
    head = a["page_size"] * a["d"] * 9 // 16 if a["dtype"] == E2M1 else a["page_size"] * a["d"]
    a.setdefault("page_stride", a["heads"] * head)
    a.setdefault("layer_stride", a["heads"] * head * a["pages"])
    a.setdefault("head_stride", head)
    a.setdefault("slot_stride", a["d"] // 2 if a["dtype"] == E2M1 else a["d"])
    return CacheT(**a)


class RotationT(ctypes.Structure):
    _fields_ = [("table", vp), ("positions", vp), ("rows", ci), ("dims", ci), ("neighbours", ci)]


def rotated(lib, c, **kw):  # noqa: F811
    a = dict(layer=0, K=256, V=512, ts=256, hs=64, Q=256, Qout=512, Hq=8, qt=512, qh=64, ot=512, oh=64, T=4, seqs=None, qs=256,
             granted=None, n=2, table=256, positions=None, rows=100, dims=64, neighbours=0, rotation=True)
    a.update(kw)
    f = lib.attn_cache_append_rotated
    f.restype = ci
    f.argtypes = [vp, ci, vp, vp, ll, ll, vp, vp, ci, ll, ll, ll, ll, ci, vp, vp, vp, ci, vp, vp]
    r = RotationT(a["table"], a["positions"], a["rows"], a["dims"], a["neighbours"])
    return f(c, a["layer"], a["K"], a["V"], a["ts"], a["hs"], a["Q"], a["Qout"], a["Hq"], a["qt"], a["qh"], a["ot"], a["oh"],
             a["T"], a["seqs"], a["qs"], a["granted"], a["n"], ctypes.byref(r) if a["rotation"] else None, None)


def read(lib, c, **kw):  # noqa: F811
    a = dict(layer=0, K=256, V=512, ts=256, hs=64, T=4, seqs=None, qs=256, first=None, n=2)
    a.update(kw)
    f = lib.attn_cache_read
    f.restype = ci
    f.argtypes = [vp, ci, vp, vp, ll, ll, ci, vp, vp, vp, ci, vp]
    return f(c, a["layer"], a["K"], a["V"], a["ts"], a["hs"], a["T"], a["seqs"], a["qs"], a["first"], a["n"], None)


BAD = [
    (dict(K=None), -1), (dict(V=264), -1), (dict(d=48), -2), (dict(d=160), -2), (dict(page_size=8), -2), (dict(page_size=48), -2),
    (dict(dtype=4), -1), (dict(dtype=2), -2),
    (dict(slot_stride=64), -1), (dict(slot_stride=36), -1),              # codes lie d / 2 bytes apart
    (dict(head_stride=16 * 64), -1), (dict(head_stride=32, slot_stride=128), -1),   # head by head, and no other way
    (dict(page_stride=4 * 16 * 36 - 16), -1), (dict(page_stride=4 * 16 * 36 + 8), -1),
    (dict(layer_stride=4 * 16 * 36 * 9), -1), (dict(page_stride=-4 * 16 * 36), -1),
    (dict(max_pages=(1 << 26) + 1), -1), (dict(heads=1 << 26, pages=1, layers=1), -1),
]


@pytest.mark.parametrize("bad,code", BAD)
def test_every_entry_rejects_a_bad_cache(lib, bad, code):  # noqa: F811
    c = ctypes.byref(cache(**bad))
    p, big = vp(256), sz(1 << 40)
    assert lib.attn_cache_reserve(c, p, p, ci(1), p, p, big, None) == code
    assert lib.attn_cache_free(c, p, p, ci(1), None) == code
    assert lib.attn_cache_fork(c, p, p, ci(1), ci(0), p, p, big, None) == code
    assert lib.attn_cache_compact(c, p, p, p, p, big, None) == code
    assert lib.attn_cache_append(c, ci(0), p, p, ll(256), ll(64), ci(4), p, p, ci(1), None) == code
    assert paged(lib, c, Hq=8) == code
    assert rotated(lib, c) == code and read(lib, c) == code
    assert rotated(lib, None) == -1 and read(lib, None) == -1


def test_accepted_layouts(lib):  # noqa: F811
    for d in (32, 64, 96, 128):
        for page in (16, 32, 64, 128, 256):
            for heads in (1, 3):
                c = ctypes.byref(cache(d=d, page_size=page, heads=heads))
                assert rotated(lib, c, T=0, dims=d) == 0 and read(lib, c, T=0) == 0 and rotated(lib, c, n=0, dims=d, oh=d, ot=8 * d) == 0
                assert paged(lib, c, T=0, Hq=heads, qh=d, oh=d) == 0
    assert read(lib, ctypes.byref(cache(heads=1, head_stride=0)), T=0) == 0
    # K and V of a page side by side, layers inside a page
    block = 4 * 16 * 36
    assert read(lib, ctypes.byref(cache(page_stride=4 * block, layer_stride=2 * block)), T=0) == 0


@pytest.mark.parametrize("dtype", [0, 1, E2M1])
def test_rotated_append_rejection(lib, dtype):  # noqa: F811
    c = ctypes.byref(cache(dtype=dtype))
    assert rotated(lib, c, rotation=False) == -1
    for bad in (dict(layer=2), dict(layer=-1), dict(T=-1), dict(n=-1), dict(n=(1 << 20) + 1), dict(K=None), dict(V=None), dict(K=264),
                dict(V=520), dict(ts=-256), dict(ts=258), dict(hs=66), dict(qs=None), dict(qs=258), dict(seqs=257), dict(granted=258),
                dict(Q=None), dict(Qout=None), dict(Q=264), dict(Qout=520), dict(Hq=-1), dict(Hq=0), dict(qt=514), dict(qh=-64),
                dict(oh=32), dict(ot=64), dict(oh=0), dict(Q=256, Qout=256, ot=1024),
                dict(table=None), dict(table=264), dict(positions=258), dict(rows=0), dict(rows=-1), dict(dims=0), dict(dims=-2),
                dict(dims=33), dict(dims=66), dict(neighbours=2), dict(neighbours=-1)):
        assert rotated(lib, c, **bad) == -1, bad
    assert rotated(lib, c, Hq=1 << 20, oh=64, ot=1 << 27) == -2
    assert rotated(lib, c, qt=1 << 38) == -2
    # nothing to do; strides of a dimension of one are ignored; no queries
    assert rotated(lib, c, T=0) == 0 and rotated(lib, c, n=0) == 0
    assert rotated(lib, c, n=0, T=1, ts=3, qt=5, ot=7) == 0
    assert rotated(lib, c, n=0, Hq=0, Q=None, Qout=None) == 0
    assert rotated(lib, c, n=0, Hq=1, qh=3, oh=5) == 0


@pytest.mark.parametrize("dtype", [0, 1, E2M1])
def test_read_rejection(lib, dtype):  # noqa: F811
    c = ctypes.byref(cache(dtype=dtype))
    for bad in (dict(layer=2), dict(T=-1), dict(n=-1), dict(K=None), dict(V=None), dict(K=264), dict(V=520), dict(ts=258), dict(hs=-64),
                dict(hs=32), dict(hs=0), dict(ts=64), dict(ts=0), dict(qs=None), dict(seqs=257), dict(first=258), dict(V=256)):
        assert read(lib, c, **bad) == -1, bad
    assert read(lib, c, T=0) == 0 and read(lib, c, n=0) == 0
    assert read(lib, c, n=0, hs=1024, ts=64) == 0        # tokens inside heads


def test_too_many_rows_to_a_token(lib):  # noqa: F811
    c = ctypes.byref(cache(heads=1 << 19, layers=1, pages=1))
    assert rotated(lib, c, Hq=1, ts=1 << 30, qt=64, ot=64) == -2
    c = ctypes.byref(cache(heads=(1 << 19) + 1, layers=1, pages=1))
    assert read(lib, c, ts=1 << 30) == -2 and rotated(lib, c, ts=1 << 30, Hq=0, Q=None, Qout=None) == -2
    p = vp(256)
    assert lib.attn_cache_append(c, ci(0), p, p, ll(1 << 30), ll(64), ci(4), p, p, ci(1), None) == -2


def test_attention_over_4_bits(lib):  # noqa: F811
    c = ctypes.byref(cache())
    f = lib.attn_paged_workspace_size
    f.restype, f.argtypes = sz, [ci] * 5
    need = f(8, 4, 4, 64, E2M1)
    assert need > 0 and f(8, 4, 4, 48, E2M1) == 0 and f(8, 4, 4, 64, 4) == 0
    assert paged(lib, c, ws_bytes=need - 1) == -3 and paged(lib, c, ws=None) == -3
    assert paged(lib, c, Q=vp(264)) == -1 and paged(lib, c, Hq=6) == -1 and paged(lib, c, scale=0.0) == -1
    assert paged(lib, c, qt=516) == -1 and paged(lib, c, T=0) == 0 and paged(lib, c, n=0) == 0
    # a cache of 4-bit values is no type of the other entry points
    from test_abi_host import _fwd
    assert _fwd(lib, dtype=E2M1) == -1
