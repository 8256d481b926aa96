"""NaN that a paged cache of 4-bit values holds (what an infinity or a NaN becomes):
in K every row that sees the key is NaN, LSE too; in V every row that sees it, in
the 16 columns of the group.  Other rows of the same entry and kv head may be NaN in
those columns; everything else is as without it, bit by bit."""
import math

import pytest
import torch

from e2m1_ref import build4, ints, starts

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
NAN_SCALE = 255


@pytest.fixture(scope="module")
def eta():
    import exact_tiled_attention_17_gb300 as m
    return m


def queries(T, Hq, d, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn((T, Hq, d), generator=g, device="cuda").to(BF16)


def plant(cache, pool, row, head, key, group, byte):
    """Sets a group's scale; returns what it was."""
    scales = cache.parts(pool)[1]
    at = (0, int(cache.page_table[row, key // cache.page_size]), head, key % cache.page_size, group)
    was = int(scales[at])
    scales[at] = byte
    return was


def attend(eta, cache, q, new, causal=True, scale=None):
    o, lse = eta.attn_paged_fwd(q, cache, 0, None, ints(starts(new)), max_q=max(new), causal=causal, scale=scale)
    torch.cuda.synchronize()
    assert eta.attn_status() == eta.ATTN_OK
    return o, lse


def check(eta, cache, lens, new, g, where, row, head, key, group, q, causal=True, scale=None):
    """Outputs with a NaN at a key of a sequence against those with zeros in its place."""
    pool = getattr(cache, where)
    was = plant(cache, pool, row, head, key, group, 0)
    o0, l0 = attend(eta, cache, q, new, causal, scale)
    plant(cache, pool, row, head, key, group, NAN_SCALE)
    o1, l1 = attend(eta, cache, q, new, causal, scale)
    plant(cache, pool, row, head, key, group, was)
    hit = torch.zeros(o0.shape, dtype=torch.bool, device="cuda")
    hit_l = torch.zeros(l0.shape, dtype=torch.bool, device="cuda")
    may = hit.clone()      # rows that a NaN in V may reach, although they do not see it
    a, n, heads = starts(new)[row], new[row], slice(head * g, head * g + g)
    sees = [t for t in range(n) if not causal or key <= lens[row] - n + t]
    for t in sees:
        if where == "k":
            hit[a + t, heads] = True
            hit_l[a + t, heads] = True
        else:
            hit[a + t, heads, 16 * group:16 * group + 16] = True
    if where == "v":
        may[a:a + n, heads, 16 * group:16 * group + 16] = True
    what = f"{where}, sequence {row}, head {head}, key {key} of {lens[row]}, group {group}"
    assert not torch.isnan(o0).any() and not torch.isnan(l0).any()
    assert torch.isnan(o1)[hit].all(), f"{what}: lost in {(~torch.isnan(o1) & hit).sum()} of {hit.sum()} columns"
    assert torch.isnan(l1)[hit_l].all(), f"{what}: lost in LSE"
    assert not torch.isnan(o1)[~hit & ~may].any(), f"{what}: in {(torch.isnan(o1) & ~hit & ~may).sum()} other columns"
    hit |= may & torch.isnan(o1)
    # (the references of rows that see a NaN in K may move otherwise: those are NaN anyway)
    assert torch.equal(o1[~hit], o0[~hit]) and torch.equal(l1[~hit_l], l0[~hit_l]), f"{what}: other results changed"


FORMS = [(1, 4), (2, 4), (3, 5), (8, 2), (5, 4), (4, 8), (9, 3), (40, 4), (130, 2), (17, 17), (300, 1)]   # new tokens, group


@pytest.mark.parametrize("d", [32, 64, 96, 128])
@pytest.mark.parametrize("new,g", FORMS)
def test_nan_among_the_new_tokens(eta, new, g, d):
    """The keys at the causal border, which some rows of a unit see and others do not."""
    lens, news = [new + 77, new, new + 200], [new, new, 1]
    cache, _ = build4(eta, lens, 2, 16 if d != 64 else 128, d, seed=new + d)
    q = queries(sum(news), 2 * g, d, new + g)
    for where in ("v", "k"):
        for row, key in ((0, lens[0] - 1), (0, lens[0] - new), (0, lens[0] - 1 - new // 2), (1, 0), (1, new - 1), (2, lens[2] - 1)):
            check(eta, cache, lens, news, g, where, row, (key + d) % 2, key, (key + new) % (d // 16), q)


@pytest.mark.parametrize("new,g,d", [(1, 4, 128), (3, 5, 64), (5, 4, 96), (40, 4, 128), (130, 2, 64)])
def test_every_key_sees_every_row(eta, new, g, d):
    lens, news = [new + 150, new + 3], [new, new]
    cache, _ = build4(eta, lens, 2, 32, d, seed=d + g)
    q = queries(sum(news), 2 * g, d, 3)
    for where in ("v", "k"):
        for row, key in ((0, lens[0] - 1), (0, 3), (1, new)):
            check(eta, cache, lens, news, g, where, row, 1, key, 1, q, causal=False)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n,new,g", [(300, 1, 4), (6000, 1, 4), (6000, 3, 5), (6000, 5, 4), (6000, 40, 4), (20000, 200, 2), (2000, 300, 2)])
def test_nan_where_weights_vanish(eta, n, new, g, d):
    """Scores of the first half hundreds below those of the second: the parts that hold the NaN have weights that are 0 in
    float32, or (the other way round) parts that come later have."""
    for down in (False, True):
        cache, _ = build4(eta, [n], 1, 16, d, seed=n + new)
        k = torch.zeros((n, 1, d), dtype=BF16, device="cuda")
        low = torch.arange(n, device="cuda") < n // 2
        k[:, 0, 0] = torch.where(low != down, -6.0, 6.0).to(BF16)
        v = torch.randn((n, 1, d), generator=torch.Generator(device="cuda").manual_seed(n), device="cuda").to(BF16)
        eta.attn_cache_append(cache, 0, k, v, None, ints([0, n]))
        q = queries(new, g, d, 5)
        q[..., 0] = 32.0
        for where in ("v", "k"):
            for key in (5, n // 2 - 200 if n > 1000 else 140, n // 2 + 3, n - new - 1, n - 1):
                check(eta, cache, [n], [new], g, where, 0, 0, key, 0 if where == "k" else 2, q, scale=1.0)


@pytest.mark.parametrize("new,g", [(1, 4), (4, 4), (6, 4), (60, 2)])
def test_nan_and_pages_that_are_missing(eta, new, g):
    """A NaN in a page that the table does not name is seen by nobody; what lies past the end neither."""
    d, n = 64, 200
    cache, _ = build4(eta, [n], 2, 16, d, seed=9)
    q = queries(new, 2 * g, d, 1)
    id_ = int(cache.page_table[0, 3])
    cache.page_table[0, 3] = -1
    o0, l0 = eta.attn_paged_fwd(q, cache, 0, None, ints([0, new]), max_q=new)
    for pool in (cache.k, cache.v):
        cache.parts(pool)[1][0, id_] = NAN_SCALE
    o1, l1 = eta.attn_paged_fwd(q, cache, 0, None, ints([0, new]), max_q=new)
    assert eta.attn_status() == eta.ATTN_ERR_ARG        # (the page is reported)
    assert torch.equal(o0, o1) and torch.equal(l0, l1) and not torch.isnan(o0).any()
    assert math.isfinite(float(l0.abs().max()))
