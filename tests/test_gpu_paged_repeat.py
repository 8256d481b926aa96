"""Attention of few new tokens over a paged bf16 cache with many short units to a
CTA: the copy buffers are handed back and filled again all the time, so a read that
a later copy overtakes changes an output.  Every output against the definition in
float64, and the same bits each time."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def eta():
    import exact_tiled_attention_17_gb300 as m
    return m


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("seqs,longest,new,heads,g,d,page", [
    (500, 70, 1, 8, 4, 128, 16), (500, 130, 1, 8, 4, 64, 64), (300, 300, 1, 8, 16, 128, 32), (400, 200, 3, 4, 5, 96, 16),
    (300, 140, 5, 8, 4, 128, 16), (300, 260, 4, 8, 8, 64, 128),
])
def test_many_short_units(eta, seqs, longest, new, heads, g, d, page):
    """At most 16 rows: P in two bf16 parts (2^-16 of a weight); more: rounded once (2^-8).  A score is a sum of d
    products in float32, exp2 is off by 2^-22, sums of n weights by n 2^-23; O is rounded to bf16 (2^-8)."""
    gen = torch.Generator(device="cuda").manual_seed(d + g)
    lens = torch.randint(new, longest + 1, (seqs,), generator=torch.Generator().manual_seed(seqs + d)).tolist()
    cache = eta.PagedCache.empty(1, sum(-(-n // page) for n in lens) + 1, heads, page, d, seqs, longest // page + 1)
    for pool in (cache.k, cache.v):
        pool.fill_(math.nan)
    assert eta.attn_cache_reserve(cache, ints(list(range(seqs))), ints(lens)).tolist() == [1] * seqs
    ends = torch.tensor([0] + lens).cumsum(0).tolist()
    k, v = (torch.randn((ends[-1], heads, d), generator=gen, device="cuda").to(BF16) for _ in range(2))
    eta.attn_cache_append(cache, 0, k, v, None, ints(ends))
    T, Hq = seqs * new, heads * g
    q = torch.randn((T, Hq, d), generator=gen, device="cuda").to(BF16)
    runs = [eta.attn_paged_fwd(q, cache, 0, None, ints([new * i for i in range(seqs + 1)]), max_q=new) for _ in range(8)]
    torch.cuda.synchronize()
    assert eta.attn_status() == eta.ATTN_OK
    for o, lse in runs[1:]:
        assert torch.equal(o, runs[0][0]) and torch.equal(lse, runs[0][1])
    o, lse = runs[0]
    part = 2.0 ** -16 if g * new <= 16 else 2.0 ** -8
    scale = 1 / math.sqrt(d)
    for i, n in enumerate(lens):
        a, b = new * i, new * i + new
        kd, vd = (x[ends[i]:ends[i + 1]].double().repeat_interleave(g, 1) for x in (k, v))
        s = torch.einsum("thd,nhd->htn", q[a:b].double(), kd) * scale
        mass = torch.einsum("thd,nhd->htn", q[a:b].double().abs(), kd.abs()).amax(2) * scale
        see = torch.arange(n, device="cuda")[None] <= n - new + torch.arange(new, device="cuda")[:, None]
        s = s.masked_fill(~see, -math.inf)
        w = torch.softmax(s, 2)
        want, size = (torch.einsum("htn,nhd->thd", w, x) for x in (vd, vd.abs()))
        delta = ((d + 4) * 2.0 ** -23 * mass + 2.0 ** -21 + (n + 16) * 2.0 ** -23).T
        tol = 2.0 ** -8 * want.abs() + (part + 2 * delta[..., None]) * size * 1.01
        err = (o[a:b].double() - want).abs()
        assert (err <= tol).all(), f"entry {i}: off by {(err / tol).max():.3g} of the bound"
        want_l = torch.logsumexp(s, 2).T
        assert ((lse[a:b].double() - want_l).abs() <= delta + 2.0 ** -22 * (want_l.abs() + 1)).all()
