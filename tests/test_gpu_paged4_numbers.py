"""What the header promises of numbers in attention over a cache of 4-bit values:
weights rounded once to float16, small columns of Q."""
import math

import pytest
import torch

from e2m1_ref import build4, ints
from paged4_bounds import two_weights

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def eta():
    import exact_tiled_attention_17_gb300 as m
    return m


@pytest.mark.parametrize("d", [32, 64, 96, 128])
@pytest.mark.parametrize("n,new,g,page", [
    (64, 1, 8, 16), (200, 3, 5, 64), (513, 4, 4, 16), (513, 5, 4, 128), (700, 40, 2, 32), (300, 1, 17, 16),
    (20001, 1, 8, 16), (20001, 2, 8, 64), (20001, 9, 3, 32), (20001, 9, 4, 256),
])
def test_weights_are_rounded_once_to_float16(eta, n, new, g, d, page):
    known = two_weights(n, new, g, d)
    cache, _ = build4(eta, [n], 1, page, d, seed=1)
    k, v = known.k[:, None].cuda(), known.v[:, None].cuda()
    eta.attn_cache_append(cache, 0, k, v, None, ints([0, n]))
    for got, want in zip(eta.attn_cache_read(cache, 0, None, ints([0, n]), n), (k, v)):
        assert torch.equal(got, want)
    o, lse = eta.attn_paged_fwd(known.q.cuda(), cache, 0, None, ints([0, new]), max_q=new, scale=known.scale)
    torch.cuda.synchronize()
    assert eta.attn_status() == eta.ATTN_OK
    known.check(o, lse)


@pytest.mark.parametrize("g", [1, 3, 17])
@pytest.mark.parametrize("top", [1.0, 1.5, 1.9921875, 2.0 ** -40, 1.25 * 2.0 ** 60])
def test_small_columns(eta, g, top):
    """Two keys, of which one is 0 and the other 6 in a column where Q is small beside its largest (to which the keys say
    nothing): the score shows the column's error, 2^-39 of the largest at most, and none down to 2^-29 of it.  (The LSE
    moves by at most as much as the score; the rest of it is float32.)"""
    d = 64
    cache, _ = build4(eta, [2], 1, 16, d, seed=1)
    k = torch.zeros((2, 1, d), dtype=BF16, device="cuda")
    k[1, 0, 17] = 6.0
    eta.attn_cache_append(cache, 0, k, k, None, ints([0, 2]))
    for e in range(20, 44):
        for m in (1.0, 1.0078125, 1.3359375, 1.9921875):
            small = m * 2.0 ** -e * (2.0 ** math.floor(math.log2(top)))
            q = torch.zeros((1, g, d), dtype=BF16, device="cuda")
            q[..., 3], q[..., 17] = top, small
            assert float(q[0, 0, 17]) == small
            scale = 1 / (6 * small)
            _, lse = eta.attn_paged_fwd(q, cache, 0, None, ints([0, 1]), max_q=1, scale=scale)
            off = 0.0 if small >= 2.0 ** -29 * top else 2.0 ** -39 * top * 6 * scale
            assert (lse.cpu().double() - math.log(1 + math.e)).abs().max() <= off + 2.0 ** -19, (e, m)
    assert eta.attn_status() == eta.ATTN_OK
