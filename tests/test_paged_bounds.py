"""The bounds of paged_bounds.py hold for a right result and refuse planted
mistakes: a share of the keys lost, P rounded to bf16 once, products in TF32."""
import pytest
import torch

from paged_bounds import BF16, F32, close_weights, counts, fine_keys, tf32


def as_stored(known, result):
    return result[0].to(known.q.dtype), result[1].float()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n,new", [(70001, 1), (70001, 7), (20000, 40)])
def test_a_lost_share_shows(dtype, n, new):
    known = counts(n, new, 2, 64, dtype)
    known.check(*as_stored(known, known.result()))
    for at in (0, 1000, n // 2, n - 200):
        keys = torch.ones(n, dtype=torch.bool)
        keys[at:at + 100] = False    # (the smallest share of a CTA has 128)
        with pytest.raises(AssertionError):
            known.check(*as_stored(known, known.result(keys=keys)))


@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("n,new,g", [(2, 1, 8), (17, 1, 4), (40, 4, 4), (64, 16, 1)])
def test_one_rounding_of_p_shows(n, new, g, d):
    known = close_weights(n, new, g, d)
    known.check(*as_stored(known, known.result()))

    def two(p):
        hi = p.to(BF16).double()
        return hi + (p - hi).to(BF16).double()
    known.check(*as_stored(known, known.result(weight=two)))
    with pytest.raises(AssertionError):
        known.check(*as_stored(known, known.result(weight=lambda p: p.to(BF16).double())))


@pytest.mark.parametrize("n,new", [(50, 1), (5000, 3), (70001, 1)])
def test_products_in_tf32_show(n, new):
    known = fine_keys(n, new, 4)
    known.check(*as_stored(known, known.result()))
    with pytest.raises(AssertionError):
        known.check(*as_stored(known, known.result(k=tf32(known.k))))
    o, lse = as_stored(known, known.result())
    with pytest.raises(AssertionError):      # the LSE alone shows it too
        known.check(o, as_stored(known, known.result(k=tf32(known.k)))[1])
