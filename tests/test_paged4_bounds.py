"""The bounds of paged4_bounds.py hold for weights rounded once to float16 and refuse
weights rounded to bf16."""
import pytest
import torch

from paged4_bounds import two_weights
from paged_bounds import BF16


@pytest.mark.parametrize("d", [32, 64, 96, 128])
@pytest.mark.parametrize("n,new,g", [(64, 1, 8), (200, 3, 5), (513, 4, 4), (513, 5, 4), (700, 40, 2), (20001, 1, 8), (20001, 9, 4)])
def test_bf16_weights_show(n, new, g, d):
    known = two_weights(n, new, g, d)
    o, lse, _ = known.result()
    known.check(o.to(BF16), lse.float())
    known.check(known.result(weight=lambda p: (p * 128).half().double() / 128)[0].to(BF16), lse.float())
    with pytest.raises(AssertionError):
        known.check(known.result(weight=lambda p: p.to(BF16).double())[0].to(BF16), lse.float())
    for t in (known.k, known.v):      # what the cache holds exactly: 0 and the largest code under a scale of 1
        assert set(t.float().abs().unique().tolist()) <= {0.0, 6.0}
    assert torch.isfinite(o).all()
