"""Tables of the rotated append with more rows than positions can name."""
import pytest
import torch

from e2m1_ref import ints, turned

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.mark.parametrize("rows", [2 ** 31 - 1, 2 ** 31, 2 ** 31 + 5])
def test_a_table_of_more_than_2_31_rows(rows):
    """17 GB, of which the first and the last position's rows are looked at."""
    import exact_tiled_attention_17_gb300 as eta
    table = torch.empty((rows, 2), device="cuda")
    table[:40] = torch.randn((40, 2), generator=torch.Generator().manual_seed(1)).cuda()
    last = 2 ** 31 - 2
    table[last] = torch.tensor([0.5, -2.0], device="cuda")
    cache = eta.PagedCache.empty(1, 4, 2, 16, 64, 1, 4)
    assert eta.attn_cache_reserve(cache, ints([0]), ints([30])).tolist() == [1]
    k, v = (torch.randn((30, 2, 64), generator=torch.Generator().manual_seed(s)).to(BF16).cuda() for s in (2, 3))
    pos = torch.arange(30)
    pos[7] = last
    eta.attn_cache_append_rotated(cache, 0, k, v, None, ints([0, 30]), table, positions=pos.int().cuda())
    rk, rv = eta.attn_cache_read(cache, 0, None, ints([0, 30]), 30)
    assert eta.attn_status() == eta.ATTN_OK
    small = torch.cat([table[:40].cpu(), table[last:last + 1].cpu()])
    assert torch.equal(rk.cpu(), turned(k, small, torch.where(pos == last, 40, pos), False).to(BF16)) and torch.equal(rv, v)
    del table
    torch.cuda.empty_cache()
