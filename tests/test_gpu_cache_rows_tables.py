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


@pytest.mark.parametrize("dtype", [BF16, torch.float32, torch.float4_e2m1fn_x2])
def test_reading_from_before_the_first_token(dtype):
    """An entry with a negative first is left out whole; without first the rows of the tokens that are there are read."""
    import exact_tiled_attention_17_gb300 as eta
    cache = eta.PagedCache.empty(1, 4, 2, 16, 64, 2, 4, dtype=dtype)
    assert eta.attn_cache_reserve(cache, ints([0, 1]), ints([5, 20])).tolist() == [1, 1]
    k, v = (torch.full((25, 2, 64), x, dtype=cache.dtype, device="cuda") for x in (6.0, -6.0))
    eta.attn_cache_append(cache, 0, k, v, None, ints([0, 5, 25]))
    ko, vo = (torch.full((12, 2, 64), 1.0, dtype=cache.dtype, device="cuda") for _ in range(2))
    eta.attn_cache_read(cache, 0, None, ints([0, 6, 9]), first=ints([-2, 17]), k_out=ko, v_out=vo)
    assert eta.attn_status() == eta.ATTN_ERR_ARG
    assert (ko[:6] == 1).all() and (vo[:6] == 1).all() and (ko[6:9] == 6).all() and (vo[6:9] == -6).all() and (ko[9:] == 1).all()
    ko.fill_(1.0)
    eta.attn_cache_read(cache, 0, None, ints([0, 7, 9]), k_out=ko, v_out=vo)
    assert eta.attn_status() == eta.ATTN_ERR_ARG
    assert (ko[:2] == 1).all() and (ko[2:9] == 6).all() and (ko[9:] == 1).all()
