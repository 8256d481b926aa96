"""attn_decode_fwd with stages that are refilled many times: every output against
the definition in float64, and the same bits each time."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B,H,Nq,Nk,d,dtype", [
    (1, 32, 1, 32768, 128, torch.bfloat16), (4, 16, 2, 5001, 64, torch.bfloat16), (1, 8, 8, 20011, 96, torch.bfloat16),
    (2, 8, 1, 16385, 128, torch.float32), (1, 4, 3, 30000, 32, torch.float32),
])
def test_decode_again_and_again(B, H, Nq, Nk, d, dtype):
    """Bounds: a score is a sum of d products in float32, weights and sums are float32 (exp2 2^-22, sums 2^-23 each of the
    chunk's keys, at least 14 chunks or at most 4681 keys), O is rounded to its type."""
    import exact_tiled_attention_17_gb300 as eta
    gen = torch.Generator(device="cuda").manual_seed(Nk)
    q, k, v = (torch.randn((B, H, n, d), generator=gen, device="cuda").to(dtype) for n in (Nq, Nk, Nk))
    scale = 1 / math.sqrt(d)
    runs = [eta.attn_decode_fwd(q, k, v, True, scale) for _ in range(8)]
    torch.cuda.synchronize()
    assert eta.attn_status() == eta.ATTN_OK
    for o, lse in runs[1:]:
        assert torch.equal(o, runs[0][0]) and torch.equal(lse, runs[0][1])
    o, lse = runs[0]
    kd, vd = k.double(), v.double()
    s = q.double() @ kd.transpose(2, 3) * scale
    mass = (q.double().abs() @ kd.abs().transpose(2, 3)).amax(3) * scale
    see = torch.arange(Nk, device="cuda")[None] <= Nk - Nq + torch.arange(Nq, device="cuda")[:, None]
    s = s.masked_fill(~see, -math.inf)
    w = torch.softmax(s, 3)
    want, size = w @ vd, w @ vd.abs()
    delta = (d + 4) * 2.0 ** -23 * mass + 2.0 ** -21 + 4900 * 2.0 ** -23
    half = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -24
    err = (o.double() - want).abs()
    assert (err <= half * want.abs() + 2 * delta[..., None] * size * 1.01).all()
    want_l = torch.logsumexp(s, 3)
    assert ((lse.double() - want_l).abs() <= delta + 2.0 ** -22 * (want_l.abs() + 1)).all()
