"""Inputs of attn_paged_fwd whose results are known to a few roundings at any
length, so that a part lost in the merge, a probability rounded once too often
or a product in fewer bits cannot hide in a bound that grows with the context
(not collected by pytest).  One sequence, one kv head."""
import math

import torch

BF16, F32 = torch.bfloat16, torch.float32


class Known:
    """q [T, Hq, d], k, v [n, d] (CPU), and how far O (relative to its size and
    to itself) and LSE may be off."""

    def __init__(self, q, k, v, scale, of_size, of_value, of_lse):
        self.q, self.k, self.v, self.scale = q, k, v, scale
        self.of_size, self.of_value, self.of_lse = of_size, of_value, of_lse

    def result(self, keys=None, k=None, weight=None):
        """O, LSE and the size of O's sums in float64.  keys: the only ones
        seen; k: other keys; weight: what P goes through before the product
        with V (plants for the tests of the bounds)."""
        T, n = self.q.shape[0], self.k.shape[0]
        k = (self.k if k is None else k).double()
        s = torch.einsum("thd,nd->thn", self.q.double(), k) * self.scale
        see = torch.arange(n) <= (n - T + torch.arange(T))[:, None]
        if keys is not None:
            see = see & keys
        s = s.masked_fill(~see[:, None], -math.inf)
        p = torch.exp(s - s.amax(2, keepdim=True))
        total = p.sum(2, keepdim=True)
        w = p if weight is None else weight(p)
        v = self.v.double()
        return (w / total) @ v, torch.logsumexp(s, 2), (p / total) @ v.abs()

    def check(self, o, lse):
        want, want_lse, size = self.result()
        err = (o.cpu().double() - want).abs()
        tol = self.of_size * size + self.of_value * want.abs()
        assert (err <= tol).all(), f"O: off by {(err / tol).max():.3g} of the bound"
        err = (lse.cpu().double() - want_lse).abs().max()
        assert err <= self.of_lse, f"LSE: off by {err:.3g}, allowed {self.of_lse:.3g}"


def counts(n, new, g, d, dtype):
    """K = 0, and column c of V marks the c-th block of keys: O is a share of
    the keys.  Every p is 1, sums are whole numbers below 2^24, so what rounds
    is 1 / l, its product with o (2^-24 each, and as much again for the bounds'
    own second order), O in its type (bf16: 2^-8) and log2(l) ln 2 (a unit in
    the last place of a number below 32, 2^-19, times ln 2, and two roundings of
    a number below 16)."""
    q = torch.randn((new, g, d), generator=torch.Generator().manual_seed(n)).to(dtype)
    v = (torch.arange(n)[:, None] * d // n == torch.arange(d)).to(dtype)
    return Known(q, torch.zeros((n, d), dtype=dtype), v, 0.125, 0.0, 2.0 ** -22 + (2.0 ** -8 if dtype == BF16 else 0.0),
                 2.0 ** -19 + 2.0 ** -19)


def close_weights(n, new, g, d):
    """bf16, at most 16 rows: scores within about 1 of each other in one column
    of K, V of random signs, so that O is small beside the weights that make it.
    P in two bf16 parts is off by (2^-8)^2 of itself.  A score, one product of
    at most 1.1 in units of log2, is off by 2^-21 with its scaling, ex2 by 2^-22, and
    the sums over n weights (as much in l) by n 2^-23 each."""
    gen = torch.Generator().manual_seed(100 * n + new)
    q, k = torch.zeros((new, g, d)), torch.zeros((n, d))
    q[:, :, 0] = 1 + torch.arange(new * g).reshape(new, g) / 32
    k[:, 0] = -torch.rand(n, generator=gen) * 4
    v = torch.randint(0, 2, (n, d), generator=gen) * 2.0 - 1
    delta = 2.0 ** -21 + 2.0 ** -22 + (n + 16) * 2.0 ** -23
    return Known(q.to(BF16), k.to(BF16), v.to(BF16), 0.125, 2.0 ** -16 + 2 * delta, 2.0 ** -8, delta + 2.0 ** -20)


def fine_keys(n, new, g):
    """float32, d = 64: keys of 1 and, every third, of 1 + 2^-12, queries of 8 ..
    32; V tells the two apart.  TF32 would take them for equal.  Scores are
    exact sums of at most 2112 (multiples of 2^-9) where the products come first;
    where q is scaled before them, each of the 4 products and 5 exchanges of a
    sum of at most 381 (in units of log2) rounds: 10 * 381 * 2^-24.  ex2: 2^-22.
    Sums: one long unit is cut into at least a hundred shares, or into shares
    of less than 200 keys, each at worst added up key by key, and then into at
    most 640 parts."""
    q = torch.full((new, g, 64), 32.0) / (1 + torch.arange(g) % 4)[None, :, None].exp2().clamp(max=4)
    fine = torch.arange(n) % 3 == 0
    k = (1 + fine[:, None] * 2.0 ** -12).expand(n, 64).contiguous()
    v = torch.where(torch.arange(64) < 32, fine[:, None], ~fine[:, None]).float()
    delta = 10 * 381 * 2.0 ** -24 * math.log(2) + 2.0 ** -22 + (min(n, n // 100 + 840) + 16) * 2.0 ** -23
    return Known(q, k, v, 0.125, 2 * delta, 2.0 ** -22, delta + 264 * 2.0 ** -23)


def tf32(x):
    """x with 10 bits of fraction."""
    bits = x.float().contiguous().view(torch.int32)
    return ((bits + 0xFFF + ((bits >> 13) & 1)) & ~0x1FFF).view(torch.float32)
