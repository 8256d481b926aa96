"""Inputs of attn_paged_fwd over a cache of 4-bit values whose results show how often
and to what type the weights are rounded (not collected by pytest).  One sequence,
one kv head; every key and value is one that the cache holds exactly."""
import torch

from paged_bounds import BF16, Known


def two_weights(n, new, g, d):
    """Every other key scores 0, the others one value below, so a row has two
    weights, 1 and w.  V is -6 in the keys of weight 1, in column c only in the
    first (c + 1) / d of them, and 6 in all of the others: O is near 0 in some
    column, so nothing but the rounding of w is left there, and that has one sign
    in all keys.

    Bounds.  A weight is rounded once to float16: 2^-11.  A score is one product in
    one column (exact in float32, as Q and K are in float16), scaled by a float32
    number (2^-24 of a score of at most 4 in units of log2, and 2^-24 for the
    number's own rounding) and brought to its reference (a number below 16: 2^-21,
    twice where the scaling is rounded first); exp2 is off by 2^-22.  Sums: a share
    has less than 200 keys, or (at least 100 shares, at most 480) n / 100, each at
    worst added up key by key, and then come the parts: 2^-23 each."""
    gen = torch.Generator().manual_seed(n + d)
    q = torch.randn((new, g, d), generator=gen)
    q[:, :, 0] = -(0.25 + torch.arange(new * g).reshape(new, g) % 32 / 16)
    k, v = torch.zeros((n, d)), torch.zeros((n, d))
    low = torch.arange(n) % 2 == 1
    k[low, 0] = 6.0
    v[low] = 6.0
    ones = int((~low).sum())
    v[~low] = torch.where(torch.arange(ones)[:, None] * d < (torch.arange(d) + 1) * ones, -6.0, 0.0)
    delta = 2.0 ** -22 + 2.0 ** -20 + 2.0 ** -22 + (min(n, n // 100 + 680) + 16) * 2.0 ** -23
    return Known(q.to(BF16), k.to(BF16), v.to(BF16), 0.125, 2.0 ** -11 + 2 * delta, 2.0 ** -8, delta + 2.0 ** -20)
