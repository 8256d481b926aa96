"""Plain references for the paged-cache tests (not collected by pytest):
attention in float64, the page operators in Python integers, and the bounds
the kernels are held to."""
import math

import torch

EPS = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}   # half a step, relative to the value


def gather(cache, layer, row, n):
    """K and V of the first n tokens of a table row, float64 [heads, n, d], and
    which of them lie in a page of the pool."""
    S, table = cache.page_size, cache.page_table[row].tolist()
    k = torch.zeros(cache.heads, n, cache.d, dtype=torch.float64)
    v = torch.zeros_like(k)
    there = torch.zeros(n, dtype=torch.bool)
    for c in range(-(-n // S)):
        id_ = table[c]
        if not 0 <= id_ < cache.pages:
            continue
        a, b = c * S, min(n, c * S + S)
        k[:, a:b] = cache.k[layer, id_, :, :b - a].cpu().double()
        v[:, a:b] = cache.v[layer, id_, :, :b - a].cpu().double()
        there[a:b] = True
    return k, v, there


def attention(q, cache, layer, seqs, q_start, causal, scale):
    """The definition, row by row of the list: {row of q: (o, lse, tol_o,
    tol_lse)} with [Hq, d] and [Hq] float64 tensors.

    Bounds.  A score is a sum of d products in float32, off by at most
    (d + 2) 2^-23 scale sum |q_c k_c| (2^-23: the tensor core's sums may cut
    where the CUDA cores round), times log2(e) and back; exp2 is off by 2^-22.
    So each weight is off by a factor 1 + delta, the sum of n weights and the
    output by n more roundings of 2^-23 each; bf16 rounds each weight once
    (2^-8) and the output once.  A numerator and a denominator both carry the
    weights' error."""
    dt = q.dtype
    half = EPS[dt]
    out = {}
    g = q.shape[1] // cache.heads
    starts = q_start.tolist()
    rows = seqs.tolist() if seqs is not None else range(len(starts) - 1)
    lens = cache.seq_lens.tolist()
    for i, row in enumerate(rows):
        a, b = starts[i], starts[i + 1]
        if b == a:
            continue
        n = lens[row]
        k, v, there = gather(cache, layer, row, n)
        qd = q[a:b].cpu().double()
        for t in range(b - a):
            see = there.clone()
            if causal:
                see &= torch.arange(n) <= n - (b - a) + t
            o = torch.zeros(q.shape[1], cache.d, dtype=torch.float64)
            lse = torch.full((q.shape[1],), -math.inf, dtype=torch.float64)
            tol_o, tol_l = torch.zeros_like(o), torch.zeros_like(lse)
            if see.any():
                kk = k[:, see].repeat_interleave(g, 0)
                vv = v[:, see].repeat_interleave(g, 0)
                s = (kk @ qd[t][:, :, None])[..., 0] * scale
                mass = (kk.abs() @ qd[t].abs()[:, :, None])[..., 0].amax(1) * scale
                w = torch.softmax(s, 1)
                o = (w[:, None] @ vv)[:, 0]
                lse = torch.logsumexp(s, 1)
                m = int(see.sum())
                delta = (cache.d + 4) * 2.0 ** -23 * mass + 2.0 ** -21 + (m + 16) * 2.0 ** -23
                size = (w[:, None] @ vv.abs())[:, 0]
                p_round = half if dt == torch.bfloat16 else 0.0
                tol_o = half * o.abs() + size * (p_round + 2 * delta[:, None]) * 1.01 + 1e-30
                tol_l = delta + 2.0 ** -22 * (lse.abs() + 1)
            out[a + t] = (o, lse, tol_o, tol_l)
    return out


def check_attention(q, cache, layer, seqs, q_start, causal, scale, o, lse, untouched=None):
    """Every row of the list within its bound; the others as `untouched` says."""
    ref = attention(q, cache, layer, seqs, q_start, causal, scale)
    og, lg = o.cpu().double(), lse.cpu().double()
    for r in range(q.shape[0]):
        if r not in ref:
            if untouched is not None:
                assert torch.equal(og[r], untouched[0][r].cpu().double()), f"row {r} was written"
                assert torch.equal(lg[r], untouched[1][r].cpu().double()), f"LSE of row {r} was written"
            continue
        ro, rl, to, tl = ref[r]
        assert not torch.isnan(og[r]).any() and not torch.isnan(lg[r]).any(), f"NaN in row {r}"
        err = (og[r] - ro).abs()
        assert (err <= to).all(), f"row {r}: off by {(err / to).max():.3g} of the bound"
        inf = torch.isinf(rl)
        assert torch.equal(torch.isinf(lg[r]) & (lg[r] < 0), inf), f"LSE of row {r}"
        assert (og[r][inf] == 0).all()
        assert ((lg[r] - rl).abs()[~inf] <= tl[~inf]).all(), f"LSE of row {r}: {(lg[r] - rl).abs()[~inf].max():.3g}"


class Pages:
    """The page operators in plain integers, beside the tensors of a cache."""

    def __init__(self, cache):
        self.S, self.n_pages, self.cols = cache.page_size, cache.pages, cache.max_pages
        self.table = cache.page_table.tolist()
        self.lens = cache.seq_lens.tolist()
        self.refs = cache.ref_counts.tolist()
        self.copies = []   # (src, dst, slots) of the last call
        self.shared = False   # whether a sequence was refused to grow into a shared page

    def _free(self):
        return [p for p in range(self.n_pages) if self.refs[p] <= 0]

    def reserve(self, seqs, n_new):
        free, at, total, out, seen = self._free(), 0, 0, [], set()
        for s, add in zip(seqs, n_new):
            ok = 0 <= s < len(self.lens) and add >= 0 and not (add and s in seen)
            if add > 0:
                seen.add(s)
            if not ok or self.lens[s] + add > self.cols * self.S:
                out.append(0)
                continue
            if add and self.lens[s] % self.S and self.refs[self.table[s][self.lens[s] // self.S]] > 1:
                self.shared = True
                out.append(0)
                continue
            have, want = -(-self.lens[s] // self.S), -(-(self.lens[s] + add) // self.S)
            need = want - have
            total += need
            if need and total > len(free):
                out.append(0)
                continue
            ids = free[total - need:total]
            for k, p in enumerate(ids):
                self.table[s][have + k] = p
                self.refs[p] = 1
            self.lens[s] += add
            out.append(1)
        return out

    def free(self, seqs, keep=None):
        seen = set()
        for i, s in enumerate(seqs):
            if not 0 <= s < len(self.lens) or s in seen:
                continue
            seen.add(s)
            left = max(0, min(keep[i] if keep is not None else 0, self.lens[s]))
            for c in range(-(-left // self.S), self.cols):
                p = self.table[s][c]
                if p >= 0:
                    self.table[s][c] = -1
                    if p < self.n_pages:
                        self.refs[p] -= 1
            self.lens[s] = left

    def fork(self, parents, children, copy):
        free, total, out, seen = self._free(), 0, [], set()
        before, tables = list(self.lens), [list(t) for t in self.table]
        self.copies = []
        for a, b in zip(parents, children):
            ok = 0 <= a < len(before) and 0 <= b < len(before) and b not in seen and before[b] == 0
            if 0 <= b < len(before):
                seen.add(b)
            if not ok:
                out.append(0)
                continue
            n = before[a]
            shared = 0 if copy else n // self.S
            need = -(-n // self.S) - shared
            total += need
            if need and total > len(free):
                out.append(0)
                continue
            ids = free[total - need:total]
            self.table[b] = tables[a][:shared] + ids + [-1] * (self.cols - shared - need)
            for p in tables[a][:shared]:
                self.refs[p] += 1
            for k, p in enumerate(ids):
                self.refs[p] = 1
                self.copies.append((tables[a][shared + k], p, min(self.S, n - (shared + k) * self.S)))
            self.lens[b] = n
            out.append(1)
        return out

    def compact(self):
        live = sum(r > 0 for r in self.refs)
        holes = [p for p in range(live) if self.refs[p] <= 0]
        strays = [p for p in range(live, self.n_pages) if self.refs[p] > 0]
        to = dict(zip(strays, holes))
        self.copies = [(s, h, self.S) for s, h in to.items()]
        self.table = [[to.get(p, p) for p in row] for row in self.table]
        for s, h in to.items():
            self.refs[h], self.refs[s] = self.refs[s], 0
        return live

    def check(self, cache):
        assert cache.page_table.tolist() == self.table
        assert cache.seq_lens.tolist() == self.lens
        assert cache.ref_counts.tolist() == self.refs

    def consistent(self):
        names = [0] * self.n_pages
        for row in self.table:
            for p in row:
                if p >= 0:
                    names[p] += 1
        assert names == self.refs
