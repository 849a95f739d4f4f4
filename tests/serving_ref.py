"""Plain 64-bit references of the serving operators, and the error bounds their tests use.

Attention of one request, from the definition, in float64. ``Bounds`` carries what the tolerance of
a row is made of (eps below is the relative error of one rounding to that type, half a step:
bf16 2^-8, fp32 2^-24; the tensor cores' fp32 sums may truncate, which costs a whole step, 2^-23):

* a score is a sum of D exact products: off by at most ds = (D + 3) 2^-23 max_j sum_i |q_i k_ji| scale
  (the D partial sums, the factor's own rounding and its product with the score);
* every weight p is off by ds relative, by the exponential (2^-22 for the hardware's base-2 one, and
  the argument's rounding, 2^-23 (|s| + |m|) <= 2^-23 * 2 max|s|, counted in ds), and where it is
  rounded to bf16 by 2^-8;
* sums over n keys, of the weights and of weight times value: n 2^-23 each;
* the output's rounding: 2^-8 of its value.

So |out - ref| <= 2^-8 |ref| + A (2^-8 + 2 ds + 2 n 2^-23 + 2^-20), A = sum_j p_j |v_j| / sum_j p_j, the
denominator's and the numerator's ds counted separately, and
|lse - ref| <= ds + n 2^-23 + 2^-20 + 2^-22 |ref|.
"""

from __future__ import annotations

import math
from typing import NamedTuple

import torch


class Rows(NamedTuple):
    out: torch.Tensor   # [n, Hq, D] float64
    lse: torch.Tensor   # [n, Hq]
    out_tol: torch.Tensor
    lse_tol: torch.Tensor


def attend(q, k, v, see) -> Rows:
    """q [n, Hq, D] against k, v [S, Hkv, D]; see [n, S] truth values."""
    n, hq, d = q.shape
    s = k.shape[0]
    g = hq // k.shape[1]
    scale = 1.0 / math.sqrt(d)
    q64 = q.double().transpose(0, 1)                                   # [Hq, n, D]
    k64 = k.double().transpose(0, 1).repeat_interleave(g, 0)           # [Hq, S, D]
    v64 = v.double().transpose(0, 1).repeat_interleave(g, 0)
    hidden = ~see[None].expand(hq, n, s)
    x = (q64 @ k64.transpose(1, 2) * scale).masked_fill(hidden, -math.inf)
    size = (q64.abs() @ k64.abs().transpose(1, 2) * scale).masked_fill(hidden, 0.0)
    lse = torch.logsumexp(x, -1) if s else torch.full((hq, n), -math.inf, dtype=torch.float64, device=q.device)
    p = torch.exp(x - torch.where(lse == -math.inf, 0.0, lse)[..., None])
    out, mean = p @ v64, p @ v64.abs()
    ds = ((d + 7) * 2.0 ** -23 * (size.amax(-1) if s else torch.zeros_like(lse)))[..., None]
    keys = see.sum(-1).double()[None, :, None]
    out_tol = 2.0 ** -8 * out.abs() + mean * (2.0 ** -8 + 2 * ds + 2 * keys * 2.0 ** -23 + 2.0 ** -20)
    lse_tol = (ds + keys * 2.0 ** -23)[..., 0] + 2.0 ** -20 + 2.0 ** -22 * torch.where(lse == -math.inf, 0.0, lse).abs()
    return Rows(out.transpose(0, 1), lse.T, out_tol.transpose(0, 1), lse_tol.T)


def prompt(q, k, v, lens) -> Rows:
    """Packed prompts: row i of a request sees its rows j <= i."""
    at, rows = 0, []
    for n in lens:
        part = slice(at, at + n)
        at += n
        see = torch.ones((n, n), dtype=torch.bool, device=q.device).tril()
        rows.append(attend(q[part], k[part], v[part], see))
    return Rows(*(torch.cat(x) for x in zip(*rows)))


def tree(q, caches, prefix, lens, see_drafts) -> Rows:
    """caches[b] = (k, v) [S, Hkv, D] of request b; see_drafts[b] [n, n] truth values."""
    at, rows = 0, []
    for (k, v), p, n, see in zip(caches, prefix, lens, see_drafts):
        full = torch.cat([torch.ones((n, p), dtype=torch.bool, device=q.device), see.to(q.device)], 1)
        rows.append(attend(q[at:at + n], k[:p + n], v[:p + n], full))
        at += n
    return Rows(*(torch.cat(x) for x in zip(*rows)))


def mask_words(see_drafts, words, fill=0):
    """[T, words] int32 mask rows of the requests' [n, n] truth values; bits past n are `fill`."""
    rows = []
    for see in see_drafts:
        n = see.shape[0]
        bits = torch.full((n, 32 * words), fill, dtype=torch.int64)
        bits[:, :n] = see.cpu()
        w = (bits.view(n, words, 32) << torch.arange(32)).sum(-1)
        rows.append(torch.where(w >= 1 << 31, w - (1 << 32), w).to(torch.int32))
    return torch.cat(rows)


def random_tree(gen, n):
    """Visibility of a random tree: a draft sees itself and its ancestors."""
    see = torch.eye(n, dtype=torch.bool)
    for i in range(1, n):
        parent = int(torch.randint(-1, i, (1,), generator=gen))
        if parent >= 0:
            see[i] |= see[parent]
    return see


def check_rows(out, lse, ref: Rows, what=""):
    """Every element of out and lse within the bounds above; empty rows exactly 0 and -inf."""
    empty = ref.lse == -math.inf
    assert torch.equal(lse == -math.inf, empty), f"{what}: rows without keys"
    assert torch.isfinite(out).all() and torch.isfinite(lse[~empty]).all(), f"{what}: non-finite values"
    e = (out.double() - ref.out).abs()
    worst = float((e / ref.out_tol.clamp_min(1e-300)).max()) if e.numel() else 0.0
    assert bool((e <= ref.out_tol).all()), f"{what}: out off by {worst:.3f} of its bound"
    assert not out[empty].any(), f"{what}: an empty row is not zero"
    el = (lse.double() - ref.lse)[~empty].abs()
    assert bool((el <= ref.lse_tol[~empty]).all()), f"{what}: lse off by {float((el / ref.lse_tol[~empty]).max()):.3f} of its bound"
    return worst


class Pool:
    """A paged cache's state on the host, and its operators from their definitions."""

    def __init__(self, k, v, refs, table, lens):
        self.k, self.v = k.clone().cpu(), v.clone().cpu()
        self.refs, self.table, self.lens = [list(x) if x and not isinstance(x[0], list) else [list(r) for r in x]
                                            for x in (refs, table, lens)]
        self.size = k.shape[2]

    def pages(self, b):
        row = self.table[b]
        n = next((c for c, p in enumerate(row) if p < 0), len(row))
        return row[:n]

    def take(self):
        p = self.refs.index(0)
        self.refs[p] = 1
        return p

    def reserve(self, want):
        cap = len(self.table[0])
        for b, n in enumerate(want):
            have = len(self.pages(b))
            missing = min(-(-max(n, 0) // self.size), cap) - have
            if missing <= 0:
                continue
            if missing > self.refs.count(0):
                return False
            for c in range(have, have + missing):
                self.table[b][c] = self.take()
        return True

    def append(self, k_new, v_new, start, new, codes=None):
        at = 0
        for b, (p, n) in enumerate(zip(start, new)):
            for i in range(max(n, 0)):
                c, r = divmod(p + i, self.size)
                if p >= 0 and c < len(self.table[b]) and 0 <= self.table[b][c] < len(self.refs):
                    for pool, x in ((self.k, k_new), (self.v, v_new)):
                        pool[self.table[b][c], :, r] = x[at + i]
            at += max(n, 0)

    def free(self, seqs):
        for b in dict.fromkeys(seqs):
            if 0 <= b < len(self.table):
                for c, p in enumerate(self.pages(b)):
                    if p < len(self.refs) and self.refs[p] > 0:
                        self.refs[p] -= 1
                    self.table[b][c] = -1
                self.lens[b] = 0

    def fork(self, src, dst):
        rows = [(self.pages(a) if 0 <= a < len(self.table) else [], self.lens[a] if 0 <= a < len(self.lens) else 0)
                for a in src]
        seen = set()
        for (pages, n), a, b in zip(rows, src, dst):
            if not (0 <= a < len(self.table) and 0 <= b < len(self.table)) or b in seen or self.table[b][0] >= 0:
                seen.add(b)
                continue
            seen.add(b)
            full, tail = divmod(n, self.size)
            used = pages[:-(-n // self.size)]
            if len(used) < -(-n // self.size) or any(p >= len(self.refs) or self.refs[p] < 1 for p in used):
                continue
            if tail and 0 not in self.refs:
                continue
            row = used[:full]
            for p in row:
                self.refs[p] += 1
            if tail:
                row = row + [self.take()]
                for pool in (self.k, self.v):
                    pool[row[full], :, :tail] = pool[used[full], :, :tail]
            self.table[b] = row + [-1] * (len(self.table[b]) - len(row))
            self.lens[b] = n

    def compact(self, start, keep, keep_lens):
        before = list(self.refs)  # the checks see the references as they stood before the call
        for b, (a, m) in enumerate(zip(start, keep_lens)):
            if m < 0:
                continue
            kept, pages, cap = keep[b][:m], self.pages(b), len(self.table[b]) * self.size
            if a < 0 or m > len(keep[b]) or any(x >= y for x, y in zip([-1] + kept, kept)) or a + max([m] + [x + 1 for x in kept]) > cap:
                continue
            moved = [i for i, x in enumerate(kept) if x != i]
            if moved:
                first, last, wrote = (a + moved[0]) // self.size, (a + kept[-1]) // self.size, (a + m - 1) // self.size
                if last >= len(pages) or any(not 0 <= pages[c] < len(self.refs) for c in range(first, last + 1)) or \
                        any(before[pages[c]] != 1 for c in range(first, wrote + 1)):
                    continue
            for i in moved:
                (c0, r0), (c1, r1) = divmod(a + kept[i], self.size), divmod(a + i, self.size)
                for pool in (self.k, self.v):
                    pool[pages[c1], :, r1] = pool[pages[c0], :, r0]
            self.lens[b] = a + m
            for c in range(-(-(a + m) // self.size), len(pages)):
                p = pages[c]
                if p < len(self.refs) and self.refs[p] > 0:
                    self.refs[p] -= 1
                self.table[b][c] = -1
