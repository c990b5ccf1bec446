"""Plain 64-bit oracles of the target's side of a draft step: the paged cache's metadata and
copies (one Python statement a token), attention from its definition, draft verification from its
definition. NumPy and CPU torch only; nothing here is shared with the library.
"""
from __future__ import annotations

import math

import numpy as np
import torch


class CacheOracle:
    """An xpress_cache on the host, its calls carried out one row after the other."""

    def __init__(self, n_layers, n_pages, Hkv, page, D, rows, ld, dtype, seed=0):
        g = torch.Generator().manual_seed(seed)
        shape = (n_layers, n_pages, Hkv, page, D)
        self.k = torch.randn(shape, generator=g).to(dtype)
        self.v = torch.randn(shape, generator=g).to(dtype)
        self.table = np.full((rows, ld), -1, np.int32)
        self.length = np.zeros(rows, np.int32)
        self.ref = np.zeros(n_pages, np.int32)
        self.page = page

    def pages(self, n):
        return -(-int(n) // self.page)

    def release(self, r, keep):
        for j in range(self.pages(keep), self.pages(self.length[r])):
            self.ref[self.table[r, j]] -= 1
            self.table[r, j] = -1
        self.length[r] = keep

    def fork(self, src, dst):
        for a, b in zip(src, dst):
            self.release(b, 0)
            self.table[b] = self.table[a]
            self.length[b] = self.length[a]
            for j in range(self.pages(self.length[b])):
                self.ref[self.table[b, j]] += 1

    def extend(self, rows, add):
        free = [int(p) for p in np.nonzero(self.ref == 0)[0]]
        ref0 = self.ref.copy()
        plan = []
        for r, a in zip(rows, add):
            a = max(int(a), 0)
            n, after = int(self.length[r]), int(self.length[r]) + a
            if after > self.table.shape[1] * self.page:
                return -1
            cow = a > 0 and n % self.page and ref0[self.table[r, n // self.page]] > 1
            first = self.pages(n) - (1 if cow else 0)
            plan.append((r, after, first, self.pages(after) - first, cow))
        total = sum(p[3] for p in plan)
        if total > len(free):
            return total - len(free)
        copies = []
        for r, after, first, count, cow in plan:
            for j in range(count):
                p = free.pop(0)
                if j == 0 and cow:
                    old = int(self.table[r, first])
                    self.ref[old] -= 1
                    copies.append((old, p))
                self.table[r, first + j] = p
                self.ref[p] = 1
            self.length[r] = after
        for old, p in copies:
            self.k[:, p] = self.k[:, old]
            self.v[:, p] = self.v[:, old]
        return 0

    def append(self, layer, k_new, v_new, rows, B):
        for i, r in enumerate(rows):
            for b in range(B):
                pos = int(self.length[r]) - B + b
                if pos >= 0:
                    p, line = int(self.table[r, pos // self.page]), pos % self.page
                    self.k[layer, p, :, line] = k_new[i * B + b]
                    self.v[layer, p, :, line] = v_new[i * B + b]

    def trim(self, rows, drop):
        for i, r in enumerate(rows):
            d = self.length[r] if drop is None else min(max(int(drop[i]), 0), int(self.length[r]))
            self.release(r, int(self.length[r]) - int(d))

    def compact(self):
        live = int((self.ref > 0).sum())
        frm = [p for p in range(live, len(self.ref)) if self.ref[p] > 0]
        to = [p for p in range(live) if self.ref[p] == 0]
        place = dict(zip(frm, to))
        for a, b in place.items():
            self.k[:, b] = self.k[:, a]
            self.v[:, b] = self.v[:, a]
            self.ref[b], self.ref[a] = self.ref[a], 0
        for r in range(len(self.length)):
            for j in range(self.pages(self.length[r])):
                self.table[r, j] = place.get(int(self.table[r, j]), int(self.table[r, j]))
        return live


def attention(k, v, table, lengths, page, q, rows, B, Hq, scale):
    """out [N*B, Hq, D], lse [N*B, Hq], and per (token, head, channel) the weighted sum of |v| and
    per (token, head) the largest sum of |q k| * scale, all float64. k, v: one layer, [n_pages,
    Hkv, page, D]."""
    n_pages, Hkv, _, D = k.shape
    G = Hq // Hkv
    N = len(rows)
    out = torch.zeros(N * B, Hq, D, dtype=torch.float64)
    lse = torch.full((N * B, Hq), -math.inf, dtype=torch.float64)
    mass = torch.zeros(N * B, Hq, D, dtype=torch.float64)
    size = torch.zeros(N * B, Hq, dtype=torch.float64)
    q = q.double().view(N * B, Hq, D)
    for i, r in enumerate(rows):
        for b in range(B):
            see = int(lengths[r]) - B + b + 1
            if see <= 0:
                continue
            at = torch.arange(see)
            ids = torch.as_tensor(np.asarray(table[r], dtype=np.int64))[at // page]
            kk = k[ids, :, at % page].double()  # [see, Hkv, D]
            vv = v[ids, :, at % page].double()
            t = i * B + b
            for h in range(Hq):
                x = q[t, h]
                s = (kk[:, h // G] @ x) * scale
                lse[t, h] = torch.logsumexp(s, 0)
                p = torch.exp(s - lse[t, h])
                out[t, h] = p @ vv[:, h // G]
                mass[t, h] = p @ vv[:, h // G].abs()
                size[t, h] = (kk[:, h // G].abs() @ x.abs()).max() * scale
    return out, lse, mass, size


def attention_bounds(out, mass, size, keys, D, dtype):
    """How far a result may be off: (out, lse). One rounding of the result and one of every weight
    to the type (half a step each, against the weighted sum of |v|), and 32-bit sums: a score is
    off by D * 2^-24 of the sum of its products' sizes (twice: the score's and the maximum's), a
    sum of `keys` weights by keys * 2^-24, an exponential by 2^-22."""
    half = torch.finfo(dtype).eps / 2
    slack = 2 * size * D * 2.0 ** -24 + keys * 2.0 ** -24 + 2.0 ** -22
    tiny = torch.finfo(dtype).tiny * half * 2  # a step of the type's subnormals
    return (half * out.abs() + mass * (half * (1 + half) + slack[..., None] * (1 + half)) + tiny,
            slack + 2.0 ** -22)


def verify(logits, blk, draft_len, q, temperature, u):
    """out, accepted; logits [N*B, V], q [N*(B-1), V] or None, as float64 NumPy arrays."""
    N, B = blk.shape
    V = logits.shape[1]
    out = np.full((N, B), -1, np.int64)
    accepted = np.zeros(N, np.int32)
    for n in range(N):
        t = 0.0 if temperature is None or not temperature[n] > 0 else float(temperature[n])
        limit = B - 1 if draft_len is None else min(max(int(draft_len[n]), 0), B - 1)
        a = 0
        while True:
            x = logits[n * B + a]
            x = np.where(np.isnan(x), -np.inf, x)
            top = x.max()
            if top == -np.inf:
                break
            d = int(blk[n, a + 1]) if a < limit else -1
            if t == 0:
                best = int(np.argmax(x))
                if a < limit and d == best:
                    out[n, a] = d
                    a += 1
                    continue
                out[n, a] = best
                break
            with np.errstate(invalid="ignore"):
                w = np.where(x == top, 1.0, np.exp((x - top) / t))
            p = w / w.sum()
            if a < limit and 0 <= d < V:
                qd = 1.0 if q is None else q[n * (B - 1) + a, d]
                if float(u[n, a]) * qd < p[d]:
                    out[n, a] = d
                    a += 1
                    continue
            # weights need no common scale: w has no rounding of a division in it, so that running
            # sums of equal weights are exact and a border that u meets exactly stays one
            left = w
            if a < limit:
                if q is None:
                    left = w.copy()
                    if 0 <= d < V:
                        left[d] = 0
                else:
                    left = np.maximum(p - q[n * (B - 1) + a], 0)
                if not left.sum() > 0:
                    left = w
            run = np.cumsum(left)
            hit = np.nonzero((run > float(u[n, B - 1]) * run[-1]) & (left > 0))[0]
            out[n, a] = hit[0] if len(hit) else np.nonzero(left > 0)[0][-1]
            break
        accepted[n] = a
    return out, accepted
