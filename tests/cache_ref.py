"""Plain references of the paged cache's operators, in float64 and whole numbers (NumPy only).

The cache is kept in its natural form here, one [H, slots, D] array a sequence, and packed
into the library's layout by `pack`; nothing of the library is used.
"""
from __future__ import annotations

import numpy as np


def pack_k(k, t, pages, page_ids, page, E):
    """Key k [H, D] of slot t into pages [P, H, D/E, page, E]."""
    pages[page_ids[t // page], :, :, t % page, :] = k.reshape(k.shape[0], -1, E)


def pack_v(v, t, pages, page_ids, page, E):
    """Value v [H, D] of slot t into pages [P, H, page/E, D, E]."""
    pages[page_ids[t // page], :, (t % page) // E, :, t % E] = v


def unpack(k_pages, v_pages, page_ids, n, page, E):
    """Keys and values [H, n, D] of slots 0 .. n-1 of a sequence with these pages."""
    P, H, U, _, _ = k_pages.shape
    k = np.zeros((H, n, U * E), k_pages.dtype)
    v = np.zeros((H, n, U * E), k_pages.dtype)
    for t in range(n):
        k[:, t] = k_pages[page_ids[t // page], :, :, t % page, :].reshape(H, -1)
        v[:, t] = v_pages[page_ids[t // page], :, (t % page) // E, :, t % E]
    return k, v


def lineage(parent, i):
    """Node i and its ancestors, and i's depth."""
    line = [i]
    while parent[line[-1]] >= 0:
        line.append(int(parent[line[-1]]))
    return line, len(line) - 1


def seen_slots(n, m, parent, i, window, sinks):
    """The slots node i of a sequence with n committed tokens sees, ascending."""
    line, depth = lineage(parent, i)
    pos = n + depth
    slots = [t for t in range(n) if not window or pos - t < window or t < sinks]
    for j in sorted(line):
        pj = n + lineage(parent, j)[1]
        if not window or pos - pj < window or pj < sinks:
            slots.append(n + j)
    return slots


def attention(q, ks, vs, lens, news, parents, scale, window, sinks, esz):
    """out [B, N, Hq, D] in float64 and, per element, how far an evaluation with f32 scores,
    statistics and sums and with weights and outputs rounded to esz bytes may be off.

    The allowance follows the evaluation's steps, u = 2^-24 (half a step of f32), w = half a
    step of the type (2^-8 bf16, u for f32), A = sum_t p_t |v_t|:
      - a score is a sum of D exact (bf16) or rounded (f32) products in f32, times a constant:
        off by at most (D + 4) u scale sum_d |q_d k_d| =: dz; a weight then by a factor of
        e^(2 dz) at most (its own score and the normaliser), plus exp2's 2 u
      - rounding the weights: w A
      - sums over T weights or products in f32: at most (T + 8) u relative to A each, and a
        rescaling of the sums each time the maximum moves (2 u each, at most T / 32 of them)
      - the output's rounding: w |out|
    """
    B, N, Hq, D = q.shape
    u, w = 2.0 ** -24, (2.0 ** -8 if esz == 2 else 2.0 ** -24)
    out, tol = np.zeros((B, N, Hq, D)), np.zeros((B, N, Hq, D))
    for b in range(B):
        H = ks[b].shape[0]
        g = Hq // H
        par = parents[b] if parents is not None else np.arange(-1, N - 1)
        for i in range(news[b]):
            at = seen_slots(lens[b], news[b], par, i, window, sinks)
            T = len(at)
            for h in range(Hq):
                k, v = ks[b][h // g][at].astype(np.float64), vs[b][h // g][at].astype(np.float64)
                qq = q[b, i, h].astype(np.float64)
                with np.errstate(invalid="ignore", over="ignore"):
                    z = scale * (k @ qq)
                    p = np.exp(z - z.max())
                    p /= p.sum()
                    out[b, i, h] = p @ v
                    A = p @ np.abs(v)
                    dz = (D + 4) * u * abs(scale) * (np.abs(k) @ np.abs(qq)).max()
                    f = 2 * dz * 1.1 + w + (2 * (T + 8) + T / 16 + 8) * u
                    tol[b, i, h] = f * A + w * (np.abs(out[b, i, h]) + f * A) + 1e-37
    return out, tol


class Books:
    """The pool's books, kept with lists: what spec_cache_resize and spec_cache_fork do to them."""

    def __init__(self, P, S, W, page):
        self.P, self.S, self.W, self.page = P, S, W, page
        self.rows = [[] for _ in range(S)]
        self.ref = [0] * P

    def table(self):
        t = np.full((self.S, self.W), -1, np.int32)
        for b, r in enumerate(self.rows):
            t[b, :len(r)] = r
        return t

    def free_map(self):
        words = np.zeros((self.P + 31) // 32, np.uint32)
        for p, r in enumerate(self.ref):
            if r == 0:
                words[p // 32] |= np.uint32(1 << (p % 32))
        return words.view(np.int32)

    def resize(self, keep, want):
        """(status, copies): copies are (from, to, slots) triples."""
        page, status = self.page, [0] * self.S
        for b in range(self.S):
            if want[b] < 0:
                continue
            if -(-want[b] // page) > self.W or keep[b] < 0 or keep[b] > len(self.rows[b]) * page:
                status[b] = -8
                continue
            goal = -(-want[b] // page)
            for p in self.rows[b][goal:]:
                self.ref[p] -= 1
            del self.rows[b][goal:]
        free = [p for p in range(self.P) if self.ref[p] == 0]
        ref, copies, later, refused = list(self.ref), [], [], False
        for b in range(self.S):
            if want[b] < 0 or status[b] or want[b] <= keep[b]:
                continue
            row, goal, first = self.rows[b], -(-want[b] // page), keep[b] // page
            swap = [i for i in range(first, min(len(row), goal)) if ref[row[i]] > 1]
            need = len(swap) + max(0, goal - len(row))
            if need == 0:
                continue
            if refused or need > len(free):
                status[b], refused = -9, True
                continue
            for i in swap:
                new = free.pop(0)
                if i == first and keep[b] % page:
                    copies.append((row[i], new, keep[b] % page))
                later.append(row[i])
                row[i] = new
                self.ref[new] = 1
            while len(row) < goal:
                new = free.pop(0)
                row.append(new)
                self.ref[new] = 1
        for p in later:
            self.ref[p] -= 1
        return status, copies

    def fork(self, lens, src, dst):
        status = []
        for i, (s, d) in enumerate(zip(src, dst)):
            ok = 0 <= s < self.S and 0 <= d < self.S and d not in src and d not in dst[:i] and not self.rows[d]
            status.append(0 if ok else -10)
        for s, d, st in zip(src, dst, status):
            if st == 0:
                self.rows[d] = list(self.rows[s])
                lens[d] = lens[s]
                for p in self.rows[s]:
                    self.ref[p] += 1
        return status
