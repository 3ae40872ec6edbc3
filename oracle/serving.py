"""float64 definitions of the serving operators: rotary positions, the paged key/value cache and its pages.

Written from the definitions, one row and one request at a time; no code is shared with the CUDA path.
"""
from __future__ import annotations

import math

import numpy as np

from .attention import as_f64, attention_fwd_general


def rotary(x, positions, freqs, magnitude=1.0, interleaved=False, inverse=False):
    """x [B, H, N, d] with the pairs of its first 2 len(freqs) columns multiplied, as complex numbers, by
    magnitude e^(i pos f) (e^(-i pos f) for the inverse map, its transpose).  positions: [N] or [B, N]."""
    x = as_f64(x)
    f = np.asarray(freqs, np.float64)
    r = 2 * f.size
    pos = np.broadcast_to(np.asarray(positions, np.float64), (x.shape[0], x.shape[2]))
    # the angle modulo a turn, in extended precision: far positions lose nothing
    turns = pos[..., None].astype(np.longdouble) * f.astype(np.longdouble)
    angle = np.fmod(turns, 2 * np.longdouble("3.14159265358979323846264338327950288")).astype(np.float64)
    w = magnitude * np.exp((-1j if inverse else 1j) * angle)[:, None]
    y = x.copy()
    a, b = (x[..., 0:r:2], x[..., 1:r:2]) if interleaved else (x[..., :r // 2], x[..., r // 2:r])
    z = (a + 1j * b) * w
    if interleaved:
        y[..., 0:r:2], y[..., 1:r:2] = z.real, z.imag
    else:
        y[..., :r // 2], y[..., r // 2:r] = z.real, z.imag
    return y


def gather(pages, table_row, n):
    """Keys 0 .. n - 1 of one sequence, [H_kv, n, d], from pages [P, H_kv, page_size, d]."""
    page = pages.shape[2]
    rows = [pages[table_row[j // page], :, j % page] for j in range(n)]
    return np.stack(rows, axis=1) if rows else np.zeros((pages.shape[1], 0, pages.shape[3]))


def paged_decode(q, k_pages, v_pages, table, lens, scale, causal=True):
    """O [B, H, N, d], lse [B, H, N] of the last N positions of each sequence."""
    q = as_f64(q)
    o, lse = np.zeros(q.shape), np.full(q.shape[:3], -math.inf)
    for b, n in enumerate(lens):
        if n > 0:
            k, v = (gather(as_f64(p), table[b], n)[None] for p in (k_pages, v_pages))
            o[b], lse[b] = (x[0] for x in attention_fwd_general(q[b:b + 1], k, v, scale, causal))
    return o, lse


def paged_append(k_pages, v_pages, table, lens, tokens):
    """tokens: per sequence (k, v) of [H_kv, n, d], written at the sequence's last n positions; new (k_pages, v_pages)."""
    kp, vp = k_pages.copy(), v_pages.copy()
    page = kp.shape[2]
    for b, (k, v) in enumerate(tokens):
        n = k.shape[1]
        for i in range(n):
            j = lens[b] - n + i
            if j >= 0:
                kp[table[b][j // page], :, j % page] = k[:, i]
                vp[table[b][j // page], :, j % page] = v[:, i]
    return kp, vp


class Pages:
    """The bookkeeping of a paged cache, one request after the other."""

    def __init__(self, table, lens, refs, page_size):
        self.table, self.lens, self.refs = (np.array(x, np.int32) for x in (table, lens, refs))
        self.page = page_size

    def _pages(self, n):
        return -(-int(n) // self.page)

    def _grant(self, wants):
        """Pages for each request (None: refused): granted while all that was asked for so far was free."""
        free, asked, got = [p for p, n in enumerate(self.refs) if n == 0], 0, []
        for w in wants:
            asked += w
            got.append(free[asked - w:asked] if w == 0 or asked <= len(free) else None)
        return got

    def extend(self, seqs, tokens):
        S, M = self.table.shape
        named, wants, status = set(), [], []
        for s, t in zip(seqs, tokens):
            ok = 0 <= s < S and t >= 0 and 0 <= self.lens[s] <= M * self.page and self.lens[s] + t <= M * self.page \
                and s not in named
            wants.append(self._pages(self.lens[s] + t) - self._pages(self.lens[s]) if ok else 0)
            status.append(0 if ok else 1)
            if ok:
                named.add(s)
        for i, pages in enumerate(self._grant(wants)):
            if status[i] == 0 and pages is None:
                status[i] = 4
            elif status[i] == 0:
                at = self._pages(self.lens[seqs[i]])
                self.table[seqs[i], at:at + len(pages)] = pages
                self.refs[pages] = 1
                self.lens[seqs[i]] += tokens[i]
        return status

    def fork(self, src, dst):
        S, M = self.table.shape
        lens, named, status, copies = self.lens.copy(), set(), [], []
        for s, t in zip(src, dst):
            ok = 0 <= s < S and 0 <= t < S and s != t and lens[t] == 0 and 0 <= lens[s] <= M * self.page and t not in named
            status.append(0 if ok else 1)
            if ok:
                named.add(t)
        got = self._grant([int(status[i] == 0 and lens[s] % self.page != 0) for i, s in enumerate(src)])
        for i, (s, t) in enumerate(zip(src, dst)):
            if status[i] == 0 and got[i] is None:
                status[i] = 4
            elif status[i] == 0:
                full = lens[s] // self.page
                self.table[t, :full] = self.table[s, :full]
                np.add.at(self.refs, self.table[s, :full], 1)
                if got[i]:
                    copies.append([self.table[s, full], got[i][0], lens[s] % self.page])
                    self.table[t, full] = got[i][0]
                    self.refs[got[i][0]] = 1
                self.lens[t] = lens[s]
        return copies + [[-1, -1, -1]] * (len(src) - len(copies)), status

    def free(self, seqs):
        for s in seqs:
            n = self._pages(self.lens[s])
            np.add.at(self.refs, self.table[s, :n], -1)
            self.table[s, :n] = -1
            self.lens[s] = 0

    def compact(self):
        live = int((self.refs > 0).sum())
        holes = [p for p in range(live) if self.refs[p] == 0]
        moves = {p: holes.pop(0) for p in range(live, self.refs.size) if self.refs[p] > 0}
        for p, to in moves.items():
            self.refs[to], self.refs[p] = self.refs[p], 0
        for s, n in enumerate(self.lens):
            for e in range(self._pages(n)):
                self.table[s, e] = moves.get(int(self.table[s, e]), self.table[s, e])
        copies = [[p, to, self.page] for p, to in moves.items()]
        return copies + [[-1, -1, -1]] * (self.refs.size // 2 - len(copies))


def copy_pages(pages, copies):
    """pages [P, H_kv, page_size, d] after the listed copies (those with a source)."""
    new = pages.copy()
    for src, dst, rows in copies:
        if src >= 0:
            new[dst, :, :rows] = pages[src, :, :rows]
    return new
