"""The paged-cache operators written out plainly: attention in float64, page bookkeeping in
Python integers, one stream and one page after the other."""

import numpy as np


def visible(at, j, window, sinks):
    return j <= at and (window <= 0 or j > at - window or j < sinks)


def attention(q, k_pages, v_pages, table, length, cu, scale, window=0, sinks=0):
    """(out, spread) in float64.  spread[row, h, d] = sum_j p_j |v_j - out|: the factor by which a
    relative error of the weights reaches the output."""
    rows, Hq, D = q.shape
    Hkv, P = k_pages.shape[1], k_pages.shape[2]
    G = Hq // Hkv
    out = np.full((rows, Hq, D), np.nan)
    spread = np.full((rows, Hq, D), np.nan)
    for b in range(len(length)):
        n = cu[b + 1] - cu[b] + 1
        for i in range(n):
            at = length[b] + i
            js = np.array([j for j in range(at + 1) if visible(at, j, window, sinks)])
            pages = table[b][js // P]
            for h in range(Hkv):
                k = k_pages[pages, h, js % P].astype(np.float64)
                v = v_pages[pages, h, js % P].astype(np.float64)
                for g in range(G):
                    row = cu[b] + b + i
                    s = k @ q[row, h * G + g].astype(np.float64) * scale
                    w = np.exp(s - s.max())
                    w /= w.sum()
                    o = w @ v
                    out[row, h * G + g] = o
                    spread[row, h * G + g] = w @ np.abs(v - o)
    return out, spread


class Book:
    """Page bookkeeping: page_table, held, length, ref_count and the contents of pages (any labels)."""

    def __init__(self, table, held, length, refs, page_size, contents):
        self.table = [list(map(int, r)) for r in table]
        self.held, self.length, self.refs = list(map(int, held)), list(map(int, length)), list(map(int, refs))
        self.P, self.contents = page_size, list(contents)
        self.width = len(self.table[0]) if self.table else 0

    def pages_of(self, n):
        return -(-n // self.P)

    def resize(self, advance=None, room=None):
        B = len(self.held)
        advance = [0] * B if advance is None else list(map(int, advance))
        room = [0] * B if room is None else list(map(int, room))
        status, keep, want, new = [0] * B, list(self.held), list(self.held), list(self.length)
        refs0 = list(self.refs)
        ok = lambda p: 0 <= p < len(self.refs)  # noqa: E731
        for b in range(B):
            n = self.length[b] + advance[b]
            if (self.length[b] < 0 or n < 0 or room[b] < 0 or not 0 <= self.held[b] <= self.width
                    or n > self.held[b] * self.P or n + room[b] > self.width * self.P):
                status[b] = 9
                continue
            w, full = self.pages_of(n + room[b]), self.pages_of(n)
            looked = list(range(full, self.held[b])) + ([n // self.P] if n % self.P and room[b] else [])
            if not all(ok(self.table[b][j]) for j in looked):
                status[b] = 10
                continue
            lim = min(w, self.held[b])
            shared = [j for j in range(full, lim) if refs0[self.table[b][j]] > 1]
            keep[b], want[b], new[b] = (min(shared) if shared else lim), w, n
        for b in range(B):
            for j in range(keep[b], self.held[b]):
                self.refs[self.table[b][j]] -= 1
                self.table[b][j] = -1
        asks = {}
        for b in range(B):
            if status[b] == 0 and room[b] and new[b] % self.P:
                p = self.table[b][new[b] // self.P]
                if self.refs[p] > 1:
                    asks.setdefault(p, []).append(b)
        copies = set()
        for p, who in asks.items():
            copies |= set(who[1:] if len(who) == self.refs[p] else who)
        free = [p for p in range(len(self.refs)) if self.refs[p] == 0]
        at = 0
        for b in range(B):
            need = want[b] - keep[b] + (b in copies)
            mine = free[at:at + need]
            at += need
            if status[b]:
                continue
            self.length[b] = new[b]
            if need and at > len(free):
                status[b] = 8
                self.held[b] = keep[b]
                continue
            if b in copies:
                j = new[b] // self.P
                old, p = self.table[b][j], mine.pop(0)
                self.contents[p] = self.contents[old]
                self.refs[old] -= 1
                self.refs[p] = 1
                self.table[b][j] = p
            for j in range(keep[b], want[b]):
                p = mine.pop(0)
                self.table[b][j] = p
                self.refs[p] = 1
            self.held[b] = want[b]
        return status

    def fork(self, src, dst):
        B, status = len(self.held), [0] * len(src)
        held0 = list(self.held)
        for e, (s, d) in enumerate(zip(src, dst)):
            if not (0 <= s < B and 0 <= d < B) or d in list(src) or d in list(dst)[:e]:
                status[e] = 11
                continue
            if (self.length[s] < 0 or not 0 <= held0[s] <= self.width or not 0 <= held0[d] <= self.width
                    or self.length[s] > held0[s] * self.P):
                status[e] = 9
                continue
            n = self.pages_of(self.length[s])
            if not all(0 <= p < len(self.refs) for p in self.table[s][:n] + self.table[d][:held0[d]]):
                status[e] = 10
                continue
            for p in self.table[d][:held0[d]]:
                self.refs[p] -= 1
            for p in self.table[s][:n]:
                self.refs[p] += 1
            self.table[d] = self.table[s][:n] + [-1] * max(0, held0[d] - n) + self.table[d][max(n, held0[d]):]
            self.held[d], self.length[d] = n, self.length[s]
        return status
