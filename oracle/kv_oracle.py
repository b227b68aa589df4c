"""Plain CPU references of the paged key/value cache: fp64 attention and rotation, and the page
pool's bookkeeping as a sequential program.

TEST INFRASTRUCTURE ONLY.  Only the test suite may import this module.  It shares no code
with the GPU library and never imports it.

  pool       a list of free pages used as a stack; sequences are served one after the other
  rotation   (x_i + i x_j) e^(i pos freq) for the pairs (i, j) of a head
  e4m3       nearest of the 127 finite magnitudes, ties to the even code, saturating
  attention  softmax of scale q.k over the visible positions, in fp64, position by position
"""
from __future__ import annotations

import numpy as np

NO_PAGES, TOO_LONG, BAD_SLOT, CLAMPED = 1, 2, 4, 8


class Pool:
    """The page pool, one sequence and one page at a time."""

    def __init__(self, batch, npages, page, max_pages):
        self.B, self.page, self.mp = batch, page, max_pages
        self.free = list(range(npages - 1, -1, -1))     # the top is the end
        self.rows = [[] for _ in range(batch)]          # pages held
        self.len, self.end, self.err = [0] * batch, [0] * batch, 0

    def reserve(self, counts, active=None, layout=None, rows=None):
        """counts per sequence; layout "step" (row i * B + b) or "packed".  Returns slots, pos, starts."""
        packed = layout == "packed"
        n_of = [int(c) if active is None or active[b] else 0 for b, c in enumerate(counts)]
        ntok = max([0] + [c for c in counts]) if not packed else 0
        rows = ntok * self.B if rows is None else rows
        slots, pos = np.full(rows, -1, np.int64), np.full(rows, -1, np.int32)
        starts, start, asked, avail = [], 0, 0, len(self.free)
        taken = []
        for b in range(self.B):
            n = n_of[b]
            if n < 0:
                self.err |= TOO_LONG
                n = 0
            starts.append(start)
            need = max(0, -(-(self.len[b] + n) // self.page) - len(self.rows[b]))
            served = self.len[b] + n <= self.mp * self.page and (not packed or start + n <= rows)
            if not served:
                self.err |= TOO_LONG
            else:
                first, asked = asked, asked + need
                if need and asked > avail:
                    served = False
                    self.err |= NO_PAGES
                elif need:
                    new = [self.free[avail - 1 - first - i] for i in range(need)]
                    self.rows[b] += new
                    taken.append(asked)
            self.end[b] = self.len[b] + n if served else self.len[b]
            for i in range(n):
                r = start + i if packed else i * self.B + b
                if served and r < rows:
                    p = self.len[b] + i
                    slots[r] = self.rows[b][p // self.page] * self.page + p % self.page
                    pos[r] = p
            start += n
        if taken:
            del self.free[avail - max(taken):]
        return slots, pos, starts + [start]

    def commit(self, accepted=None):
        for b in range(self.B):
            n = self.end[b] - self.len[b]
            if accepted is not None:
                if not 0 <= accepted[b] <= n:
                    self.err |= CLAMPED
                n = min(max(int(accepted[b]), 0), n)
            self.len[b] += n
            self.end[b] = self.len[b]

    def release(self, mask=None):
        out = [b for b in range(self.B) if mask is None or mask[b]]
        pages = [p for b in out for p in self.rows[b]]
        self.free += pages[::-1]
        for b in out:
            self.rows[b], self.len[b], self.end[b] = [], 0, 0

    def table(self):
        t = np.full((self.B, self.mp), -1, np.int32)
        for b, r in enumerate(self.rows):
            t[b, :len(r)] = r
        return t


def rotate(x, pos, freq, axis, rot, adjacent):
    """x [N][H][D] fp64, pos [A][N], freq [rot / 2], axis [rot / 2] -> rotated copy."""
    x = np.array(x, np.float64)
    for p in range(rot // 2):
        i, j = (2 * p, 2 * p + 1) if adjacent else (p, p + rot // 2)
        if axis is not None and axis[p] >= len(pos):
            continue
        where = np.asarray(pos[0 if axis is None else axis[p]], np.float64)
        z = (x[:, :, i] + 1j * x[:, :, j]) * np.exp(1j * where * np.float64(freq[p]))[:, None]
        x[:, :, i], x[:, :, j] = z.real, z.imag
    return x


def e4m3_values():
    """The 127 nonnegative finite E4M3 values, by code."""
    v = []
    for c in range(127):
        e, m = c >> 3, c & 7
        v.append(m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
    return np.array(v)


def to_e4m3(x):
    """Codes (uint8) of fp64 values."""
    x = np.asarray(x, np.float64)
    v = e4m3_values()
    a = np.minimum(np.abs(np.where(np.isnan(x), 0.0, x)), 448.0)
    hi = np.clip(np.searchsorted(v, a), 0, 126)
    lo = np.maximum(hi - 1, 0)
    up = (a - v[lo] > v[hi] - a) | ((a - v[lo] == v[hi] - a) & (hi % 2 == 0))
    code = np.where(up, hi, lo).astype(np.uint8)
    code = np.where(v[hi] == a, hi, code).astype(np.uint8)
    code |= np.where(np.signbit(x), 0x80, 0).astype(np.uint8)
    return np.where(np.isnan(x), 0x7f, code).astype(np.uint8)


def attention(q, K, V, table, end, scale, window=0, page_ok=None):
    """q [T][B][Hq][D]; K, V [npages][Hkv][page][D] (fp64); table [B][MP]; end [B].
    Returns o, lse, and for error bounds the largest scale * sum |q k| and sum p |v| of each row."""
    T, B, Hq, D = q.shape
    npages, Hkv, page, _ = K.shape
    G = Hq // Hkv
    o, a = np.zeros((T, B, Hq, D)), np.zeros((T, B, Hq, D))
    lse, top = np.full((T, B, Hq), -np.inf), np.zeros((T, B, Hq))
    for b in range(B):
        e = min(max(int(end[b]), 0), table.shape[1] * page)
        for t in range(T):
            p = e - T + t
            lo = max(0, p - window + 1) if window else 0
            js = [j for j in range(lo, p + 1) if 0 <= table[b, j // page] < npages]
            if not js:
                continue
            at, off = table[b, np.array(js) // page], np.array(js) % page
            for h in range(Hq):
                k, v = K[at, h // G, off], V[at, h // G, off]
                s = scale * (k @ q[t, b, h])
                m = s.max()
                w = np.exp(s - m)
                o[t, b, h] = (w / w.sum()) @ v
                a[t, b, h] = (w / w.sum()) @ np.abs(v)
                lse[t, b, h] = m + np.log(w.sum())
                top[t, b, h] = abs(scale) * (np.abs(k) @ np.abs(q[t, b, h])).max()
    return o, lse, top, a
