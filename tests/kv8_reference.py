"""Plain 64-bit form of the paged 8-bit cache (NumPy, one token at a time), the
oracle of tests/test_gpu_kv8.py.  Codes are kept as the values they stand for
before the scale (float64), so that int8 and e4m3 share the code below."""
import math

import numpy as np

INT8, E4M3 = 0, 1
QMAX = {INT8: 127.0, E4M3: 448.0}


def nearest(x, fmt):
    """Nearest code values, ties to even."""
    if fmt == INT8:
        return np.rint(x)
    _, e = np.frexp(x)
    step = 2.0 ** np.maximum(e - 4, -9)  # three fraction bits; the subnormal step is 2^-9
    return np.rint(x / step) * step


def scale_for(amax, fmt):
    e = -126
    while amax > QMAX[fmt] * 2.0 ** e:
        e += 1
    return 2.0 ** e


class Refused(Exception):
    pass


class Cache:
    def __init__(self, fmt, layers, kvh, d, ps, num_pages, num_slots, max_pages):
        self.fmt, self.layers, self.kvh, self.d, self.ps = fmt, layers, kvh, d, ps
        self.num_pages, self.num_slots, self.max_pages = num_pages, num_slots, max_pages
        self.codes = np.zeros((num_pages, layers, 2, kvh, ps, d))
        self.scales = np.ones((num_pages, layers, 2, kvh))
        self.table = np.full((num_slots, max_pages), -1)
        self.lens = np.zeros(num_slots, dtype=int)
        self.refs = np.zeros(num_pages, dtype=int)

    def pages(self, n):
        return -(-n // self.ps)

    def _copy(self, a, b):
        self.codes[b], self.scales[b] = self.codes[a], self.scales[a]

    def resize(self, slots, new):
        if len(set(slots)) < len(slots) or any(not 0 <= s < self.num_slots for s in slots) or \
                any(n < 0 or self.pages(n) > self.max_pages for n in new):
            raise Refused
        refs, plan = self.refs.copy(), []
        for s, n in zip(slots, new):
            keep = min(n, self.lens[s])
            plan.append(keep % self.ps > 0 and self.refs[self.table[s, keep // self.ps]] > 1)
        for s, n in zip(slots, new):
            for j in range(self.pages(n), self.pages(self.lens[s])):
                refs[self.table[s, j]] -= 1
        free = [p for p in range(self.num_pages) if refs[p] == 0]
        if len(free) < sum(plan) + sum(max(0, self.pages(n) - self.pages(self.lens[s])) for s, n in zip(slots, new)):
            raise Refused
        self.refs, moved = refs, []
        for s, n, copy in zip(slots, new, plan):
            old, keep = self.lens[s], min(n, self.lens[s])
            if copy:
                p = free.pop(0)
                moved.append((self.table[s, keep // self.ps], p))
                self.table[s, keep // self.ps] = p
                self.refs[p] = 1
            for j in range(self.pages(old), self.pages(n)):
                self.table[s, j] = free.pop(0)
                self.refs[self.table[s, j]] = 1
            self.table[s, self.pages(n):self.pages(old)] = -1
            self.lens[s] = n
        for a, b in moved:
            self._copy(a, b)
            self.refs[a] -= 1

    def fork(self, src, dst):
        slots = list(src) + list(dst)
        if len(set(dst)) < len(dst) or set(src) & set(dst) or any(not 0 <= s < self.num_slots for s in slots) or any(self.lens[t] for t in dst):
            raise Refused
        free = [p for p in range(self.num_pages) if self.refs[p] == 0]
        if len(free) < sum(self.lens[s] % self.ps > 0 for s in src):
            raise Refused
        for s, t in zip(src, dst):
            n = self.lens[s]
            for j in range(self.pages(n)):
                p = self.table[s, j]
                if (j + 1) * self.ps > n:
                    q = free.pop(0)
                    self._copy(p, q)
                    p = q
                self.table[t, j] = p
                self.refs[p] += 1
            self.lens[t] = n

    def compact(self):
        live = int((self.refs > 0).sum())
        high = [p for p in range(live, self.num_pages) if self.refs[p] > 0]
        hole = [p for p in range(live) if self.refs[p] == 0]
        for a, b in zip(high, hole):
            self._copy(a, b)
            self.refs[b], self.refs[a] = self.refs[a], 0
            for s in range(self.num_slots):
                used = self.table[s, :self.pages(self.lens[s])]
                used[used == a] = b
        return live

    def append(self, layer, k, v, slots, cu):
        """k, v float64 [rows, kvh, d] holding bf16 values."""
        for i, s in enumerate(slots):
            row, pos = cu[i], self.lens[s] - (cu[i + 1] - cu[i])
            while pos < self.lens[s]:
                p, off = self.table[s, pos // self.ps], pos % self.ps
                m = min(self.ps - off, self.lens[s] - pos)
                for side, src in enumerate((k, v)):
                    for h in range(self.kvh):
                        self._block(p, layer, side, h, off, src[row:row + m, h])
                pos, row = pos + m, row + m

    def _block(self, p, layer, side, h, off, x):
        old, tile = self.scales[p, layer, side, h], self.codes[p, layer, side, h]
        new = scale_for(np.max(np.abs(x)), self.fmt) if np.all(np.isfinite(x)) else math.nan
        if off and (math.isnan(old) or old > new):
            new = old
        if off and new > old:
            tile[:] = nearest(tile * (old / new), self.fmt)
        self.scales[p, layer, side, h] = new
        tile[off:off + len(x)] = 0.0 if math.isnan(new) else nearest(x / new, self.fmt)

    def values(self, layer, s):
        """keys, values float64 [len, kvh, d] of slot s"""
        ids = self.table[s, :self.pages(self.lens[s])]
        x = self.codes[ids, layer] * self.scales[ids, layer][..., None, None]  # [pages, 2, kvh, ps, d]
        x = x.transpose(1, 0, 3, 2, 4).reshape(2, -1, self.kvh, self.d)[:, :self.lens[s]]
        return x[0], x[1]

    def attention(self, layer, q, slots, cu):
        """q float64 [rows, heads, d] -> out, lse, and for the error bounds
        sum_t p_t |v_t| and max_t sum |q||k| / sqrt(d); rows of no sequence stay 0."""
        rows, heads, d = q.shape
        out, mag = np.zeros(q.shape), np.zeros(q.shape)
        lse, top = np.zeros((rows, heads)), np.zeros((rows, heads))
        for i, s in enumerate(slots):
            k, v = self.values(layer, s)
            for r in range(cu[i], cu[i + 1]):
                last = self.lens[s] - (cu[i + 1] - r)
                for h in range(heads):
                    kk, vv = k[:last + 1, h * self.kvh // heads], v[:last + 1, h * self.kvh // heads]
                    z = kk @ q[r, h] / math.sqrt(d)
                    m = z.max()
                    e = np.exp(z - m)
                    out[r, h] = e @ vv / e.sum()
                    mag[r, h] = e @ np.abs(vv) / e.sum()
                    lse[r, h] = m + math.log(e.sum())
                    top[r, h] = np.max(np.abs(kk) @ np.abs(q[r, h])) / math.sqrt(d)
        return out, lse, mag, top
