"""Plain 64-bit references of the cache, the attention over it and its page
operations, for the tests (numpy and Python integers)."""
import numpy as np

PAGE = 64
E_MIN = -100


def e4m3(x):
    """Nearest e4m3 value, ties to even, |x| <= 448 (float64)."""
    x = np.asarray(x, np.float64)
    a = np.maximum(np.abs(x), 2.0 ** -6)
    step = np.exp2(np.floor(np.log2(a)) - 3)
    return np.rint(x / step) * step


def scale_of(amax):
    """Smallest 2^e with amax <= 448 * 2^e, e >= E_MIN (amax finite)."""
    e = np.full(np.shape(amax), E_MIN, np.int64)
    while True:
        small = amax > 448.0 * np.exp2(e.astype(np.float64))
        if not small.any():
            return np.exp2(e.astype(np.float64))
        e = np.where(small, e + 1, e)


class Side:
    """Keys or values of one layer: per page and head 64 values and a scale."""

    def __init__(self, pages, heads, dim):
        self.val = np.zeros((pages, heads, PAGE, dim))
        self.scale = np.zeros((pages, heads))

    def append(self, pages, start, rows):
        """rows [n, heads, dim] float64 at positions start.. of a sequence whose pages are `pages`."""
        n = rows.shape[0]
        t = start
        while t < start + n:
            p, lo = pages[t // PAGE], t % PAGE
            hi = min(PAGE, lo + start + n - t)
            part = rows[t - start:t - start + hi - lo]
            good = np.isfinite(part)
            fin = np.where(good, part, 0.0)
            s = scale_of(np.abs(fin).max(axis=(0, 2)))
            bad = ~good.all(axis=(0, 2))
            if lo:
                old = self.scale[p]
                bad |= np.isnan(old)
                s = np.where(np.isnan(old), s, np.maximum(s, old))
                self.val[p, :, :lo] = e4m3(self.val[p, :, :lo] / s[:, None, None]) * s[:, None, None]
            self.val[p, :, lo:hi] = (e4m3(fin / s[None, :, None]) * s[None, :, None]).transpose(1, 0, 2)
            self.scale[p] = np.where(bad, np.nan, s)
            t += hi - lo

    def read(self, pages, first, n):
        """[n, heads, dim]; a poisoned block reads as NaN."""
        out = np.empty((n, self.val.shape[1], self.val.shape[3]))
        for i in range(n):
            p, s = pages[(first + i) // PAGE], (first + i) % PAGE
            out[i] = self.val[p, :, s] + np.where(np.isnan(self.scale[p]), np.nan, 0.0)[:, None]
        return out


def attention(q, k, v, first, window, sinks, scale):
    """q [n, heads, dim] at positions first.., k and v [total, kv_heads, dim]:
    (out, lse, weighted sum of |v|, largest sum of |q||k| that a row sees)."""
    n, hq, d = q.shape
    total, hk, _ = k.shape
    out, mag = np.zeros((n, hq, d)), np.zeros((n, hq, d))
    lse, big = np.full((n, hq), -np.inf), np.zeros((n, hq))
    for i in range(n):
        p = first + i
        j = np.arange(total)
        see = j <= p
        if window:
            see &= (j > p - window) | (j < sinks)
        if not see.any():
            continue
        for h in range(hq):
            kk, vv = k[see, h // (hq // hk)], v[see, h // (hq // hk)]
            t = kk @ q[i, h] * scale
            m = t.max()
            w = np.exp(t - m)
            out[i, h] = w @ vv / w.sum()
            mag[i, h] = w @ np.abs(vv) / w.sum()
            lse[i, h] = m + np.log(w.sum())
            big[i, h] = (np.abs(kk) @ np.abs(q[i, h])).max() * abs(scale)
    return out, lse, mag, big


class Pool:
    """Tables, references and lengths, step by step."""

    def __init__(self, pages, max_seqs, max_pages):
        self.refs, self.max_pages = [0] * pages, max_pages
        self.rows = [[] for _ in range(max_seqs)]
        self.lens = [0] * max_seqs

    def table(self):
        return np.array([r + [-1] * (self.max_pages - len(r)) for r in self.rows], np.int32)

    def reserve(self, seqs, counts):
        """(start list, copies (src, dst)), or None when there is too little room."""
        save = (list(self.refs), [list(r) for r in self.rows], list(self.lens))
        start, copies = [], []
        try:
            for s, c in zip(seqs, counts):
                n = self.lens[s]
                row = self.rows[s]
                if c and n % PAGE and self.refs[row[-1]] > 1:
                    p = self.refs.index(0)
                    copies.append((row[-1], p))
                    self.refs[row[-1]] -= 1
                    self.refs[p] = 1
                    row[-1] = p
                while len(row) * PAGE < n + c:
                    p = self.refs.index(0)
                    if len(row) == self.max_pages:
                        raise ValueError
                    self.refs[p] = 1
                    row.append(p)
                start.append(n)
                self.lens[s] = n + c
        except ValueError:
            self.refs, self.rows, self.lens = save
            return None
        return start, copies

    def fork(self, a, b):
        self.rows[b], self.lens[b] = list(self.rows[a]), self.lens[a]
        for p in self.rows[a]:
            self.refs[p] += 1

    def free(self, s):
        for p in self.rows[s]:
            self.refs[p] -= 1
        self.rows[s], self.lens[s] = [], 0

    def compact(self):
        """Moves (src, dst)."""
        live = sum(r > 0 for r in self.refs)
        moves = list(zip([p for p in range(live, len(self.refs)) if self.refs[p]],
                         [p for p in range(live) if not self.refs[p]]))
        to = dict(moves)
        for s, d in moves:
            self.refs[d], self.refs[s] = self.refs[s], 0
        self.rows = [[to.get(p, p) for p in r] for r in self.rows]
        return moves, live
