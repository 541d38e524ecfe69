"""The paged cache's operators in numpy fp64, from their formulas: rotary
positions, the cached rows' values, attention of one token over a page table,
and a model of the pages' bookkeeping.  Shares no code with the CUDA library."""
from __future__ import annotations

import math

import numpy as np

E4M3 = np.array([math.nan if (b & 0x7F) == 0x7F else
                 (-1.0 if b & 0x80 else 1.0) * ((b & 7) / 8.0 * 2.0 ** -6 if (b >> 3) & 15 == 0 else
                                                (1 + (b & 7) / 8.0) * 2.0 ** (((b >> 3) & 15) - 7))
                 for b in range(256)])


def bf16(bits):
    """bf16 bit patterns to fp64."""
    return (np.asarray(bits).view(np.uint16).astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def rope_frequencies(rot, base, kind="none", factor=1.0, trained=0):
    """(f_i in radians a position, factor on cos and sin)."""
    if kind == "ntk":
        base = base * factor ** (rot / (rot - 2))
    f = np.array([base ** (-2.0 * i / rot) for i in range(rot // 2)])
    if kind == "linear":
        f = f / factor
    if kind == "yarn":
        d = lambda turns: rot * math.log(trained / (2 * math.pi * turns)) / (2 * math.log(base))  # noqa: E731
        lo, hi = max(0, math.floor(d(32))), min(rot - 1, math.ceil(d(1)))
        r = np.array([min(1.0, max(0.0, (i - lo) / max(1e-3, hi - lo))) for i in range(rot // 2)])
        return f / factor * r + f * (1 - r), 0.1 * math.log(factor) + 1.0
    return f, 1.0


def rope(x, pos, f, scale, layout):
    """x fp64 [T][heads][D]; layout "half" or "interleaved"."""
    rot, y = 2 * len(f), np.array(x, np.float64)
    for t, p in enumerate(pos):
        for i, fi in enumerate(f):
            a, b = (i, i + rot // 2) if layout == "half" else (2 * i, 2 * i + 1)
            c, s = math.cos(float(p) * fi), math.sin(float(p) * fi)
            y[t, :, a] = scale * (x[t, :, a] * c - x[t, :, b] * s)
            y[t, :, b] = scale * (x[t, :, b] * c + x[t, :, a] * s)
    return y


def scale_of(byte):
    """ue8m0 bytes to fp64; 255 is NaN."""
    s = byte.astype(np.float64)
    return np.where(s == 255, np.nan, 2.0 ** (s - 127))


def rows(pool, scales, pages, h, n):
    """The first n cached rows of one head over a list of pages, fp64 [n][D];
    a page id of None gives rows of NaN (to be left out)."""
    ps, D = pool.shape[2:]
    got = np.full((len(pages) * ps, D), np.nan)
    for i, p in enumerate(pages):
        if p is None:
            continue
        if scales is None:
            got[i * ps:(i + 1) * ps] = bf16(pool[p, h])
        else:
            got[i * ps:(i + 1) * ps] = E4M3[pool[p, h]] * scale_of(scales[p, h])[:, None]
    return got[:n]


def attention(q, k, v, seen, scale, softcap=0.0):
    """q [G][D], k and v [n][D] in fp64, seen bool [n].  Returns (out [G][D],
    lse [G], sum_j p_j |v_j| [G][D], max_j scale sum_i |q_i k_ij| [G], max |s|,
    p [G][seen])."""
    G, D = q.shape
    if not seen.any():
        return np.zeros((G, D)), np.full(G, -np.inf), np.zeros((G, D)), np.zeros(G), 0.0, np.zeros((G, 0))
    k, v = k[seen], v[seen]
    s = scale * (q @ k.T)
    if softcap:
        s = softcap * np.tanh(s / softcap)
    top = s.max(1, keepdims=True)
    w = np.exp(s - top)
    p = w / w.sum(1, keepdims=True)
    size = np.array([(np.abs(q[g]) * np.abs(k)).sum(1).max() for g in range(G)]) * abs(scale)
    return p @ v, top[:, 0] + np.log(w.sum(1)), p @ np.abs(v), size, float(np.abs(s).max()), p


class Pages:
    """The pages' bookkeeping with plain lists: the lowest free page and id first."""

    def __init__(self, pages, page_size, seqs, row):
        self.refs, self.ps, self.max, self.row = [0] * pages, page_size, seqs, row
        self.seqs = {}                      # id -> [length, page ids]

    def free_pages(self):
        return sum(r == 0 for r in self.refs)

    def _take(self):
        p = self.refs.index(0)
        self.refs[p] = 1
        return p

    def _id(self):
        return next((i for i in range(self.max) if i not in self.seqs), None)

    def open(self):
        i = self._id()
        if i is not None:
            self.seqs[i] = [0, []]
        return i

    def fork(self, parent):
        i = self._id()
        if i is not None:
            self.seqs[i] = [self.seqs[parent][0], list(self.seqs[parent][1])]
            for p in self.seqs[i][1]:
                self.refs[p] += 1
        return i

    def extend(self, i, n):
        """(src, dst) or None; raises MemoryError or ValueError with nothing changed."""
        length, ids = self.seqs[i]
        if n == 0:
            return None
        if length + n > self.row * self.ps:
            raise ValueError
        need = -(-(length + n) // self.ps)
        own = length % self.ps != 0 and self.refs[ids[-1]] > 1
        if need - len(ids) + own > self.free_pages():
            raise MemoryError
        copy = None
        if own:
            src = ids[-1]
            self.refs[src] -= 1
            ids[-1] = self._take()
            copy = (src, ids[-1])
        while len(ids) < need:
            ids.append(self._take())
        self.seqs[i][0] = length + n
        return copy

    def free(self, i):
        for p in self.seqs.pop(i)[1]:
            self.refs[p] -= 1

    def compact(self, most):
        used = len(self.refs) - self.free_pages()
        src = [p for p in range(used, len(self.refs)) if self.refs[p]][:most]
        dst = [p for p in range(used) if not self.refs[p]][:len(src)]
        for a, b in zip(src, dst):
            self.refs[b], self.refs[a] = self.refs[a], 0
        to = dict(zip(src, dst))
        for s in self.seqs.values():
            s[1] = [to.get(p, p) for p in s[1]]
        return list(zip(src, dst))
