"""Plain 64-bit references of the serving operators (test infrastructure only):
low-rank adapters, the paged 8-bit key/value cache, attention over it.  NumPy
and Python, one element of the definition at a time where that is fast enough.
"""
from __future__ import annotations

import math

import numpy as np

LARGEST = {"e4m3": 448.0, "int8": 127.0}


def e4m3_values() -> np.ndarray:
    """The 256 values of OCP e4m3 codes (bias 7, no infinities, 0x7F and 0xFF NaN)."""
    c = np.arange(256)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e == 0, m / 8.0 * 2.0 ** -6, (1 + m / 8.0) * 2.0 ** (e - 7.0))
    v[(c & 127) == 127] = np.nan
    return np.where(c >= 128, -v, v)


_E4M3 = e4m3_values()


def values(codes: np.ndarray, kind: str) -> np.ndarray:
    return _E4M3[codes] if kind == "e4m3" else codes.view(np.int8).astype(np.float64)


def round_to_code(x: np.ndarray, kind: str) -> np.ndarray:
    """The nearest code of finite values within the type's range, ties to the even code."""
    x = np.asarray(x, np.float64)
    if kind == "int8":
        return np.clip(np.rint(x), -127, 127).astype(np.int8).view(np.uint8)
    grid = _E4M3[:127]
    a = np.minimum(np.abs(x), 448.0)
    hi = np.searchsorted(grid, a).clip(0, 126)
    lo = np.maximum(hi - 1, 0)
    up, down = grid[hi] - a, a - grid[lo]
    code = np.where((down < up) | ((down == up) & (lo % 2 == 0)), lo, hi)
    code = np.where(grid[hi] == a, hi, code)
    return np.where(np.signbit(x), code + 128, code).astype(np.uint8)


def scale_for(amax: float, kind: str) -> float:
    """The least 2^e, e >= -60, with amax <= Q 2^e."""
    e = -60
    while amax > LARGEST[kind] * 2.0 ** e:
        e += 1
    return 2.0 ** e


class Cache:
    """The cache with its pages, in plain Python: codes as numpy bytes, values
    of keys and values per (layer, page, head) in the buffers' own layout."""

    def __init__(self, layers, kv_heads, head_dim, n_pages, max_seqs, max_pages, page_tokens=64, dtype="e4m3"):
        wide = -(-head_dim // 64) * 64
        self.kind, self.page, self.dim, self.max_pages = dtype, page_tokens, head_dim, max_pages
        self.k = np.zeros((layers, n_pages, kv_heads, page_tokens, wide), np.uint8)
        self.v = np.zeros((layers, n_pages, kv_heads, wide, page_tokens), np.uint8)
        self.scale = np.zeros((layers, n_pages, kv_heads, 2), np.float32)
        self.refs = np.zeros(n_pages, np.int32)
        self.table = np.zeros((max_seqs, max_pages), np.int32)
        self.lens = np.zeros(max_seqs, np.int32)
        self.status = 0

    def pages(self, tokens):
        return -(-int(tokens) // self.page)

    def _free(self, n):
        free = np.flatnonzero(self.refs == 0)[:n]
        return None if len(free) < n else [int(p) for p in free]

    def extend(self, rows, counts):
        need = [self.pages(self.lens[r] + c) - self.pages(self.lens[r]) for r, c in zip(rows, counts)]
        if any(self.lens[r] + c > self.max_pages * self.page for r, c in zip(rows, counts)):
            self.status |= 2
            return
        got = self._free(sum(need))
        if got is None:
            self.status |= 1
            return
        for r, c, n in zip(rows, counts, need):
            at = self.pages(self.lens[r])
            for j in range(n):
                p = got.pop(0)
                self.table[r, at + j] = p
                self.refs[p] = 1
            self.lens[r] += c

    def fork(self, parents, children):
        if any(self.lens[c] != 0 for c in children):
            self.status |= 8
            return
        need = [int(self.lens[p] % self.page != 0) for p in parents]
        got = self._free(sum(need))
        if got is None:
            self.status |= 1
            return
        for p, c, n in zip(parents, children, need):
            whole = int(self.lens[p]) // self.page
            self.table[c, :whole] = self.table[p, :whole]
            for x in self.table[p, :whole]:
                self.refs[x] += 1
            if n:
                to, at = got.pop(0), self.table[p, whole]
                self.table[c, whole] = to
                self.refs[to] = 1
                for a in (self.k, self.v, self.scale):
                    a[:, to] = a[:, at]
            self.lens[c] = self.lens[p]

    def free(self, rows):
        for r in rows:
            for x in self.table[r, :self.pages(self.lens[r])]:
                self.refs[x] -= 1
            self.lens[r] = 0

    def compact(self):
        live = [int(p) for p in np.flatnonzero(self.refs > 0)]
        n = len(live)
        holes = [p for p in range(n) if self.refs[p] == 0]
        to = {p: p for p in live}
        to.update(zip([p for p in live if p >= n], holes))
        refs, table = np.zeros_like(self.refs), np.full_like(self.table, -1)
        for p in live:
            refs[to[p]] = self.refs[p]
            if to[p] != p:
                for a in (self.k, self.v, self.scale):
                    a[:, to[p]] = a[:, p]
        for r in range(len(self.lens)):
            for j in range(self.pages(self.lens[r])):
                table[r, j] = to[int(self.table[r, j])]
        self.refs, self.table = refs, table

    def append(self, layer, k, v, rows, starts=None):
        """k, v: (tokens, heads, dim) float64 values of the inputs."""
        starts = list(range(len(rows) + 1)) if starts is None else starts
        for i, r in enumerate(rows):
            n = starts[i + 1] - starts[i]
            begin = int(self.lens[r]) - n
            for j in range(begin // self.page, self.pages(self.lens[r])):
                lo, hi = max(begin, j * self.page), min(int(self.lens[r]), (j + 1) * self.page)
                if lo >= hi:
                    continue
                p, a, b = int(self.table[r, j]), lo - j * self.page, hi - j * self.page
                for side, x in ((0, k), (1, v)):
                    for h in range(x.shape[1]):
                        new = x[starts[i] + lo - begin:starts[i] + hi - begin, h]
                        fin = np.isfinite(new)
                        if not fin.all():
                            self.status |= 16
                        old = float(self.scale[layer, p, h, side]) if a else 0.0
                        s = max(old, scale_for(float(np.abs(new[fin]).max(initial=0.0)), self.kind))
                        top = LARGEST[self.kind]
                        q = np.where(np.isnan(new), 0.0, np.clip(np.nan_to_num(new, nan=0.0, posinf=np.inf, neginf=-np.inf) / s, -top, top))
                        code = np.zeros((b - a, self.k.shape[-1]), np.uint8)
                        code[:, :self.dim] = round_to_code(q, self.kind)
                        have = self.k[layer, p, h] if side == 0 else self.v[layer, p, h].T
                        if a and old < s:
                            have[:a] = round_to_code(values(have[:a], self.kind) * (old / s), self.kind)
                        have[a:b] = code
                        self.scale[layer, p, h, side] = s

    def tokens(self, layer, row, head, side):
        """The stored values of a row's tokens: (length, dim) float64."""
        n, out = int(self.lens[row]), []
        for j in range(self.pages(n)):
            p = int(self.table[row, j])
            c = self.k[layer, p, head] if side == 0 else self.v[layer, p, head].T
            out.append(values(np.ascontiguousarray(c), self.kind) * float(self.scale[layer, p, head, side]))
        return np.concatenate(out)[:n, :self.dim] if out else np.zeros((0, self.dim))

    def attend(self, layer, q, rows, starts=None, scale=0.0, window=0, sinks=0, softcap=0.0, gone=()):
        """(out, lse, slack, spread): for each query the result, the logarithm
        of the softmax sum, the most that fp32 sums can move a logit, and the
        probability-weighted magnitude of the values.  gone: (row, column)
        entries of the table whose tokens are left out."""
        starts = list(range(len(rows) + 1)) if starts is None else starts
        scale = scale or 1.0 / math.sqrt(self.dim)
        out, spread = np.zeros(q.shape), np.zeros(q.shape)
        lse, slack = np.full(q.shape[:2], -np.inf), np.zeros(q.shape[:2])
        group = q.shape[1] // self.k.shape[2]
        for i, r in enumerate(rows):
            count, n = starts[i + 1] - starts[i], int(self.lens[r])
            for h in range(self.k.shape[2]):
                k, v = self.tokens(layer, r, h, 0), self.tokens(layer, r, h, 1)
                for j in range(count):
                    at = n - count + j
                    t = np.arange(n)
                    seen = (t <= at) & ~np.isin(t // self.page, [c for x, c in gone if x == r])
                    if window:
                        seen &= (t > at - window) | (t < sinks)
                    if not seen.any():
                        continue
                    for m in range(h * group, (h + 1) * group):
                        x = q[starts[i] + j, m]
                        logit = k[seen] @ x * scale
                        loose = np.abs(k[seen]) @ np.abs(x) * abs(scale) * (self.dim + 8) * 2.0 ** -24 + np.abs(logit) * 2.0 ** -21
                        if softcap:
                            logit = softcap * np.tanh(logit / softcap)
                            # an error in proportion to the cap where that is small, else to the capped logit
                            loose = loose + (softcap * 2.0 ** -20 if softcap <= 256 else np.abs(logit) * 2.0 ** -19)
                        top = logit.max()
                        p = np.exp(logit - top)
                        total = p.sum()
                        lse[starts[i] + j, m] = top + math.log(total)
                        slack[starts[i] + j, m] = loose.max() + 2.0 ** -20
                        out[starts[i] + j, m] = p @ v[seen] / total
                        spread[starts[i] + j, m] = p @ np.abs(v[seen]) / total
        return out, lse, slack, spread


def attend_bound(out, slack, spread):
    """How far a result may be: BF16 probabilities (8 significant bits, so rounded
    by at most 2^-8 of each term), logits
    moved by `slack` (twice: the term's and the sum's), the result's own
    rounding (2^-8)."""
    return (2.0 ** -8 * 1.01 + 2.02 * slack[..., None]) * spread + 2.0 ** -8 * 1.01 * np.abs(out) + 1e-30


def lora(y, x, of, adapters):
    """y + s B (A x) per token, and the bound of fp32 arithmetic: sums of cols
    and of 3 rank + 8 exact products, each addition rounded once, and a
    rounding when shares and factors are applied."""
    out, loose = np.array(y, np.float64), np.abs(y) * 2.0 ** -22
    for t, a in enumerate(of):
        if a < 0:
            continue
        A, B, s = adapters[a]
        inner, mag = A @ x[t], np.abs(A) @ np.abs(x[t])
        out[t] += s * (B @ inner)
        rounds = x.shape[1] + 64 + 3 * 128 + 16
        loose[t] += rounds * 2.0 ** -24 * abs(s) * (np.abs(B) @ mag)
    return out, 2 * loose
