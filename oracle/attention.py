"""What the calls around an 8-bit cache compute (norm and rotation of heads,
append, read, attention), token by token in 64 bits from the definitions in
include/qlin.h, and the cache's codes and scales in the 32-bit steps that are
defined there; test infrastructure only.
"""
from __future__ import annotations

import numpy as np

import oracle

FP8, INT8 = 0, 1
_E4M3 = []          # the value of each e4m3 code
QMAX = {FP8: np.float32(448.0), INT8: np.float32(127.0)}


def norm_rope(x, weight, eps, cos_sin, positions, rotary, interleaved):
    """x [T, heads, D] -> (y, size): size is what rounding errors are measured
    by, the absolute terms of y.  positions outside the table: y is NaN."""
    x = np.asarray(x, dtype=np.float64)
    T, H, D = x.shape
    y, size = np.full((T, H, D), np.nan), np.zeros((T, H, D))
    for t in range(T):
        if rotary and not 0 <= positions[t] < len(cos_sin):
            continue
        for h in range(H):
            v = x[t, h].copy()
            if weight is not None:
                v = v / np.sqrt(np.mean(v * v) + eps) * np.asarray(weight, dtype=np.float64)
            out, s = v.copy(), np.abs(v)
            for i in range(rotary // 2):
                a, b = (2 * i, 2 * i + 1) if interleaved else (i, rotary // 2 + i)
                cos, sin = float(cos_sin[positions[t], i]), float(cos_sin[positions[t], rotary // 2 + i])
                out[a], out[b] = v[a] * cos - v[b] * sin, v[b] * cos + v[a] * sin
                s[a], s[b] = abs(v[a] * cos) + abs(v[b] * sin), abs(v[b] * cos) + abs(v[a] * sin)
            y[t, h], size[t, h] = out, s
    return y, size


# ---------------------------------------------------------------------- cache

def key_byte(t, d, D):
    return 16 * D * (t // 16) + 1024 * (d // 64) + 256 * (d % 64 // 16) + 16 * (t % 16) + d % 16


def value_byte(t, d, D):
    return 16 * D * (t // 16) + 1024 * (d // 64) + 256 * (t % 16 // 4) + 16 * (d % 16) + 4 * (d % 64 // 16) + t % 4


def byte_index(page, D, values):
    """[page, D]: where (token, channel) lies among a page and head's codes."""
    t, d = np.arange(page)[:, None], np.arange(D)[None, :]
    return value_byte(t, d, D) if values else key_byte(t, d, D)


def decode(fmt, codes):
    codes = np.asarray(codes, dtype=np.uint8)
    if fmt == INT8:
        return codes.view(np.int8).astype(np.float64)
    if not _E4M3:
        _E4M3.append(oracle.e4m3_decode(np.arange(256, dtype=np.uint8)))
    return _E4M3[0][codes]


def encode(fmt, x, scale):
    """fp32 values -> codes under an fp32 scale: fp32 quotients, nearest even."""
    x, scale = np.asarray(x, dtype=np.float32), np.float32(scale)
    if scale == 0:
        return np.zeros(x.shape, dtype=np.uint8)
    t = (x / scale).astype(np.float32)
    if fmt == INT8:
        return np.clip(np.rint(t), -127, 127).astype(np.int8).view(np.uint8)
    return np.asarray(oracle.e4m3_encode(np.clip(t, -448, 448)), dtype=np.uint8).reshape(x.shape)


class Cache:
    """A pool of pages: codes uint8 [pages, heads, page * D] and scales fp32
    [pages, heads], of keys (0) and of values (1)."""

    def __init__(self, fmt, heads, D, page, pages, fill=0x7F):
        self.fmt, self.heads, self.D, self.page, self.pages = fmt, heads, D, page, pages
        self.codes = [np.full((pages, heads, page * D), fill, dtype=np.uint8) for _ in range(2)]
        self.scales = [np.full((pages, heads), np.nan, dtype=np.float32) for _ in range(2)]
        self.index = [byte_index(page, D, False), byte_index(page, D, True)]

    def page_of(self, table, s, position):
        """The pool's page of a sequence's position, or -1."""
        if not 0 <= position < 1 << 30 or position // self.page >= table.shape[1]:
            return -1
        p = int(table[s, position // self.page])
        return p if 0 <= p < self.pages else -1

    def append(self, offsets, lengths, table, k, v):
        """k, v [T, heads, D] in fp32."""
        for kv, x in enumerate((k, v)):
            x = np.asarray(x, dtype=np.float32)
            for s in range(len(lengths)):
                start = int(lengths[s]) - (int(offsets[s + 1]) - int(offsets[s]))
                by_page = {}
                for t in range(int(offsets[s]), int(offsets[s + 1])):
                    at = start + t - int(offsets[s])
                    if self.page_of(table, s, at) >= 0:
                        by_page.setdefault(at // self.page, []).append((at % self.page, t))
                for which, tokens in by_page.items():
                    p, had = self.page_of(table, s, which * self.page), tokens[0][0]
                    for h in range(self.heads):
                        was = self.scales[kv][p, h] if had else np.float32(0)
                        rows = x[[t for _, t in tokens], h]
                        now = max(was, np.float32(np.abs(rows).max()) / QMAX[self.fmt])
                        codes = self.codes[kv][p, h]
                        if had and now > was:
                            old = self.index[kv][:had]
                            again = (decode(self.fmt, codes[old]).astype(np.float32) * was).astype(np.float32)
                            codes[old] = encode(self.fmt, again, now)
                        for (at, _), row in zip(tokens, rows):
                            codes[self.index[kv][at]] = encode(self.fmt, row, now)
                        self.scales[kv][p, h] = now

    def token(self, kv, table, s, position):
        """[heads, D] in fp32 (code x scale, rounded once), or None."""
        p = self.page_of(table, s, position)
        if p < 0:
            return None
        codes = self.codes[kv][p][:, self.index[kv][position % self.page]]
        return (decode(self.fmt, codes).astype(np.float32) * self.scales[kv][p][:, None]).astype(np.float32)

    def exact(self, kv, table, s, positions):
        """[n, heads, D] in 64 bits: code x scale."""
        out = np.empty((len(positions), self.heads, self.D))
        for i, at in enumerate(positions):
            p = self.page_of(table, s, at)
            codes = self.codes[kv][p][:, self.index[kv][at % self.page]]
            out[i] = decode(self.fmt, codes) * self.scales[kv][p][:, None].astype(np.float64)
        return out


def attention(cache, offsets, lengths, table, q, scale, causal=True, window=0):
    """q [T, q_heads, D] -> (y, W, E, F).  W = sum p |v| / sum p.  E: by how much y
    is off when log2 p_j is off by u ((D + 8) A_j + 2 |x_j - max x|), for u = 1,
    A_j being the absolute terms of x_j = log2(e) scale q . k_j.  F = sum |v| /
    sum p, with p = 1 for the largest."""
    q = np.asarray(q, dtype=np.float64)
    T, Hq, D = q.shape
    G = Hq // cache.heads
    y, W, E, F = np.full((T, Hq, D), np.nan), *np.zeros((3, T, Hq, D))
    to_log2 = scale / np.log(2.0)
    for s in range(len(lengths)):
        first, n = int(offsets[s]), int(offsets[s + 1]) - int(offsets[s])
        if n <= 0:
            continue
        length = max(int(lengths[s]), 0)
        start = length - n
        held = [at for at in range(min(length, table.shape[1] * cache.page)) if cache.page_of(table, s, at) >= 0]
        low = max(0, start - window + 1) if window else 0
        held = np.array([at for at in held if at >= low], dtype=np.int64)
        k, v = cache.exact(0, table, s, held), cache.exact(1, table, s, held)
        for i in range(n):
            seen = np.ones(len(held), bool)
            if causal:
                seen &= held <= start + i
            if window:
                seen &= held > start + i - window
            for h in range(Hq):
                if not seen.any():
                    y[first + i, h] = 0.0
                    continue
                ks, vs, one = k[seen, h // G], v[seen, h // G], q[first + i, h]
                x = ks @ one * to_log2
                A = np.abs(ks) @ np.abs(one) * abs(to_log2)
                p = np.exp2(x - x.max())
                off = p * np.log(2.0) * ((D + 8) * A + 2 * np.abs(x - x.max()))
                F[first + i, h] = np.abs(vs).sum(0) / p.sum()
                p, off = p / p.sum(), off / p.sum()
                y[first + i, h] = p @ vs
                W[first + i, h] = p @ np.abs(vs)
                E[first + i, h] = off @ np.abs(vs) + off.sum() * np.abs(y[first + i, h])
    return y, W, E, F
