"""Oracle of the packed key/value cache, float64 NumPy: the definitions stated in
include/bitstack.h ("packed key/value cache"), one number at a time where speed allows.

The cache has no counterpart on the pages (they compress weights); it is the other
occupant of the variable memory they are about, so its format is this project's own.
"""
from __future__ import annotations

import numpy as np

CHUNK = 16        # tokens of a chunk
CLAMP = 65000.0   # largest stored size


def chunk_bytes(dim: int) -> int:
    return 20 * dim


def page_bytes(heads: int, dim: int, page_tokens: int) -> int:
    return heads * (page_tokens // CHUNK) * chunk_bytes(dim)


def code_place(dim: int, value: bool, t: int, d: int) -> tuple[int, int]:
    """(byte inside the chunk, shift) of the code of token t (0..15), dim d."""
    w = d // 8
    row = t // 2 + 8 * (t % 2) if value else t
    place = (w % 8) * (dim // 64) + w // 8 if value else (w % 4) * (dim // 32) + w // 4
    return (10 * dim if value else 0) + row * (dim // 2) + 4 * place + (d % 8) // 2, 4 * (d % 2)


def pair_place(dim: int, value: bool, t: int, g: int) -> int:
    """First byte inside the chunk of the (s, b) pair of token t, group g."""
    row = t // 2 + 8 * (t % 2) if value else t
    place = (g % 2) * (dim // 64) + g // 2 if value else g
    return (18 * dim if value else 8 * dim) + row * (dim // 8) + 4 * place


_maps: dict = {}


def _chunk_maps(dim: int):
    """For keys and values: byte and shift of every (token, dim), byte of every (token, group)."""
    if dim not in _maps:
        out = []
        for value in (False, True):
            code = np.array([[code_place(dim, value, t, d) for d in range(dim)] for t in range(CHUNK)])
            pair = np.array([[pair_place(dim, value, t, g) for g in range(dim // 32)] for t in range(CHUNK)])
            out.append((code[..., 0], code[..., 1], pair))
        _maps[dim] = out
    return _maps[dim]


def quantise(x):
    """Numbers (..., D) -> codes (..., D) ints, s and b (..., D / 32) as fp16.  In fp32, as
    the definition says: the codes at a rounding border depend on it."""
    x = np.asarray(x, dtype=np.float32)
    x = np.where(np.isnan(x), np.float32(0), np.clip(x, np.float32(-CLAMP), np.float32(CLAMP)))
    g = x.reshape(*x.shape[:-1], -1, 32)
    lo, hi = g.min(-1), g.max(-1)
    step = ((hi - lo) / np.float32(15)).astype(np.float32)
    s, b = step.astype(np.float16), (lo + np.float32(8) * step).astype(np.float16)
    sf, bf = s.astype(np.float32)[..., None], b.astype(np.float32)[..., None]
    with np.errstate(divide="ignore", invalid="ignore"):
        c = np.rint((g - bf) / sf + np.float32(8))
    c = np.where(sf > 0, np.clip(c, 0, 15), 8).astype(np.int64)
    return c.reshape(x.shape), s, b


def dequantise(c, s, b):
    """float64 b + s (c - 8)."""
    g = c.reshape(*c.shape[:-1], -1, 32).astype(np.float64)
    return (b.astype(np.float64)[..., None] + s.astype(np.float64)[..., None] * (g - 8)).reshape(c.shape)


class Pool:
    """A pool's bytes and how they are addressed."""

    def __init__(self, heads: int, dim: int, page_tokens: int, n_pages: int, data=None):
        self.heads, self.dim, self.page_tokens, self.n_pages = heads, dim, page_tokens, n_pages
        n = n_pages * page_bytes(heads, dim, page_tokens)
        self.data = np.zeros(n, np.uint8) if data is None else np.asarray(data, np.uint8)[:n].copy()

    def chunk(self, page: int, pos: int, h: int) -> int:
        return ((page * self.heads + h) * (self.page_tokens // CHUNK) + pos % self.page_tokens // CHUNK) * chunk_bytes(self.dim)

    def in_pool(self, page: int) -> bool:
        return 0 <= page < self.n_pages

    def store(self, page: int, pos: int, h: int, value: bool, x) -> None:
        code, shift, pair = _chunk_maps(self.dim)[int(value)]
        base, t = self.chunk(page, pos, h), pos % CHUNK
        c, s, b = quantise(x)
        at = base + code[t]
        even = shift[t] == 0
        self.data[at[even]] = c[even] | c[~even] << 4     # dims 2 i and 2 i + 1 share a byte
        for g in range(self.dim // 32):
            self.data[base + pair[t, g]:base + pair[t, g] + 4] = np.array([s[g], b[g]], "<f2").view(np.uint8)

    def load(self, page: int, pos: int, h: int, value: bool):
        code, shift, pair = _chunk_maps(self.dim)[int(value)]
        base, t = self.chunk(page, pos, h), pos % CHUNK
        c = self.data[base + code[t]].astype(np.int64) >> shift[t] & 15
        sb = np.stack([self.data[base + pair[t] + i] for i in range(4)], -1).copy().view("<f2")
        return dequantise(c, sb[:, 0], sb[:, 1])


def spans(n_seqs, n_tokens, max_new, cu, start, table_width, page_tokens):
    """(first row, rows, start, live, bad) of every sequence after the step's checks."""
    out = []
    for i in range(n_seqs):
        lo, hi = (int(cu[i]), int(cu[i + 1])) if cu is not None else (i, i + 1)
        bad = lo < 0 or hi < lo or hi > n_tokens
        if bad:                       # the rows inside the dense tensors, as an empty slot's
            lo, hi = max(lo, 0), min(hi, n_tokens)
        rows = max(hi - lo, 0)
        live = not bad and start[i] >= 0 and rows > 0
        if live and (rows > max_new or int(start[i]) + rows > min(table_width * page_tokens, 2 ** 31 - 512)):
            live, bad = False, True
        out.append((lo, rows, int(start[i]), live, bad))
    return out


def context(pool: Pool, table_row, h: int, end: int):
    """Keys, values (end, D) float64 and which positions are in the pool."""
    k, v = np.zeros((end, pool.dim)), np.zeros((end, pool.dim))
    ok = np.zeros(end, bool)
    for pos in range(end):
        page = int(table_row[pos // pool.page_tokens])
        if pool.in_pool(page):
            ok[pos] = True
            k[pos], v[pos] = pool.load(page, pos, h, False), pool.load(page, pos, h, True)
    return k, v, ok


def attend(q, k, v, seen, scale: float):
    """One query row: (output, lse, sum of p |v| / sum of p); zeros and -inf where nothing is seen."""
    if not seen.any():
        return np.zeros(v.shape[1]), -np.inf, np.zeros(v.shape[1])
    x = scale * (k[seen] @ q)
    m = x.max()
    p = np.exp(x - m)
    z = p.sum()
    return p @ v[seen] / z, m + np.log(z), p @ np.abs(v[seen]) / z
