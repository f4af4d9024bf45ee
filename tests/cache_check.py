"""A tight check of attention over the packed cache: every output number and every lse within what the roundings
that the kernels are allowed leave, computed from the terms that are really there.  The kernels multiply values that are
rounded to fp16 (as the header says), so the comparison is with the softmax over values rounded so, in float64.

Roundings counted (u = 2^-23, one fp32 step):
  * a matrix product of 16 terms and an accumulator aligns them to the largest and cuts each off there: 17 u / 2 of the
    largest of terms and running sum.
  * scores, few rows: per group of 32, acc = sum (64 + c) q in two products, then s acc into a running sum (one fma of
    u / 2 each), in front of which stand the (s, b) pairs times (-72 sum q, sum q), the sums in 22 bits (2 u);
  * scores, many rows: 16 numbers s (c - 8) q at a time into a running sum that begins with the b sum q.  The larger of
    the two is allowed;
  * the query in fp16, its largest entry in [1, 2): half a step of fp16's subnormals, 2^-25, where a power of two
    does not bring it there exactly;
  * a score's factor scale log2 e (2 u), its product and difference (u each), 2^x (2 u): 4 u of the scores' sizes, 2 u;
  * a weight in fp16 for bf16 rows: 2^-11 of it; in two fp16 parts for fp16 rows: 2^-22; for both half of the
    smallest step, 2^-25, with the row's largest weight at 2^7 or above: 2^-32 of the largest (1 % more, as the
    reference is a rounded number);
  * sums of n weights: rounded to nearest, n / 4 additions a lane at most: min(n / 4, 8 sqrt(n / 4)) u / 2, and 40 u / 2 for
    the joins;
  * the values' products: one for 16 tokens (two for fp16 rows), each cutting at the largest of running sum and terms;
    the running sum is at most sum p |v|: 17 u / 2 (n / 8 + 16) of it, but n / 8 no more than the tokens that weigh
    2^-24 or more of the row's largest;
  * the result: half a step of its type.
"""
from __future__ import annotations

import numpy as np

from oracle import cache as oc

U = 2.0 ** -23
CUT = 17 * U / 2
STEP = {"fp16": 2.0 ** -11, "bf16": 2.0 ** -8}          # half a step, relative


def unpack(pool: oc.Pool, table_row, h: int, first: int, end: int):
    """(codes, s, b) of keys and of values at positions first .. end - 1, and which are in the pool."""
    pos = np.arange(first, end)
    page = np.asarray(table_row, np.int64)[pos // pool.page_tokens]
    ok = (page >= 0) & (page < pool.n_pages)
    page = np.where(ok, page, 0)
    base = ((page * pool.heads + h) * (pool.page_tokens // 16) + pos % pool.page_tokens // 16) * oc.chunk_bytes(pool.dim)
    t, out = pos % 16, []
    for code, shift, pair in oc._chunk_maps(pool.dim):
        c = pool.data[base[:, None] + code[t]].astype(np.int64) >> shift[t] & 15
        at = base[:, None] + pair[t]
        sb = np.stack([pool.data[at + i] for i in range(4)], -1).copy().view("<f2").astype(np.float64)
        out.append((c, sb[..., 0], sb[..., 1]))
    return out[0], out[1], ok


def numbers(c, s, b):
    return np.repeat(b, 32, -1) + np.repeat(s, 32, -1) * (c - 8)


def expected(q, pos, keys, values, ok, first, window, scale, dtype):
    """For the query rows q (n, D) at positions pos of one sequence and head: (out, lse, allowed errors of both, the largest
    error of a score that matters).  Rows that see nothing: zeros, -inf, 0, 0."""
    q = np.asarray(q, np.float64)
    n, dim = q.shape
    (c, s, b), v = keys, numbers(*values).astype(np.float16).astype(np.float64)
    t = np.arange(first, first + len(c))
    see = ok & (t <= pos[:, None])
    if window:
        see &= t > pos[:, None] - window
    c, s, b, v = (np.where(ok.reshape(-1, *[1] * (a.ndim - 1)), a, 0) for a in (c, s, b, v))
    seen = see.any(0)                                      # what no row sees may hold anything
    c, s, b, v = (np.where(seen.reshape(-1, *[1] * (a.ndim - 1)), a, 0) for a in (c, s, b, v))
    k = numbers(c, s, b)
    x = np.where(see, scale * (q @ k.T), -np.inf)
    some = see.any(1)
    m = np.where(some, np.max(x, 1, initial=-np.inf), 0.0)
    p = np.exp(x - m[:, None])
    z = np.where(some, p.sum(1), 1.0)
    out, A = p @ v / z[:, None], p @ np.abs(v) / z[:, None]
    lse = np.where(some, m + np.log(z), -np.inf)
    # errors of scores
    g = dim // 32
    qg, sums = q.reshape(n, g, 32), q.reshape(n, g, 32).sum(-1)
    acc = np.abs(np.einsum("ngd,tgd->ngt", qg, c.reshape(-1, g, 32) + 64.0))
    top = 79 * np.abs(qg).max(-1)
    pairs = np.abs(sums) @ (72 * s + np.abs(b)).T           # (n, t)
    running = np.einsum("ngt,tg->nt", acc, s) + pairs
    few = 2 * CUT * np.einsum("ngt,tg->nt", np.maximum(acc, top[..., None]), s) + U / 2 * g * running + (2 * U + 2 * CUT) * pairs
    terms = np.repeat(s, 2, -1)[:, :, None] * (c.reshape(-1, dim // 16, 16) - 8)
    parts = np.einsum("nkd,tkd->nkt", q.reshape(n, -1, 16), terms)
    bsum = sums @ b.T
    largest = np.abs(q.reshape(n, -1, 16)).max(-1)[:, :, None] * 8 * np.repeat(s, 2, -1).T[None]
    many = CUT * (np.maximum(np.abs(np.cumsum(parts, 1) + bsum[:, None]), largest).sum(1) + (dim // 16 + 1) * (np.abs(sums) @ np.abs(b).T)) + \
        2 * U * (np.abs(sums) @ np.abs(b).T)
    with np.errstate(divide="ignore"):
        up = np.clip(127 - np.floor(np.log2(np.abs(q).max(1))), -126, 127)       # as large as a power of two may be
        up = np.where(np.abs(q).max(1) == 0, 0.0, np.minimum(up, -np.floor(np.log2(np.abs(q).max(1)))))
    rounded = 2.0 ** (-25 - up)[:, None] * np.abs(k).sum(1)
    size = np.where(see, np.abs(x), 0.0)
    e = abs(scale) * (np.maximum(few, many) + rounded) + 4 * U * (size + size.max(1, initial=0.0)[:, None]) + 2 * U
    e = np.where(see, e, 0.0)
    # of the result
    count = see.sum(1)
    adds = (np.minimum(count / 4, 8 * np.sqrt(count / 4)) + 40) * U / 2
    heavy = (p >= 2.0 ** -24).sum(1)
    weight = 2.0 ** -11 if dtype == "bf16" else 2.0 ** -22
    grow = p * np.expm1(e)
    away = grow @ np.abs(v) / z[:, None] + np.abs(out) * (grow.sum(1) / z)[:, None]
    few_v = np.where(see, 1.0, 0.0) @ np.abs(v)             # the weights' smallest step meets every value
    tol = away + (weight + adds[:, None] + CUT * (heavy / 8 + 16)[:, None]) * A + 2.0 ** -32 * 1.01 * few_v / z[:, None]
    tol = tol + STEP[dtype] * (np.abs(out) + tol) + 2.0 ** -25
    tol_lse = grow.sum(1) / z + adds + 4 * U * (np.where(some, np.abs(lse), 0.0) + size.max(1, initial=0.0) + 16)
    matters = np.where(p > 2.0 ** -20, e, 0.0).max(1, initial=0.0)
    return np.where(some[:, None], out, 0.0), lse, np.where(some[:, None], tol, 0.0), np.where(some, tol_lse, 0.0), matters


def check(pool, table, spans, q, out, lse, window, scale, dtype, sample=None, seed=1):
    """Asserts on out [rows, q_heads, D] and lse [rows, q_heads] (float64) of a step; spans as oracle.cache.spans gives them.
    Returns the largest share of a tolerance that was used."""
    group, used = q.shape[1] // pool.heads, 0.0
    gen = np.random.default_rng(seed)
    for i, (row0, rows, start, live, _) in enumerate(spans):
        if not live:
            assert (out[row0:row0 + rows] == 0).all() and (lse[row0:row0 + rows] == -np.inf).all(), i
            continue
        pick = np.arange(rows)
        if sample is not None and rows > sample:           # the last row always
            pick = np.sort(np.append(gen.choice(rows - 1, sample - 1, replace=False), rows - 1))
        first = max(0, start - window + 1) if window else 0
        for h in range(pool.heads):
            keys, values, ok = unpack(pool, table[i], h, first, start + rows)
            heads = slice(h * group, (h + 1) * group)
            flat = q[row0 + pick, heads].reshape(-1, pool.dim)
            want, wl, tol, tl, e = expected(flat, np.repeat(start + pick, group), keys, values, ok, first, window, scale, dtype)
            assert e.max(initial=0.0) < 0.05, "scores too inexact for this check to mean anything"
            got, gl = out[row0 + pick, heads].reshape(-1, pool.dim), lse[row0 + pick, heads].reshape(-1)
            blind = wl == -np.inf
            assert (got[blind] == 0).all() and (gl[blind] == -np.inf).all(), (i, h)
            got, gl, want, wl, tol, tl = (a[~blind] for a in (got, gl, want, wl, tol, tl))
            if not len(gl):
                continue
            a, bl = np.abs(got - want) / tol, np.abs(gl - wl) / tl
            assert (a <= 1).all() and (bl <= 1).all(), (i, h, "out, lse: %.3g, %.3g of the tolerance" % (np.max(a), np.max(bl)))
            used = max(used, a.max(), bl.max())
    return used


class Made:
    """A pool whose bytes are the oracle's own quantisation of random keys and values, and a step's queries over it.  What is
    not stored holds 0xff: NaN scales and bases."""

    def __init__(self, seqs, heads=2, group=4, dim=128, page=32, window=0, scale=None, size=1.5, dtype="fp16", seed=0, stored=None):
        gen = np.random.default_rng(seed)
        self.seqs, self.heads, self.group, self.dim, self.page, self.window, self.dtype = seqs, heads, group, dim, page, window, dtype
        self.scale = dim ** -0.5 if scale is None else scale
        need = [max(1, -(-(max(s, 0) + n) // page)) for s, n in seqs]
        order = gen.permutation(sum(need) + 2)
        self.table = np.zeros((len(seqs), max(need)), np.int32)
        at = 0
        for i, n in enumerate(need):
            self.table[i, :n] = order[at:at + n]
            at += n
        n_bytes = len(order) * oc.page_bytes(heads, dim, page)
        self.pool = oc.Pool(heads, dim, page, len(order), np.full(n_bytes, 0xff, np.uint8))
        for i, (s, n) in enumerate(seqs):
            if s >= 0 and n:
                self._store(gen, i, stored[i] if stored else 0, s + n)
        self.start = np.array([s for s, _ in seqs], np.int32)
        self.cu = np.concatenate([[0], np.cumsum([n for _, n in seqs])]).astype(np.int32)
        self.rows, self.max_new = int(self.cu[-1]), max(n for _, n in seqs)
        q = gen.standard_normal((self.rows, heads * group, dim)).astype(np.float32) * np.float32(size)
        # the type's own numbers
        self.q = (q.view(np.uint32) + 0x7fff + (q.view(np.uint32) >> 16 & 1) & 0xffff0000).view(np.float32) if dtype == "bf16" else \
            q.astype(np.float16).astype(np.float32)
        self.spans = oc.spans(len(seqs), self.rows, self.max_new, self.cu, self.start, self.table.shape[1], page)

    def _store(self, gen, i, first, end):
        pos = np.arange(first, end)
        x = gen.standard_normal((2, end - first, self.heads, self.dim)).astype(np.float32)
        x[..., ::13] *= 6                                   # some channels are large, as in trained models
        codes, s, b = oc.quantise(x)
        page = self.table[i, pos // self.page].astype(np.int64)
        t = pos % 16
        for value, (code, shift, pair) in enumerate(oc._chunk_maps(self.dim)):
            for h in range(self.heads):
                base = ((page * self.heads + h) * (self.page // 16) + pos % self.page // 16) * oc.chunk_bytes(self.dim)
                c = codes[value, :, h]
                at = base[:, None] + code[t]                # dims 2 i and 2 i + 1 share a byte
                self.pool.data[at[:, ::2]] = c[:, ::2] | c[:, 1::2] << 4
                sb = np.stack([s[value, :, h], b[value, :, h]], -1).astype("<f2").view(np.uint8).reshape(len(pos), -1, 4)
                for k in range(4):
                    self.pool.data[base[:, None] + pair[t] + k] = sb[..., k]

    def check(self, out, lse, **kw):
        return check(self.pool, self.table, self.spans, self.q, out, lse, self.window, self.scale, self.dtype, **kw)


# What the kernels are held to: each row count, head size, type and kind of mask, few rows a head and many.
CASES = {
    "tokens": dict(seqs=[(0, 1), (1, 1), (15, 1), (31, 1), (-1, 1), (64, 1), (257, 1), (700, 1)]),
    "tokens64": dict(seqs=[(0, 1), (63, 1), (300, 1)], dim=64, group=12, page=16),
    "tokens256": dict(seqs=[(0, 1), (63, 1), (300, 1)], dim=256, group=3, page=64),
    "window": dict(seqs=[(0, 3), (200, 5), (95, 2), (5, 0), (130, 7)], window=37),
    "draft": dict(seqs=[(500, 4), (30, 3)], group=8, dim=64, window=100),
    "chunk": dict(seqs=[(0, 40), (77, 61), (-1, 5), (300, 1)]),
    "chunk64": dict(seqs=[(0, 33), (150, 60)], dim=64, group=4),
    "chunk256": dict(seqs=[(0, 33), (150, 60)], dim=256, group=3),
    "chunk_window": dict(seqs=[(0, 40), (213, 61)], window=50),
    "peaked": dict(seqs=[(90, 1), (0, 1), (257, 2)], size=12.0),
    "peaked_chunk": dict(seqs=[(90, 40), (0, 30)], size=12.0),
    "negative": dict(seqs=[(99, 1), (0, 30)], scale=-0.11),
    "long": dict(seqs=[(2000, 1)], group=8),
}
