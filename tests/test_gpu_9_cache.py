"""GPU: the packed key/value cache against its float64 oracle: quantised writes bit for bit,
reads, and attention with tolerances derived from the roundings the header names."""
import math

import numpy as np
import pytest
import torch

import residual_block_decomp_b200 as R
from oracle import cache as oc

pytestmark = pytest.mark.gpu

HALF = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}   # half a step, relative


class Case:
    """A pool, a page table with scattered pages, and a step over sequences of given (start, new)."""

    def __init__(self, seqs, heads=2, dim=128, page=32, seed=0, cu=True, pages_more=3, garbage=True, spare_rows=0):
        self.seqs, self.heads, self.dim, self.page = seqs, heads, dim, page
        self.gen = np.random.default_rng(seed)
        need = [max(1, -(-(max(s, 0) + n) // page)) for s, n in seqs]
        self.n_pages = sum(need) + pages_more
        order = self.gen.permutation(self.n_pages)[:sum(need)]
        self.table = np.full((len(seqs), max(need) + 1), 0, np.int32)
        at = 0
        for i, n in enumerate(need):
            self.table[i, :n] = order[at:at + n]
            at += n
        self.total = sum(n for _, n in seqs)
        self.rows = self.total + spare_rows
        self.start = np.array([s for s, _ in seqs], np.int32)
        self.cu = np.concatenate([[0], np.cumsum([n for _, n in seqs])]).astype(np.int32) if cu else None
        nbytes = R.bs_cache_device_bytes(heads, dim, page, self.n_pages)
        # what was never written holds anything: NaN pairs and all-ones codes
        self.store = torch.full((nbytes,), 0xff if garbage else 0, dtype=torch.uint8, device="cuda")
        self.handle = R.bs_cache_create(heads, dim, page, self.n_pages, self.store)
        self.max_new = max(n for _, n in seqs)
        self.step = self.make_step()

    def make_step(self, max_new=None):
        dev = lambda a: None if a is None else torch.from_numpy(a).cuda()  # noqa: E731
        return R.CacheStep(dev(self.start), dev(self.table), self.rows, self.max_new if max_new is None else max_new,
                           dev(self.cu))

    def pool(self):
        return oc.Pool(self.heads, self.dim, self.page, self.n_pages, self.store.cpu().numpy())

    def numbers(self, rows, heads, dtype, scale=1.0):
        x = torch.from_numpy(self.gen.standard_normal((rows, heads, self.dim)).astype(np.float32) * scale)
        return x.to(dtype).cuda()

    def fill(self, dtype=torch.float16, upto=None):
        """Writes every sequence's positions 0 .. start + new - 1, through the library."""
        lens = [max(s, 0) + n for s, n in self.seqs] if upto is None else upto
        total = sum(lens)
        start = torch.zeros(len(lens), dtype=torch.int32, device="cuda")
        cu = torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32, device="cuda")
        step = R.CacheStep(start, torch.from_numpy(self.table).cuda(), total, max(lens), cu)
        k, v = self.numbers(total, self.heads, dtype), self.numbers(total, self.heads, dtype)
        k[:, :, ::13] *= 6
        R.bs_cache_append(self.handle, step, k, v)
        return k, v

    def attend(self, q, window=0, scale=None, step=None, ws=None, stream=None, lse=True):
        st = step or self.step
        out = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda")
        ls = torch.full(q.shape[:2], 7.0, device="cuda") if lse else None
        if ws is None:
            ws = torch.zeros(R.bs_cache_attention_workspace_bytes(self.handle, st, q.shape[1]), dtype=torch.uint8,
                             device="cuda")
        R.bs_cache_attention(self.handle, st, q, out, ws, scale, window, ls, stream)
        torch.cuda.synchronize()
        assert not ws[:148 * 4].any(), "counters are left at zero"
        return out, ls

    def close(self):
        R.bs_cache_destroy(self.handle)


def check_attention(case, q, out, lse, window=0, scale=None, sample=None):
    """Every row (or `sample` of them) against the oracle on the pool's own bytes.

    Tolerance of an output number: A = sum p |v| / sum p carries the fp16 rounding of each weight and
    of each value (2^-11 relative each, 2^-25 absolute below fp16's normal range), and twice the relative
    error of the weights, e; then half a step of the output's type.  e bounds the error of a score: a group's
    product adds 34 terms of at most (64 + 15) |q| s, its correction one of (72 s + |b|) |q|, with 40 fp32
    roundings of at most 2^-23 between them (products and additions of the matrix unit are allowed a whole
    step), the query's fp16 form is off by 2^-25 of its largest entry, the exponential by 2^-21."""
    scale = case.dim ** -0.5 if scale is None else scale
    pool = case.pool()
    qh, o = q.double().cpu().numpy(), out.double().cpu().numpy()
    ls = lse.double().cpu().numpy()
    heads, group = case.heads, q.shape[1] // case.heads
    spans = oc.spans(len(case.seqs), q.shape[0], case.step.max_new, case.cu, case.start, case.table.shape[1], case.page)
    gen = np.random.default_rng(1)
    seen_rows = np.zeros(q.shape[0], bool)
    for i, (row0, rows, start, live, _) in enumerate(spans):
        seen_rows[row0:row0 + rows] = True
        if not live:
            assert (o[row0:row0 + rows] == 0).all() and (ls[row0:row0 + rows] == -np.inf).all()
            continue
        for h in range(heads):
            k, v, ok = oc.context(pool, case.table[i], h, start + rows)
            pick = range(rows) if sample is None or rows <= sample else gen.choice(rows, sample, replace=False)
            for r in pick:
                pos = start + r
                t = np.arange(start + rows)
                vis = ok & (t <= pos)
                if window:
                    vis &= t > pos - window
                for g in range(group):
                    qr = qh[row0 + r, h * group + g]
                    want, wl, A = oc.attend(qr, k, v, vis, scale)
                    got = o[row0 + r, h * group + g]
                    if not vis.any():
                        assert (got == 0).all() and ls[row0 + r, h * group + g] == -np.inf
                        continue
                    qa = np.abs(qr).sum()
                    size = np.abs(k[vis]).max() * 80   # (79 s + |b|) of a group is below 80 times its largest number
                    e = abs(scale) * qa * (size * 40 * 2.0 ** -23 + np.abs(k[vis]).max() * case.dim * 2.0 ** -25) + 2.0 ** -21
                    vmax = np.abs(v[vis]).max()
                    tol = (2.0 ** -10 * 1.01 + 2 * e) * A + vis.sum() * 2.0 ** -25 * vmax + 2.0 ** -25
                    tol = tol + HALF[out.dtype] * (np.abs(want) + tol) + 2.0 ** -25
                    err = np.abs(got - want)
                    assert (err <= tol).all(), (i, h, r, g, float((err / tol).max()))
                    assert abs(ls[row0 + r, h * group + g] - wl) <= e + (vis.sum() ** 0.5 + 64) * 2.0 ** -23 + 2.0 ** -22 * abs(wl), (i, h, r, g)
    assert (o[~seen_rows] == 7).all() and (ls[~seen_rows] == 7).all(), "rows behind the last sequence"


# ------------------------------------------------------------------ append, read ---
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16, torch.float32])
def test_append_writes_the_defined_bytes(dim, dtype):
    c = Case([(0, 5), (13, 1), (30, 40), (7, 0), (16, 16)], heads=3, dim=dim, page=16, seed=dim)
    joined = c.numbers(c.rows, 2 * c.heads + 1, dtype)
    joined[:, ::2, 3::29] *= 30
    joined[2, 1, 5] = float("nan")
    joined[3, 2, 40] = float("inf")
    joined[4, 4, 1] = -float("inf")
    joined[6, :, :32] = 0.25
    k, v = joined[:, :c.heads], joined[:, c.heads + 1:]     # slices: strides that are not the dense ones
    want = c.pool()
    R.bs_cache_append(c.handle, c.step, k, v)
    torch.cuda.synchronize()
    kf, vf = k.float().cpu().numpy(), v.float().cpu().numpy()
    for i, (start, n) in enumerate(c.seqs):
        for r in range(n):
            for h in range(c.heads):
                page = int(c.table[i, (start + r) // c.page])
                want.store(page, start + r, h, False, kf[c.cu[i] + r, h])
                want.store(page, start + r, h, True, vf[c.cu[i] + r, h])
    assert np.array_equal(c.pool().data, want.data)          # other tokens' bytes are as they were, too
    assert R.bs_cache_get_device_error(c.handle) == R.BS_OK
    c.close()


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16, torch.float32])
def test_read_gives_the_stored_numbers(page, dtype):
    c = Case([(0, 300), (5, 1), (250, 30)], heads=2, dim=128, page=page, seed=page, spare_rows=2)
    c.fill()
    k = torch.full((c.rows, 2, 128), 7.0, dtype=dtype, device="cuda")
    v = torch.full_like(k, 7.0)
    R.bs_cache_read(c.handle, c.step, k, v)
    k2 = torch.full_like(k, 7.0)
    R.bs_cache_read(c.handle, c.step, k2, None)
    torch.cuda.synchronize()
    assert torch.equal(k, k2)
    assert (k[c.total:] == 7).all() and (v[c.total:] == 7).all()
    pool = c.pool()
    for i, (start, n) in enumerate(c.seqs):
        for r in range(n):
            for h in range(2):
                page_id = int(c.table[i, (start + r) // c.page])
                for got, value in ((k, False), (v, True)):
                    want = torch.from_numpy(pool.load(page_id, start + r, h, value)).float().to(dtype)
                    assert torch.equal(got[c.cu[i] + r, h].cpu(), want)
    c.close()


def test_large_appends_use_the_unrolled_kernels():
    """A step of more than 148 x 8 x 1024 words: every number against the torch form of the definition."""
    c = Case([(3, 9001), (0, 2000)], heads=8, dim=128, page=64, seed=3)
    k, v = c.numbers(c.rows, 8, torch.bfloat16), c.numbers(c.rows, 8, torch.bfloat16)
    R.bs_cache_append(c.handle, c.step, k, v)
    ko, vo = torch.empty(c.rows, 8, 128, device="cuda"), torch.empty(c.rows, 8, 128, device="cuda")
    R.bs_cache_read(c.handle, c.step, ko, vo)
    for x, got in ((k, ko), (v, vo)):
        want = oc.dequantise(*oc.quantise(x.float().cpu().numpy()))
        # one rounding to fp32
        assert (np.abs(got.cpu().numpy() - want) <= 2.0 ** -24 * np.abs(want) + 1e-30).all()
    c.close()


# -------------------------------------------------------------------- attention ----
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("group", [1, 3, 4, 8, 12])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_single_tokens_over_ragged_contexts(dim, group, dtype):
    seqs = [(0, 1), (1, 1), (15, 1), (16, 1), (31, 1), (-1, 1), (63, 1), (64, 1), (100, 1), (257, 1), (-5, 1), (700, 1)]
    c = Case(seqs, heads=2, dim=dim, page=32, seed=group, cu=False, spare_rows=2)
    c.fill(dtype)
    q = c.numbers(c.rows, 2 * group, dtype, 1.5)
    out, lse = c.attend(q)
    check_attention(c, q, out, lse)
    assert R.bs_cache_get_device_error(c.handle) == R.BS_OK
    c.close()


@pytest.mark.parametrize("page", [16, 64, 256])
@pytest.mark.parametrize("window", [0, 1, 2, 17, 100, 5000])
def test_windows_and_several_new_tokens(page, window):
    seqs = [(0, 3), (200, 5), (31, 1), (95, 2), (0, 1), (5, 0), (130, 7)]
    c = Case(seqs, heads=2, dim=128, page=page, seed=window)
    c.fill(torch.bfloat16)
    q = c.numbers(c.rows, 6, torch.bfloat16)
    out, lse = c.attend(q, window, 0.2)
    check_attention(c, q, out, lse, window, 0.2)
    c.close()


@pytest.mark.parametrize("dim,group", [(64, 4), (128, 1), (128, 4), (256, 3)])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_chunks_of_a_prompt(dim, group, dtype):
    """Up to 520 query rows a head: several row tiles, the last one ragged, contexts split between CTAs."""
    seqs = [(0, 130), (77, 61), (300, 1), (-1, 5), (0, 0), (513, 40)]
    c = Case(seqs, heads=2, dim=dim, page=32, seed=dim, spare_rows=3)
    c.fill()
    q = c.numbers(c.rows, 2 * group, dtype)
    out, lse = c.attend(q)
    check_attention(c, q, out, lse, sample=20)
    again, lse2 = c.attend(q)
    assert torch.equal(out, again) and torch.equal(lse, lse2)
    assert R.bs_cache_get_device_error(c.handle) == R.BS_OK
    c.close()


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("window", [1, 20, 100, 1000])
def test_chunks_under_a_window(dim, window):
    seqs = [(0, 70), (300, 90), (1500, 33)]
    c = Case(seqs, heads=1, dim=dim, page=16, seed=window)
    c.fill(torch.bfloat16)
    q = c.numbers(c.rows, 4, torch.bfloat16)
    out, lse = c.attend(q, window, -0.07)
    check_attention(c, q, out, lse, window, -0.07, sample=16)
    c.close()


@pytest.mark.parametrize("dim,rows", [(64, 40), (128, 24), (128, 25), (256, 17)])
def test_borders_of_the_row_counts(dim, rows):
    """Rows of a head around the choice of the kernel, with many sequences and with one."""
    for n in (1, 40):
        c = Case([(50 * i, rows) for i in range(n)] if n > 1 else [(700, rows)], heads=2, dim=dim, page=64, seed=rows)
        c.fill()
        q = c.numbers(c.rows, 8, torch.float16)
        out, lse = c.attend(q)
        check_attention(c, q, out, lse, sample=1 if n > 1 else 6)
        c.close()


def test_many_rows_over_one_long_context():
    """One item's tiles on all SMs: parts of 128 rows joined, few of the rows there."""
    c = Case([(9000, 60)], heads=1, dim=128, page=64, seed=3)
    c.fill()
    q = c.numbers(60, 2, torch.float16, 1.5)
    out, lse = c.attend(q)
    check_attention(c, q, out, lse, sample=5)
    c.close()


def test_many_rows_with_bad_pages_nan_and_peaked_scores():
    c = Case([(200, 60), (64, 40)], heads=2, dim=128, page=16, seed=31)
    c.fill()
    q = c.numbers(c.rows, 8, torch.bfloat16, 30.0)
    q[7, 3, 100] = float("nan")
    q[70, 0, 0] = float("inf")
    clean = q.clone()
    clean[7, 3, 100] = clean[70, 0, 0] = 1.0
    want, _ = c.attend(clean)
    out, lse = c.attend(q)
    bad = torch.zeros(c.rows, 8, dtype=torch.bool, device="cuda")
    bad[7, 3] = bad[70, 0] = True
    assert torch.equal(out[~bad], want[~bad]) and out[bad].isnan().all() and lse[bad].isnan().all()
    check_attention(c, clean, *c.attend(clean), sample=10)
    c.table[0, 3], c.table[0, 15], c.table[1, 0] = c.n_pages, -2, 1 << 20
    c.step = c.make_step()
    out, lse = c.attend(clean)
    assert R.bs_cache_get_device_error(c.handle) == R.BS_ERR_RANGE
    check_attention(c, clean, out, lse, sample=10)
    c.table[1] = -1
    c.step = c.make_step()
    out, lse = c.attend(clean)
    assert (out[60:] == 0).all() and (lse[60:] == -np.inf).all()
    assert R.bs_cache_get_device_error(c.handle) == R.BS_ERR_RANGE
    c.close()


def test_prompt_pieces_in_a_graph():
    """Append and attention of 64-token pieces captured once and replayed along a prompt."""
    c = Case([(0, 64), (0, 40)], heads=2, dim=64, page=32, seed=32, pages_more=40)
    own = list(range(c.n_pages))
    c.table = np.stack([own[:12], own[12:24]]).astype(np.int32)
    c.step = c.make_step()
    k, v, q = (c.numbers(c.rows, h, torch.float16) for h in (2, 2, 8))
    out, lse = torch.empty_like(q), torch.empty(c.rows, 8, device="cuda")
    ws = torch.zeros(R.bs_cache_attention_workspace_bytes(c.handle, c.step, 8), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        R.bs_cache_append(c.handle, c.step, k, v)
        R.bs_cache_attention(c.handle, c.step, q, out, ws, lse=lse)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        R.bs_cache_append(c.handle, c.step, k, v)
        R.bs_cache_attention(c.handle, c.step, q, out, ws, lse=lse)
    for _ in range(4):
        for x in (k, v, q):
            x.copy_(torch.from_numpy(c.gen.standard_normal(x.shape).astype(np.float32)))
        g.replay()
        torch.cuda.synchronize()
        check_attention(c, q, out, lse, sample=8)
        c.start = (c.start + [64, 40]).astype(np.int32)
        c.step.start.copy_(torch.from_numpy(c.start))
    c.close()


def test_one_long_context_over_all_sms_and_many_short_ones():
    c = Case([(20000, 1)], heads=1, dim=128, page=64, seed=1, cu=False)
    c.fill()
    q = c.numbers(1, 4, torch.float16, 2.0)
    out, lse = c.attend(q)
    check_attention(c, q, out, lse)
    again, _ = c.attend(q)
    assert torch.equal(out, again)
    c.close()
    gen = np.random.default_rng(8)
    c = Case([(int(n), 1) for n in gen.integers(0, 40, 700)], heads=1, dim=64, page=16, seed=2, cu=False)
    c.fill()
    q = c.numbers(700, 2, torch.bfloat16)
    out, lse = c.attend(q)
    check_attention(c, q, out, lse)
    c.close()


def test_peaked_scores_and_large_queries():
    """Scores of several hundred: one weight is 1 and the rest vanish; lengths of exponents beyond fp16's."""
    for dtype, size in ((torch.float16, 50.0), (torch.bfloat16, 3e5), (torch.bfloat16, 1e-30), (torch.bfloat16, 1e-39)):
        c = Case([(90, 1), (0, 1)], heads=1, dim=128, page=16, seed=4, cu=False)
        c.fill()
        q = c.numbers(2, 4, dtype, size)
        scale = None if size < 1 else 0.5 / size * 50
        out, lse = c.attend(q, 0, scale)
        check_attention(c, q, out, lse, 0, scale)
        c.close()


def test_a_row_with_nan_or_inf_stays_alone():
    c = Case([(40, 1)] * 3, heads=2, dim=64, page=16, seed=5, cu=False)
    c.fill()
    for dtype in (torch.float16, torch.bfloat16):
        q = c.numbers(3, 4, dtype)
        clean, _ = c.attend(q)
        q[1, 2, 9] = float("nan")
        q[2, 1, 3] = float("inf")
        out, _ = c.attend(q)
        bad = torch.zeros(3, 4, dtype=torch.bool, device="cuda")
        bad[1, 2] = bad[2, 1] = True
        assert torch.equal(out[~bad], clean[~bad])
        assert out[1, 2].isnan().all()
    c.close()


def test_zero_scale_is_the_mean_and_negative_scale_works():
    c = Case([(99, 1)], heads=1, dim=64, page=16, seed=6, cu=False)
    c.fill()
    q = c.numbers(1, 2, torch.float16)
    for scale in (0.0, -0.3):
        out, lse = c.attend(q, 0, scale)
        check_attention(c, q, out, lse, 0, scale)
    assert abs(c.attend(q, 0, 0.0)[1][0, 0].item() - math.log(100)) < 1e-5
    c.close()


# ------------------------------------------------------- bad steps and bad pages ---
def test_bad_pages_and_bad_steps_are_reported_and_skipped():
    c = Case([(50, 2), (40, 1), (10, 3), (70, 1)], heads=2, dim=128, page=16, seed=7)
    c.fill()
    q = c.numbers(c.rows, 4, torch.float16)
    good, _ = c.attend(q)
    keep = c.table.copy()
    c.table[0, 1], c.table[1, 2], c.table[3, 4] = c.n_pages, -1, 1 << 30      # positions 16..31, 32..40, 64..70
    c.step = c.make_step()
    out, lse = c.attend(q)
    assert R.bs_cache_get_device_error(c.handle) == R.BS_ERR_RANGE
    assert R.bs_cache_get_device_error(c.handle) == R.BS_OK
    check_attention(c, q, out, lse)
    assert torch.equal(out[3:6], good[3:6])
    before = c.pool().data
    k = c.numbers(c.rows, 2, torch.float16)
    R.bs_cache_append(c.handle, c.step, k, k)           # sequence 1's and 3's tokens fall on bad pages
    assert R.bs_cache_get_device_error(c.handle) == R.BS_ERR_RANGE
    after = oc.Pool(2, 128, 16, c.n_pages, before)
    kf = k.float().cpu().numpy()
    for i in (0, 2):
        for r in range(c.seqs[i][1]):
            for h in range(2):
                for value in (False, True):
                    after.store(int(c.table[i, (c.seqs[i][0] + r) // 16]), c.seqs[i][0] + r, h, value, kf[c.cu[i] + r, h])
    assert np.array_equal(c.pool().data, after.data)
    ko, vo = torch.full_like(k, 7.0), torch.full_like(k, 7.0)
    R.bs_cache_read(c.handle, c.step, ko, vo)
    assert R.bs_cache_get_device_error(c.handle) == R.BS_ERR_RANGE
    assert (ko[2] == 0).all() and (vo[6] == 0).all() and (ko[0] != 0).any()
    c.table = keep.copy()
    # all pages bad: rows that see nothing
    c.table[1] = -7
    c.step = c.make_step()
    out, lse = c.attend(q)
    assert (out[2] == 0).all() and (lse[2] == -np.inf).all()
    assert R.bs_cache_get_device_error(c.handle) == R.BS_ERR_RANGE
    c.table = keep.copy()
    c.step = c.make_step()
    R.bs_cache_append(c.handle, c.step, k, k)      # the appends below write the same rows at the same positions
    good, _ = c.attend(q)
    # rows backwards, out of range, more than max_new, positions past the table
    for change in ("back", "beyond", "negative", "max_new", "past"):
        cu, start, step = c.cu.copy(), c.start.copy(), None
        if change == "back":
            c.cu = np.array([0, 5, 3, 6, 7], np.int32)
        elif change == "beyond":
            c.cu = np.array([0, 2, 3, 6, 9], np.int32)
        elif change == "negative":
            c.cu = np.array([-1, 2, 3, 6, 7], np.int32)
        elif change == "past":
            c.start = np.array([50, 40, 2 ** 31 - 2, c.table.shape[1] * 16 - 1], np.int32)
        step = c.make_step(2 if change == "max_new" else None)
        out = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda")
        ws = torch.zeros(R.bs_cache_attention_workspace_bytes(c.handle, step, 4), dtype=torch.uint8, device="cuda")
        R.bs_cache_attention(c.handle, step, q, out, ws)
        assert R.bs_cache_get_device_error(c.handle) == R.BS_ERR_RANGE, change
        if change in ("max_new", "past"):
            assert (out[3:6] == 0).all() and torch.equal(out[:3], good[:3]), change
        R.bs_cache_read(c.handle, step, ko, vo)
        assert R.bs_cache_get_device_error(c.handle) == R.BS_ERR_RANGE, change
        R.bs_cache_append(c.handle, step, k, k)
        assert R.bs_cache_get_device_error(c.handle) == R.BS_ERR_RANGE, change
        c.cu, c.start = cu, start
    c.close()


def test_refusals():
    c = Case([(50, 2), (40, 1)], heads=2, dim=128, page=16, seed=7)
    q = c.numbers(c.rows, 4, torch.float16)
    out = torch.empty_like(q)
    need = R.bs_cache_attention_workspace_bytes(c.handle, c.step, 4)
    ws = torch.zeros(need + 256, dtype=torch.uint8, device="cuda")

    def status(fn, *args, **kw):
        with pytest.raises(R.BsError) as e:
            fn(*args, **kw)
        return e.value.status

    at = R.bs_cache_attention
    assert status(at, c.handle, c.step, q, out, ws[:need - 1]) == R.BS_ERR_CAPACITY
    assert status(at, c.handle, c.step, q, out, None) == R.BS_ERR_CAPACITY
    assert status(at, c.handle, c.step, q, out, ws[64:]) == R.BS_ERR_ALIGNMENT
    assert status(at, c.handle, c.step, q, out, ws, scale=float("inf")) == R.BS_ERR_INVALID_ARG
    assert status(at, c.handle, c.step, q, out, ws, window=-1) == R.BS_ERR_INVALID_ARG
    assert status(at, c.handle, c.step, q.float(), out.float(), ws) == R.BS_ERR_INVALID_ARG
    q3 = c.numbers(c.rows, 3, torch.float16)
    assert status(at, c.handle, c.step, q3, torch.empty_like(q3), ws) == R.BS_ERR_INVALID_ARG
    odd = torch.zeros(c.rows * 2 * 132 + 8, dtype=torch.float16, device="cuda")
    assert status(R.bs_cache_append, c.handle, c.step, odd[1:1 + c.rows * 256].view(-1, 2, 128),
                  q[:, :2]) == R.BS_ERR_ALIGNMENT
    strided = odd[:c.rows * 264].view(c.rows, 2, 132)[:, :, :128]        # head stride 132: not whole 16 bytes
    assert status(R.bs_cache_append, c.handle, c.step, strided, q[:, :2]) == R.BS_ERR_ALIGNMENT
    assert status(R.bs_cache_read, c.handle, c.step, None, None) == R.BS_ERR_INVALID_ARG
    for bad in (q[:1], q[:, :1], q[..., :64], q.transpose(1, 2), q.cpu()):
        with pytest.raises(ValueError):
            R.bs_cache_append(c.handle, c.step, bad, bad)
    with pytest.raises(ValueError):
        at(c.handle, c.step, q, out.bfloat16(), ws)
    with pytest.raises(ValueError):
        at(c.handle, c.step, q, out, ws, lse=torch.empty(c.rows, 4, device="cuda", dtype=torch.float16))
    host = R.CacheStep(torch.from_numpy(c.start), torch.from_numpy(c.table), c.rows, 2, torch.from_numpy(c.cu))
    with pytest.raises(ValueError):
        at(c.handle, host, q, out, ws)
    for n, m in ((-1, 2), (3, -1)):
        st = R.CacheStep(c.step.start, c.step.page_table, n, m, c.step.cu_new)
        assert R.lib.bs_cache_read(c.handle, st.ref, out.data_ptr(), None, 0, None) == R.BS_ERR_INVALID_ARG
    st = R.CacheStep(c.step.start, c.step.page_table, 1)                 # fewer rows than sequences
    assert R.lib.bs_cache_read(c.handle, st.ref, out.data_ptr(), None, 0, None) == R.BS_ERR_INVALID_ARG
    st = R.CacheStep(c.step.start, c.step.page_table, 1 << 30, 1)
    assert R.lib.bs_cache_read(c.handle, st.ref, out.data_ptr(), None, 0, None) == R.BS_ERR_RANGE
    # a step without rows does nothing
    empty = R.CacheStep(c.step.start, c.step.page_table, 0, 0, torch.zeros(3, dtype=torch.int32, device="cuda"))
    at(c.handle, empty, q[:0], out[:0], ws)
    R.bs_cache_append(c.handle, empty, q[:0, :2], q[:0, :2])
    assert R.bs_cache_get_device_error(c.handle) == R.BS_OK
    c.close()


# ------------------------------------------------------ streams, graphs, sharing ---
def test_a_token_loop_in_a_graph_follows_the_lengths():
    """Append and attention captured once, replayed while the lengths and pages move on the device."""
    c = Case([(0, 1), (15, 1), (40, 1), (-1, 1)], heads=2, dim=128, page=16, seed=9, cu=False, pages_more=20)
    c.table[:, -1] = 0
    spare = [p for p in range(c.n_pages) if p not in set(c.table.flatten())]
    wide = np.zeros((4, 8), np.int32)
    for i in range(4):
        own = list(c.table[i, :max(1, -(-(max(int(c.start[i]), 0) + 1) // 16))])
        while len(own) < 8 and spare and len(own) < 4 + i:
            own.append(spare.pop())
        wide[i, :len(own)] = own
    c.table = wide
    c.step = c.make_step()
    c.fill(upto=[max(int(s), 0) + 1 for s in c.start])
    k, v = c.numbers(4, 2, torch.bfloat16), c.numbers(4, 2, torch.bfloat16)
    q = c.numbers(4, 8, torch.bfloat16)
    out = torch.empty_like(q)
    lse = torch.empty(4, 8, device="cuda")
    ws = torch.zeros(R.bs_cache_attention_workspace_bytes(c.handle, c.step, 8), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        R.bs_cache_attention(c.handle, c.step, q, out, ws, lse=lse)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        R.bs_cache_append(c.handle, c.step, k, v)
        R.bs_cache_attention(c.handle, c.step, q, out, ws, lse=lse)
    for turn in range(12):
        for x in (k, v, q):
            x.copy_(torch.from_numpy(c.gen.standard_normal(x.shape).astype(np.float32)))
        g.replay()
        torch.cuda.synchronize()
        check_attention(c, q, out, lse)
        c.start = np.where(c.start >= 0, c.start + 1, c.start).astype(np.int32)
        if turn == 5:
            c.start[3], c.start[0] = 0, -1       # a slot fills, another empties
        c.step.start.copy_(torch.from_numpy(c.start))
    assert R.bs_cache_get_device_error(c.handle) == R.BS_OK
    c.close()


def test_two_streams_with_their_own_workspaces():
    c = Case([(3000, 1), (100, 1)], heads=2, dim=128, page=64, seed=10, cu=False)
    c.fill()
    q = c.numbers(2, 8, torch.float16)
    want, _ = c.attend(q)
    streams = [torch.cuda.Stream() for _ in range(2)]
    spaces = [torch.zeros(R.bs_cache_attention_workspace_bytes(c.handle, c.step, 8), dtype=torch.uint8, device="cuda")
              for _ in range(2)]
    outs = [[torch.empty_like(q) for _ in range(20)] for _ in range(2)]
    torch.cuda.synchronize()
    for i in range(20):
        for s in range(2):
            R.bs_cache_attention(c.handle, c.step, q, outs[s][i], spaces[s], stream=streams[s])
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for both in outs for o in both)
    c.close()


def test_shared_pages_and_one_workspace_for_changing_steps():
    """Two sequences read one prompt's pages; one workspace serves steps of other sizes in turn."""
    c = Case([(64, 1), (64, 1)], heads=2, dim=64, page=32, seed=11, cu=False)
    c.table[1, :2] = c.table[0, :2]
    c.step = c.make_step()
    c.fill(upto=[65, 0])
    k = c.numbers(2, 2, torch.float16)
    R.bs_cache_append(c.handle, c.step, k, k)
    q = c.numbers(2, 24, torch.float16)
    big = R.CacheStep(c.step.start, c.step.page_table, 2, 40)
    ws = torch.zeros(R.bs_cache_attention_workspace_bytes(c.handle, big, 24), dtype=torch.uint8, device="cuda")
    for heads in (24, 2, 8, 24):
        out, lse = c.attend(q[:, :heads], ws=ws)
        check_attention(c, q[:, :heads], out, lse)
    c.close()


@pytest.mark.parametrize("graph", [True, False])
def test_a_chain_of_reads_and_writes_sees_each_write(graph):
    """read, append, read, attention of the same positions, back to back: every kernel starts while the one before it
    ends, and none may work on what it, or one before it, held in a cache."""
    c = Case([(0, 9), (0, 30), (0, 1)], heads=2, dim=64, page=16, seed=41)
    k, v = c.numbers(c.rows, 2, torch.float16), c.numbers(c.rows, 2, torch.float16)
    q = c.numbers(c.rows, 4, torch.float16)
    new_k, new_v = torch.empty_like(k), torch.empty_like(v)
    first, second = torch.empty((2, *k.shape), device="cuda"), torch.empty((2, *k.shape), device="cuda")
    out = torch.empty_like(q)
    ws = torch.zeros(R.bs_cache_attention_workspace_bytes(c.handle, c.step, 4), dtype=torch.uint8, device="cuda")

    def chain():
        R.bs_cache_append(c.handle, c.step, k, v)
        R.bs_cache_read(c.handle, c.step, first[0], first[1])
        R.bs_cache_append(c.handle, c.step, new_k, new_v)
        R.bs_cache_read(c.handle, c.step, second[0], second[1])
        R.bs_cache_attention(c.handle, c.step, q, out, ws)

    if graph:
        chain()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            chain()
    for _ in range(30):
        for x in (k, v, new_k, new_v):
            x.copy_(torch.from_numpy(c.gen.standard_normal(x.shape).astype(np.float32)))
        g.replay() if graph else chain()
        torch.cuda.synchronize()
        for got, dense in ((first[0], k), (first[1], v), (second[0], new_k), (second[1], new_v)):
            codes, s, b = oc.quantise(dense.float().cpu().numpy())
            assert np.array_equal(got.double().cpu().numpy().reshape(-1), np.float32(oc.dequantise(codes, s, b)).astype(np.float64).reshape(-1))
        want, _ = c.attend(q)
        assert torch.equal(out, want)
    c.close()


@pytest.mark.parametrize("new", [3, 60])
def test_positions_up_to_the_largest(new):
    """The last positions of a context of 2^31 - 512 tokens under a window, in shared pages: as the same
    tokens at the end of a context of 512."""
    c = Case([(512 - new, new)], heads=1, dim=64, page=256, seed=new, pages_more=1)
    c.fill()
    q = c.numbers(new, 2, torch.float16)
    want = c.attend(q, 200)
    check_attention(c, q, *want, 200, sample=8)
    end = 2 ** 31 - 512
    table = torch.full((1, 2 ** 23), c.n_pages + 5, dtype=torch.int32, device="cuda")
    table[0, end // 256 - 2:end // 256] = torch.from_numpy(c.table[0, :2]).cuda()
    start = torch.tensor([end - new], dtype=torch.int32, device="cuda")
    far = R.CacheStep(start, table, new, new, torch.tensor([0, new], dtype=torch.int32, device="cuda"))
    got = c.attend(q, 200, step=far)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    k, v = c.numbers(new, 1, torch.float16), c.numbers(new, 1, torch.float16)
    R.bs_cache_append(c.handle, far, k, v)
    here, there = torch.empty((2, 2, *k.shape), dtype=torch.float16, device="cuda")
    R.bs_cache_read(c.handle, far, there[0], there[1])
    R.bs_cache_read(c.handle, c.step, here[0], here[1])
    assert torch.equal(here, there) and (here[0] - k).abs().max() < 0.5
    assert R.bs_cache_get_device_error(c.handle) == R.BS_OK
    start += 1
    out, lse = c.attend(q, 200, step=far)
    R.bs_cache_append(c.handle, far, k * 0, v * 0)
    R.bs_cache_read(c.handle, far, there[0], there[1])
    assert (out == 0).all() and (lse == -np.inf).all() and (there == 0).all()
    assert R.bs_cache_get_device_error(c.handle) == R.BS_ERR_RANGE
    R.bs_cache_read(c.handle, c.step, there[0], there[1])
    assert torch.equal(here, there)
    c.close()


@pytest.mark.parametrize("new", [1, 40])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_slices_of_a_joined_projection_and_broadcast_heads(new, dim):
    """q, k and v as slices of one tensor, heads before tokens, one row for all: as their contiguous copies."""
    c = Case([(30, new), (5, new)], heads=2, dim=dim, page=16, seed=dim + new)
    c.fill()
    joined = c.numbers(c.rows, 8 + 2 + 2, torch.bfloat16)
    q, k, v = joined[:, :8], joined[:, 8:10], joined[:, 10:]
    want = c.attend(q.contiguous())
    assert all(torch.equal(x, y) for x, y in zip(c.attend(q), want))
    turned = q.transpose(0, 1).contiguous().transpose(0, 1)
    assert all(torch.equal(x, y) for x, y in zip(c.attend(turned), want))
    got = torch.empty((4, c.rows, 2, dim), device="cuda")
    R.bs_cache_append(c.handle, c.step, k, v)
    R.bs_cache_read(c.handle, c.step, got[0], got[1])
    R.bs_cache_append(c.handle, c.step, k.contiguous(), v.contiguous())
    R.bs_cache_read(c.handle, c.step, got[2], got[3])
    assert torch.equal(got[:2], got[2:])
    one = joined[:1, 8:9].expand(c.rows, 2, dim)
    R.bs_cache_append(c.handle, c.step, one, one)
    R.bs_cache_read(c.handle, c.step, got[0], got[1])
    assert (got[:2] == got[0, 0, 0]).all()
    same = joined[:1, :1].expand(c.rows, 8, dim)
    assert all(torch.equal(x, y) for x, y in zip(c.attend(same), c.attend(same.contiguous())))
    c.close()


def test_an_error_on_another_stream_is_read_without_waiting_for_it():
    c = Case([(0, 3)], heads=1, dim=64, page=16, seed=51)
    k = c.numbers(3, 1, torch.float16)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)             # some 10 ms
        c.step.page_table.fill_(c.n_pages)
        R.bs_cache_append(c.handle, c.step, k, k)
    assert R.bs_cache_get_device_error(c.handle) == R.BS_ERR_RANGE
    assert R.bs_cache_get_device_error(c.handle) == R.BS_OK
    c.close()


def test_the_most_sequences_of_a_step():
    gen = np.random.default_rng(52)
    starts = gen.integers(0, 40, 4096)
    c = Case([(int(s) if s % 9 else -1, 1) for s in starts], heads=1, dim=64, page=16, seed=52, cu=False)
    c.fill(upto=[max(int(s), 0) + 1 for s in c.start])
    q = c.numbers(4096, 2, torch.bfloat16)
    out, lse = c.attend(q)
    check_attention(c, q, out, lse)
    assert R.bs_cache_get_device_error(c.handle) == R.BS_OK
    c.close()


@pytest.mark.parametrize("dim,n", [(64, 4096), (128, 400), (128, 2500), (256, 300)])
def test_many_rows_of_many_sequences(dim, n):
    """Row counts for the kernel for many rows, with as many sequences as its shared memory holds, and more."""
    c = Case([(i % 50 if i % 31 == 0 else -1, 7) for i in range(n)], heads=1, dim=dim, page=16, seed=n, pages_more=0)
    c.fill(upto=[int(s) + 7 if s >= 0 else 0 for s in c.start])
    q = c.numbers(c.rows, 8, torch.bfloat16)
    out, lse = c.attend(q)
    check_attention(c, q, out, lse, sample=1)
    c.close()


def test_pages_beyond_four_gib():
    heads, dim, page = 8, 128, 64
    n_pages = (9 << 29) // R.bs_cache_page_bytes(heads, dim, page)
    store = torch.empty(R.bs_cache_device_bytes(heads, dim, page, n_pages), dtype=torch.uint8, device="cuda")
    handle = R.bs_cache_create(heads, dim, page, n_pages, store)
    c = Case([(150, 1)], heads=heads, dim=dim, page=page, seed=12, cu=False)
    c.fill()
    q = c.numbers(1, 16, torch.float16)
    want, _ = c.attend(q)
    far = np.array([[n_pages - 1, n_pages - 5, n_pages - 2, 0]], np.int32)
    small = c.store[:c.n_pages * R.bs_cache_page_bytes(heads, dim, page)].view(c.n_pages, -1)
    pages = store[:n_pages * R.bs_cache_page_bytes(heads, dim, page)].view(n_pages, -1)
    for i in range(3):
        pages[int(far[0, i])] = small[int(c.table[0, i])]
    step = R.CacheStep(c.step.start, torch.from_numpy(far).cuda(), 1)
    out = torch.empty_like(q)
    ws = torch.zeros(R.bs_cache_attention_workspace_bytes(handle, step, 16), dtype=torch.uint8, device="cuda")
    R.bs_cache_attention(handle, step, q, out, ws)
    assert torch.equal(out, want)
    k = c.numbers(1, heads, torch.float16)
    R.bs_cache_append(handle, step, k, k)
    back = torch.empty_like(k)
    R.bs_cache_read(handle, step, back, None)
    assert torch.equal(back.float().cpu(), torch.from_numpy(oc.dequantise(*oc.quantise(k.float().cpu().numpy()))).half().float())
    assert R.bs_cache_get_device_error(handle) == R.BS_OK
    R.bs_cache_destroy(handle)
    c.close()
