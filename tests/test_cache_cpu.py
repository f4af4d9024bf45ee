"""CPU tests of the packed key/value cache: the layout of a chunk, the quantisation's
bounds, the ABI's sizes and refusals, and a mirror of the attention kernel's work split
and lane reads.  No GPU is needed; no compute call is made."""
import ctypes

import numpy as np
import pytest

import residual_block_decomp_b200 as R
from oracle import cache as oc

DIMS = (64, 128, 256)


# ------------------------------------------------------------------ layout -------
@pytest.mark.parametrize("dim", DIMS)
def test_chunk_places_cover_every_byte_once(dim):
    seen = np.zeros((oc.chunk_bytes(dim), 2), int)
    for value in (False, True):
        for t in range(16):
            for d in range(dim):
                byte, shift = oc.code_place(dim, value, t, d)
                seen[byte, shift // 4] += 1
            for g in range(dim // 32):
                at = oc.pair_place(dim, value, t, g)
                seen[at:at + 4] += 1
    assert (seen == 1).all()


@pytest.mark.parametrize("dim", DIMS)
def test_store_and_load_round_trip(dim):
    gen = np.random.default_rng(dim)
    pool = oc.Pool(2, dim, 32, 3)
    x = gen.standard_normal((40, 2, 2, dim)).astype(np.float32)
    for pos in range(40):
        for h in range(2):
            for value in (False, True):
                pool.store(2 - pos // 32, pos, h, value, x[pos, h, int(value)])
    for pos in range(40):
        for h in range(2):
            for value in (False, True):
                got = pool.load(2 - pos // 32, pos, h, value)
                assert np.array_equal(got, oc.dequantise(*oc.quantise(x[pos, h, int(value)])))


# -------------------------------------------------------------- quantisation -----
def _bound(x):
    """The header's bound on |stored - x|: half a step, and half a step of fp16 of b and of 8 s
    (2^-25 for subnormals), with the fp32 arithmetic's own roundings (a few 2^-24 of the sizes)."""
    c, s, b = oc.quantise(x)
    s, b = (np.repeat(v.astype(np.float64), 32, -1) for v in (s, b))
    size = np.abs(b) + 8 * s
    return s / 2 + 2.0 ** -11 * size + 9 * 2.0 ** -25 + 8 * 2.0 ** -24 * size


@pytest.mark.parametrize("kind", ["normal", "outlier", "offset", "equal", "zero", "tiny", "large"])
def test_quantisation_error_bound(kind):
    gen = np.random.default_rng(5)
    x = gen.standard_normal((200, 128)).astype(np.float32)
    if kind == "outlier":
        x[:, ::37] *= 50
    elif kind == "offset":
        x = x * 0.01 + 100
    elif kind == "equal":
        x[:] = 0.7
    elif kind == "zero":
        x[:] = 0
    elif kind == "tiny":
        x *= 1e-7
    elif kind == "large":
        x *= 20000
    x = np.clip(x, -oc.CLAMP, oc.CLAMP)
    err = np.abs(oc.dequantise(*oc.quantise(x)) - x)
    assert (err <= _bound(x)).all()
    if kind == "normal":   # a planted code one step off breaks the bound
        c, s, b = oc.quantise(x)
        assert (np.abs(oc.dequantise((c + 1) % 16, s, b) - x) > _bound(x)).any()


def test_stored_numbers_are_finite_in_fp16():
    """The clamp keeps b + s (c - 8) inside fp16 for the most extreme groups, infinities and NaN."""
    ext = np.array([np.inf, -np.inf, np.nan, 65504, -65504, 3e38, 1e-30, 0], np.float32)
    gen = np.random.default_rng(6)
    x = gen.choice(ext, size=(5000, 64))
    y = oc.dequantise(*oc.quantise(x))
    assert np.isfinite(y).all() and np.abs(y).max() <= 65504


# ------------------------------------------------------------ sizes, refusals ----
def test_sizes():
    for heads, dim, page in [(8, 128, 64), (1, 64, 16), (3, 256, 256)]:
        pb = oc.page_bytes(heads, dim, page)
        assert R.bs_cache_page_bytes(heads, dim, page) == pb == heads * page * dim * 5 // 4
        assert R.bs_cache_device_bytes(heads, dim, page, 7) == (7 * pb + 255) // 256 * 256 + 256
    for bad in [(0, 128, 64), (1025, 128, 64), (8, 96, 64), (8, 128, 8), (8, 128, 48), (8, 128, 512)]:
        assert R.bs_cache_page_bytes(*bad) == 0
    assert R.bs_cache_device_bytes(8, 128, 64, 0) == 0
    # beyond 32 bits
    assert R.bs_cache_device_bytes(8, 128, 64, 100000) == 100000 * 81920 + 256


def test_create_validates_before_touching_a_device():
    h = ctypes.c_void_p()
    fake = ctypes.c_void_p(1 << 20)
    need = R.bs_cache_device_bytes(8, 128, 64, 4)
    create = R.lib.bs_cache_create
    assert create(8, 128, 64, 4, None, need, None, ctypes.byref(h)) == R.BS_ERR_INVALID_ARG
    assert create(8, 128, 64, 4, fake, need, None, None) == R.BS_ERR_INVALID_ARG
    assert create(8, 128, 64, 0, fake, need, None, ctypes.byref(h)) == R.BS_ERR_INVALID_ARG
    assert create(8, 100, 64, 4, fake, need, None, ctypes.byref(h)) == R.BS_ERR_UNSUPPORTED_SHAPE
    assert create(8, 128, 20, 4, fake, need, None, ctypes.byref(h)) == R.BS_ERR_UNSUPPORTED_SHAPE
    assert create(8, 128, 64, 4, ctypes.c_void_p((1 << 20) + 16), need, None, ctypes.byref(h)) == R.BS_ERR_ALIGNMENT
    assert create(8, 128, 64, 4, fake, need - 1, None, ctypes.byref(h)) == R.BS_ERR_CAPACITY
    import torch
    if not torch.cuda.is_available():
        assert create(8, 128, 64, 4, fake, need, None, ctypes.byref(h)) == R.BS_ERR_NO_DEVICE
        assert h.value is None


def test_null_handles_are_rejected():
    assert R.lib.bs_cache_destroy(None) == R.BS_ERR_INVALID_ARG
    assert R.lib.bs_cache_append(None, None, None, 0, 0, None, 0, 0, 0, None) == R.BS_ERR_INVALID_ARG
    assert R.lib.bs_cache_read(None, None, None, None, 0, None) == R.BS_ERR_INVALID_ARG
    assert R.lib.bs_cache_attention(None, None, None, 0, 0, 8, 0, 1.0, 0, None, None, None, 0,
                                    None) == R.BS_ERR_INVALID_ARG
    assert R.lib.bs_cache_attention_workspace_bytes(None, None, 8) == 0
    assert R.lib.bs_cache_get_device_error(None) == R.BS_ERR_INVALID_ARG


def test_step_refuses_wrong_tensors():
    import torch
    table = torch.zeros(2, 3, dtype=torch.int32)
    start = torch.zeros(2, dtype=torch.int32)
    R.CacheStep(start, table, 2)
    for args in [(start.long(), table, 2), (start, table.long(), 2), (start, table[0], 2), (start[:1], table, 1),
                 (start, table.t().contiguous().t(), 2), (start, table, 2, 1, start)]:
        with pytest.raises(ValueError):
            R.CacheStep(*args)


# ------------------------------------------------ the attention kernel's split ----
def _split(tiles, grid, warps):
    """The kernel's tiles of a CTA, and its runs: [(cta, warp, first tile, last tile + 1)] of a list of `tiles`."""
    per = max(-(-tiles // grid), warps)
    out = []
    for c in range(grid):
        c0 = per * c
        c1 = max(min(c0 + per, tiles), c0)
        for w in range(warps):
            a, b = c0 + (c1 - c0) * w // warps, c0 + (c1 - c0) * (w + 1) // warps
            if a < b:
                out.append((c, w, a, b))
    return per, out


@pytest.mark.parametrize("seed", range(40))
def test_work_split_covers_the_list_once_and_counts_arrivals(seed):
    gen = np.random.default_rng(seed)
    grid, warps = 148, int(gen.choice([8, 12]))
    items = gen.integers(1, int(gen.choice([2, 5, 60, 3000])), size=int(gen.integers(1, 200)))
    begin = np.concatenate([[0], np.cumsum(items)])
    T = int(begin[-1])
    per, runs = _split(T, grid, warps)
    assert [r[2] for r in runs[1:]] == [r[3] for r in runs[:-1]] and runs[0][2] == 0 and runs[-1][3] == T
    counts = {}
    for i, size in enumerate(items):
        a, b = int(begin[i]), int(begin[i + 1])
        ctas = sorted({c for c, _, x, y in runs if x < b and y > a})
        f0, f1 = a // per, (b - 1) // per                               # the kernel's cta_of
        assert ctas == list(range(f0, f1 + 1)) and f1 < grid
        if f1 > f0:
            # the counter of CTA f0 belongs to this item alone, and every CTA of it has a part of its own
            assert f0 not in counts
            counts[f0] = i
            assert per * f0 <= a
            for c in range(f0 + 1, f1 + 1):
                assert per * c > a            # parts 2 c of the later ones, 2 f0 + 1 of the first
    # a warp holds at most two partial results: of its run's first and last item
    for c, w, x, y in runs:
        cut = [i for i in range(len(items)) if begin[i] < y and begin[i + 1] > x and not (x <= begin[i] and begin[i + 1] <= y)]
        assert len(cut) <= 2 and all(begin[i] < x or begin[i + 1] > y for i in cut)


@pytest.mark.parametrize("dim", DIMS)
def test_lane_reads_hit_their_numbers(dim):
    """Mirror of the kernel's copies and fragment reads: every 16-byte unit of a tile lands once inside
    its 5120-byte stage, and every lane's word and pair is the one the layout names."""
    gr, jn, uc = dim // 32, dim // 64, oc.chunk_bytes(dim) // 16
    tm = 4096 // dim // 16
    unit = {}
    for k in range(10):
        for lane in range(32):
            u = k * 32 + lane
            if dim == 64:
                half = k // 5
                v = u - half * 160
                m, o = 2 * half + (v >= uc), v - uc if v >= uc else v
            else:
                m = k // (uc // 32)
                o = u - m * uc
            d = o
            if dim == 256:
                if o < 128:
                    d = o ^ ((o >> 3) & 1)
                elif 160 <= o < 288:
                    d = o ^ ((((o - 160) >> 3) & 3) << 1)
            assert 0 <= m < tm and 0 <= o < uc and 0 <= d < uc and (m, d) not in unit
            unit[m, d] = o
    assert len(unit) == 320
    at = lambda off: unit[0, off // 16] * 16 + off % 16  # noqa: E731
    for lane in range(32):
        t, cc = lane >> 2, lane & 3
        for row in (t, t + 8):
            if dim == 256:
                words = [row * 128 + ((cc * 2 + i) ^ (t & 1)) * 16 + 4 * e for i in range(2) for e in range(4)]
            else:
                words = [row * (dim // 2) + cc * (dim // 8) + 4 * g for g in range(gr)]
            for g, off in enumerate(words):
                assert (at(off), 0) == oc.code_place(dim, False, row, 32 * g + 8 * cc)
                assert at(8 * dim + row * (dim // 8) + 4 * g) == oc.pair_place(dim, False, row, g)
        for i in range(4):
            tok, row = 2 * cc + (i & 1) + (i >> 1) * 8, cc + (i & 1) * 8 + (i >> 1) * 4
            for j in range(jn):
                w = t + 8 * j
                base = 10 * dim + (row * 128 + (t ^ ((row & 3) << 1)) * 16 if dim == 256 else row * (dim // 2) + t * (dim // 16))
                assert (at(base + 4 * j), 0) == oc.code_place(dim, True, tok, 8 * w)
                assert at(18 * dim + row * (dim // 8) + (t >> 2) * (dim // 16) + 4 * j) == oc.pair_place(dim, True, tok, w // 4)


# ------------------------------------------------------------------- page table ---
def test_page_table_hands_out_each_page_once_and_takes_them_back():
    t = R.PageTable(10, 16)
    a, b = t.open(), t.open()
    start, pages = t.advance([a, b], [16, 17])
    assert start == [0, 0] and [len(p) for p in pages] == [1, 2]
    start, pages = t.advance([b, a], [15, 0])
    assert start == [17, 16] and [len(p) for p in pages] == [2, 1]
    start, pages = t.advance([a], [1], room=40)      # 17 tokens, pages for 57
    assert start == [16] and len(pages[0]) == 4 and t.length[a] == 17
    assert t.advance([a], [40])[0] == [17] and len(t.pages[a]) == 4
    held = t.pages[a] + t.pages[b]
    assert len(set(held + t.free)) == 10 and len(held + t.free) == 10
    mine = list(t.pages[a])
    t.close(a)
    c = t.open()
    assert c not in (a, b) and t.advance([c], [64])[1][0] == mine


def test_page_table_refusals_change_nothing():
    t = R.PageTable(4, 32)
    a, b = t.open(), t.open()
    t.advance([a], [33])
    before = (dict(t.length), {k: list(v) for k, v in t.pages.items()}, list(t.free))
    for seqs, new, room, error in [([a, a], [1, 1], 0, ValueError), ([a], [1, 2], 0, ValueError), ([], [], 0, ValueError),
                                   ([a], [-1], 0, ValueError), ([a], [1], -1, ValueError), ([a, 9], [1, 1], 0, KeyError),
                                   ([a, b], [32, 64], 0, R.BsError), ([b], [1], 100, R.BsError),
                                   ([a], [2 ** 31 - 33], 0, R.BsError)]:
        with pytest.raises(error):
            t.advance(seqs, new, room)
        assert before == (dict(t.length), {k: list(v) for k, v in t.pages.items()}, list(t.free))
    t.advance([a, b], [31, 64])
    with pytest.raises(KeyError):
        t.close(17)


def _cache_of(table):
    """A BitStackCache without a pool: what step() does on the host."""
    cache = R.BitStackCache.__new__(R.BitStackCache)
    cache.table, cache.handles = table, []
    cache.device = "cpu"
    return cache


def _state(t):
    return dict(t.length), {k: list(v) for k, v in t.pages.items()}, list(t.free)


def test_a_refused_step_changes_nothing(monkeypatch):
    import torch
    cache = _cache_of(R.PageTable(5000, 16))
    seqs = [cache.open() for _ in range(4097)]
    before = _state(cache.table)
    with pytest.raises(R.BsError) as e:
        cache.step(seqs, [1] * 4097)
    assert e.value.status == R.BS_ERR_RANGE and _state(cache.table) == before
    # rows that pass 32 bits together, though no sequence does
    cache = _cache_of(R.PageTable(2 ** 23 + 8, 256))
    seqs = [cache.open(), cache.open()]
    with pytest.raises(R.BsError) as e:
        cache.step(seqs, [2 ** 30, 2 ** 30 + 1])
    assert e.value.status == R.BS_ERR_RANGE
    assert cache.table.length == {0: 0, 1: 0} and len(cache.table.free) == 2 ** 23 + 8
    # no memory for the step's arrays
    cache = _cache_of(R.PageTable(20, 16))
    seqs = [cache.open() for _ in range(3)]
    cache.table.advance(seqs, [20, 1, 0])
    before = _state(cache.table)

    def none(self):
        raise RuntimeError("out of memory")

    monkeypatch.setattr(torch.Tensor, "pin_memory", none)
    for new, room in (([40, 16, 1], 0), ([1, 1, 1], 30), ([0, 0, 0], 0)):
        with pytest.raises(RuntimeError, match="out of memory"):
            cache.step(seqs, new, room)
        assert _state(cache.table) == before
    # during a capture
    monkeypatch.setattr(torch.cuda, "is_initialized", lambda: True)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
    with pytest.raises(RuntimeError, match="capture"):
        cache.step(seqs, [1, 1, 1])
    assert _state(cache.table) == before


def test_numbers_that_no_c_int_holds_are_refused(monkeypatch):
    """They would be cut to 32 bits: a window of 2^32 taken for none, 2^32 + 4 pages for 4."""
    import torch
    from residual_block_decomp_b200 import binding as B
    big = 2 ** 32
    assert R.bs_cache_device_bytes(8, 128, 64, big + 4) == 0 and R.bs_cache_device_bytes(big + 8, 128, 64, 4) == 0
    assert R.bs_cache_page_bytes(8, big + 128, 64) == 0 and R.bs_cache_page_bytes(8, 128, big + 64) == 0
    table, start = torch.zeros(1, 3, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    assert R.CacheStep(start, table, big + 1).c.n_tokens < 0
    assert R.CacheStep(start, table, 1, big + 1).c.max_new < 0
    seen, real = {}, B.lib

    class Lib:
        def __getattr__(self, name):
            return getattr(real, name)

        def bs_cache_attention(self, handle, step, q, tok, head, heads, dt, scale, window, *rest):
            seen["window"] = window
            return B.BS_OK

        def bs_cache_create(self, *a):
            seen["create"] = a[:4]
            return B.BS_ERR_INVALID_ARG

        def bs_cache_attention_workspace_bytes(self, handle, step, heads):
            return max(0, heads)

    monkeypatch.setattr(B, "lib", Lib())
    monkeypatch.setattr(B, "_cache_stream", lambda *a: None)
    monkeypatch.setitem(B._cache_shapes, 77, (1, 64, torch.device("cpu"), 0))
    q = torch.zeros(1, 1, 64, dtype=torch.float16)
    for window, given in ((0, 0), (7, 7), (2 ** 31 - 1, 2 ** 31 - 1), (2 ** 31, -1), (big, -1), (big + 7, -1), (-5, -5)):
        R.bs_cache_attention(77, R.CacheStep(start, table, 1), q, torch.empty_like(q), None, window=window)
        assert seen["window"] == given
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)

    class Pool(torch.Tensor):                                # of GPU 0, as far as the binding sees
        is_cuda = True

        def get_device(self):
            return 0

    with pytest.raises(R.BsError):
        R.bs_cache_create(1, 64, 16, big + 1, torch.zeros(16).as_subclass(Pool), stream=0)
    assert seen["create"] == (1, 64, 16, -1)
    assert R.bs_cache_attention_workspace_bytes(77, R.CacheStep(start, table, 1), big + 2) == 0


def test_memory_that_is_not_what_it_looks_like_is_refused(monkeypatch):
    """A pool in host memory, on another GPU, or of one byte seen a million times; a workspace of one byte."""
    import torch
    from residual_block_decomp_b200 import binding as B
    real = B.lib

    class Lib:
        def __getattr__(self, name):
            assert name == "bs_status_string", f"{name} was called"
            return getattr(real, name)

    class Pool(torch.Tensor):
        is_cuda = True

        def get_device(self):
            return 1

    monkeypatch.setattr(B, "lib", Lib())
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    for pool in (torch.zeros(1 << 20, dtype=torch.uint8), torch.zeros(1 << 20, dtype=torch.uint8).as_subclass(Pool),
                 torch.zeros(1, dtype=torch.uint8).expand(1 << 20)):
        with pytest.raises(ValueError, match="pool"):
            R.bs_cache_create(1, 64, 16, 4, pool)
    monkeypatch.setitem(B._cache_shapes, 77, (1, 64, torch.device("cpu"), 0))
    table, start = torch.zeros(1, 3, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    q = torch.zeros(1, 1, 64, dtype=torch.float16)
    with pytest.raises(ValueError, match="workspace"):
        R.bs_cache_attention(77, R.CacheStep(start, table, 1), q, torch.empty_like(q), torch.zeros(1, dtype=torch.uint8).expand(1 << 24))


def test_a_handle_that_is_made_again_while_it_is_destroyed_keeps_its_shape(monkeypatch):
    from residual_block_decomp_b200 import binding as B

    class Lib:
        def bs_cache_destroy(self, handle):
            B._cache_shapes[handle] = "another thread's"     # as its bs_cache_create does with the memory just freed
            return B.BS_OK

    monkeypatch.setattr(B, "lib", Lib())
    monkeypatch.setitem(B._cache_shapes, 77, "mine")
    R.bs_cache_destroy(77)
    assert B._cache_shapes[77] == "another thread's"
