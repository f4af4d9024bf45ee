"""GPU: the cache's layer and the attention block: q/k/v linears, packed cache and output linear in a run, as a
model uses them."""
import numpy as np
import pytest
import torch

import residual_block_decomp_b200 as R
import workloads as wl
from residual_block_decomp_b200.layer import record_from_parts
from tests.gpu_util import assert_close
from tests.test_gpu_9_cache import check_attention

pytestmark = pytest.mark.gpu

D_MODEL, DIM, HEADS, Q_HEADS = 512, 64, 2, 8


def random_linear(m, d, gen, blocks=3):
    lin = R.BitStackLinear(m, d, blocks, wl.synthetic_inv_scale(d, gen))
    for i in range(blocks):
        words = gen.integers(0, 2 ** 32, size=m * d // 32, dtype=np.uint64).astype(np.uint32)
        U = wl.random_factors(m, 16, gen, 0.12 / np.sqrt(i + 1.0))
        V = wl.random_factors(d, 16, gen, 0.12 / np.sqrt(i + 1.0))
        lin.add_record(record_from_parts(words, U, V))
    lin.set_loaded(blocks)
    return lin


def block(gen, cache, **kw):
    kv = HEADS * DIM
    lins = [random_linear(m, d, gen) for m, d in
            ((Q_HEADS * DIM, D_MODEL), (kv, D_MODEL), (kv, D_MODEL), (D_MODEL, Q_HEADS * DIM))]
    return R.BitStackAttention(*lins, cache, **kw)


def inputs(gen, rows, dtype):
    return torch.from_numpy(gen.standard_normal((rows, D_MODEL)).astype(np.float32)).to(dtype).cuda()


class View:
    """The pool of a cache's layer under a step, as check_attention reads it."""

    def __init__(self, cache, step, layer, new):
        from oracle import cache as oc
        self.dim, self.heads, self.page = cache.dim, cache.heads, cache.table.page_tokens
        self.seqs, self.step = new, step
        self.start = step.start.cpu().numpy()
        self.table = step.page_table.cpu().numpy()
        self.cu = None if step.cu_new is None else step.cu_new.cpu().numpy()
        self.pool = lambda: oc.Pool(cache.heads, cache.dim, self.page, cache.table.n_pages,
                                    cache.dev_pages[layer].cpu().numpy())


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_two_blocks_answer_prompts_and_tokens(dtype):
    """Prompts, then tokens of two sequences, a third one that joins, a piece of a prompt; blocks dropped on the way.
    Each call's attention against the float64 oracle on the pool's bytes, its linears against the rebuilt weights."""
    gen = np.random.default_rng(5)
    cache = R.BitStackCache(HEADS, DIM, 40, 16, layers=2)
    blocks = [block(gen, cache, layer=0), block(gen, cache, layer=1, window=20, scale=0.2)]
    a, b, c = cache.open(), cache.open(), cache.open()
    for n, (seqs, new) in enumerate([([a, b], [37, 20]), ([a, b], [1, 1]), ([b, a, c], [1, 1, 90]), ([c, a], [1, 1]),
                                     ([a, c, b], [4, 0, 1])]):
        if n == 3:
            blocks[0].q.set_loaded(1)
            blocks[1].v.set_loaded(2)
            blocks[1].o.set_loaded(1)
        step = cache.step(seqs, new)
        x = inputs(gen, sum(new), dtype)
        for i, blk in enumerate(blocks):
            seen = {}

            def between(q, k):
                seen["q"], seen["k"] = q * 1.25, k.flip(2)
                return seen["q"], seen["k"]

            y = blk(x, step, between)
            x64 = x.double().cpu().numpy()
            W = {name: getattr(blk, name).reconstruct(dtype=torch.float32).double().cpu().numpy() for name in "qkvo"}
            assert_close(seen["k"].flip(2).reshape(len(x), -1), x64 @ W["k"].T, what="k")
            lse = torch.empty(len(x), Q_HEADS, device="cuda")
            out = cache.attention(step, seen["q"], i, blk.scale, blk.window, lse=lse)
            check_attention(View(cache, step, i, new), seen["q"], out, lse, blk.window, blk.scale, sample=4)
            o64 = out.reshape(len(x), -1).double().cpu().numpy() @ W["o"].T
            assert_close(y, o64, what="o")
            got_k, got_v = cache.read(step, i, torch.float32)
            want_v = blk.v(x).float().view(len(x), HEADS, DIM)
            for got, want in ((got_k, seen["k"].float()), (got_v, want_v)):   # a step of 4 bits, and its fp16 pair
                r = want.reshape(len(x), HEADS, DIM // 32, 32)
                width = (r.amax(3) - r.amin(3)) / 15
                # half a step, off by fp16 roundings of (s, b): 2^-11 (8 s + |b|), and 2^-24 below fp16's range
                tol = 0.5 * width + 2.0 ** -11 * 1.01 * (8.5 * width + r.abs().amax(3)) + 2.0 ** -20
                assert ((got.reshape(r.shape) - r).abs() <= tol[..., None]).all()
            assert blk.device_error() == R.BS_OK
            x = y
    cache.close_sequence(b)
    assert len(cache.table.free) == 40 - len(cache.table.pages[a]) - len(cache.table.pages[c])


def test_same_bits_as_the_single_calls():
    gen = np.random.default_rng(6)
    cache, twin = (R.BitStackCache(HEADS, DIM, 12, 32) for _ in range(2))
    blk = block(gen, cache)
    s, t = cache.open(), twin.open()
    for rows in (70, 1, 4, 5):
        step, other = cache.step([s], [rows]), twin.step([t], [rows])
        x = inputs(gen, rows, torch.bfloat16)
        y = blk(x, step)
        q, k, v = (lin(x).view(rows, -1, DIM) for lin in (blk.q, blk.k, blk.v))
        twin.append(other, k, v)
        assert torch.equal(blk.o(twin.attention(other, q).view(rows, -1)), y)
    assert torch.equal(cache.read(step)[0], twin.read(other)[0])
    assert blk.device_error() == R.BS_OK


def test_a_longer_cache_leaves_fewer_blocks():
    """The cache's bytes come off the memory budget that decides how many blocks stay loaded."""
    gen = np.random.default_rng(7)
    blk = block(gen, R.BitStackCache(HEADS, DIM, 8, 16))
    lins = (blk.q, blk.k, blk.v, blk.o)
    weight, _ = R.bs_plan_order([3] * 4, R.BS_ORDER_AVERAGE)
    sizes = [lin.block_bytes for lin in lins]
    budget = sum(sizes) * 3 + blk.cache.device_bytes
    loaded, pages = [], [8, 40, 64]
    for n in pages:
        cache = R.BitStackCache(HEADS, DIM, n, 16)
        plan = R.bs_plan_budget(weight, sizes, max(0, budget - cache.device_bytes))
        for lin, count in zip(lins, plan):
            lin.set_loaded(int(count))
        loaded.append([lin.n_blocks for lin in lins])
        assert sum(c * s for c, s in zip(loaded[-1], sizes)) + cache.device_bytes <= budget
        layer = R.BitStackAttention(*lins, cache)
        x = inputs(gen, 3, torch.float16)
        seq = cache.open()
        y = layer(x, cache.step([seq], [3]))
        assert torch.isfinite(y).all() and layer.device_error() == R.BS_OK
    assert loaded[0] == [3] * 4 and sum(loaded[0]) > sum(loaded[1]) > sum(loaded[2])


def test_token_steps_in_a_graph():
    gen = np.random.default_rng(8)
    cache, twin = (R.BitStackCache(HEADS, DIM, 24, 16) for _ in range(2))
    blk = block(gen, cache)
    eager = R.BitStackAttention(blk.q, blk.k, blk.v, blk.o, twin)
    seqs, others = [cache.open() for _ in range(3)], [twin.open() for _ in range(3)]
    x = inputs(gen, 17 + 30 + 1, torch.float16)
    blk(x, cache.step(seqs, [17, 30, 1]))
    eager(x, twin.step(others, [17, 30, 1]))
    x = inputs(gen, 3, torch.float16)
    step = cache.step(seqs, [1] * 3, room=40)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        y = blk(x, step)                          # workspaces are there before the capture
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = blk(x, step)
    for n in range(30):
        if n:
            step.start.copy_(cache.step(seqs, [1] * 3).start)
            x.copy_(inputs(gen, 3, torch.float16))
        g.replay()
        assert torch.equal(y, eager(x, twin.step(others, [1] * 3))), n
    assert blk.device_error() == R.BS_OK and eager.device_error() == R.BS_OK


def test_a_capture_needs_its_workspaces_first():
    gen = np.random.default_rng(9)
    cache = R.BitStackCache(HEADS, DIM, 24, 16)
    q = torch.zeros(1, Q_HEADS, DIM, dtype=torch.float16, device="cuda")
    step = cache.step([cache.open()], [1])
    blk = block(gen, cache)
    x = inputs(gen, 1, torch.float16)
    for call in (lambda: cache.attention(step, q), lambda: blk(x, step)):
        with pytest.raises(RuntimeError, match="captur"):
            with torch.cuda.graph(torch.cuda.CUDAGraph()):
                torch.zeros(1, device="cuda")     # a capture that is not empty
                call()
        torch.cuda.synchronize()
    cache.append(step, *torch.ones(2, 1, HEADS, DIM, dtype=torch.float16, device="cuda"))
    assert (cache.attention(step, q) == 1).all()


def test_refusals():
    gen = np.random.default_rng(10)
    with pytest.raises(R.BsError):
        R.BitStackCache(2, 96, 4)
    with pytest.raises(R.BsError):
        R.BitStackCache(2, 64, 4, layers=0)
    cache = R.BitStackCache(HEADS, DIM, 4, 16)
    blk = block(gen, cache)
    with pytest.raises(R.BsError):
        R.BitStackAttention(blk.q, blk.k, blk.q, blk.o, cache)
    with pytest.raises(R.BsError):
        R.BitStackAttention(blk.q, blk.k, blk.v, random_linear(D_MODEL, 256, gen), cache)
    with pytest.raises(IndexError):
        R.BitStackAttention(blk.q, blk.k, blk.v, blk.o, cache, layer=1)
    seq = cache.open()
    with pytest.raises(R.BsError):
        cache.step([seq], [65])
    step = cache.step([seq], [2])
    with pytest.raises(ValueError):
        blk(inputs(gen, 3, torch.float16), step)
    with pytest.raises(KeyError):
        cache.step([seq + 1], [1])
    nothing = cache.step([seq], [0])
    assert blk(inputs(gen, 0, torch.float16), nothing).shape == (0, D_MODEL)
