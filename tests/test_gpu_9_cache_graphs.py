"""GPU: the attention block in captured graphs beside eager calls of the same layers."""
import numpy as np
import pytest
import torch

import residual_block_decomp_b200 as R
from tests.test_gpu_9_cache_layer import DIM, HEADS, block, inputs

pytestmark = pytest.mark.gpu


def eager_of(blk, cache):
    return R.BitStackAttention(blk.q, blk.k, blk.v, blk.o, cache)


@pytest.mark.parametrize("rows", [3, 8])
def test_a_captured_block_outlives_larger_calls_of_its_layers(rows):
    """Eager calls that need larger workspaces replace them; the graph goes on with those that it was captured with."""
    gen = np.random.default_rng(21)
    cache, twin, other = (R.BitStackCache(HEADS, DIM, 40, 16) for _ in range(3))
    blk = block(gen, cache)
    same, larger = eager_of(blk, twin), eager_of(blk, other)
    step, step2 = cache.step([cache.open()], [rows]), twin.step([twin.open()], [rows])
    x = inputs(gen, rows, torch.float16)
    want = same(x, step2)
    blk(x, step)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = blk(x, step)
    large = inputs(gen, 300, torch.float16)
    larger(large, other.step([other.open()], [300]))
    cache.attention(cache.step([cache.open()], [200]), torch.zeros(200, 64, DIM, dtype=torch.float16, device="cuda"))
    torch.cuda.synchronize()
    junk = [torch.full((n,), 0x5a, dtype=torch.uint8, device="cuda") for n in [1 << k for k in range(9, 24)] * 4]
    for _ in range(3):
        y.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want)
    assert all((j == 0x5a).all() for j in junk)
    assert blk.device_error() == R.BS_OK


def test_a_refused_capture_leaves_the_layers_as_they_were():
    """Nothing ran before: the linears' workspaces would be made, and zeroed, inside the capture that the cache then refuses."""
    gen = np.random.default_rng(22)
    cache, twin = (R.BitStackCache(HEADS, DIM, 24, 16) for _ in range(2))
    blk = block(gen, cache)
    torch.full((1 << 24,), 0x5a, dtype=torch.uint8, device="cuda")   # freed at once: what the next allocations may hold
    step = cache.step([cache.open()], [8])
    x = inputs(gen, 8, torch.float16)
    with pytest.raises(RuntimeError, match="captur"):
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            blk(x, step)
    torch.cuda.synchronize()
    got = blk(x, step)
    q, k, v = (lin(x).view(8, -1, DIM) for lin in (blk.q, blk.k, blk.v))
    other = twin.step([twin.open()], [8])
    twin.append(other, k, v)
    assert torch.equal(got, blk.o(twin.attention(other, q).view(8, -1)))
    assert blk.device_error() == R.BS_OK and np.isfinite(got.float().cpu().numpy()).all()


def test_a_step_is_refused_during_a_capture():
    cache = R.BitStackCache(HEADS, DIM, 24, 16)
    seq = cache.open()
    with pytest.raises(RuntimeError, match="captur"):
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            torch.zeros(1, device="cuda")
            cache.step([seq], [5])
    torch.cuda.synchronize()
    assert cache.table.length[seq] == 0 and len(cache.table.free) == 24
    assert cache.step([seq], [5]).n_tokens == 5
