"""GPU: the bounded waits of the many-row kernel of cache attention.

The timeout is injected on the host: the call is told to leave out the first copy of its first CTA, with a 2 ms bound on each
wait.  The kernel records BS_ERR_TIMEOUT in the pool's error word, waits for its copies and products in flight, frees tensor
memory and returns; the context stays usable, which the next call shows.  Nothing here faults, traps or hangs the GPU."""
import pytest
import torch

import residual_block_decomp_b200 as R
from tests.test_gpu_9_cache import Case, check_attention

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("seqs", [[(0, 60)], [(3000, 60), (100, 40)]])     # one tile in all; runs of tiles, split items
def test_bounded_wait_times_out_and_context_survives(dim, seqs):
    c = Case(seqs, heads=2, dim=dim, page=64, seed=dim)
    c.fill()
    q = c.numbers(c.rows, 8, torch.bfloat16)
    want, want_lse = c.attend(q)
    ws = torch.zeros(R.bs_cache_attention_workspace_bytes(c.handle, c.step, 8), dtype=torch.uint8, device="cuda")
    out = torch.empty_like(q)
    R.bs_cache_debug_set_wait(c.handle, 2_000_000, unreachable_flag=True)
    R.bs_cache_attention(c.handle, c.step, q, out, ws)
    assert R.bs_cache_get_device_error(c.handle) == R.BS_ERR_TIMEOUT
    assert R.bs_cache_get_device_error(c.handle) == R.BS_OK          # the word was cleared by the read
    R.bs_cache_debug_set_wait(c.handle, 500_000_000, unreachable_flag=False)
    ws.zero_()
    for _ in range(2):
        out, lse = c.attend(q, ws=ws)
        assert R.bs_cache_get_device_error(c.handle) == R.BS_OK
        assert torch.equal(out, want) and torch.equal(lse, want_lse)
    check_attention(c, q, out, lse, sample=3)
    c.close()


def test_the_cache_zeroes_its_workspaces_after_a_timeout():
    cache = R.BitStackCache(2, 64, 40, 16)
    seq = cache.open()
    k, v, q = (torch.randn(200, h, 64, device="cuda").half() for h in (2, 2, 8))
    step = cache.step([seq], [200])
    cache.append(step, k, v)
    want = cache.attention(step, q)
    R.bs_cache_debug_set_wait(cache.handles[0], 2_000_000, unreachable_flag=True)
    cache.attention(step, q)
    assert cache.device_error() == R.BS_ERR_TIMEOUT
    R.bs_cache_debug_set_wait(cache.handles[0], 500_000_000, unreachable_flag=False)
    assert torch.equal(cache.attention(step, q), want) and cache.device_error() == R.BS_OK


def test_refusals():
    c = Case([(0, 3)], heads=1, dim=64, page=16, seed=1)
    for ns in (0, -1):
        with pytest.raises(R.BsError) as e:
            R.bs_cache_debug_set_wait(c.handle, ns)
        assert e.value.status == R.BS_ERR_INVALID_ARG
    c.close()
