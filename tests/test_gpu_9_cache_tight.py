"""GPU: attention over the packed cache within the roundings that its kernels are allowed (tests/cache_check.py), few query
rows a head and many, all head sizes, both types, with masks, peaked scores and long contexts."""
import numpy as np
import pytest
import torch

import residual_block_decomp_b200 as R
from tests import cache_check as cc
from tests.test_gpu_9_cache import Case

pytestmark = pytest.mark.gpu

TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}


def attend(made):
    """(out, lse) in float64 of a cc.Made step, its pool's bytes on the GPU as the oracle made them."""
    pool = made.pool
    nbytes = R.bs_cache_device_bytes(pool.heads, pool.dim, pool.page_tokens, pool.n_pages)
    store = torch.zeros(nbytes, dtype=torch.uint8, device="cuda")
    store[:len(pool.data)] = torch.from_numpy(pool.data).cuda()
    handle = R.bs_cache_create(pool.heads, pool.dim, pool.page_tokens, pool.n_pages, store)
    start, table, cu = (torch.from_numpy(a).cuda() for a in (made.start, made.table, made.cu))
    step = R.CacheStep(start, table, made.rows, made.max_new, cu)
    q = torch.from_numpy(made.q).cuda().to(TYPES[made.dtype])
    assert np.array_equal(q.float().cpu().numpy(), made.q)
    out = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda")
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    ws = torch.zeros(R.bs_cache_attention_workspace_bytes(handle, step, q.shape[1]), dtype=torch.uint8, device="cuda")
    R.bs_cache_attention(handle, step, q, out, ws, made.scale, made.window, lse)
    assert R.bs_cache_get_device_error(handle) == R.BS_OK
    R.bs_cache_destroy(handle)
    return out.double().cpu().numpy(), lse.double().cpu().numpy()


@pytest.mark.parametrize("name", cc.CASES)
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_within_the_roundings(name, dtype):
    for seed in (0, 1):
        made = cc.Made(**cc.CASES[name], dtype=dtype, seed=10 * len(name) + seed)
        used = made.check(*attend(made))
        print(f"{name} {dtype}: {used:.3f} of the tolerance")


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("new,group", [(1, 4), (1, 9), (3, 20), (140, 2)])
def test_long_and_many(dim, new, group):
    """One context over all SMs, and sequences by the dozen."""
    made = cc.Made([(9000, new)], heads=1, dim=dim, group=group, page=64, dtype="fp16", seed=new)
    made.check(*attend(made), sample=4)
    made = cc.Made([(7 * i - 1, new) for i in range(70)], heads=2, dim=dim, group=group, page=16, dtype="bf16", seed=dim)
    made.check(*attend(made), sample=2)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("new", [1, 5, 70])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_only_the_windows_tokens_are_stored(dim, new, dtype):
    """Positions that the window hides from every row hold NaN scales, also those in the same chunk as the first that is
    seen: few rows and many, contexts whose windows begin at each place of a chunk."""
    window = 20
    seqs = [(100 + i, new) for i in range(16)] + [(19, new), (20, new), (5, new), (16 * 40 + 3, new)]
    made = cc.Made(seqs, dim=dim, page=16, window=window, dtype=dtype, seed=dim + new, stored=[max(0, s - window + 1) for s, _ in seqs])
    made.check(*attend(made))


@pytest.mark.parametrize("new", [2, 60])
def test_rows_outside_the_tensors_are_an_empty_slots(new):
    """A sequence whose rows begin before 0, end behind the last one, run backwards or lie far out: those inside the tensors
    are attended and read as zeros, the others' results are as without it, nothing else is written."""
    c = Case([(40, new), (50, new), (10, new)], heads=2, dim=64, page=16, seed=new, spare_rows=3)
    c.fill()
    q = c.numbers(c.rows, 8, torch.float16)
    good, good_lse = c.attend(q)
    cu = c.cu.copy()
    for change, zero in [((0, -5), [(0, new)]), ((3, c.rows + 9), [(2 * new, c.rows)]), ((0, -2 ** 31), [(0, new)]),
                         ((3, 2 ** 31 - 1), [(2 * new, c.rows)]), ((3, 2 * new - 1), []), ((0, new + 1), [])]:
        c.cu = cu.copy()
        c.cu[change[0]] = change[1]
        step = c.make_step()
        out, lse = c.attend(q, step=step)
        assert R.bs_cache_get_device_error(c.handle) == R.BS_ERR_RANGE, change
        k = torch.full((c.rows, 2, 64), 7.0, device="cuda")
        v = k.clone()
        R.bs_cache_read(c.handle, step, k, v)
        assert R.bs_cache_get_device_error(c.handle) == R.BS_ERR_RANGE, change
        bad = 0 if change[0] == 0 else 2                      # the sequence that is an empty slot
        rest = torch.ones(c.rows, dtype=torch.bool, device="cuda")
        rest[bad * new:(bad + 1) * new if bad == 0 else c.rows] = False
        rest[3 * new:] = False
        assert torch.equal(out[rest], good[rest]) and torch.equal(lse[rest], good_lse[rest]), change
        assert (k[rest] != 7).any(2).all()
        for a, b in zero:
            assert (out[a:b] == 0).all() and (lse[a:b] == -np.inf).all() and (k[a:b] == 0).all() and (v[a:b] == 0).all(), change
        if not zero:
            rows = slice(bad * new, (bad + 1) * new)
            assert (out[rows] == 7).all() and (lse[rows] == 7).all() and (k[rows] == 7).all(), change
        before = c.store.clone()
        R.bs_cache_append(c.handle, step, k, v)
        torch.cuda.synchronize()
        assert R.bs_cache_get_device_error(c.handle) == R.BS_ERR_RANGE, change
        pages = torch.ones(c.n_pages, dtype=torch.bool, device="cuda")
        pages[torch.from_numpy(np.unique(np.delete(c.table, bad, 0))).long().cuda()] = False
        size = R.bs_cache_page_bytes(2, 64, 16)
        now, was = (x[:c.n_pages * size].view(c.n_pages, size) for x in (c.store, before))
        assert torch.equal(now[pages], was[pages]), change    # the empty slot's pages are as they were
        c.store.copy_(before)
    c.close()
