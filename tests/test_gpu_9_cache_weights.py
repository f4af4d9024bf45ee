"""GPU: what the attention kernels of the packed cache make of small weights, of positions that nobody stored, and of
very large scores: exact constructions, whose results are known in closed form."""
import math

import numpy as np
import pytest
import torch

import residual_block_decomp_b200 as R

pytestmark = pytest.mark.gpu

HALF = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}   # half a step, relative
LOG2E = 1.4426950408889634


def pool_of(keys, values, heads, page, spare=1):
    """A pool that holds one sequence of constant rows: token t's numbers are keys[t] and values[t] (exact: a group of
    equal numbers is its fp16 base).  (handle, the sequence's pages, the store)."""
    dim, n = keys[1], len(keys[0])
    n_pages = -(-n // page) + spare
    store = torch.full((R.bs_cache_device_bytes(heads, dim, page, n_pages),), 0xff, dtype=torch.uint8, device="cuda")
    handle = R.bs_cache_create(heads, dim, page, n_pages, store)
    table = torch.arange(n_pages, dtype=torch.int32, device="cuda")[None]
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    k, v = (torch.as_tensor(x, dtype=torch.float16, device="cuda")[:, None, None].expand(n, heads, dim).contiguous()
            for x in (keys[0], values))
    R.bs_cache_append(handle, R.CacheStep(zero, table, n, n, cu), k, v)
    return handle, table, store


def attend(handle, step, q, scale, window=0):
    out = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda")
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    ws = torch.zeros(R.bs_cache_attention_workspace_bytes(handle, step, q.shape[1]), dtype=torch.uint8, device="cuda")
    R.bs_cache_attention(handle, step, q, out, ws, scale, window, lse)
    torch.cuda.synchronize()
    return out.double().cpu(), lse.double().cpu()


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("group", [2, 64])                # the kernel for few rows, and the one for many
def test_a_long_flat_tail_behind_one_large_score(group, dim, dtype):
    """One key whose score is `gap` (in powers of two) above that of all others, as an attention sink is; its value is 0
    and theirs are 1, so the result is the others' share.  A weight enters the product of the values in fp16 with the
    largest at 2^7 or above: half of the smallest step, 2^-25, is 2^-32 of the largest weight, and a bf16 row's
    weights are rounded once (2^-11).  A score is off by a few fp32 steps of itself.  The sum of the weights is off by half
    a step, 2^-24 of it, an addition to the lane's share that holds the large one: n / 16 additions (few rows), n / 128."""
    heads, n, seqs = 4, 20000, 64
    keys = np.zeros(n)
    keys[0] = 1.0
    values = np.ones(n)
    values[0] = 0.0
    handle, table, _ = pool_of((keys, dim), values, heads, 64)
    step = R.CacheStep(torch.full((seqs,), n - 1, dtype=torch.int32, device="cuda"), table.repeat(seqs, 1), seqs)
    q = torch.ones(seqs, heads * group, dim, dtype=dtype, device="cuda")
    for gap in (12.0, 23.7, 25.2, 27.6, 30.0):
        out, lse = attend(handle, step, q, gap / (dim * LOG2E))
        p = 2.0 ** -gap
        z = 1 + (n - 1) * p
        want = (n - 1) * p / z
        part = (gap * 8 * 2.0 ** -23 + (n / 8) * 2.0 ** -23) * want + (n - 1) * 2.0 ** -32 * 1.01 / z
        if dtype == torch.bfloat16:
            part += 2.0 ** -11 * want
        tol = part + HALF[dtype] * (want + part) + 2.0 ** -25
        err = (out - want).abs().max().item()
        assert err <= tol, (gap, want, err, tol)
        want_lse = gap * math.log(2) + math.log(z)
        assert (lse - want_lse).abs().max().item() <= 2.0 ** -20 * want_lse + n / (16 if group == 2 else 128) * 2.0 ** -24, gap
    R.bs_cache_destroy(handle)


def test_more_tiles_of_a_sequence_than_32_bits_count():
    """1024 heads of a context of 12.3 million tokens, 48 rows each: 4.7 10^9 tiles of 16 tokens.  Every page is the same
    one; keys are zeros, so the weights are equal, and a head's values are 1 or 2: all sums are exact.  (About 5 seconds.)"""
    heads, dim, group, page = 1024, 256, 48, 256
    n = 12_300_032
    assert n // 16 * heads * (group // 8) > 2 ** 32 + 2 ** 28 and n % page == 0
    handle, _, _ = pool_of((np.zeros(page), dim), np.zeros(page), heads, page, spare=0)
    level = 1.0 + torch.arange(heads, device="cuda") // 512
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    write = R.CacheStep(zero, zero[None], page, page, torch.tensor([0, page], dtype=torch.int32, device="cuda"))
    R.bs_cache_append(handle, write, torch.zeros(page, heads, dim, dtype=torch.float16, device="cuda"),
                      level.half()[None, :, None].expand(page, heads, dim).contiguous())
    step = R.CacheStep(torch.full((1,), n - 1, dtype=torch.int32, device="cuda"), torch.zeros(1, n // page, dtype=torch.int32, device="cuda"), 1)
    q = torch.randn(1, heads * group, dim, device="cuda").bfloat16()
    out, lse = attend(handle, step, q, 0.0625)
    assert R.bs_cache_get_device_error(handle) == R.BS_OK
    want = level.double().cpu().repeat_interleave(group)[None, :, None]
    assert torch.equal(out, want.expand_as(out))
    assert (lse - math.log(n)).abs().max().item() <= 2.0 ** -21 * math.log(n)
    R.bs_cache_destroy(handle)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("group", [2, 64])                # the kernel for few rows, and the one for many
def test_scores_of_any_size_that_fp32_holds(group, dim, dtype):
    """Keys and queries of up to 10^4, and bf16 queries of 10^9 and 10^20: scores of 10^8 to 10^25, whose fp32 steps are far
    larger than 1.  The largest score's value is the result wherever it is clear which that is.  A score is a sum of terms
    s (64 + c) q and (72 s - b) sum q, 79 s at most for each q, where 15 s is a group's range, so 10.6 times its largest
    number, with some 40 steps of 2^-23 of it in all: off by up to 2^-14 of sum |q| max |k|."""
    heads, n, page = 2, 60, 16
    gen = np.random.default_rng(dim + group)
    n_pages = n // page + 1
    store = torch.full((R.bs_cache_device_bytes(heads, dim, page, n_pages),), 0xff, dtype=torch.uint8, device="cuda")
    handle = R.bs_cache_create(heads, dim, page, n_pages, store)
    table = torch.arange(n_pages, dtype=torch.int32, device="cuda")[None]
    zero, cu = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.tensor([0, n], dtype=torch.int32, device="cuda")
    write = R.CacheStep(zero, table, n, n, cu)
    k, v = (torch.from_numpy(gen.standard_normal((n, heads, dim)).astype(np.float32) * s).cuda() for s in (5e3, 1.0))
    R.bs_cache_append(handle, write, k, v)
    R.bs_cache_read(handle, write, k, v)
    k, v = k.double().cpu(), v.double().cpu()
    for size in (1e4, 1.0) if dtype == torch.float16 else (1e4, 1e9, 1e20, 1.0):
        for sign in (1, -1):
            seqs = 40                                       # contexts of 1 to n tokens
            start = torch.arange(seqs, dtype=torch.int32) * (n - 1) // (seqs - 1)
            step = R.CacheStep(start.cuda(), table.repeat(seqs, 1), seqs)
            q = (torch.from_numpy(gen.standard_normal((seqs, heads * group, dim)).astype(np.float32)) * size).to(dtype)
            if sign < 0:                                    # every score far below zero
                q = q.abs() * -k.mean((0, 1)).sign().to(dtype)
            out, lse = attend(handle, step, q.cuda(), 1.0)
            clear = 0
            for i in range(seqs):
                x = torch.einsum("hgd,thd->hgt", q[i].double().view(heads, group, dim), k[:int(start[i]) + 1]).flatten(0, 1)
                top, at = x.max(-1)
                rest = x.clone()
                rest.scatter_(1, at[:, None], -math.inf)
                off = 2.0 ** -14 * q[i].double().abs().sum(-1) * k.abs().max()
                sure = top - rest.amax(-1) > 2 * off + 40
                want = v[at, torch.arange(heads).repeat_interleave(group)]
                err = (out[i] - want).abs()[sure] / (want.abs()[sure] * (HALF[dtype] + 2.0 ** -10) + 2.0 ** -25)
                assert err.numel() == 0 or err.max().item() <= 1, (size, sign, i)
                assert ((lse[i] - top).abs() <= off + 2.0 ** -21 * top.abs())[sure].all(), (size, sign, i)
                assert torch.isfinite(out[i]).all() and torch.isfinite(lse[i]).all()
                clear += int(sure.sum())
            assert clear > 0.9 * seqs * heads * group
    R.bs_cache_destroy(handle)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("group,seqs", [(4, 222), (9, 222), (64, 19)])     # one run of tiles a warp, and one a CTA
@pytest.mark.parametrize("n", [8192 + 256, 1 << 18])
def test_sums_over_long_runs_are_not_cut_short(dim, group, seqs, n):
    """Equal weights over n tokens that one run of tiles takes, values about 1 (a page of them, again and again).  A product
    cuts its terms at the accumulator's last place, 2^-28 of the sum a token at most as measured; a run's output is
    added up apart after 8192 tokens at most, with one rounding each.  The sum of equal weights is exact."""
    heads, page = 8, 256
    gen = np.random.default_rng(dim + group)
    handle, _, _ = pool_of((np.zeros(page), dim), np.zeros(page), heads, page, spare=0)
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    write = R.CacheStep(zero, zero[None], page, page, torch.tensor([0, page], dtype=torch.int32, device="cuda"))
    k = torch.zeros(page, heads, dim, device="cuda")
    R.bs_cache_append(handle, write, k, torch.from_numpy(gen.standard_normal((page, heads, dim)).astype(np.float32)).cuda() + 1)
    v = torch.empty_like(k)
    R.bs_cache_read(handle, write, None, v)
    v = v.half().double().cpu()                             # as it enters the product
    step = R.CacheStep(torch.full((seqs,), n - 1, dtype=torch.int32, device="cuda"),
                       torch.zeros(seqs, n // page, dtype=torch.int32, device="cuda"), seqs)
    q = torch.from_numpy(gen.standard_normal((seqs, heads * group, dim)).astype(np.float32)).half().cuda()
    out, lse = attend(handle, step, q, 0.1)
    want = v.mean(0).repeat_interleave(group, 0)[None]
    size = v.abs().mean(0).repeat_interleave(group, 0)[None]
    tol = size * (2.0 ** -28 * 8192 + n / 4096 * 2.0 ** -24 + 2.0 ** -22)
    tol = tol + HALF[torch.float16] * (want.abs() + tol) + 2.0 ** -25
    assert ((out - want).abs() <= tol).all(), float(((out - want).abs() / tol).max())
    assert (lse - math.log(n)).abs().max().item() <= 2.0 ** -21 * math.log(n)
    R.bs_cache_destroy(handle)


@pytest.mark.parametrize("group", [2, 64])
def test_a_row_whose_scores_pass_fp32_leaves_the_others_alone(group):
    heads, n, dim = 2, 60, 64
    gen = np.random.default_rng(group)
    handle, table, _ = pool_of((gen.standard_normal(n), dim), gen.standard_normal(n), heads, 16)
    step = R.CacheStep(torch.full((5,), n - 1, dtype=torch.int32, device="cuda"), table.repeat(5, 1), 5)
    q = torch.from_numpy(gen.standard_normal((5, heads * group, dim)).astype(np.float32)).bfloat16().cuda()
    clean, clean_lse = attend(handle, step, q, 0.5)
    for size in (1e38, -1e38, 3e38):
        wild = q.clone()
        wild[2, 1] = wild[3, -1] = size
        out, lse = attend(handle, step, wild, 0.5)
        rest = torch.ones(5, heads * group, dtype=torch.bool)
        rest[2, 1] = rest[3, -1] = False
        assert torch.equal(out[rest], clean[rest]) and torch.equal(lse[rest], clean_lse[rest])
    R.bs_cache_destroy(handle)
