"""CPU: the tight check of cache attention accepts what the kernels' roundings give, and rejects planted mistakes, in every
case that it is used for on the GPU."""
import numpy as np
import pytest

from oracle import cache as oc
from tests import cache_check as cc


def rounded(x, dtype):
    """The result's type, as float64."""
    if dtype == "fp16":
        return x.astype(np.float16).astype(np.float64)
    w = x.astype(np.float32).view(np.uint32)
    return (w + 0x7fff + (w >> 16 & 1) & 0xffff0000).astype(np.uint32).view(np.float32).astype(np.float64)


def stand_in(made, fault=None):
    """What a kernel computes, in float64 with its roundings of weights, values and result, and one planted mistake."""
    out = np.full(made.q.shape, 7.0)
    lse = np.full(made.q.shape[:2], 7.0)
    for i, (row0, rows, start, live, _) in enumerate(made.spans):
        out[row0:row0 + rows], lse[row0:row0 + rows] = 0.0, -np.inf
        if not live:
            continue
        for h in range(made.heads):
            (c, s, b), (vc, vs, vb), ok = cc.unpack(made.pool, made.table[i], h, 0, start + rows)
            k, v = np.nan_to_num(cc.numbers(c, s, b)), np.nan_to_num(cc.numbers(vc, vs, vb))
            if fault == "one part of the keys":              # the remainder of s (c - 8) / 2 in fp16 left out
                k = np.nan_to_num(np.repeat(b, 32, -1) + 2 * (np.repeat(s, 32, -1) * (c - 8) / 2).astype(np.float16))
            if fault == "a code one off":
                k[:, 5] += np.repeat(s, 32, -1)[:, 5]
            if fault == "values of the next token":
                v = np.roll(v, 1, 0)
            v = v.astype(np.float16).astype(np.float64)
            pos = np.repeat(np.arange(start, start + rows), made.group)
            t = np.arange(start + rows)
            window = made.window - 1 if fault == "window one short" and made.window else made.window
            see = ok & (t <= pos[:, None])
            if fault == "own token dropped":
                see = ok & (t < pos[:, None])
            if window:
                see &= t > pos[:, None] - window
            q = made.q[row0:row0 + rows, h * made.group:(h + 1) * made.group].reshape(-1, made.dim).astype(np.float64)
            scale = made.scale * (1.01 if fault == "scale 1 % off" else 1.0)
            x = np.where(see, scale * (q @ k.T), -np.inf)
            some = see.any(1)
            m = np.where(some, x.max(1, initial=-np.inf), 0.0)
            p = np.exp(x - m[:, None])
            z = np.where(some, p.sum(1), 1.0)
            hi = (p * 128).astype(np.float16).astype(np.float64)
            if made.dtype == "fp16" and fault != "one part of the weights":
                hi = hi + (p * 128 - hi).astype(np.float16)
            o = hi @ v / 128 / z[:, None]
            at = np.s_[row0:row0 + rows, h * made.group:(h + 1) * made.group]
            out[at] = rounded(np.where(some[:, None], o, 0.0), made.dtype).reshape(out[at].shape)
            lse[at] = np.where(some, m + np.log(z), -np.inf).reshape(lse[at].shape).astype(np.float32)
    if fault == "zeros":
        out[:] = 0.0
    if fault == "lse in 11 bits":
        lse = lse.astype(np.float16).astype(np.float64)
    return out, lse


FAULTS = ("own token dropped", "scale 1 % off", "a code one off", "values of the next token", "zeros", "lse in 11 bits")


@pytest.mark.parametrize("name", cc.CASES)
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_the_check_accepts_the_roundings_and_rejects_mistakes(name, dtype):
    made = cc.Made(**cc.CASES[name], dtype=dtype, seed=len(name))
    assert made.check(*stand_in(made)) <= 1
    faults = list(FAULTS)
    if made.window:
        faults.append("window one short")
    if "chunk" in name:                                      # the kernel that has these parts
        faults.append("one part of the keys")
    for fault in faults:
        with pytest.raises(AssertionError, match="of the tolerance"):
            made.check(*stand_in(made, fault))
            print("accepted:", fault)              # shown if it was


@pytest.mark.parametrize("seed", range(4))
def test_the_check_rejects_one_part_of_an_fp16_rows_weights(seed):
    """(In the case whose rows have the fewest numbers a weight; elsewhere the result's own rounding is as large.)"""
    made = cc.Made(**cc.CASES["chunk64"], dtype="fp16", seed=seed)
    with pytest.raises(AssertionError, match="of the tolerance"):
        made.check(*stand_in(made, "one part of the weights"))
