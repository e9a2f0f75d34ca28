"""Helpers of the tests of the transformer block's operators.

Tolerances: a bf16 result is rounded once, by at most 2^-8 of its value (half a
step; below the normal range half of 2^-133); float32 arithmetic in front of it,
and float32 results, may lose LOST of the sum of the magnitudes of the terms (the
oracle gives it).  The longest chain of float32 roundings in the tests' rows of up
to 16384 values is 16 or 32 values a thread, 10 additions between threads and waves
and about 12 operations around the statistics, which enter twice (two norms one
after the other): below 128 half steps of 2^-24, so LOST = 2^-17.
"""

import numpy as np
import torch

from oracle import e4m3, moe
from tests.gpu_util import bf16_to_f64, dev, host

LOST = 2.0 ** -17
FILL = 0x5A        # what unwritten codes keep
UNWRITTEN = -3.0   # and unwritten scales
SENTINEL = 0x7FC1  # a bf16 NaN that no kernel writes


def padded(bits, pad):
    """Device matrix of bf16 bits inside one with `pad` more columns, which hold NaN."""
    t = dev(np.pad(bits, ((0, 0), (0, pad)), constant_values=0x7FC0))
    return t[:, :bits.shape[1]]


def empty_rows(rows, cols, pad=0):
    return torch.full((rows, cols + pad), SENTINEL, dtype=torch.int16, device="cuda")[:, :cols]


def pads_kept(t):
    """Whether the columns behind a view of empty_rows() are as they were."""
    whole = t._base if t._base is not None else t
    return bool((whole[:, t.shape[1]:] == SENTINEL).all())


def f32(v):
    return None if v is None else torch.as_tensor(np.asarray(v, dtype=np.float32), device="cuda")


def check_rows(got, want, mag, what):
    """bf16 results."""
    got = bf16_to_f64(host(got))
    bound = 2.0 ** -8 * np.abs(want) + LOST * mag + 2.0 ** -134
    bad = ~(np.abs(got - want) <= bound)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size}, worst {np.max(np.abs(got - want) / bound):.3f}, first at {np.argwhere(bad)[0]}"


def check_f32(got, want, mag, what, lost=LOST):
    got = host(got).astype(np.float64)
    bad = ~(np.abs(got - want) <= 2.0 ** -24 * np.abs(want) + lost * mag + 2.0 ** -149)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size}, first at {np.argwhere(bad)[0]}, {got[bad][0]} for {np.broadcast_to(want, got.shape)[bad][0]}"


def check_scales(got, amax, mag, what):
    """float32 scales amax / 448 (at least 2^-126, 0 for a tile of zeros), with what amax may be off by."""
    want = np.where(amax > 0, np.maximum(amax / 448.0, 2.0 ** -126), 0.0)
    off = np.abs(got.astype(np.float64) - want)
    bad = ~(off <= 2.0 ** -22 * want + LOST * mag / 448.0)
    assert not bad.any(), f"{what}: {bad.sum()} scales, first at {np.argwhere(bad)[0]}"


def check_exponents(got, amax, mag, what):
    """UE8M0 exponents ceil(log2(amax / 448)) + 127; next to a power of two either one."""
    low, high = np.maximum(amax - LOST * mag, 0.0), amax + LOST * mag

    def exponent(v):
        with np.errstate(divide="ignore"):
            return np.where(v > 0, np.clip(np.ceil(np.log2(np.where(v > 0, v, 1.0) / 448.0)), -127, 127) + 127, 0)

    got = got.astype(np.int64)
    bad = ~((got >= exponent(low * (1 - 2.0 ** -22))) & (got <= exponent(high * (1 + 2.0 ** -22))))
    assert not bad.any(), f"{what}: {bad.sum()} exponents, first at {np.argwhere(bad)[0]}"


def check_codes(q, s, v, mag, what):
    """Codes q with the scales s that came with them (one a value) against v: nearest e4m3 numbers of v / s but
    for what v may be off by (2^-20 for the quotient)."""
    q = e4m3.decode(q).astype(np.float64)
    t = v / np.where(s > 0, s, 1.0)
    off = (2.0 ** -20 * np.abs(v) + LOST * mag) / np.where(s > 0, s, 1.0)
    near = np.minimum(np.abs(t), 448.0)
    bad = ~(np.abs(q - np.clip(t, -448.0, 448.0)) <= moe.half_step(near + off) + off)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} codes, first at {np.argwhere(bad)[0]}"


def check_row_codes(q, sf, v, mag, ue8m0, what):
    """Row-wise codes q [R][C] and scales sf [C/128][ld]; scales past the rows unwritten."""
    q, sf = host(q), host(sf)
    rows = len(v)
    amax = np.abs(v).reshape(rows, -1, 128).max(2).T
    top = mag.reshape(rows, -1, 128).max(2).T
    if ue8m0:
        assert np.all(sf[:, rows:] == FILL)
        check_exponents(sf[:, :rows], amax, top, what)
        s = np.exp2(sf[:, :rows].astype(np.float64) - 127)
    else:
        assert np.all(sf[:, rows:] == UNWRITTEN)
        check_scales(sf[:, :rows], amax, top, what)
        s = sf[:, :rows].astype(np.float64)
    check_codes(q, np.repeat(s.T, 128, axis=1), v, mag, what)


def code_buffers(rows, cols, ld, ue8m0=False):
    q = torch.full((rows, cols), FILL, dtype=torch.uint8, device="cuda")
    if ue8m0:
        return q, torch.full((cols // 128, ld), FILL, dtype=torch.uint8, device="cuda")
    return q, torch.full((cols // 128, ld), UNWRITTEN, device="cuda")


def workspace(size, fill=0xA5):
    return torch.full((max(16, size),), fill, dtype=torch.uint8, device="cuda")
