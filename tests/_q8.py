"""Checks shared by the GPU tests of the 8-bit operators.

Codes decided from values that are exact in float32 (a checkpoint's h, gate, up; a
cache's V; weight * h of the row-scaled norm, one float32 rounding) must equal the
oracle's.  Where the kernel's value is itself a float32 result (a rotated K, a
gated unit), it may be off by ``win``; then a code must lie between the codes of
the exact value moved down and up by what that allows, rounding being monotone.
"""

import numpy as np
import torch

import oracle
from oracle import q8

CODE = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}


def codes64(t):
    """The codes as numbers."""
    return t.detach().float().cpu().numpy().astype(np.float64)


def check_exact(codes, scale, v64, fmt, what, group=None):
    c, s = q8.quantize(v64, fmt, group)
    got_c, got_s = codes64(codes), codes64(scale)
    assert got_c.shape == c.shape and got_s.shape == s.shape, (what, got_c.shape, c.shape)
    assert np.array_equal(got_s, s, equal_nan=True), f"{what}: {int((got_s != s).sum())} scales differ"
    bad = (got_c != c) & np.isfinite(q8.values(c, s, group))
    assert not bad.any(), f"{what}: {int(bad.sum())} codes differ, first at {tuple(np.argwhere(bad)[0])}"


def check_window(codes, scale, v64, win, fmt, what, max_ambiguous=4e-3):
    """win: how far the kernel's float32 value of each v64 may be off (absolute).  The group's
    maximum is then off by at most the largest of the group's windows, and code and scale
    by three more float32 roundings."""
    v = np.asarray(v64, dtype=np.float64)
    win = np.broadcast_to(np.asarray(win, dtype=np.float64), v.shape)
    a = np.maximum(np.abs(v).max(axis=-1), q8.AMAX_MIN)
    wa = win.max(axis=-1)
    s = codes64(scale)
    assert s.shape == a.shape, (what, s.shape, a.shape)
    assert (np.abs(s * q8.QMAX[fmt] - a) <= wa + 2.0 ** -23 * a).all(), f"{what}: scales off"
    t = v / a[..., None] * q8.QMAX[fmt]
    w = (win + np.abs(v) * (wa / a)[..., None]) / a[..., None] * q8.QMAX[fmt] + 2.0 ** -22 * np.abs(t)
    near = np.rint if fmt == "int8" else oracle.round_to_e4m3
    lo, hi = near(t - w), near(t + w)
    got = codes64(codes)
    bad = ~((got >= lo) & (got <= hi))
    assert not bad.any(), f"{what}: {int(bad.sum())} codes off, first at {tuple(np.argwhere(bad)[0])}"
    if lo.size >= 4096:  # too few codes say nothing about the rate
        assert (lo != hi).mean() <= max_ambiguous, f"{what}: {(lo != hi).mean():.2g} of the codes sit on a border"
