"""8-bit storage with float32 scales: the definition, in numpy.

TEST INFRASTRUCTURE ONLY, like the rest of this package; it shares nothing with
the CUDA library.  A group of values v shares one float32 scale:

    a = max(max |v|, 2**-100);  code = nearest(v * (qmax / a));  scale = a / qmax

with qmax = 127 and integer codes (INT8) or qmax = 448 and E4M3 codes, ties to even.
Each of these operations is a float32 operation rounded to nearest: the roundings
are part of the definition, because they decide a code next to a border, so this
one function works in numpy's float32 (whose elementary operations are IEEE's).
Everything around it is float64.
"""

from __future__ import annotations

import numpy as np

from . import act, round_io, round_to_e4m3

QMAX = {"int8": 127.0, "e4m3": 448.0}
AMAX_MIN = 2.0 ** -100
CKPT_GROUP = 128


def _one_group(v, fmt):
    v = np.asarray(v, dtype=np.float64).astype(np.float32)
    q = np.float32(QMAX[fmt])
    amax = np.max(np.abs(v), axis=-1, keepdims=True)  # NaN if any value is NaN
    a = np.maximum(amax, np.float32(AMAX_MIN))
    with np.errstate(invalid="ignore", over="ignore"):
        t = (v * (q / a)).astype(np.float64)
        codes = np.rint(t) if fmt == "int8" else round_to_e4m3(t)
        scale = np.where(np.isfinite(amax), a / q, np.float32(np.nan))
    return codes, scale[..., 0].astype(np.float64)


def quantize(v, fmt, group=None):
    """Codes (as numbers) of float32 values v [..., N] and the scales [..., ceil(N / group)] of
    its groups of consecutive values (group None: the whole last axis, scales [...])."""
    v = np.asarray(v, dtype=np.float64)
    if group is None:
        return _one_group(v, fmt)
    parts = [_one_group(v[..., j:j + group], fmt) for j in range(0, v.shape[-1], group)]
    return np.concatenate([p[0] for p in parts], axis=-1), np.stack([p[1] for p in parts], axis=-1)


def values(codes, scale, group=None):
    """code * scale."""
    scale = np.asarray(scale, dtype=np.float64)
    if group is None:
        return codes * scale[..., None]
    return codes * np.repeat(scale, group, axis=-1)[..., :codes.shape[-1]]


def rmsnorm_fwd_fp8(x, residual, weight, eps, io=None):
    """``(codes, scale, y, h, rstd)``: the row-scaled E4M3 output of the RMSNorm forward.
    With u = weight * h in float32, codes = E4M3 of u * (448 / max|u|) and
    scale = max|u| * rstd / 448; y is the exact output."""
    x = np.asarray(x, dtype=np.float64)
    w = np.asarray(weight, dtype=np.float64)
    h = x if residual is None else round_io(x + np.asarray(residual, dtype=np.float64), io)
    rstd = 1.0 / np.sqrt(np.mean(h * h, axis=-1) + eps)
    u = (h.astype(np.float32) * w.astype(np.float32)).astype(np.float64)
    codes, _ = quantize(u, "e4m3")
    scale = np.maximum(np.max(np.abs(u), axis=-1), AMAX_MIN) * rstd / QMAX["e4m3"]
    return codes, scale, w * h * rstd[..., None], h, rstd


def rmsnorm_bwd_kept(dy, dres, kept, weight, rstd):
    """``(dx, dw)`` of the RMSNorm backward that has ``kept`` in the place of h, and the
    forward's rstd: n = kept * rstd, dx = rstd * (dy w - n mean(dy w n)) + dres, dw = sum dy n."""
    dy, w = np.asarray(dy, dtype=np.float64), np.asarray(weight, dtype=np.float64)
    n = np.asarray(kept, dtype=np.float64) * rstd[..., None]
    g = dy * w
    dx = rstd[..., None] * (g - n * np.mean(g * n, axis=-1)[..., None])
    if dres is not None:
        dx = dx + np.asarray(dres, dtype=np.float64)
    return dx, np.sum(dy * n, axis=0)


def glu_out(name, gate, up):
    """f(gate) * up."""
    return act(name, np.asarray(gate, dtype=np.float64)) * np.asarray(up, dtype=np.float64)
