"""Per-head RMSNorm of Q and K, rotary embedding with several position axes, and attention
over cached keys and values: the definitions, in numpy float64.

TEST INFRASTRUCTURE ONLY, like the rest of this package; it shares nothing with the CUDA
library.  Operators: "Fast-LLM: 高效大语言模型训练框架", §三 框架结构 (attention with RoPE) and
训练配置示例 (rms_norm, rotary).
"""

from __future__ import annotations

import numpy as np


def _angles(pos, axis, theta, D):
    """Angle of every token's pairs [T, 1, D / 2]: pos [n, T], axis [D / 2]."""
    f = theta ** (-2.0 * np.arange(D // 2) / D)
    return (np.asarray(pos, dtype=np.float64)[np.asarray(axis)].T * f)[:, None, :]


def rotate(x, pos, axis, theta, pairing="half", back=False):
    """Heads x [T, H, D], pair i of each turned by pos[axis[i]] * theta^(-2i/D) (or back)."""
    x = np.asarray(x, dtype=np.float64)
    D = x.shape[-1]
    a = _angles(pos, axis, theta, D) * (-1.0 if back else 1.0)
    one, two = (slice(0, D // 2), slice(D // 2, D)) if pairing == "half" else (slice(0, D, 2), slice(1, D, 2))
    out = np.empty_like(x)
    out[..., one] = x[..., one] * np.cos(a) - x[..., two] * np.sin(a)
    out[..., two] = x[..., two] * np.cos(a) + x[..., one] * np.sin(a)
    return out


def norm_rotate(x, w, pos, axis, theta, eps, pairing="half"):
    """Every head of x [T, H, D] divided by sqrt(mean square + eps), times w [D], rotated."""
    x = np.asarray(x, dtype=np.float64)
    r = 1.0 / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps)
    return rotate(x * r * np.asarray(w, dtype=np.float64), pos, axis, theta, pairing)


def norm_rotate_bwd(dy, x, w, pos, axis, theta, eps, pairing="half"):
    """Gradients ``(dx, dw)`` of sum(dy * norm_rotate(x, w, ...)).  The rotation's transpose is the
    rotation back; with d its result, g = d w, n = x r: dx = r (g - n mean(g n)), dw = sum d n."""
    x = np.asarray(x, dtype=np.float64)
    w = np.asarray(w, dtype=np.float64)
    d = rotate(dy, pos, axis, theta, pairing, back=True)
    r = 1.0 / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps)
    n, g = x * r, d * w
    return r * (g - n * np.mean(g * n, axis=-1, keepdims=True)), np.sum(d * n, axis=(0, 1))


def attend(q, k, v, scale, first, causal=True, window=0):
    """Attention of the rows q [m, H, D] over keys and values [n, Hk, D]: row i stands at position
    first + i and sees the keys j <= its position (causal) with j > position - window (window > 0).
    Returns ``(o [m, H, D], lse [m, H])``; a row that sees nothing gives zeros and -inf."""
    q, k, v = (np.asarray(t, dtype=np.float64) for t in (q, k, v))
    m, H, D = q.shape
    n, Hk = k.shape[:2]
    o, lse = np.zeros((m, H, D)), np.full((m, H), -np.inf)
    p = first + np.arange(m)[:, None]
    j = np.arange(n)[None]
    seen = np.ones((m, n), dtype=bool)
    if causal:
        seen &= j <= p
    if window:
        seen &= j > p - window
    rows = seen.any(axis=1)
    for h in range(H):
        kv = h // (H // Hk)
        with np.errstate(invalid="ignore"):
            s = np.where(seen, scale * (q[:, h] @ k[:, kv].T), -np.inf)[rows]
        if not s.size:
            continue
        top = s.max(axis=1, keepdims=True)
        e = np.exp(s - top)
        z = e.sum(axis=1, keepdims=True)
        # a value that a row does not see has no part in it, whatever it holds
        with np.errstate(invalid="ignore"):
            part = np.where(seen[rows][..., None], (e / z)[..., None] * v[None, :, kv], 0.0).sum(axis=1)
        o[rows, h], lse[rows, h] = part, (top + np.log(z))[:, 0]
    return o, lse
