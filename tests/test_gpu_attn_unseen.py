"""GPU: keys that a row does not see, pages outside the cache and rows whose reference moves in every step,
in each of the kernels of attention over the paged 8-bit cache.

The first test compares calls with one another, bit for bit: a row's result may depend on nothing that
the row does not see.  Where values are compared, the bounds are those of ``test_gpu_attn`` and, for
weights rounded to fp16 relative to the power of two R above the row's scales of V (R at most twice the
largest), half a step below fp16's normal range: 2^-25 / 2^13 of R for every key, times its code.
"""

import numpy as np
import pytest
import torch

import rmsnorm_fwd_bwd_03_gb300 as gb
from oracle import heads

from _checks import to64
from test_gpu_attn import F32_TERMS, _args, _check, _make

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module", autouse=True)
def _library():
    from rmsnorm_fwd_bwd_03_gb300._build import build_library
    build_library()
    gb.library()


def _place(s, b, j):
    page = s["cache"][0].shape[1]
    return int(s["table"][b, j // page]), j % page


def _call(s, **kw):
    lse = torch.zeros((s["T"], s["Hq"]), device="cuda")
    return gb.attn_cache8(*_args(s), lse=lse, **kw), lse


def _same(got, want, rows):
    return all(torch.equal(g[rows], w[rows]) for g, w in zip(got, want))


# heads of the kernel for few rows, of the one for many, of the one for any other
KINDS = [("bf16", 128, 8, 2, [3], [40]), ("bf16", 128, 8, 2, [2, 1, 4], [300, 7, 16]), ("bf16", 128, 2, 2, [5], [1000]),
         ("bf16", 64, 14, 2, [2], [90]), ("bf16", 96, 8, 2, [3, 2], [33, 130]), ("bf16", 256, 4, 2, [4], [70]),
         ("bf16", 128, 8, 2, [150], [400]), ("bf16", 64, 4, 1, [70, 90], [70, 300]), ("bf16", 80, 4, 2, [3, 40], [60, 90]),
         ("f32", 64, 4, 2, [5], [77])]


@pytest.mark.parametrize("window", [0, 20])
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("io,D,Hq,Hk,new,kv", KINDS)
def test_a_neighbours_key_changes_nothing(io, D, Hq, Hk, new, kv, fmt, window):
    """The last key of each sequence is seen by its last new token only, and with a window the first key
    of the first token's window by that token only: whatever its scales and codes are, no other row changes."""
    s = _make(new, kv, Hq, Hk, D, io=io, fmt=fmt)
    plain = _call(s, window=window)
    last = np.cumsum(new) - 1
    first = last - np.array(new) + 1
    edges = [(b, kv[b] - 1, last[b]) for b in range(len(new))]
    if window:
        edges += [(b, kv[b] - new[b] - window + 1, first[b]) for b in range(len(new)) if kv[b] - new[b] - window + 1 >= 0]
    changes = [(3, v) for v in (2.0 ** 25, 2.0 ** 32, 2.0 ** 40, 1e30, INF, -2.0 ** 40, NAN)] + [(1, v) for v in (INF, 2.0 ** 100, NAN)]
    for b, j, row in edges:
        page, off = _place(s, b, j)
        others = np.delete(np.arange(s["T"]), row)
        for tensor, value in changes:
            kept = s["cache"][tensor][page, off].clone()
            s["cache"][tensor][page, off] = value
            got = _call(s, window=window)
            s["cache"][tensor][page, off] = kept
            assert _same(got, plain, others), f"sequence {b} key {j}: {'K' if tensor == 1 else 'V'} scale {value}"
        # codes of NaN (E4M3) with a scale of NaN, as the cache's writers store a head that is not finite
        kept = [c[page, off].clone() for c in s["cache"]]
        for i in (0, 2):
            s["cache"][i].view(torch.uint8)[page, off] = 0x7f
            s["cache"][i + 1][page, off] = NAN
        got = _call(s, window=window)
        for c, k in zip(s["cache"], kept):
            c[page, off] = k
        assert _same(got, plain, others) and got[0][row].isnan().all()
        if fmt == "e4m3":  # such codes alone
            for i in (0, 2):
                codes = s["cache"][i].view(torch.uint8)[page, off]
                kept = codes.clone()
                codes.fill_(0xff)
                got = _call(s, window=window)
                codes.copy_(kept)
                assert _same(got, plain, others), f"sequence {b} key {j}: codes of NaN"
    assert _same(_call(s, window=window), plain, np.arange(s["T"]))
    assert gb.device_error() == 0


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("D,Hq,Hk,new,kv", [(128, 8, 2, [3], [200]), (256, 4, 2, [2, 3], [40, 90]), (64, 2, 2, [6], [300])])
def test_scales_of_v_far_apart(D, Hq, Hk, new, kv, fmt):
    """Scales of V from 2^-40 to 2^40 in one sequence, the largest seen by some rows only."""
    s = _make(new, kv, Hq, Hk, D, fmt=fmt)
    r = np.random.default_rng(3)
    for b, n in enumerate(kv):
        power = np.exp2(r.integers(-40, 20, n))
        power[-(new[b] - 1):] = 2.0 ** 40  # what the first new token does not see
        for j in range(n):
            s["cache"][3][_place(s, b, j)] *= float(power[j])
        s["values"][1][b] = s["values"][1][b] * power[:, None, None]
    out, _ = _call(s)
    got, q64, t = to64(out), to64(s["q"]), 0
    for b, (m, n) in enumerate(zip(new, kv)):
        k, v = s["values"][0][b], s["values"][1][b]
        o, _ = heads.attend(q64[t:t + m], k, v, D ** -0.5, n - m)
        a, _ = heads.attend(q64[t:t + m], k, np.abs(v), D ** -0.5, n - m)
        top = np.stack([np.abs(v[:n - m + i + 1]).max(axis=(0, 2)) for i in range(m)])  # [m, Hk]: qmax * the largest scale seen
        # each weight off by 2^-38 of R at most, R <= 2 * the largest scale = 2 * top / qmax (every head's largest code is the
        # format's largest, qmax), codes at most qmax, the weights' sum at least 1 (the largest weight's): 2^-37 top a key
        lost = 2.0 ** -37 * n * np.repeat(top, Hq // Hk, axis=1)[..., None]
        bad = np.abs(got[t:t + m] - o) > 2.0 ** -8 * np.abs(o) + (2.0 ** -8 * (1 + 2.0 ** -8) + F32_TERMS) * a + lost
        assert not bad.any(), f"sequence {b}: {int(bad.sum())} off, first at {tuple(np.argwhere(bad)[0])}"
        t += m


@pytest.mark.parametrize("D,Hq,Hk,new,kv", [(128, 8, 2, [150, 30], [300, 40]), (64, 4, 2, [200], [200]), (128, 8, 2, [2, 1], [300, 40]), (80, 4, 2, [20, 3], [300, 40])])
def test_any_entry_outside_the_cache_is_reported(D, Hq, Hk, new, kv):
    s = _make(new, kv, Hq, Hk, D)
    plain = _call(s)
    pages = s["cache"][0].shape[0]
    assert gb.device_error() == 0
    for column in (3, (kv[0] - 1) // 16):  # in the middle, and the last page
        kept = int(s["table"][0, column])
        for bad in (-1, pages, -2 ** 31, 2 ** 31 - 1, -2 ** 31 + 1):
            s["table"][0, column] = bad
            got = _call(s)
            assert gb.device_error(clear=True) == gb.ERR_BAD_SLOT, bad
            see = torch.arange(new[0], device="cuda") + kv[0] - new[0] >= 16 * column
            assert got[0][:new[0]][see].isnan().all(), bad
            others = torch.cat([torch.nonzero(~see).flatten(), torch.arange(new[0], s["T"], device="cuda")])
            assert _same(got, plain, others), bad
        s["table"][0, column] = kept


@pytest.mark.parametrize("D,new,kv", [(128, [130, 70], [700, 200]), (64, [300], [900]), (96, [64], [500])])
def test_references_that_move_in_every_step(D, new, kv):
    """Scores that rise by up to 9 from one 64 keys to the next (another rise for every third row): rows whose
    weights are computed anew beside rows whose are not."""
    s = _make(new, kv, 4, 2, D)
    r = np.random.default_rng(1)
    s["q"][:] = (torch.arange(s["T"], device="cuda") % 3 / 2).to(torch.bfloat16)[:, None, None]
    for b, n in enumerate(kv):
        scale = ((9.0 * (np.arange(n) // 64) + r.random(n)) / (127 * D ** 0.5)).astype(np.float32)
        for j in range(n):
            at = _place(s, b, j)
            s["cache"][0][at] = 127
            s["cache"][1][at] = float(scale[j])
        s["values"][0][b] = np.broadcast_to(127.0 * scale.astype(np.float64)[:, None, None], s["values"][0][b].shape)
    out, lse = _call(s)
    # scores up to 130 here (188 in powers of two), sums of D equal products, exact; then five roundings of scales and
    # products: 5 * 2^-24 * 188 = 2^-14 in a weight's exponent, below the bound's 2^-11
    _check(s, out, lse)
    for _ in range(3):
        again = _call(s)
        assert torch.equal(again[0], out) and torch.equal(again[1], lse)
