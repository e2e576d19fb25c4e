"""GPU vs oracle: attention of the new tokens of a ragged batch over the paged 8-bit cache.

Bounds, derived.  bf16 rows: the result is rounded to bf16 (half a step, by the eps / 2 rule:
finfo(bf16).eps / 2 = 2^-8) and every weight times v's scale once to bf16 (2^-8 of the weight at
most), so that with w_j the normalised weights
    |err| <= 2^-8 |o| + 2^-8 sum_j w_j |v_j| (1 + 2^-8) + float32 terms.
The scores are float32 sums of exact products: off by at most (D + 3) 2^-24 sum |q||k| scale, which
changes a weight by that relative amount, and 2^-21 for the exponential: D = 512 and scores of
magnitude 16 stay below 2^-11.  float32 rows: the same terms without bf16, in all below 2^-17 of
sum_j w_j |v_j| for the scores here (below 16, D up to 512: 515 * 2^-24 * 16 = 2^-10.9 in the worst case of
one sign; the sums here are of random signs, sqrt(512) terms: 2^-15.5, so 2^-14 is taken).
"""

import numpy as np
import pytest
import torch

import rmsnorm_fwd_bwd_03_gb300 as gb
from oracle import heads, q8

from _checks import to64
from _q8 import CODE, codes64

pytestmark = pytest.mark.gpu

IO = {"f32": torch.float32, "bf16": torch.bfloat16}
F32_TERMS = 2.0 ** -11


@pytest.fixture(scope="module", autouse=True)
def _library():
    from rmsnorm_fwd_bwd_03_gb300._build import build_library
    build_library()
    gb.library()


def _make(new, kv, Hq, Hk, D, io="bf16", fmt="int8", page=16, layout="NHD", pad=0, off=0, seed=0, extra_cols=2):
    """A batch: q, its offsets and lengths, page table, caches (scattered pages, junk everywhere else)."""
    r = np.random.default_rng(seed + sum(new) + 7 * sum(kv) + D)
    B, T = len(new), int(sum(new)) + pad
    q = torch.from_numpy(r.normal(size=(T, Hq * D + off)).astype(np.float32)).cuda().to(IO[io])[:, off:].unflatten(1, (Hq, D))
    need = [-(-n // page) for n in kv]
    pages = sum(need) + 3
    order = r.permutation(pages)
    table = np.full((B, max(need + [0]) + extra_cols), -1, np.int32)
    table[:, -1:] = 2 ** 31 - 1  # never to be read
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    ctx = [(r.normal(size=(n, Hk, D)), r.normal(size=(n, Hk, D))) for n in kv]
    cache, values = [], []
    for i in range(2):
        codes = np.full((pages, page, Hk, D), 0x7f, np.uint8)  # E4M3: NaN codes
        scale = np.full((pages, page, Hk), np.nan, np.float32)
        kept = []
        for b, n in enumerate(kv):
            c, s = q8.quantize(ctx[b][i], fmt)
            j = np.arange(n)
            p = table[b, j // page] if n else j
            t = torch.from_numpy(c).to(CODE[fmt]) if fmt == "int8" else torch.from_numpy(c.astype(np.float32)).to(CODE[fmt])
            codes[p, j % page] = t.view(torch.uint8).numpy()
            scale[p, j % page] = s
            kept.append(q8.values(c, s))
        codes, scale = torch.from_numpy(codes).cuda().view(CODE[fmt]), torch.from_numpy(scale).cuda()
        if layout == "HND":
            codes, scale = codes.transpose(1, 2).contiguous().transpose(1, 2), scale.transpose(1, 2).contiguous().transpose(1, 2)
        cache += [codes, scale]
        values.append(kept)
    cu = torch.from_numpy(np.concatenate([[0], np.cumsum(new)]).astype(np.int32)).cuda()
    return dict(q=q, cu=cu, kv=torch.tensor(kv, dtype=torch.int32, device="cuda"), table=torch.from_numpy(table).cuda(), cache=cache,
                values=values, new=list(new), lens=list(kv), io=io, pad=pad, T=T, Hq=Hq, D=D)


def _args(s):
    return (s["q"], s["cu"], s["kv"], s["table"], *s["cache"])


def _check(s, out, lse=None, what="", scale=None, causal=True, window=0):
    scale = s["D"] ** -0.5 if scale is None else scale
    got, t = to64(out), 0
    q64 = to64(s["q"])
    eps = 2.0 ** -8 if s["io"] == "bf16" else 2.0 ** -24
    for b, (m, n) in enumerate(zip(s["new"], s["lens"])):
        k, v = s["values"][0][b], s["values"][1][b]
        o, z = heads.attend(q64[t:t + m], k, v, scale, n - m, causal, window)
        a, _ = heads.attend(q64[t:t + m], k, np.abs(v), scale, n - m, causal, window)
        terms = eps * (1 + 2.0 ** -8) + F32_TERMS if s["io"] == "bf16" else 2.0 ** -14
        bad = np.abs(got[t:t + m] - o) > eps * np.abs(o) + terms * a + 1e-30
        assert not bad.any(), f"{what} sequence {b} ({m} of {n}): {int(bad.sum())} off, first at {tuple(np.argwhere(bad)[0])}"
        assert np.isfinite(got[t:t + m]).all()
        if lse is not None:
            l64 = to64(lse)[t:t + m]
            none = np.isneginf(z)
            assert np.array_equal(np.isneginf(l64), none)
            # scores in float32 as above (absolute, as they stand in the exponent), the sum and its logarithm 2^-21
            assert (np.abs(l64[~none] - z[~none]) <= F32_TERMS + 2.0 ** -20 * np.abs(z[~none])).all(), what + " lse"
        t += m


def _run(new, kv, Hq, Hk, D, causal=True, window=0, scale=None, **kw):
    s = _make(new, kv, Hq, Hk, D, **kw)
    out = torch.full((s["T"], Hq, D), 7.0, dtype=s["q"].dtype, device="cuda")
    lse = torch.full((s["T"], Hq), 7.0, device="cuda")
    got = gb.attn_cache8(*_args(s), out=out, lse=lse, causal=causal, window=window, scale=scale)
    assert got is out
    what = f"{new} of {kv}, {Hq}/{Hk}x{D} {kw} causal={causal} window={window}"
    _check(s, out, lse, what, scale, causal, window)
    n = s["T"] - s["pad"]
    assert (out[n:] == 7).all() and (lse[n:] == 7).all(), what + ": rows behind the last sequence changed"
    assert gb.device_error() == 0
    return s


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("io,D,Hq,Hk", [("bf16", 128, 32, 8), ("bf16", 64, 14, 2), ("bf16", 96, 8, 1), ("bf16", 256, 4, 2), ("bf16", 128, 3, 3),
                                        ("bf16", 80, 4, 2), ("bf16", 72, 2, 1), ("bf16", 33, 3, 1), ("f32", 64, 14, 2), ("f32", 128, 4, 1),
                                        ("f32", 512, 2, 1), ("bf16", 1, 2, 2)])
def test_head_sizes_and_formats(io, D, Hq, Hk, fmt):
    _run([1], [1], Hq, Hk, D, io=io, fmt=fmt)
    _run([1, 1, 3, 1], [300, 17, 3, 129], Hq, Hk, D, io=io, fmt=fmt, pad=2)
    _run([5, 40], [70, 40], Hq, Hk, D, io=io, fmt=fmt, layout="HND", page=5)


@pytest.mark.parametrize("G", [1, 2, 4, 5, 7, 8, 16, 17, 48])
def test_groups(G):
    _run([1, 1, 2, 7], [33, 500, 90, 7], 2 * G, 2, 64, pad=1)
    _run([70], [200], G, 1, 128)


@pytest.mark.parametrize("page", [1, 3, 16, 48, 64, 256])
@pytest.mark.parametrize("layout", ["NHD", "HND"])
def test_pages(page, layout):
    _run([1, 2, 1], [1000, 77, 256], 8, 2, 128, page=page, layout=layout)
    _run([150, 1], [400, 33], 8, 2, 128, page=page, layout=layout, fmt="e4m3")


@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 31, 127, 128, 129, 255, 256, 257, 1023, 4097, 20011])
def test_lengths(n):
    _run([1], [n], 8, 2, 128)
    _run([min(n, 9)], [n], 8, 2, 64, fmt="e4m3")
    if n < 2000:
        _run([n], [n], 4, 1, 128, fmt="e4m3")
        _run([n, 1, n], [n + 5, 200, n], 2, 2, 64)


@pytest.mark.parametrize("new,kv", [([0, 0, 1, 0], [0, 50, 9, 3]), ([1, 1], [0, 4]), ([5, 3], [2, 0]), ([300], [100]), ([1] * 70, list(range(1, 71))),
                                    ([0, 33, 0, 1, 64], [5, 40, 0, 600, 64])])
def test_empty_rows_and_sequences(new, kv):
    """Sequences without new tokens, without a context, and rows before the first key."""
    _run(new, kv, 8, 2, 128, pad=3)
    _run(new, kv, 4, 2, 96)
    _run(new, kv, 4, 2, 64, io="f32")


@pytest.mark.parametrize("window", [1, 2, 16, 100, 129, 5000])
@pytest.mark.parametrize("causal", [True, False])
def test_windows_and_full_masks(window, causal):
    _run([1, 6, 200], [900, 400, 333], 8, 2, 128, window=window, causal=causal)
    _run([1, 6, 100], [900, 400, 100], 4, 2, 64, window=window, causal=causal, fmt="e4m3")
    _run([4], [90], 4, 2, 64, window=window, causal=causal, io="f32")
    if window == 1:
        _run([3, 130], [70, 200], 8, 2, 128, causal=causal)


def test_alignment_of_rows():
    for off in (1, 2, 4, 8):
        _run([1, 30], [50, 60], 4, 2, 64, off=off)
        _run([1, 300], [50, 300], 4, 1, 128, off=off)
        s = _make([2, 200], [80, 300], 4, 2, 128)
        buf = torch.zeros((202, 4 * 128 + off), dtype=torch.bfloat16, device="cuda")
        out = buf[:, off:].unflatten(1, (4, 128))
        gb.attn_cache8(*_args(s), out=out)
        _check(s, out)
        assert (buf[:, :off] == 0).all()


def test_unaligned_cache():
    s = _make([1, 40], [100, 60], 4, 2, 64)
    moved = []
    for c in s["cache"]:
        if c.element_size() == 1:  # heads 65 bytes apart
            wide = torch.zeros((*c.shape[:3], 65), dtype=torch.uint8, device="cuda")
            wide[..., 1:] = c.view(torch.uint8)
            moved.append(wide[..., 1:].view(c.dtype))
        else:
            moved.append(c)
    s["cache"] = moved
    _check(s, gb.attn_cache8(*_args(s)))


@pytest.mark.parametrize("new,kv", [([1, 1], [700, 300]), ([150, 200], [700, 300])])
def test_masked_places_hold_anything(new, kv):
    """Keys behind the rows, with infinite scales, and pages before a window: no part in a result."""
    for fmt in ("int8", "e4m3"):
        s = _make(new, kv, 8, 2, 128, fmt=fmt)
        plain = gb.attn_cache8(*_args(s), window=90)
        for b, (m, n) in enumerate(zip(new, kv)):  # pages wholly before the first new token's window
            s["table"][b, :max(0, n - m + 1 - 90) // 16] = -5
        assert torch.equal(gb.attn_cache8(*_args(s), window=90), plain)
        assert gb.device_error() == 0
    # the last key is NaN: only the rows that see it are
    s = _make([150], [400], 8, 2, 128, fmt="e4m3")
    good = gb.attn_cache8(*_args(s))
    kc, ks, vc, vs = s["cache"]
    page, off = int(s["table"][0, 399 // 16]), 399 % 16
    vs[page, off] = float("nan")
    vc.view(torch.uint8)[page, off] = 0x7f
    out = gb.attn_cache8(*_args(s))
    assert out[149].isnan().all() and torch.equal(out[:149], good[:149])
    vs[page, off] = 1.0
    vc.view(torch.uint8)[page, off] = 0
    ks[page, off, 1] = float("nan")  # K/V head 1: query heads 4 .. 7
    out = gb.attn_cache8(*_args(s))
    assert out[149, 4:].isnan().all() and torch.equal(out[:149], good[:149]) and out[149, :4].isfinite().all()


def test_not_finite_rows_stay_alone():
    for new, kv in (([1, 3], [40, 50]), ([140], [300])):
        s = _make(new, kv, 8, 2, 128)
        good = gb.attn_cache8(*_args(s))
        s["q"][1, 2, 5] = float("nan")
        s["q"][2, 3, 0] = float("inf")
        out = gb.attn_cache8(*_args(s))
        assert out[1, 2].isnan().all() and out[2, 3].isnan().any()
        keep = torch.ones(out.shape[:2], dtype=torch.bool, device="cuda")
        keep[1, 2] = keep[2, 3] = False
        assert torch.equal(out[keep], good[keep])


def test_large_and_small_scores():
    """Scores far apart (weights underflow), all equal, of tiny scales."""
    for scale in (30.0, 0.0, -2.0, 1e-20):
        for new, kv in (([2, 1], [200, 90]), ([160], [300])):
            s = _make(new, kv, 4, 2, 64)
            out = gb.attn_cache8(*_args(s), scale=scale)
            if scale == 30.0:
                # scores up to 30 * 64: their float32 error (67 * 2^-24 * 30 * 64) moves weights by 2^-7; compare where one key leads
                t = 0
                for b, (m, n) in enumerate(zip(new, kv)):
                    o, _ = heads.attend(to64(s["q"])[t:t + m], s["values"][0][b], s["values"][1][b], scale, n - m)
                    a, _ = heads.attend(to64(s["q"])[t:t + m], s["values"][0][b], np.abs(s["values"][1][b]), scale, n - m)
                    assert (np.abs(to64(out)[t:t + m] - o) <= (2.0 ** -7 + 2.0 ** -6) * a + 1e-6).all()
                    t += m
            else:
                _check(s, out, scale=scale)


def test_bad_pages_are_nan_and_reported():
    for D in (128, 80):
        s = _make([1, 2], [100, 60], 4, 2, D)
        good = gb.attn_cache8(*_args(s))
        for bad in (-1, 10 ** 6):
            s["table"][0, 3] = bad
            out = gb.attn_cache8(*_args(s))
            assert out[0].isnan().all() and torch.equal(out[1:], good[1:])
            assert gb.device_error(clear=True) == gb.ERR_BAD_SLOT


def test_lengths_beyond_the_tables_are_cut():
    for D in (128, 80):
        s = _make([2, 3], [64, 40], 4, 2, D, extra_cols=0)  # four columns of 16 slots
        good = gb.attn_cache8(*_args(s))
        s["kv"][0] = 10 ** 9
        assert torch.equal(gb.attn_cache8(*_args(s)), good)
        s["kv"][0] = 64
        s["cu"][2] = 10 ** 9
        assert torch.equal(gb.attn_cache8(*_args(s)), good)


def test_in_place_streams_and_graphs():
    for new, kv in (([1] * 9, [333] * 9), ([200, 1, 130], [700, 900, 130])):
        s = _make(new, kv, 8, 2, 128)
        good = gb.attn_cache8(*_args(s))
        for _ in range(3):
            assert torch.equal(gb.attn_cache8(*_args(s)), good)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):  # two calls at once, a workspace each
            other = gb.attn_cache8(*_args(s))
        again = gb.attn_cache8(*_args(s))
        torch.cuda.synchronize()
        assert torch.equal(other, good) and torch.equal(again, good)
        ws = torch.empty(gb.attn_cache8_workspace(s["T"], len(new), 8, 2, 128), dtype=torch.uint8, device="cuda")
        out = torch.zeros_like(good)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            gb.attn_cache8(*_args(s), out=out, workspace=ws)
        ws.fill_(255)
        g.replay()
        assert torch.equal(out, good)
        # the graph follows the lengths
        s["kv"] -= 3
        s2 = dict(s, lens=[n - 3 for n in s["lens"]], values=[[t[:-3] for t in v] for v in s["values"]])
        g.replay()
        _check(s2, out)
        want = out.clone()
        gb.attn_cache8(*_args(s), out=s["q"])
        assert torch.equal(s["q"], want)


def test_a_long_cache_passes_32_bits():
    """Slots whose codes lie beyond 2^31 bytes."""
    pages, page, Hk, D = 66000, 16, 16, 128  # 2.16e9 bytes of codes
    codes = torch.zeros((pages, page, Hk, D), dtype=torch.int8, device="cuda")
    scale = torch.zeros((pages, page, Hk), device="cuda")
    k, ks = codes, scale
    v, vs = torch.zeros_like(codes), torch.zeros_like(scale)
    s = _make([1, 20], [40, 40], Hk * 2, Hk, D, page=page)
    n = s["cache"][0].shape[0]
    for big, small in zip((k, ks, v, vs), s["cache"]):
        big[-n:] = small.flip(0)
    t = s["table"]
    t[t >= 0] = pages - 1 - t[t >= 0]
    s["cache"] = [k, ks, v, vs]
    _check(s, gb.attn_cache8(*_args(s)))


def test_two_heads_do_not_depend_on_the_batch():
    """A sequence alone and in a batch: the same up to how its keys were divided among blocks."""
    s = _make([1, 1, 1], [500, 900, 100], 8, 2, 128)
    both = gb.attn_cache8(*_args(s))
    one = gb.attn_cache8(s["q"][1:2], torch.tensor([0, 1], dtype=torch.int32, device="cuda"), s["kv"][1:2], s["table"][1:2], *s["cache"])
    assert (both[1:2].float() - one.float()).abs().max() <= 2.0 ** -7 * one.float().abs().max()


def test_binding_refuses():
    s = _make([2, 3], [64, 40], 4, 2, 64)
    ok = list(_args(s))

    def refused(exc, i, bad, **kw):
        a = list(ok)
        a[i] = bad
        with pytest.raises(exc):
            gb.attn_cache8(*a, **kw)
    refused(ValueError, 0, s["q"].cpu())
    refused(ValueError, 0, s["q"][:, :, :32])
    refused(ValueError, 0, s["q"].transpose(1, 2))
    refused(TypeError, 0, s["q"].half())
    refused(gb.GblnError, 0, s["q"][:, :3])  # three heads over two
    refused(ValueError, 1, s["cu"][:2])
    refused(TypeError, 1, s["cu"].long())
    refused(TypeError, 2, s["kv"].long())
    refused(ValueError, 3, s["table"][:1])
    refused(ValueError, 3, s["table"].long())
    refused(ValueError, 3, s["table"].T.contiguous().T)
    refused(TypeError, 4, ok[4].view(torch.uint8))
    refused(ValueError, 5, ok[5][:1])
    refused(ValueError, 0, s["q"], out=s["q"].float())
    refused(ValueError, 0, s["q"], lse=torch.zeros(3, device="cuda"))
    refused(TypeError, 0, s["q"], workspace=torch.zeros(9, device="cuda"))
    refused(gb.GblnError, 0, s["q"], workspace=torch.zeros(16, dtype=torch.uint8, device="cuda"))
    refused(gb.GblnError, 0, s["q"], window=-1)
    refused(gb.GblnError, 0, s["q"], scale=float("nan"))
    assert gb.attn_cache8(s["q"][:0], s["cu"][:1], s["kv"][:0], s["table"][:0], *s["cache"]).shape == (0, 4, 64)


def test_a_layer_serves_prompts_then_decodes():
    """The calls as a serving program makes them: projections' rows, norm + rotation + store, attention;
    a prompt in chunks, then single tokens, against the whole in float64."""
    Hq, Hk, D, page, n = 8, 2, 128, 16, 61
    r = np.random.default_rng(5)
    x = torch.from_numpy(r.normal(size=(2, n, (Hq + 2 * Hk) * D)).astype(np.float32)).cuda().bfloat16()
    wq, wk = (torch.from_numpy((1 + 0.1 * r.normal(size=D)).astype(np.float32)).cuda().bfloat16() for _ in range(2))
    table, theta, eps = gb.rope_table(n, D, 1e4), 1e4, 1e-6
    pages = torch.from_numpy(r.permutation(10)[:8].reshape(2, 4).astype(np.int32)).cuda()
    cache = [t for _ in range(2) for t in (torch.zeros((10, page, Hk, D), dtype=torch.int8, device="cuda"), torch.zeros((10, page, Hk), device="cuda"))]
    got = torch.zeros((2, n, Hq, D), dtype=torch.bfloat16, device="cuda")
    at = 0
    for m in [40, 17] + [1] * 4:
        rows = x[:, at:at + m].reshape(2 * m, -1)
        q, k, v = (t.unflatten(1, (-1, D)) for t in rows.split([Hq * D, Hk * D, Hk * D], dim=1))
        pos = torch.arange(at, at + m, device="cuda", dtype=torch.int32).repeat(2)
        j = pos.long()
        slots = pages.long().repeat_interleave(m, 0)[torch.arange(2 * m, device="cuda"), j // page] * page + j % page
        q = gb.qk_norm_rope_fwd_cache8(q, k, v, wq, wk, pos, table, eps, slots, *cache)
        cu = torch.tensor([0, m, 2 * m], dtype=torch.int32, device="cuda")
        kv = torch.tensor([at + m] * 2, dtype=torch.int32, device="cuda")
        got[:, at:at + m] = gb.attn_cache8(q, cu, kv, pages, *cache).view(2, m, Hq, D)
        at += m
    assert at == n
    p = np.arange(n)[None]
    for b in range(2):
        q, k, v = np.split(to64(x[b]).reshape(n, -1, D), [Hq, Hq + Hk], axis=1)
        q, k = (heads.norm_rotate(t, to64(w), p, np.zeros(D // 2, int), theta, eps) for t, w in ((q, wq), (k, wk)))
        o, _ = heads.attend(q, k, v, D ** -0.5, 0)
        # the cache's own rounding: K and V off by a / 254 each (1.4% of a normal head's standard deviation), q by 2^-8
        assert np.linalg.norm(to64(got[b]) - o) <= 0.02 * np.linalg.norm(o)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("io,D", [("bf16", 80), ("bf16", 72), ("bf16", 33), ("f32", 64), ("f32", 200)])
def test_other_sizes_over_long_contexts(io, D, fmt):
    """Rows whose keys several warps share, also where a window or the context leaves some of them none."""
    _run([1, 6, 3], [700, 300, 2000], 4, 2, D, io=io, fmt=fmt, pad=1)
    _run([2, 1, 40], [257, 31, 600], 4, 2, D, io=io, fmt=fmt, window=100)
    _run([3, 1], [2, 0], 4, 2, D, io=io, fmt=fmt, causal=False)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("off", [1, 2, 4, 8, 16])
def test_codes_at_any_address(off, fmt):
    s = _make([1, 40], [300, 200], 4, 2, 128, fmt=fmt)
    for i in (0, 2):
        c = s["cache"][i]
        moved = torch.empty(c.numel() + off, dtype=torch.uint8, device="cuda")[off:]
        moved.copy_(c.view(torch.uint8).flatten())
        s["cache"][i] = moved.view(c.dtype).view(c.shape)
    _check(s, gb.attn_cache8(*_args(s)), what=f"{fmt} {off}")
    assert gb.device_error() == 0


@pytest.mark.parametrize("new,kv,Hq,Hk", [([1] * 64, [1024] * 64, 32, 8), ([80] * 12, [400] * 12, 8, 2), ([64], [2000], 4, 1), ([1], [3000], 4, 1)])
def test_divided_units_are_joined(new, kv, Hq, Hk):
    """Many units of few parts (warps with rows of their own), one unit of many (a block for a row)."""
    _run(new, kv, Hq, Hk, 128)
    _run(new, kv, Hq, Hk, 64, fmt="e4m3", window=300)
