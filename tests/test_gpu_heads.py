"""GPU vs oracle: per-head RMSNorm of Q and K with the rotation, position axes, their
gradients, and the form that stores K and V in the 8-bit cache."""

import numpy as np
import pytest
import torch

import rmsnorm_fwd_bwd_03_gb300 as gb
from oracle import heads

from _checks import check_dw, check_io, dx_scale, to64
from _q8 import CODE, check_exact, check_window

pytestmark = pytest.mark.gpu

IO = {"f32": torch.float32, "bf16": torch.bfloat16}
THETA, EPS, MAXP = 1e4, 1e-5, 60


@pytest.fixture(scope="module", autouse=True)
def _library():
    from rmsnorm_fwd_bwd_03_gb300._build import build_library
    build_library()
    gb.library()


def _randn(shape, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def _heads_of(T, H, D, io, seed, off, packed):
    """[T, H, D], its rows contiguous or inside wider ones, `off` values past an aligned address."""
    if H == 0:
        return None
    width = H * D + (D if packed else 0)
    return _randn((T, width + off), IO[io], seed)[:, off:off + H * D].unflatten(1, (H, D)) if packed or off \
        else _randn((T, H, D), IO[io], seed)


def _setup(T, Hq, Hk, D, io, wt, n, pairing, packed, off, seed):
    r = np.random.default_rng(seed + T + D + n)
    s = {"q": _heads_of(T, Hq, D, io, seed, off, packed), "k": _heads_of(T, Hk, D, io, seed + 1, off, packed),
         "dq": _heads_of(T, Hq, D, io, seed + 2, off, packed), "dk": _heads_of(T, Hk, D, io, seed + 3, off, packed)}
    pos = r.integers(0, MAXP, (n, T)).astype(np.int32)
    axis = r.integers(0, n, D // 2)
    s["pos"], s["axis"] = pos, axis
    s["positions"] = torch.from_numpy(pos if n > 1 else pos[0]).cuda()
    s["axes"] = bytes(axis.tolist()) if n > 1 else None
    s["table"] = gb.rope_table(MAXP, D, THETA)
    s["wq"], s["wk"] = (1 + 0.2 * _randn((D,), torch.float32, seed + 4 + i) for i in range(2))
    s["wq"], s["wk"] = s["wq"].to(IO[wt]), s["wk"].to(IO[wt])
    return s


def _case(T, Hq, Hk, D, io="bf16", wt="bf16", n=1, pairing="half", packed=False, off=0, seed=0):
    s = _setup(T, Hq, Hk, D, io, wt, n, pairing, packed, off, seed)
    what = f"{T}x{Hq}/{Hk}x{D} {io}/{wt} {n} axes {pairing} packed={packed} off={off}"
    where = (s["positions"], s["table"])
    how = {"pairing": pairing}
    wk = s["wk"] if Hk else None
    q, k = gb.qk_norm_rope_fwd(s["q"], s["k"], s["wq"], wk, *where, EPS, axes=s["axes"], **how)
    dq, dk, part, P = gb.qk_norm_rope_bwd(s["dq"], s["dk"], s["q"], s["k"], s["wq"], wk, *where, EPS, axes=s["axes"], **how)
    dwq, dwk = gb.qk_norm_dw_finalize(part, P)
    assert P == gb.qk_norm_rope_bwd_num_partials(T, Hq, Hk, D)
    pos2 = s["positions"] if n > 1 else s["positions"][None]
    axes2 = s["axes"] if n > 1 else bytes(D // 2)
    rq, rk = gb.rope_axes_fwd(s["q"], s["k"], pos2, s["table"], axes2, **how)
    bq, bk = gb.rope_axes_bwd(s["dq"], s["dk"], pos2, s["table"], axes2, **how)
    args = (s["pos"], s["axis"], THETA)
    for x, d, w, y, dx, dw, rx, bx, name in ((s["q"], s["dq"], s["wq"], q, dq, dwq, rq, bq, " q"),
                                            (s["k"], s["dk"], s["wk"], k, dk, dwk, rk, bk, " k")):
        if x is None:
            assert y is None and dx is None and rx is None and bx is None and not dw.any()
            continue
        x64, d64, w64 = to64(x), to64(d), to64(w)
        check_io(to64(y), heads.norm_rotate(x64, w64, *args, EPS, pairing), io, what + name)
        dx_r, dw_r = heads.norm_rotate_bwd(d64, x64, w64, *args, EPS, pairing)
        rstd = 1 / np.sqrt((x64 ** 2).mean(-1) + EPS)
        # a gradient before its rotation is at most sqrt(2) of its pair's largest value
        scale = None if D > 16 else dx_scale(2 ** 0.5 * np.abs(d64).max(-1, keepdims=True) * np.ones(D), np.abs(w64), rstd)
        if io == "bf16" and D <= 16:  # the terms cancel: bound by float32 roundings of the largest
            err = np.abs(to64(dx) - dx_r)
            assert (err <= 1e-2 * np.abs(dx_r) + 1e-3 + 2.0 ** -20 * scale).all(), what + name + " dx"
        else:
            check_io(to64(dx), dx_r, io, what + name + " dx", scale=scale)
        if dw_r.any():
            # both sums of n = x rstd products; where T and D are 1 or 2 they may cancel
            err = np.linalg.norm(to64(dw) - dw_r)
            assert err <= 1e-3 * np.linalg.norm(dw_r) + 2.0 ** -20 * np.abs(d64).max() * x.shape[1] * T, what + name + " dw"
        check_io(to64(rx), heads.rotate(x64, *args, pairing), io, what + name + " rotated")
        check_io(to64(bx), heads.rotate(d64, *args, pairing, back=True), io, what + name + " rotated back")
    assert gb.device_error() == 0


@pytest.mark.parametrize("pairing", ["half", "interleaved"])
@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("D", [2, 6, 8, 16, 40, 64, 72, 80, 96, 128, 192, 256, 512])
def test_head_sizes(D, io, pairing):
    wt = "f32" if io == "f32" or D % 3 == 0 else "bf16"
    _case(1, 3, 1, D, io, wt, 1 + D % 3, pairing)
    _case(37, 4, 2, D, io, wt, 1 + (D // 2) % 4, pairing, packed=True)


@pytest.mark.parametrize("Hq,Hk", [(1, 0), (1, 1), (8, 8), (32, 8), (7, 1), (28, 4), (64, 8), (5, 3), (40, 40), (130, 2), (300, 3)])
def test_head_counts(Hq, Hk):
    _case(19, Hq, Hk, 64, "bf16", "bf16", 3)
    _case(5, Hq, Hk, 128, "bf16", "f32", 1, packed=True)


@pytest.mark.parametrize("D,Hq,Hk", [(512, 300, 3), (512, 40, 20), (256, 200, 8)])
def test_many_wide_heads(D, Hq, Hk):
    """More chunks of a token than a few tokens bring blocks."""
    _case(1, Hq, Hk, D, "bf16", "bf16", 2)
    _case(3, Hq, Hk, D, "f32" if D == 256 else "bf16", "f32", 1)
    _case(150, Hq, Hk, D, "bf16", "f32", 1)


@pytest.mark.parametrize("off", [1, 2, 4, 8])
@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_alignment(io, off):
    _case(23, 4, 2, 64, io, "f32", 2, packed=True, off=off)
    _case(23, 4, 2, 136, io, "f32", 1, "interleaved", packed=True, off=off)


@pytest.mark.parametrize("T", [1, 2, 3, 31, 257, 1000, 4099])
def test_token_counts(T):
    _case(T, 16, 8, 128, "bf16", "bf16", 1, packed=True)
    _case(T, 14, 2, 64, "f32", "f32", 3)


@pytest.mark.parametrize("Hq,Hk,D", [(16, 8, 128), (2, 1, 64), (7, 1, 96), (64, 8, 64), (1, 0, 128), (4, 4, 256), (3, 1, 72)])
@pytest.mark.parametrize("pairing", ["half", "interleaved"])
def test_many_tokens(Hq, Hk, D, pairing):
    """Enough for the persistent kernels: warps that take several steps, several tokens at once."""
    _case(9001, Hq, Hk, D, "bf16", "bf16", 1 + Hq % 3, pairing, packed=True)
    _case(6007, Hq, Hk, D, "f32", "f32", 2, pairing)


def test_in_place_and_packed_gradient():
    s = _setup(50, 4, 2, 64, "bf16", "bf16", 2, "half", True, 0, 3)
    a = (s["wq"], s["wk"], s["positions"], s["table"], EPS)
    q, k = gb.qk_norm_rope_fwd(s["q"], s["k"], *a, axes=s["axes"])
    dq, dk, part, P = gb.qk_norm_rope_bwd(s["dq"], s["dk"], s["q"], s["k"], *a, axes=s["axes"])
    grad = torch.full((50, 8 * 64), 7.0, dtype=torch.bfloat16, device="cuda")  # dq, dk, dv of one packed row
    gq, gk = grad[:, :256].unflatten(1, (4, 64)), grad[:, 256:384].unflatten(1, (2, 64))
    part2 = torch.full((P + 2, 128), 3.0, device="cuda")
    gb.qk_norm_rope_bwd(s["dq"], s["dk"], s["q"], s["k"], *a, axes=s["axes"], dq_in=gq, dk_in=gk, dw_partial=part2)
    assert torch.equal(gq, dq) and torch.equal(gk, dk) and torch.equal(part2[:P], part) and (part2[P:] == 3).all()
    assert (grad[:, 384:] == 7).all()
    d1, d2 = s["dq"].clone(), s["dk"].clone()
    gb.qk_norm_rope_bwd(d1, d2, s["q"], s["k"], *a, axes=s["axes"], dq_in=d1, dk_in=d2)
    assert torch.equal(d1, dq) and torch.equal(d2, dk)
    gb.qk_norm_rope_fwd(s["q"], s["k"], *a, axes=s["axes"], q_out=s["q"], k_out=s["k"])
    assert torch.equal(s["q"], q) and torch.equal(s["k"], k)
    w1, w2 = gb.qk_norm_dw_finalize(part, P)
    v1, v2 = w1.clone(), w2.clone()
    gb.qk_norm_dw_finalize(part, P, w1, w2, accumulate=True)
    assert torch.equal(w1, 2 * v1) and torch.equal(w2, 2 * v2)


def test_bad_positions_are_nan_and_reported():
    s = _setup(9, 2, 1, 64, "bf16", "bf16", 3, "half", False, 0, 1)
    for D_path in (0, 1):  # vector and element path
        q, k = (t if not D_path else _heads_of(9, t.shape[1], 64, "bf16", 5, 1, True) for t in (s["q"], s["k"]))
        pos = s["positions"].clone()
        pos[1, 4], pos[2, 7] = MAXP, -1
        o, p = gb.rope_axes_fwd(q, k, pos, s["table"], s["axes"])
        assert gb.device_error(clear=True) == gb.ERR_BAD_POSITION
        bad = torch.zeros(9, dtype=torch.bool, device="cuda")
        bad[4] = bad[7] = True
        for t in (o, p):
            assert t[bad].isnan().all() and t[~bad].isfinite().all()


def test_extreme_heads():
    """A head of zeros gives zeros; an infinity or a NaN stays in its own head."""
    s = _setup(4, 3, 1, 128, "bf16", "bf16", 1, "half", False, 0, 2)
    s["q"][1, 1] = 0
    s["q"][2, 0, 5] = float("inf")
    s["q"][3, 2, 7] = float("nan")
    a = (s["wq"], s["wk"], s["positions"], s["table"], EPS)
    q, _ = gb.qk_norm_rope_fwd(s["q"], s["k"], *a)
    assert (q[1, 1] == 0).all() and q[2, 0].isnan().any() and q[3, 2].isnan().all()
    ok = torch.ones((4, 3), dtype=torch.bool, device="cuda")
    ok[2, 0] = ok[3, 2] = False
    assert q[ok].isfinite().all()


def _cache(pages, page, Hk, D, fmt):
    c = [torch.full((pages, page, Hk, D), 0x55, dtype=torch.uint8, device="cuda").view(CODE[fmt]) for _ in range(2)]
    s = [torch.full((pages, page, Hk), -7.0, device="cuda") for _ in range(2)]
    return c[0], s[0], c[1], s[1]


def _norm_window(x64, w64):
    """t = rotation of x * w in float32: the product, the turn's c and s, two products and a sum
    rounded (2^-24 each): five roundings of at most |u1| + |u2|, with the head's largest for both."""
    return 12 * 2.0 ** -24 * np.abs(x64 * w64).max(axis=-1, keepdims=True)


@pytest.mark.parametrize("pairing", ["half", "interleaved"])
@pytest.mark.parametrize("io,D,Hq,Hk", [("bf16", 128, 32, 8), ("bf16", 64, 14, 2), ("bf16", 96, 4, 1), ("bf16", 72, 8, 8), ("bf16", 66, 2, 2),
                                        ("bf16", 256, 8, 4), ("f32", 64, 14, 2), ("f32", 128, 4, 4), ("f32", 6, 2, 1), ("bf16", 512, 3, 2),
                                        ("bf16", 128, 0, 8)])
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_cache(io, D, Hq, Hk, fmt, pairing):
    for T, n, norm in ((1, 1, True), (45, 3, True), (700, 1, True), (5003, 2, True), (33, 2, False)):
        s = _setup(T, max(Hq, 1), Hk, D, io, "f32" if io == "f32" or n > 1 else "bf16", n, pairing, True, 0, T)
        q = s["q"] if Hq else None
        r = np.random.default_rng(T)
        page, pages = 7, -(-T // 7) + 2
        slots = torch.from_numpy(r.permutation(pages * page)[:T]).cuda()
        if T > 40:
            slots[3] = -2
        cache = _cache(pages, page, Hk, D, fmt)
        v = _heads_of(T, Hk, D, io, 99, 0, True)
        wq, wk = (s["wq"] if Hq else None, s["wk"]) if norm else (None, None)
        qo = gb.qk_norm_rope_fwd_cache8(q, s["k"], v, wq, wk, s["positions"], s["table"], EPS, slots, *cache, axes=s["axes"], pairing=pairing)
        args = (s["pos"], s["axis"], THETA)
        if Hq:
            q64 = to64(q)
            want = heads.norm_rotate(q64, to64(wq), *args, EPS, pairing) if norm else heads.rotate(q64, *args, pairing)
            check_io(to64(qo), want, io, "q")
        keep = (slots >= 0).cpu().numpy()
        sl = slots[slots >= 0]
        at = (sl // page, sl % page)
        kc, ks, vc, vs = cache
        k64 = to64(s["k"])[keep]
        w64 = to64(wk) if norm else np.ones(D)
        rstd = 1 / np.sqrt((k64 ** 2).mean(-1) + EPS) if norm else np.ones(k64.shape[:2])
        t64 = heads.rotate(to64(s["k"]) * w64, *args, pairing)[keep]
        # the stored scale without the head's rstd (float32: relative 2^-20 with its sum's and roots' roundings)
        got_s = torch.from_numpy((to64(ks[at]) / rstd)).cuda()
        win = _norm_window(k64, w64) + 2.0 ** -20 * np.abs(t64).max(-1, keepdims=True)
        check_window(kc.view(torch.uint8)[at].view(CODE[fmt]), got_s, t64, win, fmt, "k", max_ambiguous=2e-2)
        check_exact(vc.view(torch.uint8)[at].view(CODE[fmt]), vs[at], to64(v)[keep], fmt, "v")
        left = torch.ones(pages * page, dtype=torch.bool, device="cuda")
        left[sl] = False
        left = left.nonzero()[:, 0]
        for c, sc in ((kc, ks), (vc, vs)):
            assert (c.view(torch.uint8)[left // page, left % page] == 0x55).all() and (sc[left // page, left % page] == -7).all()
        if not norm and n == 1:
            break
    assert gb.device_error() == 0


@pytest.mark.parametrize("io,D", [("bf16", 128), ("bf16", 80), ("f32", 64), ("bf16", 66)])
def test_without_norms_the_cache_gets_the_plain_bits(io, D):
    s = _setup(61, 8, 2, D, io, "f32", 1, "half", True, 0, 8)
    v = _heads_of(61, 2, D, io, 9, 0, True)
    slots = torch.arange(61, device="cuda").flip(0)
    a, b = _cache(8, 8, 2, D, "int8"), _cache(8, 8, 2, D, "int8")
    q1 = gb.rope_fwd_cache8(s["q"], s["k"], v, s["positions"], s["table"], slots, *a)
    q2 = gb.qk_norm_rope_fwd_cache8(s["q"], s["k"], v, None, None, s["positions"], s["table"], EPS, slots, *b)
    assert torch.equal(q1, q2)
    for x, y in zip(a, b):
        assert torch.equal(x, y)


def test_chunks_of_a_prompt_store_the_same_bits():
    s = _setup(700, 32, 8, 128, "bf16", "bf16", 3, "half", True, 0, 4)
    v = _heads_of(700, 8, 128, "bf16", 9, 0, True)
    slots = torch.arange(700, device="cuda")
    whole, parts = _cache(50, 16, 8, 128, "e4m3"), _cache(50, 16, 8, 128, "e4m3")
    call = lambda i, j, c: gb.qk_norm_rope_fwd_cache8(  # noqa: E731
        s["q"][i:j], s["k"][i:j], v[i:j], s["wq"], s["wk"], s["positions"][:, i:j].contiguous(), s["table"], EPS, slots[i:j], *c, axes=s["axes"])
    q = call(0, 700, whole)
    qs = [call(i, j, parts) for i, j in ((0, 1), (1, 34), (34, 690), (690, 700))]
    assert torch.equal(q, torch.cat(qs))
    for x, y in zip(whole, parts):
        assert torch.equal(x.view(torch.uint8) if x.element_size() == 1 else x, y.view(torch.uint8) if y.element_size() == 1 else y)


def test_runs_repeat_and_graphs_replay():
    s = _setup(513, 16, 8, 128, "bf16", "bf16", 2, "half", True, 0, 6)
    a = (s["wq"], s["wk"], s["positions"], s["table"], EPS)

    def step():
        q, k = gb.qk_norm_rope_fwd(s["q"], s["k"], *a, axes=s["axes"])
        dq, dk, part, P = gb.qk_norm_rope_bwd(s["dq"], s["dk"], s["q"], s["k"], *a, axes=s["axes"])
        return (q, k, dq, dk, *gb.qk_norm_dw_finalize(part, P))

    first = [t.clone() for t in step()]
    for x, y in zip(first, step()):
        assert torch.equal(x, y)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = step()
    torch.cuda.current_stream().wait_stream(side)
    for x, y in zip(first, again):
        assert torch.equal(x, y)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step()
    for t in out:
        t.zero_()
    g.replay()
    for x, y in zip(first, out):
        assert torch.equal(x, y)


def test_binding_refuses():
    s = _setup(6, 4, 2, 64, "bf16", "bf16", 2, "half", False, 0, 7)
    a = dict(axes=s["axes"])
    ok = (s["q"], s["k"], s["wq"], s["wk"], s["positions"], s["table"], EPS)

    def refused(exc, i, bad, **kw):
        args = list(ok)
        args[i] = bad
        with pytest.raises(exc):
            gb.qk_norm_rope_fwd(*args, **{**a, **kw})
    refused(ValueError, 0, s["q"].cpu())
    refused(ValueError, 0, s["q"].transpose(1, 2))
    refused(ValueError, 1, s["k"][:5])
    refused(ValueError, 1, s["k"].float())
    refused(ValueError, 2, s["wq"][:32])
    refused(TypeError, 3, s["wk"].float())
    refused(ValueError, 3, None)
    refused(ValueError, 4, s["positions"][0])
    refused(ValueError, 4, s["positions"][:, :5])
    refused(TypeError, 4, s["positions"].long())
    refused(ValueError, 4, s["positions"].T.contiguous().T)
    refused(ValueError, 5, s["table"][:, :16])
    refused(ValueError, 0, s["q"], axes=bytes(31))
    refused(ValueError, 0, s["q"], axes=bytes([2] * 32))
    refused(ValueError, 0, s["q"], q_out=s["k"])
    with pytest.raises(ValueError):
        gb.qk_norm_rope_bwd(s["dq"][:5], s["dk"], *ok, **a)
    with pytest.raises(gb.GblnError):
        gb.qk_norm_rope_fwd(*ok[:6], -1.0, **a)
    with pytest.raises(gb.GblnError):
        gb.qk_norm_rope_bwd(s["dq"], s["dk"], *ok, dw_partial=torch.zeros((0, 128), device="cuda"), **a)


@pytest.mark.parametrize("n", [1, 3])
@pytest.mark.parametrize("pairing", ["half", "interleaved"])
def test_autograd(n, pairing):
    """The wrappers on slices of one packed projection output: the gradients of the formulas."""
    from rmsnorm_fwd_bwd_03_gb300 import autograd as ga
    T, Hq, Hk, D = 40, 4, 2, 64
    s = _setup(T, Hq, Hk, D, "bf16", "bf16", n, pairing, False, 0, 11)
    qkv = _randn((T, (Hq + 2 * Hk) * D), torch.bfloat16, 12).requires_grad_()
    wq, wk = s["wq"].clone().requires_grad_(), s["wk"].clone().requires_grad_()
    q, k, v = (t.unflatten(1, (-1, D)) for t in qkv.split([Hq * D, Hk * D, Hk * D], dim=1))
    yq, yk = ga.qk_norm_rotary(q, k, wq, wk, s["positions"], s["table"], EPS, axes=s["axes"], pairing=pairing)
    torch.autograd.backward([yq, yk, v], [s["dq"], s["dk"], torch.ones_like(v)])
    args = (s["pos"], s["axis"], THETA, EPS, pairing)
    g64, x64 = to64(qkv.grad).reshape(T, -1, D), to64(qkv).reshape(T, -1, D)
    for sl, y, d, w in ((slice(0, Hq), yq, s["dq"], wq), (slice(Hq, Hq + Hk), yk, s["dk"], wk)):
        check_io(to64(y), heads.norm_rotate(x64[:, sl], to64(w), *args), "bf16", "y")
        dx, dw = heads.norm_rotate_bwd(to64(d), x64[:, sl], to64(w), *args)
        check_io(g64[:, sl], dx, "bf16", "dx")
        check_io(to64(w.grad), dw, "bf16", "dw")
    assert (g64[:, Hq + Hk:] == 1).all()
    a, b = s["q"].clone().requires_grad_(), s["k"].clone().requires_grad_()
    out = ga.rotary(a, b, s["positions"], s["table"], axes=s["axes"], pairing=pairing)
    torch.autograd.backward(out, [s["dq"], s["dk"]])
    for x, y, d in ((a, out[0], s["dq"]), (b, out[1], s["dk"])):
        check_io(to64(y), heads.rotate(to64(x), *args[:3], pairing), "bf16", "rotated")
        check_io(to64(x.grad), heads.rotate(to64(d), *args[:3], pairing, back=True), "bf16", "rotated back")
