"""8-bit storage with float32 scales, without a GPU: the oracle's definition is
pinned by hand-worked groups, error bounds and torch's own casts; the C entry
points and the Python binding refuse bad arguments on the host."""

import ctypes

import numpy as np
import pytest
import torch

import oracle
import rmsnorm_fwd_bwd_03_gb300 as gb
from oracle import q8

OK, INVALID, UNSUPPORTED = 0, 1, 2
F32, BF16 = 0, 1
FAKE = 0x10000  # never dereferenced: every call below returns before touching memory
f32, bf = torch.float32, torch.bfloat16


# ---------------------------------------------------------------------------
# The definition
# ---------------------------------------------------------------------------

def test_hand_worked_groups():
    # amax 127/8: scale 1/8, so eighths are kept exactly and halves of them tie to even
    v = np.array([15.875, -0.125, 0.0, 0.0625, 0.1875, -0.3125, 7.9375])
    codes, scale = q8.quantize(v, "int8")
    assert scale == 0.125
    assert codes.tolist() == [127, -1, 0, 0, 2, -2, 64]  # 0.5 -> 0, 1.5 -> 2, -2.5 -> -2, 63.5 -> 64
    # amax 448: scale 1, E4M3 values are kept, ties to even mantissas, subnormals of 2^-9
    v = np.array([448.0, -448.0, 17.0, 19.0, 0.0009765625, 0.0029296875, -1.0625])
    codes, scale = q8.quantize(v, "e4m3")
    assert scale == 1.0
    assert codes.tolist() == [448, -448, 16, 20, 0.0, 0.00390625, -1.0]


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_zero_tiny_and_non_finite_groups(fmt):
    codes, scale = q8.quantize(np.zeros((2, 5)), fmt)
    assert (codes == 0).all() and np.allclose(scale, 2.0 ** -100 / q8.QMAX[fmt], rtol=1e-6)
    # below the floor the step stays the floor's: nothing overflows
    codes, scale = q8.quantize(np.array([2.0 ** -103, -2.0 ** -120]), fmt)
    assert abs(codes[0] * scale - 2.0 ** -103) <= 2.0 ** -101 / 127 and codes[1] * scale <= 0
    for bad in (np.inf, -np.inf, np.nan):
        _, scale = q8.quantize(np.array([[1.0, bad], [1.0, 2.0]]), fmt)
        assert np.isnan(scale[0]) and np.isfinite(scale[1])


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("N", [1, 5, 128, 129, 300])
def test_groups_and_error_bounds(fmt, N):
    rng = np.random.default_rng(N)
    v = rng.standard_normal((7, N)).astype(np.float32).astype(np.float64) * 10.0 ** rng.integers(-6, 6, (7, 1))
    codes, scale = q8.quantize(v, fmt, 128)
    assert scale.shape == (7, -(-N // 128)) and np.abs(codes).max() == q8.QMAX[fmt]
    err = np.abs(q8.values(codes, scale, 128) - v)
    step = np.repeat(scale, 128, axis=-1)[:, :N]
    slack = 2.0 ** -21 * np.abs(v)  # the float32 roundings of v * inv, inv and scale: 3 * 2^-24 of v
    if fmt == "int8":
        assert (err <= 0.5 * step + slack).all()
    else:
        assert (err <= np.maximum(2.0 ** -4 * np.abs(v), 2.0 ** -10 * step) + slack).all()
    # each group by itself
    for g in range(scale.shape[1]):
        c, s = q8.quantize(v[:, 128 * g:128 * (g + 1)], fmt)
        assert np.array_equal(c, codes[:, 128 * g:128 * (g + 1)]) and np.array_equal(s, scale[:, g])


def test_codes_equal_torchs_float32_steps():
    # the same float32 steps in torch: division, product, round / cast
    g = torch.Generator().manual_seed(3)
    v = torch.randn(64, 96, generator=g) * torch.exp(4 * torch.randn(64, 1, generator=g))
    for fmt in ("int8", "e4m3"):
        a = v.abs().amax(-1).clamp(min=2.0 ** -100)
        t = v * torch.div(torch.tensor(q8.QMAX[fmt]), a)[:, None]
        want = t.round() if fmt == "int8" else t.to(torch.float8_e4m3fn).float()
        codes, scale = q8.quantize(v.double().numpy(), fmt)
        assert np.array_equal(codes, want.double().numpy())
        assert np.array_equal(scale, torch.div(a, q8.QMAX[fmt]).double().numpy())


def test_row_scaled_rmsnorm_output():
    rng = np.random.default_rng(0)
    x, r = (oracle.round_to_bf16(rng.standard_normal((9, 40))) for _ in range(2))
    w = oracle.round_to_bf16(1 + 0.1 * rng.standard_normal(40))
    codes, scale, y, h, rstd = q8.rmsnorm_fwd_fp8(x, r, w, 1e-5, "bf16")
    y0, h0, rstd0 = oracle.rmsnorm_fwd(x, r, w, 1e-5, "bf16")
    assert np.allclose(y, y0, rtol=1e-14) and np.array_equal(h, h0) and np.allclose(rstd, rstd0, rtol=1e-14)
    # the value of each code is the output up to half an E4M3 step, and the row's largest is 448
    err = np.abs(codes * scale[:, None] - y)
    assert (err <= np.maximum(2.0 ** -4 * np.abs(y), 2.0 ** -10 * scale[:, None]) + 2.0 ** -21 * np.abs(y)).all()
    assert (np.abs(codes).max(axis=-1) == 448).all()
    assert np.allclose(scale * 448, np.abs(y).max(axis=-1), rtol=1e-6)  # 3 float32 roundings of u


def test_backward_from_kept_values():
    # kept = h: the plain backward; and central differences of sum(dy * y) where kept = h
    rng = np.random.default_rng(1)
    h, dy, dres = (rng.standard_normal((4, 6)) for _ in range(3))
    w, eps = 1 + 0.1 * rng.standard_normal(6), 1e-3
    _, _, rstd = oracle.rmsnorm_fwd(h, None, w, eps)
    dx, dw = q8.rmsnorm_bwd_kept(dy, dres, h, w, rstd)
    dx0, dw0 = oracle.rmsnorm_bwd(dy, dres, h, w, eps)
    assert np.allclose(dx, dx0, rtol=1e-13, atol=1e-13) and np.allclose(dw, dw0, rtol=1e-13, atol=1e-13)
    loss = lambda h, w: float((dy * oracle.rmsnorm_fwd(h, None, w, eps)[0]).sum() + (dres * h).sum())  # noqa: E731
    d = 1e-6
    for idx in np.ndindex(4, 6):
        e = np.zeros((4, 6))
        e[idx] = d
        assert abs((loss(h + e, w) - loss(h - e, w)) / (2 * d) - dx[idx]) < 1e-7
    for j in range(6):
        e = np.zeros(6)
        e[j] = d
        assert abs((loss(h, w + e) - loss(h, w - e)) / (2 * d) - dw[j]) < 1e-7


# ---------------------------------------------------------------------------
# Refusals of the C entry points
# ---------------------------------------------------------------------------

@pytest.fixture(scope="module")
def lib():
    from rmsnorm_fwd_bwd_03_gb300._build import build_library
    build_library()
    return gb.library()


def test_norm_entries_refuse(lib):
    f = FAKE

    def fp8(x=f, r=None, w=f, y=None, q=f, sc=f, ho=None, rs=f, T=4, H=8, eps=1e-5, io=BF16, wt=BF16):
        return lib.gbln_rmsnorm_fwd_fp8(x, r, w, y, q, sc, ho, rs, T, H, eps, io, wt, None)

    def ck(x=f, r=None, w=f, y=f, ho=None, rs=f, q=f, sc=f, T=4, H=8, eps=1e-5, fmt=0, io=BF16, wt=BF16):
        return lib.gbln_rmsnorm_fwd_ckpt8(x, r, w, y, ho, rs, q, sc, T, H, eps, fmt, io, wt, None)

    for fn in (fp8, ck):
        for kw in ({"x": None}, {"w": None}, {"q": None}, {"sc": None}, {"rs": None}, {"r": f}, {"T": -1},
                   {"T": 1 << 31}, {"H": 0}, {"H": (1 << 24) + 1}, {"eps": -1e-6}, {"eps": float("nan")},
                   {"eps": float("inf")}, {"io": 7}, {"wt": 7}):
            assert fn(**kw) == INVALID, (fn, kw)
        assert fn(io=F32, wt=BF16) == UNSUPPORTED
        assert fn(T=0, x=None, w=None, q=None, sc=None, rs=None) == OK
    assert ck(y=None) == INVALID and ck(fmt=2) == INVALID and ck(fmt=-1) == INVALID

    def bwd(dy=f, q=f, sc=f, w=f, rs=f, dx=f, part=f, P=10, T=4, H=8, fmt=1, io=BF16, wt=BF16):
        return lib.gbln_rmsnorm_bwd_ckpt8(dy, None, q, sc, w, rs, dx, part, P, T, H, fmt, io, wt, None)
    for kw in ({"dy": None}, {"q": None}, {"sc": None}, {"w": None}, {"rs": None}, {"dx": None}, {"part": None},
               {"P": -1}, {"T": -1}, {"H": 0}, {"fmt": 5}, {"io": 9}):
        assert bwd(**kw) == INVALID, kw
    assert bwd(io=F32, wt=BF16) == UNSUPPORTED
    assert bwd(T=0, dy=None, q=None, part=None) == OK
    n = lib.gbln_rmsnorm_bwd_ckpt8_num_partials
    assert n(-1, 8, BF16) == -1 and n(4, 0, BF16) == -1 and n(4, 8, 9) == -1 and n(0, 8, BF16) == 0


def test_glu_entries_refuse(lib):
    f = FAKE

    def fp8(g=f, u=f, q=f, sc=f, T=4, I=8, ldg=8, ldu=8, act=0, io=BF16):
        return lib.gbln_glu_fwd_fp8(g, u, q, sc, T, I, ldg, ldu, act, io, None)

    def fwd(g=f, u=f, o=f, gq=f, gs=f, uq=f, us=f, T=4, I=8, ldg=8, ldu=8, ldo=8, act=0, fmt=0, io=BF16):
        return lib.gbln_glu_fwd_ckpt8(g, u, o, gq, gs, uq, us, T, I, ldg, ldu, ldo, act, fmt, io, None)

    def bwd(d=f, gq=f, gs=f, uq=f, us=f, dg=f, du=f, T=4, I=8, ldd=8, lddg=8, lddu=8, act=0, fmt=0, io=BF16):
        return lib.gbln_glu_bwd_ckpt8(d, gq, gs, uq, us, dg, du, T, I, ldd, lddg, lddu, act, fmt, io, None)

    common = ({"T": -1}, {"I": 0}, {"act": 4}, {"act": -1}, {"io": 2}, {"T": 1 << 40, "I": 1 << 30})
    for fn, own in ((fp8, ({"g": None}, {"u": None}, {"q": None}, {"sc": None}, {"ldg": 7}, {"ldu": 7}, {"T": 1 << 31})),
                    (fwd, ({"g": None}, {"u": None}, {"o": None}, {"gq": None}, {"gs": None}, {"uq": None}, {"us": None},
                           {"ldg": 7}, {"ldu": 7}, {"ldo": 7}, {"fmt": 2})),
                    (bwd, ({"d": None}, {"gq": None}, {"gs": None}, {"uq": None}, {"us": None}, {"dg": None},
                           {"du": None}, {"ldd": 7}, {"lddg": 7}, {"lddu": 7}, {"fmt": -1}))):
        for kw in common + own:
            assert fn(**kw) == INVALID, (fn, kw)
    assert fp8(T=0, g=None, u=None, q=None, sc=None) == OK
    assert fwd(T=0, g=None, o=None, gq=None) == OK
    assert bwd(T=0, d=None, gq=None, dg=None) == OK


def _cache(pages=4, page_size=2, Hk=2, D=16, **kw):
    st = dict(codes=FAKE, scale=FAKE, pages=pages, page_size=page_size, page_stride=page_size * Hk * D,
              slot_stride=Hk * D, head_stride=D, scale_page_stride=page_size * Hk, scale_slot_stride=Hk,
              scale_head_stride=1)
    st.update(kw)
    return gb._Cache8(*[st[n] for n, _ in gb._Cache8._fields_])


BAD_CACHES = [
    {"pages": -1}, {"page_size": 0}, {"page_size": -2}, {"codes": None}, {"scale": None},
    {"head_stride": 15}, {"slot_stride": 16},           # heads or slots on one another
    {"page_stride": 32}, {"scale_head_stride": 0}, {"scale_slot_stride": 1}, {"scale_page_stride": 3},
    {"head_stride": -16}, {"page_stride": 1 << 60}, {"pages": 1 << 41}, {"pages": 1 << 30, "page_size": 1 << 30},
]


def test_cache_entries_refuse(lib):
    f, ref = FAKE, ctypes.byref

    def write(q=f, k=f, v=f, qo=f, pos=f, cs=f, mp=9, sl=f, kc=None, vc=None, T=4, Hq=4, Hk=2, D=16, ldq=64, ldk=32,
              ldv=32, ldqo=64, pairing=0, fmt=0, io=BF16):
        kc, vc = kc or _cache(), vc or _cache()
        return lib.gbln_rope_fwd_cache8(q, k, v, qo, pos, cs, mp, sl, ref(kc), ref(vc), T, Hq, Hk, D, ldq, ldk, ldv, ldqo,
                                        pairing, fmt, io, None)

    def read(sl=f, kc=None, vc=None, ko=f, vo=f, T=4, Hk=2, D=16, ldk=32, ldv=32, fmt=0, io=BF16):
        kc, vc = kc or _cache(), vc or _cache()
        return lib.gbln_cache8_read(sl, ref(kc), ref(vc), ko, vo, T, Hk, D, ldk, ldv, fmt, io, None)

    for kw in ({"q": None}, {"k": None}, {"v": None}, {"qo": None}, {"pos": None}, {"cs": None}, {"sl": None},
               {"cs": FAKE + 4}, {"sl": FAKE + 4}, {"mp": -1}, {"T": -1}, {"T": 1 << 34}, {"Hq": -1}, {"Hk": 0}, {"D": 7},
               {"D": 0}, {"ldq": 63}, {"ldk": 31}, {"ldv": 31}, {"ldqo": 63}, {"ldk": 1 << 60}, {"pairing": 2},
               {"fmt": 2}, {"io": 2}, {"Hq": 1 << 30, "ldq": 1 << 40, "ldqo": 1 << 40}):
        assert write(**kw) == INVALID, kw
    for kw in ({"sl": None}, {"ko": None}, {"vo": None}, {"sl": FAKE + 4}, {"T": -1}, {"T": 1 << 34}, {"Hk": 0}, {"D": 0},
               {"ldk": 31}, {"ldv": 31}, {"fmt": -1}, {"io": 2}):
        assert read(**kw) == INVALID, kw
    for bad in BAD_CACHES:
        for fn in (write, read):
            assert fn(kc=_cache(**bad)) == INVALID, bad
            assert fn(vc=_cache(**bad)) == INVALID, bad
    assert write(vc=_cache(pages=3)) == INVALID and read(vc=_cache(page_size=4, page_stride=128, scale_page_stride=8)) == INVALID
    none = ctypes.POINTER(gb._Cache8)()
    assert lib.gbln_cache8_read(f, none, ref(_cache()), f, f, 4, 2, 16, 32, 32, 0, BF16, None) == INVALID
    assert write(T=0, q=None, k=None, v=None, pos=None, sl=None) == OK
    assert read(T=0, sl=None, ko=None, vo=None) == OK


# ---------------------------------------------------------------------------
# Refusals of the binding (before any CUDA call, so CPU tensors show them)
# ---------------------------------------------------------------------------

def _t(*shape, dtype=bf):
    return torch.zeros(shape, dtype=dtype)


def test_binding_refuses_norm_and_glu_tensors():
    T, H = 4, 200
    x, w = _t(T, H), _t(H)
    for fn in (gb.rmsnorm_fwd_fp8, gb.rmsnorm_fwd_ckpt8):
        with pytest.raises(ValueError, match="weight"):
            fn(x, _t(H - 1), 1e-6)
        with pytest.raises(ValueError, match="residual"):
            fn(x, w, 1e-6, _t(T, H, dtype=f32))
        with pytest.raises(ValueError, match="residual_out"):
            fn(x, w, 1e-6, _t(T, H), residual_out=_t(T + 1, H))
        with pytest.raises(ValueError, match="CUDA"):
            fn(x, w, 1e-6)
    with pytest.raises(ValueError, match="format"):
        gb.rmsnorm_fwd_ckpt8(x, w, 1e-6, fmt="int4")
    h8, sc, rstd = _t(T, H, dtype=torch.int8), _t(T, 2, dtype=f32), _t(T, dtype=f32)
    for bad, match in (((_t(T, H - 1, dtype=torch.int8), sc), "h8"), ((h8, _t(T, 1, dtype=f32)), "h8_scale"),
                       ((h8, _t(T, 2)), "h8_scale"), ((_t(T, H), sc), "h8")):
        with pytest.raises((ValueError, TypeError), match=match):
            gb.rmsnorm_bwd_ckpt8(x, *bad, w, rstd)
    with pytest.raises(ValueError, match="weight"):
        gb.rmsnorm_bwd_ckpt8(x, h8, sc, _t(H + 1), rstd)
    with pytest.raises(TypeError, match="rstd"):
        gb.rmsnorm_bwd_ckpt8(x, h8, sc, w, _t(T))
    with pytest.raises(ValueError, match="dw_partial"):
        gb.rmsnorm_bwd_ckpt8(x, h8, sc, w, rstd, dw_partial=_t(4, H))
    for fn in (gb.glu_fwd_fp8, gb.glu_fwd_ckpt8):
        with pytest.raises(ValueError, match="up"):
            fn(x, _t(T, H + 8))
        with pytest.raises(ValueError, match="CUDA"):
            fn(x, x)
    with pytest.raises(ValueError, match="gate8"):
        gb.glu_bwd_ckpt8(x, _t(T, H - 1, dtype=torch.int8), sc, h8, sc)
    with pytest.raises(ValueError, match="up8_scale"):
        gb.glu_bwd_ckpt8(x, h8, sc, h8, _t(T, 3, dtype=f32))
    with pytest.raises(TypeError, match="same dtype"):
        gb.glu_bwd_ckpt8(x, h8, sc, _t(T, H, dtype=torch.float8_e4m3fn), sc)
    with pytest.raises(ValueError, match="dgate"):
        gb.glu_bwd_ckpt8(x, h8, sc, h8, sc, dgate=_t(T, H, dtype=f32))


def test_binding_refuses_cache_tensors():
    # _heads and the device checks come first for CUDA-only properties, so the
    # shape checks of the caches are exercised on their own helper
    codes, scale = _t(3, 4, 2, 16, dtype=torch.int8), _t(3, 4, 2, dtype=f32)
    for c, s, match in ((_t(3, 4, 2, 16), scale, "k_cache"), (codes[0], scale, "k_cache"),
                        (_t(3, 4, 3, 16, dtype=torch.int8), scale, "k_cache"),
                        (_t(3, 0, 2, 16, dtype=torch.int8), scale, "k_cache"),
                        (codes, scale[:2], "k_scale"), (codes, scale.to(bf), "k_scale"),
                        (codes.transpose(2, 3).contiguous().transpose(2, 3), scale, "next to one another"),
                        (codes, scale, "CUDA")):
        with pytest.raises((ValueError, TypeError), match=match):
            gb._cache8(c, s, 2, 16, "k")
    with pytest.raises(ValueError, match="CUDA"):
        gb.rope_fwd_cache8(None, _t(2, 2, 16), _t(2, 2, 16), None, None, None, codes, scale, codes, scale)
    with pytest.raises(TypeError, match="slots"):
        gb.cache8_read(torch.zeros(3, dtype=torch.int32), codes, scale, codes, scale)
    with pytest.raises(ValueError, match="k_out"):
        gb.cache8_read(torch.zeros(3, dtype=torch.int64), codes, scale, codes, scale, k_out=_t(3, 2, 16, dtype=f32))


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_stated_bounds_hold_beside_outliers(fmt):
    # the bound the header states, in the group's largest magnitude a: values from 2^-30 of it to
    # itself, where E4M3 codes run through its normal range, its subnormals and zero.  Four float32
    # roundings (q / a, v * inv, a / q, code * scale): under 5 * 2^-24 < 2^-21 of the value
    rng = np.random.default_rng(7)
    a = 10.0 ** rng.uniform(-6, 6, (400, 1))
    v = (a * 2.0 ** -rng.uniform(0, 30, (400, 96)) * rng.choice([-1.0, 1.0], (400, 96)))
    v[:, :1] = a
    v = v.astype(np.float32).astype(np.float64)
    a = np.abs(v).max(-1, keepdims=True)
    codes, scale = q8.quantize(v, fmt)
    value = (codes.astype(np.float32) * scale.astype(np.float32)[:, None]).astype(np.float64)
    own = a / 254 if fmt == "int8" else np.maximum(2.0 ** -4 * np.abs(v), a / 448 * 2.0 ** -10)
    assert (np.abs(value - v) <= own + 2.0 ** -21 * np.abs(v)).all()
    if fmt == "e4m3":
        small = np.abs(v) < a / 448 * 2.0 ** -10 * (1 - 2.0 ** -20)
        assert small.any() and (codes[small] == 0).all()
        assert (np.abs(value - v) > 2.0 ** -4 * np.abs(v))[np.abs(v) < a * 2.0 ** -16].any()  # not 2^-4 of all values


def test_cache_write_refuses_one_cache_for_k_and_v(lib):
    # stored into the same memory, K and V would leave either's codes with the other's scale; every
    # other refusal stands with caches of their own too
    f, ref = FAKE, ctypes.byref
    own = {"codes": FAKE + (1 << 20), "scale": FAKE + (2 << 20)}

    def write(q=f, k=f, v=f, qo=f, pos=f, cs=f, mp=9, sl=f, kc=None, vc=None, T=4, Hq=4, Hk=2, D=16, ldq=64, ldk=32,
              ldv=32, ldqo=64, pairing=0, fmt=0, io=BF16):
        kc, vc = kc or _cache(), vc or _cache(**own)
        return lib.gbln_rope_fwd_cache8(q, k, v, qo, pos, cs, mp, sl, ref(kc), ref(vc), T, Hq, Hk, D, ldq, ldk, ldv, ldqo,
                                        pairing, fmt, io, None)

    for shared in ("codes", "scale"):
        assert write(vc=_cache(**{**own, shared: FAKE})) == INVALID, shared
    assert write(vc=_cache()) == INVALID
    assert write(T=0, vc=_cache()) == OK  # nothing is written
    for kw in ({"q": None}, {"k": None}, {"v": None}, {"qo": None}, {"pos": None}, {"cs": None}, {"sl": None},
               {"cs": FAKE + 4}, {"sl": FAKE + 4}, {"mp": -1}, {"T": -1}, {"T": 1 << 34}, {"Hq": -1}, {"Hk": 0}, {"D": 7},
               {"D": 0}, {"ldq": 63}, {"ldk": 31}, {"ldv": 31}, {"ldqo": 63}, {"ldk": 1 << 60}, {"pairing": 2},
               {"fmt": 2}, {"io": 2}, {"Hq": 1 << 30, "ldq": 1 << 40, "ldqo": 1 << 40}):
        assert write(**kw) == INVALID, kw
    for bad in BAD_CACHES:
        assert write(kc=_cache(**bad)) == INVALID, bad
        assert write(vc=_cache(**{**own, **bad})) == INVALID, bad
    assert write(vc=_cache(pages=3, **own)) == INVALID
