"""Per-head norms, position axes and attention: the oracle's pins, the axis helper and the
refusals of the C entry points (decided on the host before any CUDA call).  CPU only."""

import ctypes

import numpy as np
import pytest

import oracle
from oracle import heads

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
F32, BF16 = 0, 1
FAKE = 0x10000  # never dereferenced


@pytest.fixture(scope="module")
def lib():
    from rmsnorm_fwd_bwd_03_gb300._build import build_library
    import rmsnorm_fwd_bwd_03_gb300 as gb
    build_library()
    return gb.library()


def _inputs(T=3, H=2, D=6, n=3, seed=0):
    r = np.random.default_rng(seed)
    axis = r.integers(0, n, D // 2)
    return r, r.normal(size=(T, H, D)), 1 + 0.1 * r.normal(size=D), r.integers(0, 9, (n, T)), axis


@pytest.mark.parametrize("pairing", ["half", "interleaved"])
def test_one_axis_is_the_plain_rotation(pairing):
    _, x, _, pos, _ = _inputs()
    np.testing.assert_allclose(heads.rotate(x, pos[:1], np.zeros(3, int), 1e4, pairing), oracle.rope_fwd(x, pos[0], 1e4, pairing), atol=1e-12)


def test_each_pair_turns_by_its_own_axis():
    _, x, _, pos, axis = _inputs()
    got = heads.rotate(x, pos, axis, 100.0)
    for t in range(3):
        for i in range(3):
            z = complex(x[t, 0, i], x[t, 0, i + 3]) * np.exp(1j * pos[axis[i], t] * 100.0 ** (-2 * i / 6))
            assert abs(complex(got[t, 0, i], got[t, 0, i + 3]) - z) < 1e-12


@pytest.mark.parametrize("pairing", ["half", "interleaved"])
def test_norm_rotate_is_the_norm_then_the_rotation(pairing):
    _, x, w, pos, axis = _inputs()
    y, _, _ = oracle.rmsnorm_fwd(x.reshape(-1, 6), None, w, 1e-3)
    np.testing.assert_allclose(heads.norm_rotate(x, w, pos, axis, 50.0, 1e-3, pairing), heads.rotate(y.reshape(x.shape), pos, axis, 50.0, pairing), atol=1e-12)


@pytest.mark.parametrize("pairing", ["half", "interleaved"])
def test_backward_is_the_difference_quotient(pairing):
    r, x, w, pos, axis = _inputs(T=2, H=2, D=4, n=2)
    dy = r.normal(size=x.shape)
    f = lambda x, w: np.sum(dy * heads.norm_rotate(x, w, pos, axis, 10.0, 1e-2, pairing))  # noqa: E731
    dx, dw = heads.norm_rotate_bwd(dy, x, w, pos, axis, 10.0, 1e-2, pairing)
    for a, g, call in ((x, dx, lambda v: f(v, w)), (w, dw, lambda v: f(x, v))):
        for i in np.ndindex(a.shape):
            e = np.zeros_like(a)
            e[i] = 1e-5
            assert abs((call(a + e) - call(a - e)) / 2e-5 - g[i]) < 1e-8


def test_attention_by_hand():
    # scores 0, ln 3 of the first row's two keys: weights 1/4, 3/4
    q, k = np.array([[[1.0]], [[1.0]]]), np.array([[[0.0]], [[np.log(3.0)]], [[np.log(4.0)]]])
    v = np.array([[[4.0]], [[8.0]], [[16.0]]])
    o, lse = heads.attend(q, k, v, 1.0, first=1)
    np.testing.assert_allclose(o[:, 0, 0], [7.0, (4 + 24 + 64) / 8])
    np.testing.assert_allclose(lse[:, 0], [np.log(4.0), np.log(8.0)])
    o, _ = heads.attend(q, k, v, 1.0, first=1, window=1)
    np.testing.assert_allclose(o[:, 0, 0], [8.0, 16.0])
    o, _ = heads.attend(q, k, v, 1.0, first=1, causal=False)
    np.testing.assert_allclose(o[:, 0, 0], [11.5, 11.5])
    o, lse = heads.attend(q, k, v, 1.0, first=-1)  # the first row stands before every key
    assert o[0, 0, 0] == 0 and lse[0, 0] == -np.inf and o[1, 0, 0] == 4.0


def test_attention_takes_nothing_from_masked_values():
    r = np.random.default_rng(1)
    q, k, v = r.normal(size=(2, 4, 8)), r.normal(size=(5, 2, 8)), r.normal(size=(5, 2, 8))
    o, _ = heads.attend(q, k, v, 0.3, first=2)
    k[4], v[4] = np.nan, np.inf
    o2, _ = heads.attend(q, k, v, 0.3, first=2)
    np.testing.assert_array_equal(o, o2)
    for h in range(4):  # heads in groups share keys and values
        p = np.exp(0.3 * q[1, h] @ k[:4, h // 2].T)
        np.testing.assert_allclose(o[1, h], p @ v[:4, h // 2] / p.sum(), atol=1e-12)


def test_axes_of_sections():
    import rmsnorm_fwd_bwd_03_gb300 as gb
    assert list(gb.rope_axes((1, 2, 1))) == [0, 1, 1, 2]
    assert list(gb.rope_axes((3, 1, 2), "cyclic")) == [0, 1, 2, 0, 2, 0]
    assert list(gb.rope_axes((0, 2))) == [1, 1]
    for bad in ((), (1, 1, 1, 1, 1), (2, -1)):
        with pytest.raises(ValueError):
            gb.rope_axes(bad)
    with pytest.raises(ValueError):
        gb.rope_axes((1, 1), "rows")


def _axis(D, *values):
    a = (ctypes.c_uint8 * (D // 2))(*values)
    return ctypes.addressof(a), a


def _rope(lib, fn="gbln_rope_axes_fwd", q=FAKE, k=FAKE, qo=FAKE, ko=FAKE, pos=FAKE, ldp=4, n=2, axis=(0, 1, 1, 0), tab=FAKE, T=4,
          Hq=2, Hk=1, D=8, ldq=16, ldk=8, ldqo=16, ldko=8, pairing=0, io=BF16):
    p, keep = _axis(8, *axis) if axis else (None, None)
    return getattr(lib, fn)(q, k, qo, ko, pos, ldp, n, p, tab, 5, T, Hq, Hk, D, ldq, ldk, ldqo, ldko, pairing, io, None)


@pytest.mark.parametrize("fn", ["gbln_rope_axes_fwd", "gbln_rope_axes_bwd"])
def test_rope_axes_rejects(lib, fn):
    bad = [dict(q=None), dict(k=None), dict(qo=None), dict(ko=None), dict(pos=None), dict(tab=None), dict(tab=FAKE + 4), dict(n=0), dict(n=5),
           dict(axis=None), dict(axis=(0, 1, 2, 0)), dict(ldp=3), dict(T=-1), dict(Hq=0), dict(Hk=-1), dict(D=7), dict(D=0), dict(D=514),
           dict(ldq=15), dict(ldk=7), dict(ldqo=15), dict(ldko=7), dict(pairing=2), dict(io=3)]
    for b in bad:
        assert _rope(lib, fn, **b) == INVALID, b
    assert _rope(lib, fn, T=0, q=None, k=None, qo=None, ko=None, pos=None, tab=None) == OK
    assert _rope(lib, fn, T=0, n=1, axis=None, Hk=0, k=None, ko=None) == OK


def _norm(lib, q=FAKE, k=FAKE, wq=FAKE, wk=FAKE, qo=FAKE, ko=FAKE, T=4, Hq=2, Hk=1, D=8, eps=1e-6, io=BF16, wt=BF16, ldq=16):
    return lib.gbln_qk_norm_rope_fwd(q, k, wq, wk, qo, ko, FAKE, 0, 1, None, FAKE, 5, T, Hq, Hk, D, ldq, 8, 16, 8, eps, 0, io, wt, None)


def test_qk_norm_rope_rejects(lib):
    for b in (dict(q=None), dict(k=None), dict(wq=None), dict(wk=None), dict(qo=None), dict(ko=None), dict(T=-1), dict(D=6, ldq=11),
              dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(Hq=0), dict(ldq=8)):
        assert _norm(lib, **b) == INVALID, b
    assert _norm(lib, io=F32, wt=BF16) == UNSUPPORTED
    assert _norm(lib, T=0) == OK

    def bwd(dq=FAKE, dk=FAKE, q=FAKE, part=FAKE, P=1 << 20, T=4, ldd=16, eps=1e-6, wt=BF16):
        return lib.gbln_qk_norm_rope_bwd(dq, dk, q, FAKE, FAKE, FAKE, FAKE, FAKE, part, P, FAKE, 0, 1, None, FAKE, 5, T, 2, 1, 8, ldd,
                                         8, 16, 8, 16, 8, eps, 0, BF16, wt, None)
    for b in (dict(dq=None), dict(dk=None), dict(q=None), dict(part=None), dict(part=FAKE + 2), dict(T=-1), dict(ldd=15), dict(eps=-1.0)):
        assert bwd(**b) == INVALID, b
    assert bwd(wt=7) == UNSUPPORTED
    assert bwd(T=0) == OK
    assert lib.gbln_qk_norm_rope_bwd_num_partials(0, 2, 1, 8) == 0
    assert lib.gbln_qk_norm_rope_bwd_num_partials(4, 2, 1, 7) == -1
    assert lib.gbln_qk_norm_rope_bwd_num_partials(-1, 2, 1, 8) == -1
    for a in ((None, 1, 8, FAKE, FAKE), (FAKE, -1, 8, FAKE, FAKE), (FAKE, 1, 0, FAKE, FAKE), (FAKE, 1, 8, None, FAKE), (FAKE, 1, 8, FAKE, None)):
        assert lib.gbln_qk_norm_dw_finalize(*a, 0, None) == INVALID


def test_qk_norm_rope_cache_rejects(lib):
    import rmsnorm_fwd_bwd_03_gb300 as gb

    def cache(codes=FAKE, scale=FAKE, pages=4, head=8):
        return gb._pack_cache8(codes, scale, pages, 16, 16 * head, head, head, 16, 1, 1)

    def call(q=FAKE, k=FAKE, v=FAKE, wq=FAKE, wk=FAKE, slots=FAKE, kc=cache(), vc=cache(FAKE * 2, FAKE * 2), T=4, Hq=2, Hk=1, eps=1e-6, fmt=0,
             ldv=8, wt=BF16):
        return lib.gbln_qk_norm_rope_fwd_cache8(q, k, v, wq, wk, FAKE, FAKE, 0, 1, None, FAKE, 5, slots, kc, vc, T, Hq, Hk, 8, 16, 8, ldv, 16,
                                                eps, 0, fmt, BF16, wt, None)
    for b in (dict(q=None), dict(k=None), dict(v=None), dict(wq=None), dict(wk=None), dict(slots=None), dict(slots=FAKE + 4), dict(kc=None),
              dict(vc=cache()), dict(vc=cache(FAKE * 2, FAKE * 2, 5)), dict(kc=cache(head=7)), dict(Hk=0), dict(eps=-1.0), dict(fmt=2), dict(ldv=7)):
        assert call(**b) == INVALID, b
    assert call(wt=5) == UNSUPPORTED
    assert call(T=0) == OK


def test_attention_rejects(lib):
    import rmsnorm_fwd_bwd_03_gb300 as gb

    def cache(codes=FAKE, scale=FAKE, pages=4, page=16, head=8):
        return gb._pack_cache8(codes, scale, pages, page, page * head, head, head, page, 1, 1)

    def call(q=FAKE, cu=FAKE, kv=FAKE, table=FAKE, most=4, kc=cache(), vc=cache(FAKE * 2, FAKE * 2), out=FAKE, lse=None, T=4, B=2, Hq=2, Hk=1,
             D=8, ldq=16, ldo=16, scale=1.0, window=0, fmt=0, io=BF16):
        return lib.gbln_attn_cache8(q, cu, kv, table, most, kc, vc, out, lse, None, 0, T, B, Hq, Hk, D, ldq, ldo, scale, 1, window, fmt, io, None)
    for b in (dict(q=None), dict(cu=None), dict(kv=None), dict(table=None), dict(out=None), dict(kc=None), dict(vc=None), dict(T=-1), dict(B=-1),
              dict(Hq=3, Hk=2), dict(Hk=0), dict(D=0), dict(D=513), dict(ldq=15), dict(ldo=15), dict(scale=float("nan")), dict(scale=float("inf")),
              dict(window=-1), dict(fmt=2), dict(io=4), dict(most=-1), dict(most=1 << 30), dict(vc=cache(pages=5)), dict(kc=cache(head=7)),
              dict(kc=cache(0)), dict(cu=FAKE + 2), dict(kv=FAKE + 1), dict(table=FAKE + 2), dict(lse=FAKE + 2), dict(T=1 << 30)):
        assert call(**b) == INVALID, b
    assert call(T=0) == OK and call(B=0, q=None) == OK
    assert lib.gbln_attn_cache8_workspace(4, 2, 3, 2, 64, BF16) == -1
    assert lib.gbln_attn_cache8_workspace(4, 2, 2, 1, 80, BF16) == 0
    assert lib.gbln_attn_cache8_workspace(0, 2, 2, 1, 64, BF16) == 0


def test_attention_scales_stay_finite_in_powers_of_two(lib):
    """The largest scale that is taken, times log2(e), is a float32; a larger one is refused."""
    import rmsnorm_fwd_bwd_03_gb300 as gb
    c = gb._pack_cache8(FAKE, FAKE, 4, 16, 128, 8, 8, 16, 1, 1), gb._pack_cache8(2 * FAKE, 2 * FAKE, 4, 16, 128, 8, 8, 16, 1, 1)
    call = lambda scale: lib.gbln_attn_cache8(None, None, None, None, 4, *c, None, None, None, 0, 0, 2, 2, 1, 8, 16, 16, scale, 1, 0, 0, BF16, None)  # noqa: E731
    for sign in (1.0, -1.0):
        assert call(sign * 2e38) == OK
        assert call(sign * 2.4e38) == INVALID
    assert np.float32(2e38) * np.float32(np.log2(np.e)) < np.inf
