"""GPU vs oracle for the row-scaled FP8 outputs and the 8-bit activation checkpoints
of RMSNorm and the gated units, forward and backward."""

import numpy as np
import pytest
import torch

import oracle
import rmsnorm_fwd_bwd_03_gb300 as gb
from oracle import q8
from rmsnorm_fwd_bwd_03_gb300 import autograd as ga

from _checks import Guarded, check_dw, check_io, check_rstd, dx_scale, sample_rows, to64
from _q8 import CODE, check_exact, check_window, codes64

pytestmark = pytest.mark.gpu

IO = {"f32": torch.float32, "bf16": torch.bfloat16}
TYPES = [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")]


@pytest.fixture(scope="module", autouse=True)
def _library():
    from rmsnorm_fwd_bwd_03_gb300._build import build_library
    build_library()
    gb.library()


def _randn(shape, dtype, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def _weight(H, dtype, seed=9):
    return (1 + 0.1 * _randn((H,), torch.float32, seed)).to(dtype)


def _unaligned(t):
    """The same values one element past a 16-byte boundary."""
    buf = torch.empty(t.numel() + 1, dtype=t.dtype, device=t.device)
    buf[1:] = t.reshape(-1)
    return buf[1:].view(t.shape)


def _same_bits(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


# One row group per warp, per two warps, per block of 64 to 512 threads; one value,
# odd widths, a short last checkpoint group, widths around the limits of the
# element path's registers (16384) and of the vector path's (8192 f32, 16384 bf16).
WIDTHS = [1, 2, 7, 32, 64, 127, 128, 129, 264, 513, 896, 1021, 1024, 2048, 4096, 5000, 8192]
WIDE = [8200, 16384, 16385, 16512, 20001]


def _norm_case(T, H, io, wt, residual, fmt, want_y=True, x=None, seed=0):
    dt = IO[io]
    eps = 1e-5
    x = _randn((T, H), dt, seed + 1) if x is None else x
    r = _randn((T, H), dt, seed + 2) if residual else None
    w = _weight(H, IO[wt])
    X, R, W = to64(x), None if r is None else to64(r), to64(w)
    c64, s64, y64, h64, rs64 = q8.rmsnorm_fwd_fp8(X, R, W, eps, io)

    y, yq, ys, h, rstd = gb.rmsnorm_fwd_fp8(x, w, eps, r, want_y=want_y)
    assert np.array_equal(to64(h), h64)
    check_rstd(to64(rstd), rs64)
    assert yq.dtype == torch.float8_e4m3fn and np.array_equal(codes64(yq), c64), "row-scaled codes"
    check_rstd(to64(ys), s64, "row scale")  # rstd's bound, and two roundings far below it
    if want_y:
        check_io(to64(y), y64, io, "y")
    else:
        assert y is None

    y, h, rstd, h8, hs = gb.rmsnorm_fwd_ckpt8(x, w, eps, r, fmt=fmt)
    assert np.array_equal(to64(h), h64)
    check_io(to64(y), y64, io, "y")
    check_rstd(to64(rstd), rs64)
    assert h8.dtype == CODE[fmt]
    check_exact(h8, hs, h64, fmt, f"h8 {T}x{H}", 128)

    dy, dres = _randn((T, H), dt, seed + 3), _randn((T, H), dt, seed + 4) if residual else None
    dx, part, P = gb.rmsnorm_bwd_ckpt8(dy, h8, hs, w, rstd, dres)
    dw = gb.rmsnorm_dw_finalize(part, P)
    kept = q8.values(codes64(h8), codes64(hs), 128)
    dx64, dw64 = q8.rmsnorm_bwd_kept(to64(dy), None if dres is None else to64(dres), kept, W, rs64)
    check_io(to64(dx), dx64, io, "dx", dx_scale(to64(dy), W, rs64, None if dres is None else to64(dres)))
    check_dw(to64(dw), dw64)
    assert gb.device_error() == 0


@pytest.mark.parametrize("io,wt", TYPES)
@pytest.mark.parametrize("H", WIDTHS)
def test_norm_widths(io, wt, H):
    # T: one row; more rows than a block holds, not a multiple of it
    fmt = "int8" if (H + len(io)) % 2 else "e4m3"
    _norm_case(1, H, io, wt, residual=H % 3 != 0, fmt=fmt, want_y=False)
    _norm_case(37, H, io, wt, residual=H % 3 != 1, fmt="e4m3" if fmt == "int8" else "int8")


@pytest.mark.parametrize("io,wt", TYPES)
@pytest.mark.parametrize("H", WIDE)
def test_norm_wide_rows(io, wt, H):
    _norm_case(5, H, io, wt, residual=True, fmt="int8")
    _norm_case(3, H, io, wt, residual=False, fmt="e4m3", want_y=False)


@pytest.mark.parametrize("T,H", [(5000, 128), (3001, 896), (2500, 1021), (1200, 4096), (700, 8192)])
def test_norm_many_rows(T, H):
    # several rows per block of the persistent backward
    _norm_case(T, H, "bf16", "bf16", residual=True, fmt="int8")


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("H", [96, 1024, 4096])
def test_norm_unaligned_pointers(io, H):
    T = 19
    x, r, dy, dres = (_unaligned(_randn((T, H), IO[io], s)) for s in range(4))
    w = _unaligned(_weight(H, IO[io]))
    aligned = [t.clone() for t in (x, r, dy, dres, w)]
    a = gb.rmsnorm_fwd_ckpt8(x, w, 1e-5, r)
    b = gb.rmsnorm_fwd_ckpt8(aligned[0], aligned[4], 1e-5, aligned[1])
    for p, q in zip(a[1:2] + a[3:], b[1:2] + b[3:]):
        assert _same_bits(p, q)  # h, h8 and its scale do not depend on the path
    h64 = to64(a[1])
    W, rs64 = to64(w), 1 / np.sqrt((h64 ** 2).mean(-1) + 1e-5)
    check_io(to64(a[0]), W * h64 * rs64[:, None], io, "y")
    h8 = _unaligned(a[3].view(torch.uint8)).view(a[3].dtype)  # codes at an odd address
    dx, part, P = gb.rmsnorm_bwd_ckpt8(dy, h8, a[4], w, a[2], dres)
    dx64, dw64 = q8.rmsnorm_bwd_kept(to64(dy), to64(dres), q8.values(codes64(a[3]), codes64(a[4]), 128), W, rs64)
    check_io(to64(dx), dx64, io, "dx")
    check_dw(to64(gb.rmsnorm_dw_finalize(part, P)), dw64)
    _, yq, ys, _, _ = gb.rmsnorm_fwd_fp8(x, w, 1e-5, r)
    _, yq2, ys2, _, _ = gb.rmsnorm_fwd_fp8(aligned[0], aligned[4], 1e-5, aligned[1])
    assert _same_bits(yq, yq2)


def test_norm_outlier_channels_and_special_rows():
    # one channel in a hundred fifty times as large; an all-zero row, a tiny one, a
    # huge one, rows with an infinity and with a NaN
    T, H, io = 64, 1024, "bf16"
    x = _randn((T, H), torch.bfloat16, 1)
    x[:, ::100] *= 50
    x[3] = 0
    x[4] = 2.0 ** -110
    x[5] *= 2.0 ** 40
    _norm_case(T, H, io, "bf16", residual=False, fmt="e4m3", x=x)
    _norm_case(T, H, io, "bf16", residual=False, fmt="int8", x=x)
    x[6, 17] = float("inf")
    x[7, 1000] = float("nan")
    w = _weight(H, torch.bfloat16)
    _, yq, ys, _, _ = gb.rmsnorm_fwd_fp8(x, w, 1e-5)
    val = codes64(yq) * codes64(ys)[:, None]
    assert np.isnan(val[6:8]).all() and np.isfinite(np.delete(val, [6, 7], 0)).all()
    for fmt in ("int8", "e4m3"):
        _, _, _, h8, hs = gb.rmsnorm_fwd_ckpt8(x, w, 1e-5, fmt=fmt)
        kept = q8.values(codes64(h8), codes64(hs), 128)
        assert np.isnan(kept[6, :128]).all() and np.isnan(kept[7, 896:]).all()  # their groups, and no other
        kept[6, :128] = kept[7, 896:] = 0
        assert np.isfinite(kept).all()


@pytest.mark.parametrize("io,H", [("bf16", 1024), ("bf16", 4096), ("f32", 256), ("bf16", 777)])
def test_norm_aliases_and_guards(io, H):
    # residual_out over x or residual, dx over dy or dres; nothing outside the outputs is written
    T, dt = 33, IO[io]
    x, r, dy, dres = (_randn((T, H), dt, s) for s in (1, 2, 3, 4))
    w = _weight(H, dt)
    want = gb.rmsnorm_fwd_ckpt8(x, w, 1e-5, r)
    for target in (0, 1):
        a, b = x.clone(), r.clone()
        got = gb.rmsnorm_fwd_ckpt8(a, w, 1e-5, b, residual_out=(a, b)[target])
        for p, q in zip(got, want):
            assert _same_bits(p, q)
    dx, part, P = gb.rmsnorm_bwd_ckpt8(dy, want[3], want[4], w, want[2], dres)
    for target in (0, 1):
        a, b = dy.clone(), dres.clone()
        got, part2, _ = gb.rmsnorm_bwd_ckpt8(a, want[3], want[4], w, want[2], b, dx=(a, b)[target])
        assert _same_bits(got, dx) and _same_bits(part2[:P], part[:P])
    lib, s = gb.library(), torch.cuda.current_stream().cuda_stream
    io_ = 1 if io == "bf16" else 0
    ng = -(-H // 128)
    g = {n: Guarded(sh, d) for n, sh, d in (("y", (T, H), dt), ("h", (T, H), dt), ("rstd", (T,), torch.float32),
                                            ("q", (T, H), torch.uint8), ("sc", (T, ng), torch.float32),
                                            ("dx", (T, H), dt), ("part", (P, H), torch.float32))}
    p = {n: t.tensor.data_ptr() for n, t in g.items()}
    assert lib.gbln_rmsnorm_fwd_ckpt8(x.data_ptr(), r.data_ptr(), w.data_ptr(), p["y"], p["h"], p["rstd"], p["q"], p["sc"],
                                      T, H, 1e-5, 0, io_, io_, s) == 0
    assert lib.gbln_rmsnorm_bwd_ckpt8(dy.data_ptr(), dres.data_ptr(), p["q"], p["sc"], w.data_ptr(), p["rstd"], p["dx"],
                                      p["part"], P, T, H, 0, io_, io_, s) == 0
    torch.cuda.synchronize()
    assert all(t.intact() for t in g.values())
    assert _same_bits(g["q"].tensor, want[3].view(torch.uint8)) and _same_bits(g["dx"].tensor, dx)
    assert lib.gbln_rmsnorm_bwd_ckpt8(dy.data_ptr(), None, p["q"], p["sc"], w.data_ptr(), p["rstd"], p["dx"],
                                      p["part"], P - 1, T, H, 0, io_, io_, s) == 3  # GBLN_ERR_WORKSPACE
    assert lib.gbln_rmsnorm_fwd_fp8(x.data_ptr(), r.data_ptr(), w.data_ptr(), None, p["q"], p["sc"], p["h"], p["rstd"],
                                    T, H, 1e-5, io_, io_, s) == 0
    torch.cuda.synchronize()
    assert all(t.intact() for t in g.values())


# ---------------------------------------------------------------------------
# Gated units
# ---------------------------------------------------------------------------

def _glu_window(act, g, u, io):
    """How far a float32 gated unit may be from the exact one: relative 1e-5 (the float32
    bound of this library), and for the erf form also 1e-5 of |g u| where x Phi(x) cancels."""
    out = q8.glu_out(act, g, u)
    return 1e-5 * np.abs(out) + (1e-5 * np.abs(g * u) if act == "gelu_erf" else 0.0)


def _glu_case(T, I, io, act, fmt, packed, unaligned=False, seed=0):
    dt = IO[io]
    if packed:
        gate, up = _randn((T, 2 * I + (1 if unaligned else 0)), dt, seed + 1)[:, (1 if unaligned else 0):].chunk(2, dim=-1)
    else:
        gate, up = _randn((T, I), dt, seed + 1), _randn((T, I), dt, seed + 2)
        if unaligned:
            gate, up = _unaligned(gate), _unaligned(up)
    G, U = to64(gate), to64(up)
    q, s = gb.glu_fwd_fp8(gate, up, act)
    assert q.dtype == torch.float8_e4m3fn and tuple(s.shape) == (T,)
    check_window(q, s, q8.glu_out(act, G, U), _glu_window(act, G, U, io), "e4m3", f"glu fp8 {T}x{I} {act}")
    out, gq, gs, uq, us = gb.glu_fwd_ckpt8(gate, up, act, fmt=fmt)
    check_io(to64(out), q8.glu_out(act, G, U), io, "out")
    check_exact(gq, gs, G, fmt, "gate8", 128)
    check_exact(uq, us, U, fmt, "up8", 128)
    dout = _randn((T, I), dt, seed + 3)
    if unaligned:
        dout = _unaligned(dout)
    KG, KU = q8.values(codes64(gq), codes64(gs), 128), q8.values(codes64(uq), codes64(us), 128)
    dg64, du64 = oracle.glu_bwd(act, to64(dout), KG, KU)
    dgate, dup = gb.glu_bwd_ckpt8(dout, gq, gs, uq, us, act)
    check_io(to64(dgate), dg64, io, "dgate")
    check_io(to64(dup), du64, io, "dup")
    if packed:  # one packed gradient
        both = torch.empty((T, 2 * I), dtype=dt, device="cuda")
        a, b = both.chunk(2, dim=-1)
        gb.glu_bwd_ckpt8(dout, gq, gs, uq, us, act, dgate=a, dup=b)
        assert _same_bits(a, dgate) and _same_bits(b, dup)
    return out, (gq, gs, uq, us), dgate, dup


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("I", [1, 8, 100, 128, 136, 512, 1000, 1023, 2048, 4864, 8192])
def test_glu_widths(io, I):
    acts = list(gb.ACT)
    for k, (T, packed) in enumerate(((1, True), (2, False), (7, True), (33, False))):
        _glu_case(T, I, io, acts[(I + k) % 4], ("int8", "e4m3")[k % 2], packed)


@pytest.mark.parametrize("act", list(gb.ACT))
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_glu_activations(act, fmt):
    for io in ("bf16", "f32"):
        _glu_case(65, 640, io, act, fmt, packed=True)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("I", [14336, 16384, 16392, 28672, 32768, 32776, 40001])
def test_glu_wide_rows(io, I):
    _glu_case(3, I, io, "silu", "int8", packed=True)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("packed", [False, True])
def test_glu_unaligned(io, packed):
    _glu_case(17, 264, io, "silu", "int8", packed, unaligned=True)


def test_glu_out_over_its_inputs_and_dgate_over_dout():
    T, I = 40, 1024
    for n in (I, I - 1):
        gate, up, dout = (_randn((T, n), torch.bfloat16, s) for s in (1, 2, 3))
        want = gb.glu_fwd_ckpt8(gate, up)
        for target in (0, 1):
            a, b = gate.clone(), up.clone()
            for p, q in zip(gb.glu_fwd_ckpt8(a, b, out=(a, b)[target]), want):
                assert _same_bits(p, q)
        dg, du = gb.glu_bwd_ckpt8(dout, *want[1:])
        for name in ("dgate", "dup"):
            d = dout.clone()
            p, q = gb.glu_bwd_ckpt8(d, *want[1:], **{name: d})
            assert _same_bits(p, dg) and _same_bits(q, du)


def test_glu_special_rows():
    T, I = 6, 512
    gate, up = _randn((T, I), torch.bfloat16, 1), _randn((T, I), torch.bfloat16, 2)
    gate[0] = 0                    # out = 0
    gate[1] = -200                 # silu underflows to -0
    up[2, 7] = float("inf")
    gate[3, 300] = float("nan")
    up[4] = 3e38                   # finite inputs whose product may overflow
    q, s = gb.glu_fwd_fp8(gate, up)
    v = codes64(q) * codes64(s)[:, None]
    assert (v[:2] == 0).all() and np.isnan(v[2]).all() and np.isnan(v[3]).all() and np.isfinite(v[5]).all()
    for fmt in ("int8", "e4m3"):
        _, gq, gs, uq, us = gb.glu_fwd_ckpt8(gate, up, fmt=fmt)
        kg, ku = q8.values(codes64(gq), codes64(gs), 128), q8.values(codes64(uq), codes64(us), 128)
        assert np.isnan(ku[2, :128]).all() and np.isfinite(ku[2, 128:]).all()
        assert np.isnan(kg[3, 256:384]).all() and np.isfinite(kg[3, :256]).all() and np.isfinite(kg[3, 384:]).all()
        assert (kg[0] == 0).all() and np.allclose(kg[1], -200) and np.allclose(ku[4], 3e38, rtol=2.0 ** -8)


# ---------------------------------------------------------------------------
# Large sizes (sampled rows), differences, autograd, graphs and streams
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("T,I", [(8193, 14336), (2047, 28672)])
def test_glu_large(T, I):
    gate, up = _randn((T, 2 * I), torch.bfloat16, 1).chunk(2, dim=-1)
    dout = _randn((T, I), torch.bfloat16, 2)
    q, s = gb.glu_fwd_fp8(gate, up)
    out, gq, gs, uq, us = gb.glu_fwd_ckpt8(gate, up)
    dgate, dup = gb.glu_bwd_ckpt8(dout, gq, gs, uq, us)
    for r in sample_rows(T, 20):
        r = slice(int(r), int(r) + 1)
        G, U = to64(gate[r]), to64(up[r])
        check_window(q[r], s[r], q8.glu_out("silu", G, U), _glu_window("silu", G, U, "bf16"), "e4m3", "glu fp8")
        check_io(to64(out[r]), q8.glu_out("silu", G, U), "bf16", "out")
        check_exact(gq[r], gs[r], G, "int8", "gate8", 128)
        check_exact(uq[r], us[r], U, "int8", "up8", 128)
        dg, du = oracle.glu_bwd("silu", to64(dout[r]), q8.values(codes64(gq[r]), codes64(gs[r]), 128),
                                q8.values(codes64(uq[r]), codes64(us[r]), 128))
        check_io(to64(dgate[r]), dg, "bf16", "dgate")
        check_io(to64(dup[r]), du, "bf16", "dup")


def test_norm_large():
    T, H = 33001, 4096
    x, r, dy, dres = (_randn((T, H), torch.bfloat16, s) for s in range(4))
    w = _weight(H, torch.bfloat16)
    y, h, rstd, h8, hs = gb.rmsnorm_fwd_ckpt8(x, w, 1e-5, r, fmt="e4m3")
    dx, part, P = gb.rmsnorm_bwd_ckpt8(dy, h8, hs, w, rstd, dres)
    dw = gb.rmsnorm_dw_finalize(part, P)
    W = to64(w)
    for t in sample_rows(T, 20):
        t = slice(int(t), int(t) + 1)
        c, s, y64, h64, rs = q8.rmsnorm_fwd_fp8(to64(x[t]), to64(r[t]), W, 1e-5, "bf16")
        assert np.array_equal(to64(h[t]), h64)
        check_io(to64(y[t]), y64, "bf16", "y")
        check_exact(h8[t], hs[t], h64, "e4m3", "h8", 128)
        kept = q8.values(codes64(h8[t]), codes64(hs[t]), 128)
        check_io(to64(dx[t]), q8.rmsnorm_bwd_kept(to64(dy[t]), to64(dres[t]), kept, W, rs)[0], "bf16", "dx")
    dw64 = torch.zeros(H, dtype=torch.float64, device="cuda")
    for i in range(0, T, 4096):
        n = h8[i:i + 4096].double() * hs[i:i + 4096].double().repeat_interleave(128, 1)
        hh = h[i:i + 4096].double()
        dw64 += (dy[i:i + 4096].double() * n / torch.sqrt(hh.square().mean(-1, keepdim=True) + 1e-5)).sum(0)
    check_dw(to64(dw), dw64.cpu().numpy())


def _lattice(T, N, seed):
    """Float32 values that an INT8 checkpoint keeps exactly: multiples of 2^-5, the largest of
    each group 127 * 2^-5 (scale 2^-5)."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    v = torch.randint(-100, 101, (T, N), generator=g, device="cuda").float()
    v[:, ::128] = 127
    return v / 32


def test_gradients_against_differences():
    # where the checkpoint keeps its input exactly, the gradients are those of the
    # exact function: central differences of the oracle's float64 forward.  Step 1e-4:
    # truncation d^2/6 * f''' ~ 1e-8, cancellation 1e-16 * 1e3 / 1e-4 ~ 1e-9; float32
    # outputs are held to 1e-5 of the largest as everywhere.
    T, H, d = 3, 140, 1e-4
    x, w = _lattice(T, H, 1), _weight(H, torch.float32)
    dy = _randn((T, H), torch.float32, 2)
    y, h, rstd, h8, hs = gb.rmsnorm_fwd_ckpt8(x, w, 1e-5)
    assert np.array_equal(q8.values(codes64(h8), codes64(hs), 128), to64(x))
    dx, part, P = gb.rmsnorm_bwd_ckpt8(dy, h8, hs, w, rstd)
    dw = gb.rmsnorm_dw_finalize(part, P)
    X, W, DY = to64(x), to64(w), to64(dy)
    num = np.zeros((T, H))
    numw = np.zeros(H)
    for j in range(H):
        e = np.zeros(H)
        e[j] = d
        num[:, j] = (DY * (oracle.rmsnorm_fwd(X + e, None, W, 1e-5)[0] - oracle.rmsnorm_fwd(X - e, None, W, 1e-5)[0])).sum(-1) / (2 * d)
        numw[j] = (DY * (oracle.rmsnorm_fwd(X, None, W + e, 1e-5)[0] - oracle.rmsnorm_fwd(X, None, W - e, 1e-5)[0])).sum() / (2 * d)
    check_io(to64(dx), num, "f32", "dx")
    check_dw(to64(dw), numw)
    gate, up = _lattice(T, H, 3), _lattice(T, H, 4)
    for act in ("silu", "gelu_tanh", "gelu_erf"):
        _, *saved = gb.glu_fwd_ckpt8(gate, up, act)
        dg, du = gb.glu_bwd_ckpt8(dy, *saved, act)
        G, U = to64(gate), to64(up)
        check_io(to64(dg), DY * (q8.glu_out(act, G + d, U) - q8.glu_out(act, G - d, U)) / (2 * d), "f32", "dgate")
        check_io(to64(du), DY * (q8.glu_out(act, G, U + d) - q8.glu_out(act, G, U - d)) / (2 * d), "f32", "dup")


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_autograd_layer_with_checkpoints(fmt):
    # residual add + norm, a packed projection, the gated unit, a second projection: the
    # gradients that arrive at each operator are passed through the oracle's backward.
    T, H, I, dt = 70, 264, 200, torch.bfloat16
    x, r = (_randn((2, T // 2, H), dt, s).requires_grad_() for s in (1, 2))
    w = _weight(H, dt).requires_grad_()
    wgu = (_randn((H, 2 * I), dt, 3) / H ** 0.5).requires_grad_()
    y, h = ga.rms_norm(x, w, 1e-5, r, checkpoint=fmt)
    y0, h0 = ga.rms_norm(x, w, 1e-5, r)
    check_io(to64(y), oracle.rmsnorm_fwd(to64(x), to64(r), to64(w), 1e-5, "bf16")[0], "bf16", "y")
    assert torch.equal(h, h0)
    gate, up = (y @ wgu).chunk(2, dim=-1)
    gate.retain_grad(), up.retain_grad(), y.retain_grad()
    out = ga.swiglu(gate, up, checkpoint=fmt)
    check_io(to64(out), q8.glu_out("silu", to64(gate), to64(up)), "bf16", "out")
    co, ch = _randn(out.shape, dt, 5), _randn(h.shape, dt, 6)
    torch.autograd.backward([out, h], [co, ch])

    def kept(t, n):
        v = to64(t).reshape(-1, n)
        return q8.values(*q8.quantize(v, fmt, 128), 128)
    dg, du = oracle.glu_bwd("silu", to64(co).reshape(-1, I), kept(gate, I), kept(up, I))
    check_io(to64(gate.grad).reshape(-1, I), dg, "bf16", "dgate")
    check_io(to64(up.grad).reshape(-1, I), du, "bf16", "dup")
    H64 = to64(h).reshape(-1, H)
    rs = 1 / np.sqrt((H64 ** 2).mean(-1) + 1e-5)
    dx, dw = q8.rmsnorm_bwd_kept(to64(y.grad).reshape(-1, H), to64(ch).reshape(-1, H), kept(h, H), to64(w), rs)
    check_io(to64(x.grad).reshape(-1, H), dx, "bf16", "dx")
    assert torch.equal(x.grad, r.grad) and w.grad.dtype == dt
    check_io(to64(w.grad), dw, "bf16", "dw")
    assert wgu.grad is not None


def test_autograd_saves_less_and_handles_partial_use():
    T, H = 256, 4096
    x = _randn((T, H), torch.bfloat16, 1).requires_grad_()
    w = _weight(H, torch.bfloat16).requires_grad_()
    saved = []
    with torch.autograd.graph.saved_tensors_hooks(lambda t: saved.append(t) or t, lambda t: t):
        y = ga.rms_norm(x, w, 1e-5, checkpoint="int8")
        out = ga.swiglu(*y.chunk(2, dim=-1), checkpoint="e4m3")
    big = [t for t in saved if t.numel() >= T * H // 2]
    assert {t.dtype for t in big} == {torch.int8, torch.float8_e4m3fn}  # nothing of that size in 16 bits
    out.sum().backward()  # an expanded upstream gradient
    assert torch.isfinite(x.grad).all()
    # only the residual stream used: the norm passes its gradient on
    r = _randn((T, H), torch.bfloat16, 2).requires_grad_()
    x2 = x.detach().clone().requires_grad_()
    _, h = ga.rms_norm(x2, w, 1e-5, r, checkpoint="int8")
    g = _randn((T, H), torch.bfloat16, 3)
    h.backward(g)
    assert torch.equal(x2.grad, g) and torch.equal(r.grad, g)
    with pytest.raises(RuntimeError):  # no second derivatives
        x3 = x.detach().clone().requires_grad_()
        y = ga.rms_norm(x3, w, 1e-5, checkpoint="int8")
        (gx,) = torch.autograd.grad(y.float().square().sum(), x3, create_graph=True)
        gx.float().sum().backward()


def _step(s):
    y, h, rstd, h8, hs = gb.rmsnorm_fwd_ckpt8(s["x"], s["w"], 1e-5, s["r"], y=s["y"], residual_out=s["h"])
    out, *kept = gb.glu_fwd_ckpt8(*y.chunk(2, dim=-1), out=s["out"])
    dg, du = gb.glu_bwd_ckpt8(s["dout"], *kept)
    dx, part, P = gb.rmsnorm_bwd_ckpt8(torch.cat([dg, du], dim=-1), h8, hs, s["w"], rstd, s["dres"])
    q, qs = gb.glu_fwd_fp8(*y.chunk(2, dim=-1))
    _, yq, ys, _, _ = gb.rmsnorm_fwd_fp8(s["x"], s["w"], 1e-5, s["r"], want_y=False)
    return [y, h, out, dg, du, dx, gb.rmsnorm_dw_finalize(part, P), q, qs, yq, ys]


@pytest.mark.parametrize("T,H", [(1, 4096), (300, 1024), (65, 1022)])
def test_graph_replay_and_side_stream_give_the_same_bits(T, H):
    dt = torch.bfloat16

    def state(seed):
        s = {n: _randn((T, H), dt, seed + i) for i, n in enumerate(("x", "r", "dres", "y", "h"))}
        return s | {"w": _weight(H, dt), "dout": _randn((T, H // 2), dt, seed + 7), "out": _randn((T, H // 2), dt, 0)}
    a, b = state(1), state(50)
    want_a, want_b = [t.clone() for t in _step(a)], [t.clone() for t in _step(b)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = _step(a)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    for p, q in zip(got, want_a):
        assert _same_bits(p, q)
    # two graphs captured from different states share nothing
    graphs = []
    for s in (a, b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = _step(s)
        graphs.append((g, out))
    for _ in range(2):
        for g, _o in graphs:
            g.replay()
    torch.cuda.synchronize()
    for (_g, out), want in zip(graphs, (want_a, want_b)):
        for p, q in zip(out, want):
            assert _same_bits(p, q)
    a["x"].copy_(b["x"])  # new inputs in place are what the replay sees
    graphs[0][0].replay()
    torch.cuda.synchronize()
    for p, q in zip(graphs[0][1], _step(a)):
        assert _same_bits(p, q)


def test_empty_inputs():
    x, w = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda"), _weight(64, torch.bfloat16)
    _, q, s, _, _ = gb.rmsnorm_fwd_fp8(x, w, 1e-5)
    assert q.shape == (0, 64) and s.shape == (0,)
    y, h, rstd, h8, hs = gb.rmsnorm_fwd_ckpt8(x, w, 1e-5)
    dx, part, P = gb.rmsnorm_bwd_ckpt8(x, h8, hs, w, rstd)
    assert dx.shape == (0, 64) and P == 0 and (gb.rmsnorm_dw_finalize(part, P) == 0).all()
    out, *kept = gb.glu_fwd_ckpt8(x, x)
    assert out.shape == (0, 64) and gb.glu_bwd_ckpt8(x, *kept)[0].shape == (0, 64)
    assert gb.glu_fwd_fp8(x, x)[0].shape == (0, 64)


def test_more_than_two_to_the_31_values():
    # element offsets pass 32 bits: rows on both sides of the border
    T, I = 150001, 14336  # 2.15e9 values
    gate = torch.empty((T, I), dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    gate.normal_(generator=g)
    out, gq, gs, uq, us = gb.glu_fwd_ckpt8(gate, gate, "relu")
    q, s = gb.glu_fwd_fp8(gate, gate, "relu")
    rows = [0, 74898, 74899, 149796, 149797, T - 1]  # 2^30 / I, 2^31 / I
    for r in rows:
        r = slice(r, r + 1)
        G = to64(gate[r])
        check_exact(gq[r], gs[r], G, "int8", "gate8", 128)
        check_exact(uq[r], us[r], G, "int8", "up8", 128)
        v = q8.glu_out("relu", G, G)
        check_io(to64(out[r]), v, "bf16", "out")
        check_window(q[r], s[r], v, 2.0 ** -23 * np.abs(v), "e4m3", "fp8")
    dgate, dup = gb.glu_bwd_ckpt8(out, gq, gs, uq, us, "relu")
    for r in rows:
        r = slice(r, r + 1)
        k = q8.values(codes64(gq[r]), codes64(gs[r]), 128)
        dg, du = oracle.glu_bwd("relu", to64(out[r]), k, k)
        check_io(to64(dgate[r]), dg, "bf16", "dgate")
        check_io(to64(dup[r]), du, "bf16", "dup")


def test_captured_training_step_matches_eager():
    # forward, backward and dW of a norm and a gated unit with checkpoints, through
    # autograd, captured once and replayed on new inputs
    T, H, dt = 96, 512, torch.bfloat16
    x = _randn((T, H), dt, 1).requires_grad_()
    r = _randn((T, H), dt, 2).requires_grad_()
    w = _weight(H, dt).requires_grad_()
    cy, ch = _randn((T, H // 2), dt, 3), _randn((T, H), dt, 4)
    leaves = (x, r, w)

    def step():
        y, h = ga.rms_norm(x, w, 1e-5, r, checkpoint="int8")
        out = ga.swiglu(*y.chunk(2, dim=-1), checkpoint="e4m3")
        return torch.autograd.grad([out, h], leaves, [cy, ch])

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        grads = step()
    for seed in (10, 20):
        with torch.no_grad():
            x.copy_(_randn((T, H), dt, seed))
            r.copy_(_randn((T, H), dt, seed + 1))
            cy.copy_(_randn((T, H // 2), dt, seed + 2))
        graph.replay()
        torch.cuda.synchronize()
        got = [g.clone() for g in grads]
        for a, b in zip(got, step()):
            assert _same_bits(a, b)


def test_fp8_operands_through_a_layer():
    # norm -> projection -> gated unit -> projection, the projections on the E4M3 operands
    # and their row scales (float64 products of the values they stand for)
    T, H, I = 40, 256, 384
    x, r = _randn((T, H), torch.bfloat16, 1), _randn((T, H), torch.bfloat16, 2)
    w = _weight(H, torch.bfloat16)
    w1, w2 = _randn((H, 2 * I), torch.float32, 3).double() / H ** 0.5, _randn((I, H), torch.float32, 4).double() / I ** 0.5
    _, y8, ys, h, _ = gb.rmsnorm_fwd_fp8(x, w, 1e-5, r, want_y=False)
    gate_up = ((y8.double() @ w1) * ys.double()[:, None]).to(torch.bfloat16)
    o8, os_ = gb.glu_fwd_fp8(*gate_up.chunk(2, dim=-1))
    got = to64((o8.double() @ w2) * os_.double()[:, None])
    # each operand is within 2^-4 of its value (normal E4M3 range), so is every term of a product:
    # the first projection's error passes a slope of at most 1.1 (silu) and a factor up
    y64 = q8.rmsnorm_fwd_fp8(to64(x), to64(r), to64(w), 1e-5, "bf16")[2]
    W1, W2 = w1.cpu().numpy(), w2.cpu().numpy()
    gu = y64 @ W1
    G, U = gu[:, :I], gu[:, I:]
    dgu = (2.0 ** -4 + 2.0 ** -8) * (np.abs(y64) @ np.abs(W1)) + 2.0 ** -8 * np.abs(gu)
    out = q8.glu_out("silu", G, U)
    f = oracle.act("silu", G)
    dout = 1.1 * dgu[:, :I] * (np.abs(U) + dgu[:, I:]) + np.abs(f) * dgu[:, I:]
    dout = dout + (2.0 ** -4 + 2.0 ** -8) * (np.abs(out) + dout) + np.abs(out).max(-1, keepdims=True) / 448 * 2.0 ** -9
    assert (np.abs(got - out @ W2) <= dout @ np.abs(W2)).all()


def test_backward_is_reproducible_and_accumulates():
    for T, H in ((3000, 640), (700, 4096), (500, 1023), (40, 20001)):
        dt = torch.bfloat16
        x, dy = _randn((T, H), dt, 1), _randn((T, H), dt, 2)
        w = _weight(H, dt)
        _, _, rstd, h8, hs = gb.rmsnorm_fwd_ckpt8(x, w, 1e-5)
        dx, part, P = gb.rmsnorm_bwd_ckpt8(dy, h8, hs, w, rstd)
        dw = gb.rmsnorm_dw_finalize(part, P)
        for _ in range(3):
            dx2, part2, _ = gb.rmsnorm_bwd_ckpt8(dy, h8, hs, w, rstd)
            assert _same_bits(dx, dx2) and _same_bits(dw, gb.rmsnorm_dw_finalize(part2, P))
        acc = gb.rmsnorm_dw_finalize(part, P, dw=dw.clone(), accumulate=True)
        assert torch.equal(acc, dw + dw)
        assert P == gb.rmsnorm_bwd_ckpt8_num_partials(T, H, dt)


def test_norm_of_more_than_two_to_the_31_values():
    T, H = 150001, 14336
    x = torch.empty((T, H), dtype=torch.bfloat16, device="cuda")
    x.normal_(generator=torch.Generator(device="cuda").manual_seed(2))
    w = _weight(H, torch.bfloat16)
    y, _, rstd, h8, hs = gb.rmsnorm_fwd_ckpt8(x, w, 1e-5, fmt="e4m3")
    _, yq, ys, _, _ = gb.rmsnorm_fwd_fp8(x, w, 1e-5, want_y=False)
    dx, part, P = gb.rmsnorm_bwd_ckpt8(x, h8, hs, w, rstd, x)
    W = to64(w)
    for t in (0, 74898, 74899, 149796, 149797, T - 1):
        t = slice(t, t + 1)
        X = to64(x[t])
        c, s, y64, _, rs = q8.rmsnorm_fwd_fp8(X, None, W, 1e-5)
        check_io(to64(y[t]), y64, "bf16", "y")
        assert np.array_equal(codes64(yq[t]), c)
        check_rstd(to64(ys[t]), s)
        check_exact(h8[t], hs[t], X, "e4m3", "h8", 128)
        kept = q8.values(codes64(h8[t]), codes64(hs[t]), 128)
        check_io(to64(dx[t]), q8.rmsnorm_bwd_kept(X, X, kept, W, rs)[0], "bf16", "dx")


def test_two_streams_at_once():
    T, H = 2000, 2048
    states = []
    for seed in (1, 100):
        s = {n: _randn((T, H), torch.bfloat16, seed + i) for i, n in enumerate(("x", "r", "dres", "y", "h"))}
        s |= {"w": _weight(H, torch.bfloat16), "dout": _randn((T, H // 2), torch.bfloat16, seed + 7), "out": _randn((T, H // 2), torch.bfloat16, 0)}
        states.append((s, [t.clone() for t in _step(s)]))
    streams = [torch.cuda.Stream() for _ in states]
    torch.cuda.synchronize()
    got = []
    for st, (s, _) in zip(streams, states):
        with torch.cuda.stream(st):
            got.append(_step(s))
    torch.cuda.synchronize()
    for g, (_, want) in zip(got, states):
        for p, q in zip(g, want):
            assert _same_bits(p, q)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("act", list(gb.ACT))
def test_gated_units_give_the_same_bits_on_every_path(io, act):
    # out of the forward that saves checkpoints is glu_fwd's, and the row-scaled codes do not
    # depend on alignment; 20000 and 28672: unaligned rows are read twice
    for T, I in ((2001, 1024), (301, 5000), (300, 20000), (200, 28672)):
        gate, up = 2 * _randn((T, I), IO[io], 1), _randn((T, I), IO[io], 2)
        want = gb.glu_fwd(gate, up, act)
        q, s = gb.glu_fwd_fp8(gate, up, act)
        for g, u in ((gate, up), (_unaligned(gate), _unaligned(up))):
            assert _same_bits(gb.glu_fwd(g, u, act), want)
            assert _same_bits(gb.glu_fwd_ckpt8(g, u, act)[0], want)
            q2, s2 = gb.glu_fwd_fp8(g, u, act)
            assert _same_bits(q2, q) and _same_bits(s2, s)


@pytest.mark.parametrize("io,wt", TYPES)
@pytest.mark.parametrize("H", [64, 896, 1021, 4095, 4096, 8200, 16384, 20001])
def test_norm_outputs_beside_the_plain_forward(io, wt, H):
    # h to the bit.  rstd: the row's sum of squares takes at most 60 float32 additions in a row in any of
    # the kernels (all terms positive: 60 * 2^-24 of it, half of that in rstd), the mean, eps and rsqrt
    # another 6 * 2^-24: two kernels are within 2 * 36 * 2^-24 < 2^-17 of one another.  y adds two
    # roundings, and at bf16 the final one may fall to the neighbour: 2^-7 of the value.
    T, dt = 61, IO[io]
    x, r, w = _randn((T, H), dt, 1), _randn((T, H), dt, 2), _weight(H, IO[wt])
    tol_y = 2.0 ** -16 if io == "f32" else 2.0 ** -7 + 2.0 ** -14
    for unaligned in (False, True):
        a, b, c = (_unaligned(t) if unaligned else t for t in (x, r, w))
        for res in (None, b):
            y0, h0, rstd0 = gb.rmsnorm_fwd(a, c, 1e-5, res)
            H64 = to64(h0)
            ref = 1 / np.sqrt((H64 ** 2).mean(-1) + 1e-5)
            y1, h1, rstd1, _, _ = gb.rmsnorm_fwd_ckpt8(a, c, 1e-5, res)
            y2, yq, ys, h2, rstd2 = gb.rmsnorm_fwd_fp8(a, c, 1e-5, res)
            for y, h, rstd in ((y1, h1, rstd1), (y2, h2, rstd2)):
                assert _same_bits(h, h0)
                assert ((rstd.double() - rstd0.double()).abs() <= 2.0 ** -17 * rstd0.double()).all()
                assert ((y.double() - y0.double()).abs() <= tol_y * y0.double().abs()).all()
            u = np.abs(H64.astype(np.float32) * to64(c).astype(np.float32)).astype(np.float64)
            check_rstd(to64(ys), u.max(-1) * ref / 448, "row scale")
            assert np.array_equal(codes64(yq), q8.rmsnorm_fwd_fp8(H64, None, to64(c), 1e-5, io)[0])
    xa, ra, wa = (t.clone().requires_grad_() for t in (x, r, w))
    y1, h1 = ga.rms_norm(xa, wa, 1e-5, ra, checkpoint="int8")
    y0, h0 = ga.rms_norm(xa, wa, 1e-5, ra)
    assert _same_bits(h1, h0) and ((y1.double() - y0.double()).abs() <= tol_y * y0.double().abs()).all()


@pytest.mark.parametrize("H", [256, 777, 4096, 16384, 17001])
def test_fp8_norm_residual_out_over_its_inputs(H):
    T = 33
    x, r, w = _randn((T, H), torch.bfloat16, 1), _randn((T, H), torch.bfloat16, 2), _weight(H, torch.bfloat16)
    want = gb.rmsnorm_fwd_fp8(x, w, 1e-5, r)
    for target in (0, 1):
        a, b = x.clone(), r.clone()
        for p, q in zip(gb.rmsnorm_fwd_fp8(a, w, 1e-5, b, residual_out=(a, b)[target]), want):
            assert _same_bits(p, q)


# ---------------------------------------------------------------------------
# Launch geometries that small calls do not reach
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("act", list(gb.ACT))
@pytest.mark.parametrize("io,I", [("bf16", 16392), ("bf16", 20000), ("bf16", 32760), ("bf16", 32768),
                                  ("f32", 8196), ("f32", 12300), ("f32", 16384)])
def test_glu_wide_rows_of_many_tokens(io, I, act):
    # 2049 to 4096 vectors per row and more rows than SMs: rows stream through shared memory, the
    # last stage of a row holding 16 bytes (2049 vectors), a part or a whole of its size
    T = 3 * torch.cuda.get_device_properties(0).multi_processor_count + 1
    gate, up = _randn((T, 2 * I), IO[io], 1).chunk(2, dim=-1)
    q, s = gb.glu_fwd_fp8(gate, up, act)
    r = torch.from_numpy(sample_rows(T, 12)).cuda()
    G, U = to64(gate[r]), to64(up[r])
    check_window(q[r], s[r], q8.glu_out(act, G, U), _glu_window(act, G, U, io), "e4m3", f"{io} {I} {act}")
    q2, s2 = gb.glu_fwd_fp8(gate[:100], up[:100], act)  # the same rows, fewer than SMs: another kernel
    assert _same_bits(q2, q[:100]) and _same_bits(s2, s[:100])
    assert gb.device_error() == 0


@pytest.mark.parametrize("io,I", [("bf16", 32776), ("bf16", 65536), ("bf16", 65544), ("bf16", 131072), ("bf16", 131080),
                                  ("f32", 32768), ("f32", 32772), ("f32", 65536), ("f32", 65540)])
def test_glu_rows_of_a_cluster_and_beyond(io, I):
    # four and eight blocks per row, and rows too wide for those
    T = 5
    gate, up = _randn((T, 2 * I), IO[io], 3).chunk(2, dim=-1)
    q, s = gb.glu_fwd_fp8(gate, up)
    G, U = to64(gate), to64(up)
    check_window(q, s, q8.glu_out("silu", G, U), _glu_window("silu", G, U, io), "e4m3", f"{io} {I}")


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_glu_checkpoints_of_more_groups_than_run_at_once(io, fmt):
    # odd width: a warp takes several units one after the other
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    T, I = 8 * 64 * sms + 4321, 129
    gate, up, dout = (_randn((T, I), IO[io], s) for s in (1, 2, 3))
    out, gq, gs, uq, us = gb.glu_fwd_ckpt8(gate, up, "gelu_tanh", fmt=fmt)
    dgate, dup = gb.glu_bwd_ckpt8(dout, gq, gs, uq, us, "gelu_tanh")
    rows = sample_rows(T, 200, extra=(8 * 64 * sms - 1, 8 * 64 * sms))
    r = torch.from_numpy(rows).cuda()
    G, U = to64(gate[r]), to64(up[r])
    check_io(to64(out[r]), q8.glu_out("gelu_tanh", G, U), io, "out")
    check_exact(gq[r], gs[r], G, fmt, "gate8", 128)
    check_exact(uq[r], us[r], U, fmt, "up8", 128)
    dg, du = oracle.glu_bwd("gelu_tanh", to64(dout[r]), q8.values(codes64(gq[r]), codes64(gs[r]), 128),
                            q8.values(codes64(uq[r]), codes64(us[r]), 128))
    check_io(to64(dgate[r]), dg, io, "dgate")
    check_io(to64(dup[r]), du, io, "dup")


@pytest.mark.parametrize("T,H,io,wt", [
    (1500, 2500, "bf16", "bf16"), (1201, 5001, "bf16", "f32"), (1001, 8190, "bf16", "bf16"),    # blocks of 320 to 1024 threads per row
    (1500, 2050, "f32", "f32"), (1001, 8193, "bf16", "bf16"), (1003, 8200, "f32", "f32"), (1001, 20001, "bf16", "f32"),
    (3001, 512, "f32", "f32"), (3001, 64, "bf16", "bf16"), (1001, 16384, "bf16", "bf16"), (5001, 257, "f32", "f32")])
def test_norm_checkpoint_step_of_many_rows(T, H, io, wt):
    # several rows per block of the backward, one after the other: dW over all of them in
    # float64, the rest on sampled rows
    dt, eps = IO[io], 1e-5
    x, r, dy, dres = (_randn((T, H), dt, s) for s in (1, 2, 3, 4))
    w = _weight(H, IO[wt])
    W = to64(w)
    for res, fmt in ((True, "int8"), (False, "e4m3")):
        y, h, rstd, h8, hs = gb.rmsnorm_fwd_ckpt8(x, w, eps, r if res else None, fmt=fmt)
        dx, part, P = gb.rmsnorm_bwd_ckpt8(dy, h8, hs, w, rstd, dres if res else None)
        assert P < T
        kept = h8.double() * hs.double().repeat_interleave(128, 1)[:, :H]
        rs = 1 / torch.sqrt(h.double().square().mean(-1, keepdim=True) + eps)
        check_dw(to64(gb.rmsnorm_dw_finalize(part, P)), (dy.double() * kept * rs).sum(0).cpu().numpy())
        rows = sample_rows(T, 60)
        i = torch.from_numpy(rows).cuda()
        H64, RS = to64(h[i]), rs[i].cpu().numpy()[:, 0]
        check_rstd(to64(rstd[i]), RS)
        check_io(to64(y[i]), W * H64 * RS[:, None], io, "y")
        check_exact(h8[i], hs[i], H64, fmt, "h8", 128)
        dx64, _ = q8.rmsnorm_bwd_kept(to64(dy[i]), to64(dres[i]) if res else None, kept[i].cpu().numpy(), W, RS)
        check_io(to64(dx[i]), dx64, io, "dx")
