"""GPU vs oracle for RoPE with a quantised paged K/V cache and its read-back."""

import numpy as np
import pytest
import torch

import oracle
import rmsnorm_fwd_bwd_03_gb300 as gb
from oracle import q8

from _checks import check_io, to64
from _q8 import CODE, check_exact, check_window, codes64

pytestmark = pytest.mark.gpu

IO = {"f32": torch.float32, "bf16": torch.bfloat16}
THETA = 1e4


@pytest.fixture(scope="module", autouse=True)
def _library():
    from rmsnorm_fwd_bwd_03_gb300._build import build_library
    build_library()
    gb.library()


def _randn(shape, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def _caches(pages, page, Hk, D, fmt, layout="NHD", fill=0x55):
    """Caches filled with a pattern: what a call does not name has to keep it."""
    out = []
    if layout == "KV":  # K and V interleaved in one allocation
        codes = torch.full((pages, 2, page, Hk, D), fill, dtype=torch.uint8, device="cuda").view(CODE[fmt])
        scale = torch.full((pages, 2, page, Hk), -7.0, device="cuda")
        return codes[:, 0], scale[:, 0], codes[:, 1], scale[:, 1]
    for _ in range(2):
        shape = (pages, page, Hk, D) if layout == "NHD" else (pages, Hk, page, D)
        c = torch.full(shape, fill, dtype=torch.uint8, device="cuda").view(CODE[fmt])
        s = torch.full(shape[:3], -7.0, device="cuda")
        out += [c, s] if layout == "NHD" else [c.transpose(1, 2), s.transpose(1, 2)]
    return tuple(out)


def _at(t, slots, page):
    """Rows of a paged tensor at slots, by plain indexing."""
    t = t.view(torch.uint8) if t.element_size() == 1 else t
    return t[slots // page, slots % page]


def _rotation_window(x64):
    """A rotated value x1 c - x2 s in float32: c and s each rounded (2^-24 of at most 1), two
    products and a sum rounded (2^-24 each): at most 4 * 2^-24 * (|x1| + |x2|), with the
    head's largest magnitude for both."""
    return 8 * 2.0 ** -24 * np.abs(x64).max(axis=-1, keepdims=True)


def _case(T, Hq, Hk, D, io, fmt, page=16, layout="NHD", pairing="half", packed=True, in_place=False, unaligned=False, seed=0,
          shift=None):
    dt = IO[io]
    r = np.random.default_rng(seed + T + D)
    width = (Hq + 2 * Hk) * D
    off = shift or (1 if unaligned else 0)  # values before the first token's row
    qkv = _randn((T, width + off), dt, seed)[:, off:]
    q, k, v = (t.unflatten(1, (-1, D)) if t.shape[1] else None for t in qkv.split([Hq * D, Hk * D, Hk * D], dim=1))
    if not packed:
        q, k, v = (None if t is None else t.contiguous() for t in (q, k, v))
    max_pos = 50
    pos = torch.from_numpy(r.integers(0, max_pos, T).astype(np.int32)).cuda()
    pages = -(-T // page) + 3
    slots = torch.from_numpy(r.permutation(pages * page)[:T]).cuda()
    pad = r.random(T) < 0.1
    slots[torch.from_numpy(pad).cuda()] = -1 - int(r.integers(0, 5))
    table = gb.rope_table(max_pos, D, THETA)
    cache = _caches(pages, page, Hk, D, fmt, layout)
    q64, k64, v64 = (None if t is None else to64(t) for t in (q, k, v))
    qo = gb.rope_fwd_cache8(q, k, v, pos, table, slots, *cache, pairing=pairing, q_out=q if in_place else None)
    p = pos.cpu().numpy()
    what = f"{T}x{Hq}/{Hk}x{D} {io} {fmt} {layout} {pairing}"
    if Hq:
        assert (qo is q) == in_place
        check_io(to64(qo), oracle.rope_fwd(q64, p, THETA, pairing), io, what + " q")
    else:
        assert qo is None
    keep = ~pad
    s = slots[torch.from_numpy(keep).cuda()]
    kc, ks, vc, vs = cache
    k_rot = oracle.rope_fwd(k64, p, THETA, pairing)[keep]
    check_window(_at(kc, s, page).view(CODE[fmt]), _at(ks, s, page), k_rot, _rotation_window(k64[keep]), fmt, what + " k")
    check_exact(_at(vc, s, page).view(CODE[fmt]), _at(vs, s, page), v64[keep], fmt, what + " v")
    # slots that were not named keep their contents
    left = torch.ones(pages * page, dtype=torch.bool, device="cuda")
    left[s] = False
    left = left.nonzero()[:, 0]
    for c, sc in ((kc, ks), (vc, vs)):
        assert (_at(c, left, page) == 0x55).all() and (_at(sc, left, page) == -7.0).all()
    # read back in another order, with repeats and padding
    order = torch.from_numpy(r.integers(0, max(len(s), 1), T + 5)).cuda()
    rd = s[order] if len(s) else torch.zeros(0, dtype=torch.int64, device="cuda")
    rd[::7] = -3
    ko, vo = gb.cache8_read(rd, *cache, dtype=dt)
    for got, c, sc in ((ko, kc, ks), (vo, vc, vs)):
        val = _at(c, rd.clamp(min=0), page).view(CODE[fmt]).float() * _at(sc, rd.clamp(min=0), page)[..., None]
        want = torch.where((rd >= 0)[:, None, None], val, torch.zeros_like(val)).to(dt)
        assert torch.equal(got, want), what + " read"
    assert gb.device_error() == 0


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("D", [2, 6, 8, 16, 32, 64, 72, 80, 96, 128, 192, 256, 512, 576, 1024])
@pytest.mark.parametrize("pairing", ["half", "interleaved"])
def test_head_sizes(io, D, pairing):
    k = D + len(pairing)
    _case(1, 3, 1, D, io, ("int8", "e4m3")[k % 2], pairing=pairing)
    _case(29, 4, 2, D, io, ("e4m3", "int8")[k % 2], pairing=pairing, page=(1, 16, 7)[k % 3])


@pytest.mark.parametrize("Hq,Hk", [(0, 1), (0, 8), (1, 1), (8, 8), (32, 8), (7, 1), (28, 4), (64, 8), (5, 3), (40, 40), (128, 1)])
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_head_counts(Hq, Hk, fmt):
    _case(33, Hq, Hk, 128, "bf16", fmt)
    _case(9, Hq, Hk, 64, "f32", fmt, packed=False)


@pytest.mark.parametrize("layout", ["NHD", "HND", "KV"])
@pytest.mark.parametrize("page", [1, 3, 16, 64, 1000])
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_layouts_and_pages(layout, page, fmt):
    _case(70, 8, 4, 64, "bf16", fmt, page=page, layout=layout)
    _case(11, 2, 2, 40, "f32", fmt, page=page, layout=layout, pairing="interleaved")


@pytest.mark.parametrize("pairing", ["half", "interleaved"])
@pytest.mark.parametrize("D", [8, 24, 40, 72, 200, 256])
def test_eight_byte_runs(D, pairing):
    """bf16 heads that 8-byte, but not 16-byte, accesses divide."""
    _case(37, 5, 3, D, "bf16", "int8", pairing=pairing, shift=4)
    _case(300, 0, 2, D, "bf16", "e4m3", pairing=pairing, layout="HND", shift=4)
    _case(9, 33, 8, D, "bf16", "int8", pairing=pairing, in_place=True, shift=4)


@pytest.mark.parametrize("D", [18, 50, 100, 250])
@pytest.mark.parametrize("Hq,Hk", [(0, 1), (1, 1), (5, 3), (7, 2), (2, 4)])
def test_single_values_across_heads(D, Hq, Hk):
    """Heads of single values, several of Q, K and V to a warp."""
    _case(19, Hq, Hk, D, "bf16", "int8", layout="HND")
    _case(6, Hq, Hk, D, "f32", "e4m3", pairing="interleaved", unaligned=True)


@pytest.mark.parametrize("pairing", ["half", "interleaved"])
@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 128, 50])
def test_in_place_and_unaligned(io, D, pairing):
    _case(21, 4, 2, D, io, "int8", pairing=pairing, in_place=True)
    _case(21, 4, 2, D, io, "e4m3", pairing=pairing, unaligned=True)
    _case(21, 4, 2, D, io, "int8", pairing=pairing, unaligned=True, in_place=True, packed=False)


@pytest.mark.parametrize("T", [1, 2, 7, 8, 9, 255, 4097])
def test_token_counts(T):
    _case(T, 8, 2, 128, "bf16", "int8", page=16)


@pytest.mark.parametrize("T,Hq,Hk,D,io", [
    (5000, 32, 8, 128, "bf16"), (2501, 7, 12, 128, "bf16"), (5003, 16, 3, 128, "bf16"), (4999, 40, 4, 96, "bf16"),
    (2600, 0, 5, 256, "bf16"), (5001, 12, 2, 64, "f32"), (2500, 17, 8, 64, "f32"), (2511, 9, 6, 72, "bf16"),
    (1300, 70, 2, 40, "bf16"), (1703, 5, 3, 100, "bf16")])
def test_more_tokens_than_run_at_once(T, Hq, Hk, D, io):
    """Enough of them that the heads are dealt to few, busy lanes."""
    _case(T, Hq, Hk, D, io, "int8", page=64, layout="HND")
    _case(T, Hq, Hk, D, io, "e4m3", pairing="interleaved", packed=False)


@pytest.mark.parametrize("io,Hq,Hk,D", [("bf16", 32, 8, 128), ("bf16", 8, 8, 72), ("bf16", 12, 3, 100), ("f32", 12, 8, 64)])
@pytest.mark.parametrize("pairing", ["half", "interleaved"])
def test_chunks_of_a_prompt_give_the_same_bits(io, Hq, Hk, D, pairing):
    T, page = 5000, 16
    dt = IO[io]
    qkv = _randn((T, (Hq + 2 * Hk) * D), dt, D)
    q, k, v = (t.unflatten(1, (-1, D)) for t in qkv.split([Hq * D, Hk * D, Hk * D], dim=1))
    pos = torch.arange(T, device="cuda", dtype=torch.int32)
    slots = torch.randperm(T, device="cuda")
    table = gb.rope_table(T, D, THETA)
    whole = _caches(-(-T // page), page, Hk, D, "int8")
    parts = _caches(-(-T // page), page, Hk, D, "int8")
    qo = gb.rope_fwd_cache8(q, k, v, pos, table, slots, *whole, pairing=pairing)
    got = torch.empty_like(qo)
    for a, b in ((0, 1), (1, 17), (17, 500), (500, 2100), (2100, T)):
        gb.rope_fwd_cache8(q[a:b], k[a:b], v[a:b], pos[a:b], table, slots[a:b], *parts, pairing=pairing, q_out=got[a:b])
    assert torch.equal(got, qo)
    for x, y in zip(parts, whole):
        assert torch.equal(x, y)
    assert gb.device_error() == 0


def test_rotation_equals_rope_fwd():
    # the queries are those of rope_fwd, bit for bit, and the keys quantised are its float32 rotation
    T, Hq, Hk, D = 100, 8, 4, 128
    table = gb.rope_table(200, D, THETA)
    pos = torch.arange(T, dtype=torch.int32, device="cuda") + 60
    for pairing in ("half", "interleaved"):
        q, k, v = (_randn((T, h, D), torch.float32, 3 + h) for h in (Hq, Hk, Hk))
        cache = _caches(T, 1, Hk, D, "int8")
        slots = torch.arange(T, device="cuda")
        qo = gb.rope_fwd_cache8(q, k, v, pos, table, slots, *cache, pairing=pairing)
        q2, k2 = gb.rope_fwd_ex(q, k, pos, table, pairing=pairing)
        check_io(to64(qo), to64(q2), "f32", "q")
        check_window(cache[0][:, 0], cache[1][:, 0], to64(k2), _rotation_window(to64(k)), "int8", "k")


def test_bad_positions_and_slots_are_reported_and_harmless():
    T, Hq, Hk, D, page = 8, 4, 2, 64, 4
    for io, width in (("bf16", D), ("f32", 50)):  # vector path, element path
        D = width
        q, k, v = (_randn((T, h, D), IO[io], h) for h in (Hq, Hk, Hk))
        table = gb.rope_table(10, D, THETA)
        pos = torch.tensor([0, 1, -1, 10, 9, 2 ** 31 - 1, 3, 4], dtype=torch.int32, device="cuda")
        slots = torch.tensor([0, 1, 2, 3, 4, 5, 12, 2 ** 40], device="cuda")  # 12 slots
        cache = _caches(3, page, Hk, D, "int8")
        qo = gb.rope_fwd_cache8(q, k, v, pos, table, slots, *cache)
        assert gb.device_error(clear=True) == gb.ERR_BAD_POSITION | gb.ERR_BAD_SLOT
        bad = torch.tensor([2, 3, 5], device="cuda")
        good = torch.tensor([0, 1, 4, 6, 7], device="cuda")
        assert torch.isnan(qo[bad]).all() and torch.isfinite(qo[good]).all()
        kc, ks, vc, vs = cache
        assert torch.isnan(_at(ks, bad, page)).all() and torch.isfinite(_at(vs, bad, page)).all()
        assert (_at(ks, torch.arange(6, 12, device="cuda"), page) == -7).all()
        ko, vo = gb.cache8_read(torch.tensor([2, 0, 12, -1], device="cuda"), *cache, dtype=IO[io])
        assert gb.device_error(clear=True) == gb.ERR_BAD_SLOT
        assert torch.isnan(ko[0]).all() and torch.isfinite(vo[0]).all() and torch.isfinite(ko[1]).all()
        assert torch.isnan(ko[2]).all() and torch.isnan(vo[2]).all() and (ko[3] == 0).all() and (vo[3] == 0).all()
        # padding only: no store, and no error for its positions where there are no queries
        before = [t.clone() for t in cache]
        gb.rope_fwd_cache8(None, k, v, pos, table, torch.full_like(slots, -1), *cache)
        assert gb.device_error() == 0
        for a, b in zip(before, cache):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_non_finite_heads():
    T, Hk, D = 4, 2, 128
    k, v = _randn((T, Hk, D), torch.bfloat16, 1), _randn((T, Hk, D), torch.bfloat16, 2)
    v[0, 1, 5] = float("inf")
    k[1, 0, 7] = float("nan")
    v[2] = 0
    table = gb.rope_table(4, D, THETA)
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    for fmt in ("int8", "e4m3"):
        cache = _caches(T, 1, Hk, D, fmt)
        gb.rope_fwd_cache8(None, k, v, pos, table, torch.arange(T, device="cuda"), *cache)
        ko, vo = gb.cache8_read(torch.arange(T, device="cuda"), *cache)
        assert torch.isnan(vo[0, 1]).all() and torch.isfinite(vo[0, 0]).all() and torch.isfinite(vo[1:]).all()
        assert torch.isnan(ko[1, 0]).all() and torch.isfinite(ko[1, 1]).all() and (vo[2] == 0).all()


def test_slots_beyond_32_bits_of_bytes():
    # a cache of 4.4e9 bytes for each of K and V: the last pages' offsets pass 2^32
    Hk, D, page, pages = 8, 128, 64, 67000
    cache = [torch.empty((pages, page, Hk, D), dtype=torch.int8, device="cuda"), torch.empty((pages, page, Hk), device="cuda"),
             torch.empty((pages, page, Hk, D), dtype=torch.int8, device="cuda"), torch.empty((pages, page, Hk), device="cuda")]
    slots = torch.tensor([0, pages * page - 1, 2 ** 21, 2 ** 22, 2 ** 22 - 1, 2 ** 22 + 12345], device="cuda")
    T = len(slots)
    k, v = _randn((T, Hk, D), torch.bfloat16, 1), _randn((T, Hk, D), torch.bfloat16, 2)
    table = gb.rope_table(8, D, THETA)
    gb.rope_fwd_cache8(None, k, v, torch.zeros(T, dtype=torch.int32, device="cuda"), table, slots, *cache)  # position 0: identity
    ko, vo = gb.cache8_read(slots, *cache)
    for got, x in ((ko, k), (vo, v)):
        val = q8.values(*q8.quantize(to64(x), "int8"))
        check_io(to64(got), val, "bf16", "read")
    check_exact(_at(cache[2], slots, page).view(torch.int8), _at(cache[3], slots, page), to64(v), "int8", "v")


def test_strided_outputs_and_refusals():
    T, Hk, D, page = 12, 2, 64, 4
    k, v = _randn((T, Hk, D), torch.bfloat16, 1), _randn((T, Hk, D), torch.bfloat16, 2)
    table = gb.rope_table(16, D, THETA)
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    cache = _caches(3, page, Hk, D, "int8")
    slots = torch.arange(T, device="cuda")
    gb.rope_fwd_cache8(None, k, v, pos, table, slots, *cache)
    ko, vo = gb.cache8_read(slots, *cache)
    both = torch.full((T, 3 * Hk * D), 5.0, dtype=torch.bfloat16, device="cuda")
    a, b = both[:, :Hk * D].unflatten(1, (Hk, D)), both[:, Hk * D:2 * Hk * D].unflatten(1, (Hk, D))
    gb.cache8_read(slots, *cache, k_out=a, v_out=b)
    assert torch.equal(a, ko) and torch.equal(b, vo) and (both[:, 2 * Hk * D:] == 5).all()
    e4 = _caches(3, page, Hk, D, "e4m3")
    for bad in (lambda: gb.rope_fwd_cache8(None, k, v, pos, table, slots, *cache[:2], *e4[2:]),
                lambda: gb.rope_fwd_cache8(None, k, v[:, :1], pos, table, slots, *cache),
                lambda: gb.rope_fwd_cache8(k.float(), k, v, pos, table, slots, *cache),
                lambda: gb.rope_fwd_cache8(None, k, v, pos[:-1], table, slots, *cache),
                lambda: gb.rope_fwd_cache8(None, k, v, pos, table, slots.int(), *cache),
                lambda: gb.rope_fwd_cache8(None, k, v, pos, gb.rope_table(16, 32, THETA), slots, *cache),
                lambda: gb.rope_fwd_cache8(None, k, v, pos, table, slots, cache[0][:, :, :1], cache[1][:, :, :1], *cache[2:]),
                lambda: gb.rope_fwd_cache8(None, k, v, pos, table, slots, cache[0][:1].expand(3, -1, -1, -1), *cache[1:]),
                lambda: gb.cache8_read(slots, *cache, k_out=ko.float()),
                lambda: gb.cache8_read(slots, *cache[:2], *e4[2:])):
        with pytest.raises((ValueError, TypeError, gb.GblnError)):
            bad()


def test_decode_loop_in_a_graph_on_a_side_stream():
    # three sequences grow one token per step; the step (rotate, store, read the
    # whole context back) is captured once and replayed with new inputs
    B, Hq, Hk, D, page, steps = 3, 8, 2, 128, 4, 9
    table = gb.rope_table(steps, D, THETA)
    blocks = torch.randperm(B * 3, generator=torch.Generator().manual_seed(1)).view(B, 3).cuda()
    cache = _caches(B * 3, page, Hk, D, "e4m3", "HND")
    qkv = torch.zeros((B, (Hq + 2 * Hk) * D), dtype=torch.bfloat16, device="cuda")
    q, k, v = (t.unflatten(1, (-1, D)) for t in qkv.split([Hq * D, Hk * D, Hk * D], dim=1))
    pos = torch.zeros(B, dtype=torch.int32, device="cuda")
    new = torch.full((B,), -1, device="cuda")
    ctx = torch.full((B * steps,), -1, device="cuda")

    def step():
        qo = gb.rope_fwd_cache8(q, k, v, pos, table, new, *cache)
        return (qo, *gb.cache8_read(ctx, *cache))

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    all_k, all_v = [], []
    for t in range(steps):
        qkv.copy_(_randn(qkv.shape, torch.bfloat16, 100 + t))
        pos.fill_(t)
        new.copy_(blocks[:, t // page] * page + t % page)
        ctx.view(B, steps)[:, t] = new
        graph.replay()
        all_k.append(oracle.rope_fwd(to64(k), np.full(B, t), THETA))
        all_v.append(to64(v))
        qo, ko, vo = out
        check_io(to64(qo), oracle.rope_fwd(to64(q), np.full(B, t), THETA), "bf16", "q")
        for got, want in ((ko, all_k), (vo, all_v)):
            got = to64(got).reshape(B, steps, Hk, D)
            assert (got[:, t + 1:] == 0).all()
            want = np.stack(want, axis=1)
            # half an E4M3 step of the value (or of the scale's subnormals), and bf16's own half step
            err = np.abs(got[:, :t + 1] - want)
            amax = np.abs(want).max(-1, keepdims=True)
            assert (err <= (2.0 ** -4 + 2.0 ** -8 + 2.0 ** -12) * np.abs(want) + amax / 448 * 2.0 ** -10 * 1.01).all()
    assert gb.device_error() == 0


def test_empty_calls():
    Hk, D = 2, 64
    cache = _caches(2, 4, Hk, D, "int8")
    none = _caches(0, 4, Hk, D, "int8")
    table = gb.rope_table(4, D, THETA)
    kv = torch.empty((0, Hk, D), dtype=torch.bfloat16, device="cuda")
    i32, i64 = (torch.empty(0, dtype=t, device="cuda") for t in (torch.int32, torch.int64))
    assert gb.rope_fwd_cache8(None, kv, kv, i32, table, i64, *cache) is None
    assert gb.rope_fwd_cache8(torch.empty((0, 4, D), dtype=torch.bfloat16, device="cuda"), kv, kv, i32, table, i64, *cache).shape == (0, 4, D)
    ko, vo = gb.cache8_read(i64, *cache)
    assert ko.shape == vo.shape == (0, Hk, D)
    # a cache of no pages: padding stores nothing and reads as zeros, any slot is outside it
    one = _randn((1, Hk, D), torch.bfloat16, 1)
    pad = torch.full((1,), -1, device="cuda")
    gb.rope_fwd_cache8(None, one, one, torch.zeros(1, dtype=torch.int32, device="cuda"), table, pad, *none)
    ko, vo = gb.cache8_read(pad, *none)
    assert (ko == 0).all() and (vo == 0).all() and gb.device_error() == 0
    ko, _ = gb.cache8_read(torch.zeros(1, dtype=torch.int64, device="cuda"), *none)
    assert torch.isnan(ko).all() and gb.device_error(clear=True) == gb.ERR_BAD_SLOT


def test_prefill_then_decode_attention():
    # a prompt stored at once, tokens stored one by one, attention over what is read back:
    # against the same attention in float64 over the quantised values
    Hq, Hk, D, page, n, new = 4, 2, 64, 8, 37, 5
    table = gb.rope_table(n + new, D, THETA)
    cache = _caches(8, page, Hk, D, "int8", "HND")
    blocks = torch.tensor([5, 2, 7, 0, 1, 6], device="cuda")
    slot = lambda p: blocks[p // page] * page + p % page  # noqa: E731
    qkv = _randn((n + new, (Hq + 2 * Hk) * D), torch.bfloat16, 1)
    q, k, v = (t.unflatten(1, (-1, D)) for t in qkv.split([Hq * D, Hk * D, Hk * D], dim=1))
    pos = torch.arange(n + new, dtype=torch.int32, device="cuda")
    Q64 = oracle.rope_fwd(to64(q), pos.cpu().numpy(), THETA)
    K64 = q8.values(*q8.quantize(oracle.rope_fwd(to64(k), pos.cpu().numpy(), THETA), "int8"))
    V64 = q8.values(*q8.quantize(to64(v), "int8"))

    def attend(Q, K, V):
        out = np.zeros((Hq, D))
        for h in range(Hq):
            s = K[:, h // (Hq // Hk)] @ Q[h] / D ** 0.5
            p = np.exp(s - s.max())
            out[h] = p @ V[:, h // (Hq // Hk)] / p.sum()
        return out

    steps = [slice(0, n)] + [slice(i, i + 1) for i in range(n, n + new)]
    for s in steps:
        qo = gb.rope_fwd_cache8(q[s], k[s], v[s], pos[s], table, slot(pos[s].long()), *cache)
        ko, vo = gb.cache8_read(slot(torch.arange(s.stop, device="cuda")), *cache, dtype=torch.float32)
        got = attend(to64(qo)[-1], to64(ko), to64(vo))
        want = attend(Q64[s.stop - 1], K64[:s.stop], V64[:s.stop])
        # q is rounded to bf16 (2^-9 of each value): a score moves by at most 2^-9 sum |q k| / sqrt(D), a
        # weight by twice that, relatively; a rotated K next to a tie may take the other code (a step of
        # its scale: 1/127 of its largest value) in a few of its values, far less than that
        d = 2 * 2.0 ** -9 * max((np.abs(K64[:s.stop, h // (Hq // Hk)]) @ np.abs(Q64[s.stop - 1, h])).max() for h in range(Hq)) / D ** 0.5
        assert (np.abs(got - want) <= 1.5 * d * np.abs(V64[:s.stop]).max()).all()


def test_more_than_two_to_the_31_slots():
    # slot numbers past 31 bits (13 GB for each of K and V): page and offset come from a
    # 64-bit division
    Hk, D, page, pages = 1, 2, 16, 2 ** 27 + 5
    cache = [torch.empty((pages, page, Hk, D), dtype=torch.int8, device="cuda"), torch.empty((pages, page, Hk), device="cuda"),
             torch.empty((pages, page, Hk, D), dtype=torch.int8, device="cuda"), torch.empty((pages, page, Hk), device="cuda")]
    slots = torch.tensor([0, 2 ** 31 - 1, 2 ** 31, pages * page - 1, 12345678], device="cuda")
    T = len(slots)
    k, v = _randn((T, Hk, D), torch.float32, 1), _randn((T, Hk, D), torch.float32, 2)
    gb.rope_fwd_cache8(None, k, v, torch.zeros(T, dtype=torch.int32, device="cuda"), gb.rope_table(1, D, THETA), slots, *cache)
    ko, vo = gb.cache8_read(slots, *cache, dtype=torch.float32)
    for got, x in ((ko, k), (vo, v)):
        assert np.array_equal(to64(got), q8.values(*q8.quantize(to64(x), "int8")).astype(np.float32).astype(np.float64))
    gb.cache8_read(torch.tensor([pages * page], device="cuda"), *cache)
    assert gb.device_error(clear=True) == gb.ERR_BAD_SLOT


def test_two_streams_write_and_read_the_same_caches():
    # two halves of a batch stored at once from two streams, then read at once
    T, Hq, Hk, D, page = 4096, 8, 4, 128, 16
    qkv = _randn((T, (Hq + 2 * Hk) * D), torch.bfloat16, 1)
    q, k, v = (t.unflatten(1, (-1, D)) for t in qkv.split([Hq * D, Hk * D, Hk * D], dim=1))
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    table = gb.rope_table(T, D, THETA)
    slots = torch.randperm(T, generator=torch.Generator().manual_seed(3)).cuda()
    one, two = _caches(T // page, page, Hk, D, "e4m3"), _caches(T // page, page, Hk, D, "e4m3")
    qo = gb.rope_fwd_cache8(q, k, v, pos, table, slots, *one)
    ko, vo = gb.cache8_read(slots, *one)
    streams = [torch.cuda.Stream() for _ in range(2)]
    halves = (slice(0, 2050), slice(2050, T))
    torch.cuda.synchronize()
    outs = []
    for st, s in zip(streams, halves):
        with torch.cuda.stream(st):
            outs.append(gb.rope_fwd_cache8(q[s], k[s], v[s], pos[s], table, slots[s], *two))
    torch.cuda.synchronize()
    assert torch.equal(torch.cat(outs), qo)
    for a, b in zip(one, two):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    outs = []
    for st, s in zip(streams, halves):
        with torch.cuda.stream(st):
            outs.append(gb.cache8_read(slots[s], *two))
    torch.cuda.synchronize()
    assert torch.equal(torch.cat([o[0] for o in outs]), ko) and torch.equal(torch.cat([o[1] for o in outs]), vo)


def _rotated(x, cs, pairing):
    """The rotation in float32 with its roundings: one product rounded, the other exact within a
    multiply-add.  Products of float32 are exact in float64, and so is a sum but for one rounding far
    below float32's."""
    x64 = x.double()
    c, s = (cs[..., i].double()[:, None] for i in (0, 1))
    a, b = (x64[..., 0::2], x64[..., 1::2]) if pairing == "interleaved" else x64.chunk(2, dim=-1)
    f32 = lambda t: t.float().double()  # noqa: E731
    y = f32(a * c - f32(b * s)), f32(b * c + f32(a * s))
    return (torch.stack(y, dim=-1).flatten(-2) if pairing == "interleaved" else torch.cat(y, dim=-1)).float()


@pytest.mark.parametrize("pairing", ["half", "interleaved"])
@pytest.mark.parametrize("io,T,Hq,Hk,D", [
    ("f32", 16, 8, 2, 128), ("f32", 3000, 8, 2, 128), ("f32", 2001, 9, 8, 64), ("f32", 300, 4, 2, 50), ("f32", 200, 5, 3, 100),
    ("f32", 60, 3, 2, 250), ("f32", 40, 3, 2, 576), ("bf16", 300, 8, 2, 64), ("bf16", 300, 3, 2, 40), ("bf16", 2500, 32, 8, 128),
    ("bf16", 60, 3, 2, 50)])
def test_rotation_is_the_same_on_every_path(io, T, Hq, Hk, D, pairing):
    # the roundings of a rotated value depend on no launch: aligned rows and rows one value off
    # give the same queries, and the same codes and scales of K and V
    table = gb.rope_table(T, D, THETA)
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    slots = torch.arange(T, device="cuda")
    r = np.random.default_rng(D)
    table = torch.cat([table, table])[torch.from_numpy(r.permutation(2 * T)[:T].copy()).cuda()].contiguous()
    x = [_randn((T, h, D), IO[io], 3 + h) for h in (Hq, Hk, Hk)]
    for off in (0, 1):
        q, k, v = (torch.empty(t.numel() + off, dtype=t.dtype, device="cuda")[off:].view(t.shape).copy_(t) for t in x)
        cache = _caches(T, 1, Hk, D, "int8")
        qo = gb.rope_fwd_cache8(q, k, v, pos, table, slots, *cache, pairing=pairing)
        assert torch.equal(qo, _rotated(q, table, pairing).to(IO[io])), f"queries, {off} off"
        kr = to64(_rotated(k, table, pairing))
        check_exact(cache[0][:, 0], cache[1][:, 0], kr, "int8", f"k, {off} off")
        check_exact(cache[2][:, 0], cache[3][:, 0], to64(v), "int8", f"v, {off} off")
    assert gb.device_error() == 0
