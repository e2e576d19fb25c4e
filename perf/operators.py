"""What is measured of the library's 8-bit operators, each beside its plain form.

Five operators, each a row-parallel, memory-bound pass of a transformer layer:

* ``norm_fp8``   RMSNorm with the fused residual add, output in E4M3 with one float32 scale per row;
* ``glu_fp8``    the gated MLP unit, output in E4M3 with one float32 scale per row;
* ``norm_ckpt``  a training step of RMSNorm whose forward saves its input in 8 bits (one float32 scale
  per 128 values of a row) and whose backward reads it: y, h, rstd, dx, dW;
* ``glu_ckpt``   the same of the gated unit: out, dgate, dup;
* ``cache``      RoPE on Q and K with K and V quantised into a paged cache (one float32 scale per token
  and head), then the read-back of the sequences' slots.

Quantisation of a group of values v, in float32 with each operation rounded: a = max(max|v|, 2^-100),
code = round(v * (qmax / a)) to nearest even, scale = a / qmax, value = code * scale; qmax is 127 for
INT8 and 448 for E4M3.  The float32 roundings belong to the definition: they decide a code next to a border.
"""

import math

import numpy as np
import torch

own = False

QMAX = {"int8": 127.0, "e4m3": 448.0}
AMIN = 2.0 ** -100
GROUP = 128
THETA = 5e5
IO = {"bf16": torch.bfloat16, "f32": torch.float32}
CODE = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # decode step of a batch of 32 sequences: the norm before a row-scaled FP8 projection
        {"name": "norm_fp8 decode", "op": "norm_fp8", "T": 32, "H": 4096, "io": "bf16", "wt": "bf16", "outliers": False},
        # prefill of two 16k sequences at the 70B width
        {"name": "norm_fp8 70B width", "op": "norm_fp8", "T": 32768, "H": 8192, "io": "bf16", "wt": "bf16", "outliers": True},
        # the down projection's operand in a small decode step, gate and up packed in one projection output
        {"name": "glu_fp8 decode", "op": "glu_fp8", "T": 8, "I": 14336, "io": "bf16", "packed": True, "act": "silu"},
        # the same over a ragged prefill at the 70B width
        {"name": "glu_fp8 70B width", "op": "glu_fp8", "T": 16383, "I": 28672, "io": "bf16", "packed": True, "act": "silu"},
        # the small float32 training workload: latency counts
        {"name": "norm_ckpt small f32", "op": "norm_ckpt", "T": 256, "H": 896, "io": "f32", "wt": "f32", "fmt": "int8", "outliers": False},
        # rows that are no multiple of 16 bytes
        {"name": "norm_ckpt odd rows", "op": "norm_ckpt", "T": 8191, "H": 1021, "io": "bf16", "wt": "f32", "fmt": "int8", "outliers": False},
        # packed documents with outlier channels: E4M3 keeps the small values of a group beside its outlier
        {"name": "norm_ckpt packed outliers", "op": "norm_ckpt", "T": 65536, "H": 4096, "io": "bf16", "wt": "bf16", "fmt": "e4m3", "outliers": True},
        # the small float32 training workload: latency counts
        {"name": "glu_ckpt small f32", "op": "glu_ckpt", "T": 256, "I": 4864, "io": "f32", "packed": False, "act": "silu", "fmt": "int8"},
        # a training step of four 8k sequences, gate and up packed in one projection output
        {"name": "glu_ckpt 8k packed", "op": "glu_ckpt", "T": 32768, "I": 14336, "io": "bf16", "packed": True, "act": "silu", "fmt": "int8"},
        # one decode step of 16 sequences, the new tokens read back: latency counts
        {"name": "cache decode", "op": "cache", "T": 16, "ctx": 16, "seqs": 16, "pad": 0, "Hq": 32, "Hk": 8, "D": 128,
         "page": 16, "layout": "NHD", "pairing": "half", "fmt": "int8", "io": "bf16"},
        # a chunk of a prefill, the whole context read back for the attention over it, a ragged batch with padding
        {"name": "cache chunked prefill", "op": "cache", "T": 2048, "ctx": 32761, "seqs": 5, "pad": 37, "Hq": 32, "Hk": 8, "D": 128,
         "page": 64, "layout": "NHD", "pairing": "half", "fmt": "int8", "io": "bf16"},
        # the packed documents of the largest workload, written and read back whole, pages with the heads outside
        {"name": "cache packed prefill", "op": "cache", "T": 65536, "ctx": 65536, "seqs": 76, "pad": 0, "Hq": 32, "Hk": 8, "D": 128,
         "page": 16, "layout": "HND", "pairing": "interleaved", "fmt": "e4m3", "io": "bf16"},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, lo, hi):
    """A row width: half of them multiples of 128, a quarter of 8, the rest as drawn."""
    w, k = _log(rng, lo, hi), rng.randrange(4)
    q = 128 if k < 2 else 8 if k == 2 else 1
    return max(lo, w // q * q)


def draw(rng):
    op = rng.choice(["norm_fp8", "glu_fp8", "norm_ckpt", "glu_ckpt", "cache"])
    io = rng.choice(["bf16", "bf16", "bf16", "f32"])
    half = 2 if io == "f32" else 1
    c = {"op": op}
    if op.startswith("norm"):
        H = _width(rng, 64, 8192)
        c |= {"T": _log(rng, 1, min(65536, 2 ** 27 // half // H)), "H": H, "io": io,
              "wt": "f32" if io == "f32" else rng.choice(["bf16", "f32"]), "outliers": rng.random() < 0.3}
    elif op.startswith("glu"):
        I = _width(rng, 128, 28672)
        c |= {"T": _log(rng, 1, min(65536, 2 ** 28 // half // I)), "I": I, "io": io, "packed": rng.random() < 0.5,
              "act": rng.choice(["silu", "silu", "gelu_tanh", "gelu_erf", "relu"])}
    else:
        T = _log(rng, 1, 16384)
        ctx = _log(rng, T, max(T, 32768))
        Hk = rng.choice([1, 2, 4, 8])
        c |= {"T": T, "ctx": ctx, "seqs": _log(rng, 1, min(T, 64)), "pad": rng.choice([0, 0, 1, 7]), "Hq": Hk * rng.choice([1, 2, 4, 7]),
              "Hk": Hk, "D": rng.choice([64, 64, 96, 128, 128, 256]), "page": rng.choice([1, 16, 48, 64, 256]),
              "layout": rng.choice(["NHD", "HND"]), "pairing": rng.choice(["half", "half", "interleaved"]), "io": "bf16"}
    if "fp8" not in op:
        c["fmt"] = rng.choice(["int8", "e4m3"])
    return c


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _randn(g, shape, io):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(IO[io]) if io == "f32" else \
        torch.randn(shape, generator=g, device="cuda", dtype=IO[io])


def _prepare_norm(c, g):
    T, H = c["T"], c["H"]
    s = {"x": _randn(g, (T, H), c["io"]), "residual": _randn(g, (T, H), c["io"]),
         "w": (1 + 0.1 * torch.randn(H, generator=g, device="cuda")).to(IO[c["wt"]]), "eps": 1e-5}
    if c["outliers"]:  # one channel in a hundred is fifty times as large
        s["x"][:, torch.randperm(H, generator=g, device="cuda")[:max(1, round(0.01 * H))]] *= 50
    if c["op"] == "norm_ckpt":
        s |= {"dy": _randn(g, (T, H), c["io"]), "dres": _randn(g, (T, H), c["io"])}
    return s


def _prepare_glu(c, g):
    T, I = c["T"], c["I"]
    if c["packed"]:  # the halves of one projection output
        gate, up = _randn(g, (T, 2 * I), c["io"]).chunk(2, dim=-1)
    else:
        gate, up = _randn(g, (T, I), c["io"]), _randn(g, (T, I), c["io"])
    s = {"gate": gate, "up": up}
    if c["op"] == "glu_ckpt":
        s["dout"] = _randn(g, (T, I), c["io"])
    return s


def _prepare_cache(c, g, seed):
    """Sequences of ragged lengths that fill `ctx` slots; each one's last tokens are the new ones."""
    r = np.random.default_rng(seed)
    T, ctx, B, page, Hq, Hk, D = c["T"], c["ctx"], c["seqs"], c["page"], c["Hq"], c["Hk"], c["D"]
    cuts = np.sort(r.choice(np.arange(1, ctx), size=B - 1, replace=False)) if B > 1 else np.zeros(0, np.int64)
    length = np.diff(np.concatenate([[0], cuts, [ctx]])).astype(np.int64)
    new = np.minimum(length, T // B)
    room = np.cumsum(length - new)
    new += np.diff(np.concatenate([[0], np.minimum(room, T - new.sum())]))
    seq = np.repeat(np.arange(B), length)
    pos = np.arange(ctx) - np.repeat(np.cumsum(length) - length, length)
    blocks = -(-length // page)
    first = np.cumsum(blocks) - blocks
    pages = int(blocks.sum()) + 3
    table = r.permutation(pages)
    slot = table[first[seq] + pos // page] * page + pos % page
    fresh = pos >= np.repeat(length - new, length)
    pad = np.full(c["pad"], -1, np.int64)
    dev = lambda a, t: torch.from_numpy(np.ascontiguousarray(a)).to("cuda", t)  # noqa: E731
    qkv = _randn(g, (T + c["pad"], (Hq + 2 * Hk) * D), c["io"])
    q, k, v = (t.unflatten(1, (-1, D)) for t in qkv.split([Hq * D, Hk * D, Hk * D], dim=1))
    max_pos = int(length.max())
    ang = torch.arange(max_pos, device="cuda", dtype=torch.float64)[:, None] * \
        THETA ** (-2 * torch.arange(D // 2, device="cuda", dtype=torch.float64) / D)
    s = {"q": q, "k": k, "v": v, "positions": dev(np.concatenate([pos[fresh], 0 * pad]), torch.int32),
         "slots": dev(np.concatenate([slot[fresh], pad]), torch.int64), "read": dev(slot, torch.int64),
         "table": torch.stack([ang.cos(), ang.sin()], dim=-1).float().contiguous()}
    shape = (pages, page, Hk, D) if c["layout"] == "NHD" else (pages, Hk, page, D)
    for n in "kv":  # what earlier steps wrote
        t = torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)
        a = t.abs().amax(-1)
        codes, scale = _quant(t, c["fmt"], a)
        if c["layout"] == "HND":
            codes, scale = codes.transpose(1, 2), scale.transpose(1, 2)
        s[n + "_cache"], s[n + "_scale"] = codes, scale
    return s


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    s = _prepare_cache(case, g, seed) if case["op"] == "cache" else _prepare_norm(case, g) if case["op"].startswith("norm") else _prepare_glu(case, g)
    return s | {"case": case}


# ---------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------

def _quant(v, fmt, amax):
    """Codes (as their type) and scales of the last axis of float32 v, whose largest magnitudes are amax."""
    a = amax.clamp(min=AMIN)
    qmax = torch.full((), QMAX[fmt], device=v.device)
    t = v * torch.div(qmax, a)[..., None]
    return (t.round() if fmt == "int8" else t).to(CODE[fmt]), torch.div(a, qmax)


def _checkpoint(v, fmt):
    """Float32 rows as they come back from an 8-bit checkpoint with one scale per GROUP values."""
    T, H = v.shape
    n = -(-H // GROUP)
    p = torch.nn.functional.pad(v, (0, n * GROUP - H)).view(T, n, GROUP)
    codes, scale = _quant(p, fmt, p.abs().amax(-1))
    return (codes.float() * scale[..., None]).view(T, n * GROUP)[:, :H]


def _act(x, act):
    """f(x) and f'(x), in the type of x."""
    if act == "silu":
        s = 1 / (1 + torch.exp(-x))
        return x * s, s * (1 + x * (1 - s))
    if act == "gelu_tanh":
        k = 2 * math.sqrt(2 / math.pi)
        s = 1 / (1 + torch.exp(-k * (x + 0.044715 * x * x * x)))
        return x * s, s + x * s * (1 - s) * k * (1 + 3 * 0.044715 * x * x)
    if act == "gelu_erf":
        cdf = 0.5 * torch.erfc(-x * math.sqrt(0.5))
        return x * cdf, cdf + x * torch.exp(-0.5 * x * x) / math.sqrt(2 * math.pi)
    return torch.where(x > 0, x, torch.zeros_like(x)), (x > 0).to(x.dtype)


def _plain_norm(s):
    c, io = s["case"], s["x"].dtype
    h = (s["x"].float() + s["residual"].float()).to(io)
    hf, w = h.float(), s["w"].float()
    rstd = 1 / torch.sqrt((hf * hf).mean(-1) + s["eps"])
    if c["op"] == "norm_fp8":
        u = hf * w
        a = u.abs().amax(-1)
        codes, _ = _quant(u, "e4m3", a)
        return {"y8": codes, "scale": a.clamp(min=AMIN) * rstd / QMAX["e4m3"], "h": h, "rstd": rstd}
    y = (w * (hf * rstd[:, None])).to(io)
    n = _checkpoint(hf, c["fmt"]) * rstd[:, None]
    dy = s["dy"].float()
    d = dy * w
    dx = rstd[:, None] * (d - n * (d * n).mean(-1, keepdim=True)) + s["dres"].float()
    return {"y": y, "h": h, "rstd": rstd, "dx": dx.to(io), "dw": (dy * n).sum(0, dtype=torch.float64).float()}


def _plain_glu(s):
    c, io = s["case"], s["gate"].dtype
    g, u = s["gate"].float(), s["up"].float()
    out = _act(g, c["act"])[0] * u
    if c["op"] == "glu_fp8":
        codes, scale = _quant(out, "e4m3", out.abs().amax(-1))
        return {"y8": codes, "scale": scale}
    f, fp = _act(_checkpoint(g, c["fmt"]), c["act"])
    d = s["dout"].float()
    return {"out": out.to(io), "dgate": (d * _checkpoint(u, c["fmt"]) * fp).to(io), "dup": (d * f).to(io)}


def _rotate(x, cos, sin, pairing):
    """Rotate the pairs of the last axis of x [T, H, D] by cos, sin [T, 1, D / 2]."""
    x1, x2 = x.chunk(2, dim=-1) if pairing == "half" else (x[..., 0::2], x[..., 1::2])
    y1, y2 = x1 * cos - x2 * sin, x2 * cos + x1 * sin
    return torch.cat([y1, y2], dim=-1) if pairing == "half" else torch.stack([y1, y2], dim=-1).flatten(-2)


def _plain_cache(s):
    c, io = s["case"], s["q"].dtype
    cs = s["table"][s["positions"].long()][:, None]
    q = _rotate(s["q"].float(), cs[..., 0], cs[..., 1], c["pairing"]).to(io)
    n = len(s["slots"]) - c["pad"]
    at = s["slots"][:n]
    at = (at // c["page"], at % c["page"])
    rd = (s["read"] // c["page"], s["read"] % c["page"])
    back = []
    for name, t in (("k", _rotate(s["k"].float(), cs[..., 0], cs[..., 1], c["pairing"])), ("v", s["v"].float())):
        codes, scale = _quant(t[:n], c["fmt"], t[:n].abs().amax(-1))
        s[name + "_cache"].view(torch.uint8)[at] = codes.view(torch.uint8)
        s[name + "_scale"][at] = scale
        codes = s[name + "_cache"].view(torch.uint8)[rd].view(CODE[c["fmt"]])
        back.append((codes.float() * s[name + "_scale"][rd][..., None]).to(io))
    return {"q": q, "k": back[0], "v": back[1]}


# ---------------------------------------------------------------------------
# The library's calls
# ---------------------------------------------------------------------------

def _own_run(s):
    import rmsnorm_fwd_bwd_03_gb300 as gb
    c = s["case"]
    if c["op"] == "norm_fp8":
        _, y8, scale, h, rstd = gb.rmsnorm_fwd_fp8(s["x"], s["w"], s["eps"], s["residual"], want_y=False)
        return {"y8": y8, "scale": scale, "h": h, "rstd": rstd}
    if c["op"] == "glu_fp8":
        y8, scale = gb.glu_fwd_fp8(s["gate"], s["up"], c["act"])
        return {"y8": y8, "scale": scale}
    if c["op"] == "norm_ckpt":
        y, h, rstd, h8, h_scale = gb.rmsnorm_fwd_ckpt8(s["x"], s["w"], s["eps"], s["residual"], fmt=c["fmt"])
        dx, part, P = gb.rmsnorm_bwd_ckpt8(s["dy"], h8, h_scale, s["w"], rstd, s["dres"])
        return {"y": y, "h": h, "rstd": rstd, "dx": dx, "dw": gb.rmsnorm_dw_finalize(part, P)}
    if c["op"] == "glu_ckpt":
        out, *saved = gb.glu_fwd_ckpt8(s["gate"], s["up"], c["act"], fmt=c["fmt"])
        dgate, dup = gb.glu_bwd_ckpt8(s["dout"], *saved, c["act"])
        return {"out": out, "dgate": dgate, "dup": dup}
    cache = (s["k_cache"], s["k_scale"], s["v_cache"], s["v_scale"])
    q = gb.rope_fwd_cache8(s["q"], s["k"], s["v"], s["positions"], s["table"], s["slots"], *cache, pairing=c["pairing"])
    k, v = gb.cache8_read(s["read"], *cache, dtype=s["q"].dtype)
    return {"q": q, "k": k, "v": v}


def run(state):
    if own:
        return _own_run(state)
    op = state["case"]["op"]
    return _plain_cache(state) if op == "cache" else _plain_norm(state) if op.startswith("norm") else _plain_glu(state)


# ---------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    c = case
    b = 4 if c["io"] == "f32" else 2
    if c["op"] == "cache":
        n, e = c["T"] + c["pad"], c["Hk"] * c["D"]
        head = 2 * c["Hk"] * (c["D"] + 4)  # codes and scales of one token's K and V
        return {"bytes": n * (2 * c["Hq"] * c["D"] * b + 2 * e * b + 12) + c["T"] * head + min(n, c["ctx"]) * c["D"] * 4
                + c["ctx"] * (8 + head + 2 * e * b),
                "flops": n * c["D"] * (3 * c["Hq"] + 8 * c["Hk"]) + 2 * c["ctx"] * e}
    T, N = c["T"], c.get("H") or c.get("I")
    groups = -(-N // GROUP)
    if c["op"] == "norm_fp8":
        wb = 4 if c["wt"] == "f32" else 2
        return {"bytes": T * N * (3 * b + 1) + 8 * T + N * wb, "flops": 8 * T * N}
    if c["op"] == "glu_fp8":
        return {"bytes": T * N * (2 * b + 1) + 4 * T, "flops": 8 * T * N}
    if c["op"] == "norm_ckpt":
        wb = 4 if c["wt"] == "f32" else 2
        return {"bytes": T * N * (7 * b + 2) + 8 * T * groups + 8 * T + N * (2 * wb + 4), "flops": 22 * T * N}
    return {"bytes": T * N * (6 * b + 4) + 16 * T * groups, "flops": 30 * T * N}


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------

def _nearest_e4m3(t):
    """The E4M3 value (3 bits behind the point, exponents from -6, up to 448) nearest to float64 t, ties to even."""
    _, e = torch.frexp(t)
    ulp = torch.exp2((e - 1).clamp(min=-6).double() - 3)
    return (torch.round(t / ulp) * ulp).clamp(-448, 448)


def _f32(t):
    return t.float().double()


def _codes64(v, fmt, amax):
    """The value of each code, the float32 scale, of float64 v; both decided where the definition decides them, in float32."""
    a = amax.clamp(min=AMIN)
    t = _f32(v * _f32(QMAX[fmt] / a)[..., None])
    return torch.round(t) if fmt == "int8" else _nearest_e4m3(t), _f32(a / QMAX[fmt])


def _kept64(v, fmt):
    parts = []
    for p in v.split(GROUP, dim=-1):
        codes, scale = _codes64(p, fmt, p.abs().amax(-1))
        parts.append(codes * scale[:, None])
    return torch.cat(parts, dim=-1)


def _exact_norm(s, c):
    io = s["x"].dtype
    h = (s["x"].double() + s["residual"].double()).to(io).double()  # the stored sum is what gets normalised
    w = s["w"].double()
    rstd = 1 / torch.sqrt(h.square().mean(-1) + s["eps"])
    if c["op"] == "norm_fp8":
        y = h * rstd[:, None] * w
        a = y.abs().amax(-1)
        return {"y8": _nearest_e4m3(y * (448 / a)[:, None]), "scale": a / 448, "h": h, "rstd": rstd}
    kept = _kept64(h, c["fmt"])
    xhat = kept * rstd[:, None]
    dy = s["dy"].double()
    g = dy * w
    c1 = (g * xhat).sum(-1, keepdim=True) / c["H"]
    return {"y": h * rstd[:, None] * w, "h": h, "rstd": rstd, "dx": s["dres"].double() + rstd[:, None] * (g - c1 * xhat),
            "dw": (dy * xhat).sum(0)}


def _exact_glu(s, c):
    gate, up = s["gate"].double(), s["up"].double()

    def value_and_slope(x):
        if c["act"] == "silu":
            p = torch.sigmoid(x)
            return x * p, p + x * p * (1 - p)
        if c["act"] == "gelu_tanh":
            t = torch.tanh(math.sqrt(2 / math.pi) * (x + 0.044715 * x ** 3))
            return 0.5 * x * (1 + t), 0.5 * (1 + t) + 0.5 * x * (1 - t * t) * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * x * x)
        if c["act"] == "gelu_erf":
            p = 0.5 * (1 + torch.erf(x / math.sqrt(2)))
            return x * p, p + x * torch.exp(-x * x / 2) / math.sqrt(2 * math.pi)
        return x.clamp(min=0), (x > 0).double()

    out = value_and_slope(gate)[0] * up
    if c["op"] == "glu_fp8":
        a = out.abs().amax(-1).clamp(min=AMIN)
        return {"y8": _nearest_e4m3(out * (448 / a)[:, None]), "scale": a / 448}
    f, fp = value_and_slope(_kept64(gate, c["fmt"]))
    d = s["dout"].double()
    return {"out": out, "dgate": d * _kept64(up, c["fmt"]) * fp, "dup": d * f}


def _exact_cache(s, c):
    D, page, n = c["D"], c["page"], len(s["slots"]) - c["pad"]
    f = s["positions"].double()[:, None] * THETA ** (-2 * torch.arange(D // 2, device="cuda", dtype=torch.float64) / D)
    turn = torch.polar(torch.ones_like(f), f)[:, None]

    def rotated(x):
        x = x.double()
        if c["pairing"] == "half":
            z = torch.complex(x[..., :D // 2].contiguous(), x[..., D // 2:].contiguous()) * turn
            return torch.cat([z.real, z.imag], dim=-1)
        return torch.view_as_real(torch.view_as_complex(x.contiguous().unflatten(-1, (-1, 2))) * turn).flatten(-2)

    read, back = s["read"], {"q": rotated(s["q"])}
    order = torch.full((s["k_cache"].shape[0] * page,), -1, dtype=torch.int64, device="cuda")
    order[s["slots"][:n]] = torch.arange(n, device="cuda")  # the new token in each slot
    src = order[read]
    for name, t in (("k", rotated(s["k"])[:n]), ("v", s["v"][:n].double())):
        a = t.abs().amax(-1).clamp(min=AMIN)
        q = t * (QMAX[c["fmt"]] / a)[..., None]
        q = (torch.round(q) if c["fmt"] == "int8" else _nearest_e4m3(q)) * (a / QMAX[c["fmt"]])[..., None]
        flat = s[name + "_cache"].reshape(-1, c["Hk"], D)[read].double() * s[name + "_scale"].reshape(-1, c["Hk"])[read].double()[..., None]
        back[name] = torch.where((src >= 0)[:, None, None], q[src.clamp(min=0)], flat)
    return back


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_cache(s, case) if case["op"] == "cache" else _exact_norm(s, case) if case["op"].startswith("norm") else _exact_glu(s, case)
