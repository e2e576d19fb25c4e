"""What is measured of the operators between the QKV projection and the attention output, each beside its plain form.

* ``norm_rope``  a training step of the per-head RMSNorm of Q and K with the rotary embedding in the same
  pass: q', k' and, from their gradients, dq, dk, dWq, dWk;
* ``axes``       a training step of the rotary embedding with several position axes (time, height, width):
  q', k' and, from their gradients, dq, dk;
* ``cache``      the serving form of the first: Q normalised and rotated, K normalised, rotated and quantised
  with V into a paged 8-bit cache; then the read-back of the new slots;
* ``attn``       attention of the new tokens of a ragged batch over that paged cache.

With x one head of one token, w its norm's weight, and (c, s)_i the cosine and sine of pos_{axis(i)} * theta^(-2i/D):
u = w * x * rstd, rstd = 1 / sqrt(mean x^2 + eps); a pair (u1, u2) becomes (u1 c - u2 s, u2 c + u1 s).  A stored head t
has a = max(max|t|, 2^-100), code = round(t * (qmax / a)) to nearest even, value = code * scale; rstd cancels out of the
codes, which are those of rot(w * x), and enters the scale a * rstd / qmax.  Attention: the new tokens are a
sequence's last ones; one at position p sees the keys j <= p (causal) with j > p - window (window > 0),
o = sum_j softmax_j(scale q.k_j) v_j, and one that sees nothing gives zeros.
"""

import math

import numpy as np
import torch

own = False

QMAX = {"int8": 127.0, "e4m3": 448.0}
AMIN = 2.0 ** -100
THETA = 1e6
EPS = 1e-6
IO = {"bf16": torch.bfloat16, "f32": torch.float32}
CODE = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}
MOST_PAIRS = 2048 * 32768 * 32 * 128  # query-key pairs x heads x head size of the largest attention
MOST_CODES = 64 * 8192 * 8 * 128      # values of K of the largest cache


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # the small float32 training workload: latency counts
        {"name": "norm_rope small f32", "op": "norm_rope", "T": 256, "Hq": 14, "Hk": 2, "D": 64, "io": "f32", "wt": "f32",
         "packed": False, "pairing": "half", "sections": "", "order": ""},
        # eight 2k sequences of a 0.6B model with Q/K norms, inside one projection output
        {"name": "norm_rope 0.6B", "op": "norm_rope", "T": 16384, "Hq": 16, "Hk": 8, "D": 128, "io": "bf16", "wt": "bf16",
         "packed": True, "pairing": "half", "sections": "", "order": ""},
        # 70B widths over images and text: three axes in turns; a ragged count of tokens
        {"name": "norm_rope 70B width, three axes", "op": "norm_rope", "T": 32761, "Hq": 64, "Hk": 8, "D": 128, "io": "bf16",
         "wt": "f32", "packed": True, "pairing": "half", "sections": "24 20 20", "order": "cyclic"},
        # the tokens of one small image: latency counts
        {"name": "axes one image", "op": "axes", "T": 259, "Hq": 14, "Hk": 2, "D": 64, "io": "bf16", "packed": False,
         "pairing": "half", "sections": "8 12 12", "order": "blocks"},
        # long videos packed with text at 8B widths
        {"name": "axes packed video", "op": "axes", "T": 65536, "Hq": 32, "Hk": 8, "D": 128, "io": "bf16", "packed": True,
         "pairing": "half", "sections": "16 24 24", "order": "blocks"},
        # one decode step of 16 sequences: latency counts
        {"name": "cache decode", "op": "cache", "T": 16, "seqs": 16, "pad": 0, "Hq": 32, "Hk": 8, "D": 128, "page": 16,
         "layout": "NHD", "pairing": "half", "fmt": "int8", "io": "bf16", "wt": "bf16", "sections": "", "order": ""},
        # the prompts of a ragged batch, written whole, pages with the heads outside
        {"name": "cache prompts", "op": "cache", "T": 32768, "seqs": 37, "pad": 11, "Hq": 32, "Hk": 8, "D": 128, "page": 64,
         "layout": "HND", "pairing": "half", "fmt": "e4m3", "io": "bf16", "wt": "bf16", "sections": "16 24 24", "order": "blocks"},
        # one sequence decodes over its 8k context: latency counts
        {"name": "attn decode one", "op": "attn", "N": 1, "ctx": 8192, "seqs": 1, "pad": 0, "Hq": 32, "Hk": 8, "D": 128,
         "page": 16, "layout": "NHD", "fmt": "int8", "window": 0},
        # 64 sequences decode over half a million cached tokens
        {"name": "attn decode batch", "op": "attn", "N": 64, "ctx": 524288, "seqs": 64, "pad": 0, "Hq": 32, "Hk": 8, "D": 128,
         "page": 64, "layout": "NHD", "fmt": "int8", "window": 0},
        # a few draft tokens each, a sliding window, a padded batch, small heads
        {"name": "attn draft window", "op": "attn", "N": 57, "ctx": 70001, "seqs": 19, "pad": 7, "Hq": 14, "Hk": 2, "D": 64,
         "page": 16, "layout": "HND", "fmt": "e4m3", "window": 1024},
        # packed prompts without any past: the whole triangle of each
        {"name": "attn prompts", "op": "attn", "N": 32768, "ctx": 32768, "seqs": 19, "pad": 0, "Hq": 32, "Hk": 8, "D": 128,
         "page": 64, "layout": "NHD", "fmt": "e4m3", "window": 0},
        # a chunk of a long prompt over all that was stored before it
        {"name": "attn chunk over 32k", "op": "attn", "N": 2048, "ctx": 32768, "seqs": 1, "pad": 0, "Hq": 32, "Hk": 8, "D": 128,
         "page": 64, "layout": "NHD", "fmt": "int8", "window": 0},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _sections(rng, D, least=1):
    """Pairs of each position axis; none for plain positions."""
    n = rng.randint(least, 4)
    if n == 1:
        return "", ""
    cuts = sorted(rng.sample(range(1, D // 2), n - 1))
    return " ".join(str(b - a) for a, b in zip([0] + cuts, cuts + [D // 2])), rng.choice(["blocks", "cyclic"])


def draw(rng):
    op = rng.choice(["norm_rope", "axes", "cache", "attn", "attn"])
    Hk = rng.choice([1, 2, 4, 8])
    c = {"op": op, "Hq": Hk * rng.choice([1, 2, 4, 7, 8]), "Hk": Hk}
    if op in ("norm_rope", "axes"):
        D = rng.choice([64, 80, 96, 128, 128, 256])
        io = rng.choice(["bf16", "bf16", "bf16", "f32"])
        row = (c["Hq"] + 2 * Hk) * D * (2 if io == "f32" else 1)
        c |= {"T": _log(rng, 1, min(65536, 2 ** 28 // row)), "D": D, "io": io, "packed": rng.random() < 0.5,
              "pairing": rng.choice(["half", "half", "interleaved"])}
        c["sections"], c["order"] = _sections(rng, D, 2 if op == "axes" else 1)
        if op == "norm_rope":
            c["wt"] = "f32" if io == "f32" else rng.choice(["bf16", "f32"])
        return c
    c |= {"pad": rng.choice([0, 0, 1, 7]), "page": rng.choice([1, 16, 48, 64, 256]), "layout": rng.choice(["NHD", "HND"]),
          "fmt": rng.choice(["int8", "e4m3"])}
    if op == "cache":
        D = rng.choice([64, 96, 128, 128, 256])
        T = _log(rng, 1, 32768)
        c |= {"T": T, "seqs": _log(rng, 1, min(T, 64)), "D": D, "io": "bf16", "wt": rng.choice(["bf16", "f32"]),
              "pairing": rng.choice(["half", "half", "interleaved"])}
        c["sections"], c["order"] = _sections(rng, D)
        return c
    D = rng.choice([64, 96, 128, 128])
    seqs = _log(rng, 1, 64)
    N = seqs if rng.random() < 0.4 else _log(rng, seqs, 8192)
    # several times the largest sequence's share, so that a ragged split stays below the largest listed case
    most = min(524288, MOST_CODES // (Hk * D), max(N, MOST_PAIRS * seqs // (4 * N * c["Hq"] * D)))
    return c | {"N": N, "ctx": _log(rng, N, max(N, most)), "seqs": seqs, "D": D, "window": rng.choice([0, 0, 0, 128, 1000])}


def _lengths(c):
    """New tokens and whole length of each sequence: fixed by the case."""
    B = c["seqs"]
    r = np.random.default_rng([c["N"], c["ctx"], B])

    def split(total, least):
        cuts = np.sort(r.integers(0, total - least * B + 1, B - 1))
        return np.diff(np.concatenate([[0], cuts, [total - least * B]])).astype(np.int64) + least

    new = split(c["N"], 1)
    return new, new + split(c["ctx"] - c["N"], 0)


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _randn(g, shape, io):
    return torch.randn(shape, generator=g, device="cuda", dtype=IO[io])


def _dev(a, t):
    return torch.from_numpy(np.ascontiguousarray(a)).to("cuda", t)


def _table(max_pos, D):
    ang = torch.arange(max_pos, device="cuda", dtype=torch.float64)[:, None] * \
        THETA ** (-2 * torch.arange(D // 2, device="cuda", dtype=torch.float64) / D)
    return torch.stack([ang.cos(), ang.sin()], dim=-1).float().contiguous()


def _axis_of(c):
    """The position axis of each pair: runs of the sections' lengths, or in turns as long as a section has pairs left."""
    left, out = [int(n) for n in c["sections"].split()], []
    if not left:
        return None
    if c["order"] == "blocks":
        return np.repeat(np.arange(len(left)), left)
    while len(out) < c["D"] // 2:
        for a in range(len(left)):
            if left[a]:
                left[a] -= 1
                out.append(a)
    return np.array(out)


def _positions(c, r, T):
    """Plain positions of packed documents, or text between grids of (time, height, width) on up to four axes."""
    n = max(1, len(c["sections"].split()))
    pos = np.zeros((n, T), np.int64)
    t = p = 0
    while t < T:
        if n == 1:
            k = min(T - t, int(np.clip(round(math.exp(r.normal(math.log(512), 1))), 32, 8192)))
            pos[0, t:t + k] = np.arange(k)
        elif r.random() < 0.5:  # text: every axis alike
            k = min(T - t, int(r.integers(1, 400)))
            pos[:, t:t + k] = p + np.arange(k)
            p += k
        else:
            size = [int(r.integers(1, 12)) if a == 0 else int(r.integers(1, 33)) for a in range(n)]
            k = min(T - t, math.prod(size))
            pos[:, t:t + k] = p + np.stack(np.unravel_index(np.arange(k), size))
            p += max(size)
        if p > 30000:  # the next document
            p = 0
        t += k
    return pos


def _prepare_heads(c, g, r, pad=0):
    T, Hq, Hk, D = c["T"] + pad, c["Hq"], c["Hk"], c["D"]
    if c["op"] == "cache" or c["packed"]:
        qkv = _randn(g, (T, (Hq + 2 * Hk) * D), c["io"])
        q, k, v = (t.unflatten(1, (-1, D)) for t in qkv.split([Hq * D, Hk * D, Hk * D], dim=1))
    else:
        q, k, v = _randn(g, (T, Hq, D), c["io"]), _randn(g, (T, Hk, D), c["io"]), None
    axis = _axis_of(c)
    pos = _positions(c, r, T)
    s = {"q": q, "k": k, "v": v, "positions": _dev(pos if axis is not None else pos[0], torch.int32),
         "table": _table(int(pos.max()) + 1, D), "axes": None if axis is None else bytes(axis.tolist()),
         "axis": None if axis is None else _dev(axis, torch.int64)}
    if "wt" in c:
        s |= {n: (1 + 0.1 * torch.randn(D, generator=g, device="cuda")).to(IO[c["wt"]]) for n in ("wq", "wk")}
    if c["op"] != "cache":
        s |= {"dq": _randn(g, (T, Hq, D), c["io"]), "dk": _randn(g, (T, Hk, D), c["io"])}
    return s


def _prepare_cache(c, g, length, r):
    """A cache that holds sequences of these lengths on scattered pages, and their page table."""
    page, Hk, D = c["page"], c["Hk"], c["D"]
    blocks = -(-length // page)
    pages = int(blocks.sum()) + 3
    order = r.permutation(pages)
    table = np.full((len(length), max(1, int(blocks.max()))), -1, np.int64)
    at = 0
    for b, n in enumerate(blocks):
        table[b, :n] = order[at:at + n]
        at += n
    s = {}
    shape = (pages, page, Hk, D) if c["layout"] == "NHD" else (pages, Hk, page, D)
    for n in "kv":
        codes = torch.empty(shape, dtype=CODE[c["fmt"]], device="cuda")
        scale = torch.empty(shape[:3], device="cuda")
        for i in range(0, pages, max(1, 2 ** 27 // math.prod(shape[1:]))):
            j = min(pages, i + max(1, 2 ** 27 // math.prod(shape[1:])))
            t = torch.randn((j - i, *shape[1:]), generator=g, device="cuda")
            codes[i:j], scale[i:j] = _quant(t, c["fmt"], t.abs().amax(-1))
        if c["layout"] == "HND":
            codes, scale = codes.transpose(1, 2), scale.transpose(1, 2)
        s[n + "_cache"], s[n + "_scale"] = codes, scale
    return s, table


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    r = np.random.default_rng(seed)
    if c["op"] in ("norm_rope", "axes"):
        return _prepare_heads(c, g, r) | {"case": c}
    if c["op"] == "cache":
        T, B = c["T"], c["seqs"]
        cuts = np.sort(r.choice(np.arange(1, T), size=B - 1, replace=False)) if B > 1 else np.zeros(0, np.int64)
        length = np.diff(np.concatenate([[0], cuts, [T]])).astype(np.int64)
        cache, table = _prepare_cache(c, g, length, r)
        at = np.arange(T) - np.repeat(np.cumsum(length) - length, length)
        slots = table[np.repeat(np.arange(B), length), at // c["page"]] * c["page"] + at % c["page"]
        return _prepare_heads(c, g, r, c["pad"]) | cache | {
            "slots": _dev(np.concatenate([slots, np.full(c["pad"], -1)]), torch.int64), "read": _dev(slots, torch.int64), "case": c}
    new, length = _lengths(c)
    cache, table = _prepare_cache(c, g, length, r)
    q = _randn(g, (c["N"] + c["pad"], c["Hq"], c["D"]), "bf16")
    return cache | {"q": q, "out": torch.zeros_like(q), "cu": _dev(np.concatenate([[0], np.cumsum(new)]), torch.int32),
                    "lens": _dev(length, torch.int32), "pages": _dev(table, torch.int32), "new": new, "length": length, "case": c}


# ---------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------

def _quant(v, fmt, amax):
    """Codes (as their type) and scales of the last axis of float32 v, whose largest magnitudes are amax."""
    a = amax.clamp(min=AMIN)
    qmax = torch.full((), QMAX[fmt], device=v.device)
    t = v * torch.div(qmax, a)[..., None]
    return (t.round() if fmt == "int8" else t).to(CODE[fmt]), torch.div(a, qmax)


def _turns(s):
    """cos and sin [T, 1, D / 2] of every token's pairs."""
    if s["axis"] is None:
        cs = s["table"][s["positions"].long()]
    else:
        cs = s["table"][s["positions"].long()[s["axis"]].T, torch.arange(len(s["axis"]), device="cuda")]
    return cs[:, None, :, 0], cs[:, None, :, 1]


def _rotate(x, cos, sin, pairing):
    """Rotate the pairs of the last axis of x [T, H, D] by cos, sin [T, 1, D / 2]."""
    x1, x2 = x.chunk(2, dim=-1) if pairing == "half" else (x[..., 0::2], x[..., 1::2])
    y1, y2 = x1 * cos - x2 * sin, x2 * cos + x1 * sin
    return torch.cat([y1, y2], dim=-1) if pairing == "half" else torch.stack([y1, y2], dim=-1).flatten(-2)


def _plain_heads(s):
    c, io = s["case"], s["q"].dtype
    cos, sin = _turns(s)
    out = {}
    for n in "qk":
        x, dy = s[n].float(), _rotate(s["d" + n].float(), cos, -sin, c["pairing"])
        if c["op"] == "axes":
            out[n] = _rotate(x, cos, sin, c["pairing"]).to(io)
            out["d" + n] = dy.to(io)
            continue
        w = s["w" + n].float()
        rstd = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS)
        xhat = x * rstd
        out[n] = _rotate(xhat * w, cos, sin, c["pairing"]).to(io)
        d = dy * w
        out["d" + n] = (rstd * (d - xhat * (d * xhat).mean(-1, keepdim=True))).to(io)
        out["dw" + n] = (dy * xhat).sum((0, 1), dtype=torch.float64).float()
    return out


def _plain_cache(s):
    c, io = s["case"], s["q"].dtype
    cos, sin = _turns(s)
    q, k = s["q"].float(), s["k"].float()
    u = q * (1 / torch.sqrt((q * q).mean(-1, keepdim=True) + EPS)) * s["wq"].float()
    out = {"q": _rotate(u, cos, sin, c["pairing"]).to(io)}
    n = c["T"]
    rstd = 1 / torch.sqrt((k * k).mean(-1) + EPS)
    at = (s["read"] // c["page"], s["read"] % c["page"])
    for name, t, r in (("k", _rotate(k * s["wk"].float(), cos, sin, c["pairing"]), rstd), ("v", s["v"].float(), None)):
        a = t[:n].abs().amax(-1)
        codes, scale = _quant(t[:n], c["fmt"], a)
        if r is not None:
            scale = a.clamp(min=AMIN) * r[:n] / QMAX[c["fmt"]]
        s[name + "_cache"].view(torch.uint8)[at] = codes.view(torch.uint8)
        s[name + "_scale"][at] = scale
        codes = s[name + "_cache"].view(torch.uint8)[at].view(CODE[c["fmt"]])
        out[name] = (codes.float() * s[name + "_scale"][at][..., None]).to(io)
    return out


def _context(s, b, n):
    """Codes and scales [n, Hk, D], [n, Hk] of K and of V of the first n tokens of sequence b."""
    page = s["case"]["page"]
    j = torch.arange(n, device="cuda")
    at = (s["pages"][b].long()[j // page], j % page)
    return [(s[x + "_cache"].view(torch.uint8)[at].view(s[x + "_cache"].dtype), s[x + "_scale"][at]) for x in "kv"]


def _plain_attn(s):
    c, out, t0 = s["case"], s["out"], 0
    Hk, G, D = c["Hk"], c["Hq"] // c["Hk"], c["D"]
    for b, (m, n) in enumerate(zip(s["new"].tolist(), s["length"].tolist())):
        k, v = ((codes.float() * scale[..., None]).transpose(0, 1) for codes, scale in _context(s, b, n))
        rows = max(1, 2 ** 29 // (n * c["Hq"]))
        for i in range(0, m, rows):
            e = min(m, i + rows)
            q = s["q"][t0 + i:t0 + e].float().view(e - i, Hk, G, D).permute(1, 0, 2, 3).reshape(Hk, -1, D)
            x = torch.matmul(q * D ** -0.5, k.transpose(1, 2)).view(Hk, e - i, G, n)
            gap = torch.arange(n - m + i, n - m + e, device="cuda")[:, None] - torch.arange(n, device="cuda")
            hide = (gap < 0) | (gap >= c["window"]) if c["window"] else gap < 0
            x.masked_fill_(hide[:, None], -math.inf)
            p = torch.exp(x - x.amax(-1, keepdim=True))
            o = torch.matmul(p.view(Hk, -1, n), v).view(Hk, e - i, G, D) / p.sum(-1, keepdim=True)
            out[t0 + i:t0 + e] = o.permute(1, 0, 2, 3).reshape(e - i, c["Hq"], D).to(out.dtype)
        t0 += m
    return out


# ---------------------------------------------------------------------------
# The library's calls
# ---------------------------------------------------------------------------

def _own_run(s):
    import rmsnorm_fwd_bwd_03_gb300 as gb
    c = s["case"]
    if c["op"] == "norm_rope":
        where = (s["wq"], s["wk"], s["positions"], s["table"], EPS)
        how = {"axes": s["axes"], "pairing": c["pairing"]}
        q, k = gb.qk_norm_rope_fwd(s["q"], s["k"], *where, **how)
        dq, dk, part, P = gb.qk_norm_rope_bwd(s["dq"], s["dk"], s["q"], s["k"], *where, **how)
        dwq, dwk = gb.qk_norm_dw_finalize(part, P)
        return {"q": q, "dq": dq, "dwq": dwq, "k": k, "dk": dk, "dwk": dwk}
    if c["op"] == "axes":
        q, k = gb.rope_axes_fwd(s["q"], s["k"], s["positions"], s["table"], s["axes"], pairing=c["pairing"])
        dq, dk = gb.rope_axes_bwd(s["dq"], s["dk"], s["positions"], s["table"], s["axes"], pairing=c["pairing"])
        return {"q": q, "dq": dq, "k": k, "dk": dk}
    cache = (s["k_cache"], s["k_scale"], s["v_cache"], s["v_scale"])
    if c["op"] == "cache":
        q = gb.qk_norm_rope_fwd_cache8(s["q"], s["k"], s["v"], s["wq"], s["wk"], s["positions"], s["table"], EPS, s["slots"],
                                       *cache, axes=s["axes"], pairing=c["pairing"])
        k, v = gb.cache8_read(s["read"], *cache, dtype=s["q"].dtype)
        return {"q": q, "k": k, "v": v}
    return gb.attn_cache8(s["q"], s["cu"], s["lens"], s["pages"], *cache, window=c["window"], out=s["out"])


def run(state):
    if own:
        return _own_run(state)
    op = state["case"]["op"]
    return _plain_attn(state) if op == "attn" else _plain_cache(state) if op == "cache" else _plain_heads(state)


# ---------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    c = case
    D, Hq, Hk = c["D"], c["Hq"], c["Hk"]
    if c["op"] == "attn":
        keys = pairs = 0
        w = c["window"]
        for m, n in zip(*(a.tolist() for a in _lengths(c))):
            keys += min(n, w + m - 1) if w else n
            k = min(m, max(0, w - 1 - (n - m))) if w else m  # rows that see all before them; the others see w keys
            pairs += k * (n - m) + k * (k + 1) // 2 + (m - k) * w
        return {"bytes": 4 * c["N"] * Hq * D + keys * (2 * Hk * (D + 4)) + 4 * -(-keys // c["page"]), "flops": 4 * D * Hq * pairs}
    b = 4 if c["io"] == "f32" else 2
    T, n = c["T"] + c.get("pad", 0), max(1, len(c["sections"].split()))
    heads = T * (Hq + Hk) * D
    if c["op"] == "cache":
        # K's and V's codes and scales are written and read back, K and V come back in io
        return {"bytes": T * (2 * Hq + 2 * Hk) * D * b + T * (4 * n + 8) + c["T"] * (8 + 4 * Hk * (D + 4) + 2 * Hk * D * b),
                "flops": heads * 7 + 6 * T * Hk * D}
    if c["op"] == "axes":
        return {"bytes": 4 * heads * b + 8 * T * n, "flops": 6 * heads}
    return {"bytes": 5 * heads * b + 8 * T * n + 4 * D * (b + 2), "flops": 22 * heads}


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------

def _nearest_e4m3(t):
    """The E4M3 value (3 bits behind the point, exponents from -6, up to 448) nearest to float64 t, ties to even."""
    _, e = torch.frexp(t)
    ulp = torch.exp2((e - 1).clamp(min=-6).double() - 3)
    return (torch.round(t / ulp) * ulp).clamp(-448, 448)


def _turned64(x, s, c, back=False):
    """The pairs of x [T, H, D] as complex numbers, each turned by its angle (or back)."""
    half = c["D"] // 2
    f = THETA ** (-2 * torch.arange(half, device="cuda", dtype=torch.float64) / c["D"])
    p = s["positions"].double()
    angle = (p[:, None] if s["axis"] is None else torch.stack([p[a] for a in s["axis"].tolist()], dim=1)) * f
    turn = torch.polar(torch.ones_like(angle), -angle if back else angle)[:, None]
    if c["pairing"] == "half":
        z = torch.complex(x[..., :half].contiguous(), x[..., half:].contiguous()) * turn
        return torch.cat([z.real, z.imag], dim=-1)
    return torch.view_as_real(torch.view_as_complex(x.contiguous().unflatten(-1, (-1, 2))) * turn).flatten(-2)


def _exact_heads(s, c):
    out = {}
    for n in "qk":
        x, dy = s[n].double(), _turned64(s["d" + n].double(), s, c, back=True)
        if c["op"] == "axes":
            out[n], out["d" + n] = _turned64(x, s, c), dy
            continue
        w = s["w" + n].double()
        length = torch.sqrt(x.square().mean(-1, keepdim=True) + EPS)
        out[n] = _turned64(x * w / length, s, c)
        g = dy * w
        out["d" + n] = g / length - x * (g * x).mean(-1, keepdim=True) / length ** 3
        out["dw" + n] = (dy * x / length).sum((0, 1))
    return out


def _exact_cache(s, c):
    n, fmt = c["T"], c["fmt"]

    def normed(x, w):
        x = x.double()
        return _turned64(x * w.double() / torch.sqrt(x.square().mean(-1, keepdim=True) + EPS), s, c)

    out = {"q": normed(s["q"], s["wq"])}
    for name, t in (("k", normed(s["k"], s["wk"])[:n]), ("v", s["v"][:n].double())):
        a = t.abs().amax(-1, keepdim=True).clamp(min=AMIN)
        code = t * (QMAX[fmt] / a)
        out[name] = (torch.round(code) if fmt == "int8" else _nearest_e4m3(code)) * a / QMAX[fmt]
    return out


def _exact_attn(s, c):
    out, t0 = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda"), 0
    G = c["Hq"] // c["Hk"]
    for b, (m, n) in enumerate(zip(s["new"].tolist(), s["length"].tolist())):
        (kc, ks), (vc, vs) = _context(s, b, n)
        for h in range(c["Hk"]):
            k = kc[:, h].to(torch.float64) * ks[:, h, None].double()
            v = vc[:, h].to(torch.float64) * vs[:, h, None].double()
            rows = max(1, 2 ** 28 // n)
            for g in range(h * G, (h + 1) * G):
                for i in range(0, m, rows):
                    e = min(m, i + rows)
                    x = s["q"][t0 + i:t0 + e, g].double() @ k.T / math.sqrt(c["D"])
                    row = torch.arange(n - m + i, n - m + e, device="cuda")[:, None]
                    col = torch.arange(n, device="cuda")[None]
                    seen = (col <= row) & (col > row - c["window"]) if c["window"] else col <= row
                    out[t0 + i:t0 + e, g] = torch.softmax(x.masked_fill(~seen, -math.inf), dim=-1) @ v
        t0 += m
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_attn(s, case) if case["op"] == "attn" else _exact_cache(s, case) if case["op"] == "cache" else _exact_heads(s, case)
