"""Performance cases of the decoder-layer operators: 4-bit weights with group
scales, the query/key norms with the position rotation, the 4-bit paged
key/value cache, and attention over it.

``run(state)`` is one call of an operator: in plain torch operations where
``own`` is false, through ``bit_mixed_precision_amd.bq`` where it is true.
``exact`` computes the same outputs in 64 bits from the definitions.

A page of the cache holds, for each kv head, PAGE tokens as
  K codes   [PAGE][D/2]               byte d/2 holds d even in its low nibble
  V codes   [PAGE/4][units][4][U]     U = 2 bytes (D = 64) or 4: unit u of a
                                      token holds d = 2Uu .. 2Uu + 2U - 1
  K params  [PAGE][2] fp16            scale, min: value = code * scale + min
  V params  [PAGE][2] fp16
"""
import math

import torch

own = False

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------

def listed():
    return [
        # one token through a square projection: the smallest call
        {"name": "w4g m1 4096x4096", "op": "gemm", "m": 1, "n": 4096, "k": 4096, "group": 128, "zero": False, "dtype": "fp16"},
        # four sequences through a widening layer, weights with zero points
        {"name": "w4g m4 11008x4096", "op": "gemm", "m": 4, "n": 11008, "k": 4096, "group": 64, "zero": True, "dtype": "bf16"},
        # a ragged decode batch through the narrowing layer
        {"name": "w4g m37 4096x11008", "op": "gemm", "m": 37, "n": 4096, "k": 11008, "group": 128, "zero": True, "dtype": "bf16"},
        # a prompt's tokens through the square projection
        {"name": "w4g m2048 4096x4096", "op": "gemm", "m": 2048, "n": 4096, "k": 4096, "group": 32, "zero": False, "dtype": "fp16"},
        # a decode batch's queries and keys, out of the fused projection's rows
        {"name": "norm-rope 16 tokens", "op": "rope", "tokens": 16, "hq": 32, "hkv": 8, "d": 128, "rot": 128, "inter": False, "norm": True, "dtype": "bf16"},
        # a long prompt's, rotated in part and in neighbouring pairs
        {"name": "norm-rope 8191 tokens", "op": "rope", "tokens": 8191, "hq": 32, "hkv": 8, "d": 128, "rot": 64, "inter": True, "norm": True, "dtype": "fp16"},
        # a decode step's keys and values into the cache, and back
        {"name": "cache 33 tokens", "op": "cache", "tokens": 33, "hq": 32, "hkv": 8, "d": 128, "rot": 128, "inter": False, "norm": True, "page": 16, "dtype": "bf16"},
        # a prompt's
        {"name": "cache 4097 tokens", "op": "cache", "tokens": 4097, "hq": 16, "hkv": 16, "d": 64, "rot": 64, "inter": False, "norm": False, "page": 64, "dtype": "fp16"},
        # one short conversation: latency counts
        {"name": "attn b1 len 700", "op": "attn", "batch": 1, "q": 1, "len": 700, "ragged": False, "hq": 32, "hkv": 8, "d": 128, "page": 16, "window": 0, "dtype": "fp16"},
        # a serving batch of ragged lengths
        {"name": "attn b32 len <= 8192", "op": "attn", "batch": 32, "q": 1, "len": 8192, "ragged": True, "hq": 32, "hkv": 8, "d": 128, "page": 16, "window": 0, "dtype": "bf16"},
        # a few very long contexts
        {"name": "attn b3 len 100001", "op": "attn", "batch": 3, "q": 1, "len": 100001, "ragged": False, "hq": 64, "hkv": 8, "d": 128, "page": 64, "window": 0, "dtype": "fp16"},
        # a chunk of a prompt behind what the cache holds, with a sliding window
        {"name": "attn b2 q301 len 5000", "op": "attn", "batch": 2, "q": 301, "len": 5000, "ragged": True, "hq": 32, "hkv": 8, "d": 64, "page": 32, "window": 2048, "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    dtype = rng.choice(["fp16", "bf16"])
    op = rng.choice(["gemm", "gemm", "rope", "cache", "attn", "attn"])
    if op == "gemm":
        group = rng.choice([32, 64, 128])
        n = _log(rng, 64, 12288)
        k = 128 * _log(rng, 2, 90)
        m = min(_log(rng, 1, 2048), max(1, 2048 * 4096 * 4096 // (n * k)))
        return {"op": op, "m": m, "n": n, "k": k, "group": group, "zero": rng.random() < 0.5, "dtype": dtype}
    d = rng.choice([64, 128, 128, 256])
    hkv = rng.choice([1, 2, 4, 8])
    hq = hkv * rng.choice([1, 3, 4, 8])
    if op in ("rope", "cache"):
        case = {"op": op, "tokens": _log(rng, 1, 4000), "hq": hq, "hkv": hkv, "d": d, "rot": rng.choice([d, d, d // 2]),
                "inter": rng.random() < 0.3, "norm": rng.random() < 0.7, "dtype": dtype}
        return case if op == "rope" else {**case, "page": rng.choice([16, 32, 64, 128])}
    q = rng.choice([1, 1, 1, _log(rng, 2, 300)])
    length = _log(rng, max(16, q), 60000)
    most = int(min(3e5 * 8 * 128 / (hkv * d), 6e9 / (hq * q * d)))  # tokens of all sequences
    length = max(q, min(length, most))
    return {"op": op, "batch": max(1, min(_log(rng, 1, 64), most // length)), "q": q, "len": length,
            "ragged": rng.random() < 0.6, "hq": hq, "hkv": hkv, "d": d, "page": rng.choice([16, 32, 64, 128]),
            "window": rng.choice([0, 0, 0, 1024]), "dtype": dtype}


def work(case):
    c = case
    if c["op"] == "gemm":
        groups = c["n"] * (c["k"] // c["group"])
        return {"bytes": c["n"] * c["k"] // 2 + groups * (4 if c["zero"] else 2) + 2 * c["m"] * (c["k"] + c["n"]),
                "flops": 2 * c["m"] * c["n"] * c["k"]}
    if c["op"] in ("rope", "cache"):
        q, kv = c["tokens"] * c["hq"] * c["d"], c["tokens"] * c["hkv"] * c["d"]
        table = c["tokens"] * c["rot"] * 4
        if c["op"] == "rope":
            return {"bytes": 4 * (q + kv) + table, "flops": 8 * (q + kv)}
        codes = c["tokens"] * c["hkv"] * (c["d"] + 8)
        # q in and out, k and v in, the codes written and read, k and v out
        return {"bytes": 4 * q + 4 * kv + table + 2 * codes + 4 * kv, "flops": 8 * (q + kv) + 12 * kv}
    lens = _lengths(c)
    seen, pairs = 0, 0
    for n in lens:
        first = max(0, n - c["q"] - c["window"] + 1) if c["window"] else 0
        seen += n - first
        for i in range(c["q"]):
            pos = n - c["q"] + i
            pairs += min(pos + 1, c["window"]) if c["window"] else pos + 1
    return {"bytes": seen * c["hkv"] * (c["d"] + 8) + 4 * c["batch"] * c["q"] * c["hq"] * c["d"],
            "flops": 4 * c["d"] * c["hq"] * pairs}


def _lengths(c):
    """The sequences' lengths: all `len`, or ragged from a third of it up."""
    if not c["ragged"]:
        return [c["len"]] * c["batch"]
    return [max(c["q"], c["len"] - (c["len"] * 2 // 3) * ((7 * i) % 16) // 15 - i) for i in range(c["batch"])]


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _pack_weights(w, group, zero):
    """Signed 4-bit codes with a scale (and zero point) per group of a row of w."""
    n, k = w.shape
    x = w.view(n, k // group, group)
    if zero:
        lo, hi = x.amin(2).clamp(max=0), x.amax(2).clamp(min=0)
        scale = ((hi - lo) / 15).half()
        z = (-8 - (lo / scale.float()).round()).clamp(-8, 7)
        codes = ((x / scale.float()[..., None]).round() + z[..., None]).clamp(-8, 7)
    else:
        scale = (x.abs().amax(2) / 7).half()
        z = None
        codes = (x / scale.float()[..., None]).round().clamp(-7, 7)
    codes = codes.view(n, k).to(torch.int16)
    packed = ((codes[:, 0::2] & 15) | ((codes[:, 1::2] & 15) << 4)).to(torch.uint8)
    return packed, scale, None if z is None else z.half()


def _quantize_tokens(x):
    """4-bit codes, scale and min (fp16) of each row of x (its last dimension)."""
    x = x.float()
    lo = x.amin(-1, keepdim=True).half().float()
    scale = ((x.amax(-1, keepdim=True) - lo) / 15).half().float()
    codes = torch.where(scale > 0, ((x - lo) / scale).round(), torch.zeros_like(x)).clamp(0, 15)
    return codes, scale, lo


def _unit(d):
    return 2 if d == 64 else 4


def _fill_cache(k, v, page):
    """Pages [pages, hkv, PAGE, D] of keys and values as the cache's bytes [pages, bytes]."""
    pages, hkv, _, d = k.shape
    parts, params = [], []
    for x, is_v in ((k, False), (v, True)):
        codes, scale, lo = _quantize_tokens(x)
        codes = codes.to(torch.uint8)
        b = codes[..., 0::2] | (codes[..., 1::2] << 4)
        if is_v:
            u = _unit(d)
            b = b.view(pages, hkv, page // 4, 4, d // 2 // u, u).transpose(3, 4)
        parts.append(b.reshape(pages, hkv, -1))
        params.append(torch.cat([scale, lo], -1).half().view(pages, hkv, -1).view(torch.uint8))
    return torch.cat(parts + params, 2).view(pages, -1)


def _page_values(raw, hkv, d, page):
    """Bytes of pages [n, page bytes] -> (k codes, v codes [n, hkv, PAGE, D], k and v params [n, hkv, PAGE, 2] fp16)."""
    n = raw.shape[0]
    raw = raw.view(n, hkv, page * (d + 8))
    kb = raw[..., : page * d // 2].reshape(n, hkv, page, d // 2)
    u = _unit(d)
    vb = raw[..., page * d // 2: page * d].reshape(n, hkv, page // 4, d // 2 // u, 4, u).transpose(3, 4).reshape(n, hkv, page, d // 2)
    kp = raw[..., page * d: page * d + 4 * page].contiguous().view(torch.float16).view(n, hkv, page, 2)
    vp = raw[..., page * d + 4 * page:].contiguous().view(torch.float16).view(n, hkv, page, 2)
    spread = lambda b: torch.stack([b & 15, b >> 4], -1).view(n, hkv, page, d)  # noqa: E731
    return spread(kb), spread(vb), kp, vp


def prepare(case, seed):
    c, g = case, _generator(seed)
    T = DTYPES[c["dtype"]]
    normal = lambda *shape: torch.randn(*shape, generator=g, device="cuda")  # noqa: E731
    s = dict(c)
    if c["op"] == "gemm":
        w = normal(c["n"], c["k"]) * 0.02
        s["A"] = normal(c["m"], c["k"]).to(T)
        s["B"], s["scale"], s["z"] = _pack_weights(w, c["group"], c["zero"])
        return s
    if c["op"] in ("rope", "cache"):
        t, hq, hkv, d = c["tokens"], c["hq"], c["hkv"], c["d"]
        rows = (normal(t, hq + 2 * hkv, d) * 2).to(T)  # the fused projection's rows
        s["x"], s["k"], s["v"] = rows[:, :hq], rows[:, hq: hq + hkv], rows[:, hq + hkv:]
        s["wq"] = (1 + 0.2 * normal(d)).to(T) if c["norm"] else None
        s["wk"] = (1 + 0.2 * normal(d)).to(T) if c["norm"] else None
        ang = torch.arange(8192, device="cuda", dtype=torch.float64)[:, None] * (
            10000.0 ** (-torch.arange(0, c["rot"], 2, device="cuda", dtype=torch.float64) / c["rot"]))
        s["cos"], s["sin"] = ang.cos().float(), ang.sin().float()
        s["pos"] = torch.randint(0, 8192, (t,), generator=g, device="cuda", dtype=torch.int32)
        if c["op"] == "cache":
            page = c["page"]
            pages = -(-t // page) + 8
            s["cache"] = torch.zeros(pages, hkv * page * (d + 8), dtype=torch.uint8, device="cuda")
            s["slots"] = torch.randperm(pages * page, generator=g, device="cuda")[:t].contiguous()
        return s
    lens, page, hkv, d = _lengths(c), c["page"], c["hkv"], c["d"]
    most = max(-(-n // page) for n in lens)
    pages = sum(-(-n // page) for n in lens)
    blocks = torch.full((c["batch"], most), -1, dtype=torch.int32)
    order = torch.randperm(pages, generator=torch.Generator().manual_seed(seed)).to(torch.int32)
    at = 0
    for i, n in enumerate(lens):
        w = -(-n // page)
        blocks[i, :w] = order[at: at + w]
        at += w
    s["blocks"] = blocks.cuda()
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    cache = torch.empty(pages, hkv * page * (d + 8), dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 27) // (hkv * page * d))
    for i in range(0, pages, step):
        n = min(step, pages - i)
        # keys carry a channel's own offset, as they do after a projection's bias
        cache[i: i + n] = _fill_cache((normal(n, hkv, page, d) + 0.5 * normal(1, hkv, 1, d)).to(T), normal(n, hkv, page, d).to(T), page)
    s["cache"] = cache
    s["x"] = (normal(c["batch"] * c["q"], c["hq"], d) * 1.5).to(T)
    return s


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------

def run(state):
    return {"gemm": _gemm, "rope": _rope, "cache": _cache, "attn": _attn}[state["op"]](state)


def _gemm(s):
    if own:
        from bit_mixed_precision_amd import bq
        return bq.gemm_w4g_a16(s["A"], s["B"], s["scale"], s["z"])
    n, k = s["n"], s["k"]
    codes = torch.stack([s["B"] & 15, s["B"] >> 4], -1).view(n, s["k"] // s["group"], s["group"])
    codes = (codes ^ 8).float() - 8
    if s["z"] is not None:
        codes = codes - s["z"].float()[..., None]
    w = (codes * s["scale"].float()[..., None]).view(n, k)
    return (s["A"].float() @ w.t()).to(s["A"].dtype)


def _norm_rope(x, w, s, wide):
    x = x.to(wide)
    if w is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w.to(wide)
    rot = s["rot"]
    at = s["pos"].long()
    cos, sin = s["cos"][at].to(wide)[:, None], s["sin"][at].to(wide)[:, None]
    if s["inter"]:
        a, b = x[..., :rot:2], x[..., 1:rot:2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., : rot // 2], x[..., rot // 2: rot]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([y, x[..., rot:]], -1) if rot < x.shape[-1] else y


def _rope(s):
    if own:
        from bit_mixed_precision_amd import bq
        return bq.qk_norm_rope(s["x"], s["k"], s["cos"], s["sin"], s["pos"], s["wq"], s["wk"], interleaved=s["inter"])
    T = s["x"].dtype
    return _norm_rope(s["x"], s["wq"], s, torch.float32).to(T), _norm_rope(s["k"], s["wk"], s, torch.float32).to(T)


def _cache(s):
    """Norm, rotate, write to the cache, and read the written tokens back."""
    T, hkv, d, page = s["x"].dtype, s["hkv"], s["d"], s["page"]
    if own:
        from bit_mixed_precision_amd import bq
        q = bq.qk_norm_rope_kv4(s["x"], s["k"], s["v"], s["cos"], s["sin"], s["pos"], s["cache"], s["slots"], page, s["wq"], s["wk"],
                                interleaved=s["inter"])
        return (q,) + bq.kv4_read(s["cache"], s["slots"], page, hkv, d, T)
    q = _norm_rope(s["x"], s["wq"], s, torch.float32).to(T)
    # codes turn over at borders between two values: 64 bits up to the key's own rounding
    k = _norm_rope(s["k"], s["wk"], s, torch.float64).to(T)
    out = []
    head, tok = s["slots"] // page, s["slots"] % page
    raw = s["cache"].view(-1, hkv, page * (d + 8))
    u = _unit(d)
    for x, is_v in ((k, False), (s["v"], True)):
        codes, scale, lo = _quantize_tokens(x)
        c8 = codes.to(torch.uint8)
        b = c8[..., 0::2] | (c8[..., 1::2] << 4)
        if is_v:
            raw[:, :, page * d // 2: page * d].unflatten(2, (page // 4, d // 2 // u, 4, u))[head, :, tok // 4, :, tok % 4] = b.unflatten(2, (d // 2 // u, u))
        else:
            raw[:, :, : page * d // 2].unflatten(2, (page, d // 2))[head, :, tok] = b
        at = page * d + (4 * page if is_v else 0)
        raw[:, :, at: at + 4 * page].unflatten(2, (page, 4))[head, :, tok] = torch.cat([scale, lo], -1).half().view(torch.uint8)
    kc, vc, kp, vp = _page_values(s["cache"], hkv, d, page)
    for codes, par in ((kc, kp), (vc, vp)):
        codes, par = codes[head, :, tok], par[head, :, tok].float()
        out.append((codes.float() * par[..., :1] + par[..., 1:]).to(T))
    return q, out[0], out[1]


def _attn(s):
    b, q, hq, hkv, d, page = s["batch"], s["q"], s["hq"], s["hkv"], s["d"], s["page"]
    if own:
        from bit_mixed_precision_amd import bq
        return bq.attn_kv4(s["x"], s["cache"], s["blocks"], s["lens"], page, hkv, window=s["window"], return_lse=True)
    T = s["x"].dtype
    most = s["blocks"].shape[1]
    kc, vc, kp, vp = _page_values(s["cache"][s["blocks"].clamp(min=0).view(-1).long()], hkv, d, page)

    def dense(codes, par):
        par = par.float()
        x = codes.float() * par[..., :1] + par[..., 1:]
        return x.view(b, most, hkv, page, d).transpose(1, 2).reshape(b * hkv, most * page, d)

    x = s["x"].float().view(b, q, hkv, hq // hkv, d).transpose(1, 2).reshape(b * hkv, -1, d) / math.sqrt(d)
    scores = torch.bmm(x, dense(kc, kp).transpose(1, 2).contiguous()).view(b, hkv, q, hq // hkv, most * page)
    key = torch.arange(most * page, device="cuda")
    pos = s["lens"][:, None].long() - q + torch.arange(q, device="cuda")
    gone = key > pos[..., None]
    if s["window"]:
        gone |= key <= pos[..., None] - s["window"]
    scores = scores.masked_fill(gone[:, None, :, None], float("-inf"))
    top = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - top)
    total = p.sum(-1, keepdim=True)
    o = torch.bmm((p / total).view(b * hkv, -1, most * page), dense(vc, vp)).view(b, hkv, q, hq // hkv, d)
    lse = (top + total.log()).squeeze(-1).transpose(1, 2).reshape(b * q, hq)
    return o.transpose(1, 2).reshape(b * q, hq, d).to(T), lse


# --------------------------------------------------------------------------
# the definitions, in 64 bits
# --------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    f = torch.float64
    if s["op"] == "gemm":
        n, k, group = s["n"], s["k"], s["group"]
        nib = torch.empty(n, k, dtype=torch.int32, device="cuda")
        nib[:, 0::2], nib[:, 1::2] = s["B"].int() % 16, s["B"].int() // 16
        w = torch.where(nib > 7, nib - 16, nib).to(f)
        if s["z"] is not None:
            w -= s["z"].to(f).repeat_interleave(group, 1)
        w *= s["scale"].to(f).repeat_interleave(group, 1)
        return torch.mm(s["A"].to(f), w.t().contiguous())

    if s["op"] in ("rope", "cache"):
        def turn(x, w):
            y = x.to(f).clone()
            if w is not None:
                y = y / ((y * y).sum(-1, keepdim=True) / s["d"] + 1e-6).sqrt() * w.to(f)
            half = s["rot"] // 2
            i = torch.arange(half, device="cuda")
            first, second = (2 * i, 2 * i + 1) if s["inter"] else (i, i + half)
            z = torch.complex(y[..., first], y[..., second])
            e = torch.complex(s["cos"].to(f), s["sin"].to(f)).index_select(0, s["pos"])
            z = z * e[:, None, :]
            y[..., first], y[..., second] = z.real, z.imag
            return y

        T = s["x"].dtype
        if s["op"] == "rope":
            return turn(s["x"], s["wq"]), turn(s["k"], s["wk"])

        def stored(x):
            x = x.to(f)
            lo = x.min(-1, keepdim=True)[0].half().to(f)
            scale = ((x.max(-1, keepdim=True)[0] - lo) / 15).float().half().to(f)
            u = ((x - lo) / torch.where(scale > 0, scale, torch.ones_like(scale))).round().clamp(0, 15)
            return u * scale + lo

        return turn(s["x"], s["wq"]), stored(turn(s["k"], s["wk"]).to(T)), stored(s["v"])

    b, q, hq, hkv, d, page = s["batch"], s["q"], s["hq"], s["hkv"], s["d"], s["page"]
    out = torch.empty(b * q, hq, d, dtype=f, device="cuda")
    lse = torch.empty(b * q, hq, dtype=f, device="cuda")
    for i in range(b):
        n = int(s["lens"][i])
        ids = s["blocks"][i, : -(-n // page)].long()
        kc, vc, kp, vp = _page_values(s["cache"][ids], hkv, d, page)
        rows = torch.arange(n - q, n, device="cuda")
        for h in range(hkv):
            kk = (kc[:, h].to(f) * kp[:, h, :, 0, None].to(f) + kp[:, h, :, 1, None].to(f)).reshape(-1, d)[:n]
            vv = (vc[:, h].to(f) * vp[:, h, :, 0, None].to(f) + vp[:, h, :, 1, None].to(f)).reshape(-1, d)[:n]
            at = slice(h * (hq // hkv), (h + 1) * (hq // hkv))
            x = s["x"][i * q: (i + 1) * q, at].to(f).reshape(-1, d)
            z = torch.mm(x, kk.t().contiguous()) / math.sqrt(d)
            pos = rows.repeat_interleave(hq // hkv)[:, None]
            key = torch.arange(n, device="cuda")
            hide = key > pos
            if s["window"]:
                hide = hide | (key <= pos - s["window"])
            z = z.masked_fill(hide, float("-inf"))
            lse[i * q: (i + 1) * q, at] = torch.logsumexp(z, 1).view(q, -1)
            out[i * q: (i + 1) * q, at] = torch.mm(torch.softmax(z, 1), vv).view(q, -1, d)
    return out, lse
