"""The decoder-layer operators (4-bit weights with group scales, query/key
norm and rotation, the 4-bit paged cache, attention over it) in 64 bits.

TEST INFRASTRUCTURE ONLY (same rules as the rest of this package): torch on
the CPU, float64, straight from the formulas; shares no code with the HIP
library.  Each function also returns what the error bounds of the tests need.
"""
from __future__ import annotations

import math

import torch

F64 = torch.float64


# ---- 4-bit weights with group scales ----

def weights_w4g(Bp, scale, zero, group):
    """W [N, K] = (c - zero) * scale, exact; c the signed nibbles, low first."""
    n, k2 = Bp.shape
    codes = torch.empty(n, 2 * k2, dtype=F64)
    codes[:, 0::2] = (Bp & 15).to(F64)
    codes[:, 1::2] = (Bp >> 4).to(F64)
    codes = torch.where(codes > 7, codes - 16, codes)
    if zero is not None:
        codes = codes - zero.to(F64).repeat_interleave(group, 1)
    return codes * scale.to(F64).repeat_interleave(group, 1)


def quantize_w4g(w, group, zero=True):
    """Packed codes, scale and zero point (fp16) of w [N, K] by groups."""
    n, k = w.shape
    x = w.to(F64).view(n, k // group, group)
    if zero:
        lo, hi = x.amin(2).clamp(max=0), x.amax(2).clamp(min=0)
        s = ((hi - lo) / 15).half().to(F64)
        z = (-8 - (lo / s.clamp(min=1e-30)).round()).clamp(-8, 7)
        c = ((x / s.clamp(min=1e-30)[..., None]).round() + z[..., None]).clamp(-8, 7)
    else:
        s = (x.abs().amax(2) / 7).half().to(F64)
        z = None
        c = (x / s.clamp(min=1e-30)[..., None]).round().clamp(-7, 7)
    c = c.view(n, k).to(torch.int64) & 15
    return (c[:, 0::2] | (c[:, 1::2] << 4)).to(torch.uint8), s.half(), None if z is None else z.half()


def round_once(x, dtype):
    """float64 -> dtype (as float64) in one rounding, ties to even; no overflow."""
    bits, least = (11, -24) if dtype == torch.float16 else (8, -133)
    step = torch.ldexp(torch.ones_like(x), (torch.frexp(x)[1] - bits).clamp(min=least))
    return (x / step).round() * step


def w4g_bound(A, Bp, scale, zero, group):
    """The product S [M, N] and the bound of an output of A's type, for A whose
    rows are independent of the weights (random signs: partial sums stay within
    seven times the root of their terms' squares, or the terms' sum if smaller).

    u = 2^-23 is a whole step of fp32 below the largest of what an addition
    takes in: 32 products and the accumulator, 34 of them with the result, per
    matrix step of 32 k; all errors of one output are added up.

    M <= 16: the weights are exact.  Steps sum a (c + b) and a by themselves and
    in groups, b = 8 (fp16) or 136 (bf16); what a step takes in is at most a
    code's alignment times |a| (bf16: 144; fp16 codes are subnormal and aligned
    as 2^-14: 64, times 2 for the product's own carry, in matrix steps, and
    1024 in the dot products of M = 1, which a lane takes 32 at a time) or the
    group's sum so far.  The group's end and the sum over groups: eight
    roundings of both parts, and one a group, and 16 in joins, of the sum.

    M > 16: S is of the weights rounded once to A's type, each step takes in
    products and the sum so far.  (c - z) s is formed in fp32, with one rounding
    (c s and z s are exact in it), on its way to the type, or with none where the
    multiply-add rounds to the type itself: the two differ only where fp32 rounds
    onto a tie, and the bound takes in their difference there.
    """
    M, K = A.shape
    u, e = 2.0 ** -23, torch.finfo(A.dtype).eps / 2
    bf16 = A.dtype == torch.bfloat16
    a, W = A.to(F64), weights_w4g(Bp, scale, zero, group)
    floor = 0.0 if bf16 else 2.0 ** -25  # half a step of fp16 subnormals
    either = 0.0
    if M > 16:
        twice = W.to(torch.float32).to(A.dtype).to(F64)
        W = round_once(W, A.dtype)
        if not torch.equal(W, twice):
            either = a.abs() @ (W - twice).abs().t()
    S = a @ W.t()
    sums = torch.minimum(7 * ((a * a) @ (W * W).t()).sqrt(), a.abs() @ W.abs().t())
    if M > 16:
        term = a.abs().amax(1, keepdim=True) * W.abs().amax(1)
        return S, e * S.abs() * (1 + 2.0 ** -10) + u * (34 * (K // 32) * torch.maximum(term, sums) + 20 * sums) + floor + either
    n, blocks, per = Bp.shape[0], K // 32, group // 32
    s = scale.to(F64).repeat_interleave(per, 1)                                       # [N, blocks]
    z = torch.zeros_like(s) if zero is None else zero.to(F64).repeat_interleave(per, 1)
    b = 136.0 if bf16 else 8.0
    codes = weights_w4g(Bp, torch.ones_like(scale), None, group) + b
    x = a.view(M, blocks, 32)
    part = torch.einsum("mbk,nbk->mnb", x, codes.view(n, blocks, 32))                 # a step's own sums
    ones = x.sum(2)

    def running(t):  # sums of a group at each of its steps
        return t.unflatten(-1, (blocks // per, per)).cumsum(-1).flatten(-2)

    def taken(first, t):  # the most that a step takes in: terms, the sum before, the sum after
        r = running(t)
        return torch.maximum(torch.maximum(first, r.abs()), (r - t).abs())

    if M == 1:
        size = x.abs().sum(2)
        top = torch.maximum(size * (144.0 if bf16 else 15.0), x.abs().amax(2) * (0.0 if bf16 else 1024.0))
    else:
        size = x.abs().amax(2)
        top = size * (144.0 if bf16 else 128.0)
    step = taken(top[:, None], part) + taken(size, ones)[:, None] * (b + z.abs())
    ends = running(part).abs() + running(ones).abs()[:, None] * (b + z.abs())
    err = 34 * (step * s).sum(2) + 8 * (ends * s)[..., per - 1:: per].sum(2) + (K // group + 16) * sums
    return S, e * S.abs() * (1 + 2.0 ** -10) + u * err + floor


# ---- norm and rotation ----

def norm_rope(x, w, eps, cos, sin, pos, interleaved):
    """x [tokens, heads, D] -> (y, the sum of the magnitudes of y's terms)."""
    y = x.to(F64)
    if w is not None:
        y = y / torch.sqrt(y.pow(2).mean(-1, keepdim=True) + eps) * w.to(F64)
    size = y.abs()
    if cos is None or cos.shape[1] == 0:
        return y, size
    half = cos.shape[1]
    c, s = cos[pos.long()].to(F64)[:, None], sin[pos.long()].to(F64)[:, None]
    i = torch.arange(half)
    ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    a, b = y[..., ia].clone(), y[..., ib].clone()
    y, size = y.clone(), size.clone()
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    size[..., ia] = (a * c).abs() + (b * s).abs()
    size[..., ib] = (b * c).abs() + (a * s).abs()
    return y, size


def round_to(x, dtype):
    """float64 -> dtype, through fp32."""
    return x.to(torch.float32).to(dtype)


# ---- the cache ----

def kv4_codes(x):
    """Codes, scale, min of the rows of x (16-bit values), in the fp32 steps
    of the definition: min = fp16(min x), scale = fp16((max - min) / 15), both
    held at the ends of fp16's range and the scale at 0."""
    x = x.to(torch.float32)
    lo = x.amin(-1, keepdim=True).clamp(-65504, 65504).half().float()
    s = ((x.amax(-1, keepdim=True) - lo) / 15).clamp(0, 65504).half().float()
    q = torch.where(s > 0, ((x - lo) / torch.where(s > 0, s, torch.ones_like(s))).round(), torch.zeros_like(x))
    return q.clamp(0, 15).to(torch.uint8), s.half(), lo.half()


class Cache:
    """Pages as the library stores them, written and read token by token."""

    def __init__(self, pages, kv_heads, dim, page_size, fill=0):
        self.pages, self.hkv, self.dim, self.size = pages, kv_heads, dim, page_size
        self.bytes = torch.full((pages, kv_heads, page_size * (dim + 8)), fill, dtype=torch.uint8)

    def _places(self, t):
        """Byte places of token t's K codes, V codes, K params, V params."""
        p, d = self.size, self.dim
        b = torch.arange(d // 2)
        u = 2 if d == 64 else 4
        v = p * d // 2 + (t // 4) * 2 * d + (b // u) * 4 * u + (t % 4) * u + b % u
        four = torch.arange(4)
        return t * d // 2 + b, v, p * d + 4 * t + four, p * d + 4 * p + 4 * t + four

    def write(self, slot, k, v):
        """k, v [kv_heads, D] 16-bit values."""
        page, t = divmod(int(slot), self.size)
        if not 0 <= page < self.pages:
            return
        pk, pv, ak, av = self._places(t)
        for x, at, par in ((k, pk, ak), (v, pv, av)):
            q, s, lo = kv4_codes(x)
            self.bytes[page, :, at] = q[:, 0::2] | (q[:, 1::2] << 4)
            self.bytes[page, :, par] = torch.cat([s, lo], -1).contiguous().view(torch.uint8)

    def read(self, slot):
        """(codes, scale, min) of K and of V, [kv_heads, D] and [kv_heads, 1], float64."""
        page, t = divmod(int(slot), self.size)
        pk, pv, ak, av = self._places(t)
        out = []
        for at, par in ((pk, ak), (pv, av)):
            b = self.bytes[page][:, at]
            q = torch.stack([b & 15, b >> 4], -1).view(self.hkv, self.dim).to(F64)
            p = self.bytes[page][:, par].contiguous().view(torch.float16).to(F64)
            out.append((q, p[:, :1], p[:, 1:]))
        return out

    def flat(self):
        return self.bytes.view(self.pages, -1)


# ---- attention ----

def attention(q, cache, table, seq_lens, starts, scale, window=0):
    """q [total, hq, D]; sequence b's queries are starts[b] .. starts[b+1].
    -> out, lse, and per row the bounds' ingredients: the sum of p times the
    magnitude of the uncentred value, and the score error bound (see the
    tests)."""
    total, hq, d = q.shape
    hkv = cache.hkv
    group = hq // hkv
    out = torch.zeros(total, hq, d, dtype=F64)
    size = torch.zeros(total, hq, d, dtype=F64)
    lse = torch.full((total, hq), -math.inf, dtype=F64)
    delta = torch.zeros(total, hq, dtype=F64)
    for b, n in enumerate(seq_lens):
        q0, q1 = starts[b], starts[b + 1]
        keys = [(t, int(table[b][t // cache.size])) for t in range(max(n, 0))]
        keys = [(t, page * cache.size + t % cache.size) for t, page in keys if 0 <= page < cache.pages]
        if not keys or q1 <= q0:
            continue
        at = torch.tensor([t for t, _ in keys])
        rows = [cache.read(s) for _, s in keys]
        uk, sk, mk = (torch.stack([r[0][i] for r in rows], 1) for i in range(3))  # [hkv, n, D or 1]
        uv, sv, mv = (torch.stack([r[1][i] for r in rows], 1) for i in range(3))
        for i in range(q0, q1):
            pos = n - (q1 - q0) + (i - q0)
            on = at <= pos
            if window:
                on &= at > pos - window
            if not bool(on.any()):
                continue
            for h in range(hq):
                k = h // group
                x = q[i, h].to(F64)
                z = ((uk[k] * sk[k] + mk[k])[on] @ x) * scale
                lse[i, h] = torch.logsumexp(z, 0)
                p = torch.softmax(z, 0)
                val = (uv[k] * sv[k] + mv[k])[on]
                out[i, h] = p @ val
                size[i, h] = p @ (uv[k] * sv[k] + mv[k].abs())[on]
                big = (x.abs().sum() * (15 * sk[k] + mk[k].abs())[on].max()) * abs(scale)
                trunc = d * 2.0 ** -14 * x.abs().max() * sk[k][on].max() * abs(scale)
                delta[i, h] = trunc + 2.0 ** -21 * big + 2.0 ** -22 * z.abs().max()
    return out, lse, size, delta
