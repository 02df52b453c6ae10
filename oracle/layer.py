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
