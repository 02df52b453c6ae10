"""GPU parity of the decoder-layer operators against the 64-bit formulas of
oracle/layer.py.

Bounds (u = 2^-24; e = half a step of the output type, 2^-11 fp16, 2^-8 bf16):

* w4g, M <= 16: |C - S| <= e |S| + T, T = 2^-13 sum_k |a| s (twice the
  truncation of a matrix step: products with the subnormal codes are aligned
  24 bits below the largest exponent, 2^-13 of a code unit times |a|)
  + (K + 64) u sum_k |a| s (151 + |z|) (fp32 sums of a (c + 136) and of
  (136 + z) sum a).  M > 16 rounds each weight: + e sum_k |a W|.
* norm and rotation: fp32, at most 40 roundings per term (D = 256: 8 + 5 for
  the sum of squares, the root, the products): e |y| + 40 u size, size the sum
  of the magnitudes of y's terms.
* cache: codes, scales and minima equal bit for bit (keys are computed in
  fp64 up to their rounding, then the definition's fp32 steps).
* attention: a score is off by at most delta (oracle.layer.attention: the
  truncation D 2^-14 max|q| sk, 8 u of its terms' magnitude, 4 u of itself for
  the exponential's argument), so p by 2 delta and the exponential's 4 u
  relative; p sv is held to 2^-21 (fp16 output) or 2^-10 (bf16: toward zero,
  a whole step of 11 bits), all relative to size = sum p (u sv + |mv|):
  e |o| + (2 delta + r) size, r = 2^-20 or 2^-10 + 2^-20; sums of n terms in
  fp32 add n u, n <= 4096 here, 2^-12: r has it where n is large.
  lse: delta + 2^-20 (1 + |lse|).
"""
import math

import pytest
import torch

from gpu_util import banner, need_gpu
from layer_cases import W4G_ALL, W4G_LARGE, W4G_TALL, w4g_inputs, w4g_windows
from oracle import layer

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
F64 = torch.float64
TYPES = [torch.float16, torch.bfloat16]


@pytest.fixture(scope="module")
def dev():
    return need_gpu()


@pytest.fixture(scope="module")
def bq(dev):
    from bit_mixed_precision_amd import bq as _bq

    return _bq


def half_step(t):
    return torch.finfo(t).eps / 2


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def within(got, want, tol, what):
    got = got.cpu().to(F64)
    assert torch.isfinite(got).all(), f"{what}: not finite"
    over = (got - want).abs() - tol
    assert (over <= 0).all(), f"{what}: {int((over > 0).sum())} of {got.numel()} outside the bound, worst by {float(over.max()):.3g}"


# ---------------------------------------------------------------- w4g

def check_w4g(bq, dev, M, N, K, group, zero, T, seed=0, workspace=None, A=None):
    g = gen(seed + M + 3 * N + K)
    if A is None:
        A = torch.randn(M, K, generator=g).to(T)
    B, s, z = layer.quantize_w4g(torch.randn(N, K, generator=g) * 0.02 + (0.01 if zero else 0), group, zero)
    if zero:  # zero points need not be whole
        z = (z.float() + torch.rand(z.shape, generator=g) * 0.5).half()
    out = bq.gemm_w4g_a16(A.to(dev), B.to(dev), s.to(dev), None if z is None else z.to(dev), workspace=workspace)
    torch.cuda.synchronize()
    W = layer.weights_w4g(B, s, z, group)
    S = A.to(F64) @ W.t()
    big = s.to(F64).repeat_interleave(group, 1)
    zz = z.to(F64).abs().repeat_interleave(group, 1) if zero else 0.0
    a = A.to(F64).abs()
    tol = half_step(T) * S.abs() + 2.0 ** -13 * (a @ big.t()) + (K + 64) * U * (a @ (big * (151 + zz)).t()) + 2.0 ** -25
    if M > 16:
        tol = tol + half_step(T) * (a @ W.abs().t()) * (1 + 2.0 ** -8)
    within(out, S, tol, f"w4g {M}x{N}x{K} g{group} {T}")
    return out, S


W4G = [(1, 1, 64, 32), (1, 7, 64, 64), (1, 300, 192, 64), (1, 4096, 4096, 128), (2, 33, 128, 32), (2, 1000, 2048, 128),
       (3, 17, 320, 64), (4, 515, 4160, 32), (4, 64, 65536, 128), (5, 16, 128, 128), (8, 100, 320, 64), (16, 1030, 4096, 128),
       (17, 70, 192, 32), (31, 333, 1024, 64), (32, 4096, 4096, 128), (37, 260, 11008, 128), (48, 65, 640, 64),
       (49, 128, 8192, 32), (64, 200, 448, 64), (65, 130, 64, 32), (100, 257, 320, 64), (128, 128, 256, 128),
       (300, 1000, 1152, 128), (513, 140, 4096, 32)]


@pytest.mark.parametrize("shape", W4G)
@pytest.mark.parametrize("T", TYPES)
@pytest.mark.parametrize("zero", [False, True])
def test_w4g(bq, dev, shape, T, zero):
    M, N, K, group = shape
    banner(f"w4g M={M} N={N} K={K} group={group} zero={zero} {T}")
    check_w4g(bq, dev, M, N, K, group, zero, T)


@pytest.mark.parametrize("M", [1, 4, 16, 20, 64, 70])
@pytest.mark.parametrize("T", TYPES)
def test_w4g_weights_one_by_one(bq, dev, M, T):
    """One-hot rows pick single weights: C[m, n] = T(W[n, k]) to the bound of
    one product (M > 16: exactly, the weight's own rounding)."""
    banner(f"w4g one-hot M={M} {T}")
    N, K, group = 96, 256, 32
    A = torch.zeros(M, K)
    A[torch.arange(M), torch.randperm(K, generator=gen(M))[:M]] = 1
    check_w4g(bq, dev, M, N, K, group, True, T, seed=5, A=A.to(T))


def test_w4g_from_quantize_pack(bq, dev):
    """quantize_pack over the groups gives the operator's weights: W within
    half a code of the weight."""
    banner("w4g from quantize_pack")
    N, K, group = 64, 512, 64
    w = (torch.randn(N, K, generator=gen(2)) * 0.05).half()
    p, s = bq.quantize_pack(w.to(dev).view(N * K // group, group), 4)
    eye = torch.eye(K).half()[:64].to(dev)
    for rows in (slice(0, 1), slice(0, 4), slice(0, 16), slice(0, 64)):
        C = bq.gemm_w4g_a16(eye[rows].contiguous(), p.view(N, K // 2), s.view(N, K // group))
        torch.cuda.synchronize()
        want = w[:, rows].t().to(F64)
        step = s.cpu().to(F64).view(N, K // group)[:, :1].t()
        assert ((C.cpu().to(F64) - want).abs() <= step * 0.51 + want.abs() * 2.0 ** -10).all()


@pytest.mark.parametrize("M", [1, 2, 3, 9, 33, 64, 200])
def test_w4g_more(bq, dev, M):
    """Without a workspace, with a given one, K = 0, the output given, and
    twice the same result."""
    banner(f"w4g workspace, K = 0, repeat M={M}")
    out, S = check_w4g(bq, dev, M, 520, 8192, 128, True, torch.float16)
    again, _ = check_w4g(bq, dev, M, 520, 8192, 128, True, torch.float16)
    assert torch.equal(out, again)
    check_w4g(bq, dev, M, 520, 8192, 128, True, torch.float16, workspace=torch.empty(16, dtype=torch.uint8, device=dev))
    n = max(bq.gemm_w4g_workspace_bytes(M, 520, 8192), 16)
    given, _ = check_w4g(bq, dev, M, 520, 8192, 128, True, torch.float16,
                         workspace=torch.full((n,), 255, dtype=torch.uint8, device=dev))
    assert torch.equal(out, given)
    C = torch.full((M, 5), 3.0, dtype=torch.float16, device=dev)
    bq.gemm_w4g_a16(torch.empty((M, 0), dtype=torch.float16, device=dev), torch.empty((5, 0), dtype=torch.uint8, device=dev),
                    torch.empty((5, 0), dtype=torch.float16, device=dev), out=C)
    torch.cuda.synchronize()
    assert torch.count_nonzero(C).item() == 0


# ---------------------------------------------------------------- norm and rotation

def table(n, rot):
    ang = torch.arange(n, dtype=F64)[:, None] * 10000.0 ** (-torch.arange(0, rot, 2, dtype=F64) / max(rot, 1))
    return ang.cos().float(), ang.sin().float()


ROPE = [(1, 1, 1, 128, 128, False, True), (3, 8, 2, 64, 64, False, True), (5, 4, 4, 64, 32, True, True),
        (17, 5, 1, 128, 64, False, True), (33, 32, 8, 128, 128, True, True), (7, 3, 3, 256, 256, False, True),
        (9, 6, 2, 256, 96, False, True), (4, 2, 1, 128, 16, True, False), (12, 8, 8, 64, 48, False, False),
        (6, 4, 2, 128, 0, False, True), (1000, 16, 4, 128, 128, False, True)]


@pytest.mark.parametrize("c", ROPE)
@pytest.mark.parametrize("T", TYPES)
def test_qk_norm_rope(bq, dev, c, T):
    tokens, hq, hkv, d, rot, inter, norm = c
    banner(f"norm-rope {c} {T}")
    g = gen(tokens + hq + d)
    rows = (torch.randn(tokens, hq + hkv + 1, d, generator=g) * 3).to(T)
    wq, wk = (((torch.randn(d, generator=g) * 0.3 + 1).to(T)) if norm else None for _ in range(2))
    cos, sin = table(64, rot) if rot else (None, None)
    pos = torch.randint(0, 64, (tokens,), generator=g, dtype=torch.int32) if rot else None
    if rot and tokens > 2:
        pos[1], pos[2] = -1, 64
    x = rows.to(dev)
    to = lambda t: None if t is None else t.to(dev)  # noqa: E731
    qo = torch.full((tokens, hq, d), 7.0, dtype=T, device=dev)
    ko = torch.full((tokens, hkv, d), 7.0, dtype=T, device=dev)
    bq.qk_norm_rope(x[:, :hq], x[:, hq: hq + hkv], to(cos), to(sin), to(pos), to(wq), to(wk), 1e-5, inter, qo, ko)
    torch.cuda.synchronize()
    for got, src, w in ((qo, rows[:, :hq], wq), (ko, rows[:, hq: hq + hkv], wk)):
        safe = pos.clamp(0, 63) if rot else None
        y, size = layer.norm_rope(src, w, 1e-5, cos, sin, safe, inter)
        tol = half_step(T) * y.abs() + 40 * U * size + 2.0 ** -25
        if rot and tokens > 2:  # left out
            assert (got[1:3] == 7.0).all()
            keep = torch.tensor([i for i in range(tokens) if i not in (1, 2)])
            got, y, tol = got.cpu()[keep], y[keep], tol[keep]
        within(got, y, tol, f"norm-rope {c}")


CACHE = [(1, 1, 1, 128, 128, False, True, 16), (5, 4, 2, 64, 64, False, True, 32), (33, 8, 2, 128, 128, True, True, 16),
         (9, 3, 3, 256, 128, False, True, 64), (40, 0, 4, 64, 0, False, False, 128), (21, 2, 1, 256, 256, True, False, 16),
         (300, 4, 4, 128, 64, False, True, 256)]


@pytest.mark.parametrize("c", CACHE)
@pytest.mark.parametrize("T", TYPES)
def test_qk_norm_rope_kv4_and_read(bq, dev, c, T):
    tokens, hq, hkv, d, rot, inter, norm, page = c
    banner(f"cache {c} {T}")
    g = gen(tokens + d + page)
    rows = (torch.randn(tokens, hq + 2 * hkv, d, generator=g) * 2).to(T)
    if tokens > 8:
        rows[3] = 0.75                      # one value: scale 0
        rows[4, :, 5] = 3000.0              # an outlier
        rows[5] = rows[5] * 1e-6            # small
        rows[6, hq + hkv:] = torch.arange(d).to(T) % 16  # quotients on whole codes
    wk = (torch.randn(d, generator=g) * 0.3 + 1).to(T) if norm else None
    wq = (torch.randn(d, generator=g) * 0.3 + 1).to(T) if norm else None
    cos, sin = table(64, rot) if rot else (None, None)
    pos = torch.randint(0, 64, (tokens,), generator=g, dtype=torch.int32) if rot else None
    pages = -(-tokens // page) + 3
    slots = torch.randperm(pages * page, generator=g)[:tokens].contiguous()
    if tokens > 8:
        slots[0], slots[7] = -1, pages * page  # not written
    to = lambda t: None if t is None else t.to(dev)  # noqa: E731
    x = rows.to(dev)
    cache = torch.full((pages, bq.kv4_page_bytes(hkv, d, page)), 0xA5, dtype=torch.uint8, device=dev)
    q = bq.qk_norm_rope_kv4(x[:, :hq] if hq else None, x[:, hq: hq + hkv], x[:, hq + hkv:], to(cos), to(sin), to(pos), cache,
                            to(slots), page, to(wq) if hq else None, to(wk), 1e-6, inter)
    ref = layer.Cache(pages, hkv, d, page, 0xA5)
    k = layer.round_to(layer.norm_rope(rows[:, hq: hq + hkv], wk, 1e-6, cos, sin, pos, inter)[0], T)
    for t in range(tokens):
        ref.write(slots[t], k[t], rows[t, hq + hkv:])
    ko = torch.full((tokens, hkv, d), 7.0, dtype=T, device=dev)
    vo = torch.full((tokens, hkv, d), 7.0, dtype=T, device=dev)
    bq.kv4_read(cache, to(slots), page, hkv, d, T, ko, vo)
    torch.cuda.synchronize()
    assert torch.equal(cache.cpu(), ref.flat()), f"{int((cache.cpu() != ref.flat()).sum())} cache bytes differ"
    if hq:
        y, size = layer.norm_rope(rows[:, :hq], wq, 1e-6, cos, sin, pos, inter)
        within(q, y, half_step(T) * y.abs() + 40 * U * size + 2.0 ** -25, "cache: q")
    for t in range(tokens):
        if not 0 <= int(slots[t]) < pages * page:
            assert (ko[t] == 7.0).all() and (vo[t] == 7.0).all()
            continue
        for got, (u, s, m) in zip((ko, vo), ref.read(slots[t])):
            want = u * s + m
            within(got[t], want, half_step(T) * want.abs() * (1 + 2.0 ** -10) + 2.0 ** -25, "cache: read")


# calls long enough for several heads a row of lanes; head counts that no group divides
@pytest.mark.parametrize("c", [(2500, 17, 3, 128, 128, False, True), (820, 17, 15, 256, 96, True, True),
                               (3301, 17, 15, 64, 64, False, True), (2600, 18, 1, 128, 64, False, False)])
@pytest.mark.parametrize("T", TYPES)
def test_qk_norm_rope_long(bq, dev, c, T):
    test_qk_norm_rope(bq, dev, c, T)


@pytest.mark.parametrize("c", [(1410, 17, 9, 128, 128, False, True, 16), (707, 17, 9, 256, 64, True, True, 32),
                               (2811, 17, 9, 64, 64, False, True, 64), (3109, 0, 8, 128, 0, False, False, 16)])
@pytest.mark.parametrize("T", TYPES)
def test_qk_norm_rope_kv4_and_read_long(bq, dev, c, T):
    test_qk_norm_rope_kv4_and_read(bq, dev, c, T)


def test_kv4_nonfinite_stays_in_its_head(bq, dev):
    """NaN and infinities make unspecified codes of their own token and head only."""
    banner("cache, non-finite values")
    tokens, hkv, d, page = 4, 3, 128, 16
    x = torch.randn(tokens, 2 * hkv, d, generator=gen(1)).half()
    y = x.clone()
    y[1, 1, 7], y[2, 4, 9] = float("nan"), float("inf")  # a key head, a value head
    slots = torch.arange(tokens)
    out = []
    for r in (x, y):
        cache = torch.zeros(1, bq.kv4_page_bytes(hkv, d, page), dtype=torch.uint8, device=dev)
        bq.qk_norm_rope_kv4(None, r[:, :hkv].to(dev), r[:, hkv:].to(dev), None, None, None, cache, slots.to(dev), page)
        out.append([t.cpu() for t in bq.kv4_read(cache, slots.to(dev), page, hkv, d)])
    for i, (a, b) in enumerate(zip(*out)):
        same = (a == b).all(-1)
        bad = (1, 1) if i == 0 else (2, 1)
        same[bad] = True
        assert same.all()


# ---------------------------------------------------------------- attention

def make_cache(g, pages, hkv, d, page, T, k_off=0.5, v_mul=1.0):
    """Random pages; returns the oracle's cache."""
    c = layer.Cache(pages, hkv, d, page)
    off = torch.randn(hkv, d, generator=g) * k_off
    for s in range(pages * page):
        c.write(s, (torch.randn(hkv, d, generator=g) + off).to(T), (torch.randn(hkv, d, generator=g) * v_mul).to(T))
    return c


def run_attn(bq, dev, q, cache, tab, lens, hkv, page, starts=None, maxq=None, window=0, scale=None, ws="auto", q_dev=None):
    d = q.shape[2]
    kw = {}
    if ws == "none":
        kw["workspace"] = torch.empty(16, dtype=torch.uint8, device=dev)
    elif ws == "full":
        n = bq.attn_kv4_workspace_bytes(len(lens), maxq or q.shape[0] // len(lens), q.shape[1], hkv, d, tab.shape[1] * page)
        kw["workspace"] = torch.full((max(n, 16),), 255, dtype=torch.uint8, device=dev)
    out = torch.full(q.shape, 7.0, dtype=q.dtype, device=dev)
    lse = torch.full(q.shape[:2], 7.0, device=dev)
    bq.attn_kv4(q.to(dev) if q_dev is None else q_dev, cache.flat().to(dev), tab.to(dev),
                torch.tensor(lens, dtype=torch.int32, device=dev), page, hkv, scale,
                None if starts is None else torch.tensor(starts, dtype=torch.int32, device=dev), maxq, window, out, lse, **kw)
    torch.cuda.synchronize()
    return out, lse


def check_attn(got, q, cache, tab, lens, starts, window=0, scale=None, what="attn"):
    out, lse = got
    T, d = q.dtype, q.shape[2]
    scale = d ** -0.5 if scale is None else scale
    want, wlse, size, delta = layer.attention(q, cache, tab, lens, starts, scale, window)
    n = max(max(lens), 1)
    r = (2.0 ** -20 if T == torch.float16 else 2.0 ** -10 + 2.0 ** -20) + n * U
    tol = half_step(T) * want.abs() + (2 * delta[..., None] + r) * size * (1 + 2.0 ** -6) + 2.0 ** -25
    last = starts[-1]
    within(out[:last], want[:last], tol[:last], what)
    empty = torch.isinf(wlse)
    got_lse = lse.cpu().to(F64)
    assert (got_lse[:last][empty[:last]] == -math.inf).all(), f"{what}: lse of empty rows"
    assert (out.cpu()[:last][empty[:last]] == 0).all(), f"{what}: empty rows are not zero"
    full = ~empty[:last]
    off = (got_lse[:last] - wlse[:last])[full].abs() - (delta[:last] + 2.0 ** -20 * (1 + wlse[:last].abs()))[full]
    assert (off <= 0).all(), f"{what}: lse off by {float(off.max()):.3g} over"
    assert (out[last:] == 7.0).all() and (lse[last:] == 7.0).all(), f"{what}: rows behind the last sequence"


def tables(g, lens, page, pages, extra=1):
    """Block tables over shuffled pages; unused entries are out of range."""
    most = max(-(-max(n, 0) // page) for n in lens) + extra
    order = torch.randperm(pages, generator=g)
    tab = torch.full((len(lens), most), 1 << 30, dtype=torch.int32)
    tab[:, -1] = -5
    at = 0
    for b, n in enumerate(lens):
        w = -(-max(n, 0) // page)
        tab[b, :w] = order[at: at + w].to(torch.int32)
        at += w
    assert at <= pages
    return tab


# lens, q per sequence, hq, hkv, d, page, window
ATTN = [
    ([1], 1, 1, 1, 128, 16, 0),
    ([2, 0, 17], 1, 4, 2, 64, 16, 0),
    ([31, 32, 33, 16, 15], 1, 3, 1, 128, 16, 0),
    ([700], 1, 8, 2, 128, 16, 0),
    ([129, 5, 300], 1, 16, 1, 128, 32, 0),
    ([257, 640], 1, 20, 1, 64, 64, 0),
    ([400, 128], 1, 5, 5, 256, 16, 0),
    ([1000, 3], 1, 14, 2, 128, 128, 100),
    ([511], 1, 6, 2, 256, 256, 33),
    ([90, 4, 33], 7, 6, 2, 128, 16, 0),
    ([300, 40], 40, 4, 2, 64, 32, 0),
    ([10, 70], 33, 2, 1, 128, 16, 20),
    ([5], 9, 3, 1, 64, 16, 0),
    ([150], 64, 8, 8, 256, 16, 48),
    ([1100, 37, 1025], 1, 4, 1, 128, 64, 0),
    ([1500], 1, 3, 1, 64, 32, 0),
    ([1200, 260], 5, 8, 2, 128, 16, 700),
    ([1300], 1, 2, 1, 256, 16, 0),
]


@pytest.mark.parametrize("c", ATTN)
@pytest.mark.parametrize("T", TYPES)
@pytest.mark.parametrize("ws", ["auto", "none", "full"])
def test_attn_kv4(bq, dev, c, T, ws):
    lens, ql, hq, hkv, d, page, window = c
    banner(f"attn {c} {T} {ws}")
    g = gen(sum(lens) + d + hq)
    pages = sum(-(-n // page) for n in lens) + 2
    cache = make_cache(g, pages, hkv, d, page, T)
    tab = tables(g, lens, page, pages)
    # what lies behind the sequences' ends must not matter: NaN and infinities
    for b, n in enumerate(lens):
        if n % page:
            raw = cache.bytes[int(tab[b, n // page])]
            for t in range(n % page, page):
                _, _, ak, av = cache._places(t)
                raw[:, ak] = torch.tensor([0, 126, 0, 124], dtype=torch.uint8)  # NaN, inf
                raw[:, av] = torch.tensor([0, 124, 0, 126], dtype=torch.uint8)  # inf, NaN
    B = len(lens)
    q = (torch.randn(B * ql, hq, d, generator=g) * 1.5).to(T)
    got = run_attn(bq, dev, q, cache, tab, lens, hkv, page, window=window, ws=ws)
    check_attn(got, q, cache, tab, lens, [ql * i for i in range(B + 1)], window, what=str(c))


@pytest.mark.parametrize("T", TYPES)
def test_attn_kv4_ragged_queries(bq, dev, T):
    """q_start: sequences of 3, 0, 1 and 25 queries, rows behind the last left
    as they were, queries strided as a fused projection's."""
    banner(f"attn ragged queries {T}")
    lens, starts, hq, hkv, d, page = [50, 9, 33, 20], [0, 3, 3, 4, 29], 6, 2, 128, 16
    g = gen(4)
    cache = make_cache(g, 12, hkv, d, page, T)
    tab = tables(g, lens, page, 12)
    rows = torch.randn(33, hq + 4, d, generator=g).to(T)
    x = rows.to(dev)
    got = run_attn(bq, dev, rows[:, :hq], cache, tab, lens, hkv, page, starts, 25, q_dev=x[:, :hq])
    check_attn(got, rows[:, :hq], cache, tab, lens, starts, what="ragged")


@pytest.mark.parametrize("T", TYPES)
@pytest.mark.parametrize("ws", ["auto", "full"])
def test_attn_kv4_many_short_one_long(bq, dev, T, ws):
    """More sequences than a wavefront has lanes, the longest of them last,
    short ones whose later splits are empty."""
    banner(f"attn: many sequences {T} {ws}")
    g = gen(99)
    lens = [(7 * i) % 23 for i in range(69)] + [1300]
    hq, d, page = 3, 64, 16
    pages = sum(-(-n // page) for n in lens) + 2
    cache = make_cache(g, pages, 1, d, page, T)
    tab = tables(g, lens, page, pages)
    q = (torch.randn(len(lens), hq, d, generator=g) * 1.5).to(T)
    got = run_attn(bq, dev, q, cache, tab, lens, 1, page, ws=ws)
    check_attn(got, q, cache, tab, lens, list(range(len(lens) + 1)), what="many sequences")


@pytest.mark.parametrize("T", TYPES)
@pytest.mark.parametrize("batch,top,hq,hkv,d,window", [(40, 333, 16, 8, 64, 0), (33, 290, 8, 8, 128, 50), (17, 1400, 16, 8, 128, 0),
                                                       (65, 150, 40, 5, 64, 0)])
def test_attn_kv4_many_workgroups(bq, dev, T, batch, top, hq, hkv, d, window):
    """Enough sequences and heads that every one of them is one workgroup's."""
    banner(f"attn: many workgroups {batch} {top} {hq} {hkv} {d} {window} {T}")
    g = gen(batch + top)
    page = 16
    lens = [(37 * i + 1) % (top // 4) for i in range(batch - 1)] + [top]
    pages = sum(-(-n // page) for n in lens) + 2
    cache = make_cache(g, pages, hkv, d, page, T)
    tab = tables(g, lens, page, pages)
    q = (torch.randn(len(lens), hq, d, generator=g) * 1.5).to(T)
    got = run_attn(bq, dev, q, cache, tab, lens, hkv, page, window=window)
    check_attn(got, q, cache, tab, lens, list(range(len(lens) + 1)), window, what="many workgroups")


@pytest.mark.parametrize("T", TYPES)
def test_attn_kv4_bad_pages_and_lengths(bq, dev, T):
    """Pages outside the cache are not attended to; lengths are taken within
    the block table; max_q_len and the queries' range bound what is written."""
    banner(f"attn bad pages {T}")
    hq, hkv, d, page = 4, 2, 128, 16
    g = gen(8)
    cache = make_cache(g, 8, hkv, d, page, T)
    tab = torch.tensor([[0, -1, 2, 8], [3, 1 << 30, -(1 << 31), 4], [-1, -1, -1, -1], [5, 6, 7, 1]], dtype=torch.int32)
    q = torch.randn(4, hq, d, generator=g).to(T)
    got = run_attn(bq, dev, q, cache, tab, [60, 64, 64, 64], hkv, page)
    check_attn(got, q, cache, tab, [60, 64, 64, 64], [0, 1, 2, 3, 4], what="bad pages")
    got = run_attn(bq, dev, q, cache, tab, [60, -7, 1 << 30, 1 << 20], hkv, page)  # clamped to 0 and 64
    check_attn(got, q, cache, tab, [60, 0, 64, 64], [0, 1, 2, 3, 4], what="lengths")
    # starts outside the queries: nothing is read or written there
    got = run_attn(bq, dev, q, cache, tab, [60, 64, 64, 64], hkv, page, [0, 1, 2, 2, 50], 2)
    want = run_attn(bq, dev, q, cache, tab, [60, 64, 64, 64], hkv, page, [0, 1, 2, 2, 4], 2)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("T", TYPES)
@pytest.mark.parametrize("k_off,v_mul,q_mul", [(0.0, 1e-4, 1.0), (4.0, 300.0, 3.0), (0.0, 4000.0, 0.01), (1.0, 1.0, 30.0)])
def test_attn_kv4_ranges(bq, dev, T, k_off, v_mul, q_mul):
    """Small and large values, keys with a large common offset, peaked softmax."""
    banner(f"attn ranges {k_off} {v_mul} {q_mul} {T}")
    lens, hq, hkv, d, page = [333, 1064], 8, 2, 128, 16
    g = gen(9)
    cache = make_cache(g, 90, hkv, d, page, T, k_off, v_mul)
    tab = tables(g, lens, page, 90)
    q = (torch.randn(2, hq, d, generator=g) * q_mul).to(T)
    got = run_attn(bq, dev, q, cache, tab, lens, hkv, page)
    check_attn(got, q, cache, tab, lens, [0, 1, 2], what="ranges")


def test_attn_kv4_growing_scales(bq, dev):
    """V scales that grow along the sequence, by 2^16 over it."""
    banner("attn growing V scales")
    T, lens, hq, hkv, d, page = torch.float16, [1090], 4, 1, 128, 16
    g = gen(10)
    cache = layer.Cache(72, hkv, d, page)
    for s in range(1152):
        cache.write(s, torch.randn(hkv, d, generator=g).to(T), (torch.randn(hkv, d, generator=g) * 2.0 ** (s / 72 - 6)).to(T))
    tab = torch.arange(72, dtype=torch.int32)[None]
    q = torch.randn(1, hq, d, generator=g).to(T)
    for ws in ("none", "full"):
        check_attn(run_attn(bq, dev, q, cache, tab, lens, hkv, page, ws=ws), q, cache, tab, lens, [0, 1], what="growing")


@pytest.mark.parametrize("scale", [0.0, -0.1, 1.0])
@pytest.mark.parametrize("T", TYPES)
def test_attn_kv4_scales(bq, dev, T, scale):
    """Any sign of the softmax scale; 0 is the plain average."""
    banner(f"attn scale {scale} {T}")
    lens, hq, hkv, d, page = [77, 300], 4, 2, 64, 16
    g = gen(14)
    cache = make_cache(g, 26, hkv, d, page, T)
    tab = tables(g, lens, page, 26)
    q = torch.randn(2, hq, d, generator=g).to(T)
    got = run_attn(bq, dev, q, cache, tab, lens, hkv, page, scale=scale)
    check_attn(got, q, cache, tab, lens, [0, 1, 2], scale=scale, what="scale")


@pytest.mark.parametrize("T", TYPES)
@pytest.mark.parametrize("hq,d", [(2, 64), (8, 128), (64, 64), (2, 256)])
def test_attn_kv4_masked_places_may_be_anything(bq, dev, T, hq, d):
    """NaN and infinite parameters of keys that a row does not see (before its
    window, after its own position) change nothing for it; a row that sees one
    gets NaN."""
    banner(f"attn masked places {hq} {d} {T}")
    n, ql, hkv, page, window = 150, 8, 1, 16, 40
    g = gen(15)
    cache = make_cache(g, 10, hkv, d, page, T)
    tab = torch.arange(10, dtype=torch.int32)[None]
    q = torch.randn(ql, hq, d, generator=g).to(T)
    want = run_attn(bq, dev, q, cache, tab, [n], hkv, page, window=window)
    check_attn(want, q, cache, tab, [n], [0, ql], window, what="clean")
    bad = torch.tensor([0, 126, 0, 124], dtype=torch.uint8)  # NaN, inf
    for t in list(range(0, n - ql - window + 1)) + [n - 1]:  # before every window; the last key, seen by the last row
        _, _, ak, av = cache._places(t % page)
        cache.bytes[t // page][:, ak] = bad
        cache.bytes[t // page][:, av] = bad
    out, lse = run_attn(bq, dev, q, cache, tab, [n], hkv, page, window=window)
    assert torch.equal(out[:-1], want[0][:-1]) and torch.equal(lse[:-1], want[1][:-1])
    assert torch.isnan(out[-1]).all()


def test_attn_kv4_large_cache_offsets(bq, dev):
    """A page more than 2^32 bytes into the cache."""
    banner("attn offsets past 32 bits")
    T, hq, hkv, d, page = torch.float16, 4, 2, 128, 16
    g = gen(12)
    small = make_cache(g, 3, hkv, d, page, T)
    n = (1 << 32) // small.flat().shape[1] + 5
    cache = torch.zeros(n, small.flat().shape[1], dtype=torch.uint8, device=dev)
    ids = [n - 1, 7, n - 3]
    cache[torch.tensor(ids, device=dev)] = small.flat().to(dev)
    q = torch.randn(1, hq, d, generator=g).to(T)
    lens = torch.tensor([45], dtype=torch.int32, device=dev)
    a = bq.attn_kv4(q.to(dev), cache, torch.tensor([ids], dtype=torch.int32, device=dev), lens, page, hkv)
    b = bq.attn_kv4(q.to(dev), small.flat().to(dev), torch.tensor([[0, 1, 2]], dtype=torch.int32, device=dev), lens, page, hkv)
    k1, v1 = bq.kv4_read(cache, torch.tensor([(n - 1) * page + 3], device=dev), page, hkv, d)
    k2, v2 = bq.kv4_read(small.flat().to(dev), torch.tensor([3], device=dev), page, hkv, d)
    bq.qk_norm_rope_kv4(None, k1, v1, None, None, None, cache, torch.tensor([(n - 1) * page + 9], device=dev), page)
    k3, _ = bq.kv4_read(cache, torch.tensor([(n - 1) * page + 9], device=dev), page, hkv, d)
    torch.cuda.synchronize()
    assert torch.equal(a, b) and torch.equal(k1, k2) and torch.equal(v1, v2)
    # values on a grid of codes keep it, up to the fp16 rounding of their ends
    assert ((k3.float() - k1.float()).abs() <= (k1.float().amax(-1, keepdim=True) - k1.float().amin(-1, keepdim=True)) * 0.04).all()


# ---------------------------------------------------------------- together

def _layer_step(bq, o):
    """One decode step of an attention layer: QKV product, norm, rotation and
    cache write, attention, output product."""
    qkv = bq.gemm_w4g_a16(o["x"], o["wqkv"], o["sqkv"], out=o["qkv"], workspace=o["ws1"])
    r = qkv.view(o["x"].shape[0], o["hq"] + 2 * o["hkv"], o["d"])
    q = bq.qk_norm_rope_kv4(r[:, :o["hq"]], r[:, o["hq"]: o["hq"] + o["hkv"]], r[:, o["hq"] + o["hkv"]:], o["cos"], o["sin"],
                            o["pos"], o["cache"], o["slots"], o["page"], o["wq"], o["wk"], q_out=o["q"])
    bq.attn_kv4(q, o["cache"], o["table"], o["lens"], o["page"], o["hkv"], out=o["o"], lse=o["lse"], workspace=o["ws2"])
    bq.gemm_w4g_a16(o["o"].view(o["x"].shape[0], -1), o["wo"], o["so"], out=o["y"], workspace=o["ws1"])


def _layer_state(bq, dev, T, B=20):
    g = gen(77)
    hq, hkv, d, page, hidden = 8, 2, 128, 16, 512
    lens = [5 + 61 * i for i in range(B)]
    pages = sum(-(-n // page) for n in lens)
    tab = tables(g, lens, page, pages)
    o = dict(hq=hq, hkv=hkv, d=d, page=page)
    dv = lambda t: t.to(dev)  # noqa: E731
    o["x"] = dv(torch.randn(B, hidden, generator=g).to(T))
    n = (hq + 2 * hkv) * d
    for name, shape in (("qkv", (n, hidden)), ("o", (hidden, hq * d))):
        B4, s, _ = layer.quantize_w4g(torch.randn(*shape, generator=g) * 0.04, 64, False)
        o["w" + name], o["s" + name] = dv(B4), dv(s)
    o["cos"], o["sin"] = (dv(t) for t in table(2048, d))
    o["pos"] = dv(torch.tensor(lens, dtype=torch.int32) - 1)
    o["lens"], o["table"] = dv(torch.tensor(lens, dtype=torch.int32)), dv(tab)
    o["slots"] = dv(torch.tensor([int(tab[b, (x - 1) // page]) * page + (x - 1) % page for b, x in enumerate(lens)]))
    o["wq"], o["wk"] = (dv((1 + 0.1 * torch.randn(d, generator=g)).to(T)) for _ in range(2))
    k = torch.randn(pages * page, hkv, d, generator=g).to(T)
    v = torch.randn(pages * page, hkv, d, generator=g).to(T)
    o["cache"] = torch.zeros(pages, bq.kv4_page_bytes(hkv, d, page), dtype=torch.uint8, device=dev)
    bq.qk_norm_rope_kv4(None, dv(k), dv(v), None, None, None, o["cache"], torch.arange(pages * page, device=dev), page)
    o["qkv"] = torch.empty(B, n, dtype=T, device=dev)
    o["q"] = torch.empty(B, hq, d, dtype=T, device=dev)
    o["o"] = torch.empty(B, hq, d, dtype=T, device=dev)
    o["lse"] = torch.empty(B, hq, device=dev)
    o["y"] = torch.empty(B, hidden, dtype=T, device=dev)
    w1 = max(bq.gemm_w4g_workspace_bytes(B, n, hidden), bq.gemm_w4g_workspace_bytes(B, hidden, hq * d), 16)
    w2 = max(bq.attn_kv4_workspace_bytes(B, 1, hq, hkv, d, tab.shape[1] * page), 16)
    o["ws1"], o["ws2"] = (torch.empty(w, dtype=torch.uint8, device=dev) for w in (w1, w2))
    return o, lens, tab


@pytest.mark.parametrize("T", TYPES)
def test_layer_step_together(bq, dev, T):
    """The operators run one after another, each checked against the formulas
    on the inputs it was given."""
    banner(f"layer step {T}")
    o, lens, tab = _layer_state(bq, dev, T)
    _layer_step(bq, o)
    torch.cuda.synchronize()
    B, hq, hkv, d = len(lens), o["hq"], o["hkv"], o["d"]
    qkv = o["qkv"].cpu().view(B, hq + 2 * hkv, d)
    y, size = layer.norm_rope(qkv[:, :hq], o["wq"].cpu(), 1e-6, o["cos"].cpu(), o["sin"].cpu(), o["pos"].cpu(), False)
    within(o["q"], y, half_step(T) * y.abs() + 40 * U * size + 2.0 ** -25, "layer: q")
    ref = layer.Cache(o["cache"].shape[0], hkv, d, o["page"])
    ref.bytes = o["cache"].cpu().view(ref.bytes.shape).clone()
    before = ref.bytes.clone()
    k = layer.round_to(layer.norm_rope(qkv[:, hq: hq + hkv], o["wk"].cpu(), 1e-6, o["cos"].cpu(), o["sin"].cpu(), o["pos"].cpu(),
                                       False)[0], T)
    for b in range(B):
        ref.write(o["slots"][b], k[b], qkv[b, hq + hkv:])
    assert torch.equal(ref.bytes, before), "the cache holds other keys and values"
    check_attn((o["o"], o["lse"]), o["q"].cpu(), ref, tab, lens, list(range(B + 1)), what="layer: attention")
    for a, w, s, c in ((o["x"], "wqkv", "sqkv", o["qkv"]), (o["o"].view(B, -1), "wo", "so", o["y"])):
        W = layer.weights_w4g(o[w].cpu(), o[s].cpu(), None, 64)
        A = a.cpu().to(F64)
        S = A @ W.t()
        big = o[s].cpu().to(F64).repeat_interleave(64, 1)
        tol = half_step(T) * S.abs() + 2.0 ** -13 * (A.abs() @ big.t()) + (A.shape[1] + 64) * U * (A.abs() @ (big * 151).t())
        tol = tol + half_step(T) * (A.abs() @ W.abs().t()) * (1 + 2.0 ** -8)  # 20 rows: each weight rounded once
        within(c, S, tol, "layer: product")


@pytest.mark.parametrize("T", TYPES)
def test_layer_step_captured(bq, dev, T):
    """The step captured in a graph: every replay equals the eager results bit
    for bit, with eager work between replays, on lengths changed in place."""
    banner(f"layer step in a graph {T}")
    o, lens, _ = _layer_state(bq, dev, T)
    outs = ("qkv", "q", "o", "lse", "y", "cache")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        _layer_step(bq, o)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    first = {k: o[k].clone() for k in outs}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        _layer_step(bq, o)
    for rep in range(4):
        if rep == 2:  # other lengths through the same graph
            o["lens"].copy_((o["lens"] + 1) // 2)
            _layer_step(bq, o)
            torch.cuda.synchronize()
            first = {k: o[k].clone() for k in outs}
        for k in outs[:-1]:
            o[k].fill_(3)
        for k in ("ws1", "ws2"):
            o[k].fill_(255)
        _ = (o["cos"] * 2).sum()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for k in outs:
            assert torch.equal(o[k], first[k]), f"replay {rep}: {k}"


def test_layer_other_stream(bq, dev):
    """Calls on a stream of the caller's, ordered with its other work there."""
    banner("layer step on another stream")
    o, _, _ = _layer_state(bq, dev, torch.float16)
    _layer_step(bq, o)
    torch.cuda.synchronize()
    want = o["y"].clone()
    p, _, _ = _layer_state(bq, dev, torch.float16)
    x = p["x"].clone()
    p["x"].zero_()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        torch.cuda._sleep(2_000_000)
        p["x"].copy_(x)
        _layer_step(bq, p)
    s.synchronize()
    assert torch.equal(p["y"], want)


def test_layer_two_streams_at_once(bq, dev):
    """Two streams' calls, each with workspaces of its own, at the same time."""
    banner("layer steps on two streams")
    states = [_layer_state(bq, dev, T)[0] for T in TYPES]
    wants = []
    for o in states:
        _layer_step(bq, o)
        torch.cuda.synchronize()
        wants.append(o["y"].clone())
        o["y"].zero_()
    streams = [torch.cuda.Stream() for _ in states]
    torch.cuda.synchronize()
    for _ in range(8):
        for o, s in zip(states, streams):
            with torch.cuda.stream(s):
                _layer_step(bq, o)
    torch.cuda.synchronize()
    for o, want in zip(states, wants):
        assert torch.equal(o["y"], want)


def test_layer_workspaces_from_the_graphs_pool(bq, dev):
    """Workspaces that the calls allocate themselves under capture: two graphs
    replayed in turn, each against the eager results."""
    banner("layer products and attention in two graphs, workspaces allocated under capture")
    graphs, wants, outs = [], [], []
    for T in TYPES:
        o, _, _ = _layer_state(bq, dev, T, B=18)

        def step(o=o):
            bq.gemm_w4g_a16(o["x"], o["wqkv"], o["sqkv"], out=o["qkv"])
            bq.attn_kv4(o["qkv"].view(18, -1, o["d"])[:, :o["hq"]], o["cache"], o["table"], o["lens"], o["page"], o["hkv"],
                        out=o["o"], lse=o["lse"])

        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            step()
        torch.cuda.synchronize()
        wants.append((o["qkv"].clone(), o["o"].clone(), o["lse"].clone()))
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            step()
        graphs.append(g)
        outs.append((o["qkv"], o["o"], o["lse"]))
    for rep in range(3):
        for g, got, want in zip(graphs, outs, wants):
            for t in got:
                t.fill_(3)
            torch.cuda.synchronize()
            g.replay()
            torch.cuda.synchronize()
            for a, b in zip(got, want):
                assert torch.equal(a, b), f"replay {rep}"


# ---------------------------------------------------------------- index arrays that hold anything

@pytest.mark.parametrize("T", TYPES)
@pytest.mark.parametrize("keys", [40, 1500])
def test_attn_kv4_query_starts_anywhere(bq, dev, T, keys):
    """q_start values at the ends of 32 bits: the queries taken within
    [0, total_q) are computed, every other row stays as it was.  With 1500
    keys the sequences are split."""
    banner(f"attn: q_start at the ends of 32 bits, {keys} keys {T}")
    hq, hkv, d, page = 4, 2, 128, 16
    big, small = 2**31 - 1, -(2**31)
    g = gen(21)
    cache = make_cache(g, -(-keys // page), hkv, d, page, T)
    tab = torch.arange(-(-keys // page), dtype=torch.int32)[None]
    q = torch.randn(6, hq, d, generator=g).to(T)
    for starts, used in (([big, -2], (0, 0)), ([5, small], (0, 0)), ([small, big], (0, 6)), ([small, 2], (0, 2)),
                         ([4, big], (4, 6)), ([6, 9], (0, 0)), ([-1, -2], (0, 0)), ([big, small], (0, 0))):
        out, lse = run_attn(bq, dev, q, cache, tab, [keys], hkv, page, starts, 6)
        lo, hi = used
        if hi > lo:
            check_attn((out[lo:hi], lse[lo:hi]), q[lo:hi], cache, tab, [keys], [0, hi - lo], what=f"starts {starts}")
        for t in (out, lse):
            assert (t[:lo] == 7.0).all() and (t[hi:] == 7.0).all(), f"starts {starts}"


@pytest.mark.parametrize("T", TYPES)
@pytest.mark.parametrize("longest", [50, 1500])
def test_attn_kv4_sequences_longer_than_max_q_len(bq, dev, T, longest):
    """Of sequences with more queries than max_q_len the first max_q_len are
    computed, each at its own position; the others stay as they were.  With
    1500 keys the sequences are split."""
    banner(f"attn: more queries than max_q_len, {longest} keys {T}")
    lens, starts, most, hq, hkv, d, page = [longest, 30, 21], [0, 12, 14, 23], 5, 4, 2, 64, 16
    g = gen(22)
    pages = sum(-(-n // page) for n in lens)
    cache = make_cache(g, pages, hkv, d, page, T)
    tab = tables(g, lens, page, pages)
    q = torch.randn(23, hq, d, generator=g).to(T)
    out, lse = run_attn(bq, dev, q, cache, tab, lens, hkv, page, starts, most)
    want, wlse = run_attn(bq, dev, q, cache, tab, lens, hkv, page, starts, 12)
    check_attn((want, wlse), q, cache, tab, lens, starts, what="all queries")
    for b in range(3):
        n = starts[b + 1] - starts[b]
        # the sequence's computed queries alone, at the end of a shorter cache
        k = min(n, most)
        part = slice(starts[b], starts[b] + k)
        check_attn((out[part], lse[part]), q[part], cache, tab[b: b + 1], [lens[b] - n + k], [0, k], what=f"sequence {b}")
        left = slice(starts[b] + k, starts[b + 1])
        assert (out[left] == 7.0).all() and (lse[left] == 7.0).all(), f"sequence {b}: queries left out"


# ---------------------------------------------------------------- the cache at the ends of fp16's range

def test_kv4_values_outside_fp16s_range(bq, dev):
    """Finite bf16 rows wholly below fp16's range, wholly above it, across its
    ends, and constant: finite parameters, a scale of at least 0, values held
    at what they can express; attention over them stays finite."""
    banner("cache, bf16 values outside fp16's range")
    T, d, page = torch.bfloat16, 128, 16
    g = gen(31)
    u = torch.rand(14, d, generator=g)
    rows = torch.stack([-2e6 - 0 * u[0], -2e6 * (1 + u[1]), -65504 * (1 + u[2]), -1e38 * (0.5 + u[3]), 2e6 + 0 * u[4],
                        7e4 * (1 + u[5]), 1e38 * (0.5 + u[6]), (u[7] - 0.5) * 4e5, (u[8] - 0.5) * 2e38, -1e6 + 0 * u[9],
                        1e-6 + 0 * u[10], -1e-6 - 0 * u[11], 1e-40 * u[12], (u[13] - 0.5) * 1e-6]).to(T)
    n = rows.shape[0]
    cache = torch.full((1, bq.kv4_page_bytes(1, d, page)), 0xA5, dtype=torch.uint8, device=dev)
    x = rows[:, None].to(dev)
    bq.qk_norm_rope_kv4(None, x, x, None, None, None, cache, torch.arange(n, device=dev), page)
    k, v = bq.kv4_read(cache, torch.arange(n, device=dev), page, 1, d, T)
    torch.cuda.synchronize()
    ref = layer.Cache(1, 1, d, page, 0xA5)
    for t in range(n):
        ref.write(t, rows[t][None], rows[t][None])
    assert torch.equal(cache.cpu(), ref.flat())
    x = rows.to(F64)
    for t in range(n):
        (q, s, m), _ = ref.read(t)
        assert torch.isfinite(s).all() and torch.isfinite(m).all() and float(s) >= 0
        # the nearest code's value, where the parameters reach the value: half a
        # step, the parameters' own roundings (15 codes of the scale's, the
        # minimum's) and bf16's on reading
        want = x[t].clamp(-65504, float(m) + 15 * 65504)
        tol = float(s) * (0.5 + 15 * 2.0 ** -11) + 15 * 2.0 ** -25 + abs(float(m)) * 2.0 ** -11 + 2.0 ** -25
        for got in (k, v):
            got = got[t, 0].cpu().to(F64)
            assert torch.isfinite(got).all()
            assert ((got - want).abs() <= tol + (want.abs() + tol) * 2.0 ** -8).all(), f"row {t}"
    q = torch.zeros(1, 2, d, dtype=T)
    q[0, 0, 0] = 1e-3
    out, lse = run_attn(bq, dev, q, ref, torch.zeros(1, 1, dtype=torch.int32), [n], 1, page)
    assert torch.isfinite(out).all() and torch.isfinite(lse).all()
    check_attn((out, lse), q, ref, torch.zeros(1, 1, dtype=torch.int32), [n], [0, 1], what="ends of the range")


# ---------------------------------------------------------------- keys that a row does not see

def _set_params(cache, tokens, k, v, page):
    """fp16 (scale, min) of K and of V at the tokens of pages 0, 1, ..."""
    for t in tokens:
        _, _, ak, av = cache._places(t % page)
        for at, par in ((ak, k), (av, v)):
            cache.bytes[t // page][:, at] = torch.tensor(par).half().view(torch.uint8)


@pytest.mark.parametrize("T", TYPES)
@pytest.mark.parametrize("hq,d", [(2, 64), (8, 128), (64, 64), (2, 256)])
@pytest.mark.parametrize("k,v", [([65504.0, 65504.0], [65504.0, 65504.0]), ([0.0, -65504.0], [65504.0, -65504.0]),
                                 ([0.0, 0.0], [1000.0, 0.0])])
def test_attn_kv4_unseen_keys_change_no_bit(bq, dev, T, hq, d, k, v):
    """Large finite parameters of keys before every window, and of the last
    keys, which only the last rows see: the other rows, whose own V scales are
    small, keep every bit."""
    banner(f"attn: unseen keys of large scale {hq} {d} {k} {v} {T}")
    n, ql, hkv, page = 150, 8, 1, 16
    g = gen(41)
    q = torch.randn(ql, hq, d, generator=g).to(T)
    for window, last in ((40, 1), (0, 4)):
        cache = make_cache(g, 10, hkv, d, page, T, v_mul=1e-2)
        tab = torch.arange(10, dtype=torch.int32)[None]
        want = run_attn(bq, dev, q, cache, tab, [n], hkv, page, window=window)
        check_attn(want, q, cache, tab, [n], [0, ql], window, what="clean")
        before = list(range(0, n - ql - window + 1)) if window else []
        _set_params(cache, before + list(range(n - last, n)), k, v, page)
        out, lse = run_attn(bq, dev, q, cache, tab, [n], hkv, page, window=window)
        assert torch.equal(out[:-last], want[0][:-last]) and torch.equal(lse[:-last], want[1][:-last])
        assert not torch.equal(out[-last:], want[0][-last:])


@pytest.mark.parametrize("T", TYPES)
@pytest.mark.parametrize("spread", [2.0 ** 8, 2.0 ** 14])
def test_attn_kv4_one_large_v_scale(bq, dev, T, spread):
    """A key that every row sees, of a V scale far above the others' and of
    small weight: p times a scale is also held to 2^-29 of the row's largest p
    times that scale, which is then the larger error (centred codes of
    magnitude at most 8, n keys)."""
    banner(f"attn: one V scale {spread} times the others {T}")
    n, hq, hkv, d, page = 300, 4, 1, 128, 16
    g = gen(42)
    cache = make_cache(g, 19, hkv, d, page, T, k_off=0.0, v_mul=1e-2)
    tab = torch.arange(19, dtype=torch.int32)[None]
    s = 1e-2 * 5 / 15 * spread
    _set_params(cache, [77], [0.0, 0.0], [s, -8 * s], page)
    q = torch.randn(1, hq, d, generator=g).to(T) * 4
    out, lse = run_attn(bq, dev, q, cache, tab, [n], hkv, page)
    want, wlse, size, delta = layer.attention(q, cache, tab, [n], [0, 1], d ** -0.5)
    r = (2.0 ** -20 if T == torch.float16 else 2.0 ** -10 + 2.0 ** -20) + n * U
    tol = half_step(T) * want.abs() + (2 * delta[..., None] + r) * size * (1 + 2.0 ** -6) + 2.0 ** -25 + n * 8 * s * 2.0 ** -29
    within(out, want, tol, "one large V scale")


@pytest.mark.parametrize("T", TYPES)
@pytest.mark.parametrize("d,ql", [(64, 20), (128, 1), (256, 3)])
@pytest.mark.parametrize("v_mul", [1.0, 3000.0])
def test_attn_kv4_negative_scales(bq, dev, T, d, ql, v_mul):
    """A page may hold negative scales: all of V's, or every third one, and
    half of K's."""
    banner(f"attn: negative scales d={d} q={ql} {v_mul} {T}")
    n, hq, hkv, page = 200, 4, 2, 16
    g = gen(43)
    for every in (1, 3):
        cache = make_cache(g, 13, hkv, d, page, T, v_mul=v_mul)
        plain = layer.Cache(13, hkv, d, page)
        for t in range(n):
            _, _, ak, av = cache._places(t % page)
            if t % 2:
                cache.bytes[t // page][:, ak[1]] ^= 128
        plain.bytes = cache.bytes.clone()
        for t in range(0, n, every):
            _, _, ak, av = cache._places(t % page)
            cache.bytes[t // page][:, av[1]] ^= 128
        tab = torch.arange(13, dtype=torch.int32)[None]
        q = torch.randn(ql, hq, d, generator=g).to(T)
        out, lse = run_attn(bq, dev, q, cache, tab, [n], hkv, page)
        want, wlse, _, delta = layer.attention(q, cache, tab, [n], [0, ql], d ** -0.5)
        _, _, size, _ = layer.attention(q, plain, tab, [n], [0, ql], d ** -0.5)  # the terms' magnitudes
        # K's scales of either sign: the score's bound takes their sizes
        for t in range(n):
            _, _, ak, _ = plain._places(t % page)
            plain.bytes[t // page][:, ak[1]] &= 127
        _, _, _, delta = layer.attention(q, plain, tab, [n], [0, ql], d ** -0.5)
        r = (2.0 ** -20 if T == torch.float16 else 2.0 ** -10 + 2.0 ** -20) + n * U
        within(out, want, half_step(T) * want.abs() + (2 * delta[..., None] + r) * size * (1 + 2.0 ** -6) + 2.0 ** -25, f"every {every}")
        off = (lse.cpu().to(F64) - wlse).abs() - (delta + 2.0 ** -20 * (1 + wlse.abs()))
        assert (off <= 0).all()


def test_attn_kv4_room_for_many_queries(bq, dev):
    """max_q_len far above the queries that there are: 2^24 query rows of room
    on 2^19 workgroups, none split."""
    banner("attn: room for 2^24 query rows")
    T, B, most, hkv, d, page = torch.float16, 8, 2**18, 8, 64, 16
    g = gen(51)
    lens, starts = [20] * B, list(range(B + 1))
    cache = make_cache(g, 2 * B, hkv, d, page, T)
    tab = tables(g, lens, page, 2 * B)
    q = torch.randn(B, hkv, d, generator=g).to(T)
    got = run_attn(bq, dev, q, cache, tab, lens, hkv, page, starts, most)
    check_attn(got, q, cache, tab, lens, starts, what="room")


@pytest.mark.parametrize("T", TYPES)
def test_layer_empty_calls(bq, dev, T):
    """A batch of no sequences, sequences of no queries, no tokens: empty
    results, nothing launched, nothing written."""
    banner(f"empty calls {T}")
    hq, hkv, d, page = 4, 2, 128, 16
    cache = torch.full((3, bq.kv4_page_bytes(hkv, d, page)), 0xA5, dtype=torch.uint8, device=dev)
    q = torch.empty(0, hq, d, dtype=T, device=dev)
    k = torch.empty(0, hkv, d, dtype=T, device=dev)
    ints = lambda *s: torch.zeros(s, dtype=torch.int32, device=dev)  # noqa: E731
    for batch in (0, 2):
        out, lse = bq.attn_kv4(q, cache, ints(batch, 3), ints(batch), page, hkv, return_lse=True)
        assert out.shape == q.shape and lse.shape == (0, hq)
        out = bq.attn_kv4(q, cache, ints(batch, 3), ints(batch), page, hkv, q_start=ints(batch + 1), max_q_len=4)
        assert out.shape == q.shape
    with pytest.raises(ValueError):
        bq.attn_kv4(torch.empty(1, hq, d, dtype=T, device=dev), cache, ints(0, 3), ints(0), page, hkv)
    assert bq.qk_norm_rope_kv4(q, k, k, None, None, None, cache, torch.empty(0, dtype=torch.int64, device=dev), page).shape == q.shape
    a, b = bq.qk_norm_rope(q, k, None, None, None)
    assert a.shape == q.shape and b.shape == k.shape
    a, b = bq.kv4_read(cache, torch.empty(0, dtype=torch.int64, device=dev), page, hkv, d, T)
    assert a.shape == k.shape and b.shape == k.shape
    w = torch.zeros(8, 64, dtype=torch.uint8, device=dev)
    s = torch.ones(8, 1, dtype=torch.float16, device=dev)
    assert bq.gemm_w4g_a16(torch.empty(0, 128, dtype=T, device=dev), w, s).shape == (0, 8)
    assert bq.gemm_w4g_a16(torch.zeros(3, 128, dtype=T, device=dev), w[:0], s[:0]).shape == (3, 0)
    torch.cuda.synchronize()
    assert (cache == 0xA5).all()


# ---------------------------------------------------------------- w4g, to the sums' own bound

def run_w4g(bq, dev, A, B, s, z, **kw):
    return bq.gemm_w4g_a16(A.to(dev), B.to(dev), s.to(dev), None if z is None else z.to(dev), **kw)


@pytest.mark.parametrize("shape", W4G_ALL)
@pytest.mark.parametrize("T", TYPES)
@pytest.mark.parametrize("zero", [False, True])
def test_w4g_closely(bq, dev, shape, T, zero):
    """Every kernel and tile to oracle.layer.w4g_bound, which notices a lost
    step of K or another group's scale; twice the same bits; and without a
    workspace."""
    M, N, K, group = shape
    banner(f"w4g closely M={M} N={N} K={K} group={group} zero={zero} {T}")
    A, B, s, z = w4g_inputs(M, N, K, group, zero, T)
    S, tol = layer.w4g_bound(A, B, s, z, group)
    out = run_w4g(bq, dev, A, B, s, z)
    torch.cuda.synchronize()
    within(out, S, tol, f"w4g {shape} {T}")
    again = run_w4g(bq, dev, A, B, s, z)
    alone = run_w4g(bq, dev, A, B, s, z, workspace=torch.empty(16, dtype=torch.uint8, device=dev))
    torch.cuda.synchronize()
    assert torch.equal(out, again)
    within(alone, S, tol, f"w4g {shape} {T} without a workspace")


@pytest.mark.parametrize("shape", W4G_ALL)
@pytest.mark.parametrize("T", TYPES)
def test_w4g_windows(bq, dev, shape, T):
    """Rows of A that are zero but for 32 k, the first and the last among them:
    the codes, scales and zero points of exactly those."""
    M, N, K, group = shape
    banner(f"w4g windows M={M} N={N} K={K} group={group} {T}")
    _, B, s, z = w4g_inputs(M, N, K, group, True, T)
    for A, _ in w4g_windows(M, K, T):
        S, tol = layer.w4g_bound(A, B, s, z, group)
        out = run_w4g(bq, dev, A, B, s, z)
        torch.cuda.synchronize()
        within(out, S, tol, f"w4g windows {shape} {T}")


@pytest.mark.parametrize("shape", W4G_LARGE + W4G_TALL)
def test_w4g_large_tiles_write_their_outputs_only(bq, dev, shape):
    """Ragged edges of the large tiles: nothing before or behind the output."""
    M, N, K, group = shape
    banner(f"w4g large tiles' edges M={M} N={N} K={K}")
    A, B, s, z = w4g_inputs(M, N, K, group, True, torch.float16)
    whole = torch.full((M * N + 512,), 7.0, dtype=torch.float16, device=dev)
    out = whole[256: 256 + M * N].view(M, N)
    run_w4g(bq, dev, A, B, s, z, out=out)
    torch.cuda.synchronize()
    assert (whole[:256] == 7.0).all() and (whole[256 + M * N:] == 7.0).all()
    S, tol = layer.w4g_bound(A, B, s, z, group)
    within(out, S, tol, f"w4g {shape}")


# ---------------------------------------------------------------- attention: splits of two row tiles, and of ragged queries

@pytest.mark.parametrize("T", TYPES)
@pytest.mark.parametrize("ws", ["auto", "none", "full"])
@pytest.mark.parametrize("lens,ql,hq,hkv,d,page,window", [([1300], 20, 2, 2, 64, 16, 0), ([1100, 70, 1537], 9, 4, 1, 64, 32, 0),
                                                          ([2100, 3], 17, 2, 2, 64, 64, 1500), ([1400, 1200], 40, 2, 2, 128, 16, 0)])
def test_attn_kv4_split_row_tiles(bq, dev, T, ws, lens, ql, hq, hkv, d, page, window):
    """More than 16 query rows a kv head over sequences that are split."""
    banner(f"attn: split, two row tiles {lens} {ql} {d} {window} {T} {ws}")
    test_attn_kv4(bq, dev, (lens, ql, hq, hkv, d, page, window), T, ws)


@pytest.mark.parametrize("T", TYPES)
@pytest.mark.parametrize("d,hkv", [(64, 1), (128, 2), (256, 1)])
@pytest.mark.parametrize("window", [0, 1100])
def test_attn_kv4_split_ragged_queries(bq, dev, T, d, hkv, window):
    """q_start over sequences that are split: of 0, 1, 13 and 3 queries, one
    of more queries than keys, rows behind the last left as they were."""
    banner(f"attn: split, ragged queries d={d} {window} {T}")
    lens, starts, hq, page = [1500, 1203, 1300, 0, 5, 40], [0, 1, 1, 14, 17, 26, 29], 4, 32
    g = gen(61)
    pages = sum(-(-n // page) for n in lens)
    cache = make_cache(g, pages, hkv, d, page, T)
    tab = tables(g, lens, page, pages)
    rows = torch.randn(33, hq + 2, d, generator=g).to(T)
    x = rows.to(dev)
    for ws in ("auto", "none"):
        got = run_attn(bq, dev, rows[:, :hq], cache, tab, lens, hkv, page, starts, 13, window=window, ws=ws, q_dev=x[:, :hq])
        check_attn(got, rows[:, :hq], cache, tab, lens, starts, window, what="split, ragged")


@pytest.mark.parametrize("T", TYPES)
@pytest.mark.parametrize("sign", [1, -1])
def test_attn_kv4_large_scales_and_rising_scores(bq, dev, T, sign):
    """V scales of about 2000, of either sign, and scores that rise along the
    sequence by just less than what raises the reference maximum (2^7.5 of
    2^8): p times the scale stays within fp16's range."""
    banner(f"attn: rising scores over large V scales of sign {sign} {T}")
    n, hq, hkv, d, page = 700, 2, 1, 64, 16
    g = gen(44)
    cache = make_cache(g, 44, hkv, d, page, T, v_mul=6000.0)
    tab = torch.arange(44, dtype=torch.int32)[None]
    for t in range(n):
        _, _, ak, av = cache._places(t % page)
        rise = 7.5 * math.log(2) * (t >= 256)  # of the score: 1/8 per unit of q's sum, which is 8
        cache.bytes[t // page][:, ak] = torch.tensor([0.0, rise]).half().view(torch.uint8)
        if sign < 0:
            cache.bytes[t // page][:, av[1]] ^= 128
    q = torch.full((1, hq, d), 0.125).to(T)
    out, lse = run_attn(bq, dev, q, cache, tab, [n], hkv, page)
    want, wlse, size, delta = layer.attention(q, cache, tab, [n], [0, 1], d ** -0.5)
    if sign < 0:  # the terms' magnitudes: |scale|
        for t in range(n):
            cache.bytes[t // page][:, cache._places(t % page)[3][1]] &= 127
        _, _, size, delta = layer.attention(q, cache, tab, [n], [0, 1], d ** -0.5)
    r = (2.0 ** -20 if T == torch.float16 else 2.0 ** -10 + 2.0 ** -20) + n * U
    within(out, want, half_step(T) * want.abs() + (2 * delta[..., None] + r) * size * (1 + 2.0 ** -6) + 2.0 ** -25, "rising")
    assert ((lse.cpu().to(F64) - wlse).abs() <= delta + 2.0 ** -20 * (1 + wlse.abs())).all()


@pytest.mark.parametrize("T", TYPES)
@pytest.mark.parametrize("c", [(40, 4, 2, 128, 16), (2600, 8, 8, 64, 32), (33, 0, 3, 256, 64)])
def test_qk_norm_rope_kv4_positions_outside_the_table(bq, dev, T, c):
    """A token left out for its position writes neither its query nor the
    cache; slots at the ends of 64 bits are not followed; the others are
    written as alone."""
    banner(f"cache, positions outside the table {c} {T}")
    tokens, hq, hkv, d, page = c
    g = gen(71 + tokens)
    rows = (torch.randn(tokens, hq + 2 * hkv, d, generator=g) * 2).to(T)
    cos, sin = table(64, d)
    pos = torch.randint(0, 64, (tokens,), generator=g, dtype=torch.int32)
    slots = torch.randperm(tokens + 9, generator=g)[:tokens].contiguous()
    bad = {1: -1, 2: 64, 5: 2**31 - 1, 30: -(2**31)}
    for t, p in bad.items():
        pos[t] = p
    slots[3], slots[7], slots[20] = 2**63 - 1, -(2**63), 1 << 40
    pages = -(-(tokens + 9) // page)
    out = []
    for keep in (None, [t for t in range(tokens) if t not in bad and t not in (3, 7, 20)]):
        x, p, s = (rows, pos, slots) if keep is None else (rows[keep], pos[keep], slots[keep])
        x = x.to(dev)
        cache = torch.full((pages, bq.kv4_page_bytes(hkv, d, page)), 0xA5, dtype=torch.uint8, device=dev)
        q = torch.full((x.shape[0], hq, d), 7.0, dtype=T, device=dev) if hq else None
        bq.qk_norm_rope_kv4(x[:, :hq] if hq else None, x[:, hq: hq + hkv], x[:, hq + hkv:], cos.to(dev), sin.to(dev), p.to(dev),
                            cache, s.to(dev), page, q_out=q)
        torch.cuda.synchronize()
        out.append((cache, q))
    assert torch.equal(out[0][0], out[1][0])
    if hq:
        assert torch.equal(out[0][1][keep], out[1][1])
        assert (out[0][1][list(bad)] == 7.0).all()
        assert (out[0][1][[3, 7, 20]] != 7.0).any(-1).all()  # their queries are written
    k, v = bq.kv4_read(out[0][0], torch.tensor([2**63 - 1, -(2**63), -1, 1 << 40], device=dev), page, hkv, d, T,
                       *(torch.full((4, hkv, d), 7.0, dtype=T, device=dev) for _ in range(2)))
    torch.cuda.synchronize()
    assert (k == 7.0).all() and (v == 7.0).all()
