"""GPU parity of the decoding operators against oracle/decode.py.

Bounds: masks, positions, paths, tokens and moved bytes are whole numbers and
equal.  A sampled token's choice lies at a border between two sums; the kernel
holds weights as multiples of 2^-F of the greatest, F = min(46, 61 -
ceil(log2 vocab)): each is off by 2^-(F + 1) for its rounding and by at most
2^-50 (2^-(F + 4)) before it, so a sum of up to vocab of them by 1.125 vocab
2^-(F + 1), and two sums that are compared by 1.125 vocab 2^-F of the greatest
weight, which all kept ones together are not less than: an input whose nearest
border is farther than that, relative to the kept sum, decides its token (that
all inputs here are such ones is asserted).  Log probabilities: the logarithm's
argument is exact to 2^-24, its rounding 2^-24 of itself: 2^-22 (1 + |lp|).
Attention: the bounds of attn_kv4 (test_gpu_layer.py).
"""
import math

import numpy as np
import pytest
import torch

from decode_cases import gen, logits_row, sample_wants, trees
from gpu_util import banner, need_gpu
from oracle import decode, layer
from test_gpu_layer import half_step, make_cache, table, tables, within

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


def i32(x, dev):
    return torch.as_tensor(x, dtype=torch.int32).to(dev)


# ---------------------------------------------------------------- trees

@pytest.mark.parametrize("nodes", [1, 2, 25, 31, 32, 33, 64, 65, 200, 257, 1000, 1024])
def test_tree_mask(bq, dev, nodes):
    banner(f"tree_mask {nodes}")
    for chain in (0.0, 0.4, 1.0):
        parents, see, want, depths = trees(gen(nodes), [nodes] * 3, chain=chain)
        lens = [nodes, nodes + 77, 5]
        mask, pos = bq.tree_mask(parents.view(3, nodes).to(dev), i32(lens, dev))
        assert torch.equal(mask.cpu(), want)
        assert pos.tolist() == [lens[i // nodes] - nodes + d for i, d in enumerate(depths)]
        _, depth = bq.tree_mask(parents.view(3, nodes).to(dev))
        assert depth.tolist() == depths


def test_tree_mask_ragged(bq, dev):
    """Trees of several sizes, none among them, rows behind the last left as
    they were, more words than the nodes need and fewer, parents that are none."""
    banner("tree_mask ragged")
    nodes = [7, 0, 40, 1, 70]
    parents, see, _, depths = trees(gen(1), nodes)
    parents[3], parents[9], parents[20] = 99, -7, 15  # roots of their own: after, before, itself (node 13 of tree 2)
    parents[7 + 13] = 13
    starts = [0, 7, 7, 47, 48, 118]
    want, depths = [], []
    for a, b in zip(starts, starts[1:]):
        s, d = decode.ancestors(parents[a:b].tolist())
        want.append(s)
        depths += d
    lens = [10, 4, 100, 1, 70]
    first = [n - (b - a) for n, a, b in zip(lens, starts, starts[1:])]
    for words in (1, 2, 3, 9):
        mask = torch.full((125, words), 7, dtype=torch.int32, device=dev)
        pos = torch.full((125,), 7, dtype=torch.int32, device=dev)
        padded = torch.cat([parents, torch.full((7,), 3, dtype=torch.int32)])
        bq.tree_mask(padded.to(dev), i32(lens, dev), i32(starts, dev), 70, mask, pos)
        got = mask.cpu()
        for b, (a, e) in enumerate(zip(starts, starts[1:])):
            assert torch.equal(got[a:e], decode.words_of(want[b], words)), (words, b)
            assert pos[a:e].tolist() == [first[b] + d for d in depths[a:e]]
        assert (got[118:] == 7).all() and (pos[118:] == 7).all()
    # the first 30 nodes of each tree only
    mask = torch.full((118, 2), 7, dtype=torch.int32, device=dev)
    bq.tree_mask(parents.to(dev), None, i32(starts, dev), 30, mask)
    got = mask.cpu()
    for b, (a, e) in enumerate(zip(starts, starts[1:])):
        m = min(30, e - a)
        assert torch.equal(got[a: a + m], decode.words_of(want[b][:m], 2))
        assert (got[a + m: e] == 7).all()
    # starts outside the nodes are taken within them
    a, _ = bq.tree_mask(parents.to(dev), None, i32([-5, 7, 7, 47, 48, 1 << 30], dev), 70)
    b, _ = bq.tree_mask(parents.to(dev), None, i32(starts, dev), 70)
    assert torch.equal(a, b)


@pytest.mark.parametrize("nodes", [1, 2, 25, 64, 65, 300, 1024])
def test_tree_accept(bq, dev, nodes):
    banner(f"tree_accept {nodes}")
    g = gen(nodes)
    for chain, vocab in ((0.2, 3), (1.0, 1), (0.5, 2)):
        parents, _, _, _ = trees(g, [nodes] * 5, chain=chain)
        tokens = torch.randint(0, vocab, (5, nodes), generator=g, dtype=torch.int32)
        sampled = torch.randint(0, vocab, (5, nodes), generator=g, dtype=torch.int32)
        parents = parents.view(5, nodes)
        for most in (None, 1, 3, nodes):
            path, count, last = bq.tree_accept(tokens.to(dev), parents.to(dev), sampled.to(dev).view(-1), max_path=most)
            for b in range(5):
                want, end = decode.accept(tokens[b].tolist(), parents[b].tolist(), sampled[b].tolist(), most or nodes)
                assert path[b].tolist() == want + [-1] * (path.shape[1] - len(want))
                assert int(count[b]) == len(want) and int(last[b]) == end


def test_tree_accept_ragged(bq, dev):
    """No nodes, one node, nodes that no node before them is the parent of."""
    banner("tree_accept ragged")
    g = gen(2)
    nodes, starts = [3, 0, 1, 40], [0, 3, 3, 4, 44]
    parents, _, _, _ = trees(g, nodes)
    tokens = torch.zeros(44, dtype=torch.int32)
    sampled = torch.zeros(44, dtype=torch.int32)
    parents[2], parents[10], parents[12] = 2, 30, -4
    path, count, last = bq.tree_accept(tokens.to(dev), parents.to(dev), sampled.to(dev), i32(starts, dev), 40)
    for b, (a, e) in enumerate(zip(starts, starts[1:])):
        p = [x if 0 <= x < i else -9 for i, x in enumerate(parents[a:e].tolist())]
        want, end = decode.accept(tokens[a:e].tolist(), p, sampled[a:e].tolist(), 40)
        assert path[b].tolist() == want + [-1] * (40 - len(want)) and int(count[b]) == len(want) and int(last[b]) == end


# ---------------------------------------------------------------- the cache's move

@pytest.mark.parametrize("hkv,d,page", [(1, 64, 16), (2, 128, 16), (3, 256, 32), (5, 64, 128), (8, 128, 256)])
@pytest.mark.parametrize("layers", [1, 3])
def test_kv4_compact(bq, dev, hkv, d, page, layers):
    banner(f"kv4_compact {hkv} {d} {page} x {layers}")
    g = gen(hkv + d + page + layers)
    nodes = [20, 1, 33, 0, 7, 50]
    starts = np.cumsum([0] + nodes).tolist()
    lens = [20, 77, 33 + page, 3, 5, 2 * page + 51]  # no prefix; fewer keys than nodes in sequence 4
    paths = [[0, 1, 2, 3], [0], [0, 2, 3, 9, 32, 32, 40], [0, 1], [0, 3, 4, 5, 6], [0, 3, 1, 3, 17, 49, -1, 48]]
    counts = [4, 1, 7, 2, 5, 99]
    most = 8
    pages = sum(-(-n // page) for n in lens) + 1
    tab = tables(g, lens, page, pages)
    caches = []
    for _ in range(layers):
        c = layer.Cache(pages, hkv, d, page)
        c.bytes = torch.randint(0, 256, c.bytes.shape, generator=g, dtype=torch.uint8)
        caches.append(c)
    room = torch.full((layers, pages * caches[0].flat().shape[1] + 48), 7, dtype=torch.uint8, device=dev)
    cache = room[:, : pages * caches[0].flat().shape[1]].view(layers, pages, -1)  # layers that lie apart
    for i, c in enumerate(caches):
        cache[i].copy_(c.flat())
    path = torch.full((len(nodes), most), -1, dtype=torch.int32)
    for b, p in enumerate(paths):
        path[b, : len(p)] = torch.tensor(p)
    got = bq.kv4_compact(cache if layers > 1 else cache[0], tab.to(dev), i32(lens, dev), path.to(dev), i32(counts, dev), page, hkv, d,
                         i32(starts, dev), total_q=starts[-1])
    torch.cuda.synchronize()
    assert got.data_ptr() == cache.data_ptr()
    for i, c in enumerate(caches):
        for b, n in enumerate(nodes):
            decode.compact(c, tab[b], lens[b], n, path[b, : counts[b]].tolist())
        assert torch.equal(cache[i].cpu(), c.flat()), f"layer {i}"
    assert (room[:, pages * caches[0].flat().shape[1]:] == 7).all()


def test_kv4_compact_bad_pages(bq, dev):
    """Pages outside the cache, lengths outside the table, counts below 0."""
    banner("kv4_compact bad pages")
    g = gen(31)
    hkv, d, page = 2, 128, 16
    c = layer.Cache(6, hkv, d, page)
    c.bytes = torch.randint(0, 256, c.bytes.shape, generator=g, dtype=torch.uint8)
    tab = torch.tensor([[0, 1 << 30], [-1, 2], [3, 4], [5, 5]], dtype=torch.int32)
    lens, counts, nodes = [32, 32, 1 << 30, 32], [4, 4, 4, -3], 20
    path = torch.tensor([[0, 3, 9, 19]] * 4, dtype=torch.int32)
    cache = c.flat().to(dev)
    bq.kv4_compact(cache, tab.to(dev), i32(lens, dev), path.to(dev), i32(counts, dev), page, hkv, d, max_q_len=nodes)
    for b in range(4):
        decode.compact(c, tab[b], lens[b], nodes, path[b, : max(counts[b], 0)].tolist())
    assert torch.equal(cache.cpu(), c.flat())


# ---------------------------------------------------------------- sampling

def border(vocab):
    return 1.125 * vocab * 2.0 ** -min(46, 61 - math.ceil(math.log2(vocab)))


def check_sample(got, x, u, t=None, k=None, p=None, m=None, exact=False):
    tokens, logp = got
    want, lp, margin = sample_wants(x, u, t, k, p, m)
    assert exact or (margin > border(x.shape[1])).all(), "an input at a border"
    got_tokens, got_lp = tokens.cpu().numpy(), logp.cpu().numpy().astype(np.float64)
    bad = np.nonzero(got_tokens != want)[0]
    assert not len(bad), f"rows {bad[:5]}: {got_tokens[bad[:5]]} for {want[bad[:5]]}, margins {margin[bad[:5]]}"
    none = want < 0
    assert (got_lp[none] == -math.inf).all()
    off = np.abs(got_lp[~none] - lp[~none]) - 2.0 ** -22 * (1 + np.abs(lp[~none]))
    assert (off <= 0).all(), f"log probability off by {off.max()}"


def on(v, dev):
    return None if v is None else v.to(dev)


SIZES = [(3, 1), (5, 2), (4, 7), (3, 63), (3, 64), (3, 65), (2, 1000), (3, 1023), (2, 1024), (3, 1025), (2, 4097), (9, 8191), (3, 32000),
         (2, 50021), (5, 131072), (1, 200001)]
FILTERS = ["", "k", "p", "m", "kp", "km", "pm", "kpm"]


def sample_settings(g, rows, filters, vocab):
    u = torch.rand(rows, generator=g)
    t = 0.3 + 1.2 * torch.rand(rows, generator=g)
    k = torch.randint(1, min(vocab, 200) + 1, (rows,), generator=g, dtype=torch.int32) if "k" in filters else None
    p = torch.rand(rows, generator=g) if "p" in filters else None
    m = torch.rand(rows, generator=g) * 0.2 if "m" in filters else None
    return u, t, k, p, m


@pytest.mark.parametrize("rows,vocab", SIZES)
@pytest.mark.parametrize("T", TYPES + [torch.float32])
def test_sample(bq, dev, rows, vocab, T):
    banner(f"sample {rows} x {vocab} {T}")
    g = gen(vocab)
    for filters in FILTERS:
        x = torch.stack([logits_row(g, vocab, 12.0 * (i % 3) / 2, T) for i in range(rows)])
        args = sample_settings(g, rows, filters, vocab)
        got = bq.sample(x.to(dev), *(on(v, dev) for v in args))
        check_sample(got, x, *args)


@pytest.mark.parametrize("T", TYPES + [torch.float32])
@pytest.mark.parametrize("ws", ["auto", "none", "full"])
def test_sample_many_rows(bq, dev, T, ws):
    """Many rows, each with other settings, some off and some greedy; rows
    strided and off 16-byte boundaries; with and without a workspace."""
    banner(f"sample many rows {T} {ws}")
    g = gen(77)
    rows, vocab = 300, 1531
    x = torch.stack([logits_row(g, vocab, 9.0 * (i % 4) / 3, T) for i in range(rows)])
    u, t, k, p, m = sample_settings(g, rows, "kpm", vocab)
    off = torch.rand(rows, 4, generator=g) < 0.4
    t, k, p, m = t * ~off[:, 0], k * ~off[:, 1], torch.where(off[:, 2], torch.ones(rows), p), m * ~off[:, 3]
    kw = {}
    if ws == "none":
        kw["workspace"] = torch.empty(16, dtype=torch.uint8, device=dev)
    elif ws == "full":
        kw["workspace"] = torch.full((max(16, bq.sample_workspace_bytes(rows, vocab, T)),), 255, dtype=torch.uint8, device=dev)
    for lead, tail in ((0, 0), (1, 2), (3, 10)):
        room = torch.full((rows, lead + vocab + tail), 99.0, dtype=T, device=dev)
        view = room[:, lead: lead + vocab]
        view.copy_(x)
        got = bq.sample(view, *(on(v, dev) for v in (u, t, k, p, m)), **kw)
        check_sample(got, x, u, t, k, p, m)


@pytest.mark.parametrize("T", TYPES + [torch.float32])
@pytest.mark.parametrize("vocab", [70, 3001, 40000])
def test_sample_flat_and_equal(bq, dev, T, vocab):
    """Rows of equal logits, where all sums are exact: the choice falls where
    the definition puts it, equal logits by index."""
    banner(f"sample equal logits {vocab} {T}")
    x = torch.full((8, vocab), -2.5).to(T)
    x[4:, vocab // 3:] = -math.inf
    n = [vocab] * 4 + [vocab // 3] * 4
    u = torch.tensor([0.0, 0.5, 0.71, 1 - 2.0 ** -24] * 2)
    for t in (None, torch.full((8,), 0.37)):
        tokens, logp = bq.sample(x.to(dev), u.to(dev), on(t, dev))
        assert tokens.tolist() == [math.floor(float(u[i]) * n[i]) for i in range(8)]
        assert np.allclose(logp.cpu().numpy(), [-math.log(v) for v in n], rtol=1e-6)
        k = torch.tensor([1, 3, 50, 60] * 2, dtype=torch.int32)
        tokens, _ = bq.sample(x.to(dev), u.to(dev), on(t, dev), k.to(dev))
        assert tokens.tolist() == [math.floor(float(u[i]) * min(int(k[i]), n[i])) for i in range(8)]
        p = torch.tensor([0.5, 0.25, 0.125, 0.0] * 2)
        keep = [max(1, math.ceil(float(p[i]) * n[i])) for i in range(8)]
        tokens, _ = bq.sample(x.to(dev), u.to(dev), on(t, dev), None, p.to(dev))
        assert tokens.tolist() == [math.floor(float(u[i]) * keep[i]) for i in range(8)]
        k, p = torch.full((8,), 40, dtype=torch.int32), torch.full((8,), 0.5)
        keep = [math.ceil(0.5 * min(40, n[i])) for i in range(8)]
        tokens, _ = bq.sample(x.to(dev), u.to(dev), on(t, dev), k.to(dev), p.to(dev))
        assert tokens.tolist() == [math.floor(float(u[i]) * keep[i]) for i in range(8)]


@pytest.mark.parametrize("T", TYPES + [torch.float32])
def test_sample_few_values(bq, dev, T):
    """Logits of few distinct values: the limit falls among equals."""
    banner(f"sample few values {T}")
    g = gen(6)
    rows, vocab = 40, 5003
    x = (torch.randint(0, 6, (rows, vocab), generator=g).float() * 0.75 - 3).to(T)
    for filters in FILTERS:
        args = list(sample_settings(g, rows, filters, vocab))
        if args[2] is not None:
            args[2] = args[2] * 20
        check_sample(bq.sample(x.to(dev), *(on(v, dev) for v in args)), x, *args)


@pytest.mark.parametrize("T", TYPES + [torch.float32])
@pytest.mark.parametrize("vocab", [65, 2500, 33000])
def test_sample_masked_and_odd_logits(bq, dev, T, vocab):
    """-inf, NaN, +inf, the type's lowest value, -0 against 0, all of them."""
    banner(f"sample masked logits {vocab} {T}")
    g = gen(vocab + 1)
    low = torch.finfo(T).min
    base = logits_row(g, vocab, 6.0, T).float()
    rows = []
    for fill in (-math.inf, math.nan, low):
        r = base.clone()
        r[torch.rand(vocab, generator=g) < 0.7] = fill
        rows.append(r)
    for fill in (-math.inf, math.nan, low):
        rows.append(torch.full((vocab,), fill))
    r = torch.full((vocab,), -math.inf)
    r[vocab // 2] = low
    rows.append(r)
    r = base.clone()
    r[[3, vocab - 2]] = math.inf
    rows.append(r)
    r = torch.full((vocab,), -0.0)
    r[::2] = 0.0
    rows.append(r)
    r = torch.full((vocab,), low)
    r[vocab - 1] = torch.finfo(T).max
    rows.append(r)
    x = torch.stack(rows).to(T)
    n = len(rows)
    for filters in FILTERS:
        for temp in (0.0, 0.05, 1.0, 50.0):
            u, t, k, p, m = sample_settings(g, n, filters, vocab)
            t = torch.full((n,), temp)
            u = u * 0.98 + 0.01 if filters else u
            # sums of equal weights are exact
            check_sample(bq.sample(x.to(dev), *(on(v, dev) for v in (u, t, k, p, m))), x, u, t, k, p, m, exact=True)


def test_sample_odd_settings(bq, dev):
    """Settings that are no numbers or out of range."""
    banner("sample odd settings")
    g = gen(12)
    vocab = 3000
    x = logits_row(g, vocab, 5.0, torch.float32)
    nan, inf = math.nan, math.inf
    u = [0.0, 0.3, 1.0, 2.0, -1.0, nan, inf, -inf, 1 - 2.0 ** -24]
    t = [1.0, 0.0, -3.0, nan, inf, 1e-30, 1e-45, 3e38, 0.7]
    k = [0, -5, 1, vocab - 1, vocab, vocab + 1, 1 << 30, -(1 << 31), 2]
    p = [1.0, 0.0, -1.0, nan, 2.0, inf, 1e-30, 1 - 2.0 ** -24, 0.5]
    m = [0.0, 1.0, 2.0, nan, -1.0, inf, 1e-30, 1e-3, 0.9]
    base = [0.4, 0.9, 0, 1.0, 0.0]
    rows = []
    for i, values in enumerate((u, t, k, p, m)):
        for v in values:
            rows.append([v if i == j else b for j, b in enumerate(base)])
    cols = [torch.tensor([r[j] for r in rows], dtype=torch.int32 if j == 2 else torch.float32) for j in range(5)]
    X = x.expand(len(rows), vocab).contiguous()
    got = bq.sample(X.to(dev), *(c.to(dev) for c in cols))
    fix = [c.clone() for c in cols]
    fix[3][torch.isnan(fix[3])] = 1.0
    fix[4][torch.isnan(fix[4])] = 0.0
    check_sample(got, X, *fix, exact=True)
    assert got[0][1 + 9].item() == int(x.argmax())


def test_sample_settings_left_out(bq, dev):
    banner("sample defaults")
    g = gen(13)
    x = torch.stack([logits_row(g, 777, 5.0, torch.float16) for _ in range(6)])
    u = torch.rand(6, generator=g)
    ones, zeros = torch.ones(6).to(dev), torch.zeros(6).to(dev)
    a = bq.sample(x.to(dev), u.to(dev))
    b = bq.sample(x.to(dev), u.to(dev), ones, zeros.int(), ones, zeros)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    check_sample(a, x, u)


@pytest.mark.parametrize("vocab", [32759, 32760, 32761, 32762, 32764, 32765, 32766, 32768, 32769, 65536, 65537])
@pytest.mark.parametrize("T", TYPES + [torch.float32])
def test_sample_about_the_longest_held_row(bq, dev, T, vocab):
    banner(f"sample {vocab} {T}")
    g = gen(vocab)
    rows = 4
    room = torch.full((rows, vocab + 9), 99.0, dtype=T, device=dev)
    for i, filters in enumerate(FILTERS):
        x = torch.stack([logits_row(g, vocab, 6.0 * (i % 3), T) for i in range(rows)])
        x[1, :20], x[1, -20:] = x[1, :20] + 4, x[1, -20:] + 4  # the ends count
        args = sample_settings(g, rows, filters, vocab)
        room[:, i: i + vocab].copy_(x)
        check_sample(bq.sample(room[:, i: i + vocab], *(on(v, dev) for v in args)), x, *args)


@pytest.mark.parametrize("T", TYPES + [torch.float32])
@pytest.mark.parametrize("ws", ["auto", "none", "full"])
@pytest.mark.parametrize("rows,vocab", [(24, 40007), (3, 262147)])
def test_sample_long_rows(bq, dev, T, ws, rows, vocab):
    """Rows past a workgroup's registers: other settings in each, off ones and
    greedy ones, strides and rows off 16-byte boundaries, any workspace."""
    banner(f"sample long rows {rows} x {vocab} {T} {ws}")
    g = gen(78)
    x = torch.stack([logits_row(g, vocab, 9.0 * (i % 4) / 3, T) for i in range(rows)])
    u, t, k, p, m = sample_settings(g, rows, "kpm", vocab)
    off = torch.rand(rows, 4, generator=g) < 0.4
    t, k, p, m = t * ~off[:, 0], k * ~off[:, 1], torch.where(off[:, 2], torch.ones(rows), p), m * ~off[:, 3]
    kw = {}
    if ws == "none":
        kw["workspace"] = torch.empty(16, dtype=torch.uint8, device=dev)
    elif ws == "full":
        kw["workspace"] = torch.full((bq.sample_workspace_bytes(rows, vocab, T),), 255, dtype=torch.uint8, device=dev)
    for lead, tail in ((0, 0), (1, 2), (3, 10)):
        room = torch.full((rows, lead + vocab + tail), 99.0, dtype=T, device=dev)
        view = room[:, lead: lead + vocab]
        view.copy_(x)
        check_sample(bq.sample(view, *(on(v, dev) for v in (u, t, k, p, m)), **kw), x, u, t, k, p, m)


@pytest.mark.parametrize("T", TYPES + [torch.float32])
@pytest.mark.parametrize("vocab", [3001, 40000])
def test_sample_top_k_of_any_size(bq, dev, T, vocab):
    """Up to and past the numbers of groups, of threads and of listed tokens."""
    banner(f"sample top-k {vocab} {T}")
    g = gen(20)
    k = [v for v in (1, 2, 63, 64, 65, 255, 256, 257, 1000, 1023, 1024, 1025, 2999, 3000, 3001, 6144, 6145, 20000, 39999) if v <= vocab]
    x = torch.stack([logits_row(g, vocab, 3.0, T) for _ in k])
    for filters in ("", "p", "m"):
        u, t, _, p, m = sample_settings(g, len(k), filters, vocab)
        args = (u, t, torch.tensor(k, dtype=torch.int32), p, m)
        check_sample(bq.sample(x.to(dev), *(on(v, dev) for v in args)), x, *args)


@pytest.mark.parametrize("T", TYPES + [torch.float32])
@pytest.mark.parametrize("vocab", [30000, 50003])
def test_sample_crowded(bq, dev, T, vocab):
    """Tokens that crowd where the limit lies, in the whole row or in a run of it:
    more than are listed.  A long tail of equal weights beside one token."""
    banner(f"sample crowded {vocab} {T}")
    g = gen(21)
    rows = []
    rows.append(torch.randn(vocab, generator=g) * 0.01)
    rows.append(torch.randn(vocab, generator=g) * 2)
    rows[-1][7000:10000] = 6 + torch.rand(3000, generator=g) * 0.02
    rows.append(torch.randn(vocab, generator=g) * 2)
    rows[-1][vocab - 6200:] = 5.0
    rows.append(torch.full((vocab,), -9.0))
    rows[-1][vocab // 2] = 3.0
    rows.append(torch.rand(vocab, generator=g) * 1e-3)
    rows.append(torch.linspace(-20, 0, vocab))
    x = torch.stack(rows).to(T)
    n = len(rows)
    for filters in FILTERS:
        for _ in range(3):
            args = sample_settings(g, n, filters, vocab)
            check_sample(bq.sample(x.to(dev), *(on(v, dev) for v in args)), x, *args)


@pytest.mark.parametrize("T", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("vocab", [3000, 70001])
def test_sample_captured(bq, dev, T, vocab):
    """Two captured calls with workspaces of their own, replayed side by side with
    other logits and settings, equal the definition and the eager call."""
    banner(f"sample captured {vocab} {T}")
    g = gen(22)
    rows = 6
    sets, graphs = [], []
    for i in range(2):
        new = lambda T, *shape: torch.ones(*shape, dtype=T, device=dev)  # noqa: E731
        s = dict(x=new(T, rows, vocab), u=new(torch.float32, rows) * 0.5, t=new(torch.float32, rows), k=new(torch.int32, rows),
                 p=new(torch.float32, rows), m=new(torch.float32, rows), tokens=new(torch.int32, rows),
                 logprobs=new(torch.float32, rows),
                 ws=torch.empty(max(16, bq.sample_workspace_bytes(rows, vocab, T)), dtype=torch.uint8, device=dev))
        sets.append(s)

    def call(s):
        return bq.sample(s["x"], s["u"], s["t"], s["k"], s["p"], s["m"], s["tokens"], s["logprobs"], s["ws"])

    for s in sets:
        call(s)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call(s)
        graphs.append(graph)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for filters in ("kpm", "p", "k", "", "pm"):
        given = []
        for s in sets:
            x = torch.stack([logits_row(g, vocab, 4.0, T) for _ in range(rows)])
            u, t, k, p, m = sample_settings(g, rows, filters, vocab)
            k = torch.zeros(rows, dtype=torch.int32) if k is None else k
            p = torch.ones(rows) if p is None else p
            m = torch.zeros(rows) if m is None else m
            for name, v in zip(("x", "u", "t", "k", "p", "m"), (x, u, t, k, p, m)):
                s[name].copy_(v)
            s["tokens"].fill_(-7)
            given.append((x, u, t, k, p, m))
        torch.cuda.synchronize()
        for graph, stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                graph.replay()
        torch.cuda.synchronize()
        for s, args in zip(sets, given):
            check_sample((s["tokens"], s["logprobs"]), *args)
            first = s["tokens"].clone(), s["logprobs"].clone()
            call(s)
            torch.cuda.synchronize()
            assert torch.equal(first[0], s["tokens"]) and torch.equal(first[1], s["logprobs"])


# ---------------------------------------------------------------- attention over a tree

def run_tree(bq, dev, q, cache, tab, lens, hkv, page, mask, starts=None, maxq=None, window=0, scale=None, ws="auto", q_dev=None):
    d = q.shape[2]
    kw = {}
    if ws == "none":
        kw["workspace"] = torch.empty(16, dtype=torch.uint8, device=dev)
    elif ws == "full":
        n = bq.attn_kv4_tree_workspace_bytes(len(lens), maxq or q.shape[0] // len(lens), q.shape[1], hkv, d, tab.shape[1] * page)
        kw["workspace"] = torch.full((max(n, 16),), 255, dtype=torch.uint8, device=dev)
    out = torch.full(q.shape, 7.0, dtype=q.dtype, device=dev)
    lse = torch.full(q.shape[:2], 7.0, device=dev)
    flat = cache.flat() if isinstance(cache, layer.Cache) else cache
    bq.attn_kv4_tree(q.to(dev) if q_dev is None else q_dev, flat.to(dev), tab.to(dev), i32(lens, dev), page, hkv, mask.to(dev), scale,
                     None if starts is None else i32(starts, dev), maxq, window, out, lse, **kw)
    torch.cuda.synchronize()
    return out, lse


def check_tree(got, q, cache, tab, lens, starts, see, window=0, scale=None, what="tree"):
    out, lse = got
    T, d = q.dtype, q.shape[2]
    scale = d ** -0.5 if scale is None else scale
    want, wlse, size, delta = decode.attention_tree(q, cache, tab, lens, starts, see, scale, window)
    n = min(max(max(lens), 1), tab.shape[1] * cache.size)
    r = (2.0 ** -20 if T == torch.float16 else 2.0 ** -10 + 2.0 ** -20) + n * U
    tol = half_step(T) * want.abs() + (2 * delta[..., None] + r) * size * (1 + 2.0 ** -6) + 2.0 ** -25
    last = starts[-1]
    within(out[:last], want[:last], tol[:last], what)
    empty = torch.isinf(wlse)[:last]
    got_lse = lse.cpu().to(F64)[:last]
    assert (got_lse[empty] == -math.inf).all(), f"{what}: lse of empty rows"
    assert (out.cpu()[:last][empty] == 0).all(), f"{what}: empty rows are not zero"
    off = ((got_lse - wlse[:last]).abs() - (delta[:last] + 2.0 ** -20 * (1 + wlse[:last].abs())))[~empty]
    assert (off <= 0).all(), f"{what}: lse off by {float(off.max()):.3g} over"
    assert (out[last:] == 7.0).all() and (lse[last:] == 7.0).all(), f"{what}: rows behind the last sequence"


# lens, nodes, hq, hkv, d, page, window
TREES = [
    ([1], 1, 1, 1, 128, 16, 0),
    ([2, 17], 2, 4, 2, 64, 16, 0),
    ([8], 8, 8, 2, 128, 16, 0),           # no prefix
    ([31, 32, 33, 40, 63, 64, 65], 7, 3, 1, 128, 16, 0),
    ([700], 25, 8, 2, 128, 16, 0),
    ([129, 40, 300], 33, 16, 2, 128, 32, 0),
    ([257, 640], 31, 20, 4, 64, 64, 0),
    ([400, 128], 12, 5, 5, 256, 16, 0),
    ([1000, 65], 64, 14, 2, 128, 128, 100),
    ([511], 3, 6, 2, 256, 256, 33),
    ([90, 70, 66], 65, 2, 2, 128, 16, 0),
    ([300, 140], 130, 4, 2, 64, 32, 0),
    ([200, 190], 33, 2, 1, 128, 16, 20),  # a window inside the tree
    ([150], 64, 8, 8, 256, 16, 5),
    ([1100, 60, 1025], 9, 4, 1, 128, 64, 0),
    ([1500], 16, 3, 1, 64, 32, 0),
    ([1200, 260], 40, 8, 2, 128, 16, 700),
    ([2300, 90], 17, 8, 1, 128, 16, 0),
    ([1300], 5, 2, 1, 256, 16, 0),
    ([300], 256, 4, 2, 64, 16, 0),
    ([40], 9, 3, 1, 64, 16, 1),
]


@pytest.mark.parametrize("c", TREES)
@pytest.mark.parametrize("T", TYPES)
@pytest.mark.parametrize("ws", ["auto", "none"])
def test_attn_kv4_tree(bq, dev, c, T, ws):
    lens, nodes, hq, hkv, d, page, window = c
    banner(f"tree attention {c} {T} {ws}")
    g = gen(sum(lens) + d + hq)
    pages = sum(-(-n // page) for n in lens) + 2
    cache = make_cache(g, pages, hkv, d, page, T)
    tab = tables(g, lens, page, pages)
    for b, n in enumerate(lens):  # NaN and infinities behind the ends
        if n % page:
            raw = cache.bytes[int(tab[b, n // page])]
            for t in range(n % page, page):
                _, _, ak, av = cache._places(t)
                raw[:, ak] = torch.tensor([0, 126, 0, 124], dtype=torch.uint8)
                raw[:, av] = torch.tensor([0, 124, 0, 126], dtype=torch.uint8)
    B = len(lens)
    _, see, mask, _ = trees(g, [nodes] * B)
    q = (torch.randn(B * nodes, hq, d, generator=g) * 1.5).to(T)
    got = run_tree(bq, dev, q, cache, tab, lens, hkv, page, mask, window=window, ws=ws)
    check_tree(got, q, cache, tab, lens, [nodes * i for i in range(B + 1)], see, window, what=str(c))


@pytest.mark.parametrize("T", TYPES)
@pytest.mark.parametrize("window", [0, 6, 50])
@pytest.mark.parametrize("d,hq,hkv,nodes", [(64, 2, 1, 40), (128, 8, 1, 40), (256, 2, 2, 40), (128, 2, 2, 5)])
def test_attn_kv4_tree_any_bits(bq, dev, T, window, d, hq, hkv, nodes):
    """Masks of any bits: rows that see no node, nodes behind their own, bits
    past the last node; sequences with fewer keys than nodes, rows that see
    nothing at all."""
    banner(f"tree attention any bits {T} {window} {d} {hq} {nodes}")
    g = gen(5 + window)
    page, lens = 16, [nodes + 23, nodes, nodes - 3, 100]
    cache = make_cache(g, 20, hkv, d, page, T)
    tab = tables(g, lens, page, 20)
    bits = torch.rand(4 * nodes, 64, generator=g) < 0.4
    bits[::5] = False
    mask = decode.words_of(bits.numpy(), 2)
    see = [bits[b * nodes: (b + 1) * nodes, :nodes] for b in range(4)]
    q = torch.randn(4 * nodes, hq, d, generator=g).to(T)
    got = run_tree(bq, dev, q, cache, tab, lens, hkv, page, mask, window=window)
    check_tree(got, q, cache, tab, lens, [nodes * i for i in range(5)], see, window)


@pytest.mark.parametrize("T", TYPES)
@pytest.mark.parametrize("group", [1, 6])
def test_attn_kv4_tree_ragged(bq, dev, T, group):
    """Trees of several sizes by q_start, none among them, rows behind the last
    left as they were, strided queries; fewer words than nodes; only the first
    nodes computed."""
    banner(f"tree attention ragged {T} {group}")
    hkv, d, page = 2, 128, 16
    hq = group * hkv
    lens, nodes = [50, 9, 133, 90], [13, 0, 1, 70]
    starts = [0, 13, 13, 14, 84]
    g = gen(4)
    cache = make_cache(g, 22, hkv, d, page, T)
    tab = tables(g, lens, page, 22)
    _, see, mask, _ = trees(g, nodes)
    rows = torch.randn(90, hq + 4, d, generator=g).to(T)
    x = rows.to(dev)
    padded = torch.cat([mask, torch.full((6, mask.shape[1]), -1, dtype=torch.int32)])
    got = run_tree(bq, dev, rows[:, :hq], cache, tab, lens, hkv, page, padded, starts, 70, q_dev=x[:, :hq])
    check_tree(got, rows[:, :hq], cache, tab, lens, starts, see, what="ragged")
    # the first word alone: no row sees a node past 31
    got = run_tree(bq, dev, rows[:, :hq], cache, tab, lens, hkv, page, padded[:, :1].contiguous(), starts, 70, q_dev=x[:, :hq])
    cut = [s.clone() for s in see]
    for s in cut:
        s[:, 32:] = False
    check_tree(got, rows[:, :hq], cache, tab, lens, starts, cut, what="one word")
    # max_q_len 20: the others' rows stay as they were, and nothing else changes
    some = run_tree(bq, dev, rows[:, :hq], cache, tab, lens, hkv, page, padded, starts, 20, q_dev=x[:, :hq])
    full = run_tree(bq, dev, rows[:, :hq], cache, tab, lens, hkv, page, padded, starts, 70, q_dev=x[:, :hq])
    assert torch.equal(some[0][34:], torch.full_like(some[0][34:], 7.0))
    want = decode.attention_tree(rows[:, :hq], cache, tab, lens, starts, see, d ** -0.5)[0]
    assert ((some[0][:34].cpu().to(F64) - want[:34]).abs() <= 0.02).all() and ((full[0][:34] - some[0][:34]).abs() <= 0.02).all()
    # starts outside the queries
    a = run_tree(bq, dev, rows[:84, :hq], cache, tab, lens, hkv, page, mask, [-9, 13, 13, 14, 1 << 30], 70)
    b = run_tree(bq, dev, rows[:84, :hq], cache, tab, lens, hkv, page, mask, starts, 70)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("T", TYPES)
def test_attn_kv4_tree_bad_pages_and_lengths(bq, dev, T):
    banner(f"tree attention bad pages {T}")
    hq, hkv, d, page, nodes = 4, 2, 128, 16, 6
    g = gen(8)
    cache = make_cache(g, 8, hkv, d, page, T)
    tab = torch.tensor([[0, -1, 2, 8], [3, 1 << 30, -(1 << 31), 4], [-1, -1, -1, -1], [5, 6, 7, 1]], dtype=torch.int32)
    _, see, mask, _ = trees(g, [nodes] * 4)
    q = torch.randn(4 * nodes, hq, d, generator=g).to(T)
    starts = [nodes * i for i in range(5)]
    for lens in ([60, 64, 64, 64], [60, -7, 1 << 30, 1 << 20], [3, 0, 1, 6]):
        got = run_tree(bq, dev, q, cache, tab, lens, hkv, page, mask)
        check_tree(got, q, cache, tab, lens, starts, see, what=str(lens))


@pytest.mark.parametrize("T", TYPES)
@pytest.mark.parametrize("k_off,v_mul,q_mul", [(0.0, 1e-4, 1.0), (4.0, 300.0, 3.0), (0.0, 4000.0, 0.01), (1.0, 1.0, 30.0)])
@pytest.mark.parametrize("nodes", [3, 33])
def test_attn_kv4_tree_ranges(bq, dev, T, k_off, v_mul, q_mul, nodes):
    """Small and large values, keys with a large common offset, peaked softmax."""
    banner(f"tree attention ranges {k_off} {v_mul} {q_mul} {nodes} {T}")
    lens, hq, hkv, d, page = [333, 1064], 8, 2, 128, 16
    g = gen(9)
    cache = make_cache(g, 90, hkv, d, page, T, k_off, v_mul)
    tab = tables(g, lens, page, 90)
    _, see, mask, _ = trees(g, [nodes] * 2)
    q = (torch.randn(2 * nodes, hq, d, generator=g) * q_mul).to(T)
    got = run_tree(bq, dev, q, cache, tab, lens, hkv, page, mask)
    check_tree(got, q, cache, tab, lens, [0, nodes, 2 * nodes], see, what="ranges")


def test_attn_kv4_tree_growing_scales(bq, dev):
    """V scales that grow along the sequence, by 2^16 over it, and of either sign."""
    banner("tree attention growing V scales")
    T, lens, hq, hkv, d, page, nodes = torch.float16, [1090], 16, 1, 128, 16, 10
    g = gen(10)
    cache = layer.Cache(72, hkv, d, page)
    for s in range(1152):
        cache.write(s, torch.randn(hkv, d, generator=g).to(T), (torch.randn(hkv, d, generator=g) * 2.0 ** (s / 72 - 6)).to(T))
    for s in range(0, 1152, 3):
        _, _, _, av = cache._places(s % page)
        raw = cache.bytes[s // page, :, av]
        raw[:, 1] ^= 128  # the scale's sign
        cache.bytes[s // page, :, av] = raw
    tab = torch.arange(72, dtype=torch.int32)[None]
    _, see, mask, _ = trees(g, [nodes])
    q = torch.randn(nodes, hq, d, generator=g).to(T)
    for ws in ("none", "full"):
        out, lse = run_tree(bq, dev, q, cache, tab, lens, hkv, page, mask, ws=ws)
        want, wlse, _, delta = decode.attention_tree(q, cache, tab, lens, [0, nodes], see, d ** -0.5)
        # the values' magnitudes by their scales' own
        rows = [cache.read(t) for t in range(lens[0])]
        mag = torch.stack([(r[1][0] * r[1][1].abs() + r[1][2].abs())[0] for r in rows]).amax(0)
        tol = half_step(T) * want.abs() + (2 * delta[..., None] + 2.0 ** -20 + 1090 * U) * mag + 2.0 ** -25
        within(out, want, tol, "growing")


@pytest.mark.parametrize("scale", [0.0, -0.1, 1.0])
@pytest.mark.parametrize("T", TYPES)
@pytest.mark.parametrize("nodes", [4, 20])
def test_attn_kv4_tree_scales(bq, dev, T, scale, nodes):
    banner(f"tree attention scale {scale} {nodes} {T}")
    lens, hq, hkv, d, page = [77, 300], 4, 1, 64, 16
    g = gen(14)
    cache = make_cache(g, 26, hkv, d, page, T)
    tab = tables(g, lens, page, 26)
    _, see, mask, _ = trees(g, [nodes] * 2)
    q = torch.randn(2 * nodes, hq, d, generator=g).to(T)
    got = run_tree(bq, dev, q, cache, tab, lens, hkv, page, mask, scale=scale)
    check_tree(got, q, cache, tab, lens, [0, nodes, 2 * nodes], see, scale=scale, what="scale")


@pytest.mark.parametrize("T", TYPES)
@pytest.mark.parametrize("hq,d,nodes", [(2, 64, 8), (8, 128, 8), (64, 64, 8), (2, 256, 8), (4, 128, 60)])
def test_attn_kv4_tree_masked_places_may_be_anything(bq, dev, T, hq, d, nodes):
    """NaN and infinite parameters of a node that a row does not see change no
    bit of it; a row that sees one gets NaN."""
    banner(f"tree attention masked places {hq} {d} {nodes} {T}")
    n, hkv, page = 150, 1, 16
    g = gen(15)
    cache = make_cache(g, 10, hkv, d, page, T)
    tab = torch.arange(10, dtype=torch.int32)[None]
    _, see, mask, _ = trees(g, [nodes])
    bad_node = nodes // 3
    q = torch.randn(nodes, hq, d, generator=g).to(T)
    want = run_tree(bq, dev, q, cache, tab, [n], hkv, page, mask)
    check_tree(want, q, cache, tab, [n], [0, nodes], see, what="clean")
    t = n - nodes + bad_node
    _, _, ak, av = cache._places(t % page)
    cache.bytes[t // page][:, ak] = torch.tensor([0, 126, 0, 124], dtype=torch.uint8)  # NaN, inf
    cache.bytes[t // page][:, av] = torch.tensor([0, 126, 0, 124], dtype=torch.uint8)
    out, lse = run_tree(bq, dev, q, cache, tab, [n], hkv, page, mask)
    sees = see[0][:, bad_node]
    assert torch.equal(out.cpu()[~sees], want[0].cpu()[~sees]) and torch.equal(lse.cpu()[~sees], want[1].cpu()[~sees])
    assert torch.isnan(out.cpu()[sees]).all()


@pytest.mark.parametrize("T", TYPES)
@pytest.mark.parametrize("batch,top,hq,hkv,d,nodes,window", [(40, 333, 16, 8, 64, 5, 0), (33, 290, 8, 8, 128, 20, 50),
                                                             (9, 2400, 16, 4, 128, 12, 0), (65, 150, 40, 5, 64, 3, 0)])
def test_attn_kv4_tree_many_workgroups(bq, dev, T, batch, top, hq, hkv, d, nodes, window):
    banner(f"tree attention many workgroups {batch} {top} {hq} {hkv} {d} {nodes} {window} {T}")
    g = gen(batch + top)
    page = 16
    lens = [nodes + (37 * i + 1) % (top // 4) for i in range(batch - 1)] + [top]
    pages = sum(-(-n // page) for n in lens) + 2
    cache = make_cache(g, pages, hkv, d, page, T)
    tab = tables(g, lens, page, pages)
    _, see, mask, _ = trees(g, [nodes] * batch)
    q = (torch.randn(batch * nodes, hq, d, generator=g) * 1.5).to(T)
    got = run_tree(bq, dev, q, cache, tab, lens, hkv, page, mask, window=window)
    check_tree(got, q, cache, tab, lens, [nodes * i for i in range(batch + 1)], see, window, what="many workgroups")


@pytest.mark.parametrize("T", TYPES)
@pytest.mark.parametrize("d,hq,hkv,nodes", [(64, 4, 2, 21), (128, 8, 2, 50), (256, 3, 1, 12), (128, 2, 2, 5)])
@pytest.mark.parametrize("window", [0, 70])
def test_a_chain_is_attn_kv4(bq, dev, T, d, hq, hkv, nodes, window):
    """A chain's nodes see what attn_kv4's queries see: both within the bound
    of the same formula."""
    banner(f"tree attention: a chain {d} {hq} {nodes} {window} {T}")
    g = gen(21)
    lens, page = [400, nodes + 3], 32
    cache = make_cache(g, 20, hkv, d, page, T)
    tab = tables(g, lens, page, 20)
    see, _ = decode.ancestors(list(range(-1, nodes - 1)))
    mask = decode.words_of(np.concatenate([see, see]), 2)
    q = torch.randn(2 * nodes, hq, d, generator=g).to(T)
    got = run_tree(bq, dev, q, cache, tab, lens, hkv, page, mask, window=window)
    check_tree(got, q, cache, tab, lens, [0, nodes, 2 * nodes], [torch.from_numpy(see)] * 2, window)
    o, lse = bq.attn_kv4(q.to(dev), cache.flat().to(dev), tab.to(dev), i32(lens, dev), page, hkv, window=window, return_lse=True)
    assert ((o.float() - got[0].float()).abs() <= 2 * half_step(T) * o.float().abs() + 2.0 ** -6 * half_step(T) * 300).all()


def test_attn_kv4_tree_large_cache_offsets(bq, dev):
    """A page more than 2^32 bytes into the cache; the move there too."""
    banner("tree attention offsets past 32 bits")
    T, hq, hkv, d, page, nodes = torch.float16, 16, 2, 128, 16, 9
    g = gen(12)
    small = make_cache(g, 3, hkv, d, page, T)
    n = (1 << 32) // small.flat().shape[1] + 5
    cache = torch.zeros(n, small.flat().shape[1], dtype=torch.uint8, device=dev)
    ids = [n - 1, 7, n - 3]
    at = torch.tensor(ids, device=dev)
    cache[at] = small.flat().to(dev)
    _, _, mask, _ = trees(g, [nodes])
    q = torch.randn(nodes, hq, d, generator=g).to(T).to(dev)
    lens = i32([45], dev)
    far, near = i32([ids], dev), i32([[0, 1, 2]], dev)
    tiny = small.flat().to(dev)
    a = bq.attn_kv4_tree(q, cache, far, lens, page, hkv, mask.to(dev))
    b = bq.attn_kv4_tree(q, tiny, near, lens, page, hkv, mask.to(dev))
    path, count = i32([[0, 4, 7]], dev), i32([3], dev)
    bq.kv4_compact(cache, far, lens, path, count, page, hkv, d, max_q_len=nodes)
    bq.kv4_compact(tiny, near, lens, path, count, page, hkv, d, max_q_len=nodes)
    torch.cuda.synchronize()
    assert torch.equal(a, b) and torch.equal(cache[at], tiny)
    assert not torch.equal(tiny.cpu(), small.flat())


# ---------------------------------------------------------------- together

def _state(bq, dev, T, B=6, nodes=20, seed=50):
    """A step of decoding with drafted trees: everything but what the calls compute."""
    g = gen(seed)
    hq, hkv, d, page, hidden, vocab, layers = 8, 2, 128, 16, 512, 1200, 2
    lens = [nodes + 3 + 47 * i for i in range(B)]
    pages = sum(-(-n // page) for n in lens)
    tab = tables(g, lens, page, pages)
    dv = lambda t: t.to(dev)  # noqa: E731
    o = dict(hq=hq, hkv=hkv, d=d, page=page, B=B, nodes=nodes, layers=layers, lens_list=lens, tab=tab)
    o["x"] = dv(torch.randn(B * nodes, hidden, generator=g).to(T))
    n = (hq + 2 * hkv) * d
    for name, shape in (("qkv", (n, hidden)), ("o", (hidden, hq * d)), ("head", (vocab, hidden))):
        B4, s, _ = layer.quantize_w4g(torch.randn(*shape, generator=g) * 0.04, 64, False)
        o["w" + name], o["s" + name] = dv(B4), dv(s)
    o["cos"], o["sin"] = (dv(t) for t in table(2048, d))
    o["wq"], o["wk"] = (dv((1 + 0.1 * torch.randn(d, generator=g)).to(T)) for _ in range(2))
    o["lens"], o["table"] = i32(lens, dev), dv(tab)
    parents, o["see"], _, _ = trees(g, [nodes] * B)
    o["parents"] = dv(parents.view(B, nodes))
    o["tokens"] = dv(torch.randint(0, 3, (B, nodes), generator=g, dtype=torch.int32))
    keys = [(b, t) for b, m in enumerate(lens) for t in range(m - nodes, m)]
    o["slots"] = dv(torch.tensor([int(tab[b, t // page]) * page + t % page for b, t in keys]))
    o["cache"] = torch.zeros(layers, pages, bq.kv4_page_bytes(hkv, d, page), dtype=torch.uint8, device=dev)
    for i in range(layers):
        k, v = (torch.randn(pages * page, hkv, d, generator=g).to(T) for _ in range(2))
        bq.qk_norm_rope_kv4(None, dv(k), dv(v), None, None, None, o["cache"][i], torch.arange(pages * page, device=dev), page)
    o["u"] = dv(torch.rand(B * nodes, generator=g))
    o["t"], o["p"] = dv(0.5 + torch.rand(B * nodes, generator=g)), dv(0.5 + 0.5 * torch.rand(B * nodes, generator=g))
    o["k"] = dv(torch.randint(1, 50, (B * nodes,), generator=g, dtype=torch.int32))
    N = B * nodes
    o["mask"], o["pos"] = torch.empty(N, 1, dtype=torch.int32, device=dev), torch.empty(N, dtype=torch.int32, device=dev)
    for name, shape, dt in (("qkv", (N, n), T), ("q", (N, hq, d), T), ("o", (N, hq, d), T), ("y", (N, hidden), T),
                            ("logits", (N, vocab), T), ("drawn", (N,), torch.int32), ("logp", (N,), torch.float32),
                            ("path", (B, 8), torch.int32), ("count", (B,), torch.int32), ("next", (B,), torch.int32)):
        o[name] = torch.empty(shape, dtype=dt, device=dev)
    w1 = max([16] + [bq.gemm_w4g_workspace_bytes(N, a, b) for a, b in ((n, hidden), (hidden, hq * d), (vocab, hidden))])
    w2 = max(bq.attn_kv4_tree_workspace_bytes(B, nodes, hq, hkv, d, tab.shape[1] * page), 16)
    w3 = max(bq.sample_workspace_bytes(N, vocab, T), 16)
    o["ws1"], o["ws2"], o["ws3"] = (torch.empty(w, dtype=torch.uint8, device=dev) for w in (w1, w2, w3))
    return o


OUTS = ("mask", "pos", "qkv", "q", "o", "y", "logits", "drawn", "logp", "path", "count", "next", "cache")


def _step(bq, o):
    """Masks, one layer (its cache: the first), logits, sampling, the walk, the move in all layers."""
    N, hq, hkv, page = o["x"].shape[0], o["hq"], o["hkv"], o["page"]
    bq.tree_mask(o["parents"], o["lens"], mask=o["mask"], positions=o["pos"])
    qkv = bq.gemm_w4g_a16(o["x"], o["wqkv"], o["sqkv"], out=o["qkv"], workspace=o["ws1"])
    r = qkv.view(N, hq + 2 * hkv, o["d"])
    q = bq.qk_norm_rope_kv4(r[:, :hq], r[:, hq: hq + hkv], r[:, hq + hkv:], o["cos"], o["sin"], o["pos"], o["cache"][0], o["slots"],
                            page, o["wq"], o["wk"], q_out=o["q"])
    bq.attn_kv4_tree(q, o["cache"][0], o["table"], o["lens"], page, hkv, o["mask"], out=o["o"], workspace=o["ws2"])
    bq.gemm_w4g_a16(o["o"].view(N, -1), o["wo"], o["so"], out=o["y"], workspace=o["ws1"])
    bq.gemm_w4g_a16(o["y"], o["whead"], o["shead"], out=o["logits"], workspace=o["ws1"])
    bq.sample(o["logits"], o["u"], o["t"], o["k"], o["p"], tokens=o["drawn"], logprobs=o["logp"], workspace=o["ws3"])
    o["drawn"].remainder_(3)  # a model that agrees with the draft now and then
    bq.tree_accept(o["tokens"], o["parents"], o["drawn"], path=o["path"], count=o["count"], next_token=o["next"])
    bq.kv4_compact(o["cache"], o["table"], o["lens"], o["path"], o["count"], page, hkv, o["d"], max_q_len=o["nodes"])


@pytest.mark.parametrize("T", TYPES)
def test_step_together(bq, dev, T):
    """The operators one after another, each checked on the inputs it was
    given; then attn_kv4 over the moved cache."""
    banner(f"tree step {T}")
    o = _state(bq, dev, T)
    before = o["cache"].clone()
    _step(bq, o)
    torch.cuda.synchronize()
    B, nodes, hq, hkv, d, page, lens, tab = (o[k] for k in ("B", "nodes", "hq", "hkv", "d", "page", "lens_list", "tab"))
    starts = [nodes * i for i in range(B + 1)]
    want_mask = torch.cat([decode.words_of(s.numpy(), 1) for s in o["see"]])
    assert torch.equal(o["mask"].cpu(), want_mask)
    # layer 0's cache with the nodes written, before the move
    ref = layer.Cache(before.shape[1], hkv, d, page)
    ref.bytes = before[0].cpu().view(ref.bytes.shape).clone()
    r = o["qkv"].cpu().view(B * nodes, hq + 2 * hkv, d)
    k = layer.round_to(layer.norm_rope(r[:, hq: hq + hkv], o["wk"].cpu(), 1e-6, o["cos"].cpu(), o["sin"].cpu(), o["pos"].cpu(),
                                       False)[0], T)
    for i in range(B * nodes):
        ref.write(o["slots"][i], k[i], r[i, hq + hkv:])
    lse = torch.zeros(B * nodes, hq, device=dev)
    check = decode.attention_tree(o["q"].cpu(), ref, tab, lens, starts, o["see"], d ** -0.5)
    rr = (2.0 ** -20 if T == torch.float16 else 2.0 ** -10 + 2.0 ** -20) + 400 * U
    within(o["o"], check[0], half_step(T) * check[0].abs() + (2 * check[3][..., None] + rr) * check[2] * 1.02 + 2.0 ** -25, "step: attention")
    want, lp, margin = sample_wants(o["logits"].cpu(), o["u"].cpu(), o["t"].cpu(), o["k"].cpu(), o["p"].cpu())
    clear = margin > border(1200)
    assert clear.mean() > 0.9 and (o["drawn"].cpu().numpy() == want % 3)[clear].all()
    drawn = o["drawn"].cpu().view(B, nodes).tolist()
    caches = [ref, layer.Cache(before.shape[1], hkv, d, page)]
    caches[1].bytes = before[1].cpu().view(ref.bytes.shape).clone()
    moved = 0
    for b in range(B):
        path, last = decode.accept(o["tokens"][b].tolist(), o["parents"][b].tolist(), drawn[b], 8)
        assert o["path"][b].tolist() == path + [-1] * (8 - len(path)) and int(o["next"][b]) == last
        moved += sum(j != p for j, p in enumerate(path))
        for c in caches:
            decode.compact(c, tab[b], lens[b], nodes, path)
    assert moved > 0, "no path that moves anything"
    for i, c in enumerate(caches):
        assert torch.equal(o["cache"][i].cpu(), c.flat()), f"layer {i}"
    # the next step's plain attention over what was accepted
    after = [n - nodes + int(c) for n, c in zip(lens, o["count"])]
    q = torch.randn(B, hq, d, generator=gen(1)).to(T)
    got = bq.attn_kv4(q.to(dev), o["cache"][0], o["table"], i32(after, dev), page, hkv)
    w, _, size, delta = layer.attention(q, caches[0], tab, after, list(range(B + 1)), d ** -0.5)
    within(got, w, half_step(T) * w.abs() + (2 * delta[..., None] + rr) * size * 1.02 + 2.0 ** -25, "step: next attention")
    del lse


@pytest.mark.parametrize("T", TYPES)
def test_step_captured(bq, dev, T):
    """The step in a graph: every replay equals the eager results, with eager
    work between replays, on trees and lengths changed in place."""
    banner(f"tree step in a graph {T}")
    o = _state(bq, dev, T)
    start = o["cache"].clone()

    def eager():
        o["cache"].copy_(start)
        _step(bq, o)
        torch.cuda.synchronize()
        return {k: o[k].clone() for k in OUTS}

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        _step(bq, o)
    torch.cuda.current_stream().wait_stream(s)
    first = eager()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        _step(bq, o)
    for rep in range(4):
        if rep == 2:  # other trees, settings and lengths through the same graph
            p = _state(bq, dev, T, seed=51)
            for k in ("parents", "tokens", "u", "k"):
                o[k].copy_(p[k])
            o["lens"].sub_(2)
            first = eager()
        for k in OUTS[:-1]:
            o[k].fill_(3)
        for k in ("ws1", "ws2", "ws3"):
            o[k].fill_(255)
        o["cache"].copy_(start)
        _ = (o["cos"] * 2).sum()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for k in OUTS:
            assert torch.equal(o[k], first[k]), f"replay {rep}: {k}"


def test_step_on_other_streams(bq, dev):
    """Two streams at once, each with its own state, behind work of their own."""
    banner("tree steps on two streams")
    wants = []
    for T in TYPES:
        o = _state(bq, dev, T)
        _step(bq, o)
        torch.cuda.synchronize()
        wants.append({k: o[k].clone() for k in OUTS})
    states = [_state(bq, dev, T) for T in TYPES]
    keep = [(o["x"].clone(), o["cache"].clone()) for o in states]
    for o in states:
        o["x"].zero_()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in states]
    for _ in range(3):
        for o, s, (x, c) in zip(states, streams, keep):
            with torch.cuda.stream(s):
                torch.cuda._sleep(1_000_000)
                o["x"].copy_(x)
                o["cache"].copy_(c)
                _step(bq, o)
    torch.cuda.synchronize()
    for o, w in zip(states, wants):
        for k in OUTS:
            assert torch.equal(o[k], w[k]), k


# ---------------------------------------------- trees by way of shared operands

def wide_run(bq, dev, q, cache, tab, lens, hkv, page, mask, *a, **kw):
    """run_tree with a table so wide that rows times keys take the kernel whose
    rows share decoded codes; no entry of the added ones is read."""
    maxq = kw.get("maxq") or (a[1] if len(a) > 1 and a[1] else q.shape[0] // len(lens))
    per = len(lens) * hkv * max(maxq * (q.shape[1] // hkv), 1)
    blocks = -(-(1 << 26) // (per * page))
    more = torch.full((tab.shape[0], max(blocks - tab.shape[1], 1)), 1 << 30, dtype=torch.int32)
    return run_tree(bq, dev, q, cache, torch.cat([tab, more], 1), lens, hkv, page, mask, *a, **kw)


SHARED = [
    ([1], 70, 1, 1, 128, 16, 0),
    ([700], 25, 16, 2, 128, 16, 0),
    ([31, 32, 33, 40, 63, 64, 65, 127, 128, 129], 30, 3, 1, 128, 16, 0),
    ([129, 40, 300], 33, 16, 2, 128, 32, 0),      # three tiles of 128 rows
    ([257, 640], 31, 20, 4, 64, 64, 0),
    ([1000, 65], 64, 14, 2, 128, 128, 100),
    ([90, 70, 66], 65, 4, 2, 128, 16, 0),
    ([300, 140], 130, 4, 2, 64, 32, 0),
    ([200, 190], 33, 6, 2, 128, 16, 20),          # a window inside the tree
    ([5000, 3, 64, 2999], 24, 4, 1, 64, 16, 0),
    ([4000, 90], 17, 8, 1, 128, 16, 1500),
    ([300], 1000, 2, 2, 64, 16, 0),               # fewer keys than nodes
    ([700, 130], 1024, 1, 1, 128, 256, 0),
    ([40, 45], 70, 1, 1, 64, 16, 1),
    ([190], 19, 64, 1, 128, 64, 0),               # 1216 rows: a tile that is not full
]


@pytest.mark.parametrize("c", SHARED)
@pytest.mark.parametrize("T", TYPES)
@pytest.mark.parametrize("ws", ["auto", "none", "full"])
def test_attn_kv4_tree_shared(bq, dev, monkeypatch, c, T, ws):
    shared(monkeypatch)
    test_attn_kv4_tree(bq, dev, c, T, ws)


def shared(monkeypatch):
    narrow = run_tree

    def run(*a, **kw):
        with monkeypatch.context() as m:
            m.setitem(globals(), "run_tree", narrow)
            return wide_run(*a, **kw)

    monkeypatch.setitem(globals(), "run_tree", run)


@pytest.mark.parametrize("T", TYPES)
@pytest.mark.parametrize("window", [0, 6, 50])
@pytest.mark.parametrize("d,hq,hkv,nodes", [(64, 4, 1, 40), (128, 8, 1, 40), (128, 4, 2, 36), (64, 6, 2, 30)])
def test_attn_kv4_tree_shared_any_bits(bq, dev, monkeypatch, T, window, d, hq, hkv, nodes):
    shared(monkeypatch)
    test_attn_kv4_tree_any_bits(bq, dev, T, window, d, hq, hkv, nodes)


@pytest.mark.parametrize("T", TYPES)
@pytest.mark.parametrize("group", [1, 6])
def test_attn_kv4_tree_shared_ragged(bq, dev, monkeypatch, T, group):
    shared(monkeypatch)
    test_attn_kv4_tree_ragged(bq, dev, T, group)


@pytest.mark.parametrize("T", TYPES)
@pytest.mark.parametrize("k_off,v_mul,q_mul", [(0.0, 1e-4, 1.0), (4.0, 300.0, 3.0), (0.0, 4000.0, 0.01), (1.0, 1.0, 30.0)])
def test_attn_kv4_tree_shared_ranges(bq, dev, monkeypatch, T, k_off, v_mul, q_mul):
    shared(monkeypatch)
    test_attn_kv4_tree_ranges(bq, dev, T, k_off, v_mul, q_mul, 33)


def test_attn_kv4_tree_shared_growing_scales(bq, dev, monkeypatch):
    shared(monkeypatch)
    test_attn_kv4_tree_growing_scales(bq, dev)


@pytest.mark.parametrize("scale", [0.0, -0.1, 1.0])
@pytest.mark.parametrize("T", TYPES)
def test_attn_kv4_tree_shared_scales(bq, dev, monkeypatch, T, scale):
    shared(monkeypatch)
    test_attn_kv4_tree_scales(bq, dev, T, scale, 20)


@pytest.mark.parametrize("T", TYPES)
@pytest.mark.parametrize("hq,d,nodes", [(64, 64, 8), (16, 128, 8), (4, 128, 60), (2, 64, 64)])
def test_attn_kv4_tree_shared_masked_places_may_be_anything(bq, dev, monkeypatch, T, hq, d, nodes):
    shared(monkeypatch)
    test_attn_kv4_tree_masked_places_may_be_anything(bq, dev, T, hq, d, nodes)


@pytest.mark.parametrize("T", TYPES)
@pytest.mark.parametrize("batch,top,hq,hkv,d,nodes,window", [(40, 333, 16, 1, 64, 5, 0), (130, 290, 4, 1, 128, 20, 50),
                                                             (9, 2400, 16, 2, 128, 12, 0), (65, 150, 40, 5, 64, 9, 0),
                                                             (300, 90, 24, 1, 64, 3, 0), (3, 20000, 4, 1, 64, 17, 0)])
def test_attn_kv4_tree_shared_many_workgroups(bq, dev, monkeypatch, T, batch, top, hq, hkv, d, nodes, window):
    shared(monkeypatch)
    test_attn_kv4_tree_many_workgroups(bq, dev, T, batch, top, hq, hkv, d, nodes, window)


@pytest.mark.parametrize("T", TYPES)
@pytest.mark.parametrize("d", [64, 128])
def test_attn_kv4_tree_shared_bad_pages_and_lengths(bq, dev, T, d):
    """Pages that are none, lengths below zero and past the table, in a table of
    its full width."""
    banner(f"tree attention shared bad pages {d} {T}")
    hq, hkv, page, nodes, B, wide = 32, 1, 16, 6, 3, 128
    g = gen(18)
    cache = make_cache(g, 40, hkv, d, page, T)
    tab = torch.randint(-3, 44, (B, wide), generator=g, dtype=torch.int32)
    tab[0, :9] = torch.arange(9)
    tab[1, 3], tab[1, 4] = 1 << 30, -(1 << 31)
    # 64 sequences more without queries make the rows times keys
    more = 200
    tab = torch.cat([tab, torch.full((more, wide), 77, dtype=torch.int32)])
    _, see, mask, _ = trees(g, [nodes] * B)
    q = torch.randn(B * nodes, hq, d, generator=g).to(T)
    starts = [min(nodes * i, B * nodes) for i in range(B + more + 1)]
    see = see + [torch.zeros(0, 0, dtype=torch.bool)] * more
    for lens in ([140, 1 << 30, 2048], [-7, 60, 1 << 20], [3, 0, 1]):
        lens = lens + [100] * more
        got = run_tree(bq, dev, q, cache, tab, lens, hkv, page, mask, starts, nodes)
        check_tree(got, q, cache, tab, [min(n, wide * page) for n in lens], starts, see, what=str(lens[:3]))


def test_attn_kv4_tree_shared_captured(bq, dev):
    """A captured call replayed with other lengths, queries and masks, beside a
    second one with a workspace of its own."""
    banner("tree attention shared captured")
    T, B, nodes, hq, hkv, d, page, wide = torch.bfloat16, 3, 40, 4, 1, 64, 16, 16384
    g = gen(19)
    cache = make_cache(g, 130, hkv, d, page, T)
    tab = torch.full((B, wide), -1, dtype=torch.int32)
    for b in range(B):
        tab[b, :42] = torch.arange(42) + 42 * b
    tab_d, cache_d = tab.to(dev), cache.flat().to(dev)
    sets = []
    for k in range(2):
        need = bq.attn_kv4_tree_workspace_bytes(B, nodes, hq, hkv, d, wide * page)
        assert need > 0
        sets.append(dict(q=torch.zeros(B * nodes, hq, d, dtype=T, device=dev), lens=i32([0] * B, dev),
                         mask=torch.zeros(B * nodes, 2, dtype=torch.int32, device=dev), out=torch.zeros(B * nodes, hq, d, dtype=T, device=dev),
                         lse=torch.zeros(B * nodes, hq, device=dev), ws=torch.empty(need, dtype=torch.uint8, device=dev)))

    def call(s):
        bq.attn_kv4_tree(s["q"], cache_d, tab_d, s["lens"], page, hkv, s["mask"], d ** -0.5, None, None, 0, s["out"], s["lse"],
                         workspace=s["ws"])

    graphs = []
    for s in sets:
        call(s)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call(s)
        graphs.append(graph)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for i, lens in enumerate([[600, 50, 41], [40, 640, 300], [0, 0, 670], [100, 100, 100]]):
        given = []
        for k, s in enumerate(sets):
            mine = lens[k:] + lens[:k]
            _, see, mask, _ = trees(g, [nodes] * B)
            q = torch.randn(B * nodes, hq, d, generator=g).to(T)
            s["q"].copy_(q)
            s["lens"].copy_(i32(mine, dev))
            s["mask"].copy_(mask)
            s["out"].fill_(7)
            given.append((q, mine, see))
        torch.cuda.synchronize()
        for graph, stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                graph.replay()
        torch.cuda.synchronize()
        for s, (q, mine, see) in zip(sets, given):
            check_tree((s["out"], s["lse"]), q, cache, tab, mine, [nodes * j for j in range(B + 1)], see, what=f"replay {i}")
            eager = [x.clone() for x in (s["out"], s["lse"])]
            call(s)
            torch.cuda.synchronize()
            assert torch.equal(eager[0], s["out"]) and torch.equal(eager[1], s["lse"])


# ---------------------------------------------------------------- past 32 bits

@pytest.mark.parametrize("T", TYPES)
@pytest.mark.parametrize("wide", [False, True])
def test_attn_kv4_tree_past_32_bits(bq, dev, T, wide):
    """Pages that lie past 4 GiB of the cache."""
    banner(f"tree attention past 32 bits {wide} {T}")
    hq, hkv, d, page, nodes, lens = 64, 8, 128, 16, 20, [333, 90]
    g = gen(31)
    cache = make_cache(g, 30, hkv, d, page, T)
    flat = cache.flat()
    off = (1 << 32) // flat.shape[1] + 1
    big = torch.zeros(off + 30, flat.shape[1], dtype=torch.uint8, device=dev)
    big[off:] = flat.to(dev)
    tab = tables(g, lens, page, 30)
    _, see, mask, _ = trees(g, [nodes] * 2)
    q = torch.randn(2 * nodes, hq, d, generator=g).to(T)
    got = (wide_run if wide else run_tree)(bq, dev, q, big, tab + off, lens, hkv, page, mask)
    check_tree(got, q, cache, tab, lens, [0, nodes, 2 * nodes], see, what="past 32 bits")


def test_kv4_compact_past_32_bits(bq, dev):
    """Pages past 4 GiB of a layer, layers further than that apart."""
    banner("compact past 32 bits")
    hkv, d, page, nodes, lens = 8, 64, 16, 12, [50, 31]
    g = gen(32)
    layers = [make_cache(g, 9, hkv, d, page, torch.float16) for _ in range(2)]
    size = layers[0].flat().shape[1]
    off = (1 << 32) // size + 1
    big = torch.zeros(2, off + 9, size, dtype=torch.uint8, device=dev)
    for i, c in enumerate(layers):
        big[i, off:] = c.flat().to(dev)
    tab = tables(g, lens, page, 9)
    path, count = [[0, 2, 5, 11, -1], [0, 1, 7, -1, -1]], [4, 3]
    bq.kv4_compact(big, (tab + off).to(dev), i32(lens, dev), i32(path, dev), i32(count, dev), page, hkv, d, max_q_len=nodes)
    for i, c in enumerate(layers):
        for b, n in enumerate(lens):
            decode.compact(c, tab[b], n, nodes, path[b][: count[b]])
        assert torch.equal(big[i, off:].cpu(), c.flat())
        assert not big[i, :off].any()


@pytest.mark.parametrize("vocab", [1000, 40001])
def test_sample_past_32_bits(bq, dev, vocab):
    """Rows that lie past 4 GiB of the logits."""
    banner(f"sample past 32 bits {vocab}")
    g = gen(33)
    rows, stride = 3, (1 << 31) + 1
    x = torch.stack([logits_row(g, vocab, 4.0, torch.bfloat16) for _ in range(rows)])
    room = torch.empty(stride * (rows - 1) + vocab, dtype=torch.bfloat16, device=dev)
    view = room.as_strided((rows, vocab), (stride, 1))
    view.copy_(x)
    for filters in ("", "p", "kpm"):
        args = sample_settings(g, rows, filters, vocab)
        check_sample(bq.sample(view, *(on(v, dev) for v in args)), x, *args)
