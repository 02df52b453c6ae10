"""The cache's move along paths longer than a wavefront, and attention over a
tree called again on the same inputs."""
import numpy as np
import pytest
import torch

from decode_cases import gen, trees
from gpu_util import banner, need_gpu
from oracle import decode, layer
from test_gpu_decode import TYPES, i32
from test_gpu_layer import half_step, make_cache, tables, within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    return need_gpu()


@pytest.fixture(scope="module")
def bq(dev):
    from bit_mixed_precision_amd import bq as _bq

    return _bq


@pytest.mark.parametrize("hkv,d,page", [(2, 64, 16), (1, 128, 32), (3, 256, 16)])
def test_kv4_compact_long_paths(bq, dev, hkv, d, page):
    """Paths of up to 1023 entries: every key one place down, so that each entry
    reads what the next one writes; every other node; 64 and 65 entries with gaps;
    one whose tail alone moves."""
    banner(f"kv4_compact long paths {hkv} {d} {page}")
    g = gen(51 + d)
    nodes = [1024, 1000, 300, 300, 200]
    paths = [[0] + list(range(2, 1024)), list(range(0, 1000, 2)), sorted(torch.randperm(300, generator=g)[:64].tolist()),
             sorted(torch.randperm(300, generator=g)[:65].tolist()), list(range(130)) + [140, 199]]
    starts = np.cumsum([0] + nodes).tolist()
    lens = [n + 7 * i for i, n in enumerate(nodes)]
    most = max(map(len, paths))
    pages = sum(-(-n // page) for n in lens) + 1
    tab = tables(g, lens, page, pages)
    want = layer.Cache(pages, hkv, d, page)
    want.bytes = torch.randint(0, 256, want.bytes.shape, generator=g, dtype=torch.uint8)
    cache = want.flat().to(dev)
    path = torch.full((len(nodes), most), -1, dtype=torch.int32)
    for b, p in enumerate(paths):
        path[b, : len(p)] = torch.tensor(p, dtype=torch.int32)
    bq.kv4_compact(cache, tab.to(dev), i32(lens, dev), path.to(dev), i32([len(p) for p in paths], dev), page, hkv, d, i32(starts, dev),
                   total_q=starts[-1])
    for b, n in enumerate(nodes):
        decode.compact(want, tab[b], lens[b], n, paths[b])
    assert torch.equal(cache.cpu(), want.flat())


@pytest.mark.parametrize("T", TYPES)
@pytest.mark.parametrize("d,nodes,wide", [(64, 40, 1), (128, 40, 1), (64, 40, 4096), (128, 40, 4096), (256, 40, 1)])
def test_attn_kv4_tree_repeats_itself(bq, dev, T, d, nodes, wide):
    """The same call gives the same bits, with whatever lies in the workspace."""
    banner(f"tree attention again {d} {nodes} {wide} {T}")
    g = gen(52)
    hq, hkv, page, lens = 32, 4, 16, [700, 90, 1501, 41]
    pages = sum(-(-n // page) for n in lens)
    cache = make_cache(g, pages, hkv, d, page, T).flat().to(dev)
    tab = tables(g, lens, page, pages)
    tab = torch.cat([tab, torch.full((len(lens), wide), -1, dtype=torch.int32)], 1).to(dev)
    _, _, mask, _ = trees(g, [nodes] * len(lens))
    q = torch.randn(len(lens) * nodes, hq, d, generator=g).to(T).to(dev)
    n = max(16, bq.attn_kv4_tree_workspace_bytes(len(lens), nodes, hq, hkv, d, tab.shape[1] * page))
    first = None
    for fill in (0, 255, 60, 127):
        ws = torch.full((n,), fill, dtype=torch.uint8, device=dev)
        got = bq.attn_kv4_tree(q, cache, tab, i32(lens, dev), page, hkv, mask.to(dev), return_lse=True, workspace=ws)
        torch.cuda.synchronize()
        first = first or [x.clone() for x in got]
        assert all(torch.equal(a, b) for a, b in zip(first, got))


@pytest.mark.parametrize("T", TYPES)
@pytest.mark.parametrize("nodes", [3, 300])
def test_attn_kv4_tree_without_pages(bq, dev, T, nodes):
    """A table of no columns over a cache of no pages: no row sees a key."""
    banner(f"tree attention without pages {nodes} {T}")
    hq, hkv, d, page, B = 8, 2, 128, 16, 2
    _, _, mask, _ = trees(gen(53), [nodes] * B)
    q = torch.randn(B * nodes, hq, d, generator=gen(54)).to(T).to(dev)
    cache = torch.empty(0, bq.kv4_page_bytes(hkv, d, page), dtype=torch.uint8, device=dev)
    tab = torch.empty(B, 0, dtype=torch.int32, device=dev)
    out, lse = bq.attn_kv4_tree(q, cache, tab, i32([nodes, 900], dev), page, hkv, mask.to(dev), return_lse=True)
    assert not out.any() and (lse == -float("inf")).all()


@pytest.mark.parametrize("T", TYPES)
@pytest.mark.parametrize("wide", [1, 4096])
def test_attn_kv4_tree_more_nodes_than_are_computed(bq, dev, T, wide):
    """2000 nodes behind one prefix, the first 1024 of them computed: their rows
    are those of a tree whose other nodes no row sees, the others' stay."""
    banner(f"tree attention 1024 of 2000 nodes {wide} {T}")
    g = gen(55)
    hq, hkv, d, page, nodes, prefix = 2, 2, 64, 16, 2000, 77
    n = prefix + nodes
    cache = make_cache(g, -(-n // page), hkv, d, page, T)
    tab = torch.cat([tables(g, [n], page, -(-n // page)), torch.full((1, wide), -1, dtype=torch.int32)], 1)
    _, see, mask, _ = trees(g, [1024])
    words = torch.full((nodes, 32), -1, dtype=torch.int32)
    words[:1024] = mask
    q = torch.randn(nodes, hq, d, generator=g).to(T)
    out = torch.full(q.shape, 7.0, dtype=T, device=dev)
    lse = torch.full(q.shape[:2], 7.0, device=dev)
    bq.attn_kv4_tree(q.to(dev), cache.flat().to(dev), tab.to(dev), i32([n], dev), page, hkv, words.to(dev), None, i32([0, nodes], dev),
                     1024, 0, out, lse)
    whole = torch.zeros(nodes, nodes, dtype=torch.bool)
    whole[:1024, :1024] = see[0]
    want, _, size, delta = decode.attention_tree(q, cache, tab, [n], [0, nodes], [whole], d ** -0.5)
    r = (2.0 ** -20 if T == torch.float16 else 2.0 ** -10 + 2.0 ** -20) + n * 2.0 ** -24
    tol = half_step(T) * want.abs() + (2 * delta[..., None] + r) * size * (1 + 2.0 ** -6) + 2.0 ** -25
    within(out[:1024], want[:1024], tol[:1024], "first nodes")
    assert (out[1024:] == 7).all() and (lse[1024:] == 7).all()
