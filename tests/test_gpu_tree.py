"""The cache's move along paths longer than a wavefront, and attention over a
tree called again on the same inputs."""
import numpy as np
import pytest
import torch

from decode_cases import gen, trees
from gpu_util import banner, need_gpu
from oracle import decode, layer
from test_gpu_decode import TYPES, i32
from test_gpu_layer import make_cache, tables

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
