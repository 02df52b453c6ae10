"""The decoding operators' oracle against cases that can be written down by
hand, and against oracle.layer's attention where a tree is a chain (CPU)."""
import math

import numpy as np
import pytest
import torch

from decode_cases import gen, logits_row, random_tree
from oracle import decode, layer

F64 = torch.float64


def test_ancestors_and_words():
    see, depth = decode.ancestors([-1, 0, 0, 1, 3, 7, 2])  # node 5's parent is none
    assert depth == [0, 1, 1, 2, 3, 0, 2]
    want = [{0}, {0, 1}, {0, 2}, {0, 1, 3}, {0, 1, 3, 4}, {5}, {0, 2, 6}]
    assert [set(np.nonzero(r)[0]) for r in see] == want
    w = decode.words_of(np.eye(70, dtype=bool), 2)
    assert w.shape == (70, 2) and int(w[31, 0]) == -(1 << 31) and int(w[32, 1]) == 1 and int(w[69].abs().sum()) == 0


def test_accept():
    tokens, parents = [5, 7, 8, 7, 9, 7], [-1, 0, 0, 1, 1, 0]
    assert decode.accept(tokens, parents, [7, 9, 1, 1, 4, 3], 9) == ([0, 1, 4], 4)
    assert decode.accept(tokens, parents, [7, 9, 1, 1, 4, 3], 2) == ([0, 1], 9)
    assert decode.accept(tokens, parents, [6, 9, 1, 1, 4, 3], 9) == ([0], 6)
    assert decode.accept([], [], [], 9) == ([], -1)


def test_sample_by_hand():
    x = np.log(np.array([1, 2, 4, 1, 8], dtype=np.float64)).astype(np.float32)
    draw = lambda u, **kw: decode.sample(x, u, **kw)[0]  # noqa: E731
    assert [draw(u) for u in (0, 0.05, 0.1, 0.3, 0.48, 0.52, 0.999, 1.0, math.nan)] == [0, 0, 1, 2, 3, 4, 4, 4, 4]
    assert {draw(u, top_k=2) for u in np.linspace(0, 0.99, 50)} == {2, 4}
    assert {draw(u, top_k=4) for u in np.linspace(0, 0.99, 50)} == {0, 1, 2, 4}  # equal ones by index
    assert {draw(u, top_p=0.6) for u in np.linspace(0, 0.99, 50)} == {2, 4}
    assert {draw(u, top_p=0.0) for u in np.linspace(0, 0.99, 50)} == {4}
    assert {draw(u, top_k=2, top_p=0.66) for u in np.linspace(0, 0.99, 50)} == {4}
    assert {draw(u, min_p=0.2) for u in np.linspace(0, 0.99, 50)} == {1, 2, 4}
    assert {draw(u, min_p=7.0) for u in np.linspace(0, 0.99, 50)} == {4}
    assert draw(0.3, t=0.0) == draw(0.3, t=-1.0) == draw(0.3, t=math.nan) == 4
    assert [draw(u, t=math.inf) for u in (0.1, 0.3, 0.5, 0.7, 0.9)] == [0, 1, 2, 3, 4]
    assert abs(decode.sample(x, 0.3)[1] - math.log(4 / 16)) < 1e-6
    assert abs(decode.sample(x, 0.3, t=0.5)[1] - math.log(64 / 86)) < 1e-6
    y = np.array([-math.inf, math.nan, -3e38, -math.inf], dtype=np.float32)
    assert decode.sample(y, 0.5)[:2] == (2, 0.0)
    assert decode.sample(y[:2], 0.5)[0] == -1
    assert {decode.sample(np.array([0, math.inf, 5, math.inf], dtype=np.float32), u)[0] for u in (0, 0.4, 0.6, 0.9)} == {1, 3}


def test_sample_draws_every_token_as_often_as_it_weighs():
    g = gen(3)
    x = logits_row(g, 50, 4.0, torch.float32)
    p = torch.softmax(x.to(F64) / 0.7, 0)
    n = 4000
    hits = np.bincount([decode.sample(x.numpy(), (i + 0.5) / n, t=0.7)[0] for i in range(n)], minlength=50) / n
    assert np.abs(hits - p.numpy()).max() <= 1.0 / n


@pytest.mark.parametrize("window", [0, 9])
def test_a_chain_is_causal(window):
    g = gen(8)
    hkv, hq, d, page, n, nodes = 2, 4, 64, 16, 37, 6
    cache = layer.Cache(3, hkv, d, page)
    for s in range(48):
        cache.write(s, torch.randn(hkv, d, generator=g).half(), torch.randn(hkv, d, generator=g).half())
    table = torch.tensor([[2, 0, 1]], dtype=torch.int32)
    q = torch.randn(nodes, hq, d, generator=g).half()
    see, _ = decode.ancestors(list(range(-1, nodes - 1)))
    a = decode.attention_tree(q, cache, table, [n], [0, nodes], [torch.from_numpy(see)], 0.2, window)
    b = layer.attention(q, cache, table, [n], [0, nodes], 0.2, window)
    for x, y in zip(a[:3], b[:3]):
        assert torch.allclose(x, y, rtol=1e-12, atol=1e-12)


def test_compact_by_hand():
    g = gen(5)
    hkv, d, page = 2, 64, 16
    cache = layer.Cache(3, hkv, d, page)
    for s in range(48):
        cache.write(s, torch.randn(hkv, d, generator=g).half(), torch.randn(hkv, d, generator=g).half())
    before = cache.bytes.clone()
    table = [2, 0]
    old = lambda t: [x for part in _read(before, cache, table, t) for x in part]  # noqa: E731
    decode.compact(cache, table, 30, 16, [0, 2, 3, 9])  # prefix 14: keys 16, 17, 23 to 15, 16, 17
    now = lambda t: [x for part in _read(cache.bytes, cache, table, t) for x in part]  # noqa: E731
    for t in range(32):
        was = {15: 16, 16: 17, 17: 23}.get(t, t)
        assert all(torch.equal(a, b) for a, b in zip(now(t), old(was))), t
    assert torch.equal(cache.bytes[1], before[1])


def _read(raw, cache, table, t):
    keep, cache.bytes = cache.bytes, raw
    try:
        return cache.read(table[t // cache.size] * cache.size + t % cache.size)
    finally:
        cache.bytes = keep


def test_trees_are_trees():
    for n in (1, 2, 33, 100):
        p = random_tree(gen(n), n)
        assert p[0] == -1 and all(0 <= p[i] < i for i in range(1, n))
