"""The decoding entry points (include/bq_decode.h): exported, and their
refusals decided on the host before any device call (no GPU needed)."""
import ctypes
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "bq_decode.h")

P = [ctypes.c_void_p(0x1000 * (i + 1)) for i in range(14)]  # never dereferenced
ODD = ctypes.c_void_p(0x1001)
NULL = ctypes.c_void_p(0)


@pytest.fixture(scope="module")
def bq():
    from bit_mixed_precision_amd import bq as _bq

    if not os.path.exists(_bq.LIB_PATH):
        import __graft_entry__

        __graft_entry__.build()
    return _bq


def test_exports_every_declared_symbol(bq):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(bq_[a-z0-9_]+)\s*\(", text)))
    assert set(names) == set(bq.DECODE_SIGNATURES)
    lib = ctypes.CDLL(bq.LIB_PATH)
    for n in names:
        assert hasattr(lib, n), n


NODES = (dict(batch=-1), dict(total=7), dict(maxq=2), dict(maxq=1025, total=2050), dict(maxq=-1), dict(batch=2**30 + 1),
         dict(total=2**30 + 1, qs=P[12]), dict(total=-1, qs=P[12]))


def _mask(bq, **change):
    a = dict(parents=P[0], qs=NULL, lens=P[1], batch=2, total=6, maxq=3, words=1, mask=P[2], pos=P[3], stream=NULL)
    a.update(change)
    return bq.lib().bq_tree_mask(*a.values())


def test_tree_mask_refusals(bq):
    for bad in NODES + (dict(words=0), dict(words=33), dict(words=-1)):
        assert _mask(bq, **bad) == bq.BQ_ERR_SHAPE, bad
    for bad in (dict(parents=NULL), dict(mask=NULL)):
        assert _mask(bq, **bad) == bq.BQ_ERR_NULL, bad
    for bad in (dict(parents=ODD), dict(mask=ODD), dict(pos=ODD), dict(lens=ODD), dict(qs=ODD)):
        assert _mask(bq, **bad) == bq.BQ_ERR_ALIGN, bad
    assert _mask(bq, batch=0, total=0, parents=NULL, mask=NULL) == bq.BQ_OK
    assert _mask(bq, maxq=0, total=0, parents=NULL, mask=NULL) == bq.BQ_OK


def _accept(bq, **change):
    a = dict(tokens=P[0], parents=P[1], sampled=P[2], qs=NULL, batch=2, total=6, maxq=3, most=3, path=P[3], count=P[4],
             next=P[5], stream=NULL)
    a.update(change)
    return bq.lib().bq_tree_accept(*a.values())


def test_tree_accept_refusals(bq):
    for bad in NODES + (dict(most=0), dict(most=1025), dict(most=-1)):
        assert _accept(bq, **bad) == bq.BQ_ERR_SHAPE, bad
    for bad in (dict(tokens=NULL), dict(parents=NULL), dict(sampled=NULL), dict(path=NULL), dict(count=NULL), dict(next=NULL),
                dict(maxq=0, total=0, path=NULL)):
        assert _accept(bq, **bad) == bq.BQ_ERR_NULL, bad
    for bad in (dict(tokens=ODD), dict(parents=ODD), dict(sampled=ODD), dict(path=ODD), dict(count=ODD), dict(next=ODD),
                dict(qs=ODD)):
        assert _accept(bq, **bad) == bq.BQ_ERR_ALIGN, bad
    assert _accept(bq, batch=0, total=0, path=NULL, count=NULL, next=NULL) == bq.BQ_OK


def _compact(bq, **change):
    a = dict(cache=P[0], layers=2, stride=4 * 2 * 16 * 136, pages=4, page=16, hkv=2, d=128, table=P[1], blocks=3, qs=NULL,
             lens=P[2], batch=2, total=6, maxq=3, path=P[3], count=P[4], most=3, stream=NULL)
    a.update(change)
    return bq.lib().bq_kv4_compact(*a.values())


def test_kv4_compact_refusals(bq):
    for bad in NODES + (dict(layers=-1), dict(layers=65537), dict(stride=4 * 2 * 16 * 136 - 16), dict(stride=-16), dict(pages=-1),
                        dict(page=17), dict(hkv=0), dict(d=96), dict(blocks=-1), dict(blocks=2**27), dict(most=0), dict(most=1025)):
        assert _compact(bq, **bad) == bq.BQ_ERR_SHAPE, bad
    for bad in (dict(cache=NULL), dict(table=NULL), dict(lens=NULL), dict(path=NULL), dict(count=NULL)):
        assert _compact(bq, **bad) == bq.BQ_ERR_NULL, bad
    for bad in (dict(cache=ODD), dict(stride=4 * 2 * 16 * 136 + 8), dict(table=ODD), dict(lens=ODD), dict(path=ODD), dict(count=ODD),
                dict(qs=ODD)):
        assert _compact(bq, **bad) == bq.BQ_ERR_ALIGN, bad
    for empty in (dict(batch=0, total=0), dict(layers=0), dict(maxq=0, total=0), dict(blocks=0), dict(pages=0)):
        assert _compact(bq, cache=NULL, table=NULL, **empty) == bq.BQ_OK, empty


def _sample(bq, **change):
    a = dict(logits=P[0], stride=1000, dtype=2, rows=3, vocab=1000, u=P[1], t=P[2], k=P[3], p=P[4], m=P[5], tokens=P[6], lp=P[7],
             ws=NULL, wsb=0, stream=NULL)
    a.update(change)
    return bq.lib().bq_sample(*a.values())


def test_sample_refusals(bq):
    for bad in (dict(dtype=3), dict(dtype=-1)):
        assert _sample(bq, **bad) == bq.BQ_ERR_ARG, bad
    for bad in (dict(rows=-1), dict(rows=2**30 + 1), dict(vocab=0), dict(vocab=-5), dict(vocab=2**24 + 1, stride=2**25),
                dict(stride=999), dict(stride=-1000), dict(wsb=-1)):
        assert _sample(bq, **bad) == bq.BQ_ERR_SHAPE, bad
    for bad in (dict(logits=NULL), dict(u=NULL), dict(tokens=NULL), dict(wsb=64)):
        assert _sample(bq, **bad) == bq.BQ_ERR_NULL, bad
    for bad in (dict(logits=ODD), dict(logits=ctypes.c_void_p(0x1002)), dict(u=ODD), dict(t=ODD), dict(k=ODD), dict(p=ODD),
                dict(m=ODD), dict(tokens=ODD), dict(lp=ODD), dict(ws=ODD, wsb=64), dict(logits=ODD, dtype=0)):
        assert _sample(bq, **bad) == bq.BQ_ERR_ALIGN, bad
    assert _sample(bq, rows=0, logits=NULL, u=NULL, tokens=NULL) == bq.BQ_OK
    f = bq.lib().bq_sample_workspace_bytes
    assert f(4, 0, 2) == -bq.BQ_ERR_SHAPE and f(-1, 10, 2) == -bq.BQ_ERR_SHAPE and f(4, 10, 7) == -bq.BQ_ERR_ARG
    assert f(0, 1000, 0) == 0 and f(5, 1000, 1) >= 0


def _attn(bq, **change):
    a = dict(q=P[0], qs=1024, dtype=0, q_start=NULL, lens=P[1], table=P[2], batch=2, total=6, maxq=3, hq=8, hkv=2, d=128,
             cache=P[3], pages=9, page=16, blocks=5, mask=P[8], words=1, scale=0.1, window=0, out=P[4], lse=P[5], ws=NULL, wsb=0,
             stream=NULL)
    a.update(change)
    return bq.lib().bq_attn_kv4_tree(*a.values())


def test_attn_kv4_tree_refusals(bq):
    assert _attn(bq, dtype=5) == bq.BQ_ERR_ARG
    for bad in (float("nan"), float("inf")):
        assert _attn(bq, scale=bad) == bq.BQ_ERR_ARG
    for bad in (dict(batch=-1), dict(total=3), dict(maxq=2), dict(hq=7), dict(hkv=0), dict(d=32), dict(page=17), dict(blocks=-1),
                dict(blocks=2**27), dict(window=-1), dict(window=2**31), dict(pages=-1), dict(pages=0), dict(wsb=-8), dict(qs=512),
                dict(total=2**30 + 1, q_start=P[6]), dict(words=0), dict(words=33), dict(maxq=1025, total=2050)):
        assert _attn(bq, **bad) == bq.BQ_ERR_SHAPE, bad
    for bad in (dict(q=NULL), dict(lens=NULL), dict(table=NULL), dict(cache=NULL), dict(out=NULL), dict(wsb=64), dict(mask=NULL)):
        assert _attn(bq, **bad) == bq.BQ_ERR_NULL, bad
    for bad in (dict(q=ODD), dict(qs=1028), dict(out=ODD), dict(cache=ODD), dict(lens=ODD), dict(table=ODD), dict(lse=ODD),
                dict(q_start=ODD), dict(ws=ODD, wsb=64), dict(mask=ODD)):
        assert _attn(bq, **bad) == bq.BQ_ERR_ALIGN, bad
    assert _attn(bq, batch=0, total=0) == bq.BQ_OK
    assert _attn(bq, maxq=0, total=0) == bq.BQ_OK
    f = bq.attn_kv4_tree_workspace_bytes
    assert f(0, 8, 8, 2, 128, 1000) == 0
    assert f(1, 8, 8, 2, 128, 100000) > 0
    for bad in ((-1, 1, 8, 2, 128, 10), (1, 1025, 8, 2, 128, 10), (1, 1, 7, 2, 128, 10), (1, 1, 8, 2, 100, 10)):
        with pytest.raises(bq.BQError):
            f(*bad)


def test_python_arguments_are_checked(bq):
    """The binding's own refusals, on CPU tensors."""
    import torch

    i32 = torch.zeros(2, 3, dtype=torch.int32)
    flat = i32.view(-1)
    for bad in (lambda: bq.tree_mask(i32), lambda: bq.tree_mask(flat), lambda: bq.tree_mask(i32, max_q_len=4),
                lambda: bq.tree_mask(i32, q_start=flat), lambda: bq.tree_mask(flat, q_start=flat),
                lambda: bq.tree_accept(i32, i32, i32), lambda: bq.tree_accept(flat, flat, flat),
                lambda: bq.sample(torch.zeros(2, 5), torch.zeros(2)), lambda: bq.sample(torch.zeros(5), torch.zeros(1)),
                lambda: bq.sample(torch.zeros(2, 5, dtype=torch.float64), torch.zeros(2)),
                lambda: bq.sample_workspace_bytes(2, 5, torch.float64),
                lambda: bq.kv4_compact(torch.zeros(2, 5, dtype=torch.uint8), i32, flat, i32, flat, 16, 2, 128, max_q_len=3),
                lambda: bq.kv4_compact(torch.zeros(5, dtype=torch.uint8), i32, flat, i32, flat, 16, 2, 128, max_q_len=3)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: bq.tree_mask(None), lambda: bq.sample(None, None), lambda: bq.tree_accept(None, i32, i32)):
        with pytest.raises(TypeError):
            bad()
    x = torch.zeros(6, 2, 128).half()
    with pytest.raises(ValueError):
        bq.attn_kv4_tree(x, torch.zeros(2, 2 * 16 * 136, dtype=torch.uint8), i32, flat[:2], 16, 2, None)
    with pytest.raises(ValueError):
        bq.attn_kv4_tree(x, torch.zeros(2, 2 * 16 * 136, dtype=torch.uint8), i32, flat[:2], 16, 2, i32)


@pytest.mark.parametrize("bad", [None, 3, [[0, 1]]])
def test_what_is_no_tensor_is_a_type_error(bq, bad):
    """Arguments whose dimensions are looked at first: no AttributeError."""
    import torch

    i32 = torch.zeros(2, 3, dtype=torch.int32)
    flat = i32.view(-1)
    given = dict(cache=torch.zeros(2, 2 * 16 * 136, dtype=torch.uint8), block_table=i32, seq_lens=flat[:2], path=i32, count=flat[:2])
    for name in ("cache", "block_table", "path"):
        with pytest.raises(TypeError, match=name):
            bq.kv4_compact(**{**given, name: bad}, page_size=16, kv_heads=2, head_dim=128, max_q_len=3)
    if bad is not None:  # None: made by the call
        with pytest.raises(TypeError, match="mask"):
            bq.tree_mask(i32, mask=bad)
        with pytest.raises(TypeError, match="path"):
            bq.tree_accept(i32, i32, i32, path=bad)
