"""The decoder-layer entry points (include/bq_layer.h): exported, and their
refusals decided on the host before any device call (no GPU needed)."""
import ctypes
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "bq_layer.h")

P = [ctypes.c_void_p(0x1000 * (i + 1)) for i in range(12)]  # never dereferenced
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
    assert set(names) == set(bq.LAYER_SIGNATURES)
    lib = ctypes.CDLL(bq.LIB_PATH)
    for n in names:
        assert hasattr(lib, n), n


def _gemm(bq, **change):
    a = dict(A=P[0], dtype=0, B=P[1], scale=P[2], zero=NULL, group=128, C=P[3], M=4, N=8, K=256, ws=NULL, wsb=0, stream=NULL)
    a.update(change)
    return bq.lib().bq_gemm_w4g_a16(*a.values())


def test_gemm_w4g_refusals(bq):
    for bad in (dict(dtype=2), dict(dtype=-1), dict(group=16), dict(group=0), dict(group=256)):
        assert _gemm(bq, **bad) == bq.BQ_ERR_ARG, bad
    for bad in (dict(M=-1), dict(N=-1), dict(K=-64), dict(K=96, group=32), dict(K=192), dict(K=65536 + 128),
                dict(M=2**30 + 1), dict(M=2**21, N=2**21 + 1), dict(wsb=-1)):
        assert _gemm(bq, **bad) == bq.BQ_ERR_SHAPE, bad
    for bad in (dict(A=NULL), dict(B=NULL), dict(scale=NULL), dict(C=NULL), dict(wsb=16)):
        assert _gemm(bq, **bad) == bq.BQ_ERR_NULL, bad
    for bad in (dict(A=ODD), dict(B=ODD), dict(scale=ODD), dict(zero=ODD), dict(C=ODD), dict(ws=ODD, wsb=16)):
        assert _gemm(bq, **bad) == bq.BQ_ERR_ALIGN, bad
    assert _gemm(bq, M=0, A=NULL, C=NULL) == bq.BQ_OK
    assert _gemm(bq, N=0, B=NULL, C=NULL) == bq.BQ_OK
    assert bq.lib().bq_gemm_w4g_workspace_bytes(4, 8, 100) == -bq.BQ_ERR_SHAPE
    assert bq.lib().bq_gemm_w4g_workspace_bytes(-1, 8, 128) == -bq.BQ_ERR_SHAPE
    assert bq.gemm_w4g_workspace_bytes(0, 8, 128) == 0


def _rope(bq, **change):
    a = dict(q=P[0], qs=1024, k=P[1], ks=256, dtype=0, tokens=3, hq=8, hkv=2, d=128, wq=P[2], wk=P[3], eps=1e-6, cos=P[4],
             sin=P[5], max_pos=10, rot=128, inter=0, pos=P[6], qo=P[7], ko=P[8], stream=NULL)
    a.update(change)
    return bq.lib().bq_qk_norm_rope(*a.values())


def test_qk_norm_rope_refusals(bq):
    for bad in (dict(dtype=3), dict(eps=-1.0), dict(eps=float("nan"))):
        assert _rope(bq, **bad) == bq.BQ_ERR_ARG, bad
    for bad in (dict(tokens=-1), dict(d=96), dict(d=0), dict(hq=-1), dict(hkv=70000), dict(rot=8), dict(rot=144), dict(rot=-16),
                dict(max_pos=-1), dict(qs=1016), dict(ks=0), dict(qs=-1024)):
        assert _rope(bq, **bad) == bq.BQ_ERR_SHAPE, bad
    for bad in (dict(q=NULL), dict(k=NULL), dict(qo=NULL), dict(ko=NULL), dict(cos=NULL), dict(sin=NULL), dict(pos=NULL),
                dict(wq=NULL), dict(wk=NULL)):
        assert _rope(bq, **bad) == bq.BQ_ERR_NULL, bad
    for bad in (dict(q=ODD), dict(qs=1028), dict(ks=260), dict(qo=ODD), dict(ko=ODD), dict(wq=ODD), dict(wk=ODD), dict(cos=ODD),
                dict(pos=ODD)):
        assert _rope(bq, **bad) == bq.BQ_ERR_ALIGN, bad
    assert _rope(bq, tokens=0, q=NULL, k=NULL) == bq.BQ_OK
    assert _rope(bq, hq=0, hkv=0, q=NULL, k=NULL) == bq.BQ_OK


def _append(bq, **change):
    a = dict(q=P[0], qs=1024, k=P[1], ks=256, v=P[9], vs=256, dtype=1, tokens=3, hq=8, hkv=2, d=128, wq=P[2], wk=P[3],
             eps=1e-6, cos=P[4], sin=P[5], max_pos=10, rot=128, inter=0, pos=P[6], qo=P[7], cache=P[8], pages=4, page=16,
             slots=P[10], stream=NULL)
    a.update(change)
    return bq.lib().bq_qk_norm_rope_kv4(*a.values())


def test_qk_norm_rope_kv4_refusals(bq):
    for bad in (dict(page=8), dict(page=48), dict(page=512), dict(pages=-1), dict(hkv=0), dict(vs=128), dict(d=80)):
        assert _append(bq, **bad) == bq.BQ_ERR_SHAPE, bad
    for bad in (dict(v=NULL), dict(cache=NULL), dict(slots=NULL), dict(wk=NULL)):
        assert _append(bq, **bad) == bq.BQ_ERR_NULL, bad
    for bad in (dict(v=ODD), dict(cache=ODD), dict(slots=ODD), dict(vs=260)):
        assert _append(bq, **bad) == bq.BQ_ERR_ALIGN, bad
    assert _append(bq, tokens=0) == bq.BQ_OK


def test_kv4_read_refusals_and_page_bytes(bq):
    f = bq.lib().bq_kv4_read
    assert f(P[0], 4, 16, 2, 128, P[1], 3, 2, P[2], P[3], NULL) == bq.BQ_ERR_ARG
    assert f(P[0], 4, 24, 2, 128, P[1], 3, 0, P[2], P[3], NULL) == bq.BQ_ERR_SHAPE
    assert f(P[0], 4, 16, 0, 128, P[1], 3, 0, P[2], P[3], NULL) == bq.BQ_ERR_SHAPE
    assert f(P[0], -1, 16, 2, 128, P[1], 3, 0, P[2], P[3], NULL) == bq.BQ_ERR_SHAPE
    assert f(P[0], 4, 16, 2, 128, NULL, 3, 0, P[2], P[3], NULL) == bq.BQ_ERR_NULL
    assert f(P[0], 4, 16, 2, 128, P[1], 3, 0, P[2], NULL, NULL) == bq.BQ_ERR_NULL
    assert f(ODD, 4, 16, 2, 128, P[1], 3, 0, P[2], P[3], NULL) == bq.BQ_ERR_ALIGN
    assert f(NULL, 4, 16, 2, 128, NULL, 0, 0, NULL, NULL, NULL) == bq.BQ_OK
    assert bq.kv4_page_bytes(2, 128, 16) == 2 * 16 * 136
    for bad in ((0, 128, 16), (2, 100, 16), (2, 128, 20)):
        with pytest.raises(bq.BQError):
            bq.kv4_page_bytes(*bad)


def _attn(bq, **change):
    a = dict(q=P[0], qs=1024, dtype=0, q_start=NULL, lens=P[1], table=P[2], batch=2, total=2, maxq=1, hq=8, hkv=2, d=128,
             cache=P[3], pages=9, page=16, blocks=5, scale=0.1, window=0, out=P[4], lse=P[5], ws=NULL, wsb=0, stream=NULL)
    a.update(change)
    return bq.lib().bq_attn_kv4(*a.values())


def test_attn_kv4_refusals(bq):
    assert _attn(bq, dtype=5) == bq.BQ_ERR_ARG
    for bad in (dict(batch=-1), dict(total=3), dict(maxq=2), dict(hq=7), dict(hkv=0), dict(hq=0), dict(d=32), dict(page=17),
                dict(blocks=-1), dict(blocks=2**27), dict(window=-1), dict(window=2**31), dict(pages=-1), dict(pages=0),
                dict(wsb=-8), dict(qs=512), dict(total=2**30 + 1, q_start=P[6])):
        assert _attn(bq, **bad) == bq.BQ_ERR_SHAPE, bad
    for bad in (dict(q=NULL), dict(lens=NULL), dict(table=NULL), dict(cache=NULL), dict(out=NULL), dict(wsb=64)):
        assert _attn(bq, **bad) == bq.BQ_ERR_NULL, bad
    for bad in (dict(q=ODD), dict(qs=1028), dict(out=ODD), dict(cache=ODD), dict(lens=ODD), dict(table=ODD), dict(lse=ODD),
                dict(q_start=ODD), dict(ws=ODD, wsb=64)):
        assert _attn(bq, **bad) == bq.BQ_ERR_ALIGN, bad
    assert _attn(bq, batch=0, total=0) == bq.BQ_OK
    assert _attn(bq, maxq=0, total=0) == bq.BQ_OK


def test_attn_kv4_workspace(bq):
    f = bq.attn_kv4_workspace_bytes
    assert f(0, 1, 8, 2, 128, 1000) == 0
    assert f(1, 1, 8, 2, 128, 16) == 0            # too short to split
    assert f(1, 1, 8, 2, 128, 1024) == 0
    assert f(1, 1, 8, 2, 128, 100000) > 0
    assert f(1, 1, 8, 2, 128, 100000) % (2 * 16 * 130 * 4) == 0
    for bad in ((-1, 1, 8, 2, 128, 10), (1, 1, 7, 2, 128, 10), (1, 1, 8, 2, 100, 10), (1, 1, 8, 2, 128, 2**31),
                (2**30, 2**30, 1, 1, 128, 16)):
        with pytest.raises(bq.BQError):
            f(*bad)


def test_python_arguments_are_checked(bq):
    """The binding's own refusals, on CPU tensors (no GPU tensor is needed to
    be refused)."""
    import torch

    A, B, s = torch.zeros(2, 128).half(), torch.zeros(4, 64, dtype=torch.uint8), torch.zeros(4, 1).half()
    with pytest.raises(ValueError):
        bq.gemm_w4g_a16(A, B, s)  # not on a GPU
    with pytest.raises(ValueError):
        bq.gemm_w4g_a16(A.float(), B, s)
    with pytest.raises(TypeError):
        bq.gemm_w4g_a16(None, B, s)
    x = torch.zeros(3, 2, 128).half()
    with pytest.raises(ValueError):
        bq.qk_norm_rope(x, x, None, None, None)
    with pytest.raises(ValueError):
        bq.kv4_read(torch.zeros(2, 5, dtype=torch.uint8), torch.zeros(3, dtype=torch.int64), 16, 2, 128, torch.float32)
    with pytest.raises(ValueError):
        bq.attn_kv4(x, torch.zeros(2, 2 * 16 * 136, dtype=torch.uint8), torch.zeros(3, 2, dtype=torch.int32),
                    torch.zeros(3, dtype=torch.int32), 16, 2)


def test_attn_kv4_refuses_scales_that_are_no_numbers(bq):
    for bad in (float("nan"), float("inf"), -float("inf")):
        assert _attn(bq, scale=bad) == bq.BQ_ERR_ARG, bad
        assert _attn(bq, scale=bad, batch=0, total=0) == bq.BQ_ERR_ARG, bad
    assert _attn(bq, scale=3e38, batch=0, total=0) == bq.BQ_OK
