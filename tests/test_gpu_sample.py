"""Sampling where a call could go wrong without its choice lying at a border:
rows that change over from one way through the kernels to another, the ends of
the random numbers, log probabilities of light tokens.  Bounds as in
test_gpu_decode.py unless a test derives its own."""
import math

import numpy as np
import pytest
import torch

from decode_cases import gen, logits_row
from gpu_util import banner, need_gpu
from test_gpu_decode import TYPES, check_sample, on, sample_settings

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    return need_gpu()


@pytest.fixture(scope="module")
def bq(dev):
    from bit_mixed_precision_amd import bq as _bq

    return _bq


@pytest.mark.parametrize("T", TYPES + [torch.float32])
def test_held_rows_that_are_selected_over(bq, dev, T):
    """Rows that a workgroup holds in registers and, their top_k being past its
    groups, then selects over in memory: among rows of nothing but -infinity and
    NaN, greedy ones, and ones that stay in the registers.  Their wavefronts use
    the same shared memory for both."""
    banner(f"sample: held rows that are selected over {T}")
    g = gen(41)
    rows, vocab = 96, 9001
    x = torch.stack([logits_row(g, vocab, 6.0, T) for _ in range(rows)])
    x[5::12] = -math.inf
    x[8::12] = math.nan
    x[11::12, 1:] = -math.inf
    u, t, k, p, m = sample_settings(g, rows, "kpm", vocab)
    k = torch.where(torch.arange(rows) % 4 < 3, torch.randint(257, vocab, (rows,), generator=g), k).to(torch.int32)
    t[::16] = 0.0
    for args in ((u, t, k, None, None), (u, t, k, p, None), (u, t, k, p, m)):
        moved = [on(v, dev) for v in args]
        first = bq.sample(x.to(dev), *moved)
        check_sample(first, x, *args)
        again = bq.sample(x.to(dev), *moved)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
