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


@pytest.mark.parametrize("T", TYPES + [torch.float32])
@pytest.mark.parametrize("rows,vocab", [(7, 30011), (5, 50021), (3, 140007)])
def test_every_unit_of_a_row_is_found_again(bq, dev, T, rows, vocab):
    """Random numbers of 1 and just below it draw from the last unit of the kept
    weights: the row that is read for the token has to sum up to exactly what the
    parts' sums said, or no token is written.  With the call's own workspace and
    with none, tokens and log probabilities are the same bits."""
    banner(f"sample: the last unit {rows} x {vocab} {T}")
    g = gen(43)
    for filters in ("", "p", "m", "pm", "k", "kpm"):
        for last in (1.0, 1 - 2.0 ** -24, math.nan):
            x = torch.stack([logits_row(g, vocab, 6.0, T) for _ in range(rows)])
            u, t, k, p, m = sample_settings(g, rows, filters, vocab)
            u, t = torch.full((rows,), last), 1.0 + torch.rand(rows, generator=g)  # no weight below 2^-40 of the greatest
            moved = [on(v, dev) for v in (u, t, k, p, m)]
            got = []
            for kw in ({}, dict(workspace=torch.empty(16, dtype=torch.uint8, device=dev))):
                tokens = torch.full((rows,), -7, dtype=torch.int32, device=dev)
                logprobs = torch.full((rows,), 7.0, device=dev)
                bq.sample(x.to(dev), *moved, tokens=tokens, logprobs=logprobs, **kw)
                got.append((tokens, logprobs))
            assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
            # 1 and NaN draw the last kept token whatever the sums are
            check_sample(got[0], x, u, t, k, p, m, exact=last != 1 - 2.0 ** -24)
