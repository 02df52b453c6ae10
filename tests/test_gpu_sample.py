"""Sampling where a call could go wrong without its choice lying at a border:
rows that change over from one way through the kernels to another, the ends of
the random numbers, log probabilities of light tokens.  Bounds as in
test_gpu_decode.py unless a test derives its own."""
import math

import numpy as np
import pytest
import torch

from decode_cases import gen, logits_row, sample_wants
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


@pytest.mark.parametrize("T", TYPES + [torch.float32])
@pytest.mark.parametrize("vocab", [50, 20011, 60013])
@pytest.mark.parametrize("ws", ["auto", "none"])
def test_log_probability_of_a_light_token(bq, dev, T, vocab, ws):
    """A random number of 0 draws the first kept token, however little it weighs:
    here e^-5 to e^-30.5 of the greatest, down to a few of the units that sums are
    held in.  Its log probability is (x - max) / t less the logarithm of the kept
    weights' sum, over the greatest.  The sum is off by less than 1.125 vocab
    2^-(F + 1) of the greatest (F as in test_gpu_decode.py), which it is not less
    than, and so is its logarithm; the other term, at most 31 here, by a few 2^-52
    of itself, below 2^-40; the result is rounded to fp32, 2^-24 of itself."""
    banner(f"sample: a light token {vocab} {T} {ws}")
    down = [5.0, 12.0, 17.0, 20.25, 25.0, 28.0, 30.5]
    x = torch.full((len(down), vocab), -1000.0)
    x[:, vocab // 2], x[:, vocab // 2 + 1] = 0.0, -0.75
    x[:, 3] = -torch.tensor(down)
    x = x.to(T)
    rows = len(down)
    kw = {} if ws == "auto" else dict(workspace=torch.empty(16, dtype=torch.uint8, device=dev))
    frac = min(46, 61 - math.ceil(math.log2(vocab)))
    u = torch.zeros(rows)
    for t in (1.0, 0.5, 2.0):
        xt = (x.float() * t).to(T)  # whole powers of two: the same weights
        temp = torch.full((rows,), t)
        for k in (None, 3, 45):
            top_k = None if k is None else torch.full((rows,), k, dtype=torch.int32)
            tokens, logp = bq.sample(xt.to(dev), u.to(dev), temp.to(dev), on(top_k, dev), **kw)
            assert tokens.tolist() == [3] * rows
            w = np.exp((xt.float().numpy().astype(np.longdouble) - xt.float().amax(1, True).numpy()) / np.longdouble(t))
            kept = np.sort(w, 1)[:, -(k or vocab):].sum(1)
            want = np.log(w[:, 3] / kept).astype(np.float64)
            off = np.abs(logp.cpu().numpy().astype(np.float64) - want)
            assert (off <= 2.0 ** -24 * np.abs(want) + 1.125 * vocab * 2.0 ** -(frac + 1) + 2.0 ** -40).all(), off


@pytest.mark.parametrize("T", TYPES + [torch.float32])
@pytest.mark.parametrize("vocab", [1 << 24, (1 << 24) - 5])
def test_longest_rows(bq, dev, T, vocab):
    """Rows of 2^24 tokens, the most there may be: 3000 of them finite, the first
    and the last among these (the others weigh nothing, so that sums are of 3000
    terms and the bound is theirs, in units of 2^-37); then all equal, whose sums
    are exact."""
    banner(f"sample: longest rows {vocab} {T}")
    g = gen(44)
    rows, n = 2, 3000
    at = torch.randperm(vocab - 2, generator=g)[: n - 2] + 1
    at = torch.cat([torch.tensor([0]), at.sort()[0], torch.tensor([vocab - 1])])
    few = torch.stack([logits_row(g, n, 5.0, T) for _ in range(rows)])
    few[:, 0], few[:, -1] = 4.0, 4.5
    x = torch.full((rows, vocab), -math.inf, dtype=T, device=dev)
    x[:, at.to(dev)] = few.to(dev)
    for filters in ("", "p", "m", "kp", "kpm"):
        args = sample_settings(g, rows, filters, n)
        want, lp, margin = sample_wants(few, *args)
        assert (margin > 1.125 * n * 2.0 ** -37).all(), "an input at a border"
        tokens, logp = bq.sample(x, *(on(v, dev) for v in args))
        assert tokens.tolist() == at[torch.from_numpy(want).long()].tolist(), filters
        assert (np.abs(logp.cpu().numpy() - lp) <= 2.0 ** -24 * np.abs(lp) + 1.125 * n * 2.0 ** -38 + 2.0 ** -40).all()
    x.fill_(-1.5)
    u = torch.tensor([0.7181, 1 - 2.0 ** -24])
    tokens, logp = bq.sample(x, u.to(dev))
    assert tokens.tolist() == [math.floor(float(v) * vocab) for v in u]
    assert np.allclose(logp.cpu().numpy(), -math.log(vocab), rtol=2.0 ** -24)
    tokens, _ = bq.sample(x, u.to(dev), None, None, torch.tensor([0.25, 0.5], device=dev))
    assert tokens.tolist() == [math.floor(float(v) * math.ceil(p * vocab)) for v, p in zip(u, (0.25, 0.5))]


@pytest.mark.parametrize("T", [torch.float16, torch.float32])
def test_more_long_rows_than_workgroups_at_once(bq, dev, T):
    """3000 rows of 33001 tokens, each with other settings: every row as one
    workgroup over the whole of it has it, some against the definition."""
    banner(f"sample: many long rows {T}")
    g = gen(45)
    rows, vocab = 3000, 33001
    x = torch.randn(rows, vocab, generator=g).to(T)
    u, t, k, p, m = sample_settings(g, rows, "kpm", vocab)
    off = torch.rand(rows, 4, generator=g) < 0.4
    t, k, p, m = t * ~off[:, 0], k * ~off[:, 1], torch.where(off[:, 2], torch.ones(rows), p), m * ~off[:, 3]
    moved = [v.to(dev) for v in (u, t, k, p, m)]
    y = x.to(dev)
    a = bq.sample(y, *moved)
    b = bq.sample(y, *moved, workspace=torch.empty(16, dtype=torch.uint8, device=dev))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    some = slice(0, rows, 100)
    check_sample((a[0][some], a[1][some]), x[some], *(v[some] for v in (u, t, k, p, m)))
