"""The group-scaled product's bound (oracle/layer.py) tells a wrong product
from a right one: mistakes planted in the oracle's own products pass it on no
shape that the GPU tests run (CPU)."""
import pytest
import torch

from layer_cases import W4G_ALL, w4g_inputs, w4g_windows
from oracle import layer

F64 = torch.float64
TYPES = [torch.float16, torch.bfloat16]


def outside(C, S, tol):
    return int(((C - S).abs() > tol).sum())


def product(A, B, s, z, group):
    """A product of the kernels' weights: exact up to 16 rows, else rounded once."""
    W = layer.weights_w4g(B, s, z, group)
    if A.shape[0] > 16:
        W = W.to(torch.float32).to(A.dtype).to(F64)
    return (A.to(F64) @ W.t()).to(torch.float32).to(A.dtype).to(F64)


@pytest.mark.parametrize("shape", W4G_ALL)
@pytest.mark.parametrize("T", TYPES)
@pytest.mark.parametrize("zero", [False, True])
def test_bound_holds_and_notices_mistakes(shape, T, zero):
    M, N, K, group = shape
    A, B, s, z = w4g_inputs(M, N, K, group, zero, T)
    S, tol = layer.w4g_bound(A, B, s, z, group)
    assert outside(product(A, B, s, z, group), S, tol) == 0
    lost = A.clone()
    lost[:, K - 32:] = 0  # the last step of K
    assert outside(product(lost, B, s, z, group), S, tol) > 0, "last 32 of K lost"
    lost = A.clone()
    mid = K // 2 // 64 * 64
    lost[:, mid: mid + 64] = 0
    assert outside(product(lost, B, s, z, group), S, tol) > 0, "64 of K lost"
    if N > 16:
        if K > group:
            assert outside(product(A, B, s.roll(1, 1), z, group), S, tol) > 0, "scales one group off"
        assert outside(product(A, B, s.roll(1, 0), z, group), S, tol) > 0, "scales one row off"
        swapped = (B >> 4) | (B << 4)
        assert outside(product(A, swapped, s, z, group), S, tol) > 0, "nibbles swapped"
        if zero:
            assert outside(product(A, B, s, torch.zeros_like(z), group), S, tol) > 0, "no zero points"


@pytest.mark.parametrize("shape", W4G_ALL)
@pytest.mark.parametrize("T", TYPES)
def test_windows_notice_one_step_or_group(shape, T):
    """Rows that are zero but for 32 k: a step lost, or one group's scale or
    zero point taken from the next group, shows in the row that has it."""
    M, N, K, group = shape
    if N < 16:
        return
    _, B, s, z = w4g_inputs(M, N, K, group, True, T)
    for A, at in w4g_windows(M, K, T):
        S, tol = layer.w4g_bound(A, B, s, z, group)
        assert outside(product(A, B, s, z, group), S, tol) == 0
        for m in sorted({0, M // 2, M - 1}):
            lost = A.clone()
            lost[m] = 0
            assert outside(product(lost, B, s, z, group)[m], S[m], tol[m]) > N // 2
            if K > group:
                for which in (s, z):
                    other = which.clone()
                    g = at[m] * 32 // group
                    other[:, g] = which[:, (g + 1) % (K // group)]
                    C = product(A, B, other if which is s else s, other if which is z else z, group)
                    assert outside(C[m], S[m], tol[m]) > N // 8


@pytest.mark.parametrize("T", TYPES)
def test_round_once(T):
    """One rounding: fp32 values as torch rounds them, and values just beside a
    tie, which fp32 rounds onto it, to their own side."""
    g = torch.Generator()
    g.manual_seed(3)
    x = torch.randn(20000, generator=g, dtype=torch.float32) * 2.0 ** torch.randint(-30, 15, (20000,), generator=g)
    assert torch.equal(layer.round_once(x.to(F64), T), x.to(T).to(F64))
    eps = torch.finfo(T).eps
    tie = 1.0 + eps / 2  # between 1 and 1 + eps; even is 1
    near = torch.tensor([tie + 2.0 ** -40, tie - 2.0 ** -40, -tie - 2.0 ** -40, tie], dtype=F64)
    assert layer.round_once(near, T).tolist() == [1 + eps, 1.0, -1 - eps, 1.0]
    assert near.to(torch.float32).to(T).tolist() == [1.0, 1.0, -1.0, 1.0]
