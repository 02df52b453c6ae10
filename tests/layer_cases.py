"""Shapes and inputs of the group-scaled product's tests, for the CPU (what
the bound notices) and the GPU (what the kernels give)."""
import torch

from oracle import layer

# M, N, K, group: every kernel and tile, K that ends inside a step, edges
W4G = [(1, 1, 64, 32), (1, 7, 64, 64), (1, 300, 192, 64), (1, 4096, 4096, 128), (2, 33, 128, 32), (2, 1000, 2048, 128),
       (3, 17, 320, 64), (4, 515, 4160, 32), (4, 64, 65536, 128), (5, 16, 128, 128), (8, 100, 320, 64), (16, 1030, 4096, 128),
       (17, 70, 192, 32), (31, 333, 1024, 64), (32, 4096, 4096, 128), (37, 260, 11008, 128), (48, 65, 640, 64),
       (49, 128, 8192, 32), (64, 200, 448, 64), (65, 130, 64, 32), (100, 257, 320, 64), (128, 128, 256, 128),
       (300, 1000, 1152, 128), (513, 140, 4096, 32)]
# few rows over a wide N (four wavefronts a workgroup), at least 160 tiles of
# 128 x 128, at least 256 of 128 x 64 and fewer than 160 of 128 x 128
W4G_WIDE = [(2, 8200, 64, 32), (3, 8209, 320, 64), (4, 8193, 1152, 128)]
W4G_LARGE = [(1500, 1990, 448, 64), (1281, 2049, 64, 32), (2048, 1300, 1152, 128), (130, 10250, 192, 64)]
W4G_TALL = [(260, 5500, 320, 32), (257, 5450, 64, 64), (385, 4097, 1152, 128), (129, 8300, 448, 64)]
W4G_ALL = W4G + W4G_WIDE + W4G_LARGE + W4G_TALL


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def w4g_inputs(M, N, K, group, zero, T, seed=100):
    """A [M, K], packed codes, scales and zero points (not all whole)."""
    g = gen(seed + M + 3 * N + K)
    A = torch.randn(M, K, generator=g).to(T)
    B, s, z = layer.quantize_w4g(torch.randn(N, K, generator=g) * 0.02 + (0.01 if zero else 0), group, zero)
    if zero:
        z = (z.float() + torch.rand(z.shape, generator=g) * 0.5).half()
    return A, B, s, z


def w4g_windows(M, K, T, seed=7):
    """A whose rows are zero but for one 32-wide block, and the blocks: the
    first and the last one among them, calls of few rows several times."""
    g = gen(seed + M + K)
    out = []
    for i in range(max(1, 4 // M)):
        at = torch.randint(0, K // 32, (M,), generator=g)
        if i == 0:
            at[0] = 0
        if i == max(1, 4 // M) - 1:
            at[-1] = K // 32 - 1
        A = torch.zeros(M, K // 32, 32)
        A[torch.arange(M), at] = torch.randn(M, 32, generator=g)
        out.append((A.view(M, K).to(T), at.tolist()))
    return out
