// 4-bit weights with a scale (and zero point) per group of K, times 16-bit
// activations:
//   C[m,n] = T(sum_k A[m,k] (c[n,k] - z[n,g]) s[n,g]),  g = k / group,
// codes c in -8..7 packed as by bq_pack_int4 (u = c + 8 = nibble ^ 8), fp32
// sums.  Three kernels by M:
//  * gemv (M <= 4): dot products, a stream over B;
//  * skinny (M <= 64): matrix instructions on the bare codes, K split over a
//    workgroup's wavefronts (and over workgroups with a workspace);
//  * tiled: the weights rounded once to T, through LDS.
// The first two keep scale and zero point outside the sums:
//   sum_g s_g (sum_k a u - (8 + z_g) sum_k a).
#include "bq_internal.h"
#include "dtype16.h"

namespace bq {
namespace {

constexpr uint32_t kFlip = 0x88888888u;  // two's complement nibble -> c + 8

// ---------------------------------------------------------------------------
// gemv
// ---------------------------------------------------------------------------

constexpr int kGemvWaves = 4;

// Eight codes of a dword, as the pairs (0,4) (1,5) (2,6) (3,7).  fp16: pairs
// 0 and 2 hold u 2^-24, 1 and 3 u 2^-20; bf16: 128 + u.
template <typename T>
__device__ __forceinline__ void codes8(uint32_t w, uint32_t p[4])
{
    if constexpr (T::kBf16) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            p[i] = ((w >> (4 * i)) & 0x000f000fu) | 0x43004300u;
    } else {
        const uint32_t h = w >> 8;
        p[0] = w & 0x000f000fu;
        p[1] = w & 0x00f000f0u;
        p[2] = h & 0x000f000fu;
        p[3] = h & 0x00f000f0u;
    }
}

// A wavefront takes ROWS rows of B; its lanes walk them in chunks of 32 codes
// (16 bytes, inside one group), lane l taking chunks l, l + 64, ...
template <typename T, int MR, int ROWS, int U>
__global__ __launch_bounds__(64 * kGemvWaves) void w4g_gemv_kernel(const uint16_t *__restrict__ A, const uint8_t *__restrict__ B,
                                                                   const uint16_t *__restrict__ scale,
                                                                   const uint16_t *__restrict__ zero, int gshift,
                                                                   uint16_t *__restrict__ C, int M, int N, int K)
{
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n0 = (blockIdx.x * kGemvWaves + wave) * ROWS;
    if (n0 >= N)
        return;
    const int chunks = K / 32, groups = K >> gshift;
    float acc[MR][ROWS] = {};
    for (int c0 = 0; c0 < chunks; c0 += 64 * U) {
        uint4 b[ROWS][U];
        uint32_t sz[ROWS][U];
        uint4 a[MR][U][4];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int c = c0 + lane + 64 * u;
            const bool ok = c < chunks;
#pragma unroll
            for (int r = 0; r < ROWS; ++r) {
                const int64_t n = min(n0 + r, N - 1);
                b[r][u] = ok ? load_nt16(B + n * (K / 2) + (int64_t)c * 16) : make_uint4(0, 0, 0, 0);
                const int64_t at = n * groups + (c >> (gshift - 5));
                sz[r][u] = ok ? scale[at] | (zero ? (uint32_t)zero[at] << 16 : 0u) : 0u;
            }
#pragma unroll
            for (int m = 0; m < MR; ++m)
#pragma unroll
                for (int h = 0; h < 4; ++h)
                    a[m][u][h] = ok && m < M ? *(const uint4 *)(A + (int64_t)m * K + (int64_t)c * 32 + 8 * h)
                                             : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float s0[MR][ROWS] = {}, s4[MR][ROWS] = {}, sum[MR] = {};
#pragma unroll
            for (int h = 0; h < 4; ++h) {
                uint32_t p[ROWS][4];
#pragma unroll
                for (int r = 0; r < ROWS; ++r) {
                    const uint32_t w[4] = {b[r][u].x, b[r][u].y, b[r][u].z, b[r][u].w};
                    codes8<T>(w[h] ^ kFlip, p[r]);
                }
#pragma unroll
                for (int m = 0; m < MR; ++m) {
                    const uint4 v = a[m][u][h];
                    const uint32_t q[4] = {pack_lo(v.x, v.z), pack_hi(v.x, v.z), pack_lo(v.y, v.w), pack_hi(v.y, v.w)};
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        sum[m] = T::dot2(q[i], T::kOnes, sum[m]);
#pragma unroll
                    for (int r = 0; r < ROWS; ++r) {
                        s0[m][r] = T::dot2(q[0], p[r][0], s0[m][r]);
                        s4[m][r] = T::dot2(q[1], p[r][1], s4[m][r]);
                        s0[m][r] = T::dot2(q[2], p[r][2], s0[m][r]);
                        s4[m][r] = T::dot2(q[3], p[r][3], s4[m][r]);
                    }
                }
            }
#pragma unroll
            for (int r = 0; r < ROWS; ++r) {
                const float s = half_bits(sz[r][u] & 0xffffu), z = half_bits(sz[r][u] >> 16);
#pragma unroll
                for (int m = 0; m < MR; ++m) {
                    const float dot = T::kBf16 ? s0[m][r] + s4[m][r] : s0[m][r] * 0x1p24f + s4[m][r] * 0x1p20f;
                    acc[m][r] += s * (dot - ((T::kBf16 ? 136.0f : 8.0f) + z) * sum[m]);
                }
            }
        }
    }
#pragma unroll
    for (int m = 0; m < MR; ++m)
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
#pragma unroll
            for (int off = 32; off > 0; off >>= 1)
                acc[m][r] += __shfl_xor(acc[m][r], off, 64);
            if (lane == m * ROWS + r && m < M && n0 + r < N)
                C[(int64_t)m * N + n0 + r] = T::from_f32(acc[m][r]);
        }
}

template <typename T, int MR, int ROWS>
hipError_t launch_gemv_t(const uint16_t *A, const uint8_t *B, const uint16_t *scale, const uint16_t *zero, int gshift,
                         uint16_t *C, int M, int N, int K, hipStream_t s)
{
    const int64_t wgs = ((int64_t)N + ROWS * kGemvWaves - 1) / (ROWS * kGemvWaves);
    if (!grid_fits(wgs, 64 * kGemvWaves))
        return kGridTooLarge;
    w4g_gemv_kernel<T, MR, ROWS, MR == 4 ? 1 : 2><<<dim3((unsigned)wgs), 64 * kGemvWaves, 0, s>>>(A, B, scale, zero, gshift, C,
                                                                                                 M, N, K);
    return hipGetLastError();
}

// ---------------------------------------------------------------------------
// skinny
// ---------------------------------------------------------------------------

// Eight codes of a dword as one matrix operand, pairs (0,4) (1,5) (2,6)
// (3,7): fp16 u 2^-20 (every pair brought to bits 4..7), bf16 128 + u.
template <typename T>
__device__ __forceinline__ u4 codes_op(uint32_t w)
{
    if constexpr (T::kBf16)
        return (u4){(w & 0x000f000fu) | 0x43004300u, ((w >> 4) & 0x000f000fu) | 0x43004300u,
                    ((w >> 8) & 0x000f000fu) | 0x43004300u, ((w >> 12) & 0x000f000fu) | 0x43004300u};
    else
        return (u4){(w << 4) & 0x00f000f0u, w & 0x00f000f0u, (w >> 4) & 0x00f000f0u, (w >> 8) & 0x00f000f0u};
}

// The 4 x 4 dwords of lanes l, l + 16, l + 32, l + 48, transposed.
__device__ __forceinline__ void transpose4(uint32_t w[4])
{
    auto s = __builtin_amdgcn_permlane32_swap(w[0], w[2], false, false);
    w[0] = s[0];
    w[2] = s[1];
    s = __builtin_amdgcn_permlane32_swap(w[1], w[3], false, false);
    w[1] = s[0];
    w[3] = s[1];
    s = __builtin_amdgcn_permlane16_swap(w[0], w[1], false, false);
    w[0] = s[0];
    w[1] = s[1];
    s = __builtin_amdgcn_permlane16_swap(w[2], w[3], false, false);
    w[2] = s[0];
    w[3] = s[1];
}

// NB tiles of 16 weight rows x NA tiles of 16 activation rows a workgroup;
// wavefront w takes the 128-wide steps w, w + WAVES, ... of the workgroup's
// part of K.  A 16-byte load hands lane (n, g) the 32 codes of row n at
// k = 32 g; the transpose makes matrix step j cover k = 32 j .. 32 j + 31,
// which lies in one group.
template <typename T, int NA, int NB, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void w4g_skinny_kernel(const uint16_t *__restrict__ A, const uint8_t *__restrict__ B,
                                                                const uint16_t *__restrict__ scale,
                                                                const uint16_t *__restrict__ zero, int gshift,
                                                                uint16_t *__restrict__ C, float *__restrict__ part, int M,
                                                                int N, int K, int ksplit)
{
    __shared__ float red[WAVES][16][16 * NB + 4];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int g = lane >> 4, l16 = lane & 15;
    const int split = blockIdx.x % ksplit, n0 = blockIdx.x / ksplit * (16 * NB);
    const int steps = (K + 127) / 128, per = (steps + ksplit - 1) / ksplit;
    const int first = split * per, last = min(first + per, steps);
    const int groups = K >> gshift;

    f4 acc[NA][NB], part_acc[NA][NB], sum[NA];
    const f4 zero4 = {0, 0, 0, 0};
#pragma unroll
    for (int a = 0; a < NA; ++a) {
        sum[a] = zero4;
#pragma unroll
        for (int b = 0; b < NB; ++b)
            acc[a][b] = part_acc[a][b] = zero4;
    }
    const u4 ones = {T::kOnes, T::kOnes, T::kOnes, T::kOnes};
    const int gmask = (1 << (gshift - 5)) - 1;  // 32-wide steps in a group, less one
    for (int st = first + wave; st < last; st += WAVES) {
        uint32_t w[NB][4];
        uint32_t sz[NB][4];
        u4 x[NA][4];
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            const int64_t n = min(n0 + 16 * b + l16, N - 1);
            const int k = st * 128 + 32 * g;
            const uint4 v = k < K ? load_nt16(B + n * (K / 2) + k / 2) : make_uint4(0, 0, 0, 0);
            w[b][0] = v.x;
            w[b][1] = v.y;
            w[b][2] = v.z;
            w[b][3] = v.w;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int kk = min(st * 128 + 32 * j, K - 32);
                const int64_t at = n * groups + (kk >> gshift);
                sz[b][j] = scale[at] | (zero ? (uint32_t)zero[at] << 16 : 0u);
            }
        }
#pragma unroll
        for (int a = 0; a < NA; ++a) {
            const int64_t m = min(16 * a + l16, M - 1);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int k = st * 128 + 32 * j + 8 * g;
                x[a][j] = k < K ? *(const u4 *)(A + m * K + k) : (u4){0, 0, 0, 0};
            }
        }
#pragma unroll
        for (int b = 0; b < NB; ++b)
            transpose4(w[b]);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
#pragma unroll
            for (int a = 0; a < NA; ++a) {
                const u4 v = x[a][j];
                x[a][j] = (u4){pack_lo(v.x, v.z), pack_hi(v.x, v.z), pack_lo(v.y, v.w), pack_hi(v.y, v.w)};
                sum[a] = T::mma(x[a][j], ones, sum[a]);
            }
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                const u4 op = codes_op<T>(w[b][j] ^ kFlip);
#pragma unroll
                for (int a = 0; a < NA; ++a)
                    part_acc[a][b] = T::mma(x[a][j], op, part_acc[a][b]);
            }
            if ((j & gmask) == gmask) {  // a group ends
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    const float s = half_bits(sz[b][j] & 0xffffu) * (T::kBf16 ? 1.0f : 0x1p20f);
                    const float z = ((T::kBf16 ? 136.0f : 8.0f) + half_bits(sz[b][j] >> 16)) * (T::kBf16 ? 1.0f : 0x1p-20f);
#pragma unroll
                    for (int a = 0; a < NA; ++a) {
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            acc[a][b][i] += s * (part_acc[a][b][i] - z * sum[a][i]);
                        part_acc[a][b] = zero4;
                    }
                }
#pragma unroll
                for (int a = 0; a < NA; ++a)
                    sum[a] = zero4;
            }
        }
    }
    // join the wavefronts, 16 activation rows at a time
#pragma unroll
    for (int a = 0; a < NA; ++a) {
        if (a)
            __syncthreads();
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                red[wave][4 * g + i][16 * b + l16] = acc[a][b][i];
        __syncthreads();
        for (int e = threadIdx.x; e < 256 * NB; e += 64 * WAVES) {
            const int m = e / (16 * NB), n = e % (16 * NB);
            float v = 0.0f;
#pragma unroll
            for (int q = 0; q < WAVES; ++q)
                v += red[q][m][n];
            if (16 * a + m < M && n0 + n < N) {
                const int64_t at = (int64_t)(16 * a + m) * N + n0 + n;
                if (part)
                    part[(int64_t)split * M * N + at] = v;
                else
                    C[at] = T::from_f32(v);
            }
        }
    }
}

template <typename T>
__global__ __launch_bounds__(256) void w4g_join_kernel(const float *__restrict__ part, uint16_t *__restrict__ C, int64_t total,
                                                       int ksplit)
{
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= total)
        return;
    float v = 0.0f;
    for (int s = 0; s < ksplit; ++s)
        v += part[s * total + i];
    C[i] = T::from_f32(v);
}

// Parts of K for the skinny kernel with a workspace.
int skinny_split(int M, int N, int K)
{
    if (M <= 16)
        return 1;
    const int tiles = (N + 63) / 64, steps = (K + 127) / 128;
    int n = (512 + tiles - 1) / tiles;
    n = n < steps / 4 ? n : steps / 4;
    return n < 1 ? 1 : n > 16 ? 16 : n;
}

template <typename T, int NA, int NB, int WAVES>
hipError_t launch_skinny_t(const uint16_t *A, const uint8_t *B, const uint16_t *scale, const uint16_t *zero, int gshift,
                           uint16_t *C, int M, int N, int K, float *ws, int ksplit, hipStream_t s)
{
    const int64_t wgs = ((int64_t)N + 16 * NB - 1) / (16 * NB) * ksplit;
    const int64_t total = (int64_t)M * N;
    if (!grid_fits(wgs, 64 * WAVES) || !grid_fits((total + 255) / 256, 256))
        return kGridTooLarge;
    w4g_skinny_kernel<T, NA, NB, WAVES><<<dim3((unsigned)wgs), 64 * WAVES, 0, s>>>(
        A, B, scale, zero, gshift, C, ksplit > 1 ? ws : nullptr, M, N, K, ksplit);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || ksplit == 1)
        return e;
    w4g_join_kernel<T><<<dim3((unsigned)((total + 255) / 256)), 256, 0, s>>>(ws, C, total, ksplit);
    return hipGetLastError();
}

// ---------------------------------------------------------------------------
// tiled
// ---------------------------------------------------------------------------

constexpr int kBM = 128, kBN = 128, kBK = 64, kPad = 8;

template <typename T>
__global__ __launch_bounds__(256) void w4g_tiled_kernel(const uint16_t *__restrict__ A, const uint8_t *__restrict__ B,
                                                        const uint16_t *__restrict__ scale, const uint16_t *__restrict__ zero,
                                                        int gshift, uint16_t *__restrict__ C, int M, int N, int K)
{
    __shared__ uint16_t sa[kBM][kBK + kPad], sb[kBN][kBK + kPad];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int g = lane >> 4, l16 = lane & 15;
    const int tilesN = (N + kBN - 1) / kBN;
    const int m0 = blockIdx.x / tilesN * kBM, n0 = blockIdx.x % tilesN * kBN;
    const int wm = (wave >> 1) * 64, wn = (wave & 1) * 64;
    const int groups = K >> gshift;
    f4 acc[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
            acc[i][j] = (f4){0, 0, 0, 0};
    // thread (row, half): 32 codes of a weight row; rows of A in 16-byte pieces
    const int br = threadIdx.x >> 1, bh = threadIdx.x & 1;
    const int64_t bn = min(n0 + br, N - 1);
    for (int k0 = 0; k0 < K; k0 += kBK) {
        const uint4 bw = *(const uint4 *)(B + bn * (K / 2) + k0 / 2 + 16 * bh);
        const int64_t at = bn * groups + ((k0 + 32 * bh) >> gshift);
        const float s = half_bits(scale[at]), off = -(8.0f + (zero ? half_bits(zero[at]) : 0.0f)) * s;
        u4 av[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int e = threadIdx.x + 256 * i;
            av[i] = *(const u4 *)(A + (int64_t)min(m0 + (e >> 3), M - 1) * K + k0 + 8 * (e & 7));
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int e = threadIdx.x + 256 * i;
            *(u4 *)&sa[e >> 3][8 * (e & 7)] = av[i];
        }
        const uint32_t wd[4] = {bw.x, bw.y, bw.z, bw.w};
#pragma unroll
        for (int h = 0; h < 4; ++h) {
            const uint32_t w = wd[h] ^ kFlip;
            u4 y;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float c0 = (float)((w >> (8 * i)) & 15u), c1 = (float)((w >> (8 * i + 4)) & 15u);
                y[i] = T::from_f32(c0 * s + off) | (uint32_t)T::from_f32(c1 * s + off) << 16;
            }
            *(u4 *)&sb[br][32 * bh + 8 * h] = y;
        }
        __syncthreads();
#pragma unroll
        for (int kk = 0; kk < kBK; kk += 32) {
            u4 fa[4], fb[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                fa[i] = *(const u4 *)&sa[wm + 16 * i + l16][kk + 8 * g];
                fb[i] = *(const u4 *)&sb[wn + 16 * i + l16][kk + 8 * g];
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    acc[i][j] = T::mma(fa[i], fb[j], acc[i][j]);
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int m = m0 + wm + 16 * i + 4 * g + r, n = n0 + wn + 16 * j + l16;
                if (m < M && n < N)
                    C[(int64_t)m * N + n] = T::from_f32(acc[i][j][r]);
            }
}

template <typename T>
hipError_t launch_any(const uint16_t *A, const uint8_t *B, const uint16_t *scale, const uint16_t *zero, int gshift,
                      uint16_t *C, int M, int N, int K, float *ws, int64_t wsBytes, hipStream_t s)
{
    if (M == 1)
        return launch_gemv_t<T, 1, 1>(A, B, scale, zero, gshift, C, M, N, K, s);
    if (M == 2)
        return launch_gemv_t<T, 2, 2>(A, B, scale, zero, gshift, C, M, N, K, s);
    if (M <= 4)
        return launch_gemv_t<T, 4, 2>(A, B, scale, zero, gshift, C, M, N, K, s);
    const int64_t need = gemm_w4g_workspace_bytes(M, N, K);
    const int ksplit = need && wsBytes >= need ? skinny_split(M, N, K) : 1;
    if (M <= 16)
        return launch_skinny_t<T, 1, 1, 8>(A, B, scale, zero, gshift, C, M, N, K, ws, 1, s);
    if (M <= 32)
        return launch_skinny_t<T, 2, 4, 4>(A, B, scale, zero, gshift, C, M, N, K, ws, ksplit, s);
    if (M <= 48)
        return launch_skinny_t<T, 3, 4, 4>(A, B, scale, zero, gshift, C, M, N, K, ws, ksplit, s);
    if (M <= 64)
        return launch_skinny_t<T, 4, 4, 4>(A, B, scale, zero, gshift, C, M, N, K, ws, ksplit, s);
    const int64_t wgs = (((int64_t)M + kBM - 1) / kBM) * (((int64_t)N + kBN - 1) / kBN);
    if (!grid_fits(wgs, 256))
        return kGridTooLarge;
    w4g_tiled_kernel<T><<<dim3((unsigned)wgs), 256, 0, s>>>(A, B, scale, zero, gshift, C, M, N, K);
    return hipGetLastError();
}

}  // namespace

int64_t gemm_w4g_workspace_bytes(int M, int N, int K)
{
    if (M <= 16 || M > 64)
        return 0;
    const int n = skinny_split(M, N, K);
    return n > 1 ? (int64_t)n * M * N * 4 : 0;
}

hipError_t launch_gemm_w4g(const uint16_t *A, const uint8_t *B, const uint16_t *scale, const uint16_t *zero, int group,
                           uint16_t *C, int M, int N, int K, bool bf16, float *ws, int64_t wsBytes, hipStream_t s)
{
    const int gshift = group == 32 ? 5 : group == 64 ? 6 : 7;
    return bf16 ? launch_any<BF16>(A, B, scale, zero, gshift, C, M, N, K, ws, wsBytes, s)
                : launch_any<F16>(A, B, scale, zero, gshift, C, M, N, K, ws, wsBytes, s);
}

}  // namespace bq
