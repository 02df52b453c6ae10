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

// Loads through a buffer descriptor: an offset at or past its size gives
// zeros, so rows and columns past the ends need no branch.
typedef __amdgpu_buffer_rsrc_t Buf;

__device__ __forceinline__ Buf buffer(const void *base, int64_t bytes)
{
    return __builtin_amdgcn_make_buffer_rsrc((void *)base, (short)0, (int)min(bytes, (int64_t)0x7fffffff), 0x00020000);
}
__device__ __forceinline__ u4 load16(Buf b, uint32_t off)
{
    return __builtin_bit_cast(u4, __builtin_amdgcn_raw_buffer_load_b128(b, off, 0, 0));
}
__device__ __forceinline__ uint16_t load2(Buf b, uint32_t off)
{
    return __builtin_bit_cast(uint16_t, __builtin_amdgcn_raw_buffer_load_b16(b, off, 0, 0));
}
constexpr uint32_t kOut = 0x80000000u;  // past every buffer

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

// A wavefront takes ROWS rows of B and walks them 2048 codes a pass, lane l
// the 32 codes (16 bytes, inside one group) from 32 l on, so a row is read in
// whole kilobytes.  The workgroup puts the pass of A into LDS once, already in
// the codes' pair order and with the sum of every 32 values; piece h of every
// lane's 32 lies in its own plane, so that reads of 16 bytes a lane are
// contiguous (planes padded by 64 bytes for the writes).  B is in flight two
// passes ahead.
constexpr int kPass = 2048, kPlane = 64 * 16 + 64;

template <int ROWS>
struct GemvLoad {
    u4 b[ROWS];
    uint16_t s[ROWS], z[ROWS];
};

template <typename T, int MR, int ROWS>
__global__ __launch_bounds__(64 * kGemvWaves) void w4g_gemv_kernel(const uint16_t *__restrict__ A, const uint8_t *__restrict__ B,
                                                                   const uint16_t *__restrict__ scale,
                                                                   const uint16_t *__restrict__ zero, int gshift,
                                                                   uint16_t *__restrict__ C, int M, int N, int K)
{
    static_assert(64 * kGemvWaves * 8 == kPass, "a 16-byte piece of a row's pass per thread");
    __shared__ __align__(16) uint8_t sa[2][MR][4 * kPlane];
    __shared__ float ssum[2][MR][64];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n0 = (blockIdx.x * kGemvWaves + wave) * ROWS;
    const int groups = K >> gshift;
    const int64_t nb = min(n0, N - 1);  // a wavefront past the end loads nothing and only helps with A
    const int rows = max(min(ROWS, N - n0), 0);
    const Buf ba = buffer(A, (int64_t)M * K * 2), bb = buffer(B + nb * (K / 2), (int64_t)rows * (K / 2));
    const Buf bs = buffer(scale + nb * groups, (int64_t)rows * groups * 2);
    const Buf bz = buffer((zero ? zero : scale) + nb * groups, zero ? (int64_t)rows * groups * 2 : 0);

    const auto load_b = [&](GemvLoad<ROWS> &x, int pass) {
        const int k = pass * kPass + 32 * lane;
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
            x.b[r] = load16(bb, k < K ? r * (K / 2) + k / 2 : kOut);
            const uint32_t at = k < K ? 2 * (r * groups + (k >> gshift)) : kOut;
            x.s[r] = load2(bs, at);
            x.z[r] = load2(bz, at);
        }
    };
    const auto load_a = [&](u4 *x, int pass) {
        const int k = pass * kPass + 8 * (int)threadIdx.x;
#pragma unroll
        for (int m = 0; m < MR; ++m)
            x[m] = load16(ba, k < K ? 2 * (m * K + k) : kOut);
    };
    const auto put_a = [&](const u4 *x, int buf) {
#pragma unroll
        for (int m = 0; m < MR; ++m) {
            const u4 v = {pack_lo(x[m].x, x[m].z), pack_hi(x[m].x, x[m].z), pack_lo(x[m].y, x[m].w), pack_hi(x[m].y, x[m].w)};
            *(u4 *)&sa[buf][m][(threadIdx.x & 3) * kPlane + (threadIdx.x >> 2) * 16] = v;
            float s = T::dot2(v.x, T::kOnes, T::dot2(v.y, T::kOnes, T::dot2(v.z, T::kOnes, T::dot2(v.w, T::kOnes, 0.0f))));
            s += __shfl_xor(s, 1, 64);
            s += __shfl_xor(s, 2, 64);
            if ((threadIdx.x & 3) == 0)
                ssum[buf][m][threadIdx.x >> 2] = s;
        }
    };

    float acc[MR][ROWS] = {};
    const auto compute = [&](const GemvLoad<ROWS> &x, int buf) {
        float s0[MR][ROWS] = {}, s4[MR][ROWS] = {};
#pragma unroll
        for (int h = 0; h < 4; ++h) {
            uint32_t p[ROWS][4];
#pragma unroll
            for (int r = 0; r < ROWS; ++r)
                codes8<T>(x.b[r][h] ^ kFlip, p[r]);
#pragma unroll
            for (int m = 0; m < MR; ++m) {
                const u4 q = *(const u4 *)&sa[buf][m][h * kPlane + lane * 16];
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
        for (int m = 0; m < MR; ++m) {
            const float sum = ssum[buf][m][lane];
#pragma unroll
            for (int r = 0; r < ROWS; ++r) {
                const float s = half_bits(x.s[r]), z = half_bits(x.z[r]);
                const float dot = T::kBf16 ? s0[m][r] + s4[m][r] : s0[m][r] * 0x1p24f + s4[m][r] * 0x1p20f;
                acc[m][r] += s * (dot - ((T::kBf16 ? 136.0f : 8.0f) + z) * sum);
            }
        }
    };

    const int passes = (K + kPass - 1) / kPass;
    if (passes > 0) {
        GemvLoad<ROWS> x, y;
        u4 av[MR];
        load_b(x, 0);
        load_a(av, 0);
        load_b(y, 1);  // past the end: zeros, no access
        put_a(av, 0);
        __syncthreads();
        for (int p = 0; p < passes; ++p) {
            load_a(av, p + 1);
            compute(x, p & 1);
            x = y;
            load_b(y, p + 2);
            put_a(av, (p + 1) & 1);
            __syncthreads();
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
    w4g_gemv_kernel<T, MR, ROWS><<<dim3((unsigned)wgs), 64 * kGemvWaves, 0, s>>>(A, B, scale, zero, gshift, C, M, N, K);
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

// What a wavefront loads for one 128-wide step.
template <int NA, int NB>
struct Step {
    u4 w[NB];
    uint16_t s[NB], z[NB];
    u4 a[NA][4];
};

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
    // B and its parameters from the workgroup's first row on, A whole
    const int rows = min(16 * NB, N - n0);
    const Buf ba = buffer(A, (int64_t)M * K * 2), bb = buffer(B + (int64_t)n0 * (K / 2), (int64_t)rows * (K / 2));
    const Buf bs = buffer(scale + (int64_t)n0 * groups, (int64_t)rows * groups * 2);
    const Buf bz = buffer((zero ? zero : scale) + (int64_t)n0 * groups, zero ? (int64_t)rows * groups * 2 : 0);
    const auto load = [&](Step<NA, NB> &x, int st) {
        const int k = st * 128 + 32 * g;
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            const uint32_t n = 16 * b + l16;
            x.w[b] = load16(bb, k < K ? n * (K / 2) + k / 2 : kOut);
            // scale and zero point of the lane's own 32 codes
            const uint32_t at = k < K ? 2 * (n * groups + (k >> gshift)) : kOut;
            x.s[b] = load2(bs, at);
            x.z[b] = load2(bz, at);
        }
#pragma unroll
        for (int a = 0; a < NA; ++a)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int ka = st * 128 + 32 * j + 8 * g;
                x.a[a][j] = load16(ba, ka < K ? 2 * ((16 * a + l16) * K + ka) : kOut);
            }
    };
    const auto step = [&](const Step<NA, NB> &x) {
        uint32_t w[NB][4];
#pragma unroll
        for (int b = 0; b < NB; ++b) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                w[b][j] = x.w[b][j];
            transpose4(w[b]);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            u4 q[NA];
#pragma unroll
            for (int a = 0; a < NA; ++a) {
                const u4 v = x.a[a][j];
                q[a] = (u4){pack_lo(v.x, v.z), pack_hi(v.x, v.z), pack_lo(v.y, v.w), pack_hi(v.y, v.w)};
                sum[a] = T::mma(q[a], ones, sum[a]);
            }
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                const u4 op = codes_op<T>(w[b][j] ^ kFlip);
#pragma unroll
                for (int a = 0; a < NA; ++a)
                    part_acc[a][b] = T::mma(q[a], op, part_acc[a][b]);
            }
            if ((j & gmask) == gmask) {  // a group ends
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    // held by the lane whose codes are this group's
                    uint32_t sz = x.s[b] | (uint32_t)x.z[b] << 16;
                    if (gmask != 3)
                        sz = __shfl(sz, l16 + 16 * j, 64);
                    const float s = half_bits(sz & 0xffffu) * (T::kBf16 ? 1.0f : 0x1p20f);
                    const float z = ((T::kBf16 ? 136.0f : 8.0f) + half_bits(sz >> 16)) * (T::kBf16 ? 1.0f : 0x1p-20f);
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
    };
    // Workgroups start at different places of K and go round: in step, all
    // would read one 64-byte column of rows K/2 bytes apart, which meet in a
    // few memory channels.
    const int n = last - first;
    int i = wave, st = n > 0 ? wave + (int)(blockIdx.x / ksplit) % n : 0;
    if (i < n) {
        if (st >= n)
            st -= n;
        // the next step's loads are in flight during a step's arithmetic
        Step<NA, NB> x;
        load(x, first + st);
        for (; i + WAVES < n; i += WAVES) {
            st += WAVES;
            if (st >= n)
                st -= n;
            Step<NA, NB> y;
            load(y, first + st);
            step(x);
            x = y;
        }
        step(x);
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
