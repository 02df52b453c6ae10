// 4-bit weights with a scale (and zero point) per group of K, times 16-bit
// activations:
//   C[m,n] = T(sum_k A[m,k] (c[n,k] - z[n,g]) s[n,g]),  g = k / group,
// codes c in -8..7 packed as by bq_pack_int4 (u = c + 8 = nibble ^ 8), fp32
// sums.  Three kernels by M:
//  * gemv (M = 1): dot products, a stream over B;
//  * skinny (M <= 16): matrix instructions on the bare codes, K split over a
//    workgroup's wavefronts;
//  * tiled: the weights rounded once to T between LDS and the matrix
//    instructions, K in parts over workgroups where tiles are few.  A choice:
//    the rounding is as large as the output's own, so the error against 64 bits
//    is 1.35 times it (bf16 2.3e-3 for 1.7e-3, fp16 2.8e-4 for 2.1e-4); bare
//    codes would take the scale to every accumulator at the end of each group,
//    32 to 128 k, in the issue slots that bound this kernel.
// The first two keep scale and zero point outside the sums:
//   sum_g s_g (sum_k a u - (8 + z_g) sum_k a).
#include "bq_layer_internal.h"
#include "dtype16.h"
#include "lds_dma.h"

namespace bq {
namespace {

// M up to which the skinny kernel is taken: 16 weight rows a workgroup and all
// of A's (M = 16, N = K = 4096, fp16: 6.8 us, tiled 12.3; bf16 with zero points
// 7.9, 17.2).
constexpr int kSkinnyM = 16;

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

// One row of A.  A wavefront takes a row of B and walks it 2048 codes a pass,
// lane l the 32 codes (16 bytes, inside one group) from 32 l on, so a row is
// read in whole kilobytes.  The workgroup puts the pass of A into LDS once,
// already in the codes' pair order and with the sum of every 32 values; piece
// h of every lane's 32 lies in its own plane, so that reads of 16 bytes a lane
// are contiguous (planes padded by 64 bytes for the writes).  B is in flight
// two passes ahead.
constexpr int kPass = 2048, kPlane = 64 * 16 + 64;

struct GemvLoad {
    u4 b;
    uint16_t s, z;
};

template <typename T>
__global__ __launch_bounds__(64 * kGemvWaves) void w4g_gemv_kernel(const uint16_t *__restrict__ A, const uint8_t *__restrict__ B,
                                                                   const uint16_t *__restrict__ scale,
                                                                   const uint16_t *__restrict__ zero, int gshift,
                                                                   uint16_t *__restrict__ C, int N, int K)
{
    static_assert(64 * kGemvWaves * 8 == kPass, "a 16-byte piece of the pass per thread");
    __shared__ __align__(16) uint8_t sa[2][4 * kPlane];
    __shared__ float ssum[2][64];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t n = (int64_t)blockIdx.x * kGemvWaves + wave;
    const int groups = K >> gshift;
    const bool in = n < N;  // a wavefront past the end loads nothing and only helps with A
    const int64_t nb = in ? n : 0;
    const Buf ba = buffer(A, (int64_t)K * 2), bb = buffer(B + nb * (K / 2), in ? K / 2 : 0);
    const Buf bs = buffer(scale + nb * groups, in ? (int64_t)groups * 2 : 0);
    const Buf bz = buffer((zero ? zero : scale) + nb * groups, in && zero ? (int64_t)groups * 2 : 0);

    const auto load_b = [&](GemvLoad &x, int pass) {
        const int k = pass * kPass + 32 * lane;
        x.b = load16(bb, k < K ? k / 2 : kOut);
        const uint32_t at = k < K ? 2 * (k >> gshift) : kOut;
        x.s = load2(bs, at);
        x.z = load2(bz, at);
    };
    const auto load_a = [&](int pass) {
        const int k = pass * kPass + 8 * (int)threadIdx.x;
        return load16(ba, k < K ? 2 * k : kOut);
    };
    const auto put_a = [&](const u4 x, int buf) {
        const u4 v = {pack_lo(x.x, x.z), pack_hi(x.x, x.z), pack_lo(x.y, x.w), pack_hi(x.y, x.w)};
        *(u4 *)&sa[buf][(threadIdx.x & 3) * kPlane + (threadIdx.x >> 2) * 16] = v;
        float s = T::dot2(v.x, T::kOnes, T::dot2(v.y, T::kOnes, T::dot2(v.z, T::kOnes, T::dot2(v.w, T::kOnes, 0.0f))));
        s += __shfl_xor(s, 1, 64);
        s += __shfl_xor(s, 2, 64);
        if ((threadIdx.x & 3) == 0)
            ssum[buf][threadIdx.x >> 2] = s;
    };

    float acc = 0.0f;
    const auto compute = [&](const GemvLoad &x, int buf) {
        float s0 = 0.0f, s4 = 0.0f;
#pragma unroll
        for (int h = 0; h < 4; ++h) {
            uint32_t p[4];
            codes8<T>(x.b[h] ^ kFlip, p);
            const u4 q = *(const u4 *)&sa[buf][h * kPlane + lane * 16];
            s0 = T::dot2(q[0], p[0], s0);
            s4 = T::dot2(q[1], p[1], s4);
            s0 = T::dot2(q[2], p[2], s0);
            s4 = T::dot2(q[3], p[3], s4);
        }
        const float s = half_bits(x.s), z = half_bits(x.z);
        const float dot = T::kBf16 ? s0 + s4 : s0 * 0x1p24f + s4 * 0x1p20f;
        acc += s * (dot - ((T::kBf16 ? 136.0f : 8.0f) + z) * ssum[buf][lane]);
    };

    const int passes = (K + kPass - 1) / kPass;
    if (passes > 0) {
        GemvLoad x, y;
        load_b(x, 0);
        u4 av = load_a(0);
        load_b(y, 1);  // past the end: zeros, no access
        put_a(av, 0);
        __syncthreads();
        for (int p = 0; p < passes; ++p) {
            av = load_a(p + 1);
            compute(x, p & 1);
            x = y;
            load_b(y, p + 2);
            put_a(av, (p + 1) & 1);
            __syncthreads();
        }
    }
#pragma unroll
    for (int off = 32; off > 0; off >>= 1)
        acc += __shfl_xor(acc, off, 64);
    if (lane == 0 && in)
        C[n] = T::from_f32(acc);
}

template <typename T>
hipError_t launch_gemv_t(const uint16_t *A, const uint8_t *B, const uint16_t *scale, const uint16_t *zero, int gshift,
                         uint16_t *C, int N, int K, hipStream_t s)
{
    const int64_t wgs = ((int64_t)N + kGemvWaves - 1) / kGemvWaves;
    if (!grid_fits(wgs, 64 * kGemvWaves))
        return kGridTooLarge;
    w4g_gemv_kernel<T><<<dim3((unsigned)wgs), 64 * kGemvWaves, 0, s>>>(A, B, scale, zero, gshift, C, N, K);
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

// What a wavefront loads for CH steps of 128.
template <int NL, int CH>
struct Steps {
    u4 w[CH], a[CH][NL];
    uint16_t s[CH], z[CH];  // four groups each, one a quarter of the lanes
};

__device__ __forceinline__ void wave_sync()
{
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// 16 weight rows x up to 4 NL activation rows a workgroup, whose wavefronts
// take neighbouring parts of its K in steps of 128, CH steps' loads at a time
// and the next CH in flight.
//  * A 16-byte load hands lane (n, g) the 32 codes of row n at k = 32 g; the
//    transpose makes matrix step j cover k = 32 j .. 32 j + 31, which lies in
//    one group.
//  * A is loaded in whole 256-byte pieces of rows, as many loads as there are
//    four rows, and goes through a part of LDS of the wavefront's own into the
//    codes' pair order: operand loads straight from memory, 64 bytes of 16
//    rows each, took longer than the codes (M = 8, N = 12288, K = 4096: 16.9
//    us, without them 10.2).  Pieces are permuted by the row's number: the 16
//    rows of an operand read fall into different banks.
//  * Scales and zero points come four groups of a row a load and are handed to
//    the lanes of their row when the group ends.
template <typename T, int NL, int WAVES, int CH>
__global__ __launch_bounds__(64 * WAVES) void w4g_skinny_kernel(const uint16_t *__restrict__ A, const uint8_t *__restrict__ B,
                                                                const uint16_t *__restrict__ scale,
                                                                const uint16_t *__restrict__ zero, int gshift,
                                                                uint16_t *__restrict__ C, int M, int N, int K)
{
    constexpr int kLoaded = 4 * NL;
    static_assert(kLoaded <= 16, "rows of A");
    __shared__ __align__(16) union {
        uint8_t a[WAVES][kLoaded][256];
        float red[WAVES][16][20];
    } sh;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int g = lane >> 4, l16 = lane & 15;
    const int n0 = blockIdx.x * 16;
    const int steps = (K + 127) / 128, per = (steps + WAVES - 1) / WAVES;
    const int first = wave * per, last = min(first + per, steps);
    const int groups = K >> gshift;
    const int sshift = 7 - gshift;  // groups of a step, as a shift

    const f4 zero4 = {0, 0, 0, 0};
    f4 acc = zero4, part_acc = zero4, sum = zero4;
    const u4 ones = {T::kOnes, T::kOnes, T::kOnes, T::kOnes};
    const int gmask = (1 << (gshift - 5)) - 1;  // 32-wide steps in a group, less one
    // B and its parameters from the workgroup's first row on, A whole
    const int rows = min(16, N - n0);
    const Buf ba = buffer(A, (int64_t)M * K * 2), bb = buffer(B + (int64_t)n0 * (K / 2), (int64_t)rows * (K / 2));
    const Buf bs = buffer(scale + (int64_t)n0 * groups, (int64_t)rows * groups * 2);
    const Buf bz = buffer((zero ? zero : scale) + (int64_t)n0 * groups, zero ? (int64_t)rows * groups * 2 : 0);
    const auto load = [&](Steps<NL, CH> &x, int c0) {
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int st = c0 + c, k = st * 128 + 32 * g, ka = st * 128 + 8 * l16;
            x.w[c] = load16(bb, st < last && k < K ? l16 * (K / 2) + k / 2 : kOut);
            // quarter g: group 4 c + g of the CH steps
            const int gi = (c0 << sshift) + 4 * c + g;
            const uint32_t at = c < (CH << sshift) / 4 + (CH < 4) && gi < groups ? 2 * (l16 * groups + gi) : kOut;
            x.s[c] = load2(bs, at);
            x.z[c] = load2(bz, at);
#pragma unroll
            for (int i = 0; i < NL; ++i)
                x.a[c][i] = load16(ba, st < last && ka < K ? 2 * ((4 * i + g) * K + ka) : kOut);
        }
    };
    uint8_t(*const sa)[256] = sh.a[wave];
    const auto step = [&](const Steps<NL, CH> &x, int c) {
#pragma unroll
        for (int i = 0; i < NL; ++i) {
            const int row = 4 * i + g;
            const u4 v = x.a[c][i];
            *(u4 *)&sa[row][16 * (l16 ^ (row & 15))] =
                (u4){pack_lo(v.x, v.z), pack_hi(v.x, v.z), pack_lo(v.y, v.w), pack_hi(v.y, v.w)};
        }
        wave_sync();
        uint32_t w[4] = {x.w[c].x, x.w[c].y, x.w[c].z, x.w[c].w};
        transpose4(w);
        const int row = l16 % kLoaded;  // rows past the loaded ones give outputs that are not written
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const u4 q = *(const u4 *)&sa[row][16 * ((4 * j + g) ^ row)];
            sum = T::mma(q, ones, sum);
            part_acc = T::mma(q, codes_op<T>(w[j] ^ kFlip), part_acc);
            if ((j & gmask) == gmask) {  // a group ends
                const int gi = (c << sshift) + (j >> (2 - sshift));  // of the CH steps
                uint32_t sz = 0;
#pragma unroll
                for (int i = 0; i < CH; ++i)
                    if (gi >> 2 == i)
                        sz = x.s[i] | (uint32_t)x.z[i] << 16;
                sz = __shfl(sz, l16 + 16 * (gi & 3), 64);
                const float s = half_bits(sz & 0xffffu) * (T::kBf16 ? 1.0f : 0x1p20f);
                const float z = ((T::kBf16 ? 136.0f : 8.0f) + half_bits(sz >> 16)) * (T::kBf16 ? 1.0f : 0x1p-20f);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    acc[i] += s * (part_acc[i] - z * sum[i]);
                part_acc = sum = zero4;
            }
        }
        wave_sync();
    };
    if (first < last) {
        Steps<NL, CH> x, y;
        load(x, first);
        for (int c0 = first; c0 < last; c0 += CH) {
            if (c0 + CH < last)
                load(y, c0 + CH);
#pragma unroll
            for (int c = 0; c < CH; ++c)
                if (c0 + c < last)
                    step(x, c);
            x = y;
        }
    }
    __syncthreads();
    // join the wavefronts
#pragma unroll
    for (int i = 0; i < 4; ++i)
        sh.red[wave][4 * g + i][l16] = acc[i];
    __syncthreads();
    for (int e = threadIdx.x; e < 256; e += 64 * WAVES) {
        const int m = e >> 4, n = e & 15;
        float v = 0.0f;
#pragma unroll
        for (int q = 0; q < WAVES; ++q)
            v += sh.red[q][m][n];
        if (m < M && n0 + n < N)
            C[(int64_t)m * N + n0 + n] = T::from_f32(v);
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

template <typename T, int NL, int WAVES, int CH>
hipError_t launch_skinny_t(const uint16_t *A, const uint8_t *B, const uint16_t *scale, const uint16_t *zero, int gshift,
                           uint16_t *C, int M, int N, int K, hipStream_t s)
{
    const int64_t wgs = ((int64_t)N + 15) / 16;
    if (!grid_fits(wgs, 64 * WAVES))
        return kGridTooLarge;
    w4g_skinny_kernel<T, NL, WAVES, CH><<<dim3((unsigned)wgs), 64 * WAVES, 0, s>>>(A, B, scale, zero, gshift, C, M, N, K);
    return hipGetLastError();
}

// ---------------------------------------------------------------------------
// tiled
// ---------------------------------------------------------------------------

// The eight codes of a dword (two's complement nibbles) times scale, in
// order, each weight rounded once to T.  A byte in both halves, masked to its
// low and high nibble, is with these exponent bits (and the sign bits turned)
// 1024 + u and 1024 + 16 u as fp16; one packed multiply-add makes both the
// integer u - 8.  Without zero points fp16 takes the product there; else
// (u - 8) s - z s goes through fp32.  Mask and bits are held in registers,
// which lets both be one instruction.
struct NibbleBits {
    uint32_t mask = 0x00f0000fu, bits = 0x64806408u;
    __device__ __forceinline__ void hold() { asm volatile("" : "+s"(mask), "+v"(bits)); }
};

template <typename T>
__device__ __forceinline__ u4 weights8(uint32_t w, const NibbleBits &k, bool plain, uint32_t s2, float s, float off)
{
    const h2 mul = {(_Float16)1.0f, (_Float16)0.0625f}, add = {(_Float16)-1032.0f, (_Float16)-72.0f};
    u4 y;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t b = __builtin_amdgcn_perm(0u, w, 0x0c000c00u | (uint32_t)i << 16 | (uint32_t)i);
        const h2 u = __builtin_elementwise_fma(__builtin_bit_cast(h2, (b & k.mask) ^ k.bits), mul, add);
        if (!T::kBf16 && plain) {
            y[i] = __builtin_bit_cast(uint32_t, u * __builtin_bit_cast(h2, s2));
        } else {
            const float a = (float)u[0] * s + off, c = (float)u[1] * s + off;
            y[i] = T::from_f32(a) | (uint32_t)T::from_f32(c) << 16;
        }
    }
    return y;
}

// Permutation of the eight 16-byte pieces of LDS row r, for 16-byte reads of
// 16 rows by lanes (l, g) with piece 2 g + h.  The hardware serves lanes {0-3,
// 12-15, 20-27} and {4-11, 16-19, 28-31} (and the same + 32) together, from 64
// banks of four bytes: rows 0-3, 12-15 of one g with rows 4-11 of the next,
// whose pieces differ in bit 1.  Rows of the first set take even pieces, of
// the second odd ones, and differ among themselves in the other two bits.
__device__ __forceinline__ int swizzle(int r)
{
    const int q = r >> 1;
    return ((q >> 1 ^ q >> 2) & 1) | (q & 1) << 1 | (q & 4);
}

constexpr int kBK = 64;

// Two bytes a lane straight to LDS, as a dword at lds_addr + 4 lane.
__device__ __forceinline__ void dma2(v4si rsrc, uint32_t lds_addr, uint32_t voff)
{
    asm volatile("buffer_load_ushort %0, %1, 0 offen lds" ::"v"(voff), "s"(rsrc), "{m0}"(lds_addr) : "memory");
}

// BM x BN outputs a workgroup, KW teams of four wavefronts.  A team's
// wavefronts lie side by side, each with all BM rows of A and BN/4 weight rows,
// so that a code is decoded once; the teams take turns at the 64-wide steps of
// K, and their sums are added at the end.  A stage of KW steps goes through
// one of three LDS buffers that loads fill without registers, two stages
// ahead.  A row's codes and parameters of a stage are loaded together: each
// cache line that a load touches costs the same, whether 32 bytes of it are
// taken or 128, and with a step's codes, scales and zeros loaded by themselves
// those lines were what bounded the kernel.  Codes stay packed in LDS and
// become operands in registers (weights8) between the matrix instructions.
// The 16-byte pieces of LDS rows are permuted by the row's number, so that
// operand reads fall into different banks.  A lane takes k = 16 g .. 16 g + 15
// of a step, its codes being one 8-byte read.
template <typename T, int BM, int BN, int KW, bool ZERO>
__global__ __launch_bounds__(256 * KW, 1) void w4g_tiled_kernel(const uint16_t *__restrict__ A, const uint8_t *__restrict__ B,
                                                                const uint16_t *__restrict__ scale,
                                                                const uint16_t *__restrict__ zero, int gshift,
                                                                uint16_t *__restrict__ C, float *__restrict__ part, int M,
                                                                int N, int K, int ksplit)
{
    constexpr int STAGES = 3, kSpan = kBK * KW;
    constexpr int FM = BM / 16, FN = BN / 64;
    constexpr int kA = BM / 32;                  // loads of A a wavefront and stage
    constexpr int nB = BN * KW / 32;             // loads of codes a stage, and of scales, and of zeros
    constexpr bool kShare = nB < 4 * KW;         // half the wavefronts load codes, half scales
    constexpr int kLoads = kA + (kShare ? 1 : 2) + (ZERO ? 1 : 0);
    constexpr int kPieces = 2 * KW, kTurn = KW == 4 ? 1 : 2;  // 16-byte pieces of a row of codes; rows of 256 bytes, as a shift
    constexpr int oB = KW * BM * 128, oS = oB + nB * 1024, oZ = oS + nB * 256, kStage = oZ + (ZERO ? nB * 256 : 0);
    constexpr int kSchedMfma = 8, kSchedValu = 2, kSchedDsRead = 0x100, kValu = (T::kBf16 || ZERO ? 24 : 16) / FM + 1;
    static_assert(BM % 32 == 0 && (KW == 2 || KW == 4) && (nB == 4 * KW || nB == 2 * KW), "whole loads");
    __shared__ __align__(1024) uint8_t lds[STAGES * kStage];
    const int lane = threadIdx.x & 63;
    const int wid = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), team = wid >> 2, wave = wid & 3;
    const int g = lane >> 4, l16 = lane & 15;
    const int tilesM = (M + BM - 1) / BM;
    // neighbouring workgroups share weight rows: a die's L2 then reads them once
    const int split = blockIdx.x % ksplit, tile = blockIdx.x / ksplit;
    const int m0 = tile % tilesM * BM, n0 = tile / tilesM * BN;
    const int groups = K >> gshift, spans = (K + kSpan - 1) / kSpan, per = (spans + ksplit - 1) / ksplit;
    const int first = split * per, last = min(first + per, spans);
    const int mrows = min(BM, M - m0), nrows = min(BN, N - n0);
    const v4si ra = make_rsrc(A + (int64_t)m0 * K, (uint32_t)mrows * K * 2);
    const v4si rb = make_rsrc(B + (int64_t)n0 * (K / 2), (uint32_t)nrows * (K / 2));
    const v4si rs = make_rsrc(scale + (int64_t)n0 * groups, (uint32_t)nrows * groups * 2);
    const v4si rz = make_rsrc((ZERO ? zero : scale) + (int64_t)n0 * groups, (uint32_t)nrows * groups * 2);
    const uint32_t base = lds_addr(lds);

    const auto load = [&](int st, int slot) {
        const uint32_t to = base + slot * kStage;
        const bool in = st < last;  // past the end: zeros, no access
        const int k0 = st * kSpan;
#pragma unroll
        for (int i = 0; i < kA; ++i) {
            const int at = wave * kA + i, row = at * 8 + (lane >> 3), piece = (lane & 7) ^ swizzle(row & 15);
            const int k = k0 + team * kBK + 8 * piece;
            dma16(ra, to + (team * BM * 128 + at * 1024), in && k < K ? (uint32_t)(2 * (row * K + k)) : kOOB, 0);
        }
        const int at = wid % nB;
        if (!kShare || wid < nB) {
            const int row = at * (64 / kPieces) + lane / kPieces, piece = (lane % kPieces) ^ (row >> kTurn & (kPieces - 1));
            const int k = k0 + 32 * piece;
            dma16(rb, to + (oB + at * 1024), in && k < K ? (uint32_t)(row * (K / 2) + k / 2) : kOOB, 0);
        }
        // a row's groups at every 32nd k of the stage
        const int row = at * (64 / kPieces) + lane / kPieces, k = k0 + 32 * (lane % kPieces);
        const uint32_t par = in && k < K ? 2u * (row * groups + (k >> gshift)) : kOOB;
        if (!kShare || wid >= nB)
            dma2(rs, to + (oS + at * 256), par);
        if constexpr (ZERO)
            dma2(rz, to + (oZ + at * 256), par);
    };

    f4 acc[FM][FN];
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j)
            acc[i][j] = (f4){0, 0, 0, 0};
    load(first, 0);
    load(first + 1, 1);
    const int wn = wave * (16 * FN);
    NibbleBits nibbles;
    nibbles.hold();
    const auto step = [&](int st, int slot) {
        // this wavefront's loads of the stage are there, then everyone's; and
        // everyone is done with the buffer that is filled next
        asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(kLoads) : "memory");
        load(st + 2, (slot + 2) % STAGES);
        const uint8_t *buf = lds + slot * kStage;
        uint2 w[FN];
        uint32_t s16[FN], z16[FN];
        u4 fa[2][FM], fb[2][FN];
#pragma unroll
        for (int j = 0; j < FN; ++j) {
            const int row = wn + 16 * j + l16;
            const int piece = 2 * team + (g >> 1);
            w[j] = *(const uint2 *)(buf + oB + row * (16 * kPieces) + 16 * (piece ^ (row >> kTurn & (kPieces - 1))) + 8 * (g & 1));
            s16[j] = *(const uint32_t *)(buf + oS + (row * kPieces + piece) * 4);
            z16[j] = ZERO ? *(const uint32_t *)(buf + oZ + (row * kPieces + piece) * 4) : 0u;
        }
        const auto read_a = [&](int h) {
#pragma unroll
            for (int i = 0; i < FM; ++i)
                fa[h][i] = *(const u4 *)(buf + team * BM * 128 + (16 * i + l16) * 128 + 16 * ((2 * g + h) ^ swizzle(l16)));
        };
        const auto decode = [&](int h) {
#pragma unroll
            for (int j = 0; j < FN; ++j) {
                const float s = half_bits(s16[j]), off = -half_bits(z16[j]) * s;
                fb[h][j] = weights8<T>(h ? w[j].y : w[j].x, nibbles, !ZERO, s16[j] | s16[j] << 16, s, off);
            }
        };
        const auto products = [&](int h) {
#pragma unroll
            for (int i = 0; i < FM; ++i)
#pragma unroll
                for (int j = 0; j < FN; ++j)
                    acc[i][j] = T::mma(fb[h][j], fa[h][i], acc[i][j]);
        };
        read_a(0);
        decode(0);
        __builtin_amdgcn_sched_barrier(0);
        // the second half's reads and decode go between the first half's products
        read_a(1);
        decode(1);
        products(0);
#pragma unroll
        for (int i = 0; i < FM * FN; ++i) {
            __builtin_amdgcn_sched_group_barrier(kSchedMfma, 1, 0);
            __builtin_amdgcn_sched_group_barrier(kSchedValu, kValu, 0);
            __builtin_amdgcn_sched_group_barrier(kSchedDsRead, 1, 0);
        }
        __builtin_amdgcn_sched_barrier(0);
        products(1);
    };
    for (int st = first; st < last; st += STAGES) {
#pragma unroll
        for (int s = 0; s < STAGES; ++s)
            if (st + s < last)
                step(st + s, s);
    }
    // no load may still be on its way to LDS when the workgroup ends
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    // the teams' sums, in order
    static_assert(STAGES * kStage >= (KW - 1) * BM * BN * 4, "room for the sums");
    f4 *const sums = (f4 *)lds;
    if (team) {
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
            for (int j = 0; j < FN; ++j)
                sums[(((team - 1) * FM + i) * FN + j) * 256 + (threadIdx.x & 255)] = acc[i][j];
    }
    __syncthreads();
    if (team)
        return;
#pragma unroll
    for (int k = 0; k < KW - 1; ++k)
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
            for (int j = 0; j < FN; ++j)
                acc[i][j] += sums[((k * FM + i) * FN + j) * 256 + threadIdx.x];
    // a lane holds four neighbouring columns of one row
#pragma unroll
    for (int i = 0; i < FM; ++i) {
        const int m = m0 + 16 * i + l16;
#pragma unroll
        for (int j = 0; j < FN; ++j) {
            const int n = n0 + wn + 16 * j + 4 * g;
            if (part) {
                float *to = part + ((int64_t)split * M + m) * N + n;
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    if (m < M && n + r < N)
                        to[r] = acc[i][j][r];
                continue;
            }
            uint16_t *dst = C + (int64_t)m * N + n;
            uint32_t y[2] = {T::from_f32(acc[i][j][0]) | (uint32_t)T::from_f32(acc[i][j][1]) << 16,
                             T::from_f32(acc[i][j][2]) | (uint32_t)T::from_f32(acc[i][j][3]) << 16};
            if (m < M) {
                if (n + 4 <= N && N % 4 == 0) {
                    *(u2 *)dst = (u2){y[0], y[1]};
                } else {
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        if (n + r < N)
                            dst[r] = (uint16_t)(y[r >> 1] >> (16 * (r & 1)));
                }
            }
        }
    }
}

template <typename T, int BM, int BN, int KW>
hipError_t launch_tiled_t(const uint16_t *A, const uint8_t *B, const uint16_t *scale, const uint16_t *zero, int gshift,
                          uint16_t *C, int M, int N, int K, float *ws, int ksplit, hipStream_t s)
{
    const int64_t wgs = (((int64_t)M + BM - 1) / BM) * (((int64_t)N + BN - 1) / BN) * ksplit;
    const int64_t total = (int64_t)M * N;
    if (!grid_fits(wgs, 256 * KW) || (ksplit > 1 && !grid_fits((total + 255) / 256, 256)))
        return kGridTooLarge;
    const dim3 grid((unsigned)wgs);
    float *part = ksplit > 1 ? ws : nullptr;
    if (zero)
        w4g_tiled_kernel<T, BM, BN, KW, true><<<grid, 256 * KW, 0, s>>>(A, B, scale, zero, gshift, C, part, M, N, K, ksplit);
    else
        w4g_tiled_kernel<T, BM, BN, KW, false><<<grid, 256 * KW, 0, s>>>(A, B, scale, zero, gshift, C, part, M, N, K, ksplit);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || ksplit == 1)
        return e;
    w4g_join_kernel<T><<<dim3((unsigned)((total + 255) / 256)), 256, 0, s>>>(ws, C, total, ksplit);
    return hipGetLastError();
}

// Tiles of BM x BN outputs.
int64_t tiles_of(int M, int N, int BM, int BN) { return (((int64_t)M + BM - 1) / BM) * (((int64_t)N + BN - 1) / BN); }

// Parts of K with a workspace: enough workgroups of the smaller tiles for the
// chip's 256 CUs, none under four 128-wide steps (M = 100, N = K = 4096, 128
// tiles: two parts 18.9 us, four 21; M = 200, 256 tiles: 21.9, two parts 27).
int k_split(int M, int N, int K)
{
    if (M <= kSkinnyM)
        return 1;
    const int64_t tiles = tiles_of(M, N, M <= 32 ? 32 : 64, 64), steps = (K + 127) / 128;
    int64_t n = (256 + tiles / 2) / tiles;
    n = n < steps / 4 ? n : steps / 4;
    return n < 1 ? 1 : n > 16 ? 16 : (int)n;
}

template <typename T>
hipError_t launch_any(const uint16_t *A, const uint8_t *B, const uint16_t *scale, const uint16_t *zero, int gshift,
                      uint16_t *C, int M, int N, int K, float *ws, int64_t wsBytes, hipStream_t s)
{
    // M = 1: a row of B a wavefront (fp16, K = 4096: N = 4096 5.2 us, the skinny
    // kernel 5.6; N = 11008 9.6, 10.9).  Above, the skinny kernel with as many
    // loads of A as it has rows; with few tiles of N the wavefronts share them
    // out further and hold more in flight (M = 4, K = 4096, bf16 with zero
    // points: N = 4096 eight wavefronts 6.7 us, four 7.8; N = 11008 16.3, 14.1).
    if (M == 1)
        return launch_gemv_t<T>(A, B, scale, zero, gshift, C, N, K, s);
    if (M <= 4)
        return N <= 16 * 512 ? launch_skinny_t<T, 1, 8, 4>(A, B, scale, zero, gshift, C, M, N, K, s)
                             : launch_skinny_t<T, 1, 4, 4>(A, B, scale, zero, gshift, C, M, N, K, s);
    if (M <= 8)
        return launch_skinny_t<T, 2, 8, 2>(A, B, scale, zero, gshift, C, M, N, K, s);
    if (M <= 16)
        return launch_skinny_t<T, 4, 8, 1>(A, B, scale, zero, gshift, C, M, N, K, s);
    // Larger tiles move less, but there have to be enough of them (M = 2048, N =
    // K = 4096: 128 x 128 80 us, 128 x 64 106; M = 256, N = 11008, 172 tiles of
    // 128 x 128: 39, 53, 64 x 64 51; M = 512, N = 4096, K = 11008, 128 tiles: 113,
    // 78, 100; M = 200, N = K = 4096: 64 x 64 21.9, 128 x 64 in two parts 25.9;
    // M = 128, N = 28672: 49, 62, 78).  The rule does not ask how many of a tile's
    // rows there are: from N = 20480 on it takes 128 x 128 for few rows too (M =
    // 20, N = 28672: 42 us, 32 x 64 29; M = 64: 44, 64 x 64 41).
    if (tiles_of(M, N, 128, 128) >= 160)
        return launch_tiled_t<T, 128, 128, 2>(A, B, scale, zero, gshift, C, M, N, K, nullptr, 1, s);
    if (tiles_of(M, N, 128, 64) >= 256)
        return launch_tiled_t<T, 128, 64, 2>(A, B, scale, zero, gshift, C, M, N, K, nullptr, 1, s);
    const int64_t need = gemm_w4g_workspace_bytes(M, N, K);
    const int ksplit = need && wsBytes >= need ? k_split(M, N, K) : 1;
    return M <= 32 ? launch_tiled_t<T, 32, 64, 4>(A, B, scale, zero, gshift, C, M, N, K, ws, ksplit, s)
                   : launch_tiled_t<T, 64, 64, 4>(A, B, scale, zero, gshift, C, M, N, K, ws, ksplit, s);
}

}  // namespace

int64_t gemm_w4g_workspace_bytes(int M, int N, int K)
{
    const int n = k_split(M, N, K);
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
