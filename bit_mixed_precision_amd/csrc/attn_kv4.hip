// Attention over the 4-bit paged cache:
//   o = softmax_t(scale q . K[t]) V[t],  K[t] = uk sk + mk,  V[t] = uv sv + mv
// (codes u = 0..15, scale and min per token and kv head), causal to the end
// of each sequence, optionally inside a sliding window.
//
// The scale and min stay outside the products:
//   q . K[t]  = sk (sum_d q uk) + mk (sum_d q)
//   sum_t p V = sum_t (p sv) (uv - 8) + sum_t p (mv + 8 sv)
// so the matrix instructions multiply by the bare codes.  K's enter them as
// the bits of subnormal fp16 numbers (dtype16.h): one shift and four masks
// for eight codes.  V's are made the fp16 integers u - 8 (nine operations):
// an average over many tokens is far smaller than its terms, and summed
// uncentred (0..15) its fp32 accumulator would carry their mean.
//
// One wavefront takes 32 tokens a step for a tile of 16 query rows (the
// queries of one kv head: q_len x heads per kv head).  It computes
//   S^T = K Q^T   (A = codes of 16 tokens, B = queries)
//   O^T = V^T P^T (A = codes of 16 channels over 32 tokens, B = p sv)
// The result layout of the first (a lane holds four tokens of one query) is
// the operand layout of the second, with the 32 tokens taken in the same
// order on both sides, so p goes from one to the other in registers, and a
// row's running maximum and sum are one value per lane.  The V codes of a
// page are stored in units of four tokens so that their 16-byte load hands a
// lane four tokens of the same channels; a byte permute per pair of tokens
// makes the operand.
//
// p sv is split in two fp16 values (high part and remainder) for an fp16
// output: one rounding of it alone would weigh as much as the output's own;
// with a bf16 output the high part is enough.
// The reference maximum is raised only when a score passes it by 2^8, and
// then for all lanes of the row; sums and accumulators are fp32.
//
// Long sequences are split over workgroups (and over a workgroup's
// wavefronts, joined through LDS); a second kernel joins the parts in order.
#include "bq_internal.h"
#include "dtype16.h"

namespace bq {
namespace {

constexpr int kWaves = 4;
constexpr int kThreads = 64 * kWaves;
constexpr int kTile = 32;      // tokens of a step
constexpr float kNoMax = -3.0e38f;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// What one tile of 16 query rows attends to.
struct Rows {
    int q0;          // first row of the sequence's queries in q / out
    int rows;        // query rows of the sequence and kv head (q_len * group)
    int base;        // position of the first query
    int pos_min, pos_max;
    int lo, hi;      // keys [lo, hi), lo a multiple of kTile
    int chunk;       // keys of one split
};

__device__ __forceinline__ Rows rows_of(const AttnKv4Args &p, int b, int tile)
{
    Rows r;
    int start, qlen;
    if (p.q_start) {
        start = max(p.q_start[b], 0);
        qlen = min(max(min(p.q_start[b + 1], p.total_q) - start, 0), p.max_q_len);
    } else {
        start = b * p.max_q_len;
        qlen = p.max_q_len;
    }
    const int len = min(max(p.seq_lens[b], 0), p.max_blocks << p.page_shift);
    r.q0 = start;
    r.rows = qlen * p.group;
    r.base = len - qlen;
    const int first = tile * 16 / p.group, last = min(tile * 16 + 15, r.rows - 1) / p.group;
    r.pos_min = r.base + first;
    r.pos_max = r.base + last;
    r.lo = p.window > 0 ? max(0, r.pos_min - p.window + 1) & ~(kTile - 1) : 0;
    r.hi = max(r.pos_max + 1, r.lo);
    const int n = r.hi - r.lo;
    constexpr int step = kTile * kWaves;
    r.chunk = p.nsplit == 1 ? n : ((n + p.nsplit - 1) / p.nsplit + step - 1) / step * step;
    return r;
}

template <int D>
struct Tile {
    static constexpr int kW = D / 32;  // dwords of codes per lane and 16 tokens
    uint32_t k[2][kW], v[2][kW];
    u4 kp[2], vp[2];
    int lim[2];  // tokens at or past lim are not there
};

template <int N>
__device__ __forceinline__ void load_dwords(uint32_t *dst, const uint8_t *src)
{
    static_assert(N == 2 || N == 4, "one load");
    if constexpr (N == 2) {
        const u2 x = *(const u2 *)src;
        dst[0] = x.x;
        dst[1] = x.y;
    } else {
        const u4 x = *(const u4 *)src;
        dst[0] = x.x;
        dst[1] = x.y;
        dst[2] = x.z;
        dst[3] = x.w;
    }
}

template <int D>
__device__ __forceinline__ void load_tile(Tile<D> &x, const AttnKv4Args &p, const int *table, int head, int t, int hi,
                                          int lane)
{
    const int g = lane >> 4, m = lane & 15;
    const int P = 1 << p.page_shift;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        // 16 tokens lie in one page; past the end the first 16 are read again
        const int tt = t + 16 * s < hi ? t + 16 * s : t;
        int page = table[tt >> p.page_shift];
        const bool there = page >= 0 && page < p.num_pages;
        page = there ? page : 0;
        x.lim[s] = there ? hi : 0;
        const uint8_t *base = p.cache + (int64_t)((int64_t)page * p.hkv + head) * ((int64_t)P * (D + 8));
        const uint32_t in = tt & (P - 1);
        const uint8_t *kb = base + in * (D / 2), *vb = base + P * (D / 2) + in * (D / 2);
        const uint8_t *pb = base + P * D + in * 4;
        if constexpr (D == 64) {
            load_dwords<2>(x.k[s], kb + m * 32 + g * 8);
            load_dwords<2>(x.v[s], vb + g * 128 + m * 8);
        } else if constexpr (D == 128) {
            load_dwords<4>(x.k[s], kb + m * 64 + g * 16);
            load_dwords<4>(x.v[s], vb + g * 256 + m * 16);
        } else {
            load_dwords<4>(x.k[s], kb + m * 128 + g * 32);
            load_dwords<4>(x.k[s] + 4, kb + m * 128 + g * 32 + 16);
            load_dwords<4>(x.v[s], vb + g * 512 + m * 16);
            load_dwords<4>(x.v[s] + 4, vb + g * 512 + 256 + m * 16);
        }
        x.kp[s] = *(const u4 *)(pb + g * 16);
        x.vp[s] = *(const u4 *)(pb + 4 * P + g * 16);
    }
}

constexpr uint32_t kM0 = 0x000f000fu, kM4 = 0x00f000f0u;

// Codes at bits 0..3 (or, high, 4..7) of each half as the fp16 integers u - 8:
// 0x6400 | u = 1024 + u, and (1024 + 16 u) / 16 - 72, both exact.
__device__ __forceinline__ uint32_t centred(bool high, uint32_t w)
{
    const h2 x = __builtin_bit_cast(h2, (w & (high ? kM4 : kM0)) | 0x64006400u);
    const h2 s = {(_Float16)0.0625f, (_Float16)0.0625f}, c = {(_Float16)-72.0f, (_Float16)-72.0f};
    const h2 b = {(_Float16)-1032.0f, (_Float16)-1032.0f};
    return __builtin_bit_cast(uint32_t, high ? __builtin_elementwise_fma(x, s, c) : x + b);
}

template <typename T, int D>
struct Wave {
    static constexpr int kQ = D / 64;   // operand pairs of the queries
    static constexpr int kMT = D / 16;  // output tiles of 16 channels
    static constexpr bool kLow = !T::kBf16;
    u4 q0[kQ], q4[kQ];
    float a1, b1;          // score = a1 sk (16 s0 + s4) + b1 mk, in powers of two
    float mt, mref;        // reference maximum, and what is subtracted: mt - shift
    float cap, shift;      // largest V scale that p sv 2^shift takes in fp16's range
    float l, z;
    f4 o[kMT];

    __device__ __forceinline__ void init(const uint16_t *q, bool ok, float scale, int lane)
    {
        const int g = lane >> 4;
        uint32_t w[D / 8];
        float sum = 0.0f, top = 0.0f;
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
            const u4 x = ok ? *(const u4 *)(q + g * (D / 4) + 8 * i) : (u4){0, 0, 0, 0};
            w[4 * i] = x.x;
            w[4 * i + 1] = x.y;
            w[4 * i + 2] = x.z;
            w[4 * i + 3] = x.w;
        }
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {
            const float a = T::to_f32(w[i] & 0xffffu), b = T::to_f32(w[i] >> 16);
            sum += a;
            sum += b;
            top = fmaxf(top, fmaxf(fabsf(a), fabsf(b)));
        }
#pragma unroll
        for (int off = 16; off < 64; off <<= 1) {
            sum += __shfl_xor(sum, off, 64);
            top = fmaxf(top, __shfl_xor(top, off, 64));
        }
        float back = 1.0f;
        if constexpr (T::kBf16) {
            // a power of two brings the row into fp16's range: bf16's eight
            // bits survive down to 2^-24 of the row's largest value
            const uint32_t e = max((__float_as_uint(top) >> 23) & 255u, 11u);
            const float f = e < 255u ? __uint_as_float((264u - e) << 23) : 1.0f;
            back = e < 255u ? __uint_as_float((e - 10u) << 23) : 1.0f;
#pragma unroll
            for (int i = 0; i < D / 8; ++i)
                w[i] = F16::from_f32(T::to_f32(w[i] & 0xffffu) * f) | (uint32_t)F16::from_f32(T::to_f32(w[i] >> 16) * f) << 16;
        }
        // codes 0, 4 and 2, 6 of a dword sit at bits 0..3 of a half, 1, 5 and 3, 7 at 4..7
#pragma unroll
        for (int i = 0; i < kQ; ++i) {
            const uint32_t *c = w + 8 * i;
            q0[i] = (u4){pack_lo(c[0], c[2]), pack_lo(c[1], c[3]), pack_lo(c[4], c[6]), pack_lo(c[5], c[7])};
            q4[i] = (u4){pack_hi(c[0], c[2]), pack_hi(c[1], c[3]), pack_hi(c[4], c[6]), pack_hi(c[5], c[7])};
        }
        a1 = back * 0x1p20f * (scale * kLog2e);
        b1 = sum * (scale * kLog2e);
        mt = mref = kNoMax;
        cap = shift = 0.0f;
        l = z = 0.0f;
#pragma unroll
        for (int i = 0; i < kMT; ++i)
            o[i] = (f4){0, 0, 0, 0};
    }

    template <bool MASK>
    __device__ __forceinline__ void step(const Tile<D> &x, int t, int pos, int window, int lane)
    {
        const int g = lane >> 4;
        float s[8], sv[8], mv[8];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            f4 s0 = {0, 0, 0, 0}, s4 = {0, 0, 0, 0};
#pragma unroll
            for (int i = 0; i < kQ; ++i) {
                const uint32_t a = x.k[h][2 * i], b = x.k[h][2 * i + 1];
                const uint32_t a8 = a >> 8, b8 = b >> 8;
                s0 = F16::mma((u4){a & kM0, a8 & kM0, b & kM0, b8 & kM0}, q0[i], s0);
                s4 = F16::mma((u4){a & kM4, a8 & kM4, b & kM4, b8 & kM4}, q4[i], s4);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float sk = half_bits(x.kp[h][i] & 0xffffu), mk = half_bits(x.kp[h][i] >> 16);
                const int j = 4 * h + i;
                s[j] = (s0[i] * 16.0f + s4[i]) * sk * a1 + mk * b1;
                sv[j] = half_bits(x.vp[h][i] & 0xffffu);
                mv[j] = half_bits(x.vp[h][i] >> 16) + 8.0f * sv[j];
                if constexpr (MASK) {
                    const int tok = t + 16 * h + 4 * g + i;
                    const bool on = tok < x.lim[h] && tok <= pos && (window <= 0 || tok > pos - window);
                    s[j] = on ? s[j] : -__builtin_inff();
                    sv[j] = on ? sv[j] : 0.0f;
                    mv[j] = on ? mv[j] : 0.0f;
                }
            }
        }
        float top = s[0], vtop = sv[0];
#pragma unroll
        for (int j = 1; j < 8; ++j) {
            top = fmaxf(top, s[j]);
            vtop = fmaxf(vtop, sv[j]);
        }
        if (__any(top > mt + 8.0f || vtop > cap)) {
#pragma unroll
            for (int off = 16; off < 64; off <<= 1) {
                top = fmaxf(top, __shfl_xor(top, off, 64));
                vtop = fmaxf(vtop, __shfl_xor(vtop, off, 64));
            }
#pragma unroll
            for (int off = 1; off < 16; off <<= 1)  // masked rows may hold back a scale
                vtop = fmaxf(vtop, __shfl_xor(vtop, off, 64));
            mt = fmaxf(mt, top);
            if (vtop > cap) {
                const int e = (int)((__float_as_uint(vtop) >> 23) & 255u) - 125;
                cap = ldexpf(1.0f, e);
                shift = (float)(6 - e);
            }
            const float now = mt - shift, f = __builtin_amdgcn_exp2f(mref - now);
            mref = now;
            l *= f;
            z *= f;
#pragma unroll
            for (int i = 0; i < kMT; ++i)
                o[i] *= f;
        }
        u4 ph, pl;
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
            const float p0 = __builtin_amdgcn_exp2f(s[j] - mref), p1 = __builtin_amdgcn_exp2f(s[j + 1] - mref);
            l += p0;
            l += p1;
            z += p0 * mv[j];
            z += p1 * mv[j + 1];
            const float v0 = p0 * sv[j], v1 = p1 * sv[j + 1];
            const h2 hi = {(_Float16)v0, (_Float16)v1};
            ph[j / 2] = __builtin_bit_cast(uint32_t, hi);
            if constexpr (kLow)
                pl[j / 2] = __builtin_bit_cast(uint32_t, (h2){(_Float16)(v0 - (float)hi[0]), (_Float16)(v1 - (float)hi[1])});
        }
#pragma unroll
        for (int c = 0; c < (D == 256 ? 2 : 1); ++c) {
            // pairs of tokens of the same channels: codes 0..3 (and 4..7) of a unit
            u4 lo, hi;
            if constexpr (D == 64) {
                lo = (u4){x.v[0][0], x.v[0][1], x.v[1][0], x.v[1][1]};
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t a = x.v[i >> 1][4 * c + 2 * (i & 1)], b = x.v[i >> 1][4 * c + 2 * (i & 1) + 1];
                    lo[i] = pack_lo(a, b);
                    hi[i] = pack_hi(a, b);
                }
            }
#pragma unroll
            for (int j = 0; j < (D == 64 ? 4 : 8); ++j) {
                const u4 w = j < 4 ? lo : hi;
                u4 a;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    a[i] = centred(j & 1, (j & 2) ? w[i] >> 8 : w[i]);
                f4 &acc = o[8 * c + j];
                acc = F16::mma(a, ph, acc);
                if constexpr (kLow)
                    acc = F16::mma(a, pl, acc);
            }
        }
    }

    // Sums of the row over its four lanes; the accumulators take in z.
    __device__ __forceinline__ void finish()
    {
#pragma unroll
        for (int off = 16; off < 64; off <<= 1) {
            l += __shfl_xor(l, off, 64);
            z += __shfl_xor(z, off, 64);
        }
#pragma unroll
        for (int i = 0; i < kMT; ++i)
            o[i] += z;
    }
};

template <typename T, int D>
__global__ __launch_bounds__(kThreads) void attn_kv4_kernel(const AttnKv4Args p)
{
    constexpr int DH = D > 128 ? 128 : D;  // channels joined at a time
    __shared__ float so[kWaves][16][DH + 4];
    __shared__ float sm[kWaves][16], sl[kWaves][16];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    int id = blockIdx.x;
    const int split = id % p.nsplit;
    const int item = id / p.nsplit;
    const int tile = item % p.row_tiles;
    const int head = item / p.row_tiles % p.hkv;
    const int b = item / p.row_tiles / p.hkv;
    const Rows r = rows_of(p, b, tile);
    if (tile * 16 >= r.rows)
        return;
    const int start = r.lo + split * r.chunk, end = min(start + r.chunk, r.hi);
    if (split > 0 && start >= r.hi)
        return;

    const int row = tile * 16 + (lane & 15);
    const int qi = row / p.group, hg = row - qi * p.group;
    const bool ok = row < r.rows;
    const int pos = ok ? r.base + qi : r.pos_max;
    Wave<T, D> w;
    w.init((const uint16_t *)p.q + (int64_t)(r.q0 + qi) * p.q_stride + (head * p.group + hg) * D, ok, p.scale, lane);
    const int *table = p.block_table + (int64_t)b * p.max_blocks;
    const auto one = [&](const Tile<D> &x, int t) {
        const int whole = min(min(x.lim[0], x.lim[1]), r.pos_min + 1);
        if (t + kTile <= whole && (p.window <= 0 || t > r.pos_max - p.window))
            w.template step<false>(x, t, pos, p.window, lane);
        else
            w.template step<true>(x, t, pos, p.window, lane);
    };
    int t = start + wave * kTile;
    if (t < end) {
        // the next tile's loads are in flight during a tile's arithmetic
        Tile<D> x;
        load_tile<D>(x, p, table, head, t, end, lane);
        for (; t + kWaves * kTile < end; t += kWaves * kTile) {
            Tile<D> y;
            load_tile<D>(y, p, table, head, t + kWaves * kTile, end, lane);
            one(x, t);
            x = y;
        }
        one(x, t);
    }
    w.finish();

    // join the wavefronts: thread (row, c) takes DH/16 channels
    const int g = lane >> 4, m = lane & 15;
    if (g == 0) {
        sm[wave][m] = w.mref;
        sl[wave][m] = w.l;
    }
    const int jr = threadIdx.x >> 4, jc = threadIdx.x & 15;
    constexpr int CH = DH / 16;
    const int orow = tile * 16 + jr;
    const int oqi = orow / p.group, ohg = orow - oqi * p.group;
    const int64_t orow_at = (int64_t)(r.q0 + oqi) * p.hq + head * p.group + ohg;
    const int64_t part = (int64_t)(item * (int64_t)p.nsplit + split) * 16 + jr;
#pragma unroll
    for (int c = 0; c < D / DH; ++c) {
        if (c)
            __syncthreads();
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < CH; j += 4)
                *(float4 *)&so[wave][m][(g * 4 + i) * CH + j] =
                    make_float4(w.o[8 * c + j][i], w.o[8 * c + j + 1][i], w.o[8 * c + j + 2][i], w.o[8 * c + j + 3][i]);
        __syncthreads();
        float mm = sm[0][jr];
#pragma unroll
        for (int k = 1; k < kWaves; ++k)
            mm = fmaxf(mm, sm[k][jr]);
        float l = 0.0f, acc[CH] = {};
#pragma unroll
        for (int k = 0; k < kWaves; ++k) {
            const float f = __builtin_amdgcn_exp2f(sm[k][jr] - mm);
            l += f * sl[k][jr];
#pragma unroll
            for (int j = 0; j < CH; ++j)
                acc[j] += f * so[k][jr][jc * CH + j];
        }
        if (orow < r.rows) {
            if (p.nsplit == 1) {
                uint16_t *dst = (uint16_t *)p.out + orow_at * D + c * DH + jc * CH;
                uint32_t y[CH / 2];
#pragma unroll
                for (int j = 0; j < CH; j += 2)
                    y[j / 2] = T::from_f32(l == 0.0f ? 0.0f : acc[j] / l) |
                               (uint32_t)T::from_f32(l == 0.0f ? 0.0f : acc[j + 1] / l) << 16;
                if constexpr (CH == 8)
                    *(u4 *)dst = (u4){y[0], y[1], y[2], y[3]};
                else
                    *(u2 *)dst = (u2){y[0], y[1]};
                if (p.lse && c == 0 && jc == 0)
                    p.lse[orow_at] = l == 0.0f ? -__builtin_inff() : (mm + __builtin_amdgcn_logf(l)) * kLn2;
            } else {
                float *dst = p.part + part * D + c * DH + jc * CH;
#pragma unroll
                for (int j = 0; j < CH; j += 4)
                    *(float4 *)(dst + j) = make_float4(acc[j], acc[j + 1], acc[j + 2], acc[j + 3]);
                if (c == 0 && jc == 0)
                    *(float2 *)(p.part_ml + part * 2) = make_float2(mm, l);
            }
        }
    }
}

// Joins the splits of one query row: 256 threads, D/4 of them a split.
template <typename T, int D>
__global__ __launch_bounds__(256) void attn_kv4_join(const AttnKv4Args p)
{
    constexpr int TPS = D / 4, G = 256 / TPS;
    __shared__ float4 so[G][TPS];
    const int item = blockIdx.x >> 4, jr = blockIdx.x & 15;
    const int tile = item % p.row_tiles;
    const int head = item / p.row_tiles % p.hkv;
    const int b = item / p.row_tiles / p.hkv;
    const Rows r = rows_of(p, b, tile);
    const int row = tile * 16 + jr;
    if (row >= r.rows)
        return;
    const int n = r.hi > r.lo ? (r.hi - r.lo + r.chunk - 1) / r.chunk : 1;
    const int64_t first = (int64_t)item * p.nsplit * 16 + jr;
    const int lane = threadIdx.x & 63;
    // every wavefront holds all splits' maxima and sums, one a lane (nsplit <= 64)
    const float2 ml = lane < n ? *(const float2 *)(p.part_ml + (first + 16 * lane) * 2) : make_float2(kNoMax, 0.0f);
    float mm = ml.x;
#pragma unroll
    for (int off = 32; off > 0; off >>= 1)
        mm = fmaxf(mm, __shfl_xor(mm, off, 64));
    const float f = __builtin_amdgcn_exp2f(ml.x - mm);
    float l = f * ml.y;
#pragma unroll
    for (int off = 32; off > 0; off >>= 1)
        l += __shfl_xor(l, off, 64);
    const int gq = threadIdx.x / TPS, c = threadIdx.x % TPS;
    float4 acc = make_float4(0, 0, 0, 0);
    for (int s0 = 0; s0 < n; s0 += G) {
        const int s = s0 + gq;
        const float fs = __shfl(f, s & 63, 64);
        if (s < n) {
            const float4 o = *(const float4 *)(p.part + (first + 16 * (int64_t)s) * D + 4 * c);
            acc.x += fs * o.x;
            acc.y += fs * o.y;
            acc.z += fs * o.z;
            acc.w += fs * o.w;
        }
    }
    so[gq][c] = acc;
    __syncthreads();
    if (gq == 0) {
#pragma unroll
        for (int k = 1; k < G; ++k) {
            const float4 o = so[k][c];
            acc.x += o.x;
            acc.y += o.y;
            acc.z += o.z;
            acc.w += o.w;
        }
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
        const int qi = row / p.group, hg = row - qi * p.group;
        const int64_t at = (int64_t)(r.q0 + qi) * p.hq + head * p.group + hg;
        *(u2 *)((uint16_t *)p.out + at * D + 4 * c) = (u2){T::from_f32(acc.x * inv) | (uint32_t)T::from_f32(acc.y * inv) << 16,
                                                           T::from_f32(acc.z * inv) | (uint32_t)T::from_f32(acc.w * inv) << 16};
        if (p.lse && c == 0)
            p.lse[at] = l == 0.0f ? -__builtin_inff() : (mm + __builtin_amdgcn_logf(l)) * kLn2;
    }
}

template <typename T, int D>
hipError_t launch_t(const AttnKv4Args &p, int64_t items, hipStream_t s)
{
    if (!grid_fits(items * p.nsplit, kThreads) || !grid_fits(items * 16, 256))
        return kGridTooLarge;
    attn_kv4_kernel<T, D><<<dim3((unsigned)(items * p.nsplit)), kThreads, 0, s>>>(p);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || p.nsplit == 1)
        return e;
    attn_kv4_join<T, D><<<dim3((unsigned)(items * 16)), 256, 0, s>>>(p);
    return hipGetLastError();
}

template <typename T>
hipError_t launch_d(const AttnKv4Args &p, int D, int64_t items, hipStream_t s)
{
    return D == 64 ? launch_t<T, 64>(p, items, s) : D == 128 ? launch_t<T, 128>(p, items, s) : launch_t<T, 256>(p, items, s);
}

}  // namespace

int attn_kv4_splits(int64_t items, int64_t max_len)
{
    const int64_t step = kTile * kWaves;
    const int64_t want = (1024 + items - 1) / items, most = (max_len + step - 1) / step;
    const int64_t n = want < most ? want : most;
    return (int)(n < 1 ? 1 : n > 64 ? 64 : n);
}

hipError_t launch_attn_kv4(const AttnKv4Args &p, int D, bool bf16, hipStream_t s)
{
    const int64_t items = (int64_t)p.batch * p.hkv * p.row_tiles;
    return bf16 ? launch_d<BF16>(p, D, items, s) : launch_d<F16>(p, D, items, s);
}

}  // namespace bq
