// The step between the QKV product and attention, one pass over its rows:
//   y = x * rsqrt(mean(x^2) + eps) * w       per head (w absent: y = x)
//   (a, b) -> (a cos - b sin, b cos + a sin) on the first rot_dim channels,
// pairs (i, i + rot_dim/2) or (2i, 2i + 1), one rounding to the 16-bit type;
// and, with a cache, keys and values quantized to 4 bits per token and head:
//   min = fp16(min y), scale = fp16((max y - min) / 15),
//   code = rint((y - min) / scale) in 0..15     (fp32, correctly rounded).
//
// Layout: D/8 lanes per head row, eight channels (16 bytes) a lane, so a
// wavefront covers 512 channels with one load instruction; the norm's sum and
// the quantizer's range are butterfly reductions inside the row's lanes, and
// a rotation pair in halves is a lane rot_dim/16 away.  Bound by moving the
// rows (and by launch latency at decode sizes); with a cache, by latency: 4097
// tokens of 16 + 16 heads of 64 take 16.9 us, of which the VALU issues for 7,
// in six wavefronts a SIMD.  Scattered slots write 19.4 MB there, neighbouring
// ones 12.8, and take 0.8 us more.
//
// Keys that go to the cache are normalized and rotated in fp64 (fp64 runs at
// the fp32 rate on this chip): a code turns over at a border between two
// values, and with 53 bits the rounded key, hence the code, is the
// definition's.  Queries (and keys without a cache) take fp32.
#include "bq_layer_internal.h"
#include "dtype16.h"

namespace bq {
namespace {

constexpr int kThreads = 256;

template <typename F, int LPR>
__device__ __forceinline__ F row_sum(F v)
{
#pragma unroll
    for (int off = LPR / 2; off > 0; off >>= 1)
        v += __shfl_xor(v, off, 64);
    return v;
}

__device__ __forceinline__ float inv_rms(float ms) { return __builtin_amdgcn_rsqf(ms); }
// Two Newton steps from the hardware's estimate (about 2^-28): a few units of
// 2^-53, which is far below where a rounding to 16 bits could turn over.
__device__ __forceinline__ double inv_rms(double ms)
{
    double r = __builtin_amdgcn_rsq(ms);
    r = r * (1.5 - 0.5 * ms * r * r);
    return r * (1.5 - 0.5 * ms * r * r);
}

template <typename T>
__device__ __forceinline__ void unpack8(const uint4 raw, float (&y)[8])
{
    const uint32_t r[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        y[2 * i] = T::to_f32(r[i] & 0xffffu);
        y[2 * i + 1] = T::to_f32(r[i] >> 16);
    }
}

// What a lane needs of a token's rotation: its channels' cosines and sines,
// and the lane that holds their partners (a rotation in halves).
struct Turn {
    float4 c[2], s[2];
    bool in, first;
    int other;  // partner's place in the row
};

__device__ __forceinline__ Turn turn_of(const float *cs, const float *sn, int rot, int inter, int sub)
{
    Turn t = {};
    const int hl = rot / 16;  // lanes of one half; rot is a multiple of 16: whole lanes
    t.in = 8 * sub < rot;
    t.first = sub < hl;
    t.other = t.in && !inter ? (t.first ? sub + hl : sub - hl) : sub;
    if (t.in) {
        const int at = inter ? 4 * sub : 8 * (t.first ? sub : sub - hl);
        t.c[0] = *(const float4 *)(cs + at);
        t.s[0] = *(const float4 *)(sn + at);
        if (!inter) {
            t.c[1] = *(const float4 *)(cs + at + 4);
            t.s[1] = *(const float4 *)(sn + at + 4);
        }
    }
    return t;
}

// Norm and rotation of one lane's eight channels in type F; the result in
// the 16-bit type's bits (through fp32, as a conversion from fp64 goes).  A
// rotation in halves needs another lane's channels: they come over as loaded
// (four dwords) and are scaled again here.
template <typename T, typename F, int LPR>
__device__ __forceinline__ void norm_rope(const uint4 raw, const uint16_t *w, double eps, const Turn &turn, int rot, int inter,
                                          int sub, uint16_t out[8])
{
    const bool in = turn.in, first = turn.first;
    const int other = turn.other;
    const float4 *c = turn.c, *s = turn.s;
    uint4 wr, wo;
    if (w) {
        wr = *(const uint4 *)(w + 8 * sub);
        wo = *(const uint4 *)(w + 8 * other);
    }
    // y = inv (x w): the product of two 16-bit values is exact in fp32, and inv
    // is the row's, so it is applied once, at the end
    float x[8];
    unpack8<T>(raw, x);
    F inv = 1;
    if (w) {
        F sq = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            sq += (F)x[i] * (F)x[i];
        inv = inv_rms(row_sum<F, LPR>(sq) * (F)(1.0 / (8 * LPR)) + (F)eps);
        float g[8];
        unpack8<T>(wr, g);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            x[i] *= g[i];
    }
    F y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        y[i] = (F)x[i];
    const float cc[8] = {c[0].x, c[0].y, c[0].z, c[0].w, c[1].x, c[1].y, c[1].z, c[1].w};
    const float ss[8] = {s[0].x, s[0].y, s[0].z, s[0].w, s[1].x, s[1].y, s[1].z, s[1].w};
    if (inter) {
        if (in) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const F a = y[2 * i], b = y[2 * i + 1];
                y[2 * i] = a * (F)cc[i] - b * (F)ss[i];
                y[2 * i + 1] = b * (F)cc[i] + a * (F)ss[i];
            }
        }
    } else if (rot) {
        const int lane = (threadIdx.x & 63) - sub + other;
        const uint4 ro = make_uint4(__shfl(raw.x, lane, 64), __shfl(raw.y, lane, 64), __shfl(raw.z, lane, 64),
                                    __shfl(raw.w, lane, 64));
        if (in) {
            float o[8];
            unpack8<T>(ro, o);
            if (w) {
                float g[8];
                unpack8<T>(wo, g);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    o[i] *= g[i];
            }
            const uint32_t sign = first ? 0x80000000u : 0u;  // a cos - b sin, b cos + a sin
#pragma unroll
            for (int i = 0; i < 8; ++i)
                y[i] = y[i] * (F)cc[i] + (F)o[i] * (F)__uint_as_float(__float_as_uint(ss[i]) ^ sign);
        }
    }
    if (w) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            y[i] *= inv;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        // fp32 first, then the 16-bit type: the empty asm keeps the compiler
        // from rounding an fp64 value straight to 16 bits
        float f = (float)y[i];
        asm volatile("" : "+v"(f));
        out[i] = T::from_f32(f);
    }
}

__device__ __forceinline__ uint4 pack8(const uint16_t o[8])
{
    return make_uint4(o[0] | (uint32_t)o[1] << 16, o[2] | (uint32_t)o[3] << 16, o[4] | (uint32_t)o[5] << 16,
                      o[6] | (uint32_t)o[7] << 16);
}

// Bytes of one head of one page: K codes, V codes, K and V parameters.
__device__ __forceinline__ int64_t head_base(int64_t page, int head, int hkv, int page_size, int D)
{
    return (page * hkv + head) * (int64_t)page_size * (D + 8);
}

template <typename T, int LPR>
__device__ __forceinline__ void store_kv4(const uint16_t x16[8], bool isV, uint8_t *base, uint32_t tok, int page_size, int sub)
{
    constexpr int D = 8 * LPR;
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        x[i] = T::to_f32(x16[i]);
    float lo = x[0], hi = x[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) {
        lo = fminf(lo, x[i]);
        hi = fmaxf(hi, x[i]);
    }
#pragma unroll
    for (int off = LPR / 2; off > 0; off >>= 1) {
        lo = fminf(lo, __shfl_xor(lo, off, 64));
        hi = fmaxf(hi, __shfl_xor(hi, off, 64));
    }
    // the stored parameters are fp16: bf16 values past its range are held at its
    // ends, and a row below it (max x < min) takes the scale 0
    const float mn = (float)(_Float16)fminf(fmaxf(lo, -65504.0f), 65504.0f);
    const float sc = (float)(_Float16)fminf(fmaxf((hi - mn) / 15.0f, 0.0f), 65504.0f);
    // The correctly rounded quotient from the scale's correctly rounded
    // reciprocal: one correction of d r by its exact remainder (Markstein).
    // A scale of 0 (or no number) makes codes 0.
    const float r = sc > 0.0f ? 1.0f / sc : 0.0f;
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float d = x[i] - mn, q0 = d * r;
        const float q = __builtin_fmaf(__builtin_fmaf(-sc, q0, d), r, q0);
        w |= (uint32_t)fminf(fmaxf(rintf(q), 0.0f), 15.0f) << (4 * i);
    }
    if (!isV) {
        *(uint32_t *)(base + tok * (D / 2) + 4 * sub) = w;
    } else {
        uint8_t *v = base + page_size * (D / 2) + (tok >> 2) * (2 * D);
        if constexpr (D >= 128) {
            *(uint32_t *)(v + 16 * sub + 4 * (tok & 3)) = w;
        } else {
            *(uint16_t *)(v + 16 * sub + 2 * (tok & 3)) = (uint16_t)w;
            *(uint16_t *)(v + 16 * sub + 8 + 2 * (tok & 3)) = (uint16_t)(w >> 16);
        }
    }
    if (sub == 0)
        *(uint32_t *)(base + page_size * D + (isV ? 4 * page_size : 0) + 4 * tok) =
            F16::from_f32(sc) | (uint32_t)F16::from_f32(mn) << 16;
}

// A wavefront takes one unit of 64 / LPR tokens: HB neighbouring heads of one
// kind (queries, keys, values), a row of lanes a token.  So all of it runs one
// kind's code, the head is the same in all lanes, and what belongs to the token
// (position, slot, cosines) is found once for HB heads, whose loads are in
// flight together.  Units of the same heads and kTokens tokens are neighbours:
// where slots are neighbours too, their codes fill cache lines together.
// (Rows that took the heads of one token after another mixed kinds in a
// wavefront: 4096 tokens of 32 + 8 heads of 128 with a cache 35.6 us, so 31.0.)
constexpr int kTokens = 16;

template <typename T, int LPR, bool CACHE, int HB>
__global__ __launch_bounds__(kThreads) void qk_norm_rope_kernel(const QkRopeArgs p)
{
    constexpr int D = 8 * LPR, kRows = 64 / LPR, kPer = kTokens / kRows;
    const uint32_t uq = (p.hq + HB - 1) / HB, uk = (p.hkv + HB - 1) / HB, units = uq + uk * (CACHE ? 2 : 1);
    // the grid limit keeps units of all tokens below 2^32
    const uint32_t wave = __builtin_amdgcn_readfirstlane(blockIdx.x * (kThreads / 64) + threadIdx.x / 64);
    const uint32_t block = wave / (units * kPer), in_block = wave - block * (units * kPer);
    uint32_t unit = in_block / kPer;
    const int64_t tok = (block * kPer + in_block % kPer) * kRows + (threadIdx.x & 63) / LPR;
    const int sub = threadIdx.x % LPR;
    if (tok >= p.tokens)
        return;
    const bool isQ = unit < uq, isV = unit >= uq + uk;
    unit -= isQ ? 0 : isV ? uq + uk : uq;
    const int heads = isQ ? p.hq : p.hkv, head0 = unit * HB;
    const uint16_t *src = isQ ? p.q + tok * p.q_stride : isV ? p.v + tok * p.v_stride : p.k + tok * p.k_stride;
    uint4 raw[HB];
#pragma unroll
    for (int i = 0; i < HB; ++i)
        raw[i] = *(const uint4 *)(src + min(head0 + i, heads - 1) * D + 8 * sub);
    // a row's lanes take one path together: every shuffle stays inside a row
    int64_t pos = 0;
    if (p.rot) {
        pos = p.positions[tok];
        if (pos < 0 || pos >= p.max_pos)
            return;
    }
    if (!CACHE || isQ) {
        const Turn turn = turn_of(p.cos + pos * (p.rot / 2), p.sin + pos * (p.rot / 2), p.rot, p.inter, sub);
        const uint16_t *w = isQ ? p.q_weight : p.k_weight;
        uint16_t *out = (isQ ? p.q_out : p.k_out) + tok * heads * D + 8 * sub;
#pragma unroll
        for (int i = 0; i < HB; ++i) {
            if (head0 + i >= heads)
                break;
            uint16_t o[8];
            norm_rope<T, float, LPR>(raw[i], w, p.eps, turn, p.rot, p.inter, sub, o);
            *(uint4 *)(out + (head0 + i) * D) = pack8(o);
        }
    }
    if constexpr (CACHE) {
        if (isQ)
            return;
        const int64_t slot = p.slots[tok];
        if (slot < 0 || slot >= p.num_pages << p.page_shift)
            return;
        const int page_size = 1 << p.page_shift;
        const uint32_t at = (uint32_t)slot & (page_size - 1);
        uint8_t *base = p.cache + head_base(slot >> p.page_shift, head0, p.hkv, page_size, D);
        Turn turn;
        if (!isV)
            turn = turn_of(p.cos + pos * (p.rot / 2), p.sin + pos * (p.rot / 2), p.rot, p.inter, sub);
#pragma unroll
        for (int i = 0; i < HB; ++i) {
            if (head0 + i >= heads)
                break;
            uint16_t o[8];
            if (isV) {
                const uint32_t r[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    o[2 * j] = (uint16_t)r[j];
                    o[2 * j + 1] = (uint16_t)(r[j] >> 16);
                }
            } else {
                norm_rope<T, double, LPR>(raw[i], p.k_weight, p.eps, turn, p.rot, p.inter, sub, o);
            }
            store_kv4<T, LPR>(o, isV, base + i * (int64_t)page_size * (D + 8), at, page_size, sub);
        }
    }
}

// Eight channels a lane of K or V of one token: codes and parameters to the
// 16-bit type, T(fp32(code * scale) + min): the product is exact.
// Wavefronts are laid out as the writer's (4097 tokens, 16 heads of 64: 8.3 us
// with rows of one token's heads, so 7.4).  Bound by latency: a wavefront lives
// for three accesses, each after the last (slot, codes and parameters, outputs),
// and moves 1 KB; its VALU is busy 8 % of that time.  Neighbouring slots gain
// little (7.2 us; 16388 tokens 28, scattered 30: 3 TB/s).
template <typename T, int LPR>
__global__ __launch_bounds__(kThreads) void kv4_read_kernel(const uint8_t *cache, int64_t num_pages, int page_shift, int hkv,
                                                            const int64_t *slots, int64_t tokens, uint16_t *k, uint16_t *v)
{
    constexpr int D = 8 * LPR;
    const int page_size = 1 << page_shift;
    constexpr int kRows = 64 / LPR, kPer = kTokens / kRows;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(blockIdx.x * (kThreads / 64) + threadIdx.x / 64);
    const uint32_t block = wave / (2 * hkv * kPer), in_block = wave - block * (2 * hkv * kPer);
    const int64_t tok = (block * kPer + in_block % kPer) * kRows + (threadIdx.x & 63) / LPR;
    const int sub = threadIdx.x % LPR;
    if (tok >= tokens)
        return;
    const int head = (int)(in_block / kPer);
    const bool isV = head >= hkv;
    const int h = isV ? head - hkv : head;
    const int64_t slot = slots[tok];
    if (slot < 0 || slot >= num_pages << page_shift)
        return;
    const uint32_t t = (uint32_t)slot & (page_size - 1);
    const uint8_t *base = cache + head_base(slot >> page_shift, h, hkv, page_size, D);
    uint32_t w;
    if (!isV) {
        w = *(const uint32_t *)(base + t * (D / 2) + 4 * sub);
    } else {
        const uint8_t *b = base + page_size * (D / 2) + (t >> 2) * (2 * D) + 16 * sub;
        if constexpr (D >= 128)
            w = *(const uint32_t *)(b + 4 * (t & 3));
        else
            w = *(const uint16_t *)(b + 2 * (t & 3)) | (uint32_t)*(const uint16_t *)(b + 8 + 2 * (t & 3)) << 16;
    }
    const uint32_t par = *(const uint32_t *)(base + page_size * D + (isV ? 4 * page_size : 0) + 4 * t);
    const float sc = half_bits(par & 0xffffu), mn = half_bits(par >> 16);
    uint16_t o[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        o[i] = T::from_f32((float)((w >> (4 * i)) & 15u) * sc + mn);
    *(uint4 *)((isV ? v : k) + (tok * hkv + h) * D + 8 * sub) = pack8(o);
}

template <typename T, int LPR, bool CACHE>
hipError_t launch_rope_t(const QkRopeArgs &p, hipStream_t s)
{
    const int64_t heads = p.hq + (int64_t)p.hkv * (CACHE ? 2 : 1);
    // Four heads a row of lanes once there are 12 wavefronts' work for each of
    // the 1024 SIMDs, one for shorter calls.  With a cache, heads of 128, 32 + 8:
    // 4096 tokens 31.0 us, with one head 37.3; 512 tokens 8.8, with one 7.5;
    // heads of 64, 16 + 16: 2048 tokens 10.5 against 10.8, 1024 8.7 against 6.1.
    constexpr int kMany = 4;
    const bool many = p.tokens * heads * LPR >= 3 * 64 * 4096;
    const auto units = [&](int64_t per) { return (p.hq + per - 1) / per + (CACHE ? 2 : 1) * ((p.hkv + per - 1) / per); };
    const int64_t waves = (p.tokens + kTokens - 1) / kTokens * (kTokens * LPR / 64) * units(many ? kMany : 1);
    const int64_t wgs = (waves + kThreads / 64 - 1) / (kThreads / 64);
    if (!grid_fits(wgs, kThreads))
        return kGridTooLarge;
    const dim3 grid((unsigned)wgs);
    if (many)
        qk_norm_rope_kernel<T, LPR, CACHE, kMany><<<grid, kThreads, 0, s>>>(p);
    else
        qk_norm_rope_kernel<T, LPR, CACHE, 1><<<grid, kThreads, 0, s>>>(p);
    return hipGetLastError();
}

template <typename T, bool CACHE>
hipError_t launch_rope_d(const QkRopeArgs &p, hipStream_t s)
{
    return p.D == 64    ? launch_rope_t<T, 8, CACHE>(p, s)
           : p.D == 128 ? launch_rope_t<T, 16, CACHE>(p, s)
                        : launch_rope_t<T, 32, CACHE>(p, s);
}

template <typename T>
hipError_t launch_read_t(const uint8_t *cache, int64_t num_pages, int page_shift, int hkv, int D, const int64_t *slots,
                         int64_t tokens, uint16_t *k, uint16_t *v, hipStream_t s)
{
    const int64_t waves = (tokens + kTokens - 1) / kTokens * (kTokens * (D / 8) / 64) * 2 * hkv;
    const int64_t wgs = (waves + kThreads / 64 - 1) / (kThreads / 64);
    if (!grid_fits(wgs, kThreads))
        return kGridTooLarge;
    const dim3 grid((unsigned)wgs);
    if (D == 64)
        kv4_read_kernel<T, 8><<<grid, kThreads, 0, s>>>(cache, num_pages, page_shift, hkv, slots, tokens, k, v);
    else if (D == 128)
        kv4_read_kernel<T, 16><<<grid, kThreads, 0, s>>>(cache, num_pages, page_shift, hkv, slots, tokens, k, v);
    else
        kv4_read_kernel<T, 32><<<grid, kThreads, 0, s>>>(cache, num_pages, page_shift, hkv, slots, tokens, k, v);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_qk_norm_rope(const QkRopeArgs &p, bool bf16, hipStream_t s)
{
    if (p.cache)
        return bf16 ? launch_rope_d<BF16, true>(p, s) : launch_rope_d<F16, true>(p, s);
    return bf16 ? launch_rope_d<BF16, false>(p, s) : launch_rope_d<F16, false>(p, s);
}

hipError_t launch_kv4_read(const uint8_t *cache, int64_t num_pages, int page_shift, int hkv, int D, const int64_t *slots,
                           int64_t tokens, uint16_t *k, uint16_t *v, bool bf16, hipStream_t s)
{
    return bf16 ? launch_read_t<BF16>(cache, num_pages, page_shift, hkv, D, slots, tokens, k, v, s)
                : launch_read_t<F16>(cache, num_pages, page_shift, hkv, D, slots, tokens, k, v, s);
}

}  // namespace bq
