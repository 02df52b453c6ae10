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
// with a bf16 output the high part, three bits more than the output has, is
// enough (its error against 64 bits grows by under 1 %).
// The reference maximum is raised only when a score passes it by 2^8, and
// then for all lanes of the row; sums and accumulators are fp32.  p sv is
// brought into fp16's range by the largest V scale that the row has seen.
//
// Long sequences are split over workgroups (and over a workgroup's
// wavefronts, joined through LDS); a second kernel joins the parts in order.
#include "attn_kv4.h"

namespace bq {
namespace {

// Codes and parameters of 32 tokens, K or V.
template <int D>
struct Tile {
    static constexpr int kW = D / 32;  // dwords of codes per lane and 16 tokens
    uint32_t c[2][kW];
    u4 par[2];
};

// Where the two 16-token halves of a tile lie.
struct Place {
    const uint8_t *base[2];  // the kv head's part of the page
    uint32_t in[2];          // first token in the page
    int lim[2];              // tokens at or past lim are not there
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

// Pages of the two 16-token halves of a tile; past the end the first half's.
__device__ __forceinline__ void load_pages(int (&page)[2], const AttnKv4Args &p, const int *table, int t, int hi)
{
    page[0] = table[t >> p.page_shift];
    page[1] = table[(t + 16 < hi ? t + 16 : t) >> p.page_shift];
}

template <int D>
__device__ __forceinline__ Place place_of(const AttnKv4Args &p, const int (&pages)[2], int head, int t, int hi)
{
    Place x;
    const int P = 1 << p.page_shift;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        // 16 tokens lie in one page
        const int tt = t + 16 * s < hi ? t + 16 * s : t;
        const bool there = (uint32_t)pages[s] < (uint32_t)p.num_pages;
        x.lim[s] = there ? hi : 0;
        x.base[s] = p.cache + (int64_t)((int64_t)(there ? pages[s] : 0) * p.hkv + head) * (P * (D + 8));
        x.in[s] = tt & (P - 1);
    }
    return x;
}

template <int D>
__device__ __forceinline__ void load_k(Tile<D> &x, const Place &at, int page_shift, int lane)
{
    const uint32_t g = lane >> 4, m = lane & 15;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        const uint8_t *kb = at.base[s] + at.in[s] * (D / 2);
        if constexpr (D == 64) {
            load_dwords<2>(x.c[s], kb + (m * 32 + g * 8));
        } else if constexpr (D == 128) {
            load_dwords<4>(x.c[s], kb + (m * 64 + g * 16));
        } else {
            load_dwords<4>(x.c[s], kb + (m * 128 + g * 32));
            load_dwords<4>(x.c[s] + 4, kb + (m * 128 + g * 32 + 16));
        }
        x.par[s] = *(const u4 *)(at.base[s] + (D << page_shift) + at.in[s] * 4 + g * 16);
    }
}

template <int D>
__device__ __forceinline__ void load_v(Tile<D> &x, const Place &at, int page_shift, int lane)
{
    const uint32_t g = lane >> 4, m = lane & 15;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        const uint8_t *vb = at.base[s] + ((D / 2) << page_shift) + at.in[s] * (D / 2);
        if constexpr (D == 64) {
            load_dwords<2>(x.c[s], vb + (g * 128 + m * 8));
        } else if constexpr (D == 128) {
            load_dwords<4>(x.c[s], vb + (g * 256 + m * 16));
        } else {
            load_dwords<4>(x.c[s], vb + (g * 512 + m * 16));
            load_dwords<4>(x.c[s] + 4, vb + (g * 512 + 256 + m * 16));
        }
        x.par[s] = *(const u4 *)(at.base[s] + ((D + 4) << page_shift) + at.in[s] * 4 + g * 16);
    }
}

constexpr uint32_t kM0 = 0x000f000fu, kM4 = 0x00f000f0u;

// Codes at bits 0..3 (or, high, 4..7) of each half as the fp16 integers u - 8:
// 0x6400 | u = 1024 + u, and (1024 + 16 u) / 16 - 72, both exact.
// `bias` is 0x64006400 held in a register, which lets mask and merge be one
// instruction.
__device__ __forceinline__ uint32_t centred(bool high, uint32_t w, uint32_t bias)
{
    const h2 x = __builtin_bit_cast(h2, (w & (high ? kM4 : kM0)) | bias);
    const h2 s = {(_Float16)0.0625f, (_Float16)0.0625f}, c = {(_Float16)-72.0f, (_Float16)-72.0f};
    const h2 b = {(_Float16)-1032.0f, (_Float16)-1032.0f};
    return __builtin_bit_cast(uint32_t, high ? __builtin_elementwise_fma(x, s, c) : x + b);
}

// RT tiles of 16 query rows of one wavefront.
template <typename T, int D, int RT>
struct Wave {
    static constexpr int kQ = D / 64;   // operand pairs of the queries
    static constexpr int kMT = D / 16;  // output tiles of 16 channels
    static constexpr bool kLow = !T::kBf16;
    u4 q0[RT][kQ], q4[RT][kQ];
    // score = a1 (sk (16 s0 + s4) + b1 mk), in powers of two; a1 >= 0
    float a1[RT], b1[RT];
    float mt[RT], mref[RT];  // the scores' reference maximum, and what is subtracted of them: mt - shift
    float l[RT], z[RT];
    float cap[RT];           // V scales up to cap = 2^(6 - shift) leave p sv 2^shift within fp16; 0 at first, with shift 0
    int pos[RT];             // the rows' positions (or nodes)
    u4 ph[RT], pl[RT];       // p sv of the tile, high and low parts
    f4 o[RT][kMT];

    // w: the lane's quarter of a query row, as loaded
    __device__ __forceinline__ void init_row(int r, uint32_t (&w)[D / 8], float scale)
    {
        float sum = 0.0f, top = 0.0f;
        if (scale < 0.0f) {  // the sign goes to the query
#pragma unroll
            for (int i = 0; i < D / 8; ++i)
                w[i] ^= 0x80008000u;
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
        float back = 1.0f, f = 1.0f;
        if constexpr (T::kBf16) {
            // a power of two brings the row into fp16's range: bf16's eight
            // bits survive down to 2^-24 of the row's largest value
            const uint32_t e = max((__float_as_uint(top) >> 23) & 255u, 11u);
            f = e < 255u ? __uint_as_float((264u - e) << 23) : 1.0f;
            back = e < 255u ? __uint_as_float((e - 10u) << 23) : 1.0f;
#pragma unroll
            for (int i = 0; i < D / 8; ++i)
                w[i] = F16::from_f32(T::to_f32(w[i] & 0xffffu) * f) | (uint32_t)F16::from_f32(T::to_f32(w[i] >> 16) * f) << 16;
        }
        // codes 0, 4 and 2, 6 of a dword sit at bits 0..3 of a half, 1, 5 and 3, 7 at 4..7
#pragma unroll
        for (int i = 0; i < kQ; ++i) {
            const uint32_t *c = w + 8 * i;
            q0[r][i] = (u4){pack_lo(c[0], c[2]), pack_lo(c[1], c[3]), pack_lo(c[4], c[6]), pack_lo(c[5], c[7])};
            q4[r][i] = (u4){pack_hi(c[0], c[2]), pack_hi(c[1], c[3]), pack_hi(c[4], c[6]), pack_hi(c[5], c[7])};
        }
        a1[r] = fmaxf(back * 0x1p20f * (fabsf(scale) * kLog2e), 0x1p-120f);  // a masked score is -inf a1
        b1[r] = sum * f * 0x1p-20f;
        mt[r] = mref[r] = kNoMax;
        l[r] = z[r] = cap[r] = 0.0f;
#pragma unroll
        for (int i = 0; i < kMT; ++i)
            o[r][i] = (f4){0, 0, 0, 0};
    }

    // Scores of a tile, over a1.
    __device__ __forceinline__ void scores(const Tile<D> &x, float (&s)[RT][8], float nothing)
    {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            f4 s0[RT], s4[RT];
#pragma unroll
            for (int r = 0; r < RT; ++r)
                s0[r] = s4[r] = (f4){0, 0, 0, 0};
#pragma unroll
            for (int i = 0; i < kQ; ++i) {
                const uint32_t a = x.c[h][2 * i], b = x.c[h][2 * i + 1];
                const uint32_t a8 = a >> 8, b8 = b >> 8;
                const u4 c0 = {a & kM0, a8 & kM0, b & kM0, b8 & kM0}, c4 = {a & kM4, a8 & kM4, b & kM4, b8 & kM4};
#pragma unroll
                for (int r = 0; r < RT; ++r) {
                    s0[r] = F16::mma(c0, q0[r][i], s0[r]);
                    s4[r] = F16::mma(c4, q4[r][i], s4[r]);
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float sk = half_bits(x.par[h][i] & 0xffffu), mk = half_bits(x.par[h][i] >> 16);
#pragma unroll
                for (int r = 0; r < RT; ++r)
                    s[r][4 * h + i] = __builtin_fmaf(s0[r][i] * 16.0f + s4[r][i], sk, __builtin_fmaf(mk, b1[r], nothing));
            }
        }
    }

    // p of a tile and its V parameters; masked if not every row sees every key.
    // TREE: `sees` has a bit for each key of the tile and row.
    template <bool TREE>
    __device__ __forceinline__ void values(const Tile<D> &x, float (&s)[RT][8], bool masked, int t, const int (&lim)[2],
                                           int window, int lane, const uint32_t (&sees)[RT])
    {
        float sv[8], mv[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t par = x.par[j >> 2][j & 3];
            sv[j] = half_bits(par & 0xffffu);
            mv[j] = half_bits(par >> 16) + 8.0f * sv[j];
        }
        if (masked) {
            const int g = lane >> 4;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int tok = t + 16 * (j >> 2) + 4 * g + (j & 3);
                const bool there = tok < lim[j >> 2];
                // What lies in a masked place may be anything: parameters that are
                // no numbers become 0, and make NaN only where a row sees them.
                const bool number = __builtin_isfinite(mv[j]) && __builtin_isfinite(sv[j]);
#pragma unroll
                for (int r = 0; r < RT; ++r) {
                    const bool on = there && (TREE ? (sees[r] >> (16 * (j >> 2) + 4 * g + (j & 3))) & 1
                                                   : tok <= pos[r] && (window <= 0 || tok > pos[r] - window));
                    s[r][j] = on ? (number ? s[r][j] : __builtin_nanf("")) : -__builtin_inff();
                }
                sv[j] = there && number ? sv[j] : 0.0f;
                mv[j] = there && number ? mv[j] : 0.0f;
            }
        }
        float vtop = fabsf(sv[0]);
#pragma unroll
        for (int j = 1; j < 8; ++j)
            vtop = fmaxf(vtop, fabsf(sv[j]));
        bool raise = false;
        float top[RT];
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            top[r] = s[r][0];
#pragma unroll
            for (int j = 1; j < 8; ++j)
                top[r] = fmaxf(top[r], s[r][j]);
            raise |= vtop > cap[r] || top[r] * a1[r] > mt[r] + 8.0f;
        }
        if (__builtin_expect(__any(raise), 0)) {
            // Each row by the keys that it sees (the others' scores are -inf): no
            // other key, and nothing that another row needs, changes a bit of it.
#pragma unroll
            for (int r = 0; r < RT; ++r) {
                float seen = 0.0f;
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    seen = fmaxf(seen, s[r][j] > -__builtin_inff() ? fabsf(sv[j]) : 0.0f);
#pragma unroll
                for (int off = 16; off < 64; off <<= 1) {
                    top[r] = fmaxf(top[r], __shfl_xor(top[r], off, 64));
                    seen = fmaxf(seen, __shfl_xor(seen, off, 64));
                }
                const bool wider = seen > cap[r];
                if (wider || top[r] * a1[r] > mt[r] + 8.0f)
                    mt[r] = fmaxf(mt[r], top[r] * a1[r]);
                // 2 to 4 times the scale
                const uint32_t e = (__float_as_uint(fminf(seen, 65504.0f)) >> 23) + 2u;
                cap[r] = wider ? __uint_as_float(e << 23) : cap[r];
                const float shift = cap[r] > 0.0f ? 133.0f - (float)(__float_as_uint(cap[r]) >> 23) : 0.0f;
                const float now = mt[r] - shift, f = __builtin_amdgcn_exp2f(mref[r] - now);  // 1 for a row that needs nothing
                mref[r] = now;
                l[r] *= f;
                z[r] *= f;
#pragma unroll
                for (int i = 0; i < kMT; ++i)
                    o[r][i] *= f;
            }
        }
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int j = 0; j < 8; j += 2) {
                const float p0 = __builtin_amdgcn_exp2f(s[r][j] * a1[r] - mref[r]);
                const float p1 = __builtin_amdgcn_exp2f(s[r][j + 1] * a1[r] - mref[r]);
                l[r] += p0;
                l[r] += p1;
                z[r] += p0 * mv[j];
                z[r] += p1 * mv[j + 1];
                const float v0 = p0 * sv[j], v1 = p1 * sv[j + 1];
                const h2 hi = {(_Float16)v0, (_Float16)v1};
                ph[r][j / 2] = __builtin_bit_cast(uint32_t, hi);
                if constexpr (kLow)
                    pl[r][j / 2] = __builtin_bit_cast(uint32_t, (h2){(_Float16)(v0 - (float)hi[0]), (_Float16)(v1 - (float)hi[1])});
            }
    }

    // o += p sv (u - 8)
    __device__ __forceinline__ void products(const Tile<D> &x, uint32_t bias)
    {
#pragma unroll
        for (int c = 0; c < (D == 256 ? 2 : 1); ++c) {
            // pairs of tokens of the same channels: codes 0..3 (and 4..7) of a unit
            u4 lo, hi;
            if constexpr (D == 64) {
                lo = (u4){x.c[0][0], x.c[0][1], x.c[1][0], x.c[1][1]};
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t a = x.c[i >> 1][4 * c + 2 * (i & 1)], b = x.c[i >> 1][4 * c + 2 * (i & 1) + 1];
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
                    a[i] = centred(j & 1, (j & 2) ? w[i] >> 8 : w[i], bias);
#pragma unroll
                for (int r = 0; r < RT; ++r) {
                    f4 &acc = o[r][8 * c + j];
                    acc = F16::mma(a, ph[r], acc);
                    if constexpr (kLow)
                        acc = F16::mma(a, pl[r], acc);
                }
            }
        }
    }

    // Sums of the rows over their four lanes; the accumulators take in z.
    __device__ __forceinline__ void finish()
    {
#pragma unroll
        for (int r = 0; r < RT; ++r) {
#pragma unroll
            for (int off = 16; off < 64; off <<= 1) {
                l[r] += __shfl_xor(l[r], off, 64);
                z[r] += __shfl_xor(z[r], off, 64);
            }
#pragma unroll
            for (int i = 0; i < kMT; ++i)
                o[r][i] += z[r];
        }
    }
};

// WAVES: kWaves, or kMany where `many_waves` says so.
template <typename T, int D, int RT, int WAVES, bool TREE>
__global__ __launch_bounds__(64 * WAVES) void attn_kv4_kernel(const AttnKv4Args p)
{
    constexpr int DH = D > 128 ? 128 : D;  // channels joined at a time
    constexpr int ROWS = 16 * RT;
    __shared__ float so[WAVES][16][DH + 4];
    __shared__ float sm[WAVES][ROWS], sl[WAVES][ROWS];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int split = blockIdx.x % p.nsplit, item = blockIdx.x / p.nsplit;
    const int tile = item % p.row_tiles;
    const int head = item / p.row_tiles % p.hkv;
    const int b = item / p.row_tiles / p.hkv;
    const QueryRows qr = query_rows(p, b);
    const int q0 = qr.first, rows = qr.count * p.group;
    if (tile * ROWS >= rows)
        return;
    // the queries are on their way while the keys are found
    uint32_t qw[RT][D / 8];
#pragma unroll
    for (int i = 0; i < RT; ++i) {
        const int row = min(tile * ROWS + 16 * i + (lane & 15), rows - 1);
        const int qi = row / p.group, hg = row - qi * p.group;
        const uint16_t *q = (const uint16_t *)p.q + (int64_t)(q0 + qi) * p.q_stride + (head * p.group + hg) * D;
#pragma unroll
        for (int k = 0; k < D / 32; ++k)
            load_dwords<4>(qw[i] + 4 * k, (const uint8_t *)(q + (lane >> 4) * (D / 4) + 8 * k));
    }
    const Rows r = rows_of<ROWS, TREE>(p, b, tile);
    const int start = r.lo + split * r.chunk, end = min(start + r.chunk, r.hi);
    if (split > 0 && start >= r.hi)
        return;

    Wave<T, D, RT> w;
#pragma unroll
    for (int i = 0; i < RT; ++i) {
        const int row = tile * ROWS + 16 * i + (lane & 15);
        w.pos[i] = TREE ? min(row, r.rows - 1) / p.group : row < r.rows ? r.base + row / p.group : r.pos_max;
        w.init_row(i, qw[i], p.scale);
    }
    const int *table = p.block_table + (int64_t)b * p.max_blocks;
    constexpr int kStep = WAVES * kTile;
    int t = start + wave * kTile;
    if (t < end) {
        // K of the next tile is loaded when the scores have used this one's, V
        // when the products have; page numbers come a tile earlier.
        uint32_t bias = 0x64006400u;
        asm volatile("" : "+v"(bias));
        // -0 that the compiler does not know: a product with a 16-bit factor then
        // is one mixed multiply-add instead of a conversion and a multiply
        float nothing = -0.0f;
        asm volatile("" : "+v"(nothing));
        Tile<D> k, v;
        int pages[2];
        load_pages(pages, p, table, t, end);
        Place at = place_of<D>(p, pages, head, t, end);
        load_k<D>(k, at, p.page_shift, lane);
        load_v<D>(v, at, p.page_shift, lane);
        load_pages(pages, p, table, min(t + kStep, end - 1), end);
        for (;;) {
            const int u = t + kStep;
            const int lim[2] = {at.lim[0], at.lim[1]};
            float s[RT][8];
            w.scores(k, s, nothing);
            if (u < end) {
                at = place_of<D>(p, pages, head, u, end);
                load_k<D>(k, at, p.page_shift, lane);
                load_pages(pages, p, table, min(u + kStep, end - 1), end);
            }
            const bool whole = t + kTile <= min(min(lim[0], lim[1]), r.pos_min + 1) && (p.window <= 0 || t > r.pos_max - p.window);
            uint32_t sees[RT] = {};
            if constexpr (TREE)
                if (!whole)
#pragma unroll
                    for (int i = 0; i < RT; ++i)
                        sees[i] = tree_row(p, r, qr.len, w.pos[i]).keys(t, r.base);
            w.template values<TREE>(v, s, !whole, t, lim, p.window, lane, sees);
            w.products(v, bias);
            if (u >= end)
                break;
            load_v<D>(v, at, p.page_shift, lane);
            t = u;
        }
    }
    w.finish();

    // join the wavefronts: thread (row, c) takes DH/16 channels
    const int g = lane >> 4, m = lane & 15;
    if (g == 0) {
#pragma unroll
        for (int i = 0; i < RT; ++i) {
            sm[wave][16 * i + m] = w.mref[i];
            sl[wave][16 * i + m] = w.l[i];
        }
    }
    const int jr = threadIdx.x >> 4 & 15, jc = threadIdx.x & 15;
    constexpr int CH = DH / 16;
#pragma unroll
    for (int i = 0; i < RT; ++i) {
        const int orow = tile * ROWS + 16 * i + jr;
        const int oqi = orow / p.group, ohg = orow - oqi * p.group;
        const int64_t orow_at = (int64_t)(r.q0 + oqi) * p.hq + head * p.group + ohg;
        const int64_t part = (item * (int64_t)p.nsplit + split) * ROWS + 16 * i + jr;
#pragma unroll
        for (int c = 0; c < D / DH; ++c) {
            if (i || c)
                __syncthreads();
#pragma unroll
            for (int k = 0; k < 4; ++k)
#pragma unroll
                for (int j = 0; j < CH; j += 4) {
                    const f4 *o = &w.o[i][8 * c + j];
                    *(float4 *)&so[wave][m][(g * 4 + k) * CH + j] = make_float4(o[0][k], o[1][k], o[2][k], o[3][k]);
                }
            __syncthreads();
            if (WAVES > kWaves && threadIdx.x >= 256)
                continue;  // 256 threads join
            float mm = sm[0][16 * i + jr];
#pragma unroll
            for (int k = 1; k < WAVES; ++k)
                mm = fmaxf(mm, sm[k][16 * i + jr]);
            float l = 0.0f, acc[CH] = {};
#pragma unroll
            for (int k = 0; k < WAVES; ++k) {
                const float f = __builtin_amdgcn_exp2f(sm[k][16 * i + jr] - mm);
                l += f * sl[k][16 * i + jr];
#pragma unroll
                for (int j = 0; j < CH; ++j)
                    acc[j] += f * so[k][jr][jc * CH + j];
            }
            if (orow < r.rows) {
                if (WAVES > kWaves || p.nsplit == 1) {
                    uint16_t *dst = (uint16_t *)p.out + orow_at * D + c * DH + jc * CH;
                    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
                    uint32_t y[CH / 2];
#pragma unroll
                    for (int j = 0; j < CH; j += 2)
                        y[j / 2] = T::from_f32(acc[j] * inv) | (uint32_t)T::from_f32(acc[j + 1] * inv) << 16;
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
}

// Sequences that are not split, one workgroup a CU at most, are walked by eight
// wavefronts a workgroup: 1 sequence of 700 keys, 8 kv heads of 128, 9.0 us
// against 10.3 with four; 32 of 1024 12.6 against 14.6; 64 of them (512
// workgroups) 24.0 against 20.7.  Not where a wavefront holds more than 128
// channels of 16 rows, whose join outlasts the gain (D = 256: 40 keys 7.6
// against 6.4, 700 keys 14.0 against 13.4).
bool many_waves(int D, int rt, int64_t items) { return D * rt <= 128 && items <= 256; }

template <typename T, int D, int RT, bool TREE>
hipError_t launch_t(const AttnKv4Args &p, hipStream_t s)
{
    const int64_t items = (int64_t)p.batch * p.hkv * p.row_tiles;
    if (!grid_fits(items * p.nsplit, 64 * kWaves) || (p.nsplit > 1 && !grid_fits(items * p.join_rows, 256)))
        return kGridTooLarge;
    if constexpr (D * RT <= 128)
        if (p.nsplit == 1 && many_waves(D, RT, items)) {
            attn_kv4_kernel<T, D, RT, kMany, TREE><<<dim3((unsigned)items), 64 * kMany, 0, s>>>(p);
            return hipGetLastError();
        }
    attn_kv4_kernel<T, D, RT, kWaves, TREE><<<dim3((unsigned)(items * p.nsplit)), 64 * kWaves, 0, s>>>(p);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || p.nsplit == 1)
        return e;
    return launch_join<T, D, RT, TREE>(p, items, s);
}

template <typename T, bool TREE>
hipError_t launch_d(const AttnKv4Args &p, int D, int rt, hipStream_t s)
{
    if (D == 64)
        return rt == 2 ? launch_t<T, 64, 2, TREE>(p, s) : launch_t<T, 64, 1, TREE>(p, s);
    if (D == 128)
        return rt == 2 ? launch_t<T, 128, 2, TREE>(p, s) : launch_t<T, 128, 1, TREE>(p, s);
    return launch_t<T, 256, 1, TREE>(p, s);
}

}  // namespace

AttnKv4Plan attn_kv4_plan(int64_t batch, int64_t max_q_len, int q_heads, int kv_heads, int D, int64_t max_len)
{
    // Two row tiles a wavefront where there are two: one decode of the codes
    // serves both (301 queries of 4 heads a kv head, D = 64: 43.5 against 45.7
    // us; 7 of 8, D = 128: 35.0 against 38.6).
    const int64_t rows = max_q_len * (q_heads / kv_heads), seqs = batch * kv_heads;
    const int rt = D < 256 && rows > 16 ? 2 : 1;
    AttnKv4Plan a;
    a.rt = rt;
    a.row_tiles = (rows + 16 * rt - 1) / (16 * rt);
    const int64_t items = seqs * a.row_tiles;
    // Splits until the workgroups that the registers let the 256 CUs hold are
    // all there, but no more: they then run in one go and end together (3 x 8
    // sequences and heads of 100001 keys: 76.5 us with 768 workgroups, 82 with
    // 1536, 89 with 576).
    const int64_t slots = 256 * (D == 256 || (D == 128 && rt == 2) ? 2 : D == 64 && rt == 1 ? 4 : 3);
    // Up to 1024 keys are not split: the second kernel costs what the shorter
    // first one gains, or nearly, and its launch costs a caller more (8 kv heads
    // of 128, in a graph: 1 sequence of 700 keys 8.9 us, split 9.1, of 1024 9.9
    // and 9.0, 8 of 1024 11.4 and 12.3; called from Python 9.2 and 12.1, 10.1 and
    // 12.2, 11.2 and 12.2; of 1500 in a graph 13.5 and 10.5).  Where eight
    // wavefronts a workgroup fill half of the CUs, up to 2048 keys (16 sequences
    // of 2048 18.1 us either way, 32 20.7 against 25.6; 16 of 4096 33.1 against
    // 26.7).
    const int64_t whole = many_waves(D, rt, items) && items >= 128 ? 2048 : 1024;
    const int64_t step = kTile * kWaves;
    const int64_t want = items > 0 && max_len > whole ? slots / items : 1, most = (max_len + step - 1) / step;
    const int64_t n = want < most ? want : most;
    a.nsplit = (int)(n < 1 ? 1 : n > 64 ? 64 : n);
    a.part_rows = a.nsplit > 1 ? items * a.nsplit * 16 * rt : 0;
    return a;
}

hipError_t launch_attn_kv4(AttnKv4Args &p, int D, int rt, bool bf16, hipStream_t s)
{
    const int64_t rows = (int64_t)p.max_q_len * p.group;
    p.join_rows = (int)(rows < 16 * rt ? rows : 16 * rt);
    if (p.tree_mask)
        return bf16 ? launch_d<BF16, true>(p, D, rt, s) : launch_d<F16, true>(p, D, rt, s);
    return bf16 ? launch_d<BF16, false>(p, D, rt, s) : launch_d<F16, false>(p, D, rt, s);
}

}  // namespace bq
