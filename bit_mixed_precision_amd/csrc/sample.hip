// Sampling with temperature, top-k, top-p and min-p from given random numbers.
//
// Every choice is made on whole numbers: a logit's order by its bits (key),
// its weight w = 2^-y, y = (max - x) log2(e) / temperature in 64 bits, as a
// multiple of 2^-frac (units).  Sums of units are exact in 64 bits, so no order
// of additions, atomics among them, changes a result, and a token is the
// definition's except where two sums lie within the weights' own rounding,
// 2^-45 of the largest for a vocabulary of 2^17 (fp32 sums would move borders
// between tokens that weigh 2^-17 of the whole).
//
// What is kept is a limit in the order of the tokens (key descending, index
// ascending): its last token's key and index.
//
// Rows of up to 32761 16-bit or 32765 fp32 logits (2^15, less what an unaligned
// row has in its first and last vector) are held in a workgroup's registers, in one
// kernel; the others take four:
//   greatest   the greatest logit of every group of a row's lanes;
//   weigh      a row with a top_k of at most as many as there are groups (48 to
//              256, by the row's length, the type and the number of rows): no
//              token below the top_k-th greatest group can be kept, those from
//              it on, a few more than top_k, are listed, of the few lanes only
//              whose greatest logit is one of them.  A row without top_k: the units
//              of each eighth of an octave of weight, per workgroup and row;
//   gather     lists the tokens of the eighth of an octave in which such a row's limit
//              lies;
//   draw       one workgroup a row: ends the kept ones of the listed tokens; the
//              sums over the others give the part of the row that the drawn token
//              is in, which is read again.
// The one kernel takes the same steps, a top_k of up to 256 (of any number up to
// 1024 in a row of up to 4096 tokens) by groups.  Without a workspace, where a list
// is too short (a row of equal logits), and for a greater top_k, one workgroup
// selects over the row itself, eight bits of key at a time.
//
// 1 x 32000 fp16 in the one kernel 21.9 us (in the four 28.4), with top-k 40 17.9,
// with top-p or min-p alone 36 to 47; 64 x 131072 bf16 with top-p: greatest 8.6, weigh
// 16.0 (25 operations in 64 bits a token), gather 13.9, draw 25.6; 487 x 100003 fp32
// with all settings: 45 (4.3 TB/s), 31 (all lanes' vectors, and the limit by ranks of
// the groups: 53), 17, 39.  One workgroup a row, each over the whole of it: 139, 528
// and 1083, and so, past the groups, for one top_k more: 1 x 32768 fp16 has 68 groups,
// top_k 40 21.4 us, 70 87.5; 64 x 131072 bf16 88, 70 35.5, 100 276.
//
// Most of a draw's time is one workgroup's way through code and dependent loads:
// code that runs once costs the instructions' way from memory, so loops are not
// unrolled there.
#include "bq_decode_internal.h"
#include "dtype16.h"

// A token's weight has the same bits wherever it is computed (a part's sum and the
// row that is read again for the drawn token have to agree to the last unit): products
// and sums are fused only where fma is written.
#pragma clang fp contract(off)

namespace bq {
namespace {

typedef unsigned long long u64;

constexpr int kThreads = 1024, kWaves = kThreads / 64;  // of a workgroup that has a row
constexpr int kPart = 4;                                // wavefronts of one that has a part of a row
constexpr uint32_t kNone = 0x007fffffu;                 // keys up to that of -infinity are no tokens
constexpr int kOct = 384;                               // eighths of octaves of weight: 48 octaves, past which nothing is a unit
constexpr int kGroups = 256;                            // groups of a row, at most
constexpr int kList = 6144;                             // tokens of a row that are listed, at most
constexpr int kFound = 1024;                            // of them by one workgroup

// The order of the numbers as unsigned integers; -0 as 0, NaN below all.
__device__ __forceinline__ uint32_t key_of(float x)
{
    const uint32_t b = __float_as_uint(x + 0.0f);
    return x != x ? 0u : b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t key)
{
    return __uint_as_float(key & 0x80000000u ? key ^ 0x80000000u : ~key);
}
// A token as one number, in the order of tokens the greater the earlier.
__device__ __forceinline__ u64 order_of(uint32_t key, int index) { return (u64)key << 32 | ~(uint32_t)index; }
__device__ __forceinline__ uint32_t key_in(u64 order) { return (uint32_t)(order >> 32); }
__device__ __forceinline__ int index_in(u64 order) { return (int)~(uint32_t)order; }

// A row of logits, as vectors of 16 bytes from the aligned address at or before
// its start; of the first and last one only what lies in the row is read.
template <int TYPE>
struct Row {
    static constexpr int kE = TYPE == 2 ? 4 : 8;  // tokens of a vector
    static constexpr int kSize = TYPE == 2 ? 4 : 2;
    const uint8_t *base;
    int lead, vocab;  // tokens of the first vector before the row

    __device__ __forceinline__ Row(const SampleArgs &p, int b)
    {
        const uint8_t *row = (const uint8_t *)p.logits + (int64_t)b * p.row_stride * kSize;
        lead = ((uintptr_t)row & 15) / kSize;
        base = row - lead * kSize;
        vocab = p.vocab;
    }
    __device__ __forceinline__ int vectors() const { return (lead + vocab + kE - 1) / kE; }
    __device__ __forceinline__ static float value(uint32_t bits)
    {
        if constexpr (TYPE == 2)
            return __uint_as_float(bits);
        else
            return TYPE == 1 ? BF16::to_f32(bits & 0xffffu) : F16::to_f32(bits & 0xffffu);
    }
    __device__ __forceinline__ static float value(const u4 &x, int e)
    {
        if constexpr (TYPE == 2)
            return __uint_as_float(x[e]);
        else
            return value(x[e >> 1] >> (16 * (e & 1)));
    }
    // Drops the first token of a vector; `next` becomes its last.
    __device__ __forceinline__ static void shift(u4 &x, uint32_t next)
    {
        if constexpr (TYPE == 2) {
            x[0] = x[1];
            x[1] = x[2];
            x[2] = x[3];
            x[3] = next;
        } else {
            x[0] = __builtin_amdgcn_alignbit(x[1], x[0], 16);
            x[1] = __builtin_amdgcn_alignbit(x[2], x[1], 16);
            x[2] = __builtin_amdgcn_alignbit(x[3], x[2], 16);
            x[3] = __builtin_amdgcn_alignbit(next, x[3], 16);
        }
    }
    // Raw vector v; what is not in the row is -infinity.
    __device__ __forceinline__ u4 load(int v) const
    {
        const int first = v * kE - lead;
        if (first >= 0 && first + kE <= vocab)
            return *(const u4 *)(base + (int64_t)v * 16);
        u4 x = {};
#pragma unroll 1
        for (int i = 0; i < kE; ++i) {
            const bool in = first + i >= 0 && first + i < vocab;
            if constexpr (TYPE == 2)
                shift(x, in ? ((const uint32_t *)base)[v * kE + i] : 0xff800000u);
            else
                shift(x, in ? ((const uint16_t *)base)[v * kE + i] : TYPE == 1 ? 0xff80u : 0xfc00u);
        }
        return x;
    }
    // f(index, key) for the tokens of vector v.
    template <typename F>
    __device__ __forceinline__ void each_token(int v, u4 x, F f) const
    {
        int at = v * kE - lead;
#pragma unroll 1
        for (int i = 0; i < kE; ++i, ++at) {
            f(at, key_of(value(x[0])));
            shift(x, 0);
        }
    }
    // f(index, key) for those whose bits are set.
    template <typename F>
    __device__ __forceinline__ void each_set(int v, const u4 &x, uint32_t on, F f) const
    {
#pragma unroll 1
        for (; on; on &= on - 1) {
            const int e = __ffs(on) - 1, w = TYPE == 2 ? e : e >> 1;
            const uint32_t lo = w & 1 ? x[1] : x[0], hi = w & 1 ? x[3] : x[2], word = w & 2 ? hi : lo;
            f(v * kE + e - lead, key_of(value(TYPE == 2 ? word : word >> (16 * (e & 1)))));
        }
    }
    // The greatest number of a vector; NaN is none.
    __device__ __forceinline__ static float greatest(const u4 &x, float m)
    {
#pragma unroll
        for (int e = 0; e < kE; ++e)
            m = fmaxf(m, value(x, e));
        return m;
    }
    // Bits of the numbers of at least `least`.
    __device__ __forceinline__ static uint32_t at_least(const u4 &x, float least)
    {
        uint32_t on = 0;
#pragma unroll
        for (int e = 0; e < kE; ++e)
            on |= (uint32_t)(value(x, e) >= least) << e;
        return on;
    }
    // The same for the whole row, by a workgroup of kThreads.
    template <typename F>
    __device__ __forceinline__ void each(F f) const
    {
        const int n = vectors();
        for (int v = threadIdx.x; v < n; v += 4 * kThreads) {
            u4 x[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (v + kThreads * i < n)
                    x[i] = load(v + kThreads * i);
#pragma unroll 1
            for (int at = v; at < min(v + 4 * kThreads, n); at += kThreads) {
                each_token(at, x[0], f);
                x[0] = x[1];
                x[1] = x[2];
                x[2] = x[3];
            }
        }
    }
};

// Weights of a row's tokens.
struct Scale {
    double max, c;      // y = (max - x) c / 8: c counts eighths of octaves
    int frac;
    const double *mid;  // [kOct] weight of the middle of each eighth of an octave, in units

    // Eighths of octaves below the greatest.
    __device__ __forceinline__ double eighths(float x) const
    {
        return x == (float)max ? 0.0 : (max - (double)x) * c;  // not infinity - infinity
    }
    __device__ __forceinline__ double eighths(uint32_t key) const { return eighths(value_of(key)); }
    // 2^-(q / 8) in units, to the nearest: from the middle of the eighth of an octave
    // `bin` = floor(q) on by the series, whose remainder is below 2^-50.
    __device__ __forceinline__ u64 units(double q, int bin) const
    {
        constexpr double l = 0.693147180559945309417 / 8;
        constexpr double c2 = l * l / 2, c3 = c2 * l / 3, c4 = c3 * l / 4, c5 = c4 * l / 5, c6 = c5 * l / 6, c7 = c6 * l / 7;
        const double r = ((double)bin + 0.5) - q;
        double s = c7;
        s = __builtin_fma(s, r, c6);
        s = __builtin_fma(s, r, c5);
        s = __builtin_fma(s, r, c4);
        s = __builtin_fma(s, r, c3);
        s = __builtin_fma(s, r, c2);
        s = __builtin_fma(s, r, l);
        s = __builtin_fma(s, r, 1.0);
        // with 2^52 added, the number's low bits are the rounded integer
        const u64 n = (u64)__double_as_longlong(__builtin_fma(s, mid[bin], 0x1p52)) & 0xfffffffffffffull;
        return q == 0.0 ? 1ull << frac : n;
    }
    __device__ __forceinline__ u64 units(double q) const { return q < kOct ? units(q, (int)q) : 0; }
    __device__ __forceinline__ u64 units_of(uint32_t key) const { return units(eighths(key)); }
};

// Fills Scale::mid.
__device__ __forceinline__ void fill_mid(double *mid, int frac)
{
    for (int i = threadIdx.x; i < kOct; i += blockDim.x) {
        // 2^-1/16, and half, quarter and eighth of an octave from there
        double x = 0.957603280698573646936;
        x *= i & 4 ? 0.707106781186547524401 : 1.0;
        x *= i & 2 ? 0.840896415253714543031 : 1.0;
        x *= i & 1 ? 0.917004043204671231744 : 1.0;
        mid[i] = x * __hiloint2double((1023 + frac - (i >> 3)) << 20, 0);
    }
}

// A row's settings.
struct Settings {
    bool greedy, has_p;
    int top_k;  // 0: off
    float top_p, min_p, u;

    __device__ __forceinline__ Settings(const SampleArgs &p, int b)
    {
        const float t = p.temperature ? p.temperature[b] : 1.0f;
        const int k = p.top_k ? p.top_k[b] : 0;
        top_p = p.top_p ? p.top_p[b] : 1.0f;
        min_p = p.min_p ? p.min_p[b] : 0.0f;
        u = p.u[b];
        temperature = fminf(t, 3.402823466e38f);
        greedy = !(t > 0.0f);
        top_k = k > 0 && k < p.vocab ? k : 0;
        has_p = top_p < 1.0f;
    }
    __device__ __forceinline__ Scale scale(uint32_t top, int frac, const double *mid) const
    {
        return {value_of(top), 8 * 1.4426950408889634074 / (double)temperature, frac, mid};
    }
    // Eighths of octaves within which min-p keeps tokens.
    __device__ __forceinline__ double far() const
    {
        return min_p > 0.0f ? 8 * (0x1p-53 - log2(fmin((double)min_p, 1.0))) : 1e300;
    }
    // The sum that top-p must reach, and the one that the drawn token must pass.
    __device__ __forceinline__ u64 reach(u64 total) const
    {
        return max((u64)ceil((double)fmaxf(top_p, 0.0f) * (double)total), 1ull);
    }
    __device__ __forceinline__ u64 pass(u64 total) const
    {
        return u < 1.0f ? min(total - 1, (u64)floor((double)fmaxf(u, 0.0f) * (double)total)) : total - 1;
    }
    // Whether weigh lists the tokens from the top_k-th greatest group on, or sums up
    // the units; else the row itself is selected over.
    __device__ __forceinline__ bool lists(int groups) const { return top_k && top_k <= groups; }
    __device__ __forceinline__ bool sums() const { return !top_k; }

private:
    float temperature;
};

// Kept: keys above `key`, and those that equal it up to index `last`.
struct Limit {
    uint32_t key;
    int last;
    __device__ __forceinline__ bool keeps(int i, uint32_t k) const { return k > key || (k == key && i <= last); }
};

struct Shared {
    u64 hist[256];
    u64 sums[kWaves];
    u64 before;
    uint32_t bin;
    int count;
    double mid[kOct];
};

__device__ __forceinline__ u64 wave_sum(u64 v)
{
#pragma unroll 1
    for (int off = 32; off > 0; off >>= 1)
        v += __shfl_xor(v, off, 64);
    return v;
}
__device__ __forceinline__ u64 wave_max(u64 v)
{
#pragma unroll 1
    for (int off = 32; off > 0; off >>= 1)
        v = max(v, __shfl_xor(v, off, 64));
    return v;
}
__device__ __forceinline__ u64 wave_scan(u64 v)  // sums over the lanes up to each
{
#pragma unroll 1
    for (int off = 1; off < 64; off <<= 1) {
        const u64 x = __shfl_up(v, off, 64);
        v += (int)(threadIdx.x & 63) >= off ? x : 0;
    }
    return v;
}

// Sums over the threads up to each, and over all of them.
__device__ __forceinline__ u64 block_scan(Shared &sh, u64 v, u64 &total)
{
    const u64 upto = wave_scan(v);
    __syncthreads();
    if ((threadIdx.x & 63) == 63)
        sh.sums[threadIdx.x >> 6] = upto;
    __syncthreads();
    u64 before = 0;
    total = 0;
#pragma unroll 4
    for (int w = 0; w < kWaves; ++w) {
        before += w < (int)(threadIdx.x >> 6) ? sh.sums[w] : 0;
        total += sh.sums[w];
    }
    return before + upto;
}
__device__ __forceinline__ u64 block_sum(Shared &sh, u64 v)
{
    v = wave_sum(v);
    __syncthreads();
    if ((threadIdx.x & 63) == 0)
        sh.sums[threadIdx.x >> 6] = v;
    __syncthreads();
    u64 total = 0;
#pragma unroll 4
    for (int w = 0; w < kWaves; ++w)
        total += sh.sums[w];
    return total;
}

// Sorts n <= kThreads different numbers in LDS, the greatest first, by counting
// the greater ones of each, by up to eight lanes a number.
__device__ __forceinline__ void sort_few(u64 *x, int n)
{
    int shift = 0;
    while (shift < 3 && n << (shift + 1) <= kThreads)
        ++shift;
    const int number = threadIdx.x >> shift, lanes = 1 << shift;
    const u64 mine = number < n ? x[number] : 0;
    int rank = 0;
    if (number < n) {
#pragma unroll 8
        for (int i = threadIdx.x & (lanes - 1); i < n; i += lanes)
            rank += x[i] > mine;
    }
#pragma unroll 1
    for (int off = 1; off < lanes; off <<= 1)
        rank += __shfl_xor(rank, off, 64);
    __syncthreads();
    if (number < n && (threadIdx.x & (lanes - 1)) == 0)
        x[rank] = mine;
    __syncthreads();
}

// First of N x 64 amounts, N a lane, at which their sum reaches `stop` (one
// does), and what lies before it.
template <int N>
__device__ __forceinline__ int wave_find(const u64 (&a)[N], u64 stop, u64 &before)
{
    u64 mine = 0;
#pragma unroll
    for (int i = 0; i < N; ++i)
        mine += a[i];
    const u64 upto = wave_scan(mine);
    const int lane = __ffsll((u64)__ballot(upto >= stop)) - 1;
    u64 sum = upto - mine;
    int at = 0;
    bool past = false;
#pragma unroll
    for (int i = 0; i < N - 1; ++i) {
        past |= sum + a[i] >= stop;
        sum += past ? 0 : a[i];
        at += !past;
    }
    before = __shfl(sum, lane, 64);
    return N * lane + __shfl(at, lane, 64);
}

// The greatest 32-bit number at which the amounts of the items that have it, or
// a greater one, sum to at least `stop`, and in `before` the sum of the greater
// ones'; false if all of them do not.  items(f) calls f(number, amount) for
// each item of this thread.
template <typename Items>
__device__ bool select(Shared &sh, Items items, u64 stop, uint32_t &number, u64 &before)
{
    number = 0;
    before = 0;
#pragma unroll 1
    for (int shift = 24; shift >= 0; shift -= 8) {
        __syncthreads();
        if (threadIdx.x < 256)
            sh.hist[threadIdx.x] = 0;
        __syncthreads();
        const uint32_t high = shift == 24 ? 0u : ~0u << (shift + 8);
        items([&](uint32_t x, u64 amount) {
            if ((x & high) == number)
                atomicAdd(&sh.hist[255 - (x >> shift & 255)], amount);
        });
        __syncthreads();
        if (threadIdx.x < 64) {
            u64 a[4], sum = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                sum += a[i] = sh.hist[4 * threadIdx.x + i];
            sum = wave_sum(sum);
            u64 less = 0;
            const int bin = sum >= stop - before ? wave_find(a, stop - before, less) : 256;
            if (threadIdx.x == 0) {
                sh.bin = bin;
                sh.before = less;
            }
        }
        __syncthreads();
        if (sh.bin == 256)
            return false;
        number |= (255 - sh.bin) << shift;
        before += sh.before;
    }
    return true;
}

// The limit at which the amounts of the tokens of `tokens`(f(index, key)) reach
// `stop`; amount(key) is the same for equal keys.  False: they do not.
template <typename Tokens, typename Amount>
__device__ bool limit_at(Shared &sh, Tokens tokens, Amount amount, u64 stop, Limit &limit)
{
    uint32_t key, place;
    u64 before, none;
    if (!select(sh, [&](auto f) { tokens([&](int, uint32_t k) { f(k, amount(k)); }); }, stop, key, before))
        return false;
    const u64 one = amount(key), ties = (stop - before + one - 1) / one;
    select(sh, [&](auto f) { tokens([&](int i, uint32_t k) { if (k == key) f(~(uint32_t)i, 1); }); }, ties, place, none);
    limit = {key, (int)~place};
    return true;
}

__device__ __forceinline__ void answer(const SampleArgs &p, int b, int token, float logprob)
{
    p.tokens[b] = token;
    if (p.logprobs)
        p.logprobs[b] = logprob;
}
__device__ __forceinline__ void answer_first(const SampleArgs &p, int b, u64 first)
{
    const bool none = key_in(first) <= kNone;
    answer(p, b, none ? -1 : index_in(first), none ? -__builtin_inff() : 0.0f);
}
// A token q eighths of octaves below the greatest, of `total` kept units.  Its log
// probability comes from q and not from its units, of which a light token that a
// random number near 0 draws has only a few; in 64 bits, rounded once.
__device__ __forceinline__ void answer_token(const SampleArgs &p, int b, int token, double q, u64 total)
{
    constexpr double l = 0.693147180559945309417 / 8;
    const double all = (double)total * __hiloint2double((1023 - p.frac) << 20, 0);  // over the greatest, at least 1
    answer(p, b, token, (float)(0.0 - (q * l + log(all))));
}

// Draws the token at which the kept units, in the order of indices, pass `want`,
// among vectors [first, last), before which `sum` of them lie.
template <int TYPE, typename Kept>
__device__ __forceinline__ void draw_from(Shared &sh, const SampleArgs &p, int b, const Row<TYPE> &row, const Scale &s,
                                          int first, int last, Kept kept, u64 want, u64 sum, u64 total)
{
    for (int v0 = first; v0 < last; v0 += kThreads) {
        const int v = v0 + threadIdx.x;
        u64 here = 0, step;
        u4 x = {};
        if (v < last) {
            x = row.load(v);
            row.each_token(v, x, [&](int i, uint32_t k) { here += kept(i, k); });
        }
        u64 upto = sum + block_scan(sh, here, step);
        if (upto > want && upto - here <= want) {
            upto -= here;
            row.each_token(v, x, [&](int i, uint32_t k) {
                const u64 n = kept(i, k);
                if (upto <= want && upto + n > want)
                    answer_token(p, b, i, s.eighths(k), total);
                upto += n;
            });
        }
        sum += step;
        if (sum > want)
            return;
    }
}

// All of a row's work over the row itself.
template <int TYPE>
__device__ __forceinline__ void draw_slowly(Shared &sh, const SampleArgs &p, int b, const Row<TYPE> &row, const Scale &s,
                                            const Settings &set)
{
    Limit limit = {kNone, 0};
    auto tokens = [&](auto f) {
        row.each([&](int i, uint32_t k) {
            if (k > kNone && limit.keeps(i, k))
                f(i, k);
        });
    };
    if (set.top_k) {
        Limit to;
        if (limit_at(sh, tokens, [](uint32_t) { return (u64)1; }, (u64)set.top_k, to))
            limit = to;
    }
    const double far = set.far();
    u64 total = 0;
#pragma unroll 1
    for (int pass = set.has_p ? 0 : 1; pass < 2; ++pass) {
        u64 mine = 0;
        tokens([&](int, uint32_t k) {
            const double q = s.eighths(k);
            mine += pass == 0 || q <= far ? s.units(q) : 0;
        });
        total = block_sum(sh, mine);
        Limit to;
        if (pass == 0 && limit_at(sh, tokens, [&](uint32_t k) { return s.units_of(k); }, set.reach(total), to))
            limit = to;
    }
    auto kept = [&](int i, uint32_t k) {
        if (k <= kNone || !limit.keeps(i, k))
            return (u64)0;
        const double q = s.eighths(k);
        return q <= far ? s.units(q) : 0;
    };
    draw_from(sh, p, b, row, s, 0, row.vectors(), kept, set.pass(total), 0, total);
}

// A row without what other kernels found.
template <int TYPE>
__device__ __noinline__ void draw_row(Shared &sh, const SampleArgs &p, int b)
{
    const Row<TYPE> row(p, b);
    u64 first = 0;
    row.each([&](int i, uint32_t k) { first = max(first, order_of(k, i)); });
    first = wave_max(first);
    __syncthreads();  // a caller's wavefronts may still read sh
    if ((threadIdx.x & 63) == 0)
        sh.sums[threadIdx.x >> 6] = first;
    fill_mid(sh.mid, p.frac);
    __syncthreads();
    for (int w = 0; w < kWaves; ++w)
        first = max(first, sh.sums[w]);
    const Settings set(p, b);
    if (key_in(first) <= kNone || set.greedy) {
        if (threadIdx.x == 0)
            answer_first(p, b, first);
        return;
    }
    draw_slowly(sh, p, b, row, set.scale(key_in(first), p.frac, sh.mid), set);
}

template <int TYPE>
__global__ __launch_bounds__(kThreads) void sample_kernel(const SampleArgs p)
{
    __shared__ Shared sh;
    draw_row<TYPE>(sh, p, blockIdx.x);
}

// Where a row that was summed up ends what it keeps.
struct Edge {
    int bin;     // heavier eighths of octaves are kept; kOct: all are
    u64 stop;    // units up to which the tokens of this one are, 0: all
    double far;  // eighths of octaves within which tokens are kept
};

// Computed by every wavefront, of the row's sums.
__device__ __forceinline__ Edge edge_of(const u64 *sums, const Settings &set)
{
    Edge x = {kOct, 0, set.far()};
    if (set.has_p) {
        constexpr int N = kOct / 64;
        u64 a[N], total = 0;
#pragma unroll
        for (int i = 0; i < N; ++i)
            total += a[i] = sums[N * (threadIdx.x & 63) + i];
        const u64 stop = set.reach(wave_sum(total));
        u64 before;
        x.bin = wave_find(a, stop, before);
        x.stop = stop - before;
    }
    if (x.far < x.bin) {
        x.bin = (int)x.far;
        x.stop = 0;
    }
    return x;
}

// The limit among the edge's tokens: a 256th of the eighth of an octave, then the
// tokens in it in order.
template <typename Tokens>
__device__ __forceinline__ Limit end_edge(Shared &sh, u64 *few, Tokens tokens, const Edge &edge, const Scale &s)
{
    Limit limit = {kNone, 0};
    __syncthreads();
    if (threadIdx.x < 256)
        sh.hist[threadIdx.x] = 0;
    if (threadIdx.x == 0)
        sh.count = 0;
    __syncthreads();
    if (!edge.stop)
        return limit;
    auto piece = [&](uint32_t k) { return min((int)((s.eighths(k) - edge.bin) * 256.0), 255); };
    tokens([&](int, uint32_t k) { atomicAdd(&sh.hist[piece(k)], s.units_of(k)); });
    __syncthreads();
    u64 a[4], before;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        a[i] = sh.hist[4 * (threadIdx.x & 63) + i];
    const int at = wave_find(a, edge.stop, before);
    tokens([&](int i, uint32_t k) {
        if (piece(k) == at) {
            const int to = atomicAdd(&sh.count, 1);
            if (to < kThreads)
                few[to] = order_of(k, i);
        }
    });
    __syncthreads();
    const int n = sh.count;
    if (n > kThreads) {  // equal ones, or nearly
        limit_at(sh, tokens, [&](uint32_t k) { return s.units_of(k); }, edge.stop, limit);
        return limit;
    }
    sort_few(few, n);
    const u64 token = (int)threadIdx.x < n ? few[threadIdx.x] : 0;
    const u64 units = (int)threadIdx.x < n ? s.units_of(key_in(token)) : 0;
    u64 all;
    const u64 sum = before + block_scan(sh, units, all);
    if (sum >= edge.stop && sum - units < edge.stop)
        sh.before = token;
    __syncthreads();
    limit = {key_in(sh.before), index_in(sh.before)};
    return limit;
}

// Draws from n <= kThreads tokens, among which all that are kept are: sorts them,
// ends the kept ones, sorts these by index; `down` keeps their eighths of octaves.
__device__ __forceinline__ void draw_few(Shared &sh, const SampleArgs &p, int b, u64 *few, u64 *down, int n, const Scale &s,
                                         const Settings &set)
{
    const int i = threadIdx.x;
    int place = 0;
    u64 mine = 0, total;
#pragma unroll 1
    for (int pass = 0;; ++pass) {
        sort_few(few, n);
        const u64 x = i < n ? few[i] : 0;
        u64 sum;
        if (pass == 0) {
            double eighths = 0.0;
            if (i < min(n, set.top_k)) {
                place = index_in(x);
                eighths = s.eighths(key_in(x));
                mine = s.units(eighths);
            }
            sum = block_scan(sh, mine, total);
            if ((set.has_p && sum - mine >= set.reach(total)) || eighths > set.far())
                mine = 0;
            down[i] = (u64)__double_as_longlong(eighths);
            n = __syncthreads_count(mine > 0);  // the kept ones are the first
            few[i] = mine ? order_of(~(uint32_t)place, i) : 0;
            __syncthreads();
        } else {
            const double eighths = i < n ? __longlong_as_double((long long)down[index_in(x)]) : 0.0;
            mine = i < n ? s.units(eighths) : 0;
            sum = block_scan(sh, mine, total);
            const u64 want = set.pass(total);
            if (sum > want && sum - mine <= want)
                answer_token(p, b, (int)~key_in(x), eighths, total);
            return;
        }
    }
}

// Draws from listed tokens, of which top-k keeps at most kThreads.
template <typename Tokens>
__device__ __forceinline__ void draw_listed(Shared &sh, const SampleArgs &p, int b, Tokens tokens, int length, u64 *few,
                                            u64 *down, const Scale &s, const Settings &set)
{
    Limit limit = {kNone, 0};
    if (length > kThreads)
        limit_at(sh, tokens, [](uint32_t) { return (u64)1; }, (u64)set.top_k, limit);
    __syncthreads();
    if (threadIdx.x == 0)
        sh.count = 0;
    __syncthreads();
    tokens([&](int i, uint32_t k) {
        if (limit.keeps(i, k))
            few[atomicAdd(&sh.count, 1)] = order_of(k, i);
    });
    __syncthreads();
    draw_few(sh, p, b, few, down, sh.count, s, set);
}

// A row that a workgroup holds in registers, NV vectors a thread.
template <int TYPE, int NV>
__global__ __launch_bounds__(kThreads) void sample_held_kernel(const SampleArgs p)
{
    constexpr int E = Row<TYPE>::kE;
    constexpr int kRoom = 4096;  // tokens listed
    __shared__ Shared sh;
    __shared__ u64 list[kRoom], few[kThreads], more[kThreads];
    u64 *const sums = more;  // of one of which there is need
    __shared__ uint32_t groups[kGroups];
    __shared__ uint32_t low;
    const int b = blockIdx.x, lane = threadIdx.x & 63;
    const Row<TYPE> row(p, b);
    const int n = row.vectors();
    u4 held[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        held[i] = (u4){0xffffffffu, 0xffffffffu, 0xffffffffu, 0xffffffffu};  // NaN: no tokens
        if ((int)threadIdx.x + i * kThreads < n)
            held[i] = row.load(threadIdx.x + i * kThreads);
    }
    // f(vector, x) for the held vectors, in a loop
    auto each_vector = [&](auto f) {
        u4 x[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i)
            x[i] = held[i];
#pragma unroll 1
        for (int v = threadIdx.x; v < n; v += kThreads) {
            f(v, x[0]);
#pragma unroll
            for (int i = 1; i < NV; ++i)
                x[i - 1] = x[i];
        }
    };
    const Settings set(p, b);
    fill_mid(sh.mid, p.frac);
    for (int i = threadIdx.x; i < kOct; i += kThreads)
        sums[i] = 0;
    if (threadIdx.x == 0) {
        sh.count = 0;
        low = 0;
    }
    float most = -__builtin_inff();
    each_vector([&](int, const u4 &x) { most = row.greatest(x, most); });
    // groups of 16 lanes, or of four where more tokens are kept than they can tell apart
    const int quad = set.top_k > 40;
    uint32_t key = key_of(most);
    key = max(key, (uint32_t)__shfl_xor(key, 1, 64));
    key = max(key, (uint32_t)__shfl_xor(key, 2, 64));
    uint32_t all = max(key, (uint32_t)__shfl_xor(key, 4, 64));
    all = max(all, (uint32_t)__shfl_xor(all, 8, 64));
    if (!quad)
        key = all;
    if ((threadIdx.x & (quad ? 3 : 15)) == 0)
        groups[threadIdx.x >> (quad ? 2 : 4)] = key;
    all = max(all, (uint32_t)__shfl_xor(all, 16, 64));
    all = max(all, (uint32_t)__shfl_xor(all, 32, 64));
    if (lane == 0)
        sh.sums[threadIdx.x >> 6] = all;
    __syncthreads();
    const uint32_t top = (uint32_t)wave_max(lane < kWaves ? sh.sums[lane] : 0);
    if (top <= kNone || set.greedy) {
        // the first of the greatest: below p.vocab, as there is one
        if (threadIdx.x == 0)
            sh.bin = p.vocab;
        __syncthreads();
        each_vector([&](int v, const u4 &x) {
            row.each_token(v, x, [&](int i, uint32_t k) {
                if (k == top)
                    atomicMin(&sh.bin, (uint32_t)i);
            });
        });
        __syncthreads();
        if (threadIdx.x == 0)
            answer_first(p, b, order_of(top, (int)sh.bin));
        return;
    }
    const bool lists = set.lists(p.vocab <= kRoom ? kThreads : kGroups);
    if (!lists && !set.sums()) {
        draw_row<TYPE>(sh, p, b);
        return;
    }
    const Scale s = set.scale(top, p.frac, sh.mid);
    auto add = [&](int v, const u4 &x, uint32_t on) {
        if (!on)
            return;
        int to = atomicAdd(&sh.count, __popc(on));
        row.each_set(v, x, on, [&](int index, uint32_t k) {
            if (to < kRoom)
                list[to] = order_of(k, index);
            ++to;
        });
    };
    if (lists) {
        // the top_k-th greatest group: at least top_k tokens are as great
        const int mine = threadIdx.x >> (quad ? 2 : 4), step = quad ? 4 : 16;
        int rank = 0;
#pragma unroll 4
        for (int i = threadIdx.x & (step - 1); i < kThreads / step; i += step)
            rank += groups[i] > key || (groups[i] == key && i < mine);
        rank += __shfl_xor(rank, 1, 64);
        rank += __shfl_xor(rank, 2, 64);
        if (!quad) {
            rank += __shfl_xor(rank, 4, 64);
            rank += __shfl_xor(rank, 8, 64);
        }
        if (rank == set.top_k - 1)
            low = key;
        __syncthreads();
        const float least = value_of(max(low, kNone + 1));
        each_vector([&](int v, const u4 &x) { add(v, x, row.at_least(x, least)); });
    }
    if (!lists)
        each_vector([&](int, const u4 &x) {
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const double eighths = s.eighths(row.value(x, e));
                if (eighths < kOct)  // no NaN, and no -infinity
                    atomicAdd(&sums[(int)eighths], s.units(eighths, (int)eighths));
            }
        });
    __syncthreads();
    const Edge edge = lists ? Edge{kOct, 0, 0.0} : edge_of(sums, set);
    if (!lists && edge.bin < kOct)
        each_vector([&](int v, const u4 &x) {
            uint32_t on = 0;
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const double eighths = s.eighths(row.value(x, e));
                on |= (uint32_t)(eighths < kOct && (int)eighths == edge.bin) << e;
            }
            add(v, x, on);
        });
    __syncthreads();
    const int length = sh.count;
    if (length > kRoom) {
        draw_row<TYPE>(sh, p, b);
        return;
    }
    auto tokens = [&](auto f) {
#pragma unroll 1
        for (int i = threadIdx.x; i < length; i += kThreads)
            f(index_in(list[i]), key_in(list[i]));
    };
    if (lists) {
        draw_listed(sh, p, b, tokens, length, few, more, s, set);
        return;
    }
    const Limit limit = end_edge(sh, few, tokens, edge, s);
    auto kept = [&](int i, uint32_t k) {
        if (k <= kNone || !limit.keeps(i, k))
            return (u64)0;
        const double eighths = s.eighths(k);
        return eighths <= edge.far ? s.units(eighths) : 0;
    };
    u64 mine = (int)threadIdx.x < edge.bin && threadIdx.x < kOct ? sums[threadIdx.x] : 0;
    tokens([&](int i, uint32_t k) { mine += kept(i, k); });
    const u64 total = block_sum(sh, mine), want = set.pass(total);
    // step by step in the order of indices
    u64 sum = 0;
#pragma unroll 1
    for (int v0 = 0; v0 < n; v0 += kThreads) {
        const int v = v0 + threadIdx.x;
        u64 here = 0, step;
        if (v < n)
            row.each_token(v, held[0], [&](int i, uint32_t k) { here += kept(i, k); });
        u64 upto = sum + block_scan(sh, here, step);
        if (upto > want && upto - here <= want) {
            upto -= here;
            row.each_token(v, held[0], [&](int i, uint32_t k) {
                const u64 units = kept(i, k);
                if (upto <= want && upto + units > want)
                    answer_token(p, b, i, s.eighths(k), total);
                upto += units;
            });
        }
        sum += step;
        if (sum > want)
            return;
#pragma unroll
        for (int i = 1; i < NV; ++i)
            held[i - 1] = held[i];
    }
}

// How rows are shared between workgroups, and where what they find is kept.
struct Parts {
    int steps;    // of 64 vectors, a wavefront
    int waves;    // a row, a multiple of kPart
    int lanes;    // of a group: 16 or 64
    int groups;
    uint32_t *greatest;  // [rows][groups]
    uint32_t *highest;   // [rows][64 waves]: the greatest logit's key of each lane's vectors
    u64 *first;          // [rows][waves / kPart]: greatest key and its first place (order_of)
    u64 *list;           // [rows][kList]: tokens (order_of)
    uint32_t *length;    // [rows]
    u64 *sums;           // [rows][kOct]: units per eighth of an octave
    u64 *units;          // [rows][waves / kPart][kOct]: the same of each part

    __host__ __device__ int parts() const { return waves / kPart; }
};

// A wavefront's vectors of its part of a row, four a lane on their way at a time.
template <int TYPE>
struct PartVectors {
    const Row<TYPE> &row;
    int first, steps, n;
    u4 x[4];

    __device__ __forceinline__ PartVectors(const Row<TYPE> &r, const Parts &q, int wave)
        : row(r), first(wave * q.steps * 64 + (int)(threadIdx.x & 63)), steps(q.steps), n(r.vectors())
    {
    }
    __device__ __forceinline__ void load(int st)
    {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (st + i < steps && first + (st + i) * 64 < n)
                x[i] = row.load(first + (st + i) * 64);
    }
    // f(vector, x), once, after load(0)
    template <typename F>
    __device__ __forceinline__ void each(F f)
    {
        for (int st = 0;;) {
#pragma unroll 1
            for (int i = st; i < min(st + 4, steps); ++i) {
                if (first + i * 64 < n)
                    f(first + i * 64, x[0]);
                x[0] = x[1];
                x[1] = x[2];
                x[2] = x[3];
            }
            st += 4;
            if (st >= steps)
                break;
            load(st);
        }
    }
};

template <int TYPE>
__global__ __launch_bounds__(64 * kPart) void greatest_kernel(const SampleArgs p, const Parts q)
{
    constexpr int E = Row<TYPE>::kE;
    __shared__ u64 firsts[kPart];
    const int b = blockIdx.x / q.parts(), part = blockIdx.x % q.parts(), lane = threadIdx.x & 63;
    const int wave = part * kPart + (threadIdx.x >> 6);
    const Row<TYPE> row(p, b);
    const int n = row.vectors(), first = wave * q.steps * 64 + lane;
    uint32_t key = 0;
    int place = 0;
    for (int st = 0; st < q.steps; st += 4) {
        u4 x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (st + i < q.steps && first + (st + i) * 64 < n)
                x[i] = row.load(first + (st + i) * 64);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (st + i < q.steps && first + (st + i) * 64 < n)
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    const uint32_t k = key_of(row.value(x[i], e));
                    if (k > key) {
                        key = k;
                        place = (first + (st + i) * 64) * E + e - row.lead;
                    }
                }
    }
    q.highest[((int64_t)b * q.waves + wave) * 64 + lane] = key;
    uint32_t g = key;
#pragma unroll 1
    for (int off = 1; off < q.lanes; off <<= 1)
        g = max(g, (uint32_t)__shfl_xor(g, off, 64));
    if (lane % q.lanes == 0)
        q.greatest[(int64_t)b * q.groups + wave * (64 / q.lanes) + lane / q.lanes] = g;
    const u64 f = wave_max(order_of(key, place));
    if (lane == 0)
        firsts[threadIdx.x >> 6] = f;
    __syncthreads();
    if (threadIdx.x == 0)
        q.first[(int64_t)b * q.parts() + part] = max(max(firsts[0], firsts[1]), max(firsts[2], firsts[3]));
    if (part == 0) {  // what the next kernels count up
        for (int i = threadIdx.x; i < kOct; i += 64 * kPart)
            q.sums[(int64_t)b * kOct + i] = 0;
        if (threadIdx.x == 0)
            q.length[b] = 0;
    }
}

// The tokens that a workgroup lists, in any order: what is drawn from a row's list
// does not depend on it.
struct Found {
    u64 token[kFound];
    int count, at;

    // The tokens of vector v whose bits are set, by one lane.
    template <int TYPE>
    __device__ __forceinline__ void add(const Row<TYPE> &row, int v, const u4 &x, uint32_t on)
    {
        int to = atomicAdd(&count, __popc(on));
        row.each_set(v, x, on, [&](int index, uint32_t k) {
            if (to < kFound)
                token[to] = order_of(k, index);
            ++to;
        });
    }
    // To the row's list; more than there is room for make the list too long.
    __device__ __forceinline__ void list(const Parts &q, int b)
    {
        __syncthreads();
        const int n = count;
        if (n == 0)
            return;
        if (threadIdx.x == 0)
            at = (int)atomicAdd(&q.length[b], n > kFound ? kList + 1u : (uint32_t)n);
        __syncthreads();
        for (int i = threadIdx.x; i < min(n, kFound) && at + i < kList; i += 64 * kPart)
            q.list[(int64_t)b * kList + at + i] = token[i];
    }
};

template <int TYPE>
__global__ __launch_bounds__(64 * kPart) void weigh_kernel(const SampleArgs p, const Parts q)
{
    constexpr int E = Row<TYPE>::kE;
    __shared__ Found found;
    u64 *const units = found.token;  // of one of which there is need
    static_assert(kOct <= kFound, "units share the list's place");
    __shared__ double mid[kOct];
    const int b = blockIdx.x / q.parts(), part = blockIdx.x % q.parts(), lane = threadIdx.x & 63;
    const int wave = part * kPart + (threadIdx.x >> 6);
    const Settings set(p, b);
    const bool lists = set.lists(q.groups);
    if (set.greedy || (!lists && !set.sums()))
        return;
    const Row<TYPE> row(p, b);
    PartVectors<TYPE> vectors(row, q, wave);
    if (lists) {
        const uint32_t highest = q.highest[((int64_t)b * q.waves + wave) * 64 + lane];
        // A limit that top_k groups' greatest reach, so that at least top_k tokens do:
        // 19 bits of the top_k-th greatest (all that 16-bit logits have), by every
        // wavefront for itself.
        uint32_t group[kGroups / 64], low = 0;
#pragma unroll
        for (int i = 0; i < kGroups / 64; ++i)
            group[i] = lane + 64 * i < q.groups ? q.greatest[(int64_t)b * q.groups + lane + 64 * i] : 0u;
        if (threadIdx.x == 0)
            found.count = 0;
        __syncthreads();
#pragma unroll 1
        for (uint32_t bit = 1u << 31; bit >= 1u << 13; bit >>= 1) {
            int n = 0;
#pragma unroll
            for (int i = 0; i < kGroups / 64; ++i)
                n += __popcll(__ballot(group[i] >= (low | bit)));
            low |= n >= set.top_k ? bit : 0;
        }
        const uint32_t limit = max(low, kNone + 1);
        const float least = value_of(limit);
        if (highest >= limit) {  // of few lanes: what the others have is not read again
            vectors.load(0);
            vectors.each([&](int v, const u4 &x) {
                const uint32_t on = row.at_least(x, least);
                if (on)
                    found.add(row, v, x, on);
            });
        }
        found.list(q, b);
        return;
    }
    vectors.load(0);  // on their way meanwhile
    const u64 top = wave_max(lane < q.parts() ? q.first[(int64_t)b * q.parts() + lane] : 0);
    if (key_in(top) <= kNone)
        return;
    const Scale s = set.scale(key_in(top), p.frac, mid);
    for (int i = threadIdx.x; i < kOct; i += 64 * kPart)
        units[i] = 0;
    fill_mid(mid, p.frac);
    __syncthreads();
    vectors.each([&](int, const u4 &x) {
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const double eighths = s.eighths(row.value(x, e));
            if (eighths < kOct) {  // no NaN, and no -infinity
                const int bin = (int)eighths;
                atomicAdd(&units[bin], s.units(eighths, bin));
            }
        }
    });
    __syncthreads();
    for (int i = threadIdx.x; i < kOct; i += 64 * kPart) {
        const u64 sum = units[i];
        q.units[((int64_t)b * q.parts() + part) * kOct + i] = sum;
        if (sum)
            atomicAdd(&q.sums[(int64_t)b * kOct + i], sum);
    }
}

template <int TYPE>
__global__ __launch_bounds__(64 * kPart) void gather_kernel(const SampleArgs p, const Parts q)
{
    constexpr int E = Row<TYPE>::kE;
    __shared__ Found found;
    const int b = blockIdx.x / q.parts(), part = blockIdx.x % q.parts(), lane = threadIdx.x & 63;
    const int wave = part * kPart + (threadIdx.x >> 6);
    const Settings set(p, b);
    if (set.greedy || !set.sums() || !(set.has_p || set.min_p > 0.0f))
        return;
    const Row<TYPE> row(p, b);
    PartVectors<TYPE> vectors(row, q, wave);
    vectors.load(0);
    const u64 top = wave_max(lane < q.parts() ? q.first[(int64_t)b * q.parts() + lane] : 0);
    if (key_in(top) <= kNone)
        return;
    const Scale s = set.scale(key_in(top), p.frac, nullptr);
    const int bin = edge_of(q.sums + (int64_t)b * kOct, set).bin;
    if (bin >= kOct)
        return;
    if (threadIdx.x == 0)
        found.count = 0;
    __syncthreads();
    vectors.each([&](int v, const u4 &x) {
        uint32_t on = 0;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const double eighths = s.eighths(row.value(x, e));
            on |= (uint32_t)(eighths < kOct && (int)eighths == bin) << e;
        }
        if (on)
            found.add(row, v, x, on);
    });
    found.list(q, b);
}

template <int TYPE>
__global__ __launch_bounds__(kThreads) void draw_kernel(const SampleArgs p, const Parts q)
{
    __shared__ Shared sh;
    __shared__ u64 few[kThreads], amount[kThreads];
    const int b = blockIdx.x, parts = q.parts(), lane = threadIdx.x & 63;
    const Settings set(p, b);
    const uint32_t length = q.length[b];
    const u64 first = wave_max(lane < parts ? q.first[(int64_t)b * parts + lane] : 0);
    if (key_in(first) <= kNone || set.greedy) {
        if (threadIdx.x == 0)
            answer_first(p, b, first);
        return;
    }
    const bool lists = set.lists(q.groups);
    if ((!lists && !set.sums()) || length > kList) {
        draw_row<TYPE>(sh, p, b);
        return;
    }
    const Scale s = set.scale(key_in(first), p.frac, sh.mid);
    const u64 *list = q.list + (int64_t)b * kList;
    fill_mid(sh.mid, p.frac);
    u64 mine[kList / kThreads];
#pragma unroll
    for (int i = 0; i < kList / kThreads; ++i)
        mine[i] = threadIdx.x + i * kThreads < length ? list[threadIdx.x + i * kThreads] : 0;
    auto tokens = [&](auto f) {
        u64 x[kList / kThreads];
#pragma unroll
        for (int i = 0; i < kList / kThreads; ++i)
            x[i] = mine[i];
#pragma unroll 1
        for (uint32_t at = threadIdx.x; at < length; at += kThreads) {
            f(index_in(x[0]), key_in(x[0]));
#pragma unroll
            for (int i = 1; i < kList / kThreads; ++i)
                x[i - 1] = x[i];
        }
    };
    if (lists) {
        draw_listed(sh, p, b, tokens, (int)length, few, amount, s, set);
        return;
    }
    const Edge edge = edge_of(q.sums + (int64_t)b * kOct, set);
    const Limit limit = end_edge(sh, few, tokens, edge, s);
    auto kept = [&](int i, uint32_t k) {
        if (k <= kNone || !limit.keeps(i, k))
            return (u64)0;
        const double eighths = s.eighths(k);
        return eighths <= edge.far ? s.units(eighths) : 0;
    };
    // what each part of the row keeps
    for (int w = threadIdx.x >> 6; w < parts; w += kWaves) {
        u64 sum = 0;
#pragma unroll
        for (int i = 0; i < kOct; i += 64)
            if (i + lane < edge.bin)
                sum += q.units[((int64_t)b * parts + w) * kOct + i + lane];
        sum = wave_sum(sum);
        if (lane == 0)
            amount[w] = sum;
    }
    __syncthreads();
    const int part_vectors = q.steps * 64 * kPart;
    const Row<TYPE> row(p, b);
    tokens([&](int i, uint32_t k) {
        const u64 x = kept(i, k);
        if (x)
            atomicAdd(&amount[(i + row.lead) / Row<TYPE>::kE / part_vectors], x);
    });
    __syncthreads();
    // every wavefront finds the part: at most 64 of them, one a lane
    const u64 here = lane < parts ? amount[lane] : 0, upto = wave_scan(here), total = __shfl(upto, 63, 64);
    const u64 want = set.pass(total);
    const int part = __ffsll((u64)__ballot(upto > want)) - 1;
    draw_from(sh, p, b, row, s, part * part_vectors, min((part + 1) * part_vectors, row.vectors()), kept, want,
              __shfl(upto - here, part, 64), total);
}

// Wavefronts that read 64 vectors a step, so many steps that a row has at most
// 256 of them and, up to eight steps, that a call has at most 2048 workgroups.
Parts parts_of(int64_t rows, int64_t vocab, int type)
{
    const int64_t e = type == 2 ? 4 : 8, steps = ((vocab + 2 * e - 1) / e + 63) / 64;  // of the row and its odd ends
    Parts q = {};
    q.steps = (int)((steps + kGroups - 1) / kGroups);
    while (q.steps < 8 && rows * ((steps + q.steps * kPart - 1) / (q.steps * kPart)) > 2048)
        ++q.steps;
    q.waves = (int)((steps + q.steps * kPart - 1) / (q.steps * kPart)) * kPart;
    q.lanes = q.waves <= kGroups / 4 ? 16 : 64;
    q.groups = q.waves * (64 / q.lanes);
    return q;
}

// Lays out the workspace; its bytes.
int64_t place(Parts &q, int64_t rows, uint8_t *at)
{
    uint8_t *const start = at;
    auto take = [&](auto *&p, int64_t n) {
        p = (decltype(p + 0))at;
        at += (n * (int64_t)sizeof(*p) + 15) / 16 * 16;
    };
    take(q.list, rows * kList);
    take(q.units, rows * q.parts() * kOct);
    take(q.sums, rows * kOct);
    take(q.first, rows * q.parts());
    take(q.greatest, rows * q.groups);
    take(q.highest, rows * q.waves * 64);
    take(q.length, rows);
    return at - start;
}

// Rows that a workgroup holds: up to four vectors of 16-bit logits a thread, eight
// of fp32.
constexpr int kHeld16 = 4, kHeld32 = 8;
bool held(int64_t vocab, int type)
{
    return type == 2 ? vocab + 3 <= 4 * kHeld32 * kThreads : vocab + 7 <= 8 * kHeld16 * kThreads;
}

template <int TYPE>
hipError_t launch_t(const SampleArgs &p, void *workspace, int64_t workspace_bytes, hipStream_t s)
{
    const dim3 rows((unsigned)p.rows);
    const int64_t need = sample_workspace_bytes(p.rows, p.vocab, TYPE);
    if (!grid_fits(p.rows, kThreads))
        return kGridTooLarge;
    if (need == 0) {
        sample_held_kernel<TYPE, TYPE == 2 ? kHeld32 : kHeld16><<<rows, kThreads, 0, s>>>(p);
        return hipGetLastError();
    }
    if (workspace_bytes < need) {
        sample_kernel<TYPE><<<rows, kThreads, 0, s>>>(p);
        return hipGetLastError();
    }
    Parts q = parts_of(p.rows, p.vocab, TYPE);
    place(q, p.rows, (uint8_t *)workspace);
    const int64_t items = (int64_t)p.rows * q.parts();
    if (!grid_fits(items, 64 * kPart))
        return kGridTooLarge;
    const dim3 grid((unsigned)items);
    greatest_kernel<TYPE><<<grid, 64 * kPart, 0, s>>>(p, q);
    weigh_kernel<TYPE><<<grid, 64 * kPart, 0, s>>>(p, q);
    if (p.top_p || p.min_p)
        gather_kernel<TYPE><<<grid, 64 * kPart, 0, s>>>(p, q);
    draw_kernel<TYPE><<<rows, kThreads, 0, s>>>(p, q);
    return hipGetLastError();
}

}  // namespace

int64_t sample_workspace_bytes(int64_t rows, int64_t vocab, int type)
{
    if (rows == 0 || held(vocab, type))
        return 0;
    Parts q = parts_of(rows, vocab, type);
    return place(q, rows, nullptr);
}

hipError_t launch_sample(const SampleArgs &p, int type, void *workspace, int64_t workspace_bytes, hipStream_t s)
{
    return type == 0   ? launch_t<0>(p, workspace, workspace_bytes, s)
           : type == 1 ? launch_t<1>(p, workspace, workspace_bytes, s)
                       : launch_t<2>(p, workspace, workspace_bytes, s);
}

}  // namespace bq
