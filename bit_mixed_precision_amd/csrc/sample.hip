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
// ascending): its last token's key and index.  Top-k finds it where a count
// is reached, top-p where a sum of units is, the drawn token where a sum in the
// order of indices is: all three are one radix select, a histogram of eight
// more bits at a time.
//
// Three kernels, each once over the logits, the first from memory and the others
// from the caches:
//   greatest   the greatest logit of every group of a row's lanes;
//   weigh      a row with a top_k of at most as many as there are groups: no
//              token below the top_k-th greatest group can be kept, those above
//              it are written out, a few more than top_k.  Another row: the
//              units of each quarter of an octave of weight, per workgroup;
//   draw       one workgroup a row.  Few tokens written out: all from these, in
//              LDS.  Units per quarter octave: the limit lies in one of them,
//              whose tokens are gathered into LDS; the sums over the others give
//              the part of the row that the drawn token is in, which is read
//              again.  If more must be gathered than LDS holds (a row of equal
//              logits), all selects run over the row itself.
// Without a workspace the last form is used alone.
#include "bq_decode_internal.h"
#include "dtype16.h"

namespace bq {
namespace {

typedef unsigned long long u64;

constexpr int kThreads = 1024, kWaves = kThreads / 64;  // of a workgroup that has a row
constexpr int kPart = 4;                                // wavefronts of one that has a part of a row
constexpr uint32_t kNone = 0x007fffffu;                 // keys up to that of -infinity are no tokens
constexpr int kOct = 192;                               // quarter octaves of weight: 48 octaves, past which nothing is a unit
constexpr int kGroups = 256;                            // groups of a row, at most
constexpr int kRowList = 2048;                          // tokens of a row that are written out, at most
constexpr int kList = 6144;                             // tokens gathered in LDS, at most

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
    // Raw vector v; what is not in the row is -infinity.
    __device__ __forceinline__ u4 load(int v) const
    {
        const int first = v * kE - lead;
        if (first >= 0 && first + kE <= vocab)
            return *(const u4 *)(base + (int64_t)v * 16);
        u4 x;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (TYPE == 2) {
                const int at = first + i;
                x[i] = at >= 0 && at < vocab ? ((const uint32_t *)base)[v * 4 + i] : 0xff800000u;
            } else {
                uint32_t h[2];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int at = first + 2 * i + j;
                    h[j] = at >= 0 && at < vocab ? ((const uint16_t *)base)[v * 8 + 2 * i + j] : (TYPE == 1 ? 0xff80u : 0xfc00u);
                }
                x[i] = h[0] | h[1] << 16;
            }
        }
        return x;
    }
    __device__ __forceinline__ static float value(const u4 &x, int e)
    {
        if constexpr (TYPE == 2)
            return __uint_as_float(x[e]);
        else
            return value(x[e >> 1] >> (16 * (e & 1)));
    }
    // f(index, key) for the tokens of vectors [first, last), as the wavefront's
    // parts of them: 64 neighbouring vectors a step, all lanes at the same step
    // and token of their vector (key 0 past the end).
    template <typename F>
    __device__ __forceinline__ void each(int first, int last, F f) const
    {
        const int part = (last - first + kThreads - 1) / kThreads * 64, lane = threadIdx.x & 63;
        const int v0 = first + (int)(threadIdx.x >> 6) * part, v1 = min(v0 + part, last);
        for (int v = v0; v < v1; v += 64) {
            u4 x = {};
            const bool in = v + lane < v1;
            if (in)
                x = load(v + lane);
#pragma unroll
            for (int e = 0; e < kE; ++e)
                f((v + lane) * kE + e - lead, in ? key_of(value(x, e)) : 0u);
        }
    }
};

// Weights of a row's tokens.
struct Scale {
    uint32_t top;     // greatest key
    double max, c;    // y = (max - x) c
    int frac;

    __device__ __forceinline__ double octaves(uint32_t key) const
    {
        return key == top ? 0.0 : (max - (double)value_of(key)) * c;
    }
    __device__ __forceinline__ static int bin(double y) { return y < 0.25 * kOct ? (int)(y * 4.0) : kOct; }
    // 2^-y in units, to the nearest: 2^r by its series, whose remainder is below
    // 2^-47, |r| <= 1/2.
    __device__ __forceinline__ u64 units(double y) const
    {
        constexpr double l = 0.693147180559945309417;
        constexpr double c1 = l, c2 = c1 * l / 2, c3 = c2 * l / 3, c4 = c3 * l / 4, c5 = c4 * l / 5, c6 = c5 * l / 6,
                         c7 = c6 * l / 7, c8 = c7 * l / 8, c9 = c8 * l / 9, c10 = c9 * l / 10, c11 = c10 * l / 11;
        if (!(y < 0.25 * kOct))
            return 0;
        const double n = __builtin_rint(y), r = n - y;
        double p = c11;
        p = __builtin_fma(p, r, c10);
        p = __builtin_fma(p, r, c9);
        p = __builtin_fma(p, r, c8);
        p = __builtin_fma(p, r, c7);
        p = __builtin_fma(p, r, c6);
        p = __builtin_fma(p, r, c5);
        p = __builtin_fma(p, r, c4);
        p = __builtin_fma(p, r, c3);
        p = __builtin_fma(p, r, c2);
        p = __builtin_fma(p, r, c1);
        p = __builtin_fma(p, r, 1.0);
        // with 2^52 added, the number's low bits are the rounded integer
        const double scale = __hiloint2double((1023 + frac - (int)n) << 20, 0);
        return (u64)__double_as_longlong(__builtin_fma(p, scale, 0x1p52)) & 0xfffffffffffffull;
    }
    __device__ __forceinline__ u64 units_of(uint32_t key) const { return units(octaves(key)); }
};

// A row's settings.
struct Settings {
    bool greedy;
    int top_k;             // 0: off
    bool has_p;
    double top_p, far, u;  // far: octaves within which min-p keeps tokens

    __device__ __forceinline__ Settings(const SampleArgs &p, int b, Scale &s)
    {
        const float t = p.temperature ? p.temperature[b] : 1.0f;
        greedy = !(t > 0.0f);
        s.max = value_of(s.top);
        s.c = 1.4426950408889634074 / (double)fminf(t, 3.402823466e38f);
        s.frac = p.frac;
        const int k = p.top_k ? p.top_k[b] : 0;
        top_k = k > 0 && k < p.vocab ? k : 0;
        const float tp = p.top_p ? p.top_p[b] : 1.0f, mp = p.min_p ? p.min_p[b] : 0.0f;
        has_p = tp < 1.0f;
        top_p = fmaxf(tp, 0.0f);
        far = mp > 0.0f ? -log2(fmin((double)mp, 1.0)) + 0x1p-53 : 1e300;
        u = p.u[b];
    }
    // The sum that top-p must reach, and the one that the drawn token must pass.
    __device__ __forceinline__ u64 reach(u64 total) const { return max((u64)ceil(top_p * (double)total), 1ull); }
    __device__ __forceinline__ u64 pass(u64 total) const
    {
        return u < 1.0 ? min(total - 1, (u64)floor(fmax(u, 0.0) * (double)total)) : total - 1;
    }
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
    uint32_t keys[kWaves];
    int places[kWaves];
    u64 before;
    uint32_t bin;
    int count;
};

template <typename V>
__device__ __forceinline__ V wave_sum(V v)
{
#pragma unroll
    for (int off = 32; off > 0; off >>= 1)
        v += __shfl_xor(v, off, 64);
    return v;
}
__device__ __forceinline__ u64 wave_scan(u64 v)  // sums over the lanes up to each
{
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
        const u64 x = __shfl_up(v, off, 64);
        v += (threadIdx.x & 63) >= off ? x : 0;
    }
    return v;
}

// Sum over the workgroup, in every thread; sh.sums has each wavefront's.
__device__ __forceinline__ u64 block_sum(Shared &sh, u64 v)
{
    v = wave_sum(v);
    __syncthreads();
    if ((threadIdx.x & 63) == 0)
        sh.sums[threadIdx.x >> 6] = v;
    __syncthreads();
    u64 total = 0;
    for (int w = 0; w < kWaves; ++w)
        total += sh.sums[w];
    return total;
}

// First of n amounts, four a lane in the first wavefront, at which their sum
// reaches `stop`: sh.bin, and sh.before what lies before it; n if none does.
__device__ __forceinline__ void find(Shared &sh, const u64 *amount, int n, bool backwards, u64 stop)
{
    if (threadIdx.x < 64) {
        u64 a[4], mine = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int at = 4 * threadIdx.x + i;
            a[i] = at < n ? amount[backwards ? n - 1 - at : at] : 0;
            mine += a[i];
        }
        const u64 upto = wave_scan(mine);
        const u64 there = __ballot(upto >= stop);
        if (there ? (int)threadIdx.x == __ffsll(there) - 1 : threadIdx.x == 63) {
            u64 sum = upto - mine;
            int i = 0;
            for (; i < 4 && sum + a[i] < stop; ++i)
                sum += a[i];
            const int at = there ? 4 * (int)threadIdx.x + i : n;
            sh.bin = backwards && at < n ? n - 1 - at : at;
            sh.before = sum;
        }
    }
    __syncthreads();
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
    for (int shift = 24; shift >= 0; shift -= 8) {
        __syncthreads();
        for (int i = threadIdx.x; i < 256; i += kThreads)
            sh.hist[i] = 0;
        __syncthreads();
        const uint32_t high = shift == 24 ? 0u : ~0u << (shift + 8);
        items([&](uint32_t x, u64 amount) {
            if ((x & high) == number)
                atomicAdd(&sh.hist[x >> shift & 255], amount);
        });
        __syncthreads();
        find(sh, sh.hist, 256, true, stop - before);
        if (sh.bin == 256)
            return false;
        number |= sh.bin << shift;
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

__device__ __forceinline__ void answer(const SampleArgs &p, int b, int token, double logprob)
{
    p.tokens[b] = token;
    if (p.logprobs)
        p.logprobs[b] = (float)logprob;
}

// Draws the token whose units, in the order of indices, pass `want` of the kept
// units of vectors [first, last), of which `sum` lie before the first.
template <int TYPE, typename Kept>
__device__ void draw_from(Shared &sh, const SampleArgs &p, int b, const Row<TYPE> &row, int first, int last, Kept kept, u64 want,
                          u64 before, u64 total)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    u64 mine = 0;
    row.each(first, last, [&](int i, uint32_t k) { mine += kept(i, k); });
    block_sum(sh, mine);
    u64 sum = before;
    for (int w = 0; w < wave; ++w)
        sum += sh.sums[w];
    if (sum > want || sum + sh.sums[wave] <= want)
        return;
    // this wavefront's part has it: one step after another, a step's tokens lane by lane
    constexpr int E = Row<TYPE>::kE;
    const int part = (last - first + kThreads - 1) / kThreads * 64;
    const int v0 = first + wave * part, v1 = min(v0 + part, last);
    for (int v = v0; v < v1; v += 64) {
        u64 n[E], lane_sum = 0;
        u4 x = {};
        const bool in = v + lane < v1;
        if (in)
            x = row.load(v + lane);
#pragma unroll
        for (int e = 0; e < E; ++e) {
            n[e] = in ? kept((v + lane) * E + e - row.lead, key_of(row.value(x, e))) : 0;
            lane_sum += n[e];
        }
        const u64 upto = wave_scan(lane_sum) + sum;
        const u64 past = __ballot(upto > want);
        if (past) {
            if (lane == __ffsll(past) - 1) {
                u64 s = upto - lane_sum;
                bool done = false;
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    s += n[e];
                    if (!done && s > want) {
                        done = true;
                        answer(p, b, (v + lane) * E + e - row.lead, log((double)n[e] / (double)total));
                    }
                }
            }
            return;
        }
        sum = __shfl(upto, 63, 64);
    }
}

// All of a row's work over the row itself; s.top is known.
template <int TYPE>
__device__ __noinline__ void draw_slowly(Shared &sh, const SampleArgs &p, int b, const Row<TYPE> &row, const Scale &s, const Settings &set)
{
    const int n = row.vectors();
    Limit limit = {kNone, 0};
    // zero units are no tokens here: they are not drawn, and add to no sum
    auto tokens = [&](auto f) {
        row.each(0, n, [&](int i, uint32_t k) {
            if (k > kNone && limit.keeps(i, k))
                f(i, k);
        });
    };
    if (set.top_k) {
        Limit to;
        if (limit_at(sh, tokens, [](uint32_t) { return (u64)1; }, (u64)set.top_k, to))
            limit = to;
    }
    if (set.has_p) {
        u64 mine = 0;
        tokens([&](int, uint32_t k) { mine += s.units_of(k); });
        const u64 stop = set.reach(block_sum(sh, mine));
        Limit to;
        if (limit_at(sh, tokens, [&](uint32_t k) { return s.units_of(k); }, stop, to))
            limit = to;
    }
    auto kept = [&](int i, uint32_t k) {
        if (k <= kNone || !limit.keeps(i, k))
            return (u64)0;
        const double y = s.octaves(k);
        return y <= set.far ? s.units(y) : 0;
    };
    u64 mine = 0;
    row.each(0, n, [&](int i, uint32_t k) { mine += kept(i, k); });
    const u64 total = block_sum(sh, mine);
    draw_from(sh, p, b, row, 0, n, kept, set.pass(total), 0, total);
}

// The greatest key, of the lowest index, of pairs over the workgroup; in every thread.
template <int WAVES>
__device__ __forceinline__ void block_greatest(uint32_t *keys, int *places, uint32_t &key, int &place)
{
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) {
        const uint32_t k = __shfl_xor(key, off, 64);
        const int i = __shfl_xor(place, off, 64);
        if (k > key || (k == key && i < place)) {
            key = k;
            place = i;
        }
    }
    __syncthreads();
    if ((threadIdx.x & 63) == 0) {
        keys[threadIdx.x >> 6] = key;
        places[threadIdx.x >> 6] = place;
    }
    __syncthreads();
#pragma unroll
    for (int w = 0; w < WAVES; ++w)
        if (keys[w] > key || (keys[w] == key && places[w] < place)) {
            key = keys[w];
            place = places[w];
        }
}

template <int TYPE>
__global__ __launch_bounds__(kThreads) void sample_kernel(const SampleArgs p)
{
    __shared__ Shared sh;
    const int b = blockIdx.x;
    const Row<TYPE> row(p, b);
    uint32_t key = 0;
    int place = p.vocab;
    row.each(0, row.vectors(), [&](int i, uint32_t k) {
        if (k > key) {
            key = k;
            place = i;
        }
    });
    block_greatest<kWaves>(sh.keys, sh.places, key, place);
    Scale s;
    s.top = key;
    const Settings set(p, b, s);
    if (key <= kNone || set.greedy) {
        if (threadIdx.x == 0)
            answer(p, b, key <= kNone ? -1 : place, key <= kNone ? -__builtin_inf() : 0.0);
        return;
    }
    draw_slowly(sh, p, b, row, s, set);
}

// How rows are shared between workgroups, and where what they find is kept.
struct Parts {
    int steps;    // of 64 vectors, a wavefront
    int waves;    // a row, a multiple of kPart
    int lanes;    // of a group: 16 or 64
    int groups;
    int64_t row_bytes;   // of lists or histograms
    uint32_t *greatest;  // [rows][groups]
    uint2 *first;        // [rows][waves / kPart]: greatest key and its first place
    uint8_t *found;      // [rows][row_bytes]

    __host__ __device__ int parts() const { return waves / kPart; }
    // a row's list and its length, or its histograms [parts][kOct] of units, then
    // of tokens
    __device__ uint2 *list(int b) const { return (uint2 *)(found + b * row_bytes); }
    __device__ uint32_t *length(int b) const { return (uint32_t *)(list(b) + kRowList); }
    __device__ u64 *units(int b) const { return (u64 *)(found + b * row_bytes); }
    __device__ uint32_t *tokens(int b) const { return (uint32_t *)(units(b) + parts() * kOct); }
};

template <int TYPE>
__global__ __launch_bounds__(64 * kPart) void greatest_kernel(const SampleArgs p, const Parts q)
{
    constexpr int E = Row<TYPE>::kE;
    __shared__ uint32_t keys[kPart];
    __shared__ int places[kPart];
    const int b = blockIdx.x / q.parts(), part = blockIdx.x % q.parts(), lane = threadIdx.x & 63;
    const int wave = part * kPart + (threadIdx.x >> 6);
    const Row<TYPE> row(p, b);
    const int n = row.vectors(), first = wave * q.steps * 64;
    uint32_t key = 0;
    int place = p.vocab;
#pragma unroll 4
    for (int s = 0; s < q.steps; ++s) {
        const int v = first + s * 64 + lane;
        if (v >= n)
            continue;
        const u4 x = row.load(v);
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const uint32_t k = key_of(row.value(x, e));
            if (k > key) {
                key = k;
                place = v * E + e - row.lead;
            }
        }
    }
    uint32_t g = key;
    for (int off = 1; off < q.lanes; off <<= 1)
        g = max(g, (uint32_t)__shfl_xor(g, off, 64));
    if (lane % q.lanes == 0)
        q.greatest[(int64_t)b * q.groups + wave * (64 / q.lanes) + lane / q.lanes] = g;
    block_greatest<kPart>(keys, places, key, place);
    if (threadIdx.x == 0) {
        q.first[(int64_t)b * q.parts() + part] = make_uint2(key, (uint32_t)place);
        if (part == 0)
            *q.length(b) = 0;
    }
}

template <int TYPE>
__global__ __launch_bounds__(64 * kPart) void weigh_kernel(const SampleArgs p, const Parts q)
{
    constexpr int E = Row<TYPE>::kE;
    static_assert(kGroups == 64 * kPart, "a thread a group");
    __shared__ uint32_t groups[kGroups];
    __shared__ uint32_t keys[kPart];
    __shared__ int places[kPart];
    __shared__ uint32_t low;
    __shared__ u64 units[kOct];
    __shared__ uint32_t tokens[kOct];
    const int b = blockIdx.x / q.parts(), part = blockIdx.x % q.parts(), lane = threadIdx.x & 63;
    const int wave = part * kPart + (threadIdx.x >> 6);
    const uint32_t mine = (int)threadIdx.x < q.groups ? q.greatest[(int64_t)b * q.groups + threadIdx.x] : 0u;
    groups[threadIdx.x] = mine;
    uint32_t key = mine;
    int place = 0;
    block_greatest<kPart>(keys, places, key, place);
    Scale s;
    s.top = key;
    const Settings set(p, b, s);
    if (key <= kNone || set.greedy)
        return;
    const Row<TYPE> row(p, b);
    const int n = row.vectors(), first = wave * q.steps * 64;
    if (set.top_k && set.top_k <= q.groups) {
        // the top_k-th greatest group: at least top_k tokens are as great
        int rank = 0;
        for (int i = 0; i < q.groups; ++i)
            rank += groups[i] > mine || (groups[i] == mine && i < (int)threadIdx.x);
        if ((int)threadIdx.x < q.groups && rank == set.top_k - 1)
            low = mine;
        __syncthreads();
        const uint32_t least = max(low, kNone + 1);
        uint2 *list = q.list(b);
        for (int st = 0; st < q.steps; ++st) {
            const int v = first + st * 64 + lane;
            u4 x = {};
            uint32_t on = 0;
            if (v < n) {
                x = row.load(v);
#pragma unroll
                for (int e = 0; e < E; ++e)
                    on |= (uint32_t)(key_of(row.value(x, e)) >= least) << e;
            }
            if (!__any(on))
                continue;
            // in any order: what is drawn from the list does not depend on it
            uint32_t at = 0;
            const uint32_t upto = (uint32_t)wave_scan(__popc(on));
            if (lane == 63)
                at = atomicAdd(q.length(b), upto);
            at = __shfl(at, 63, 64) + upto - __popc(on);
#pragma unroll
            for (int e = 0; e < E; ++e)
                if (on >> e & 1) {
                    if (at < kRowList)
                        list[at] = make_uint2(key_of(row.value(x, e)), (uint32_t)(v * E + e - row.lead));
                    ++at;
                }
        }
        return;
    }
    if (threadIdx.x < kOct) {
        units[threadIdx.x] = 0;
        tokens[threadIdx.x] = 0;
    }
    __syncthreads();
    for (int st = 0; st < q.steps; ++st) {
        const int v = first + st * 64 + lane;
        if (v >= n)
            continue;
        const u4 x = row.load(v);
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const uint32_t k = key_of(row.value(x, e));
            const double y = s.octaves(k);
            if (k > kNone && y < 0.25 * kOct) {
                atomicAdd(&units[s.bin(y)], s.units(y));
                if (set.top_k)
                    atomicAdd(&tokens[s.bin(y)], 1u);
            }
        }
    }
    __syncthreads();
    if (threadIdx.x < kOct) {
        q.units(b)[part * kOct + threadIdx.x] = units[threadIdx.x];
        if (set.top_k)
            q.tokens(b)[part * kOct + threadIdx.x] = tokens[threadIdx.x];
    }
}

template <int TYPE>
__global__ __launch_bounds__(kThreads) void draw_kernel(const SampleArgs p, const Parts q)
{
    __shared__ Shared sh;
    __shared__ uint2 list[kList];
    __shared__ u64 units[kOct], amount[kGroups];
    const int b = blockIdx.x, parts = q.parts();
    uint32_t key = 0;
    int place = p.vocab;
    for (int i = threadIdx.x; i < parts; i += kThreads) {
        const uint2 x = q.first[(int64_t)b * parts + i];
        if (x.x > key) {
            key = x.x;
            place = (int)x.y;
        }
    }
    block_greatest<kWaves>(sh.keys, sh.places, key, place);
    Scale s;
    s.top = key;
    const Settings set(p, b, s);
    if (key <= kNone || set.greedy) {
        if (threadIdx.x == 0)
            answer(p, b, key <= kNone ? -1 : place, key <= kNone ? -__builtin_inf() : 0.0);
        return;
    }
    const Row<TYPE> row(p, b);
    Limit limit = {kNone, 0};
    int n = 0;  // of the list
    auto tokens = [&](auto f) {
        for (int i = threadIdx.x; i < n; i += kThreads) {
            const uint2 x = list[i];
            if (limit.keeps((int)x.y, x.x))
                f((int)x.y, x.x);
        }
    };
    auto by_units = [&](uint32_t k) { return s.units_of(k); };
    auto by_count = [](uint32_t) { return (u64)1; };

    if (set.top_k && set.top_k <= q.groups) {
        n = (int)min(*q.length(b), (uint32_t)kRowList + 1);
        if (n > kRowList) {
            draw_slowly(sh, p, b, row, s, set);
            return;
        }
        for (int i = threadIdx.x; i < n; i += kThreads)
            list[i] = q.list(b)[i];
        __syncthreads();
        Limit to;
        if (limit_at(sh, tokens, by_count, (u64)set.top_k, to))
            limit = to;
        if (set.has_p) {
            u64 mine = 0;
            tokens([&](int, uint32_t k) { mine += s.units_of(k); });
            const u64 stop = set.reach(block_sum(sh, mine));
            if (limit_at(sh, tokens, by_units, stop, to))
                limit = to;
        }
        auto kept = [&](uint32_t k) {
            const double y = s.octaves(k);
            return y <= set.far ? s.units(y) : 0;
        };
        u64 mine = 0;
        tokens([&](int, uint32_t k) { mine += kept(k); });
        const u64 total = block_sum(sh, mine);
        uint32_t at;
        u64 before;
        select(sh, [&](auto f) { tokens([&](int i, uint32_t k) { f(~(uint32_t)i, kept(k)); }); }, set.pass(total) + 1, at, before);
        tokens([&](int i, uint32_t k) {
            if (i == (int)~at)
                answer(p, b, i, log((double)kept(k) / (double)total));
        });
        return;
    }

    // the whole row's units per quarter octave
    auto sum_up = [&](const auto *from) {
        __syncthreads();
        if (threadIdx.x < kOct)
            amount[threadIdx.x] = 0;
        __syncthreads();
        for (int i = threadIdx.x; i < parts * kOct; i += kThreads)
            if (from[i])
                atomicAdd(&amount[i % kOct], (u64)from[i]);
        __syncthreads();
    };
    // gathers the tokens of a quarter octave; false: too many
    int gathered = -1;
    auto gather = [&](int bin) {
        if (bin == gathered)
            return true;
        __syncthreads();
        if (threadIdx.x == 0)
            sh.count = 0;
        __syncthreads();
        row.each(0, row.vectors(), [&](int i, uint32_t k) {
            if (k > kNone && s.bin(s.octaves(k)) == bin) {
                const int at = atomicAdd(&sh.count, 1);
                if (at < kList)
                    list[at] = make_uint2(k, (uint32_t)i);
            }
        });
        __syncthreads();
        n = min(sh.count, kList);
        gathered = bin;
        return sh.count <= kList;
    };
    int edge = kOct;  // tokens of heavier quarter octaves are kept, those of this one by the limit
    if (set.top_k) {
        sum_up(q.tokens(b));
        find(sh, amount, kOct, false, (u64)set.top_k);
        const int bin = (int)sh.bin;
        const u64 before = sh.before;
        if (bin < kOct) {
            Limit to;
            if (!gather(bin)) {
                draw_slowly(sh, p, b, row, s, set);
                return;
            }
            limit_at(sh, tokens, by_count, (u64)set.top_k - before, to);
            limit = to;
            edge = bin;
        }
    }
    sum_up(q.units(b));
    if (threadIdx.x < kOct)
        units[threadIdx.x] = amount[threadIdx.x];
    if (set.has_p) {
        // of the edge's tokens those that top-k keeps
        u64 mine = 0;
        if (edge < kOct)
            tokens([&](int, uint32_t k) { mine += s.units_of(k); });
        const u64 in_edge = block_sum(sh, mine);
        if (edge < kOct && threadIdx.x >= (unsigned)edge && threadIdx.x < kOct)
            units[threadIdx.x] = threadIdx.x == (unsigned)edge ? in_edge : 0;
        const u64 total = block_sum(sh, threadIdx.x < kOct ? units[threadIdx.x] : 0);
        const u64 stop = set.reach(total);
        find(sh, units, kOct, false, stop);
        const int bin = (int)sh.bin;
        const u64 before = sh.before;
        if (bin < kOct) {
            if (!gather(bin)) {
                draw_slowly(sh, p, b, row, s, set);
                return;
            }
            Limit to;
            limit_at(sh, tokens, by_units, stop - before, to);
            limit = to;
            edge = bin;
        }
    }
    const int far = s.bin(set.far);
    if (far < edge) {
        if (!gather(far)) {
            draw_slowly(sh, p, b, row, s, set);
            return;
        }
        edge = far;
    }
    auto kept = [&](int i, uint32_t k) {
        if (k <= kNone || !limit.keeps(i, k))
            return (u64)0;
        const double y = s.octaves(k);
        return y <= set.far ? s.units(y) : 0;
    };
    // what each part of the row keeps
    __syncthreads();
    if (threadIdx.x < kGroups)
        amount[threadIdx.x] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < parts * kOct; i += kThreads)
        if (i % kOct < edge) {
            const u64 x = q.units(b)[i];
            if (x)
                atomicAdd(&amount[i / kOct], x);
        }
    const int part_vectors = q.steps * 64 * kPart;
    if (edge < kOct)
        tokens([&](int i, uint32_t k) {
            const u64 x = kept(i, k);
            if (x)
                atomicAdd(&amount[(i + row.lead) / Row<TYPE>::kE / part_vectors], x);
        });
    __syncthreads();
    const u64 total = block_sum(sh, threadIdx.x < kGroups ? amount[threadIdx.x] : 0);
    const u64 want = set.pass(total);
    find(sh, amount, parts, false, want + 1);
    const int part = (int)sh.bin;
    const u64 before = sh.before;
    draw_from(sh, p, b, row, part * part_vectors, min((part + 1) * part_vectors, row.vectors()), kept, want, before, total);
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
    const int64_t lists = kRowList * 8 + 4, hists = q.parts() * kOct * 12;
    q.row_bytes = ((lists > hists ? lists : hists) + 15) / 16 * 16;
    return q;
}

// Rows of fewer tokens than that are one workgroup's.
bool shared(int64_t vocab) { return vocab >= 2048; }

template <int TYPE>
hipError_t launch_t(const SampleArgs &p, void *workspace, int64_t workspace_bytes, hipStream_t s)
{
    const int64_t need = sample_workspace_bytes(p.rows, p.vocab, TYPE);
    if (need == 0 || workspace_bytes < need) {
        if (!grid_fits(p.rows, kThreads))
            return kGridTooLarge;
        sample_kernel<TYPE><<<dim3((unsigned)p.rows), kThreads, 0, s>>>(p);
        return hipGetLastError();
    }
    Parts q = parts_of(p.rows, p.vocab, TYPE);
    q.found = (uint8_t *)workspace;
    q.first = (uint2 *)(q.found + p.rows * q.row_bytes);
    q.greatest = (uint32_t *)(q.first + (int64_t)p.rows * q.parts());
    const int64_t items = (int64_t)p.rows * q.parts();
    if (!grid_fits(items, 64 * kPart) || !grid_fits(p.rows, kThreads))
        return kGridTooLarge;
    greatest_kernel<TYPE><<<dim3((unsigned)items), 64 * kPart, 0, s>>>(p, q);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess)
        return e;
    weigh_kernel<TYPE><<<dim3((unsigned)items), 64 * kPart, 0, s>>>(p, q);
    if ((e = hipGetLastError()) != hipSuccess)
        return e;
    draw_kernel<TYPE><<<dim3((unsigned)p.rows), kThreads, 0, s>>>(p, q);
    return hipGetLastError();
}

}  // namespace

int64_t sample_workspace_bytes(int64_t rows, int64_t vocab, int type)
{
    if (rows == 0 || !shared(vocab))
        return 0;
    const Parts q = parts_of(rows, vocab, type);
    return rows * (q.row_bytes + q.parts() * 8 + q.groups * 4);
}

hipError_t launch_sample(const SampleArgs &p, int type, void *workspace, int64_t workspace_bytes, hipStream_t s)
{
    return type == 0   ? launch_t<0>(p, workspace, workspace_bytes, s)
           : type == 1 ? launch_t<1>(p, workspace, workspace_bytes, s)
                       : launch_t<2>(p, workspace, workspace_bytes, s);
}

}  // namespace bq
