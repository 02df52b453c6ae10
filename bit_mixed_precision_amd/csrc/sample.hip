// Sampling with temperature, top-k, top-p and min-p from given random numbers.
//
// Every choice is made on whole numbers: a logit's order by its bits (key),
// its weight w = exp((x - max) / temperature) as a multiple of 2^-frac, from
// the 64-bit exponential.  Sums of such weights are exact in 64 bits, so no
// order of additions, atomics among them, changes a result, and a token is the
// definition's except where two sums lie within the weights' own rounding,
// 2^-45 of the largest for a vocabulary of 2^17 (fp32 sums would move borders
// between tokens that weigh 2^-17 of the whole).
//
// The tokens that are kept are those whose key is above a limit, and the first
// few that have the limit itself.  Top-k and top-p find it as a radix select:
// a histogram of the next bits of the keys that share the limit's bits so far,
// with counts (top-k) or sums of weights (top-p).
#include "bq_decode_internal.h"
#include "dtype16.h"

namespace bq {
namespace {

constexpr int kThreads = 1024, kWaves = kThreads / 64;
constexpr int kBits = 8, kBins = 1 << kBits;
constexpr uint32_t kNone = 0x007fffffu;  // keys up to that of -infinity are no tokens

typedef unsigned long long u64;

// The order of the numbers as unsigned integers; -0 as 0, NaN below all.
__device__ __forceinline__ uint32_t key_of(float x)
{
    if (x != x)
        return 0;
    const uint32_t b = __float_as_uint(x + 0.0f);
    return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t key)
{
    return __uint_as_float(key & 0x80000000u ? key ^ 0x80000000u : ~key);
}

template <int TYPE>
__device__ __forceinline__ uint32_t load_key(const void *row, int i)
{
    if constexpr (TYPE == 2)
        return key_of(((const float *)row)[i]);
    else if constexpr (TYPE == 1)
        return key_of(BF16::to_f32(((const uint16_t *)row)[i]));
    else
        return key_of(F16::to_f32(((const uint16_t *)row)[i]));
}

template <typename V>
__device__ __forceinline__ V wave_sum(V v)
{
#pragma unroll
    for (int off = 32; off > 0; off >>= 1)
        v += __shfl_xor(v, off, 64);
    return v;
}

// One row of logits, as a workgroup works on it.
template <int TYPE>
struct Row {
    const void *data;
    int vocab;
    uint32_t top;    // greatest key
    double max, inv_t, one;
    uint32_t limit;  // kept: keys above it, and the first `ties` of those that equal it
    int ties;

    // Calls f(index, key) for the wavefront's part of the row, 64 neighbouring
    // tokens a step and all lanes at the same step (key 0 past the end).
    template <typename F>
    __device__ __forceinline__ void each(F f) const
    {
        const int part = (vocab + kThreads - 1) / kThreads * 64, lane = threadIdx.x & 63;
        const int first = (threadIdx.x >> 6) * part, last = min(first + part, vocab);
        for (int i = first; i < last; i += 64)
            f(i + lane, i + lane < last ? load_key<TYPE>(data, i + lane) : 0u);
    }
    // The weight, relative to the greatest, before it is rounded to units.
    __device__ __forceinline__ double weight(uint32_t key) const
    {
        return key == top ? 1.0 : exp(((double)value_of(key) - max) * inv_t);
    }
    __device__ __forceinline__ u64 units(double w) const { return (u64)__double2ll_rn(w * one); }
};

struct Shared {
    u64 hist[kBins];
    u64 sums[kWaves];
    uint32_t keys[kWaves];
    int places[kWaves];
    u64 before;
    uint32_t bin;
};

// Sum over the workgroup, in every thread.
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

// Ends the kept tokens where their count (or weight) reaches `stop` >= 1.
template <bool WEIGHT, int TYPE>
__device__ void select(Shared &sh, Row<TYPE> &r, u64 stop)
{
    uint32_t prefix = 0;
    u64 before = 0;  // of the keys above the prefix
    for (int shift = 32 - kBits; shift >= 0; shift -= kBits) {
        for (int i = threadIdx.x; i < kBins; i += kThreads)
            sh.hist[i] = 0;
        __syncthreads();
        const uint32_t high = shift + kBits == 32 ? 0u : ~0u << (shift + kBits);
        r.each([&](int, uint32_t k) {
            if (k > kNone && k >= r.limit && (k & high) == prefix)
                atomicAdd(&sh.hist[k >> shift & (kBins - 1)], WEIGHT ? r.units(r.weight(k)) : 1ull);
        });
        __syncthreads();
        if (threadIdx.x == 0) {
            int bin = kBins - 1;
            for (; bin > 0 && before + sh.hist[bin] < stop; --bin)
                before += sh.hist[bin];
            sh.bin = bin;
            sh.before = before;
        }
        __syncthreads();
        before = sh.before;
        prefix |= sh.bin << shift;
    }
    if (prefix < max(r.limit, kNone + 1))
        return;  // fewer than `stop` are there: all stay
    const u64 unit = WEIGHT ? r.units(r.weight(prefix)) : 1ull;
    const u64 ties = unit ? (stop - before + unit - 1) / unit : 1;
    r.ties = (int)min(ties, (u64)(prefix == r.limit ? r.ties : r.vocab));
    r.limit = prefix;
}

template <int TYPE>
__global__ __launch_bounds__(kThreads) void sample_kernel(const SampleArgs p)
{
    __shared__ Shared sh;
    const int b = blockIdx.x, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    Row<TYPE> r;
    r.data = (const uint8_t *)p.logits + (int64_t)b * p.row_stride * (TYPE == 2 ? 4 : 2);
    r.vocab = p.vocab;

    // the greatest logit and its first place
    uint32_t key = 0;
    int place = p.vocab;
    r.each([&](int i, uint32_t k) {
        if (k > key) {
            key = k;
            place = i;
        }
    });
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) {
        const uint32_t k = __shfl_xor(key, off, 64);
        const int i = __shfl_xor(place, off, 64);
        if (k > key || (k == key && i < place)) {
            key = k;
            place = i;
        }
    }
    if (lane == 0) {
        sh.keys[wave] = key;
        sh.places[wave] = place;
    }
    __syncthreads();
    key = sh.keys[0];
    place = sh.places[0];
    for (int w = 1; w < kWaves; ++w)  // parts in the order of indices
        if (sh.keys[w] > key) {
            key = sh.keys[w];
            place = sh.places[w];
        }
    __syncthreads();
    const float t = p.temperature ? p.temperature[b] : 1.0f;
    if (key <= kNone || !(t > 0.0f)) {
        if (threadIdx.x == 0) {
            p.tokens[b] = key <= kNone ? -1 : place;
            if (p.logprobs)
                p.logprobs[b] = key <= kNone ? -__builtin_inff() : 0.0f;
        }
        return;
    }
    r.top = key;
    r.max = value_of(key);
    r.inv_t = 1.0 / (double)fminf(t, 3.402823466e38f);
    r.one = (double)(1ll << p.frac);
    r.limit = kNone;
    r.ties = 0;

    const int top_k = p.top_k ? p.top_k[b] : 0;
    if (top_k > 0 && top_k < p.vocab)
        select<false>(sh, r, (u64)top_k);
    const float top_p = p.top_p ? p.top_p[b] : 1.0f;
    if (top_p < 1.0f) {
        u64 mine = 0;
        r.each([&](int, uint32_t k) {
            if (k > r.limit)
                mine += r.units(r.weight(k));
        });
        const u64 total = block_sum(sh, mine) + (r.ties ? (u64)r.ties * r.units(r.weight(r.limit)) : 0);
        select<true>(sh, r, max((u64)ceil((double)fmaxf(top_p, 0.0f) * (double)total), 1ull));
    }

    // equals of the limit that lie before this wavefront's part
    int before = 0;
    if (r.ties) {
        int equal = 0;
        r.each([&](int, uint32_t k) { equal += k == r.limit; });
        equal = wave_sum(equal);
        if (lane == 0)
            sh.places[wave] = equal;
        __syncthreads();
        for (int w = 0; w < wave; ++w)
            before += sh.places[w];
    }
    const double least = p.min_p && p.min_p[b] > 0.0f ? fmin((double)p.min_p[b], 1.0) : 0.0;
    // f(index, units) for the tokens of this wavefront's part, 0 units for those that are not kept
    auto kept = [&](auto f) {
        int seen = before;
        r.each([&](int i, uint32_t k) {
            bool on = k > r.limit;
            if (r.ties) {
                const u64 equals = __ballot(k == r.limit);
                on |= k == r.limit && seen + __popcll(equals & ((1ull << lane) - 1)) < r.ties;
                seen += __popcll(equals);
            }
            u64 n = 0;
            if (on) {
                const double w = r.weight(k);
                n = k == r.top || !(w < least) ? r.units(w) : 0;
            }
            f(i, n);
        });
    };
    u64 mine = 0;
    kept([&](int, u64 n) { mine += n; });
    const u64 total = block_sum(sh, mine);
    // the token at which the sum passes u * total
    const double u = p.u[b];
    u64 want = total - 1;
    if (u < 1.0)
        want = min(want, (u64)floor(fmax(u, 0.0) * (double)total));
    u64 sum = 0;
    for (int w = 0; w < wave; ++w)
        sum += sh.sums[w];
    if (sum > want || sum + sh.sums[wave] <= want)
        return;
    bool done = false;
    kept([&](int i, u64 n) {
        if (done)
            return;
        u64 upto = n;  // sum over the lanes up to this one
#pragma unroll
        for (int off = 1; off < 64; off <<= 1) {
            const u64 x = __shfl_up(upto, off, 64);
            upto += lane >= off ? x : 0;
        }
        const u64 past = __ballot(sum + upto > want);
        sum += __shfl(upto, 63, 64);
        if (!past)
            return;
        done = true;
        if (lane == __ffsll(past) - 1) {
            p.tokens[b] = i;
            if (p.logprobs)
                p.logprobs[b] = (float)log((double)n / (double)total);
        }
    });
}

}  // namespace

int64_t sample_workspace_bytes(int64_t, int64_t, int) { return 0; }

hipError_t launch_sample(const SampleArgs &p, int type, void *, int64_t, hipStream_t s)
{
    if (!grid_fits(p.rows, kThreads))
        return kGridTooLarge;
    const dim3 grid((unsigned)p.rows);
    if (type == 0)
        sample_kernel<0><<<grid, kThreads, 0, s>>>(p);
    else if (type == 1)
        sample_kernel<1><<<grid, kThreads, 0, s>>>(p);
    else
        sample_kernel<2><<<grid, kThreads, 0, s>>>(p);
    return hipGetLastError();
}

}  // namespace bq
