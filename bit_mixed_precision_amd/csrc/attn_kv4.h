// What the kernels of attention over the 4-bit paged cache share: which keys a
// tile of query rows attends to, the masks of drafted trees, and the join of a
// split sequence's parts.
#pragma once

#include "attn_rows.h"
#include "bq_layer_internal.h"
#include "dtype16.h"

namespace bq {
namespace {

constexpr int kWaves = 4, kMany = 8;  // wavefronts of a workgroup
constexpr int kTile = 32;      // tokens of a step
constexpr float kNoMax = -3.0e38f;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// What one tile of 16 query rows attends to.
struct Rows {
    int q0;          // first row of the sequence's queries in q / out
    int rows;        // query rows of the sequence and kv head (computed queries * group)
    int base;        // position of the first query
    int pos_min, pos_max;
    int lo, hi;      // keys [lo, hi), lo a multiple of kTile
    int chunk;       // keys of one split
};

// Queries of sequence b.
__device__ __forceinline__ QueryRows query_rows(const AttnKv4Args &p, int b)
{
    if (p.q_start)
        return query_rows_of(p.q_start[b], p.q_start[b + 1], p.total_q, p.max_q_len);
    return {b * p.max_q_len, p.max_q_len, p.max_q_len};
}

// Rows `tile` * ROWS on of sequence b.  Every split takes `chunk` keys, the
// same for all sequences: workgroups then last equally long, and the shorter
// sequences' last splits are empty.  TREE: the queries are a tree's nodes, key
// base + i for node i, and see all keys before base; pos_min is the last of
// those that every row sees.
template <int ROWS, bool TREE>
__device__ __forceinline__ Rows rows_of(const AttnKv4Args &p, int b, int tile)
{
    Rows r;
    const QueryRows q = query_rows(p, b);
    r.q0 = q.first;
    r.rows = q.count * p.group;
    const int len = min(max(p.seq_lens[b], 0), p.max_blocks << p.page_shift);
    r.base = len - q.len;
    const int first = tile * ROWS / p.group, last = min(tile * ROWS + ROWS - 1, r.rows - 1) / p.group;
    r.pos_min = r.base + first;
    r.pos_max = r.base + last;
    if constexpr (TREE) {
        r.pos_min = r.base - 1;
        r.pos_max = min(len, r.base + 32 * p.mask_words) - 1;
    }
    r.lo = p.window > 0 ? max(0, r.pos_min - p.window + 1) & ~(kTile - 1) : 0;
    r.hi = max(r.pos_max + 1, r.lo);
    r.chunk = r.hi - r.lo;
    if (p.nsplit > 1) {
        int most = 0;
        for (int i = threadIdx.x & 63; i < p.batch; i += 64)
            most = max(most, p.seq_lens[i]);
#pragma unroll
        for (int off = 32; off > 0; off >>= 1)
            most = max(most, __shfl_xor(most, off, 64));
        most = min(most, p.max_blocks << p.page_shift);
        if (p.window > 0)  // keys of ROWS rows: their positions (or the nodes), the window, lo's alignment
            most = min(most, p.window + (TREE ? 32 * p.mask_words : (ROWS - 1) / p.group + 1) + kTile);
        constexpr int step = kTile * kWaves;
        r.chunk = __builtin_amdgcn_readfirstlane(((most + p.nsplit - 1) / p.nsplit + step - 1) / step * step);
    }
    return r;
}

// What one row of a tree's mask says.
struct TreeRow {
    const uint32_t *words;
    int low, high;    // its nodes are [low, high): those that are keys, and have a bit
    int first;        // first key of the prefix that it sees
    int nodes;        // nodes that it sees, with a window at most that many

    __device__ __forceinline__ uint32_t word(int k) const
    {
        if (32 * k >= high || 32 * k + 32 <= low || k < 0)
            return 0;
        uint32_t w = words[k];
        if (32 * k + 32 > high)
            w &= ~0u >> (32 * k + 32 - high);
        if (32 * k < low)
            w &= ~0u << (low - 32 * k);
        return w;
    }
    // The nodes of word k that lie in the window: the last `nodes` of the row's.
    __device__ __forceinline__ uint32_t seen(int k) const
    {
        uint32_t w = word(k);
        if (nodes < high - low) {
            int left = nodes;
            for (int i = (high - 1) >> 5; i > k; --i)
                left -= __popc(word(i));
            for (int over = __popc(w) - max(left, 0); over > 0; --over)
                w &= w - 1;
        }
        return w;
    }
    // Bits of the keys t .. t + 31 that the row sees.
    __device__ __forceinline__ uint32_t keys(int t, int base) const
    {
        const int at = t - base;  // node of key t
        uint32_t on = 0;
        if (at < 0) {
            on = at > -32 ? ~0u >> (32 + at) : ~0u;
            if (first > t)
                on = first < t + 32 ? on & (~0u << (first - t)) : 0;
            if (at > -32)
                on |= seen(0) << -at;
        } else {
            on = seen(at >> 5) >> (at & 31);
            if (at & 31)
                on |= seen((at >> 5) + 1) << (32 - (at & 31));
        }
        return on;
    }
};

__device__ __forceinline__ TreeRow tree_row(const AttnKv4Args &p, const Rows &r, int len, int qi)
{
    TreeRow x;
    x.words = p.tree_mask + (int64_t)(r.q0 + qi) * p.mask_words;
    x.low = max(-r.base, 0);
    x.high = min(len, 32 * p.mask_words);
    x.first = 0;
    x.nodes = x.high;
    if (p.window > 0) {
        int n = 0;
        for (int k = 0; 32 * k < x.high; ++k)
            n += __popc(x.word(k));
        x.nodes = min(n, p.window);
        x.first = r.base - (p.window - x.nodes);
    }
    return x;
}

// Joins the splits of one query row: D/4 threads a split, blockDim.x of them.
template <typename T, int D, int RT, bool TREE>
__global__ __launch_bounds__(256) void attn_kv4_join(const AttnKv4Args p)
{
    constexpr int TPS = D / 4, ROWS = 16 * RT;
    __shared__ float4 so[256];
    const int item = blockIdx.x / p.join_rows, jr = blockIdx.x % p.join_rows;
    const int tile = item % p.row_tiles;
    const int head = item / p.row_tiles % p.hkv;
    const int b = item / p.row_tiles / p.hkv;
    const Rows r = rows_of<ROWS, TREE>(p, b, tile);
    const int row = tile * ROWS + jr;
    if (row >= r.rows)
        return;
    const int n = r.hi > r.lo ? (r.hi - r.lo + r.chunk - 1) / r.chunk : 1;
    const int64_t first = (int64_t)item * p.nsplit * ROWS + jr;
    const int lane = threadIdx.x & 63;
    // every wavefront holds all splits' maxima and sums, one a lane (nsplit <= 64)
    const float2 ml = lane < n ? *(const float2 *)(p.part_ml + (first + ROWS * lane) * 2) : make_float2(kNoMax, 0.0f);
    float mm = ml.x;
#pragma unroll
    for (int off = 32; off > 0; off >>= 1)
        mm = fmaxf(mm, __shfl_xor(mm, off, 64));
    const float f = __builtin_amdgcn_exp2f(ml.x - mm);
    float l = f * ml.y;
#pragma unroll
    for (int off = 32; off > 0; off >>= 1)
        l += __shfl_xor(l, off, 64);
    const int G = blockDim.x / TPS, gq = threadIdx.x / TPS, c = threadIdx.x % TPS;
    float4 acc = make_float4(0, 0, 0, 0);
    for (int s0 = 0; s0 < n; s0 += G) {
        const int s = s0 + gq;
        const float fs = __shfl(f, s & 63, 64);
        if (s < n) {
            const float4 o = *(const float4 *)(p.part + (first + ROWS * (int64_t)s) * D + 4 * c);
            acc.x += fs * o.x;
            acc.y += fs * o.y;
            acc.z += fs * o.z;
            acc.w += fs * o.w;
        }
    }
    so[threadIdx.x] = acc;
    __syncthreads();
    if (gq == 0) {
        for (int k = 1; k < G; ++k) {
            const float4 o = so[k * TPS + c];
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

// Launches the join of `items` tiles of 16 * RT rows.
template <typename T, int D, int RT, bool TREE>
hipError_t launch_join(const AttnKv4Args &p, int64_t items, hipStream_t s)
{
    int groups = 1;  // splits joined side by side: whole wavefronts, up to 256 threads
    while (groups * (D / 4) < 256 && (groups < p.nsplit || groups * (D / 4) < 64))
        groups *= 2;
    attn_kv4_join<T, D, RT, TREE><<<dim3((unsigned)(items * p.join_rows)), groups * (D / 4), 0, s>>>(p);
    return hipGetLastError();
}

}  // namespace
}  // namespace bq
