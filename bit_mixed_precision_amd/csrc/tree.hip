// Trees of drafted tokens: what each node sees, the path that the sampled
// tokens take, and the move of its keys and values behind the prefix.
//
// A tree is small (at most 1024 nodes, usually a few dozen) and a path in it
// short, so all three calls last as long as their chain of dependent loads;
// one workgroup a sequence brings the whole tree into LDS with one of them.  Masks
// of 1 tree of 25 nodes 2.0 us, of 256 of 64 3.5; paths 2.1 and 3.2.
#include "attn_rows.h"
#include "bq_decode_internal.h"
#include "dtype16.h"

namespace bq {
namespace {

constexpr int kMaxNodes = 1024;

__device__ __forceinline__ QueryRows nodes_of(const TreeArgs &t, int b)
{
    if (t.q_start)
        return query_rows_of(t.q_start[b], t.q_start[b + 1], t.total_q, t.max_q_len);
    return {b * t.max_q_len, t.max_q_len, t.max_q_len};
}

// A thread a node walks up to its root.  Ancestors come in descending order,
// so a row's words are finished one after another, the last one first.
__global__ void tree_mask_kernel(const TreeArgs t, const int32_t *parents, int words, uint32_t *mask, int32_t *positions)
{
    __shared__ int up[kMaxNodes];
    const int b = blockIdx.x;
    const QueryRows n = nodes_of(t, b);
    const int first_key = positions && t.seq_lens ? (int)((uint32_t)t.seq_lens[b] - (uint32_t)n.len) : 0;
    for (int i = threadIdx.x; i < n.count; i += blockDim.x) {
        const int p = parents[n.first + i];
        up[i] = p < i ? p : -1;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < n.count; i += blockDim.x) {
        uint32_t *row = mask + (int64_t)(n.first + i) * words;
        int depth = -1, word = words - 1;
        uint32_t bits = 0;
        for (int at = i; at >= 0; at = up[at]) {
            ++depth;
            for (; word > at >> 5; --word) {
                row[word] = bits;
                bits = 0;
            }
            if (word == at >> 5)
                bits |= 1u << (at & 31);
        }
        for (; word >= 0; --word) {
            row[word] = bits;
            bits = 0;
        }
        if (positions)
            positions[n.first + i] = first_key + depth;
    }
}

// The child that each node's sampled token leads to, by a minimum over the
// children in LDS (the same whatever the order); then the walk.
__global__ void tree_accept_kernel(const TreeArgs t, const int32_t *tokens, const int32_t *parents, const int32_t *sampled,
                                   int max_path, int32_t *path, int32_t *count, int32_t *next_token)
{
    __shared__ int child[kMaxNodes], drawn[kMaxNodes], taken[kMaxNodes];
    __shared__ int steps;
    const int b = blockIdx.x;
    const QueryRows n = nodes_of(t, b);
    for (int i = threadIdx.x; i < n.count; i += blockDim.x) {
        child[i] = kMaxNodes;
        drawn[i] = sampled[n.first + i];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < n.count; i += blockDim.x) {
        const int p = parents[n.first + i];
        if (p >= 0 && p < i && tokens[n.first + i] == drawn[p])
            atomicMin(&child[p], i);
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        int c = 0, last = -1;
        for (int at = 0; at < n.count && c < max_path; at = child[at]) {  // children lie behind their parents
            taken[c++] = at;
            last = drawn[at];
        }
        steps = c;
        count[b] = c;
        next_token[b] = last;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < max_path; i += blockDim.x)
        path[(int64_t)b * max_path + i] = i < steps ? taken[i] : -1;
}

// A wavefront moves the entries of one sequence, layer and kv head.  Entry j
// reads key path[j] >= j and writes key j: what is read has not been written by
// an entry before, so entries may be read ahead of the ones before them, and are,
// kAhead at a time; where they lie is found for 64 at a time, an entry a lane.
// Bound by latency: a token is 8 lines of the cache.  32 layers of 8 heads, 64
// paths through trees of 64 nodes, D = 128: 16.0 us, one at a time 24.5, eight 17.5.
constexpr int kAhead = 4;

template <int D>
__global__ __launch_bounds__(256) void kv4_compact_kernel(const TreeArgs t, const CompactArgs c, int64_t items)
{
    const int64_t item = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (item >= items)
        return;
    const int lane = threadIdx.x & 63;
    const int head = (int)(item % c.hkv);
    const int64_t rest = item / c.hkv;
    const int b = (int)(rest % t.batch), layer = (int)(rest / t.batch);
    const QueryRows n = nodes_of(t, b);
    const int entries = min(max(c.count[b], 0), c.max_path);
    const int keys = c.max_blocks << c.page_shift;
    const int prefix = min(max(t.seq_lens[b], 0), keys) - n.len;
    const int32_t *path = c.path + (int64_t)b * c.max_path, *table = c.block_table + (int64_t)b * c.max_blocks;
    uint8_t *cache = c.cache + layer * c.layer_stride;
    constexpr int kU = D == 64 ? 2 : 4;           // bytes of a token in a V unit
    constexpr int kPieces = D / 2 / kU;           // units of a token
    const int P = 1 << c.page_shift;
    const int64_t head_bytes = (int64_t)P * (D + 8);
    // a lane's bytes of a token: of K, of a V unit, of its parameters
    const int k_at = 4 * lane, v_at = (D / 2 << c.page_shift) + lane * 4 * kU, p_at = (D << c.page_shift) + (lane & 1) * 4 * P;
    for (int base = 0; base < entries; base += 64) {
        const int j = base + lane, node = j < entries ? path[j] : -1;
        int fp = -1, tp = -1;
        const int from = prefix + node, to = prefix + j;
        if (node > j && node < n.len && to >= 0) {  // else out of range, or where it is already
            fp = table[from >> c.page_shift];
            tp = table[to >> c.page_shift];
        }
        const int at = (from & (P - 1)) | (to & (P - 1)) << 16;  // a page has at most 256 tokens
        unsigned long long left = __ballot((uint32_t)fp < (uint32_t)c.num_pages && (uint32_t)tp < (uint32_t)c.num_pages);
        while (left) {
            uint32_t k[kAhead], v[kAhead], par[kAhead];
            uint8_t *dst[kAhead];
            int tt[kAhead];
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                const int e = left ? __builtin_ctzll(left) : -1;  // uniform
                left &= left - 1;
                dst[i] = nullptr;
                if (e < 0)
                    continue;
                const uint8_t *src = cache + ((int64_t)__builtin_amdgcn_readlane(fp, e) * c.hkv + head) * head_bytes;
                dst[i] = cache + ((int64_t)__builtin_amdgcn_readlane(tp, e) * c.hkv + head) * head_bytes;
                const int both = __builtin_amdgcn_readlane(at, e), ft = both & 0xffff;
                tt[i] = both >> 16;
                if (lane < D / 8)
                    k[i] = *(const uint32_t *)(src + ft * (D / 2) + k_at);
                if (lane < kPieces) {
                    const uint8_t *u = src + v_at + (ft >> 2) * (2 * D) + (ft & 3) * kU;
                    v[i] = kU == 2 ? *(const uint16_t *)u : *(const uint32_t *)u;
                }
                if (lane < 2)
                    par[i] = *(const uint32_t *)(src + p_at + 4 * ft);
            }
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                if (!dst[i])
                    break;
                if (lane < D / 8)
                    *(uint32_t *)(dst[i] + tt[i] * (D / 2) + k_at) = k[i];
                if (lane < kPieces) {
                    uint8_t *u = dst[i] + v_at + (tt[i] >> 2) * (2 * D) + (tt[i] & 3) * kU;
                    if constexpr (kU == 2)
                        *(uint16_t *)u = (uint16_t)v[i];
                    else
                        *(uint32_t *)u = v[i];
                }
                if (lane < 2)
                    *(uint32_t *)(dst[i] + p_at + 4 * tt[i]) = par[i];
            }
        }
    }
}

int threads_for(int n) { return n <= 64 ? 64 : n <= 256 ? 256 : 1024; }

}  // namespace

hipError_t launch_tree_mask(const TreeArgs &t, const int32_t *parents, int words, uint32_t *mask, int32_t *positions,
                            hipStream_t s)
{
    const int threads = threads_for(t.max_q_len);
    if (!grid_fits(t.batch, threads))
        return kGridTooLarge;
    tree_mask_kernel<<<dim3((unsigned)t.batch), threads, 0, s>>>(t, parents, words, mask, positions);
    return hipGetLastError();
}

hipError_t launch_tree_accept(const TreeArgs &t, const int32_t *tokens, const int32_t *parents, const int32_t *sampled,
                              int max_path, int32_t *path, int32_t *count, int32_t *next_token, hipStream_t s)
{
    const int threads = threads_for(t.max_q_len);
    if (!grid_fits(t.batch, threads))
        return kGridTooLarge;
    tree_accept_kernel<<<dim3((unsigned)t.batch), threads, 0, s>>>(t, tokens, parents, sampled, max_path, path, count,
                                                                   next_token);
    return hipGetLastError();
}

hipError_t launch_kv4_compact(const TreeArgs &t, const CompactArgs &c, hipStream_t s)
{
    const int64_t items = (int64_t)c.layers * t.batch * c.hkv, groups = (items + 3) / 4;
    if (!grid_fits(groups, 256))
        return kGridTooLarge;
    const dim3 grid((unsigned)groups);
    if (c.D == 64)
        kv4_compact_kernel<64><<<grid, 256, 0, s>>>(t, c, items);
    else if (c.D == 128)
        kv4_compact_kernel<128><<<grid, 256, 0, s>>>(t, c, items);
    else
        kv4_compact_kernel<256><<<grid, 256, 0, s>>>(t, c, items);
    return hipGetLastError();
}

}  // namespace bq
