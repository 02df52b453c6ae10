// Internal declarations of the decoder-layer operators (include/bq_layer.h):
// what api_layer.hip and the operators' kernels share.  They stand apart from
// bq_internal.h, which the tiled GEMM's committed traffic summary covers.
#pragma once

#include "bq_internal.h"

namespace bq {

// Checks that the current device is gfx950 (a bq_status), once per device.
int device_status();
// The bq_status of a launcher's result.
int launch_status(hipError_t e);

// Query/key norm and rotation (decoder-layer operators, include/bq_layer.h).
// cache == nullptr: keys go to k_out, else keys and values to the cache.
struct QkRopeArgs {
    const uint16_t *q, *k, *v;
    int64_t q_stride, k_stride, v_stride;  // elements between tokens
    const uint16_t *q_weight, *k_weight;
    double eps;
    const float *cos, *sin;
    const int32_t *positions;
    int64_t max_pos;
    int rot, inter;
    int64_t tokens;
    int hq, hkv, D;
    uint16_t *q_out, *k_out;
    uint8_t *cache;
    int64_t num_pages;
    int page_shift;
    const int64_t *slots;
};
hipError_t launch_qk_norm_rope(const QkRopeArgs &p, bool bf16, hipStream_t s);
hipError_t launch_kv4_read(const uint8_t *cache, int64_t num_pages, int page_shift, int hkv, int D, const int64_t *slots,
                           int64_t tokens, uint16_t *k, uint16_t *v, bool bf16, hipStream_t s);

// Attention over the 4-bit paged cache.
struct AttnKv4Args {
    const void *q;
    int64_t q_stride;
    const int32_t *q_start, *seq_lens, *block_table;
    int batch, total_q, max_q_len;
    int hq, hkv, group;
    const uint8_t *cache;
    int num_pages;
    int page_shift, max_blocks;
    float scale;
    int window;
    void *out;
    float *lse;
    int row_tiles, nsplit, join_rows;
    float *part, *part_ml;
};
// How a call is split: rt tiles of 16 query rows a workgroup, row_tiles
// workgroups per sequence and kv head, times nsplit parts of the keys, whose
// results take part_rows rows (of head_dim + 2 floats) of workspace.
struct AttnKv4Plan {
    int rt, nsplit;
    int64_t row_tiles, part_rows;
};
AttnKv4Plan attn_kv4_plan(int64_t batch, int64_t max_q_len, int q_heads, int kv_heads, int D, int64_t max_len);
hipError_t launch_attn_kv4(AttnKv4Args &p, int D, int rt, bool bf16, hipStream_t s);

// 4-bit weights with group scales times 16-bit activations.  A call whose
// outputs are few splits K over workgroups through `ws` when it is given.
int64_t gemm_w4g_workspace_bytes(int M, int N, int K);
hipError_t launch_gemm_w4g(const uint16_t *A, const uint8_t *B, const uint16_t *scale, const uint16_t *zero, int group,
                           uint16_t *C, int M, int N, int K, bool bf16, float *ws, int64_t wsBytes, hipStream_t s);

}  // namespace bq
