// Internal declarations of the decoding operators (include/bq_decode.h): what
// api_decode.hip and the operators' kernels share.
#pragma once

#include "bq_layer_internal.h"

namespace bq {

// The nodes of the sequences (q_start, or max_q_len each).
struct TreeArgs {
    const int32_t *q_start, *seq_lens;
    int batch, total_q, max_q_len;
};

hipError_t launch_tree_mask(const TreeArgs &t, const int32_t *parents, int words, uint32_t *mask, int32_t *positions,
                            hipStream_t s);
hipError_t launch_tree_accept(const TreeArgs &t, const int32_t *tokens, const int32_t *parents, const int32_t *sampled,
                              int max_path, int32_t *path, int32_t *count, int32_t *next_token, hipStream_t s);

struct CompactArgs {
    uint8_t *cache;
    int64_t layer_stride;
    int layers, num_pages, page_shift, hkv, D;
    const int32_t *block_table;
    int max_blocks;
    const int32_t *path, *count;
    int max_path;
};
hipError_t launch_kv4_compact(const TreeArgs &t, const CompactArgs &c, hipStream_t s);

// Sampling: logits of type 0 fp16, 1 bf16, 2 fp32.
struct SampleArgs {
    const void *logits;
    int64_t row_stride;
    int rows, vocab;
    int frac;  // fractional bits of the weights
    const float *u, *temperature;
    const int32_t *top_k;
    const float *top_p, *min_p;
    int32_t *tokens;
    float *logprobs;
};
int64_t sample_workspace_bytes(int64_t rows, int64_t vocab, int type);
hipError_t launch_sample(const SampleArgs &p, int type, void *workspace, int64_t workspace_bytes, hipStream_t s);

}  // namespace bq
