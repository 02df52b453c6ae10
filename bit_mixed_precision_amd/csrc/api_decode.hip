// C ABI of the decoding operators (declared in include/bq_decode.h): host-side
// validation, then the launchers.  Every check runs before anything is
// enqueued.
#include <hip/hip_runtime.h>

#include "../../include/bq_decode.h"
#include "bq_decode_internal.h"

namespace {

bool aligned(const void *p, unsigned n) { return ((uintptr_t)p & (n - 1)) == 0; }

constexpr int64_t kMaxWords = BQ_TREE_MAX / 32;

int check_nodes(const int32_t *q_start, int64_t batch, int64_t total_q, int64_t max_q_len)
{
    if (batch < 0 || batch > BQ_MAX_DIM || total_q < 0 || total_q > BQ_MAX_DIM || max_q_len < 0 || max_q_len > BQ_TREE_MAX)
        return BQ_ERR_SHAPE;
    if (!q_start && total_q != batch * max_q_len)
        return BQ_ERR_SHAPE;
    return aligned(q_start, 4) ? BQ_OK : BQ_ERR_ALIGN;
}

bq::TreeArgs nodes(const int32_t *q_start, const int32_t *seq_lens, int64_t batch, int64_t total_q, int64_t max_q_len)
{
    bq::TreeArgs t = {};
    t.q_start = q_start;
    t.seq_lens = seq_lens;
    t.batch = (int)batch;
    t.total_q = (int)total_q;
    t.max_q_len = (int)max_q_len;
    return t;
}

}  // namespace

extern "C" {

int bq_tree_mask(const int32_t *parents, const int32_t *q_start, const int32_t *seq_lens, int64_t batch, int64_t total_q,
                 int64_t max_q_len, int64_t mask_words, uint32_t *mask, int32_t *positions, void *stream)
{
    int st = check_nodes(q_start, batch, total_q, max_q_len);
    if (st != BQ_OK)
        return st;
    if (mask_words < 1 || mask_words > kMaxWords)
        return BQ_ERR_SHAPE;
    if (batch == 0 || total_q == 0 || max_q_len == 0)
        return BQ_OK;
    if (!parents || !mask)
        return BQ_ERR_NULL;
    if (!aligned(parents, 4) || !aligned(mask, 4) || !aligned(positions, 4) || !aligned(seq_lens, 4))
        return BQ_ERR_ALIGN;
    if ((st = bq::device_status()) != BQ_OK)
        return st;
    return bq::launch_status(bq::launch_tree_mask(nodes(q_start, seq_lens, batch, total_q, max_q_len), parents,
                                                  (int)mask_words, mask, positions, (hipStream_t)stream));
}

int bq_tree_accept(const int32_t *tokens, const int32_t *parents, const int32_t *sampled, const int32_t *q_start,
                   int64_t batch, int64_t total_q, int64_t max_q_len, int64_t max_path, int32_t *path, int32_t *count,
                   int32_t *next_token, void *stream)
{
    int st = check_nodes(q_start, batch, total_q, max_q_len);
    if (st != BQ_OK)
        return st;
    if (max_path < 1 || max_path > BQ_TREE_MAX)
        return BQ_ERR_SHAPE;
    if (batch == 0)
        return BQ_OK;
    if (!path || !count || !next_token || (total_q > 0 && (!tokens || !parents || !sampled)))
        return BQ_ERR_NULL;
    if (!aligned(tokens, 4) || !aligned(parents, 4) || !aligned(sampled, 4) || !aligned(path, 4) || !aligned(count, 4) ||
        !aligned(next_token, 4))
        return BQ_ERR_ALIGN;
    if ((st = bq::device_status()) != BQ_OK)
        return st;
    return bq::launch_status(bq::launch_tree_accept(nodes(q_start, nullptr, batch, total_q, max_q_len), tokens, parents,
                                                    sampled, (int)max_path, path, count, next_token, (hipStream_t)stream));
}

int bq_kv4_compact(void *cache, int64_t num_layers, int64_t layer_stride, int64_t num_pages, int page_size, int kv_heads,
                   int head_dim, const int32_t *block_table, int64_t max_blocks, const int32_t *q_start,
                   const int32_t *seq_lens, int64_t batch, int64_t total_q, int64_t max_q_len, const int32_t *path,
                   const int32_t *count, int64_t max_path, void *stream)
{
    const int64_t page_bytes = bq_kv4_page_bytes(kv_heads, head_dim, page_size);
    if (page_bytes < 0 || num_pages < 0 || num_pages > BQ_MAX_DIM || num_layers < 0 || num_layers > 65536 || max_blocks < 0 ||
        max_blocks > BQ_MAX_DIM || max_blocks * page_size > BQ_MAX_DIM || max_path < 1 || max_path > BQ_TREE_MAX)
        return BQ_ERR_SHAPE;
    int st = check_nodes(q_start, batch, total_q, max_q_len);
    if (st != BQ_OK)
        return st;
    if (num_layers > 1 && (layer_stride < num_pages * page_bytes || layer_stride > BQ_MAX_OUT))
        return BQ_ERR_SHAPE;
    if (batch == 0 || num_layers == 0 || total_q == 0 || num_pages == 0 || max_blocks == 0)
        return BQ_OK;
    if (!cache || !block_table || !seq_lens || !path || !count)
        return BQ_ERR_NULL;
    if (!aligned(cache, 16) || (num_layers > 1 && layer_stride % 16 != 0) || !aligned(block_table, 4) || !aligned(seq_lens, 4) ||
        !aligned(path, 4) || !aligned(count, 4))
        return BQ_ERR_ALIGN;
    if ((st = bq::device_status()) != BQ_OK)
        return st;
    bq::CompactArgs c = {};
    c.cache = (uint8_t *)cache;
    c.layer_stride = num_layers > 1 ? layer_stride : 0;
    c.layers = (int)num_layers;
    c.num_pages = (int)num_pages;
    c.page_shift = __builtin_ctz((unsigned)page_size);
    c.hkv = kv_heads;
    c.D = head_dim;
    c.block_table = block_table;
    c.max_blocks = (int)max_blocks;
    c.path = path;
    c.count = count;
    c.max_path = (int)max_path;
    return bq::launch_status(bq::launch_kv4_compact(nodes(q_start, seq_lens, batch, total_q, max_q_len), c, (hipStream_t)stream));
}

static int sample_shape(int64_t rows, int64_t vocab, int dtype)
{
    if (dtype != BQ_F16 && dtype != BQ_BF16 && dtype != BQ_F32)
        return BQ_ERR_ARG;
    return rows < 0 || rows > BQ_MAX_DIM || vocab < 1 || vocab > (1 << 24) ? BQ_ERR_SHAPE : BQ_OK;
}

int64_t bq_sample_workspace_bytes(int64_t rows, int64_t vocab, int dtype)
{
    const int st = sample_shape(rows, vocab, dtype);
    return st != BQ_OK ? -st : bq::sample_workspace_bytes(rows, vocab, dtype);
}

int bq_sample(const void *logits, int64_t row_stride, int dtype, int64_t rows, int64_t vocab, const float *u,
              const float *temperature, const int32_t *top_k, const float *top_p, const float *min_p, int32_t *tokens,
              float *logprobs, void *workspace, int64_t workspace_bytes, void *stream)
{
    int st = sample_shape(rows, vocab, dtype);
    if (st != BQ_OK)
        return st;
    if (row_stride < vocab || row_stride > BQ_MAX_OUT || workspace_bytes < 0)
        return BQ_ERR_SHAPE;
    if (workspace_bytes > 0 && !workspace)
        return BQ_ERR_NULL;
    if (rows == 0)
        return BQ_OK;
    if (!logits || !u || !tokens)
        return BQ_ERR_NULL;
    if (!aligned(logits, dtype == BQ_F32 ? 4 : 2) || !aligned(u, 4) || !aligned(temperature, 4) || !aligned(top_k, 4) ||
        !aligned(top_p, 4) || !aligned(min_p, 4) || !aligned(tokens, 4) || !aligned(logprobs, 4) || !aligned(workspace, 16))
        return BQ_ERR_ALIGN;
    if ((st = bq::device_status()) != BQ_OK)
        return st;
    bq::SampleArgs a = {};
    a.logits = logits;
    a.row_stride = row_stride;
    a.rows = (int)rows;
    a.vocab = (int)vocab;
    a.frac = 61;  // sums of vocab weights stay within 2^61; 48 octaves below the greatest nothing is a unit
    while (a.frac > 46 || 1ll << (61 - a.frac) < vocab)
        --a.frac;
    a.u = u;
    a.temperature = temperature;
    a.top_k = top_k;
    a.top_p = top_p;
    a.min_p = min_p;
    a.tokens = tokens;
    a.logprobs = logprobs;
    return bq::launch_status(bq::launch_sample(a, dtype, workspace, workspace ? workspace_bytes : 0, (hipStream_t)stream));
}

}  // extern "C"
