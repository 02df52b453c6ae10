// C ABI of the decoder-layer operators (declared in include/bq_layer.h):
// host-side validation, then the launchers.  Every check runs before
// anything is enqueued.
#include <hip/hip_runtime.h>

#include "../../include/bq_layer.h"
#include "bq_layer_internal.h"

namespace {

bool aligned(const void *p, unsigned n) { return ((uintptr_t)p & (n - 1)) == 0; }

bool head_dim_ok(int d) { return d == 64 || d == 128 || d == 256; }
bool page_size_ok(int n) { return n == 16 || n == 32 || n == 64 || n == 128 || n == 256; }
int shift_of(int page_size)
{
    int s = 0;
    while ((1 << s) < page_size && s < 8)
        ++s;
    return s;
}
constexpr int kMaxHeads = 65536;

// A token-strided tensor: at least a token between tokens, whole 16-byte
// pieces, and an extent that 64-bit offsets hold.
int check_rows(const void *p, int64_t stride, int64_t token)
{
    if (!p)
        return BQ_ERR_NULL;
    if (stride < token || stride > BQ_MAX_OUT)
        return BQ_ERR_SHAPE;
    return aligned(p, 16) && stride % 8 == 0 ? BQ_OK : BQ_ERR_ALIGN;
}

int check_rope(const bq::QkRopeArgs &a, int dtype, bool cache, int page_size)
{
    if (dtype != BQ_F16 && dtype != BQ_BF16)
        return BQ_ERR_ARG;
    if (a.tokens < 0 || a.tokens > BQ_MAX_DIM || a.hq < 0 || a.hkv < 0 || a.hq > kMaxHeads || a.hkv > kMaxHeads ||
        !head_dim_ok(a.D))
        return BQ_ERR_SHAPE;
    if (a.rot < 0 || a.rot > a.D || a.rot % 16 != 0 || a.max_pos < 0 || a.max_pos > BQ_MAX_DIM)
        return BQ_ERR_SHAPE;
    if (!(a.eps >= 0.0))
        return BQ_ERR_ARG;
    if (cache && (!page_size_ok(page_size) || a.num_pages < 0 || a.num_pages > BQ_MAX_DIM))
        return BQ_ERR_SHAPE;
    if (a.tokens == 0 || a.hq + a.hkv == 0)
        return BQ_OK;
    int st;
    if (a.hq > 0) {
        if ((st = check_rows(a.q, a.q_stride, (int64_t)a.hq * a.D)) != BQ_OK)
            return st;
        if (!a.q_out)
            return BQ_ERR_NULL;
        if (!aligned(a.q_out, 16))
            return BQ_ERR_ALIGN;
    }
    if (a.hkv > 0) {
        if ((st = check_rows(a.k, a.k_stride, (int64_t)a.hkv * a.D)) != BQ_OK)
            return st;
        if (cache) {
            if ((st = check_rows(a.v, a.v_stride, (int64_t)a.hkv * a.D)) != BQ_OK)
                return st;
            if (!a.slots || !a.cache)
                return BQ_ERR_NULL;
            if (!aligned(a.slots, 8) || !aligned(a.cache, 16))
                return BQ_ERR_ALIGN;
        } else {
            if (!a.k_out)
                return BQ_ERR_NULL;
            if (!aligned(a.k_out, 16))
                return BQ_ERR_ALIGN;
        }
    }
    if ((a.q_weight != nullptr) != (a.k_weight != nullptr) && a.hq > 0 && a.hkv > 0)
        return BQ_ERR_NULL;
    if (!aligned(a.q_weight, 16) || !aligned(a.k_weight, 16))
        return BQ_ERR_ALIGN;
    if (a.rot > 0) {
        if (!a.positions || (a.max_pos > 0 && (!a.cos || !a.sin)))
            return BQ_ERR_NULL;
        if (!aligned(a.positions, 4) || !aligned(a.cos, 16) || !aligned(a.sin, 16))
            return BQ_ERR_ALIGN;
    }
    return bq::device_status();
}

}  // namespace

extern "C" {

int64_t bq_gemm_w4g_workspace_bytes(int64_t M, int64_t N, int64_t K)
{
    if (M < 0 || N < 0 || K < 0 || K > BQ_MAX_K || K % 64 != 0 || M > BQ_MAX_DIM || N > BQ_MAX_DIM || M * N > BQ_MAX_OUT)
        return -BQ_ERR_SHAPE;
    return M == 0 || N == 0 ? 0 : bq::gemm_w4g_workspace_bytes((int)M, (int)N, (int)K);
}

int bq_gemm_w4g_a16(const void *A, int dtype, const uint8_t *B, const void *scale_f16, const void *zero_f16, int group,
                    void *C, int64_t M, int64_t N, int64_t K, void *workspace, int64_t workspace_bytes, void *stream)
{
    if ((dtype != BQ_F16 && dtype != BQ_BF16) || (group != 32 && group != 64 && group != 128))
        return BQ_ERR_ARG;
    if (M < 0 || N < 0 || K < 0 || K > BQ_MAX_K || K % 64 != 0 || K % group != 0 || M > BQ_MAX_DIM || N > BQ_MAX_DIM ||
        M * N > BQ_MAX_OUT || workspace_bytes < 0)
        return BQ_ERR_SHAPE;
    if (workspace_bytes > 0 && !workspace)
        return BQ_ERR_NULL;
    if (M == 0 || N == 0)
        return BQ_OK;
    if (!C || (K > 0 && (!A || !B || !scale_f16)))
        return BQ_ERR_NULL;
    if (!aligned(C, 16) || !aligned(workspace, 16) ||
        (K > 0 && (!aligned(A, 16) || !aligned(B, 16) || !aligned(scale_f16, 16) || !aligned(zero_f16, 16))))
        return BQ_ERR_ALIGN;
    const int st = bq::device_status();
    if (st != BQ_OK)
        return st;
    return bq::launch_status(bq::launch_gemm_w4g((const uint16_t *)A, B, (const uint16_t *)scale_f16,
                                                 (const uint16_t *)zero_f16, group, (uint16_t *)C, (int)M, (int)N, (int)K,
                                                 dtype == BQ_BF16, (float *)workspace, workspace ? workspace_bytes : 0,
                                                 (hipStream_t)stream));
}

int bq_qk_norm_rope(const void *q, int64_t q_stride, const void *k, int64_t k_stride, int dtype, int64_t tokens, int q_heads,
                    int kv_heads, int head_dim, const void *q_weight, const void *k_weight, double eps, const float *cos,
                    const float *sin, int64_t max_pos, int rot_dim, int interleaved, const int32_t *positions, void *q_out,
                    void *k_out, void *stream)
{
    bq::QkRopeArgs a = {};
    a.q = (const uint16_t *)q;
    a.k = (const uint16_t *)k;
    a.q_stride = q_stride;
    a.k_stride = k_stride;
    a.q_weight = (const uint16_t *)q_weight;
    a.k_weight = (const uint16_t *)k_weight;
    a.eps = eps;
    a.cos = cos;
    a.sin = sin;
    a.positions = positions;
    a.max_pos = max_pos;
    a.rot = rot_dim;
    a.inter = interleaved != 0;
    a.tokens = tokens;
    a.hq = q_heads;
    a.hkv = kv_heads;
    a.D = head_dim;
    a.q_out = (uint16_t *)q_out;
    a.k_out = (uint16_t *)k_out;
    const int st = check_rope(a, dtype, false, 0);
    if (st != BQ_OK || tokens == 0 || q_heads + kv_heads == 0)
        return st;
    return bq::launch_status(bq::launch_qk_norm_rope(a, dtype == BQ_BF16, (hipStream_t)stream));
}

int64_t bq_kv4_page_bytes(int kv_heads, int head_dim, int page_size)
{
    if (kv_heads < 1 || kv_heads > kMaxHeads || !head_dim_ok(head_dim) || !page_size_ok(page_size))
        return -BQ_ERR_SHAPE;
    return (int64_t)kv_heads * page_size * (head_dim + 8);
}

int bq_qk_norm_rope_kv4(const void *q, int64_t q_stride, const void *k, int64_t k_stride, const void *v, int64_t v_stride,
                        int dtype, int64_t tokens, int q_heads, int kv_heads, int head_dim, const void *q_weight,
                        const void *k_weight, double eps, const float *cos, const float *sin, int64_t max_pos, int rot_dim,
                        int interleaved, const int32_t *positions, void *q_out, void *cache, int64_t num_pages,
                        int page_size, const int64_t *slots, void *stream)
{
    bq::QkRopeArgs a = {};
    a.q = (const uint16_t *)q;
    a.k = (const uint16_t *)k;
    a.v = (const uint16_t *)v;
    a.q_stride = q_stride;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.q_weight = (const uint16_t *)q_weight;
    a.k_weight = (const uint16_t *)k_weight;
    a.eps = eps;
    a.cos = cos;
    a.sin = sin;
    a.positions = positions;
    a.max_pos = max_pos;
    a.rot = rot_dim;
    a.inter = interleaved != 0;
    a.tokens = tokens;
    a.hq = q_heads;
    a.hkv = kv_heads;
    a.D = head_dim;
    a.q_out = (uint16_t *)q_out;
    a.cache = (uint8_t *)cache;
    a.num_pages = num_pages;
    a.page_shift = shift_of(page_size);
    a.slots = slots;
    if (kv_heads < 1)
        return BQ_ERR_SHAPE;
    const int st = check_rope(a, dtype, true, page_size);
    if (st != BQ_OK || tokens == 0)
        return st;
    return bq::launch_status(bq::launch_qk_norm_rope(a, dtype == BQ_BF16, (hipStream_t)stream));
}

int bq_kv4_read(const void *cache, int64_t num_pages, int page_size, int kv_heads, int head_dim, const int64_t *slots,
                int64_t tokens, int dtype, void *k_out, void *v_out, void *stream)
{
    if (dtype != BQ_F16 && dtype != BQ_BF16)
        return BQ_ERR_ARG;
    if (bq_kv4_page_bytes(kv_heads, head_dim, page_size) < 0 || num_pages < 0 || num_pages > BQ_MAX_DIM || tokens < 0 ||
        tokens > BQ_MAX_DIM)
        return BQ_ERR_SHAPE;
    if (tokens == 0)
        return BQ_OK;
    if (!cache || !slots || !k_out || !v_out)
        return BQ_ERR_NULL;
    if (!aligned(cache, 16) || !aligned(slots, 8) || !aligned(k_out, 16) || !aligned(v_out, 16))
        return BQ_ERR_ALIGN;
    const int st = bq::device_status();
    if (st != BQ_OK)
        return st;
    return bq::launch_status(bq::launch_kv4_read((const uint8_t *)cache, num_pages, shift_of(page_size), kv_heads, head_dim,
                                                 slots, tokens, (uint16_t *)k_out, (uint16_t *)v_out, dtype == BQ_BF16,
                                                 (hipStream_t)stream));
}

// Shapes of bq_attn_kv4 that its workspace depends on.
static int attn_shape(int64_t batch, int64_t max_q_len, int q_heads, int kv_heads, int head_dim, int64_t max_len)
{
    if (batch < 0 || batch > BQ_MAX_DIM || max_q_len < 0 || max_q_len > BQ_MAX_DIM || q_heads < 1 || kv_heads < 1 ||
        q_heads > kMaxHeads || q_heads % kv_heads != 0 || !head_dim_ok(head_dim) || max_len < 0 || max_len > BQ_MAX_DIM ||
        max_q_len * (q_heads / kv_heads) > BQ_MAX_DIM)
        return BQ_ERR_SHAPE;
    const int64_t tiles = (max_q_len * (q_heads / kv_heads) + 15) / 16;
    return batch * kv_heads <= BQ_MAX_OUT && (tiles == 0 || batch * kv_heads <= BQ_MAX_OUT / tiles) ? BQ_OK : BQ_ERR_SHAPE;
}

int64_t bq_attn_kv4_workspace_bytes(int64_t batch, int64_t max_q_len, int q_heads, int kv_heads, int head_dim,
                                    int64_t max_len)
{
    if (attn_shape(batch, max_q_len, q_heads, kv_heads, head_dim, max_len) != BQ_OK)
        return -BQ_ERR_SHAPE;
    return bq::attn_kv4_plan(batch, max_q_len, q_heads, kv_heads, head_dim, max_len).part_rows * (head_dim + 2) * 4;
}

int bq_attn_kv4(const void *q, int64_t q_stride, int dtype, const int32_t *q_start, const int32_t *seq_lens,
                const int32_t *block_table, int64_t batch, int64_t total_q, int64_t max_q_len, int q_heads, int kv_heads,
                int head_dim, const void *cache, int64_t num_pages, int page_size, int64_t max_blocks, float softmax_scale,
                int64_t window, void *out, float *lse, void *workspace, int64_t workspace_bytes, void *stream)
{
    if ((dtype != BQ_F16 && dtype != BQ_BF16) || !__builtin_isfinite(softmax_scale))
        return BQ_ERR_ARG;
    if (!page_size_ok(page_size) || max_blocks < 0 || max_blocks > BQ_MAX_DIM || num_pages < 0 || num_pages > BQ_MAX_DIM ||
        total_q < 0 || total_q > BQ_MAX_DIM || window < 0 || window > BQ_MAX_DIM || workspace_bytes < 0)
        return BQ_ERR_SHAPE;
    const int64_t max_len = max_blocks * page_size;
    const int st = attn_shape(batch, max_q_len, q_heads, kv_heads, head_dim, max_len);
    if (st != BQ_OK)
        return st;
    if (!q_start && total_q != batch * max_q_len)
        return BQ_ERR_SHAPE;
    if (workspace_bytes > 0 && !workspace)
        return BQ_ERR_NULL;
    if (batch == 0 || total_q == 0 || max_q_len == 0)
        return BQ_OK;
    const int rows = check_rows(q, q_stride, (int64_t)q_heads * head_dim);
    if (rows != BQ_OK)
        return rows;
    if (!seq_lens || !out || (max_len > 0 && (!block_table || !cache)))
        return BQ_ERR_NULL;
    if (max_len > 0 && num_pages == 0)
        return BQ_ERR_SHAPE;
    if (!aligned(out, 16) || !aligned(cache, 16) || !aligned(workspace, 16) || !aligned(q_start, 4) ||
        !aligned(seq_lens, 4) || !aligned(block_table, 4) || !aligned(lse, 4))
        return BQ_ERR_ALIGN;
    const int dev = bq::device_status();
    if (dev != BQ_OK)
        return dev;
    bq::AttnKv4Args a = {};
    a.q = q;
    a.q_stride = q_stride;
    a.q_start = q_start;
    a.seq_lens = seq_lens;
    a.block_table = block_table;
    a.batch = (int)batch;
    a.total_q = (int)total_q;
    a.max_q_len = (int)max_q_len;
    a.hq = q_heads;
    a.hkv = kv_heads;
    a.group = q_heads / kv_heads;
    a.cache = (const uint8_t *)cache;
    a.num_pages = (int)num_pages;
    a.page_shift = shift_of(page_size);
    a.max_blocks = (int)max_blocks;
    a.scale = softmax_scale;
    a.window = (int)window;
    a.out = out;
    a.lse = lse;
    const bq::AttnKv4Plan plan = bq::attn_kv4_plan(batch, max_q_len, q_heads, kv_heads, head_dim, max_len);
    a.row_tiles = (int)plan.row_tiles;
    a.nsplit = plan.part_rows > 0 && workspace && workspace_bytes >= plan.part_rows * (head_dim + 2) * 4 ? plan.nsplit : 1;
    a.part = (float *)workspace;
    a.part_ml = a.part + plan.part_rows * head_dim;
    return bq::launch_status(bq::launch_attn_kv4(a, head_dim, plan.rt, dtype == BQ_BF16, (hipStream_t)stream));
}

}  // extern "C"
