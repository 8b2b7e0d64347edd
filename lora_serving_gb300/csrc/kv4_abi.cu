// kv4_abi.cu -- C ABI entry points of the norm, the 4-bit cache's operators
// and drafted decoding's: host-side validation before anything is enqueued.
#include <cmath>
#include <cstdint>
#include <initializer_list>

#include "kv4.h"

namespace {

using lora::bf16_t;

constexpr int kMaxWidth = 65536;     // columns of a norm, of a fused row
constexpr int kMaxGroupHeads = 64;   // q heads to a kv head

inline bool aligned(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

lora_status_t cuda_status(cudaError_t e) { return e == cudaSuccess ? LORA_OK : LORA_ERR_CUDA; }

#define LORA_TRY(expr)                          \
    do {                                        \
        const lora_status_t _st = (expr);       \
        if (_st != LORA_OK) return _st;         \
    } while (0)

// A bf16 matrix argument of `cols` columns.
lora_status_t check_matrix(const void* p, int ld, long long cols)
{
    if (!p) return LORA_ERR_INVALID_ARG;
    if (ld < cols) return LORA_ERR_SHAPE;
    if (!aligned(p, 16) || ld % 8 != 0) return LORA_ERR_ALIGNMENT;
    return LORA_OK;
}

bool page_size_ok(int n) { return n == 16 || n == 32 || n == 64 || n == 128 || n == 256; }
bool head_dim_ok(int d) { return d == 64 || d == 128; }

lora_status_t check_cache(const lora_kv4_cache_t* c, lora::kv4::Cache& out)
{
    if (!c || !c->pages || c->n_pages <= 0 || c->n_kv <= 0) return LORA_ERR_INVALID_ARG;
    if (!page_size_ok(c->page_size) || !head_dim_ok(c->head_dim) || c->n_kv > 1024) return LORA_ERR_SHAPE;
    if (c->page_stride < static_cast<int64_t>(c->n_kv) * lora::kv4::block_bytes(c->page_size, c->head_dim))
        return LORA_ERR_SHAPE;
    if (!aligned(c->pages, 16) || c->page_stride % 16 != 0) return LORA_ERR_ALIGNMENT;
    out.pages = c->pages;
    out.page_stride = c->page_stride;
    out.n_pages = c->n_pages;
    out.page_size = c->page_size;
    out.page_shift = 0;
    while ((1 << out.page_shift) < c->page_size) ++out.page_shift;
    out.n_kv = c->n_kv;
    out.head_dim = c->head_dim;
    return LORA_OK;
}

lora_status_t check_batch(const lora_kv4_batch_t* b, const lora::kv4::Cache& c, lora::kv4::Batch& out)
{
    if (!b || b->n_seqs < 0 || b->n_rows < 0 || b->max_q_len < 0 || b->max_ctx_len < 0) return LORA_ERR_INVALID_ARG;
    if (b->n_rows > 0) {
        if (b->n_seqs == 0) return LORA_ERR_METADATA;
        if (!b->q_starts || !b->ctx_lens || !b->block_table) return LORA_ERR_INVALID_ARG;
        if (b->ld_table < (static_cast<long long>(b->max_ctx_len) + c.page_size - 1) / c.page_size) return LORA_ERR_SHAPE;
        if (!aligned(b->q_starts, 4) || !aligned(b->ctx_lens, 4) || !aligned(b->block_table, 4)) return LORA_ERR_ALIGNMENT;
    }
    out.q_starts = b->q_starts;
    out.ctx_lens = b->ctx_lens;
    out.block_table = b->block_table;
    out.ld_table = b->ld_table;
    out.n_seqs = b->n_seqs;
    out.n_rows = b->n_rows;
    out.max_q_len = b->max_q_len;
    out.max_ctx_len = b->max_ctx_len;
    return LORA_OK;
}

bool overlap(long long a0, long long an, long long b0, long long bn) { return a0 < b0 + bn && b0 < a0 + an; }

// The checks of an attention call and its launch; `a` holds what only a tree's call sets.
lora_status_t attend(lora::AttendArgs& a, lora_bf16_t* out, int ld_out, const lora_bf16_t* q, int ld_q, int n_heads, float scale,
                     int window, const lora_kv4_cache_t* cache, const lora_kv4_batch_t* batch, void* workspace, size_t ws_bytes,
                     int32_t* dev_status, lora_stream_t stream)
{
    LORA_TRY(check_cache(cache, a.cache));
    LORA_TRY(check_batch(batch, a.cache, a.batch));
    if (n_heads <= 0 || window < 0 || !std::isfinite(scale)) return LORA_ERR_INVALID_ARG;
    const int n_kv = a.cache.n_kv, D = a.cache.head_dim;
    if (n_heads % n_kv != 0 || n_heads / n_kv > kMaxGroupHeads) return LORA_ERR_SHAPE;
    if (batch->n_rows == 0) return LORA_OK;
    a.n_heads = n_heads; a.group = n_heads / n_kv;
    if (batch->max_ctx_len > lora::kMaxPositions || static_cast<long long>(batch->n_rows) * a.group > lora::kMaxPositions) return LORA_ERR_SHAPE;
    a.window = window < batch->max_ctx_len ? window : 0;   // one as wide as the longest context hides nothing
    a.group_magic = a.group > 1 ? static_cast<uint32_t>((1ULL << 32) / a.group + 1) : 0;
    if (batch->n_seqs > lora::kMaxSeqs || lora::kv4_attend_places(a) > 0x7FFFFFFFLL) return LORA_ERR_SHAPE;
    LORA_TRY(check_matrix(q, ld_q, static_cast<long long>(n_heads) * D));
    LORA_TRY(check_matrix(out, ld_out, static_cast<long long>(n_heads) * D));
    if (!workspace || ws_bytes < lora_kv4_attend_workspace_bytes(n_heads, n_kv, D, batch->max_q_len)) return LORA_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return LORA_ERR_ALIGNMENT;
    a.out = out; a.ld_out = ld_out; a.q = q; a.ld_q = ld_q; a.scale = scale;
    a.ws = workspace; a.ws_bytes = ws_bytes; a.status = dev_status;
    return cuda_status(lora::launch_kv4_attend(a, reinterpret_cast<cudaStream_t>(stream)));
}

}  // namespace

extern "C" {

lora_status_t lora_rms_norm(lora_bf16_t* y, int ld_y, uint8_t* y8, int ld_y8, float* scales, int ld_scales,
                            int group, lora_bf16_t* residual_out, int ld_res_out, const lora_bf16_t* x, int ld_x,
                            const lora_bf16_t* residual, int ld_res, const lora_bf16_t* weight, int n_rows,
                            int width, float eps, lora_stream_t stream)
{
    if (n_rows < 0 || width <= 0 || !(eps >= 0.f) || std::isinf(eps)) return LORA_ERR_INVALID_ARG;
    if (n_rows == 0) return LORA_OK;
    if ((!y && !y8) || (y8 && !scales) || (residual == nullptr) != (residual_out == nullptr) || !weight)
        return LORA_ERR_INVALID_ARG;
    if (width > kMaxWidth || (group != 0 && group != 128)) return LORA_ERR_SHAPE;
    if (width % 8 != 0 || !aligned(weight, 16)) return LORA_ERR_ALIGNMENT;
    LORA_TRY(check_matrix(x, ld_x, width));
    if (y) LORA_TRY(check_matrix(y, ld_y, width));
    if (residual) {
        LORA_TRY(check_matrix(residual, ld_res, width));
        LORA_TRY(check_matrix(residual_out, ld_res_out, width));
    }
    if (y8) {
        if (ld_y8 < width || ld_scales < (group ? (width + group - 1) / group : 1)) return LORA_ERR_SHAPE;
        if (!aligned(y8, 8) || ld_y8 % 8 != 0 || !aligned(scales, 4)) return LORA_ERR_ALIGNMENT;
    }
    lora::NormArgs a{y, ld_y, y8, ld_y8, scales, ld_scales, group, residual_out, ld_res_out, x, ld_x, residual, ld_res,
                     weight, n_rows, width, eps};
    return cuda_status(lora::launch_rms_norm(a, reinterpret_cast<cudaStream_t>(stream)));
}

size_t lora_kv4_block_bytes(int page_size, int head_dim)
{
    if (!page_size_ok(page_size) || !head_dim_ok(head_dim)) return 0;
    return static_cast<size_t>(lora::kv4::block_bytes(page_size, head_dim));
}

lora_status_t lora_kv4_append(lora_bf16_t* q_out, int ld_q, const lora_bf16_t* x, int ld_x, int n_heads, int q_off,
                              int k_off, int v_off, const float* rope, int rot_dim, int max_pos,
                              const int32_t* positions, int ld_pos, const int* axis_pairs, int n_axes,
                              const lora_kv4_cache_t* cache, const lora_kv4_batch_t* batch, int32_t* dev_status,
                              lora_stream_t stream)
{
    lora::AppendArgs a{};
    LORA_TRY(check_cache(cache, a.cache));
    LORA_TRY(check_batch(batch, a.cache, a.batch));
    const int D = a.cache.head_dim;
    if (n_heads <= 0 || q_off < 0 || k_off < 0 || v_off < 0 || rot_dim < 0) return LORA_ERR_INVALID_ARG;
    if (n_heads > kMaxWidth / D) return LORA_ERR_SHAPE;
    const long long nq = static_cast<long long>(n_heads) * D, nk = static_cast<long long>(a.cache.n_kv) * D;
    if (q_off + nq > ld_x || k_off + nk > ld_x || v_off + nk > ld_x) return LORA_ERR_SHAPE;
    if (overlap(q_off, nq, k_off, nk) || overlap(q_off, nq, v_off, nk) || overlap(k_off, nk, v_off, nk)) return LORA_ERR_SHAPE;
    if (q_off % 8 != 0 || k_off % 8 != 0 || v_off % 8 != 0) return LORA_ERR_ALIGNMENT;
    if (rot_dim > 0) {
        if (!rope || max_pos <= 0 || !axis_pairs || n_axes < 1 || n_axes > LORA_MAX_ROPE_AXES) return LORA_ERR_INVALID_ARG;
        if (rot_dim > D) return LORA_ERR_SHAPE;
        if (rot_dim % 16 != 0 || !aligned(rope, 16)) return LORA_ERR_ALIGNMENT;
        long long sum = 0;
        for (int i = 0; i < LORA_MAX_ROPE_AXES; ++i) {
            if (i < n_axes) {
                if (axis_pairs[i] < 0) return LORA_ERR_INVALID_ARG;
                sum += axis_pairs[i];
            }
            a.axis_end[i] = static_cast<int>(sum < D ? sum : D);
        }
        if (sum != rot_dim / 2) return LORA_ERR_SHAPE;
        if (positions && ld_pos < n_axes) return LORA_ERR_SHAPE;
        if (positions && !aligned(positions, 4)) return LORA_ERR_ALIGNMENT;
    }
    if (batch->n_rows == 0) return LORA_OK;
    LORA_TRY(check_matrix(x, ld_x, 0));
    LORA_TRY(check_matrix(q_out, ld_q, nq));
    a.q_out = q_out; a.ld_q = ld_q; a.x = x; a.ld_x = ld_x; a.n_heads = n_heads;
    a.q_off = q_off; a.k_off = k_off; a.v_off = v_off;
    a.rope = rope; a.rot_dim = rot_dim; a.max_pos = max_pos; a.positions = positions; a.ld_pos = ld_pos; a.n_axes = n_axes;
    a.status = dev_status;
    return cuda_status(lora::launch_kv4_append(a, reinterpret_cast<cudaStream_t>(stream)));
}

lora_status_t lora_kv4_read(lora_bf16_t* k, int ld_k, lora_bf16_t* v, int ld_v, const lora_kv4_cache_t* cache,
                            const lora_kv4_batch_t* batch, int32_t* dev_status, lora_stream_t stream)
{
    lora::ReadArgs a{};
    LORA_TRY(check_cache(cache, a.cache));
    LORA_TRY(check_batch(batch, a.cache, a.batch));
    if (batch->n_rows == 0) return LORA_OK;
    const long long nk = static_cast<long long>(a.cache.n_kv) * a.cache.head_dim;
    LORA_TRY(check_matrix(k, ld_k, nk));
    LORA_TRY(check_matrix(v, ld_v, nk));
    a.k = k; a.ld_k = ld_k; a.v = v; a.ld_v = ld_v; a.status = dev_status;
    return cuda_status(lora::launch_kv4_read(a, reinterpret_cast<cudaStream_t>(stream)));
}

size_t lora_kv4_attend_workspace_bytes(int n_heads, int n_kv, int head_dim, int max_q_len)
{
    if (n_heads <= 0 || n_kv <= 0 || max_q_len < 0 || !head_dim_ok(head_dim) || n_heads % n_kv != 0 ||
        n_heads / n_kv > kMaxGroupHeads)
        return 0;
    return lora::kv4_attend_workspace(n_heads, n_kv, head_dim, max_q_len);
}

lora_status_t lora_kv4_attend(lora_bf16_t* out, int ld_out, const lora_bf16_t* q, int ld_q, int n_heads, float scale,
                              int window, const lora_kv4_cache_t* cache, const lora_kv4_batch_t* batch,
                              void* workspace, size_t ws_bytes, int32_t* dev_status, lora_stream_t stream)
{
    lora::AttendArgs a{};
    return attend(a, out, ld_out, q, ld_q, n_heads, scale, window, cache, batch, workspace, ws_bytes, dev_status, stream);
}

lora_status_t lora_kv4_attend_tree(lora_bf16_t* out, int ld_out, const lora_bf16_t* q, int ld_q, int n_heads, float scale,
                                   int window, const uint32_t* tree, int ld_tree, const lora_kv4_cache_t* cache,
                                   const lora_kv4_batch_t* batch, void* workspace, size_t ws_bytes, int32_t* dev_status,
                                   lora_stream_t stream)
{
    lora::AttendArgs a{};
    if (batch && batch->n_rows > 0) {
        if (!tree) return LORA_ERR_INVALID_ARG;
        if (ld_tree < (batch->max_q_len + 31LL) / 32) return LORA_ERR_SHAPE;
        if (!aligned(tree, 4)) return LORA_ERR_ALIGNMENT;
    }
    a.tree = tree;
    a.ld_tree = ld_tree;
    return attend(a, out, ld_out, q, ld_q, n_heads, scale, window, cache, batch, workspace, ws_bytes, dev_status, stream);
}

lora_status_t lora_kv4_plan(int32_t* q_starts, int32_t* ctx_lens, int32_t* row_seq, int32_t* positions, int64_t* slots,
                            const int32_t* q_lens, const int32_t* lens, const int32_t* depths, int n_seqs, int max_rows,
                            int max_q_len, int max_ctx_len, const lora_kv4_pool_t* pool, int32_t* dev_status,
                            lora_stream_t stream)
{
    if (!pool || n_seqs < 0 || max_rows < 0 || max_q_len < 0 || max_ctx_len < 0 || pool->n_pages <= 0) return LORA_ERR_INVALID_ARG;
    if (!page_size_ok(pool->page_size) || n_seqs > lora::kMaxSeqs || max_ctx_len > lora::kMaxPositions ||
        max_rows > lora::kMaxPositions || pool->n_pages > lora::kMaxPositions)
        return LORA_ERR_SHAPE;
    if (pool->ld_table < (max_ctx_len + pool->page_size - 1) / pool->page_size) return LORA_ERR_SHAPE;
    if (!q_starts || !pool->free_pages || !pool->n_free || !pool->n_free_out) return LORA_ERR_INVALID_ARG;
    if (n_seqs > 0 && (!ctx_lens || !q_lens || !lens || !pool->held || !pool->held_out || !pool->block_table || ctx_lens == lens))
        return LORA_ERR_INVALID_ARG;
    for (const void* p : {static_cast<const void*>(q_starts), static_cast<const void*>(ctx_lens), static_cast<const void*>(row_seq),
                          static_cast<const void*>(positions), static_cast<const void*>(q_lens), static_cast<const void*>(lens),
                          static_cast<const void*>(depths), static_cast<const void*>(pool->free_pages), static_cast<const void*>(pool->n_free),
                          static_cast<const void*>(pool->held), static_cast<const void*>(pool->n_free_out),
                          static_cast<const void*>(pool->held_out), static_cast<const void*>(pool->block_table)})
        if (!aligned(p, 4)) return LORA_ERR_ALIGNMENT;
    if (!aligned(slots, 8)) return LORA_ERR_ALIGNMENT;
    lora::PlanArgs a{q_starts, ctx_lens, row_seq, positions, slots, q_lens, lens, depths, n_seqs, max_rows, max_q_len, max_ctx_len, *pool, 0,
                     aligned(q_lens, 16) && aligned(lens, 16) && aligned(pool->held, 16),
                     aligned(row_seq, 16) && aligned(positions, 16) && aligned(slots, 16), dev_status};
    while ((1 << a.page_shift) < pool->page_size) ++a.page_shift;
    return cuda_status(lora::launch_kv4_plan(a, reinterpret_cast<cudaStream_t>(stream)));
}

lora_status_t lora_kv4_keep(const lora_kv4_cache_t* caches, int n_caches, const lora_kv4_batch_t* batch,
                            const int32_t* n_keep, const int32_t* path, int ld_path, int32_t* lens,
                            int32_t* dev_status, lora_stream_t stream)
{
    if (n_caches < 0 || (n_caches > 0 && !caches)) return LORA_ERR_INVALID_ARG;
    lora::KeepArgs a{};
    uint64_t seen[4] = {};
    for (int i = 0; i < n_caches; ++i) {
        lora::kv4::Cache c{};
        LORA_TRY(check_cache(caches + i, c));
        if (i == 0) {
            a.cache = c;
            a.least_pages = c.n_pages;
            LORA_TRY(check_batch(batch, c, a.batch));
        }
        if (c.n_pages < a.least_pages) a.least_pages = c.n_pages;
        // the same pages twice would be moved twice: a bit for each of 256 classes of pointers, and a look at the others where it is set
        const unsigned bit = static_cast<unsigned>((reinterpret_cast<uintptr_t>(c.pages) >> 8) * 0x9E3779B97F4A7C15ull >> 56);
        if (seen[bit >> 6] >> (bit & 63) & 1u)
            for (int k = 0; k < i; ++k)
                if (caches[k].pages == c.pages) return LORA_ERR_INVALID_ARG;
        seen[bit >> 6] |= 1ull << (bit & 63);
        if (c.page_size != a.cache.page_size || c.n_kv != a.cache.n_kv || c.head_dim != a.cache.head_dim) return LORA_ERR_SHAPE;
    }
    if (n_caches == 0 || batch->n_seqs == 0) return LORA_OK;
    if (!batch->q_starts || !batch->ctx_lens || !batch->block_table || !n_keep || !path || lens == batch->ctx_lens) return LORA_ERR_INVALID_ARG;
    if (ld_path < 0 || batch->ld_table < (static_cast<long long>(batch->max_ctx_len) + a.cache.page_size - 1) / a.cache.page_size)
        return LORA_ERR_SHAPE;
    for (const void* p : {static_cast<const void*>(batch->q_starts), static_cast<const void*>(batch->ctx_lens),
                          static_cast<const void*>(batch->block_table), static_cast<const void*>(batch->held), static_cast<const void*>(n_keep),
                          static_cast<const void*>(path), static_cast<const void*>(lens)})
        if (!aligned(p, 4)) return LORA_ERR_ALIGNMENT;
    a.held = batch->held; a.n_keep = n_keep; a.path = path; a.ld_path = ld_path; a.status = dev_status;
    for (int at = 0; at < n_caches; at += LORA_KEEP_LAYERS) {
        const int n = n_caches - at < LORA_KEEP_LAYERS ? n_caches - at : LORA_KEEP_LAYERS;
        for (int i = 0; i < n; ++i)
            a.layers[i] = lora::KeepArgs::Pages{caches[at + i].pages, static_cast<long long>(caches[at + i].page_stride), caches[at + i].n_pages};
        a.lens = at == 0 ? lens : nullptr;
        LORA_TRY(cuda_status(lora::launch_kv4_keep(a, n, reinterpret_cast<cudaStream_t>(stream))));
    }
    return LORA_OK;
}

lora_status_t lora_logits_adjust(void* out, lora_dtype_t out_type, int ld_out, const void* logits, lora_dtype_t type, int ld,
                                 int n_rows, int vocab, const lora_logits_rules_t* rules, const int32_t* row_seq,
                                 const int32_t* drafts, const uint32_t* tree, int ld_tree, const int32_t* q_starts,
                                 const uint32_t* allowed, int ld_allowed, int n_allowed, const int32_t* allowed_rows,
                                 int32_t* dev_status, lora_stream_t stream)
{
    constexpr int kCounts = (1 << 20) - 1, kBiases = 2047;   // what a token's counter holds (logits.cu)
    if (n_rows < 0 || vocab <= 0 || (type != LORA_BF16 && type != LORA_F32) || (out_type != LORA_BF16 && out_type != LORA_F32))
        return LORA_ERR_INVALID_ARG;
    if (vocab > 1 << 25 || static_cast<long long>(n_rows) * ((vocab + 2047) / 2048) > 1 << 30) return LORA_ERR_SHAPE;
    if (n_rows == 0) return LORA_OK;
    LORA_TRY(check_matrix(logits, ld, vocab));
    LORA_TRY(check_matrix(out, ld_out, vocab));
    if (out == logits && (type != out_type || ld != ld_out)) return LORA_ERR_INVALID_ARG;
    lora::LogitsArgs a{};
    if (rules) {
        const lora_logits_rules_t& r = *rules;
        if (r.n_seqs <= 0 || r.ld_tokens < 0 || r.ld_bias < 0 || !r.tokens || !r.prompt_lens || !r.token_lens) return LORA_ERR_INVALID_ARG;
        if (r.bias_ids && (!r.bias || !r.n_bias)) return LORA_ERR_INVALID_ARG;
        if (!row_seq && n_rows > r.n_seqs) return LORA_ERR_INVALID_ARG;
        if ((r.bias_ids && r.ld_bias > kBiases) || r.ld_tokens + (drafts ? 32LL * ld_tree : 0LL) > kCounts) return LORA_ERR_SHAPE;
        for (const void* p : {static_cast<const void*>(r.tokens), static_cast<const void*>(r.prompt_lens), static_cast<const void*>(r.token_lens),
                              static_cast<const void*>(r.repetition), static_cast<const void*>(r.frequency), static_cast<const void*>(r.presence),
                              static_cast<const void*>(r.bias_ids), static_cast<const void*>(r.bias), static_cast<const void*>(r.n_bias)})
            if (!aligned(p, 4)) return LORA_ERR_ALIGNMENT;
        a.rules = r;
    }
    if (drafts) {
        if (!rules || !tree || !q_starts) return LORA_ERR_INVALID_ARG;
        if (ld_tree <= 0) return LORA_ERR_SHAPE;
    }
    if (allowed) {
        if (n_allowed <= 0 || (!allowed_rows && n_rows > n_allowed)) return LORA_ERR_INVALID_ARG;
        if (ld_allowed < (vocab + 31) / 32) return LORA_ERR_SHAPE;
    }
    for (const void* p : {static_cast<const void*>(row_seq), static_cast<const void*>(drafts), static_cast<const void*>(tree),
                          static_cast<const void*>(q_starts), static_cast<const void*>(allowed), static_cast<const void*>(allowed_rows)})
        if (!aligned(p, 4)) return LORA_ERR_ALIGNMENT;
    a.out = out; a.ld_out = ld_out; a.logits = logits; a.ld = ld; a.n_rows = n_rows; a.vocab = vocab;
    a.row_seq = row_seq; a.drafts = drafts; a.tree = tree; a.ld_tree = ld_tree; a.q_starts = q_starts;
    a.allowed = allowed; a.ld_allowed = ld_allowed; a.n_allowed = n_allowed; a.allowed_rows = allowed_rows;
    a.status = dev_status;
    return cuda_status(lora::launch_logits_adjust(a, type == LORA_F32, out_type == LORA_F32, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
