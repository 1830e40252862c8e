// C ABI of the decode-step operators: host-side validation, then the launches
// on the caller's stream, as in api.hip.
#include "api_checks.h"


extern "C" {

int tq_qk_norm_rope(int dtype, const void *q, int64_t q_ts, int64_t q_hs, int64_t q_heads,
                    const void *k, int64_t k_ts, int64_t k_hs, int64_t k_heads, int64_t tokens,
                    int64_t D, int64_t rot, int interleaved, int w_dtype, const void *q_weight,
                    const void *k_weight, float eps, const int32_t *positions,
                    const float *inv_freq, void *q_out, int64_t qo_ts, int64_t qo_hs, void *k_out,
                    int64_t ko_ts, int64_t ko_hs, hipStream_t stream)
{
    if (!valid_dtype(dtype) || ((q_weight || k_weight) && !valid_dtype(w_dtype)))
        return TQ_E_TYPE;
    if (!within(D, 2, 512) || D % 2 || !within(rot, 0, D) || rot % 2 ||
        !within(tokens, 0, MAX_TOKENS) || !within(q_heads, 0, MAX_HEADS) ||
        !within(k_heads, 0, MAX_HEADS) || q_heads + k_heads == 0 || !valid_strides(q_ts, q_hs) ||
        !valid_strides(k_ts, k_hs) || !apart(qo_ts, qo_hs, tokens, q_heads, D) ||
        !apart(ko_ts, ko_hs, tokens, k_heads, D) || !(eps >= 0.0f) || !std::isfinite(eps))
        return TQ_E_SHAPE;
    if (tokens == 0)
        return TQ_OK;
    if ((q_heads && (!q || !q_out)) || (k_heads && (!k || !k_out)) || !positions ||
        (rot && !inv_freq))
        return TQ_E_NULL;
    const uintptr_t al = size_of(dtype), wal = size_of(w_dtype);
    if (!aligned(q, al) || !aligned(k, al) || !aligned(q_out, al) || !aligned(k_out, al) ||
        !aligned(q_weight, wal) || !aligned(k_weight, wal) || !aligned(positions, 4) ||
        !aligned(inv_freq, 4))
        return TQ_E_ALIGN;
    const tq::NormRopeArgs a{{q, k}, {q_out, k_out}, {q_ts, k_ts}, {q_hs, k_hs}, {qo_ts, ko_ts},
                             {qo_hs, ko_hs}, {q_weight, k_weight}, {(int)q_heads, (int)k_heads},
                             w_dtype, tokens, (int)D, (int)rot, interleaved != 0, eps, positions,
                             inv_freq};
    return launch_status(tq::launch_norm_rope(dtype, a, stream));
}

size_t tq_cache_bytes(int type, int64_t n_pages, int64_t page_size, int64_t kv_heads, int64_t D)
{
    if (!tq::cache_type_ok(type) || !valid_cache(n_pages, page_size, kv_heads, D))
        return 0;
    return (size_t)n_pages * kv_heads * tq::chunk_bytes(type, D, page_size);
}

int tq_cache_write(int type, int dtype, const void *k, int64_t k_ts, int64_t k_hs, const void *v,
                   int64_t v_ts, int64_t v_hs, int64_t tokens, int64_t kv_heads, int64_t D,
                   const int32_t *slots, void *k_cache, void *v_cache, int64_t n_pages,
                   int64_t page_size, hipStream_t stream)
{
    if (!tq::cache_type_ok(type) || !valid_dtype(dtype))
        return TQ_E_TYPE;
    if (!valid_cache(n_pages, page_size, kv_heads, D) || !within(tokens, 0, MAX_TOKENS) ||
        !valid_strides(k_ts, k_hs) || !valid_strides(v_ts, v_hs) ||
        tokens * kv_heads * D >= (int64_t(1) << 34))
        return TQ_E_SHAPE;
    if (tokens == 0)
        return TQ_OK;
    if (!k || !v || !slots || !k_cache || !v_cache)
        return TQ_E_NULL;
    if (!aligned(k, size_of(dtype)) || !aligned(v, size_of(dtype)) || !aligned(slots, 4) ||
        !aligned(k_cache, 16) || !aligned(v_cache, 16))
        return TQ_E_ALIGN;
    const tq::CacheShape c{type, (int)kv_heads, (int)D, n_pages, page_size};
    return launch_status(tq::launch_cache_write(c, dtype, k, k_ts, k_hs, v, v_ts, v_hs, tokens,
                                                slots, k_cache, v_cache, stream));
}

int tq_cache_read(int type, int dtype, const void *k_cache, const void *v_cache, int64_t n_pages,
                  int64_t page_size, int64_t kv_heads, int64_t D, const int32_t *slots,
                  int64_t tokens, void *k, void *v, hipStream_t stream)
{
    if (!tq::cache_type_ok(type) || !valid_dtype(dtype))
        return TQ_E_TYPE;
    if (!valid_cache(n_pages, page_size, kv_heads, D) || !within(tokens, 0, MAX_TOKENS) ||
        tokens * kv_heads * D >= (int64_t(1) << 34))
        return TQ_E_SHAPE;
    if (tokens == 0)
        return TQ_OK;
    if (!k || !v || !slots || !k_cache || !v_cache)
        return TQ_E_NULL;
    if (!aligned(k, size_of(dtype)) || !aligned(v, size_of(dtype)) || !aligned(slots, 4) ||
        !aligned(k_cache, 16) || !aligned(v_cache, 16))
        return TQ_E_ALIGN;
    const tq::CacheShape c{type, (int)kv_heads, (int)D, n_pages, page_size};
    return launch_status(
        tq::launch_cache_read(c, dtype, k_cache, v_cache, slots, tokens, k, v, stream));
}

size_t tq_tree_attention_workspace_bytes(int64_t batch, int64_t heads, int64_t kv_heads, int64_t D,
                                         int64_t max_nodes, int64_t max_ctx)
{
    if (!within(batch, 1, MAX_BATCH) || !within(kv_heads, 1, MAX_HEADS) ||
        !within(heads, kv_heads, MAX_HEADS) || heads % kv_heads || !tq::cache_dim_ok(D) ||
        !within(max_nodes, 1, MAX_TOKENS) || !within(max_ctx, 0, MAX_POSITIONS))
        return 0;
    const tq::AttnPlan p = tq::attn_plan((int)D, batch, heads, kv_heads, max_nodes,
                                         max_ctx + max_nodes, false);
    const size_t n = tq::attn_scratch_bytes(p, (int)D, batch, kv_heads);
    return n ? TQ_NOALLOC_SCRATCH_BYTES + n : 0;
}

namespace {

// table_head_stride 0: all key heads read the same pages.
int attention(int type, int dtype, const void *q, int64_t q_ts, int64_t q_hs, int64_t tokens,
              int64_t heads, int64_t kv_heads, int64_t D, const void *k_cache, const void *v_cache,
              int64_t n_pages, int64_t page_size, const int32_t *page_table, int64_t table_stride,
              int64_t table_head_stride, int64_t table_pages, int64_t batch,
              const int32_t *ctx_lens, const int32_t *starts, const uint32_t *mask,
              int64_t mask_stride, int64_t mask_words, int64_t max_nodes, int64_t max_ctx,
              float scale, void *out, int64_t o_ts, int64_t o_hs, void *workspace,
              size_t workspace_bytes, hipStream_t stream)
{
    if (!tq::cache_type_ok(type) || (dtype != TQ_BF16 && dtype != TQ_F16))
        return TQ_E_TYPE;
    if (!valid_cache(n_pages, page_size, kv_heads, D) || !within(heads, kv_heads, MAX_HEADS) ||
        heads % kv_heads || !within(tokens, 0, MAX_TOKENS) || !within(batch, 0, MAX_BATCH) ||
        !within(table_pages, 1, MAX_PAGES) || table_pages * page_size > MAX_POSITIONS ||
        !within(table_stride, batch > 1 ? table_pages : 0, MAX_STRIDE) ||
        !within(table_head_stride, 0, MAX_STRIDE) ||
        !within(max_nodes, 1, MAX_TOKENS) || !within(max_ctx, 0, MAX_POSITIONS) ||
        !valid_strides(q_ts, q_hs) || !apart(o_ts, o_hs, tokens, heads, D) ||
        !(scale > 0.0f) || !std::isfinite(scale) ||
        (mask && (!within(mask_words, 1, MAX_TOKENS) ||
                  !within(mask_stride, tokens > 1 ? mask_words : 0, MAX_STRIDE))))
        return TQ_E_SHAPE;
    if (tokens == 0 || batch == 0)
        return TQ_OK;
    if (!q || !out || !k_cache || !v_cache || !page_table || !ctx_lens || !starts)
        return TQ_E_NULL;
    if (!aligned(q, 2) || !aligned(out, 2) || !aligned(k_cache, 16) || !aligned(v_cache, 16) ||
        !aligned(page_table, 4) || !aligned(ctx_lens, 4) || !aligned(starts, 4) ||
        !aligned(mask, 4))
        return TQ_E_ALIGN;
    const tq::AttnPlan p = tq::attn_plan((int)D, batch, heads, kv_heads, max_nodes,
                                         max_ctx + max_nodes, table_head_stride != 0);
    uint32_t *counters;                          // unused: the layout that all calls share
    void *scratch;
    const int st = scratch_of(
        workspace, workspace_bytes,
        tq_tree_attention_workspace_bytes(batch, heads, kv_heads, D, max_nodes, max_ctx),
        &counters, &scratch);
    if (st != TQ_OK)
        return st;
    const tq::AttnArgs a{q, out, q_ts, q_hs, o_ts, o_hs, (const uint8_t *)k_cache,
                         (const uint8_t *)v_cache, page_table, table_stride, table_head_stride,
                         ctx_lens, starts, mask, mask_stride, n_pages, tokens, (int)table_pages,
                         tq::log2_of(page_size), (int)batch, (int)kv_heads,
                         (int)(heads / kv_heads), (int)max_nodes, (int)mask_words, dtype, scale};
    return launch_status(tq::launch_attention(type, (int)D, a, p, scratch, stream));
}

}  // namespace

int tq_tree_attention(int type, int dtype, const void *q, int64_t q_ts, int64_t q_hs,
                      int64_t tokens, int64_t heads, int64_t kv_heads, int64_t D,
                      const void *k_cache, const void *v_cache, int64_t n_pages,
                      int64_t page_size, const int32_t *page_table, int64_t table_stride,
                      int64_t table_pages, int64_t batch, const int32_t *ctx_lens,
                      const int32_t *starts, const uint32_t *mask, int64_t mask_stride,
                      int64_t mask_words, int64_t max_nodes, int64_t max_ctx, float scale,
                      void *out, int64_t o_ts, int64_t o_hs, void *workspace,
                      size_t workspace_bytes, hipStream_t stream)
{
    return attention(type, dtype, q, q_ts, q_hs, tokens, heads, kv_heads, D, k_cache, v_cache,
                     n_pages, page_size, page_table, table_stride, 0, table_pages, batch, ctx_lens,
                     starts, mask, mask_stride, mask_words, max_nodes, max_ctx, scale, out, o_ts,
                     o_hs, workspace, workspace_bytes, stream);
}

int tq_tree_attention_heads(int type, int dtype, const void *q, int64_t q_ts, int64_t q_hs,
                            int64_t tokens, int64_t heads, int64_t kv_heads, int64_t D,
                            const void *k_cache, const void *v_cache, int64_t n_pages,
                            int64_t page_size, const int32_t *page_tables, int64_t table_stride,
                            int64_t table_head_stride, int64_t table_pages, int64_t batch,
                            const int32_t *ctx_lens, const int32_t *starts, const uint32_t *mask,
                            int64_t mask_stride, int64_t mask_words, int64_t max_nodes,
                            int64_t max_ctx, float scale, void *out, int64_t o_ts, int64_t o_hs,
                            void *workspace, size_t workspace_bytes, hipStream_t stream)
{
    return attention(type, dtype, q, q_ts, q_hs, tokens, heads, kv_heads, D, k_cache, v_cache,
                     n_pages, page_size, page_tables, table_stride, table_head_stride, table_pages,
                     batch, ctx_lens, starts, mask, mask_stride, mask_words, max_nodes, max_ctx,
                     scale, out, o_ts, o_hs, workspace, workspace_bytes, stream);
}

size_t tq_verify_draft_workspace_bytes(int64_t batch, int64_t vocab)
{
    if (!within(batch, 1, MAX_BATCH) || !within(vocab, 1, int64_t(1) << 27))
        return 0;
    return TQ_NOALLOC_SCRATCH_BYTES + tq::verify_scratch_bytes(batch, vocab);
}

int tq_verify_draft(int dtype, const void *target, int64_t target_stride, const void *draft,
                    int64_t draft_stride, int64_t nodes, int64_t vocab, const int32_t *tokens,
                    const int32_t *parents, const int32_t *starts, int64_t batch,
                    const float *uniforms, const float *final_uniforms, int64_t width,
                    int32_t *accepted, int32_t *out_tokens, int32_t *out_nodes, void *workspace,
                    size_t workspace_bytes, hipStream_t stream)
{
    if (!valid_dtype(dtype))
        return TQ_E_TYPE;
    if (!within(nodes, 0, MAX_TOKENS) || !within(batch, 0, MAX_BATCH) ||
        !within(vocab, 1, int64_t(1) << 27) || !within(width, 1, 1024) ||
        !within(target_stride, nodes > 1 ? vocab : 0, MAX_STRIDE) ||
        (draft && !within(draft_stride, nodes > 1 ? vocab : 0, MAX_STRIDE)))
        return TQ_E_SHAPE;
    if (batch == 0)
        return TQ_OK;
    if ((nodes && (!target || !tokens || !uniforms)) || !starts || !final_uniforms || !accepted ||
        !out_tokens || !out_nodes)
        return TQ_E_NULL;
    const uintptr_t al = size_of(dtype);
    if (!aligned(target, al) || !aligned(draft, al) || !aligned(tokens, 4) ||
        !aligned(parents, 4) || !aligned(starts, 4) || !aligned(uniforms, 4) ||
        !aligned(final_uniforms, 4) || !aligned(accepted, 4) || !aligned(out_tokens, 4) ||
        !aligned(out_nodes, 4))
        return TQ_E_ALIGN;
    uint32_t *counters;
    void *scratch;
    const int st = scratch_of(workspace, workspace_bytes,
                              tq_verify_draft_workspace_bytes(batch, vocab), &counters, &scratch);
    if (st != TQ_OK)
        return st;
    const tq::VerifyArgs a{target, draft, target_stride, draft_stride, tokens, parents, starts,
                           uniforms, final_uniforms, nodes, vocab, (int)batch, (int)width,
                           accepted, out_tokens, out_nodes};
    return launch_status(tq::launch_verify(dtype, a, counters, scratch, stream));
}

}  // extern "C"
