// C ABI of the serving-step operators: host-side validation, then the launches on
// the caller's stream, as in api.hip.
#include "api_checks.h"

extern "C" {

int tq_plan_step(int64_t batch, const int32_t *lens, const int32_t *new_tokens,
                 const int32_t *owned, int32_t *page_table, int64_t table_stride,
                 int64_t table_pages, int64_t page_size, const int32_t *free_pages,
                 int64_t free_capacity, const int32_t *free_count, int64_t tokens,
                 int32_t *starts, int32_t *positions, int32_t *slots, int32_t *new_lens,
                 int32_t *new_owned, int32_t *free_left, hipStream_t stream)
{
    if (!within(batch, 0, MAX_BATCH) || !tq::cache_page_ok(page_size) ||
        !within(table_pages, 1, MAX_PAGES) || table_pages * page_size > MAX_POSITIONS ||
        !within(table_stride, batch > 1 ? table_pages : 0, MAX_STRIDE) ||
        !within(free_capacity, 0, MAX_PAGES) || !within(tokens, 0, MAX_TOKENS))
        return TQ_E_SHAPE;
    if ((batch && (!lens || !new_tokens || !owned || !page_table || !new_lens || !new_owned)) ||
        (free_capacity && !free_pages) || !free_count || !starts ||
        (tokens && (!positions || !slots)) || !free_left)
        return TQ_E_NULL;
    if (!aligned(lens, 4) || !aligned(new_tokens, 4) || !aligned(owned, 4) ||
        !aligned(page_table, 4) || !aligned(free_pages, 4) || !aligned(free_count, 4) ||
        !aligned(starts, 4) || !aligned(positions, 4) || !aligned(slots, 4) ||
        !aligned(new_lens, 4) || !aligned(new_owned, 4) || !aligned(free_left, 4))
        return TQ_E_ALIGN;
    // every workgroup reads the old state for itself while others write the new one
    const struct { const void *p; int64_t n; } in[] = {
        {lens, batch}, {new_tokens, batch}, {owned, batch}, {free_pages, free_capacity}, {free_count, 1}};
    const struct { const void *p; int64_t n; } out[] = {
        {starts, batch + 1}, {positions, tokens}, {slots, tokens}, {new_lens, batch},
        {new_owned, batch}, {free_left, 1}};
    for (const auto &i : in)
        for (const auto &o : out)
            if (overlap(i.p, 4 * i.n, o.p, 4 * o.n))
                return TQ_E_SHAPE;
    // the table is read and written: no other array lies in it
    const int64_t entries = batch ? (batch - 1) * table_stride + table_pages : 0;
    for (const auto &i : in)
        if (overlap(i.p, 4 * i.n, page_table, 4 * entries))
            return TQ_E_SHAPE;
    for (const auto &o : out)
        if (overlap(o.p, 4 * o.n, page_table, 4 * entries))
            return TQ_E_SHAPE;
    const tq::PlanArgs a{lens, new_tokens, owned, page_table, table_stride, table_pages, free_pages,
                         free_count, free_capacity, batch, tokens, tq::log2_of(page_size), starts,
                         positions, slots, new_lens, new_owned, free_left};
    return launch_status(tq::launch_plan(a, stream));
}

int tq_release_pages(int64_t batch, const int32_t *done, const int32_t *owned, int32_t *page_table,
                     int64_t table_stride, int64_t table_pages, int32_t *free_pages,
                     int64_t free_capacity, const int32_t *free_count, int32_t *new_owned,
                     int32_t *free_left, hipStream_t stream)
{
    if (!within(batch, 0, MAX_BATCH) || !within(table_pages, 1, MAX_PAGES) ||
        !within(table_stride, batch > 1 ? table_pages : 0, MAX_STRIDE) ||
        !within(free_capacity, 0, MAX_PAGES))
        return TQ_E_SHAPE;
    if ((batch && (!done || !owned || !page_table || !new_owned)) ||
        (free_capacity && !free_pages) || !free_count || !free_left)
        return TQ_E_NULL;
    if (!aligned(done, 4) || !aligned(owned, 4) || !aligned(page_table, 4) ||
        !aligned(free_pages, 4) || !aligned(free_count, 4) || !aligned(new_owned, 4) ||
        !aligned(free_left, 4))
        return TQ_E_ALIGN;
    if (overlap(owned, 4 * batch, new_owned, 4 * batch) ||
        overlap(done, 4 * batch, new_owned, 4 * batch) || overlap(free_count, 4, free_left, 4))
        return TQ_E_SHAPE;
    // the table and the stack are written: no other array lies in them
    const int64_t entries = batch ? (batch - 1) * table_stride + table_pages : 0;
    const struct { const void *p; int64_t n; } others[] = {
        {done, batch}, {owned, batch}, {free_count, 1}, {new_owned, batch}, {free_left, 1}};
    for (const auto &o : others)
        if (overlap(o.p, 4 * o.n, page_table, 4 * entries) ||
            overlap(o.p, 4 * o.n, free_pages, 4 * free_capacity))
            return TQ_E_SHAPE;
    if (overlap(free_pages, 4 * free_capacity, page_table, 4 * entries))
        return TQ_E_SHAPE;
    const tq::ReleaseArgs a{done, owned, page_table, table_stride, table_pages, free_pages,
                            free_count, free_capacity, batch, new_owned, free_left};
    return launch_status(tq::launch_release(a, stream));
}

int tq_residual_norm(int dtype, int y_dtype, const void *y, int64_t y_ts, const void *x,
                     int64_t x_ts, int64_t tokens, int64_t N, int w_dtype, const void *post_weight,
                     const void *pre_weight, const void *gate, int64_t gate_ts, int64_t gate_es,
                     float scale, float eps, void *x_out, int64_t xo_ts, void *z, int64_t z_ts,
                     int8_t *q, uint16_t *d, hipStream_t stream)
{
    if (!valid_dtype(dtype) || !valid_dtype(y_dtype) ||
        ((post_weight || pre_weight || gate) && !valid_dtype(w_dtype)))
        return TQ_E_TYPE;
    if (!within(tokens, 0, MAX_TOKENS) || !within(N, 1, 32768) || ((q || d) && N % 32) ||
        !within(y_ts, 0, MAX_STRIDE) || !within(x_ts, 0, MAX_STRIDE) ||
        !within(xo_ts, tokens > 1 ? N : 0, MAX_STRIDE) ||
        (z && !within(z_ts, tokens > 1 ? N : 0, MAX_STRIDE)) ||
        (gate && (!within(gate_ts, 0, MAX_STRIDE) || !within(gate_es, 0, 1))) ||
        !std::isfinite(scale) || !(eps >= 0.0f) || !std::isfinite(eps))
        return TQ_E_SHAPE;
    if (tokens == 0)
        return TQ_OK;
    if (!y || !x || !x_out || !z == !q || !q != !d)
        return TQ_E_NULL;
    if (x == x_out && x_ts != xo_ts && tokens > 1)
        return TQ_E_SHAPE;
    const uintptr_t al = size_of(dtype), wal = size_of(w_dtype);
    if (!aligned(y, size_of(y_dtype)) || !aligned(x, al) || !aligned(x_out, al) || !aligned(z, al) ||
        !aligned(post_weight, wal) || !aligned(pre_weight, wal) || !aligned(gate, wal) ||
        !aligned(q, 4) || !aligned(d, 2))
        return TQ_E_ALIGN;
    // rows are read by other workgroups than those that write near them; only x' may take
    // x's place, and z that of x', which it then is
    const int64_t one = al, wone = wal, yone = size_of(y_dtype), T = tokens;
    const Span ins[] = {{y, y_ts * yone, N * yone, T}, {x, x_ts * one, N * one, T},
                        {post_weight, 0, N * wone, 1}, {pre_weight, 0, N * wone, 1},
                        {gate, gate_ts * wone, gate_es ? N * wone : wone, T}};
    const bool same_z = z == x_out && !pre_weight && (z_ts == xo_ts || T == 1);
    const Span outs[] = {{x_out, xo_ts * one, N * one, T},
                         {same_z ? nullptr : z, z_ts * one, N * one, T},
                         {q, N, N, T}, {d, N / 32 * 2, N / 32 * 2, T}};
    for (int o = 0; o < 4; o++) {
        for (int i = 0; i < 5; i++)
            if (!(o == 0 && i == 1 && x == x_out) && meet(outs[o], ins[i]))
                return TQ_E_SHAPE;
        for (int i = 0; i < o; i++)
            if (meet(outs[o], outs[i]))
                return TQ_E_SHAPE;
    }
    const tq::ResNormArgs a{y, x, y_ts, x_ts, y_dtype, w_dtype, post_weight, pre_weight, gate,
                            gate_ts, gate_es, scale, eps, tokens, (int)N, x_out, z, xo_ts, z_ts,
                            q, d};
    return launch_status(tq::launch_residual_norm(dtype, a, stream));
}

}  // extern "C"

namespace {

// 62 bits hold `vocab` weights, each at most 2^bits.
int weight_bits(int64_t vocab)
{
    int l = 0;
    while ((int64_t(1) << l) < vocab)
        l++;
    return l < 17 ? 45 : 62 - l;
}

int sample(int dtype, const void *logits, int64_t stride, int64_t rows, int64_t vocab,
           const float *temperature, const int32_t *top_k, const float *top_p, const float *min_p,
           const float *uniforms, int32_t *tokens, float *probs, int64_t probs_stride,
           void *workspace, size_t workspace_bytes, hipStream_t stream)
{
    if (!valid_dtype(dtype))
        return TQ_E_TYPE;
    if (!within(rows, 0, MAX_TOKENS) || !within(vocab, 1, int64_t(1) << 27) ||
        rows * vocab >= (int64_t(1) << 34) || !within(stride, 0, MAX_STRIDE) ||
        (probs && !within(probs_stride, rows > 1 ? vocab : 0, MAX_STRIDE)))
        return TQ_E_SHAPE;
    if (rows == 0)
        return TQ_OK;
    if (!logits || (!probs && (!uniforms || !tokens)))
        return TQ_E_NULL;
    if (!aligned(logits, size_of(dtype)) || !aligned(temperature, 4) || !aligned(top_k, 4) ||
        !aligned(top_p, 4) || !aligned(min_p, 4) || !aligned(uniforms, 4) || !aligned(tokens, 4) ||
        !aligned(probs, 4))
        return TQ_E_ALIGN;
    // a row's logits are read by several workgroups and launches; the last one reads
    // each element where it writes its probability, if anywhere
    const int64_t size = size_of(dtype);
    const Span ins[] = {{logits, stride * size, vocab * size, rows}, {temperature, 0, 4 * rows, 1},
                        {top_k, 0, 4 * rows, 1}, {top_p, 0, 4 * rows, 1}, {min_p, 0, 4 * rows, 1},
                        {uniforms, 0, 4 * rows, 1}};
    const Span out = probs ? Span{probs, probs_stride * 4, vocab * 4, rows}
                           : Span{tokens, 0, 4 * rows, 1};
    const bool in_place = probs == logits && dtype == TQ_F32 && (probs_stride == stride || rows == 1);
    for (int i = in_place ? 1 : 0; i < 6; i++)
        if (meet(out, ins[i]))
            return TQ_E_SHAPE;
    uint32_t *counters;                          // unused: the layout that all calls share
    void *scratch;
    const int st = scratch_of(workspace, workspace_bytes,
                              tq_sample_workspace_bytes(rows, vocab), &counters, &scratch);
    if (st != TQ_OK)
        return st;
    const tq::SampleArgs a{logits, stride, rows, vocab, dtype, weight_bits(vocab), temperature,
                           top_p, min_p, top_k, uniforms, tokens, probs, probs_stride};
    return launch_status(tq::launch_sample(a, scratch, stream));
}

}  // namespace

extern "C" {

size_t tq_sample_workspace_bytes(int64_t rows, int64_t vocab)
{
    if (!within(rows, 1, MAX_TOKENS) || !within(vocab, 1, int64_t(1) << 27) ||
        rows * vocab >= (int64_t(1) << 34))
        return 0;
    const size_t n = tq::sample_scratch_bytes(rows, vocab);
    return n ? TQ_NOALLOC_SCRATCH_BYTES + n : 0;
}

int tq_sample(int dtype, const void *logits, int64_t stride, int64_t rows, int64_t vocab,
              const float *temperature, const int32_t *top_k, const float *top_p,
              const float *min_p, const float *uniforms, int32_t *tokens, void *workspace,
              size_t workspace_bytes, hipStream_t stream)
{
    return sample(dtype, logits, stride, rows, vocab, temperature, top_k, top_p, min_p, uniforms,
                  tokens, nullptr, 0, workspace, workspace_bytes, stream);
}

int tq_sample_probs(int dtype, const void *logits, int64_t stride, int64_t rows, int64_t vocab,
                    const float *temperature, const int32_t *top_k, const float *top_p,
                    const float *min_p, float *probs, int64_t probs_stride, void *workspace,
                    size_t workspace_bytes, hipStream_t stream)
{
    if (rows > 0 && !probs)
        return TQ_E_NULL;
    return sample(dtype, logits, stride, rows, vocab, temperature, top_k, top_p, min_p, nullptr,
                  nullptr, probs, probs_stride, workspace, workspace_bytes, stream);
}

int tq_cache_bounds(int type, const void *k_cache, int64_t n_pages, int64_t page_size,
                    int64_t kv_heads, int64_t D, const int32_t *page_table, int64_t table_stride,
                    int64_t table_pages, int64_t batch, const int32_t *begin, const int32_t *end,
                    int64_t max_new, int8_t *codes, uint16_t *scales, hipStream_t stream)
{
    if (!tq::cache_type_ok(type))
        return TQ_E_TYPE;
    if (!valid_cache(n_pages, page_size, kv_heads, D) || !within(batch, 0, MAX_BATCH) ||
        !within(table_pages, 1, MAX_PAGES) || table_pages * page_size > MAX_POSITIONS ||
        !within(table_stride, batch > 1 ? table_pages : 0, MAX_STRIDE) ||
        !within(max_new, 0, MAX_POSITIONS))
        return TQ_E_SHAPE;
    const int64_t touched = (max_new + page_size - 2) / page_size + 1;
    if ((touched < table_pages ? touched : table_pages) * kv_heads * D >= (int64_t(1) << 31))
        return TQ_E_SHAPE;
    if (batch == 0 || max_new == 0)
        return TQ_OK;
    if (!k_cache || !page_table || !begin || !end || !codes || !scales)
        return TQ_E_NULL;
    if (!aligned(k_cache, 16) || !aligned(page_table, 4) || !aligned(begin, 4) || !aligned(end, 4) ||
        !aligned(codes, 16) || !aligned(scales, 2))
        return TQ_E_ALIGN;
    const tq::BoundsArgs a{(const uint8_t *)k_cache, page_table, table_stride, begin, end, codes,
                           scales, n_pages, (int)table_pages, tq::log2_of(page_size), (int)batch,
                           (int)kv_heads};
    return launch_status(tq::launch_bounds(type, (int)D, a, max_new, stream));
}

int64_t tq_select_pages_width(int64_t page_size, int64_t table_pages, int64_t first, int64_t last,
                              int64_t keep, int64_t max_nodes)
{
    if (!tq::cache_page_ok(page_size) || !within(table_pages, 1, MAX_PAGES) ||
        !within(first, 0, MAX_PAGES) || !within(last, 0, MAX_PAGES) ||
        !within(keep, 0, MAX_PAGES) || !within(max_nodes, 1, MAX_TOKENS))
        return 0;
    const int64_t n = first + last + keep + (max_nodes + page_size - 2) / page_size + 1;
    return n < table_pages ? n : table_pages;
}

size_t tq_select_pages_workspace_bytes(int64_t batch, int64_t kv_heads, int64_t table_pages)
{
    if (!within(batch, 1, MAX_BATCH) || !within(kv_heads, 1, MAX_HEADS) ||
        !within(table_pages, 1, MAX_PAGES) || batch * kv_heads > MAX_TOKENS)
        return 0;
    return TQ_NOALLOC_SCRATCH_BYTES + tq::select_scratch_bytes(batch, kv_heads, table_pages);
}

int tq_select_pages(int dtype, const void *q, int64_t q_ts, int64_t q_hs, int64_t tokens,
                    int64_t heads, int64_t kv_heads, int64_t D, const int8_t *codes,
                    const uint16_t *scales, int64_t n_pages, int64_t page_size,
                    const int32_t *page_table, int64_t table_stride, int64_t table_pages,
                    int64_t batch, const int32_t *ctx_lens, const int32_t *starts,
                    int64_t max_nodes, int64_t max_ctx, int64_t first, int64_t last, int64_t keep,
                    int64_t width, int32_t *tables, int32_t *ctx_out, void *workspace,
                    size_t workspace_bytes, hipStream_t stream)
{
    if (dtype != TQ_BF16 && dtype != TQ_F16)
        return TQ_E_TYPE;
    if (!valid_cache(n_pages, page_size, kv_heads, D) || !within(heads, kv_heads, MAX_HEADS) ||
        heads % kv_heads || !within(tokens, 0, MAX_TOKENS) || !within(batch, 0, MAX_BATCH) ||
        batch * kv_heads > MAX_TOKENS || !within(table_pages, 1, MAX_PAGES) ||
        table_pages * page_size > MAX_POSITIONS ||
        !within(table_stride, batch > 1 ? table_pages : 0, MAX_STRIDE) ||
        !within(max_nodes, 1, MAX_TOKENS) || !within(max_ctx, 0, MAX_POSITIONS) ||
        !valid_strides(q_ts, q_hs))
        return TQ_E_SHAPE;
    const int64_t least =
        tq_select_pages_width(page_size, table_pages, first, last, keep, max_nodes);
    if (least == 0 || !within(width, least, MAX_PAGES))
        return TQ_E_SHAPE;
    if (batch == 0)
        return TQ_OK;
    if ((tokens && !q) || !codes || !scales || !page_table || !ctx_lens || !starts || !tables ||
        !ctx_out)
        return TQ_E_NULL;
    if (!aligned(q, 2) || !aligned(codes, 16) || !aligned(scales, 2) || !aligned(page_table, 4) ||
        !aligned(ctx_lens, 4) || !aligned(starts, 4) || !aligned(tables, 4) || !aligned(ctx_out, 4))
        return TQ_E_ALIGN;
    if (overlap(ctx_lens, 4 * batch, ctx_out, 4 * batch) ||
        overlap(starts, 4 * (batch + 1), ctx_out, 4 * batch) ||
        overlap(ctx_lens, 4 * batch, tables, 4 * batch * kv_heads * width) ||
        overlap(starts, 4 * (batch + 1), tables, 4 * batch * kv_heads * width) ||
        overlap(page_table, 4 * ((batch - 1) * table_stride + table_pages), tables,
                4 * batch * kv_heads * width))
        return TQ_E_SHAPE;
    uint32_t *counters;
    void *scratch;
    const int st = scratch_of(workspace, workspace_bytes,
                              tq_select_pages_workspace_bytes(batch, kv_heads, table_pages),
                              &counters, &scratch);
    if (st != TQ_OK)
        return st;
    const tq::SelectArgs a{q, q_ts, q_hs, tokens, codes, scales, n_pages, page_table, table_stride,
                           ctx_lens, starts, (int)table_pages, tq::log2_of(page_size), (int)batch,
                           (int)kv_heads, (int)(heads / kv_heads), (int)max_nodes, dtype,
                           (int)first, (int)last, (int)keep, (int)width, tables, ctx_out};
    return launch_status(tq::launch_select((int)D, a, max_ctx, counters, scratch, stream));
}

}  // extern "C"
