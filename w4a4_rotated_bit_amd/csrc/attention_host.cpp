// attention_host.cpp -- argument checks and workspace sizes of attention and of
// the paged cache that it reads.  Pure C++: nothing here calls the HIP runtime.
#include <math.h>
#include <stdlib.h>

#include "../../include/convrot.h"
#include "attention_ops.h"
#include "internal.h"
#include "overlap.h"

using namespace convrot;

namespace {

bool half_type(int dtype) { return dtype == CONVROT_BF16 || dtype == CONVROT_F16; }

// The blocks of a cache's rows and of its scales.
Block rows_of(const convrot_kv_cache& c, const convrot_cache_rows& r)
{
    Block b(r.rows_dev, cache_row_bytes(c.kind, c.head_dim), 1);
    b.add(c.pages, r.page_stride, 1);
    b.add(c.heads, r.head_stride, 1);
    b.add(c.page_size, r.token_stride, 1);
    return b;
}
Block scales_of(const convrot_kv_cache& c, const convrot_cache_rows& r)
{
    Block b(r.scales_dev, c.head_dim / kBlock, 1);
    b.add(c.pages, r.scale_page_stride, 1);
    b.add(c.heads, r.scale_head_stride, 1);
    b.add(c.page_size, r.scale_token_stride, 1);
    return b;
}

bool known_cache(const convrot_kv_cache& c)
{
    const bool quantized = cache_quantized(c.kind);
    if (!quantized && !half_type(c.kind)) return false;
    if (!within(c.pages, 1, 0x7fffffff) || !within(c.heads, 1, kMaxHeads)) return false;
    if (!within(c.page_size, 8, kMaxPageSize) || (c.page_size & (c.page_size - 1))) return false;
    if (!within(c.head_dim, 8, kMaxHeadWidth) || c.head_dim % (quantized ? kBlock : 8)) return false;
    for (const convrot_cache_rows* r : {&c.k, &c.v}) {
        if (!r->rows_dev || !aligned(r->rows_dev, 16)) return false;
        if ((r->page_stride | r->head_stride | r->token_stride) % 16) return false;
        if (!reaches(c.pages, r->page_stride) || !reaches(c.heads, r->head_stride) || !within(r->token_stride, 0, kMaxCacheTokenStride)) return false;
        if ((r->scales_dev != nullptr) != quantized) return false;
        if (quantized && (!reaches(c.pages, r->scale_page_stride) || !reaches(c.heads, r->scale_head_stride) ||
                          !within(r->scale_token_stride, 0, kMaxCacheTokenStride)))
            return false;
    }
    return true;
}

// Whether `out` is apart from everything that a cache holds.
bool apart_from(const convrot_kv_cache& c, const Block& out)
{
    for (const convrot_cache_rows* r : {&c.k, &c.v}) {
        if (!apart(rows_of(c, *r), out)) return false;
        if (r->scales_dev && !apart(scales_of(c, *r), out)) return false;
    }
    return true;
}

int check_cache_call(const convrot_cache_args* args, bool write)
{
    if (!args) return CONVROT_EINVAL;
    const convrot_cache_args& a = *args;
    if (!half_type(a.dtype) || (a.slots_dtype != CONVROT_I32 && a.slots_dtype != CONVROT_I64)) return CONVROT_EINVAL;
    if (!known_cache(a.cache) || (!cache_quantized(a.cache.kind) && a.cache.kind != a.dtype)) return CONVROT_EINVAL;
    if (!within(a.tokens, 0, kMaxRows)) return CONVROT_EINVAL;
    if (!reaches(a.tokens, a.k_token_stride) || !reaches(a.tokens, a.v_token_stride)) return CONVROT_EINVAL;
    if (!reaches(a.cache.heads, a.k_head_stride) || !reaches(a.cache.heads, a.v_head_stride)) return CONVROT_EINVAL;
    if (a.tokens == 0) return CONVROT_OK;
    const int slot_bytes = a.slots_dtype == CONVROT_I64 ? 8 : 4;
    if (!a.k_dev || !a.v_dev || !a.slots_dev) return CONVROT_EINVAL;
    if (!aligned(a.k_dev, 2) || !aligned(a.v_dev, 2) || !aligned(a.slots_dev, slot_bytes)) return CONVROT_EINVAL;
    const auto dense = [&](const void* at, int64_t token, int64_t head) {
        Block b(at, a.cache.head_dim, 2);
        b.add(a.tokens, token, 2);
        b.add(a.cache.heads, head, 2);
        return b;
    };
    const Block k = dense(a.k_dev, a.k_token_stride, a.k_head_stride), v = dense(a.v_dev, a.v_token_stride, a.v_head_stride);
    const Block slots(a.slots_dev, a.tokens, slot_bytes);
    if (!apart_from(a.cache, k) || !apart_from(a.cache, v)) return CONVROT_EINVAL;
    if (!write) return k.injective() && v.injective() && apart(k, v) && apart(slots, k) && apart(slots, v) ? CONVROT_OK : CONVROT_EINVAL;
    // what is written does not meet itself
    const convrot_kv_cache& c = a.cache;
    const Block parts[4] = {rows_of(c, c.k), rows_of(c, c.v), scales_of(c, c.k), scales_of(c, c.v)};
    const int count = cache_quantized(c.kind) ? 4 : 2;
    for (int i = 0; i < count; ++i) {
        if (!parts[i].injective() || !apart(slots, parts[i])) return CONVROT_EINVAL;
        for (int j = 0; j < i; ++j)
            if (!apart(parts[i], parts[j])) return CONVROT_EINVAL;
    }
    return CONVROT_OK;
}

struct PagedBlocks {
    Block q, o, lse, lengths, table;
    explicit PagedBlocks(const convrot_attention_paged_args& a)
        : q(heads(a, a.q_dev, a.q_batch_stride, a.q_head_stride)), o(heads(a, a.o_dev, a.o_batch_stride, a.o_head_stride)),
          lse(a.lse_dev, a.batch * a.q_heads, 4), lengths(a.lengths_dev, a.batch, 4), table(a.page_table_dev, a.table_width, 4)
    {
        table.add(a.batch, a.table_stride, 4);
    }
    static Block heads(const convrot_attention_paged_args& a, const void* at, int64_t batch, int64_t head)
    {
        Block b(at, a.cache.head_dim, 2);
        b.add(a.batch, batch, 2);
        b.add(a.q_heads, head, 2);
        return b;
    }
    // Whether `out` is apart from everything that the call reads.
    bool apart_from_inputs(const convrot_kv_cache& cache, const Block& out) const
    {
        return apart(q, out) && apart(lengths, out) && (!table.at || apart(table, out)) && apart_from(cache, out);
    }
};

// Everything but the workspace; *empty: nothing to do.
int check_paged(const convrot_attention_paged_args* args, bool* empty)
{
    *empty = false;
    if (!args) return CONVROT_EINVAL;
    const convrot_attention_paged_args& a = *args;
    if (!half_type(a.dtype) || a.reserved || !isfinite(a.scale * kLog2e)) return CONVROT_EINVAL;
    if (!known_cache(a.cache) || (!cache_quantized(a.cache.kind) && a.cache.kind != a.dtype)) return CONVROT_EINVAL;
    if (!within(a.batch, 0, kMaxBatch) || !within(a.q_heads, 1, kMaxHeads) || a.q_heads % a.cache.heads) return CONVROT_EINVAL;
    if (!within(a.table_width, 0, kMaxPlaces / a.cache.page_size) || !reaches(a.batch, a.table_stride)) return CONVROT_EINVAL;
    if (!reaches(a.batch, a.q_batch_stride) || !reaches(a.batch, a.o_batch_stride)) return CONVROT_EINVAL;
    if (!reaches(a.q_heads, a.q_head_stride) || !reaches(a.q_heads, a.o_head_stride)) return CONVROT_EINVAL;
    if (a.batch * (int64_t)paged_plan(a).columns > kMaxThreads / (64 * kPagedWavesAlone)) return CONVROT_EINVAL;
    if (a.batch == 0) {
        *empty = true;
        return CONVROT_OK;
    }
    if (!a.q_dev || !a.o_dev || !a.lengths_dev || (a.table_width && !a.page_table_dev)) return CONVROT_EINVAL;
    if (!aligned(a.q_dev, 2) || !aligned(a.o_dev, 2) || !aligned(a.lse_dev, 4)) return CONVROT_EINVAL;
    if (!aligned(a.lengths_dev, 4) || !aligned(a.page_table_dev, 4)) return CONVROT_EINVAL;
    const PagedBlocks b(a);
    if (!b.o.injective()) return CONVROT_EINVAL;
    for (const Block* out : {&b.o, &b.lse})
        if (out->at && !b.apart_from_inputs(a.cache, *out)) return CONVROT_EINVAL;
    return !b.lse.at || apart(b.o, b.lse) ? CONVROT_OK : CONVROT_EINVAL;
}

struct PromptBlocks {
    Block q, k, v, o, lse, q_starts, k_starts;
    explicit PromptBlocks(const convrot_attention_args& a)
        : q(rows(a, a.q_dev, a.q_tokens, a.q_heads, a.q_batch_stride, a.q_token_stride, a.q_head_stride)),
          k(rows(a, a.k_dev, a.k_tokens, a.k_heads, a.k_batch_stride, a.k_token_stride, a.k_head_stride)),
          v(rows(a, a.v_dev, a.k_tokens, a.k_heads, a.v_batch_stride, a.v_token_stride, a.v_head_stride)),
          o(rows(a, a.o_dev, a.q_tokens, a.q_heads, a.o_batch_stride, a.o_token_stride, a.o_head_stride)),
          lse(a.lse_dev, entries(a) * a.q_tokens * a.q_heads, 4), q_starts(a.q_starts_dev, a.batch + 1, 4),
          k_starts(a.k_starts_dev, a.batch + 1, 4)
    {
    }
    static int64_t entries(const convrot_attention_args& a) { return a.q_starts_dev ? 1 : a.batch; }
    static Block rows(const convrot_attention_args& a, const void* at, int64_t tokens, int heads, int64_t batch_s, int64_t token_s, int64_t head_s)
    {
        Block b(at, a.head_dim, 2);
        b.add(entries(a), batch_s, 2);
        b.add(tokens, token_s, 2);
        b.add(heads, head_s, 2);
        return b;
    }
    // Whether `out` is apart from everything that the call reads.
    bool apart_from_inputs(const convrot_attention_args& a, const Block& out) const
    {
        if (!apart(q, out) || (a.k_tokens && (!apart(k, out) || !apart(v, out)))) return false;
        return !q_starts.at || (apart(q_starts, out) && apart(k_starts, out));
    }
};

int check_prompt(const convrot_attention_args* args, bool* empty)
{
    *empty = false;
    if (!args) return CONVROT_EINVAL;
    const convrot_attention_args& a = *args;
    if (!half_type(a.dtype) || !within(a.causal, 0, 1) || !isfinite(a.scale * kLog2e)) return CONVROT_EINVAL;
    if (!within(a.batch, 0, kMaxBatch) || !within(a.q_tokens, 0, kMaxRows) || !within(a.k_tokens, 0, kMaxRows)) return CONVROT_EINVAL;
    if (!within(a.q_heads, 1, kMaxHeads) || !within(a.k_heads, 1, kMaxHeads) || a.q_heads % a.k_heads) return CONVROT_EINVAL;
    if (!within(a.head_dim, 8, kMaxHeadWidth) || a.head_dim % 8) return CONVROT_EINVAL;
    const bool packed = a.q_starts_dev != nullptr;
    if (packed != (a.k_starts_dev != nullptr)) return CONVROT_EINVAL;
    const int64_t entries = PromptBlocks::entries(a);
    for (int64_t s : {a.q_batch_stride, a.k_batch_stride, a.v_batch_stride, a.o_batch_stride})
        if (!reaches(entries, s)) return CONVROT_EINVAL;
    for (int64_t s : {a.q_token_stride, a.o_token_stride})
        if (!reaches(a.q_tokens, s)) return CONVROT_EINVAL;
    for (int64_t s : {a.k_token_stride, a.v_token_stride})
        if (!reaches(a.k_tokens, s) || s > kMaxTokenStride) return CONVROT_EINVAL;
    for (int64_t s : {a.q_head_stride, a.o_head_stride})
        if (!reaches(a.q_heads, s)) return CONVROT_EINVAL;
    for (int64_t s : {a.k_head_stride, a.v_head_stride})
        if (!reaches(a.k_heads, s)) return CONVROT_EINVAL;
    const PromptPlan plan = prompt_plan(a);
    if (plan.tiles * a.q_heads * plan.splits > kMaxThreads / (2 * kPromptRows)) return CONVROT_EINVAL;   // two threads a query
    if (a.batch == 0 || a.q_tokens == 0) {
        *empty = true;
        return CONVROT_OK;
    }
    if (!a.q_dev || !a.o_dev || (a.k_tokens && (!a.k_dev || !a.v_dev))) return CONVROT_EINVAL;
    for (const void* p : {a.q_dev, a.k_dev, a.v_dev, (const void*)a.o_dev})
        if (!aligned(p, 2)) return CONVROT_EINVAL;
    if (!aligned(a.lse_dev, 4) || !aligned(a.q_starts_dev, 4) || !aligned(a.k_starts_dev, 4)) return CONVROT_EINVAL;
    const PromptBlocks b(a);
    if (!b.o.injective()) return CONVROT_EINVAL;
    for (const Block* out : {&b.o, &b.lse})
        if (out->at && !b.apart_from_inputs(a, *out)) return CONVROT_EINVAL;
    return !b.lse.at || apart(b.o, b.lse) ? CONVROT_OK : CONVROT_EINVAL;
}

// need > 0
int check_workspace(const void* workspace, size_t have, int64_t need)
{
    if (!workspace || have < (size_t)need) return CONVROT_EWORKSPACE;
    return aligned(workspace, 16) ? CONVROT_OK : CONVROT_EINVAL;
}

}  // namespace

extern "C" {

int convrot_validate_cache_write(const convrot_cache_args* args) { return check_cache_call(args, true); }
int convrot_validate_cache_read(const convrot_cache_args* args) { return check_cache_call(args, false); }

int convrot_attention_paged_workspace_bytes(const convrot_attention_paged_args* args, size_t* bytes)
{
    bool empty;
    const int rc = check_paged(args, &empty);
    if (rc || !bytes) return CONVROT_EINVAL;
    *bytes = empty ? 0 : (size_t)paged_plan(*args).bytes();
    return CONVROT_OK;
}

int convrot_validate_attention_paged(const convrot_attention_paged_args* args, const void* workspace, size_t ws_bytes)
{
    bool empty;
    int rc = check_paged(args, &empty);
    const int64_t need = rc || empty ? 0 : paged_plan(*args).bytes();
    if (need == 0 || (rc = check_workspace(workspace, ws_bytes, need))) return rc;
    const PagedBlocks b(*args);
    const Block space(workspace, need, 1);
    return b.apart_from_inputs(args->cache, space) && apart(b.o, space) && (!b.lse.at || apart(b.lse, space)) ? CONVROT_OK : CONVROT_EINVAL;
}

int convrot_attention_workspace_bytes(const convrot_attention_args* args, size_t* bytes)
{
    bool empty;
    const int rc = check_prompt(args, &empty);
    if (rc || !bytes) return CONVROT_EINVAL;
    *bytes = empty ? 0 : (size_t)prompt_plan(*args).bytes(args->head_dim);
    return CONVROT_OK;
}

int convrot_validate_attention(const convrot_attention_args* args, const void* workspace, size_t ws_bytes)
{
    bool empty;
    int rc = check_prompt(args, &empty);
    const int64_t need = rc || empty ? 0 : prompt_plan(*args).bytes(args->head_dim);
    if (need == 0 || (rc = check_workspace(workspace, ws_bytes, need))) return rc;
    const PromptBlocks b(*args);
    const Block space(workspace, need, 1);
    return b.apart_from_inputs(*args, space) && apart(b.o, space) && (!b.lse.at || apart(b.lse, space)) ? CONVROT_OK : CONVROT_EINVAL;
}

}  // extern "C"
