// C ABI of the paged cache's operators: argument validation and dispatch.
// Every check here runs before any launch; a failing call launches nothing.
#include "sbt_internal.cuh"

namespace {

// Messages are put together only where a check fails.
std::string say(const char* what, const char* text) { return std::string(what) + text; }

sbt_status check_dtype(sbt_dtype dtype, const char* what) {
    const int es = sbt_dtype_size(dtype);
    if (es != 2 && es != 4) return sbt_fail(SBT_ERR_UNSUPPORTED, say(what, ": unsupported dtype"));
    return SBT_OK;
}

sbt_status check_workspace(const void* ws, size_t bytes, size_t need, const char* what) {
    if (!ws || bytes < need)
        return sbt_fail(SBT_ERR_ALIGNMENT, say(what, ": workspace smaller than its size query"));
    if ((reinterpret_cast<uintptr_t>(ws) & 255u) != 0)
        return sbt_fail(SBT_ERR_ALIGNMENT, say(what, ": workspace must be 256-byte aligned"));
    return SBT_OK;
}

sbt_status check_map(const sbt_page_map* m, bool lens, bool refs, const char* what) {
    SBT_REQUIRE(m, say(what, ": map is NULL"));
    SBT_REQUIRE(m->n_seq >= 0 && m->max_pages >= 0 && m->n_pages >= 0, say(what, ": negative extent in the page map"));
    SBT_REQUIRE(m->n_pages < (1ll << 31), say(what, ": n_pages must be below 2^31"));
    SBT_REQUIRE(m->page_size >= 1, say(what, ": page_size must be at least 1"));
    SBT_REQUIRE(m->ld_table >= m->max_pages, say(what, ": ld_table < max_pages"));
    SBT_REQUIRE(m->n_seq == 0 || m->max_pages == 0 || m->page_table, say(what, ": page_table is NULL"));
    SBT_REQUIRE(!lens || m->n_seq == 0 || m->lens, say(what, ": lens is NULL"));
    SBT_REQUIRE(!refs || m->n_pages == 0 || m->refs, say(what, ": refs is NULL"));
    SBT_REQUIRE_ALIGNED(m->page_table, 4, say(what, ": page_table is not 4-byte aligned"));
    if (lens) SBT_REQUIRE_ALIGNED(m->lens, 4, say(what, ": lens is not 4-byte aligned"));
    if (refs) SBT_REQUIRE_ALIGNED(m->refs, 4, say(what, ": refs is not 4-byte aligned"));
    return SBT_OK;
}

// Strides of an array that is written: elements of different rows may not fall together.
bool apart(int64_t n, int64_t ld, int32_t dim) { return n <= 1 || ld >= dim; }

sbt_status check_cache(const sbt_kv_cache* c, const sbt_page_map* m, int es, const char* what) {
    SBT_REQUIRE(c, say(what, ": cache is NULL"));
    SBT_REQUIRE(c->heads >= 1 && c->head_dim >= 1, say(what, ": cache heads and head_dim must be positive"));
    SBT_REQUIRE(m->n_pages == 0 || (c->k && c->v), say(what, ": cache k or v is NULL"));
    SBT_REQUIRE(apart(m->n_pages, c->ld_page, c->head_dim) && apart(m->page_size, c->ld_slot, c->head_dim) &&
                    apart(c->heads, c->ld_head, c->head_dim) && c->ld_page >= 0 && c->ld_slot >= 0 && c->ld_head >= 0,
                say(what, ": cache stride smaller than head_dim"));
    SBT_REQUIRE_ALIGNED(c->k, es, say(what, ": cache k is not aligned to its element size"));
    SBT_REQUIRE_ALIGNED(c->v, es, say(what, ": cache v is not aligned to its element size"));
    return SBT_OK;
}

// A set of head rows that is read (or, with `write`, written).
sbt_status check_rows(const SbtHeadRows& r, int64_t tokens, int32_t heads, int32_t dim, int es, bool write,
                      const char* name, const char* what) {
    auto row = [&](const char* text) { return say(what, ": ") + name + text; };
    if (heads == 0) return SBT_OK;
    SBT_REQUIRE(r.p, row(" is NULL"));
    SBT_REQUIRE(r.ld >= 0 && r.ldh >= 0, row(" has a negative stride"));
    SBT_REQUIRE(!write || (apart(tokens, r.ld, dim) && apart(heads, r.ldh, dim)), row(" stride smaller than head_dim"));
    SBT_REQUIRE_ALIGNED(r.p, es, row(" is not aligned to its element size"));
    return SBT_OK;
}

// A launch has a block for every head of the queries, keys and values at most, and counts them in 32 bits.
sbt_status check_heads(int64_t tokens, int32_t q_heads, int32_t k_heads, const char* what) {
    SBT_REQUIRE(tokens >= 0 && q_heads >= 0 && k_heads >= 0, say(what, ": negative extent"));
    SBT_REQUIRE((int64_t)q_heads + 2 * (int64_t)k_heads <= 1 << 30, say(what, ": q_heads + 2 k_heads too large"));
    return SBT_OK;
}

sbt_status check_rope(const sbt_rope* r, int32_t head_dim, const char* what) {
    if (!r || r->rot_dim == 0) return SBT_OK;
    SBT_REQUIRE(r->rot_dim > 0 && r->rot_dim % 2 == 0 && r->rot_dim <= head_dim,
                say(what, ": rot_dim must be even and at most head_dim"));
    if (r->layout != SBT_ROPE_HALF && r->layout != SBT_ROPE_INTERLEAVED)
        return sbt_fail(SBT_ERR_UNSUPPORTED, say(what, ": unknown rotation layout"));
    SBT_REQUIRE(r->n_pos >= 0 && (r->n_pos == 0 || r->table), say(what, ": rotation table is NULL"));
    SBT_REQUIRE_ALIGNED(r->table, 8, say(what, ": rotation table is not 8-byte aligned"));
    return SBT_OK;
}

sbt_status check_pools(const sbt_page_pool* pools, int32_t n, int64_t n_pages, const char* what) {
    SBT_REQUIRE(n >= 1 && n <= SBT_MAX_PAGE_POOLS && pools, say(what, ": between 1 and SBT_MAX_PAGE_POOLS pools"));
    for (int32_t i = 0; i < n; ++i) {
        const sbt_page_pool& q = pools[i];
        SBT_REQUIRE(q.n_planes >= 1 && q.n_planes < (1ll << 31) && q.page_bytes >= 1,
                    say(what, ": pool planes and page_bytes must be positive"));
        SBT_REQUIRE(q.page_bytes < (1ll << 40), say(what, ": page_bytes too large"));
        SBT_REQUIRE((n_pages <= 1 || q.page_stride >= q.page_bytes) &&
                        (q.n_planes == 1 || q.plane_stride >= q.page_bytes),
                    say(what, ": pool stride smaller than page_bytes"));
        SBT_REQUIRE(n_pages == 0 || q.base, say(what, ": pool base is NULL"));
    }
    return SBT_OK;
}

}  // namespace

#define SBT_TRY(call)                   \
    do {                                \
        const sbt_status st_ = (call);  \
        if (st_) return st_;            \
    } while (0)

extern "C" {

sbt_status sbt_paged_attention_workspace_size(sbt_context* ctx, int32_t q_heads, int32_t kv_heads, int32_t head_dim,
                                              size_t* bytes) {
    SBT_REQUIRE(ctx && bytes, "paged_attention_workspace_size: NULL argument");
    SBT_REQUIRE(kv_heads >= 1 && q_heads >= 1 && q_heads % kv_heads == 0,
                "paged_attention_workspace_size: kv_heads must divide q_heads");
    SBT_REQUIRE(head_dim >= 1 && head_dim <= 256, "paged_attention_workspace_size: head_dim must be in [1, 256]");
    *bytes = sbt_paged_attention_workspace_bytes(ctx, q_heads, kv_heads, head_dim);
    return SBT_OK;
}

sbt_status sbt_paged_attention(sbt_context* ctx, sbt_dtype dtype, const void* q, int64_t ld_q, int64_t ld_qh,
                               int32_t batch, int32_t q_heads, const sbt_kv_cache* cache, const sbt_page_map* map,
                               const int32_t* seq, float scale, int32_t window, void* out, int64_t ld_out,
                               int64_t ld_oh, float* lse, void* workspace, size_t workspace_bytes, void* stream) {
    const char* const w = "paged_attention";
    SBT_REQUIRE(ctx, "ctx is NULL");
    SBT_TRY(check_dtype(dtype, w));
    const int es = sbt_dtype_size(dtype);
    SBT_TRY(check_map(map, true, false, w));
    SBT_TRY(check_cache(cache, map, es, w));
    SBT_REQUIRE(cache->head_dim <= 256, "paged_attention: head_dim must be in [1, 256]");
    SBT_REQUIRE(batch >= 0, "paged_attention: negative batch");
    SBT_REQUIRE(q_heads >= 1 && q_heads % cache->heads == 0, "paged_attention: the cache's heads must divide q_heads");
    SBT_REQUIRE((int64_t)q_heads * cache->head_dim < (1ll << 31), "paged_attention: q_heads * head_dim too large");
    SBT_REQUIRE(window >= 0, "paged_attention: negative window");
    if (batch == 0) return SBT_OK;
    const SbtHeadRows rq = {q, ld_q, ld_qh}, ro = {out, ld_out, ld_oh};
    SBT_TRY(check_rows(rq, batch, q_heads, cache->head_dim, es, false, "q", w));
    SBT_TRY(check_rows(ro, batch, q_heads, cache->head_dim, es, true, "out", w));
    SBT_REQUIRE_ALIGNED(seq, 4, "paged_attention: seq is not 4-byte aligned");
    SBT_REQUIRE_ALIGNED(lse, 4, "paged_attention: lse is not 4-byte aligned");
    SBT_TRY(check_workspace(workspace, workspace_bytes,
                            sbt_paged_attention_workspace_bytes(ctx, q_heads, cache->heads, cache->head_dim), w));
    SBT_TRY(sbt_use_device(ctx));
    return sbt_launch_paged_attention(ctx, dtype, rq, batch, q_heads, cache, map, seq, scale, window, ro, lse,
                                      workspace, (cudaStream_t)stream);
}

sbt_status sbt_rope_table(sbt_context* ctx, float* table, int64_t n_pos, int32_t rot_dim, double base,
                          sbt_rope_scaling scaling, double factor, int64_t orig_len, double low, double high,
                          double amplitude, void* stream) {
    SBT_REQUIRE(ctx, "ctx is NULL");
    if (scaling < SBT_ROPE_NONE || scaling > SBT_ROPE_BY_PARTS)
        return sbt_fail(SBT_ERR_UNSUPPORTED, "rope_table: unknown scaling");
    SBT_REQUIRE(n_pos >= 0 && n_pos < (1ll << 40), "rope_table: n_pos out of range");
    SBT_REQUIRE(rot_dim >= 0 && rot_dim % 2 == 0, "rope_table: rot_dim must be even");
    SBT_REQUIRE(rot_dim < 2 || n_pos <= (1ll << 40) / (rot_dim / 2), "rope_table: table too large");
    SBT_REQUIRE(base > 0.0 && factor > 0.0, "rope_table: base and factor must be positive");
    SBT_REQUIRE(scaling != SBT_ROPE_BY_PARTS || (high > low && orig_len > 0),
                "rope_table: scaling by parts needs high > low and orig_len > 0");
    if (n_pos == 0 || rot_dim == 0) return SBT_OK;
    SBT_REQUIRE(table, "rope_table: table is NULL");
    SBT_REQUIRE_ALIGNED(table, 8, "rope_table: table is not 8-byte aligned");
    SBT_TRY(sbt_use_device(ctx));
    return sbt_launch_rope_table(ctx, table, n_pos, rot_dim, base, (int)scaling, factor, orig_len, low, high,
                                 amplitude, (cudaStream_t)stream);
}

sbt_status sbt_qk_norm_rope(sbt_context* ctx, sbt_dtype dtype, const void* q, int64_t ld_q, int64_t ld_qh,
                            const void* k, int64_t ld_k, int64_t ld_kh, int64_t tokens, int32_t q_heads,
                            int32_t k_heads, int32_t head_dim, const int32_t* positions, const sbt_rope* rope,
                            const void* q_weight, const void* k_weight, float eps, void* q_out, int64_t ld_qo,
                            int64_t ld_qoh, void* k_out, int64_t ld_ko, int64_t ld_koh, const void* v, int64_t ld_v,
                            int64_t ld_vh, const sbt_kv_cache* cache, const sbt_page_map* map, const int32_t* seq,
                            void* stream) {
    const char* const w = "qk_norm_rope";
    SBT_REQUIRE(ctx, "ctx is NULL");
    SBT_TRY(check_dtype(dtype, w));
    const int es = sbt_dtype_size(dtype);
    SBT_TRY(check_heads(tokens, q_heads, k_heads, w));
    SBT_REQUIRE(head_dim >= 1 && head_dim <= 512, "qk_norm_rope: head_dim must be in [1, 512]");
    SBT_TRY(check_rope(rope, head_dim, w));
    SBT_REQUIRE(eps >= 0.f, "qk_norm_rope: negative eps");
    if (cache) {
        SBT_TRY(check_map(map, false, false, w));
        SBT_TRY(check_cache(cache, map, es, w));
        SBT_REQUIRE(cache->heads == k_heads && cache->head_dim == head_dim,
                    "qk_norm_rope: the cache's heads and head_dim must be those of the keys");
    }
    SBT_REQUIRE(cache || !v, "qk_norm_rope: v without a cache");
    SBT_REQUIRE(cache || k_heads == 0 || k_out, "qk_norm_rope: k_out is NULL and there is no cache");
    if (tokens == 0 || q_heads + k_heads == 0) return SBT_OK;
    const SbtHeadRows rq = {q_heads ? q : nullptr, ld_q, ld_qh}, rk = {k_heads ? k : nullptr, ld_k, ld_kh};
    const SbtHeadRows rv = {k_heads ? v : nullptr, ld_v, ld_vh};
    const SbtHeadRows rqo = {q_heads ? q_out : nullptr, ld_qo, ld_qoh}, rko = {k_heads ? k_out : nullptr, ld_ko, ld_koh};
    SBT_TRY(check_rows(rq, tokens, q_heads, head_dim, es, false, "q", w));
    SBT_TRY(check_rows(rk, tokens, k_heads, head_dim, es, false, "k", w));
    SBT_TRY(check_rows(rqo, tokens, q_heads, head_dim, es, true, "q_out", w));
    if (rko.p) SBT_TRY(check_rows(rko, tokens, k_heads, head_dim, es, true, "k_out", w));
    if (rv.p) SBT_TRY(check_rows(rv, tokens, k_heads, head_dim, es, false, "v", w));
    SBT_REQUIRE(positions, "qk_norm_rope: positions is NULL");
    SBT_REQUIRE_ALIGNED(positions, 4, "qk_norm_rope: positions is not 4-byte aligned");
    SBT_REQUIRE_ALIGNED(seq, 4, "qk_norm_rope: seq is not 4-byte aligned");
    SBT_REQUIRE_ALIGNED(q_weight, es, "qk_norm_rope: q_weight is not aligned to its element size");
    SBT_REQUIRE_ALIGNED(k_weight, es, "qk_norm_rope: k_weight is not aligned to its element size");
    SBT_TRY(sbt_use_device(ctx));
    return sbt_launch_norm_rope(ctx, dtype, rq, rk, rv, rqo, rko, tokens, q_heads, k_heads, head_dim, positions, rope,
                                q_weight, k_weight, eps, k_heads ? cache : nullptr, map, seq, (cudaStream_t)stream);
}

sbt_status sbt_qk_norm_rope_backward_workspace_size(sbt_context* ctx, int32_t head_dim, size_t* bytes) {
    SBT_REQUIRE(ctx && bytes, "qk_norm_rope_backward_workspace_size: NULL argument");
    SBT_REQUIRE(head_dim >= 1 && head_dim <= 512,
                "qk_norm_rope_backward_workspace_size: head_dim must be in [1, 512]");
    *bytes = (size_t)sbt_norm_rope_bwd_blocks(ctx) * head_dim * sizeof(float);
    return SBT_OK;
}

sbt_status sbt_qk_norm_rope_backward(sbt_context* ctx, sbt_dtype dtype, const void* gq, int64_t ld_gq, int64_t ld_gqh,
                                     const void* gk, int64_t ld_gk, int64_t ld_gkh, const void* q, int64_t ld_q,
                                     int64_t ld_qh, const void* k, int64_t ld_k, int64_t ld_kh, int64_t tokens,
                                     int32_t q_heads, int32_t k_heads, int32_t head_dim, const int32_t* positions,
                                     const sbt_rope* rope, const void* q_weight, const void* k_weight, float eps,
                                     void* dq, int64_t ld_dq, int64_t ld_dqh, void* dk, int64_t ld_dk, int64_t ld_dkh,
                                     float* dq_weight, float* dk_weight, void* workspace, size_t workspace_bytes,
                                     void* stream) {
    const char* const w = "qk_norm_rope_backward";
    SBT_REQUIRE(ctx, "ctx is NULL");
    SBT_TRY(check_dtype(dtype, w));
    const int es = sbt_dtype_size(dtype);
    SBT_TRY(check_heads(tokens, q_heads, k_heads, w));
    SBT_REQUIRE(head_dim >= 1 && head_dim <= 512, "qk_norm_rope_backward: head_dim must be in [1, 512]");
    SBT_TRY(check_rope(rope, head_dim, w));
    SBT_REQUIRE(eps >= 0.f, "qk_norm_rope_backward: negative eps");
    SBT_REQUIRE(!q_weight == !dq_weight && !k_weight == !dk_weight,
                "qk_norm_rope_backward: a weight's gradient is required exactly where the weight is given");
    if ((tokens == 0 || q_heads + k_heads == 0) && !dq_weight && !dk_weight) return SBT_OK;
    if (tokens > 0) {
        SBT_TRY(check_rows({gq, ld_gq, ld_gqh}, tokens, q_heads, head_dim, es, false, "gq", w));
        SBT_TRY(check_rows({gk, ld_gk, ld_gkh}, tokens, k_heads, head_dim, es, false, "gk", w));
        if (q_weight) SBT_TRY(check_rows({q, ld_q, ld_qh}, tokens, q_heads, head_dim, es, false, "q", w));
        if (k_weight) SBT_TRY(check_rows({k, ld_k, ld_kh}, tokens, k_heads, head_dim, es, false, "k", w));
        SBT_TRY(check_rows({dq, ld_dq, ld_dqh}, tokens, q_heads, head_dim, es, true, "dq", w));
        SBT_TRY(check_rows({dk, ld_dk, ld_dkh}, tokens, k_heads, head_dim, es, true, "dk", w));
        SBT_REQUIRE(q_heads + k_heads == 0 || positions, "qk_norm_rope_backward: positions is NULL");
    }
    SBT_REQUIRE_ALIGNED(positions, 4, "qk_norm_rope_backward: positions is not 4-byte aligned");
    SBT_REQUIRE_ALIGNED(q_weight, es, "qk_norm_rope_backward: q_weight is not aligned to its element size");
    SBT_REQUIRE_ALIGNED(k_weight, es, "qk_norm_rope_backward: k_weight is not aligned to its element size");
    SBT_REQUIRE_ALIGNED(dq_weight, 4, "qk_norm_rope_backward: dq_weight is not 4-byte aligned");
    SBT_REQUIRE_ALIGNED(dk_weight, 4, "qk_norm_rope_backward: dk_weight is not 4-byte aligned");
    if (dq_weight || dk_weight) {
        size_t need = 0;
        SBT_TRY(sbt_qk_norm_rope_backward_workspace_size(ctx, head_dim, &need));
        SBT_TRY(check_workspace(workspace, workspace_bytes, need, w));
    }
    SBT_TRY(sbt_use_device(ctx));
    // an absent side has no rows
    const SbtHeadRows none = {nullptr, 0, 0};
    const bool hq = q_heads && tokens, hk = k_heads && tokens;
    return sbt_launch_norm_rope_bwd(ctx, dtype, hq ? SbtHeadRows{gq, ld_gq, ld_gqh} : none,
                                    hk ? SbtHeadRows{gk, ld_gk, ld_gkh} : none,
                                    hq && q_weight ? SbtHeadRows{q, ld_q, ld_qh} : none,
                                    hk && k_weight ? SbtHeadRows{k, ld_k, ld_kh} : none,
                                    hq ? SbtHeadRows{dq, ld_dq, ld_dqh} : none,
                                    hk ? SbtHeadRows{dk, ld_dk, ld_dkh} : none, tokens, q_heads, k_heads, head_dim,
                                    positions, rope, q_weight, k_weight, eps, dq_weight, dk_weight, workspace,
                                    (cudaStream_t)stream);
}

sbt_status sbt_pages_workspace_size(sbt_context* ctx, int32_t n_seq, int64_t n_pages, size_t* bytes) {
    SBT_REQUIRE(ctx && bytes, "pages_workspace_size: NULL argument");
    SBT_REQUIRE(n_seq >= 0 && n_pages >= 0 && n_pages < (1ll << 31), "pages_workspace_size: extent out of range");
    *bytes = sbt_pages_workspace_bytes(n_seq, n_pages);
    return SBT_OK;
}

sbt_status sbt_pages_copy(sbt_context* ctx, const sbt_page_pool* pools, int32_t n_pools, int64_t n_pages,
                          const int32_t* src, const int32_t* dst, int64_t n, void* stream) {
    SBT_REQUIRE(ctx, "ctx is NULL");
    SBT_REQUIRE(n >= 0 && n < (1ll << 40), "pages_copy: n out of range");
    SBT_REQUIRE(n_pages >= 0 && n_pages < (1ll << 31), "pages_copy: n_pages out of range");
    SBT_TRY(check_pools(pools, n_pools, n_pages, "pages_copy"));
    if (n == 0 || n_pages == 0) return SBT_OK;
    SBT_REQUIRE(src && dst, "pages_copy: NULL src or dst");
    SBT_REQUIRE_ALIGNED(src, 4, "pages_copy: src is not 4-byte aligned");
    SBT_REQUIRE_ALIGNED(dst, 4, "pages_copy: dst is not 4-byte aligned");
    SBT_TRY(sbt_use_device(ctx));
    return sbt_launch_pages_copy(ctx, pools, n_pools, n_pages, src, dst, n, (cudaStream_t)stream);
}

sbt_status sbt_pages_reserve(sbt_context* ctx, const sbt_page_map* map, const sbt_page_pool* pools, int32_t n_pools,
                             const int32_t* target, void* workspace, size_t workspace_bytes, void* stream) {
    SBT_REQUIRE(ctx, "ctx is NULL");
    SBT_TRY(check_map(map, true, true, "pages_reserve"));
    SBT_TRY(check_pools(pools, n_pools, map->n_pages, "pages_reserve"));
    if (map->n_seq == 0) return SBT_OK;
    SBT_REQUIRE(target, "pages_reserve: target is NULL");
    SBT_REQUIRE_ALIGNED(target, 4, "pages_reserve: target is not 4-byte aligned");
    SBT_TRY(check_workspace(workspace, workspace_bytes, sbt_pages_workspace_bytes(map->n_seq, map->n_pages),
                            "pages_reserve"));
    SBT_TRY(sbt_use_device(ctx));
    return sbt_launch_pages_reserve(ctx, map, pools, n_pools, target, workspace, (cudaStream_t)stream);
}

sbt_status sbt_pages_fork(sbt_context* ctx, const sbt_page_map* map, const sbt_page_pool* pools, int32_t n_pools,
                          const int32_t* from, const int32_t* to, int32_t n, void* workspace, size_t workspace_bytes,
                          void* stream) {
    SBT_REQUIRE(ctx, "ctx is NULL");
    SBT_TRY(check_map(map, true, true, "pages_fork"));
    SBT_TRY(check_pools(pools, n_pools, map->n_pages, "pages_fork"));
    SBT_REQUIRE(n >= 0 && n <= map->n_seq, "pages_fork: n must be in [0, n_seq]");
    if (n == 0) return SBT_OK;
    SBT_REQUIRE(from && to, "pages_fork: NULL from or to");
    SBT_REQUIRE_ALIGNED(from, 4, "pages_fork: from is not 4-byte aligned");
    SBT_REQUIRE_ALIGNED(to, 4, "pages_fork: to is not 4-byte aligned");
    SBT_TRY(check_workspace(workspace, workspace_bytes, sbt_pages_workspace_bytes(map->n_seq, map->n_pages),
                            "pages_fork"));
    SBT_TRY(sbt_use_device(ctx));
    return sbt_launch_pages_fork(ctx, map, pools, n_pools, from, to, n, workspace, (cudaStream_t)stream);
}

sbt_status sbt_pages_free(sbt_context* ctx, const sbt_page_map* map, const int32_t* seqs, const int32_t* keep,
                          int32_t n, void* stream) {
    SBT_REQUIRE(ctx, "ctx is NULL");
    SBT_TRY(check_map(map, true, true, "pages_free"));
    SBT_REQUIRE(n >= 0, "pages_free: negative n");
    if (n == 0 || map->n_seq == 0) return SBT_OK;
    SBT_REQUIRE(seqs, "pages_free: seqs is NULL");
    SBT_REQUIRE_ALIGNED(seqs, 4, "pages_free: seqs is not 4-byte aligned");
    SBT_REQUIRE_ALIGNED(keep, 4, "pages_free: keep is not 4-byte aligned");
    SBT_TRY(sbt_use_device(ctx));
    return sbt_launch_pages_free(ctx, map, seqs, keep, n, (cudaStream_t)stream);
}

sbt_status sbt_pages_compact(sbt_context* ctx, const sbt_page_map* map, const sbt_page_pool* pools, int32_t n_pools,
                             int32_t* table_out, int64_t ld_out, int32_t* refs_out, int32_t* page_to, int32_t* n_live,
                             void* workspace, size_t workspace_bytes, void* stream) {
    SBT_REQUIRE(ctx, "ctx is NULL");
    SBT_TRY(check_map(map, true, true, "pages_compact"));
    SBT_TRY(check_pools(pools, n_pools, map->n_pages, "pages_compact"));
    SBT_REQUIRE(map->n_pages == 0 || (refs_out && page_to), "pages_compact: NULL refs_out or page_to");
    SBT_REQUIRE(n_live, "pages_compact: n_live is NULL");
    SBT_REQUIRE(map->n_seq == 0 || map->max_pages == 0 || table_out, "pages_compact: table_out is NULL");
    SBT_REQUIRE(ld_out >= map->max_pages, "pages_compact: ld_out < max_pages");
    SBT_REQUIRE(table_out != map->page_table || ld_out == map->ld_table,
                "pages_compact: table_out aliasing the table needs ld_out == ld_table");
    SBT_REQUIRE_ALIGNED(table_out, 4, "pages_compact: table_out is not 4-byte aligned");
    SBT_REQUIRE_ALIGNED(refs_out, 4, "pages_compact: refs_out is not 4-byte aligned");
    SBT_REQUIRE_ALIGNED(page_to, 4, "pages_compact: page_to is not 4-byte aligned");
    SBT_REQUIRE_ALIGNED(n_live, 4, "pages_compact: n_live is not 4-byte aligned");
    SBT_TRY(check_workspace(workspace, workspace_bytes, sbt_pages_workspace_bytes(map->n_seq, map->n_pages),
                            "pages_compact"));
    SBT_TRY(sbt_use_device(ctx));
    return sbt_launch_pages_compact(ctx, map, pools, n_pools, table_out, ld_out, refs_out, page_to, n_live, workspace,
                                    (cudaStream_t)stream);
}

}  // extern "C"
