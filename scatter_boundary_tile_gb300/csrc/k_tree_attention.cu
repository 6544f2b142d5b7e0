// Attention of several new tokens: which kernel, and its workspace.
#include "k_tree_attention.cuh"

using namespace sbt_tree;

namespace {

int padded(int32_t head_dim) { return head_dim <= 64 ? 64 : head_dim <= 128 ? 128 : head_dim <= 192 ? 192 : 256; }
// 256 rows a block where that many may come and their sums fit TMEM twice.
bool two_tiles(int64_t rows, int dp) { return rows > kRows && dp <= 128; }

// Widest piece that rows start on and consist of.
int piece(const void* a, int64_t ld0, int64_t ld1, int64_t ld2, int32_t head_dim) {
    const uint64_t x = (uintptr_t)a | (uint64_t)(ld0 * 2) | (uint64_t)(ld1 * 2) | (uint64_t)(ld2 * 2) | (uint64_t)(head_dim * 2);
    return x % 16 == 0 ? 16 : x % 8 == 0 ? 8 : x % 4 == 0 ? 4 : 2;
}

// The tensor copy engine takes the pages where they hold whole boxes (8, 16, 32 or a multiple of 64 positions), every
// stride and address is a multiple of 16 bytes, and the driver makes both maps; lanes copy them otherwise.
bool map_ok(const sbt_context* ctx, const sbt_kv_cache* c, const sbt_page_map* m) {
    const int32_t P = m->page_size;
    if (ctx->path == SBT_PATH_SCALAR || ctx->path == SBT_PATH_VECTOR) return false;
    if (!(P == 8 || P == 16 || P == 32 || P % kTok == 0) || m->n_pages == 0) return false;
    auto stride = [](int64_t n, int64_t ld) { return n == 1 || (ld % 8 == 0 && ld > 0 && ld < (1ll << 39)); };
    return sbt_aligned16(c->k) && sbt_aligned16(c->v) && stride(P, c->ld_slot) && stride(c->heads, c->ld_head) &&
           stride(m->n_pages, c->ld_page);
}

bool encode(sbt_context* ctx, CUtensorMap* map, const void* base, const sbt_kv_cache* c, const sbt_page_map* m) {
    auto bytes = [](int64_t n, int64_t ld) { return (cuuint64_t)(n == 1 ? 16 : ld * 2); };
    const cuuint64_t dims[4] = {(cuuint64_t)c->head_dim, (cuuint64_t)m->page_size, (cuuint64_t)c->heads,
                                (cuuint64_t)m->n_pages};
    const cuuint64_t strides[3] = {bytes(m->page_size, c->ld_slot), bytes(c->heads, c->ld_head), bytes(m->n_pages, c->ld_page)};
    const cuuint32_t box[4] = {64, (cuuint32_t)std::min(m->page_size, kTok), 1, 1}, step[4] = {1, 1, 1, 1};
    return ctx->encode_tiled(map, CU_TENSOR_MAP_DATA_TYPE_UINT16, 4, const_cast<void*>(base), dims, strides, box, step,
                             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

// For two blocks of 128 rows an SM or one of 256, whose parts take the same room: a workspace serves any max_new.
size_t sbt_tree_attention_workspace_bytes(const sbt_context* ctx, int32_t head_dim) {
    const int64_t blocks = 2 * (int64_t)ctx->sm_count;
    return (size_t)(sbt_cdiv(blocks * sizeof(TreeDesc), 256) * 256 +
                    2 * blocks * kRows * (sizeof(float2) + padded(head_dim) * sizeof(float)));
}

sbt_status sbt_launch_tree_attention(sbt_context* ctx, sbt_dtype dtype, const SbtHeadRows& q, int32_t rows,
                                     const int32_t* cu, int32_t batch, int32_t max_new, int32_t q_heads,
                                     const sbt_kv_cache* cache, const sbt_page_map* map, const int32_t* seq,
                                     float scale, const int32_t* mask, int64_t ld_mask, const SbtHeadRows& out,
                                     float* lse, void* workspace, cudaStream_t stream) {
    TreeAttnParams p = {};
    p.q = (const char*)q.p, p.ld_q = q.ld, p.ld_qh = q.ldh;
    p.k = (const char*)cache->k, p.v = (const char*)cache->v;
    p.ld_page = cache->ld_page, p.ld_slot = cache->ld_slot, p.ld_head = cache->ld_head;
    p.out = (char*)const_cast<void*>(out.p), p.ld_out = out.ld, p.ld_oh = out.ldh, p.lse = lse;
    p.cu = cu, p.table = map->page_table, p.lens = map->lens, p.seq = seq;
    p.ld_table = map->ld_table, p.n_pages = map->n_pages, p.n_seq = map->n_seq;
    p.mask = (const uint32_t*)mask, p.ld_mask = ld_mask;
    p.rows = rows, p.batch = batch, p.max_new = max_new;
    p.q_heads = q_heads, p.kv_heads = cache->heads, p.head_dim = cache->head_dim;
    p.max_len = (int32_t)std::min<int64_t>((int64_t)map->max_pages * map->page_size, INT32_MAX - 1023);
    p.group = sbt_make_fastdiv((uint32_t)(q_heads / cache->heads));
    p.page_size = sbt_make_fastdiv((uint32_t)map->page_size);
    // (a scale of zero would make NaN of a masked score of minus infinity; 2^-149 of any finite one is 2^-21 at most)
    p.scale = std::max(fabsf(scale) * 1.4426950408889634f, 0x1p-149f), p.negate = scale < 0.f;
    p.q_vec = piece(q.p, q.ld, q.ldh, 0, p.head_dim) == 16;
    p.copy_kv = std::min(piece(p.k, p.ld_page, p.ld_slot, p.ld_head, p.head_dim), piece(p.v, 0, 0, 0, p.head_dim));
    p.out_vec = piece(out.p, out.ld, out.ldh, 0, p.head_dim) == 16;
    p.status = ctx->status, p.wait_ns = ctx->wait_limit_ns;
    p.withhold = ctx->test_hook == SBT_TEST_WITHHOLD_LOAD;
    TreeMaps maps = {};
    maps.use = map_ok(ctx, cache, map) && encode(ctx, &maps.k, cache->k, cache, map) && encode(ctx, &maps.v, cache->v, cache, map);
    const int dp = padded(p.head_dim);
    if (dp > 128)
        return dtype == SBT_BF16 ? wide<kBF16>(ctx, p, maps, workspace, stream) : wide<kF16>(ctx, p, maps, workspace, stream);
    const bool two = two_tiles((int64_t)p.max_new * p.group.d, dp);
    return dtype == SBT_BF16 ? narrow<kBF16>(ctx, p, maps, two, workspace, stream)
                             : narrow<kF16>(ctx, p, maps, two, workspace, stream);
}
