// Attention of several new tokens, bf16, head sizes to 128.
#include "k_tree_attention.cuh"

namespace sbt_tree {

template <>
sbt_status narrow<kBF16>(sbt_context* ctx, TreeAttnParams& p, const TreeMaps& maps, bool two, void* ws,
                         cudaStream_t stream) {
    if (p.head_dim <= 64) return two ? enqueue<kBF16, 64, 2>(ctx, p, maps, ws, stream) : enqueue<kBF16, 64, 1>(ctx, p, maps, ws, stream);
    return two ? enqueue<kBF16, 128, 2>(ctx, p, maps, ws, stream) : enqueue<kBF16, 128, 1>(ctx, p, maps, ws, stream);
}

}  // namespace sbt_tree
