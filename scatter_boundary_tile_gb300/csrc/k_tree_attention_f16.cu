// Attention of several new tokens, f16, head sizes to 128.
#include "k_tree_attention.cuh"

namespace sbt_tree {

template <>
sbt_status narrow<kF16>(sbt_context* ctx, TreeAttnParams& p, const TreeMaps& maps, bool two, void* ws,
                         cudaStream_t stream) {
    if (p.head_dim <= 64) return two ? enqueue<kF16, 64, 2>(ctx, p, maps, ws, stream) : enqueue<kF16, 64, 1>(ctx, p, maps, ws, stream);
    return two ? enqueue<kF16, 128, 2>(ctx, p, maps, ws, stream) : enqueue<kF16, 128, 1>(ctx, p, maps, ws, stream);
}

}  // namespace sbt_tree
