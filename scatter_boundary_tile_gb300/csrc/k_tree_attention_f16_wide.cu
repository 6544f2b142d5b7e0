// Attention of several new tokens, f16, head sizes from 129 to 256.
#include "k_tree_attention.cuh"

namespace sbt_tree {

template <>
sbt_status wide<kF16>(sbt_context* ctx, TreeAttnParams& p, const TreeMaps& maps, void* ws, cudaStream_t stream) {
    return p.head_dim <= 192 ? enqueue<kF16, 192, 1>(ctx, p, maps, ws, stream) : enqueue<kF16, 256, 1>(ctx, p, maps, ws, stream);
}

}  // namespace sbt_tree
