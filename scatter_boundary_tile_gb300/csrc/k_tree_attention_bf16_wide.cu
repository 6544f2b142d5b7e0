// Attention of several new tokens, bf16, head sizes from 129 to 256.
#include "k_tree_attention.cuh"

namespace sbt_tree {

template <>
sbt_status wide<kBF16>(sbt_context* ctx, TreeAttnParams& p, const TreeMaps& maps, void* ws, cudaStream_t stream) {
    return p.head_dim <= 192 ? enqueue<kBF16, 192, 1>(ctx, p, maps, ws, stream) : enqueue<kBF16, 256, 1>(ctx, p, maps, ws, stream);
}

}  // namespace sbt_tree
