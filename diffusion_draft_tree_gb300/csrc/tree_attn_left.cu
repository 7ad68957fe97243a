// tree_attn_left.cu -- ddtree_tree_attn_paged where pairs of query tiles take the few
// rows that the tiles leave over along (left_rows in tree_attn.cuh).
#include "tree_attn_paged.cuh"

namespace ddt {

cudaError_t launch_tree_attn_left(const PagedAttnArgs& a, cudaStream_t s) {
    const bool f16 = a.cache.dtype == 2;
    if (a.cache.D == 128)
        return f16 ? launch_mode<128, kLeftFp16>(a, s) : launch_mode<128, kLeftBf16>(a, s);
    return f16 ? launch_mode<64, kLeftFp16>(a, s) : launch_mode<64, kLeftBf16>(a, s);
}

}  // namespace ddt
