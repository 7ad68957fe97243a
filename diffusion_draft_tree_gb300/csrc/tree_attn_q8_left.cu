// tree_attn_q8_left.cu -- ddtree_tree_attn_q8 where pairs of query tiles take the few rows that
// the tiles leave over along (left_rows in tree_attn.cuh).
#include "tree_attn_paged.cuh"

namespace ddt {

cudaError_t launch_tree_attn_q8_left(const Q8AttnArgs& a, cudaStream_t s) {
    const bool f16 = a.cache.dtype == 2;
    if (a.cache.D == 128) return f16 ? launch_mode<128, kQ8LeftFp16>(a, s) : launch_mode<128, kQ8LeftBf16>(a, s);
    return f16 ? launch_mode<64, kQ8LeftFp16>(a, s) : launch_mode<64, kQ8LeftBf16>(a, s);
}

}  // namespace ddt
