// tree_attn_q8.cu -- ddtree_tree_attn_q8: the tree-attention kernel (tree_attn.cuh) over an
// 8-bit paged cache.
#include "tree_attn_paged.cuh"

namespace ddt {

size_t q8_attn_workspace_bytes(int B, int N, int Hq, int Hkv, int D, int64_t cache_cap) {
    if (q8_few_rows(B, N, Hq, Hkv, cache_cap)) return few_rows_workspace_bytes(N, Hq, Hkv, D);
    const ManyPlan pl = plan_paged_many(B, N, Hq, Hkv, max_tiles(N, cache_cap), num_sms(), true);
    return pl.smax ? attn_layout(pl, B, Hkv, D, 4, pl.left).total : 0;
}

cudaError_t launch_tree_attn_q8(const Q8AttnArgs& a, cudaStream_t s) {
    const int64_t cap = (int64_t)a.cache.max_pages * a.cache.page_size;
    if (q8_few_rows(a.B, a.N, a.q.heads, a.cache.Hkv, cap)) return launch_tree_attn_q8_rows(a, s);
    if (plan_paged_many(a.B, a.N, a.q.heads, a.cache.Hkv, max_tiles(a.N, cap), num_sms(), true).left)
        return launch_tree_attn_q8_left(a, s);
    const bool f16 = a.cache.dtype == 2;
    if (a.cache.D == 128) return f16 ? launch_mode<128, kQ8Fp16>(a, s) : launch_mode<128, kQ8Bf16>(a, s);
    return f16 ? launch_mode<64, kQ8Fp16>(a, s) : launch_mode<64, kQ8Bf16>(a, s);
}

}  // namespace ddt
