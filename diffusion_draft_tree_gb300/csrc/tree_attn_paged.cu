// tree_attn_paged.cu -- ddtree_tree_attn_paged: the tree-attention kernel
// (tree_attn.cuh) over a paged cache, bf16 or fp16.
#include "tree_attn.cuh"

namespace ddt {

namespace {

template <int D, int MODE>
cudaError_t launch_mode(const PagedAttnArgs& a, cudaStream_t s) {
    int dev = 0;
    cudaGetDevice(&dev);
    if (const cudaError_t e = prepare_kernel<D, MODE>(dev)) return e;
    const int Hq = a.q.heads, Hkv = a.cache.Hkv, ps = a.cache.page_size;
    const int64_t cap = (int64_t)a.cache.max_pages * ps;
    const int G = Hq / Hkv, R = a.N + 1;
    const Plan base = plan_base(a.N, Hq, Hkv);
    const Tiles t = max_tiles(a.N, cap);
    const long units = plan_units(base, a.B, Hkv);
    const int sms = num_sms();
    PagedPlan pl{};
    if (units >= sms) {
        (Plan&)pl = plan_many(base, planned(t), units, sms);
        pl.npt = BM / G;
    } else {
        pl = plan_paged_few(a.B, a.N, G, Hkv, t, sms, [&](int S) {
            return merge_fits<D>(S) ? active_clusters<D, MODE>(dev, S) : 0;
        });
    }
    const WsLayout wl = attn_layout(pl, a.B, Hkv, D, 4);
    const uint64_t tokens = (uint64_t)a.B * R;
    constexpr bool f16 = MODE == kPagedFp16;
    CUtensorMap mq, mkc, mvc, mkt, mvt;
    if (!tree_map<D>(&mq, a.q, tokens, G, pl.npt, f16) || !tree_map<D>(&mkt, a.k_tree, tokens, 1, BN, f16) ||
        !tree_map<D>(&mvt, a.v_tree, tokens, 1, BN, f16) ||
        !page_map<D>(&mkc, a.cache, a.cache.k, BN, f16) || !page_map<D>(&mvc, a.cache, a.cache.v, BN, f16))
        return cudaErrorInvalidValue;
    PagedParams p{};
    p.prefix_len = a.prefix_len;
    p.n_nodes = a.n_nodes;
    p.anc_mask = a.anc_mask;
    p.out = (uint16_t*)a.out;
    p.lse = a.lse;
    char* ws = (char*)a.ws;
    const bool glob = pl.merge == kMergeGlobal;
    p.tickets = glob ? (unsigned int*)(ws + wl.tickets) : nullptr;
    p.part_o = glob ? (uint32_t*)(ws + wl.part_o) : nullptr;
    p.part_ml = glob ? (float*)(ws + wl.part_ml) : nullptr;
    p.B = a.B; p.N = a.N; p.Hq = Hq; p.Hkv = Hkv; p.G = G; p.W = (a.N + 1 + 31) / 32;
    p.mtiles = pl.mtiles; p.mpairs = pl.mpairs; p.tps = pl.tps; p.smax = pl.smax;
    p.merge = pl.merge;
    const int64_t plan_tiles = planned(t).prefix + t.tree, table_tiles = t.prefix + t.tree;
    p.share = (int)((pl.tps * (int64_t)65536 + plan_tiles - 1) / plan_tiles);
    p.sms = sms;
    p.lpt = (pl.merge != kMergeCluster && a.B <= kRankedSeqs) ? 1 : 0;
    if (pl.merge == kMergeGlobal && !p.lpt)  // not ranked: the plan's share of the table
        p.tps = (int)((pl.tps * table_tiles + plan_tiles - 1) / plan_tiles);
    p.cache_cap = cap;
    p.scale_log2 = a.scale * kLog2e;
    p.err = a.err;
    p.table = a.cache.table;
    p.table_stride = a.cache.table_stride;
    p.num_pages = a.cache.num_pages;
    for (p.ps_log2 = 0; (1 << p.ps_log2) < ps;) ++p.ps_log2;
    p.npt = pl.npt;
    p.single = pl.single;
    const long grid = plan_units(pl, a.B, Hkv) * pl.smax;
    if (grid > INT32_MAX) return cudaErrorInvalidValue;
    return launch_pdl_cluster(tree_attn_kernel<D, MODE>, dim3((unsigned)grid), dim3(kThreads),
                              (size_t)Cfg<D>::SMEM, s,
                              pl.merge == kMergeCluster ? (unsigned)pl.smax : 1u, mq, mkc, mvc,
                              mkt, mvt, p);
}

}  // namespace

size_t paged_attn_workspace_bytes(int B, int N, int Hq, int Hkv, int D, int64_t cache_cap) {
    if (few_rows(B, N, Hq, Hkv, cache_cap)) return few_rows_workspace_bytes(N, Hq, Hkv, D);
    const Plan base = plan_base(N, Hq, Hkv);
    const long units = plan_units(base, B, Hkv);
    if (units < num_sms()) return 0;
    return attn_layout(plan_many(base, planned(max_tiles(N, cache_cap)), units, num_sms()), B, Hkv, D, 4).total;
}

cudaError_t launch_tree_attn_paged(const PagedAttnArgs& a, cudaStream_t s) {
    if (few_rows(a.B, a.N, a.q.heads, a.cache.Hkv, (int64_t)a.cache.max_pages * a.cache.page_size))
        return launch_tree_attn_rows(a, s);
    const bool f16 = a.cache.dtype == 2;
    if (a.cache.D == 128)
        return f16 ? launch_mode<128, kPagedFp16>(a, s) : launch_mode<128, kPagedBf16>(a, s);
    return f16 ? launch_mode<64, kPagedFp16>(a, s) : launch_mode<64, kPagedBf16>(a, s);
}

}  // namespace ddt
