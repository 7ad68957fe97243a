// tree_attn_paged.cuh -- launch of the tree-attention kernel (tree_attn.cuh) over a
// paged cache.
#pragma once
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
    const Tiles t = max_tiles(a.N, cap);
    const int sms = num_sms();
    const ManyPlan many = plan_paged_many(a.B, a.N, Hq, Hkv, t, sms);
    PagedPlan pl{};
    if (many.smax) {
        (Plan&)pl = many;
        pl.npt = BM / G;
    } else if constexpr (!is_left(MODE)) {
        pl = plan_paged_few(a.B, a.N, G, Hkv, t, sms, [&](int S) {
            return merge_fits<D>(S) ? active_clusters<D, MODE>(dev, S) : 0;
        });
    }
    const WsLayout wl = attn_layout(pl, a.B, Hkv, D, 4, many.left);
    const uint64_t tokens = (uint64_t)a.B * R;
    constexpr bool f16 = is_f16(MODE);
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
    p.left = many.left;
    p.q = (const uint16_t*)a.q.data;
    p.q_ts = a.q.ts, p.q_hs = a.q.heads > 1 ? a.q.hs : D;
    if (many.left && wl.total) {
        p.tickets_left = (unsigned int*)(ws + wl.tickets_left);
        p.part_left = (float*)(ws + wl.part_left);
    }
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
    return launch_pdl_cluster(tree_attn_kernel<D, MODE>, dim3((unsigned)grid), dim3(threads_of(MODE)),
                              (size_t)Cfg<D>::SMEM, s,
                              pl.merge == kMergeCluster ? (unsigned)pl.smax : 1u, mq, mkc, mvc,
                              mkt, mvt, p);
}

}  // namespace

cudaError_t launch_tree_attn_left(const PagedAttnArgs& a, cudaStream_t s);

}  // namespace ddt
