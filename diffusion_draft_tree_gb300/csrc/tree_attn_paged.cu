// tree_attn_paged.cu -- ddtree_tree_attn_paged: the tree-attention kernel
// (tree_attn.cuh) over a paged cache, bf16 or fp16.
#include "tree_attn.cuh"

namespace ddt {

namespace {

// The stride of a dimension of one entry is never used; its map needs a legal one.
uint64_t stride_bytes(int64_t elements, int64_t size, uint64_t rowb) {
    return size > 1 ? (uint64_t)elements * 2 : rowb;
}

template <int D, int MODE>
cudaError_t launch_mode(const PagedAttnArgs& a, cudaStream_t s) {
    int dev = 0;
    cudaGetDevice(&dev);
    if (const cudaError_t e = prepare_kernel<D, MODE>(dev)) return e;
    const int Hq = a.q.heads, Hkv = a.cache.Hkv, ps = a.cache.page_size;
    const int64_t cap = (int64_t)a.cache.max_pages * ps;
    const Plan base = plan_base(a.N, Hq, Hkv);
    const Tiles t = max_tiles(a.N, cap);
    const long units = plan_units(base, a.B, Hkv);
    const int sms = num_sms();
    const Plan pl = units >= sms ? plan_many(base, t, units, sms)
                                 : plan_few(base, t, units, sms, [&](int S) {
                                       return merge_fits<D>(S) ? active_clusters<D, MODE>(dev, S) : 0;
                                   });
    const WsLayout wl = attn_layout(pl, a.B, Hkv, D, 4);
    const int G = Hq / Hkv, R = a.N + 1;
    const uint64_t rowb = (uint64_t)D * 2, tokens = (uint64_t)a.B * R;
    constexpr bool f16 = MODE == kPagedFp16;
    auto tree_map = [&](CUtensorMap* m, const RowsArg& r, uint32_t heads, uint32_t nodes) {
        const MapDim d[3] = {{(uint64_t)D, 0, 64},
                             {(uint64_t)r.heads, stride_bytes(r.hs, r.heads, rowb), heads},
                             {tokens, stride_bytes(r.ts, tokens, rowb), nodes}};
        return make_map(m, r.data, d, f16);
    };
    auto page_map = [&](CUtensorMap* m, const void* pages) {
        const PagedArgs& c = a.cache;
        const MapDim d[4] = {{(uint64_t)D, 0, 64},
                             {(uint64_t)ps, stride_bytes(c.slot_stride, ps, rowb), (uint32_t)std::min(ps, BN)},
                             {(uint64_t)Hkv, stride_bytes(c.head_stride, Hkv, rowb), 1},
                             {(uint64_t)c.num_pages, stride_bytes(c.page_stride, c.num_pages, rowb), 1}};
        return make_map(m, pages, d, f16);
    };
    CUtensorMap mq, mkc, mvc, mkt, mvt;
    if (!tree_map(&mq, a.q, G, BM / G) || !tree_map(&mkt, a.k_tree, 1, BN) ||
        !tree_map(&mvt, a.v_tree, 1, BN) || !page_map(&mkc, a.cache.k) || !page_map(&mvc, a.cache.v))
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
    p.lpt = (pl.merge != kMergeCluster && (long)a.B * pl.smax <= kLptMaxItems) ? 1 : 0;
    p.cache_cap = cap;
    p.scale_log2 = a.scale * kLog2e;
    p.err = a.err;
    p.table = a.cache.table;
    p.table_stride = a.cache.table_stride;
    p.num_pages = a.cache.num_pages;
    for (p.ps_log2 = 0; (1 << p.ps_log2) < ps;) ++p.ps_log2;
    p.npt = BM / G;
    const long grid = units * pl.smax;
    if (grid > INT32_MAX) return cudaErrorInvalidValue;
    return launch_pdl_cluster(tree_attn_kernel<D, MODE>, dim3((unsigned)grid), dim3(kThreads),
                              (size_t)Cfg<D>::SMEM, s,
                              pl.merge == kMergeCluster ? (unsigned)pl.smax : 1u, mq, mkc, mvc,
                              mkt, mvt, p);
}

}  // namespace

size_t paged_attn_workspace_bytes(int B, int N, int Hq, int Hkv, int D, int64_t cache_cap) {
    const Plan base = plan_base(N, Hq, Hkv);
    const long units = plan_units(base, B, Hkv);
    if (units < num_sms()) return 0;
    return attn_layout(plan_many(base, max_tiles(N, cache_cap), units, num_sms()), B, Hkv, D, 4).total;
}

cudaError_t launch_tree_attn_paged(const PagedAttnArgs& a, cudaStream_t s) {
    const bool f16 = a.cache.dtype == 2;
    if (a.cache.D == 128)
        return f16 ? launch_mode<128, kPagedFp16>(a, s) : launch_mode<128, kPagedBf16>(a, s);
    return f16 ? launch_mode<64, kPagedFp16>(a, s) : launch_mode<64, kPagedBf16>(a, s);
}

}  // namespace ddt
