// tree_attn.cu -- ddtree_tree_attn: the tree-attention kernel (tree_attn.cuh)
// over a dense cache, one [cap][D] block per (sequence, KV head).
#include "tree_attn.cuh"

namespace ddt {

namespace {

template <int D>
cudaError_t launch_d(const AttnArgs& a, cudaStream_t s) {
    int dev = 0;
    cudaGetDevice(&dev);
    if (const cudaError_t e = prepare_kernel<D, kDense>(dev)) return e;
    const Plan base = plan_base(a.N, a.Hq, a.Hkv);
    const Tiles t = max_tiles(a.N, a.cache_cap);
    const long units = plan_units(base, a.B, a.Hkv);
    const int sms = num_sms();
    const Plan pl = units >= sms ? plan_many(base, t, units, sms)
                                 : plan_few(base, t, units, sms,
                                            [&](int S) {
                                                return Cfg<D>::recv_fits_upto(S) ? active_clusters<D, kDense>(dev, S) : 0;
                                            });
    const WsLayout wl = attn_layout(pl, a.B, a.Hkv, D, 2);
    const int G = a.Hq / a.Hkv, R = a.N + 1;
    CUtensorMap mq, mkc, mvc, mkt, mvt;
    const uint64_t rowb = (uint64_t)D * 2;
    const uint64_t cap = a.cache_cap ? a.cache_cap : 1, caches = (uint64_t)a.B * a.Hkv;
    const MapDim dq[3] = {{(uint64_t)D, 0, 64}, {(uint64_t)a.Hq, rowb, (uint32_t)G}, {(uint64_t)a.B * R, rowb * a.Hq, (uint32_t)(BM / G)}};
    const MapDim dc[3] = {{(uint64_t)D, 0, 64}, {cap, rowb, BN}, {caches, rowb * cap, 1}};
    const MapDim dt[3] = {{(uint64_t)D, 0, 64}, {(uint64_t)a.Hkv, rowb, 1}, {(uint64_t)a.B * R, rowb * a.Hkv, BN}};
    const bool ok = make_map(&mq, a.q, dq) && make_map(&mkc, a.k_cache, dc) &&
                    make_map(&mvc, a.v_cache, dc) && make_map(&mkt, a.k_tree, dt) &&
                    make_map(&mvt, a.v_tree, dt);
    if (!ok) return cudaErrorInvalidValue;
    Params p;
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
    p.B = a.B; p.N = a.N; p.Hq = a.Hq; p.Hkv = a.Hkv; p.G = G; p.W = (a.N + 1 + 31) / 32;
    p.mtiles = pl.mtiles; p.mpairs = pl.mpairs; p.tps = pl.tps; p.smax = pl.smax;
    p.merge = pl.merge;
    p.lpt = (pl.merge != kMergeCluster && (long)a.B * pl.smax <= kLptMaxItems) ? 1 : 0;
    p.cache_cap = a.cache_cap;
    p.scale_log2 = a.scale * kLog2e;
    p.err = a.err;
    const long grid = units * pl.smax;
    return launch_pdl_cluster(tree_attn_kernel<D, kDense>, dim3((unsigned)grid), dim3(kThreads),
                              (size_t)Cfg<D>::SMEM, s,
                              pl.merge == kMergeCluster ? (unsigned)pl.smax : 1u, mq, mkc, mvc,
                              mkt, mvt, p);
}

}  // namespace

// Only plans for many units (no clusters) merge their KV splits in a workspace.
size_t attn_workspace_bytes(int B, int N, int Hq, int Hkv, int D, int64_t cache_cap) {
    const Plan base = plan_base(N, Hq, Hkv);
    if (plan_units(base, B, Hkv) < num_sms()) return 0;
    return attn_layout(plan_many(base, max_tiles(N, cache_cap), plan_units(base, B, Hkv), num_sms()),
                       B, Hkv, D, 2).total;
}

cudaError_t launch_tree_attn(const AttnArgs& a, cudaStream_t s) {
    if (a.D == 128) return launch_d<128>(a, s);
    return launch_d<64>(a, s);
}

}  // namespace ddt
