// tree_attn_q8_rows.cu -- ddtree_tree_attn_q8 for few query rows: plain decoding (N = 0, the
// G query heads of a KV head are the rows) and small trees, up to 8 NB rows a unit.
//
// The list of key tiles, its runs and their join are those of tree_attn_rows.cu; a tile is
// 128 keys, as many bytes as 64 of the 16-bit cache.  HBM-bound as well, at half the bytes a
// key, so the products have half the time: mma.sync takes 16 keys as its wide side and 8
// rows as its narrow one, S^T = K Q^T and O^T += V^T P^T, half the products of 16 rows wide.
// Codes stay codes as far as a warp's registers: ldmatrix brings 4 codes a word, which
// widen into the two operand words of a product (even codes, odd codes) with the block's
// scale on the way, exactly (q8.cuh).  Which of 16 elements of a head a word holds is the
// products' own affair for K, where Q is loaded in the same order; for V, ldmatrix
// transposes pairs of codes, and a pair's two elements are two rows of O^T.
// Warp w takes keys [32 w, 32 w + 32) of a tile.
//
// 64 sequences of 512 to 16384, 32 query and 8 KV heads, D = 128: 178 us, 93 % of the measured
// HBM rate (the tcgen05 kernel 478, its query tile 4 rows of 128; the 16-bit cache 327).
#include "q8.cuh"
#include "tree_attn_rows.cuh"

namespace ddt {

namespace {

constexpr int kTile = 128;

template <int D, int NB>
struct CfgQ {
    static constexpr int KV = kTile * D;  // a tile's K (or V)
    static constexpr int STAGE = 2 * KV;
    static constexpr int NS = D == 128 ? 3 : 6;
    static constexpr int SMEM = 1024 + NS * STAGE;
    static constexpr int TREE = 16 * 128;  // a slab of a tree's 16-bit rows
    static_assert(2 * (D / 64) * TREE <= STAGE, "a stage holds a tree");
    static_assert(kWarps * 8 * NB * D * 4 <= STAGE, "a stage holds the warps' outputs");
};

struct ParamsQ : ParamsR {
    const uint16_t* q;
    int64_t q_ts, q_hs;
    const uint8_t *k_scales, *v_scales;
    int block_log2, per_page_log2;  // log2 of positions a scale, of scales a page and head
};

// 16-byte chunk c of row r of a tile of codes, swizzled by its row's length.
template <int D>
DDT_DEV uint32_t swz8(int r, int c) {
    return D == 128 ? swz(r, c) : (uint32_t)(r * 64 + ((c ^ ((r >> 1) & 3)) << 4));
}

template <int D, bool F16, int NB>
__global__ void __launch_bounds__(kThreadsR, 2)
tree_attn_q8_rows_kernel(const __grid_constant__ CUtensorMap tm_kc, const __grid_constant__ CUtensorMap tm_vc,
                         const __grid_constant__ CUtensorMap tm_kt, const __grid_constant__ CUtensorMap tm_vt,
                         const __grid_constant__ ParamsQ p) {
    using C = CfgQ<D, NB>;
    constexpr int NS = C::NS, NH = D / 64;
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t bar_full[NS], bar_empty[NS];
    __shared__ __align__(8) uint16_t s_mult[NS][2][kTile];  // factors of the keys, of the values
    __shared__ RunList s_list;
    __shared__ float2 s_ml[kWarps][8 * NB];
    __shared__ volatile int s_abort;
    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // known to be one number a warp
    const uint32_t base_u32 = (smem_u32(smem_raw) + 1023u) & ~1023u;
    uint8_t* base = smem_raw + (base_u32 - smem_u32(smem_raw));

    if (tid == 0) {
        for (int s = 0; s < NS; ++s) {
            mbar_init(&bar_full[s], 1);
            mbar_init(&bar_empty[s], kWarps);
        }
        s_abort = 0;
        mbar_init_fence();
        tma_prefetch_desc(&tm_kc);
        tma_prefetch_desc(&tm_vc);
        tma_prefetch_desc(&tm_kt);
        tma_prefetch_desc(&tm_vt);
    }
    pdl_wait();
    const int R = p.N + 1;
    build_list<kTile>(s_list, p);
    const int64_t total = (int64_t)s_list.cum[p.B] * p.Hkv, chunk = s_list.chunk;
    const int64_t t_begin = blockIdx.x * chunk;
    int64_t t_end = min(total, t_begin + chunk);
    if (t_begin >= t_end) {
        if (tid == 0) p.cut[blockIdx.x] = make_int4(0, 0, 0, 0);
        return;
    }
    auto prefix_of = [&](const Place& x) { return ddt::prefix_of<kTile>(s_list, x); };
    auto next_unit = [&](Place& x) { ddt::next_unit(s_list, p, x); };
    auto fail = [&]() {
        record_error(p.err, ERR_ATTN | ERR_WAIT_TIMEOUT);
        s_abort = 1;
    };
    Place at = place_of(s_list, p, t_begin);
    if (s_list.pad[at.b]) t_end = min(t_end, t_begin + at.tiles - at.tile);  // (the padding)

    if (warp == kWarps) {
        // ============================= copy warp =============================
        const int ps = 1 << p.ps_log2, box = min(ps, kTile), nb = kTile / box;
        const int box_log2 = 31 - __clz(box);
        const int per_box = 1 << max(0, box_log2 - p.block_log2);  // scales of a box
        const uint32_t lead = elect_one();
        // Page numbers come 32 boxes at a time, lane l holding box 32 k + l of its unit,
        // two batches -- of this unit or the next ones -- ahead; the boxes' scales, up to 16
        // bytes each, one ahead.  From the pool's end a copy reads zeros: pages outside
        // the pool.
        struct Batch {
            Place x;
            int k;
            int64_t left;  // tiles of the run from the unit's first (or the run's) tile on
        };
        auto ids_of = [&](const Batch& y) {
            const int64_t key = ((int64_t)y.k * 32 + lane) * box;
            return y.left > 0 && key < prefix_of(y.x)
                       ? __ldg(&p.table[y.x.b * p.table_stride + (key >> p.ps_log2)])
                       : p.num_pages;
        };
        auto checked = [&](int page, const Batch& y) {
            if ((unsigned)page < (unsigned)p.num_pages) return page;
            if (y.left > 0 && ((int64_t)y.k * 32 + lane) * box < prefix_of(y.x))
                record_error(p.err, ERR_ATTN | ERR_BAD_PAGE);
            return p.num_pages;
        };
        auto scales_of = [&](int page, const Batch& y, const uint8_t* from) {
            if (page == p.num_pages) return make_uint4(0u, 0u, 0u, 0u);
            const int slot = (int)((((int64_t)y.k * 32 + lane) * box) & (ps - 1));
            return box_scales(from + ((((int64_t)page * p.Hkv + y.x.g) << p.per_page_log2) + (slot >> p.block_log2)), per_box);
        };
        auto advance = [&](Batch& y) {
            if (y.left <= 0) return;
            if (((int64_t)y.k + 1) * 32 * box < prefix_of(y.x)) {
                ++y.k;
            } else {
                y.k = 0;
                y.left -= y.x.tiles - y.x.tile;
                if (y.left > 0) next_unit(y.x);
            }
        };
        Batch b1{at, (int)((int64_t)at.tile * nb / 32), t_end - t_begin};
        int ids = checked(ids_of(b1), b1);
        uint4 ks = scales_of(ids, b1, p.k_scales), vs = scales_of(ids, b1, p.v_scales);
        advance(b1);
        int ids1 = checked(ids_of(b1), b1);
        uint4 ks1 = scales_of(ids1, b1, p.k_scales), vs1 = scales_of(ids1, b1, p.v_scales);
        Batch b2 = b1;
        advance(b2);
        int ids2 = ids_of(b2);
        int issued = 0;
        for (int64_t t = t_begin; t < t_end; ++t) {
            const int it = (int)(t - t_begin), s = it % NS;
            if (t > t_begin) {
                const bool same = ++at.tile < at.tiles;
                if (!same) next_unit(at);
                if (!same || (at.tile * nb % 32 == 0 && at.tile < at.tiles - 1)) {
                    ids = ids1, ks = ks1, vs = vs1;
                    ids1 = checked(ids2, b2);
                    ks1 = scales_of(ids1, b2, p.k_scales), vs1 = scales_of(ids1, b2, p.v_scales);
                    advance(b2);
                    ids2 = ids_of(b2);
                }
            }
            const bool tree = at.tile == at.tiles - 1;
            const int key0 = at.tile * kTile;
            const int boxes = tree ? 0 : min(nb, (prefix_of(at) - key0 + box - 1) / box);
            // (of the warp as a whole)
            if (!mbar_wait_warp(&bar_empty[s], ((it / NS) & 1) ^ 1, &s_abort)) { fail(); break; }
            const uint32_t dk = smem_u32(base + s * C::STAGE);
            if (tree) {
#pragma unroll
                for (int h = 0; h < NH; ++h) {
                    tma_load_3d_warp(lead, dk + h * C::TREE, &tm_kt, &bar_full[s], 64 * h, at.g, at.b * R);
                    tma_load_3d_warp(lead, dk + (NH + h) * C::TREE, &tm_vt, &bar_full[s], 64 * h, at.g, at.b * R);
                }
            } else {
#pragma unroll 4
                for (int i = 0; i < boxes; ++i) {
                    const int page = __shfl_sync(0xffffffffu, ids, (at.tile * nb + i) & 31);
                    const int row = (key0 + i * box) & (ps - 1);
                    tma_load_4d_warp(lead, dk + i * box * D, &tm_kc, &bar_full[s], 0, row, at.g, page);
                    tma_load_4d_warp(lead, dk + C::KV + i * box * D, &tm_vc, &bar_full[s], 0, row, at.g, page);
                }
            }
            if (!tree) {  // (the copies are on their way while the scales still are)
#pragma unroll
                for (int v = 0; v < 2; ++v) {
                    const uint32_t m = widen_factor<F16>(tile_scale(v ? vs : ks, at.tile * nb, box_log2, p.block_log2,
                                                                    per_box, lane)) * 0x10001u;
                    *(uint2*)&s_mult[s][v][4 * lane] = make_uint2(m, m);
                }
            }
            __syncwarp();
            if (lane == 0)
                mbar_arrive_expect_tx(&bar_full[s], tree ? 4 * D * R : 2 * D * boxes * box);
            issued = it + 1;
        }
        // (where a wait gave up, here or below, no copy may land in memory given back)
        for (int it = max(0, issued - NS); it < issued; ++it)
            mbar_wait(&bar_full[it % NS], (it / NS) & 1, nullptr, 100000000ull);
        return;
    }

    // ============================ computing warps ============================
    const int gl = lane >> 2, cl = lane & 3;  // a product's rows and columns, by lane
    const float sl2 = p.scale_log2;
    for (int64_t t = t_begin; t < t_end;) {
        // ---- a unit, or the part of it in this CTA's run -------------------------
        const int left = (int)min(t_end - t, (int64_t)(at.tiles - at.tile));
        const bool has_tree = at.tile + left == at.tiles;
        const int P = prefix_of(at), n = s_list.nodes[at.b];
        // Q^T, the right operand: row gl of each block, its elements in the order of the
        // codes' words: (16 kk + 4 cl) + 0, 2 and + 1, 3.
        uint32_t q[NB][D / 16][2];
        const uint16_t* qrow[NB];
        bool qlive[NB];
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            const int r = 8 * b + gl, u = r / p.G;
            qlive[b] = r < p.rows && u <= n;
            qrow[b] = p.q + ((int64_t)at.b * R + u) * p.q_ts + (int64_t)(at.g * p.G + r - u * p.G) * p.q_hs;
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                uint2 w = make_uint2(0u, 0u);
                if (qlive[b]) w = __ldg((const uint2*)(qrow[b] + 16 * kk + 4 * cl));
                q[b][kk][0] = __byte_perm(w.x, w.y, 0x5410);
                q[b][kk][1] = __byte_perm(w.x, w.y, 0x7632);
            }
        }
        float o[NB][D / 16][4];  // O^T: elements 16 i + 2 gl (+ 1: [2], [3]) of rows 2 cl, 2 cl + 1
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int i = 0; i < D / 16; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[b][i][e] = 0.f;
        float m[NB][2], l[NB][2];
#pragma unroll
        for (int b = 0; b < NB; ++b) m[b][0] = m[b][1] = -INFINITY, l[b][0] = l[b][1] = 0.f;

        // The weights of KG groups of 16 keys from their scores, the maxima and sums; keys
        // 16 kg + gl (+ 8: [2], [3]) of rows 2 cl, 2 cl + 1.  pw: the right operand, two
        // words a group: weights rounded to the tokens' type, as a product takes both factors in
        // one (half a step a weight, independent ones; the output is rounded once more at the end).
        auto weigh = [&](auto& x, auto& pw) {
            constexpr int KG = sizeof(x[0]) / sizeof(x[0][0]);
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                float mx0 = -INFINITY, mx1 = -INFINITY;
#pragma unroll
                for (int kg = 0; kg < KG; ++kg) {
                    mx0 = fmaxf(mx0, fmaxf(x[b][kg][0], x[b][kg][2]));
                    mx1 = fmaxf(mx1, fmaxf(x[b][kg][1], x[b][kg][3]));
                }
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) {
                    mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, d));
                    mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, d));
                }
                // the sums and outputs move to a new maximum only when it is 2^8 larger
                const bool up0 = mx0 > m[b][0] + 8.f, up1 = mx1 > m[b][1] + 8.f;
                if (__any_sync(0xffffffffu, up0 || up1)) {
                    const float f0 = up0 ? fast_exp2(m[b][0] - mx0) : 1.f, f1 = up1 ? fast_exp2(m[b][1] - mx1) : 1.f;
                    m[b][0] = up0 ? mx0 : m[b][0];
                    m[b][1] = up1 ? mx1 : m[b][1];
                    l[b][0] *= f0;
                    l[b][1] *= f1;
#pragma unroll
                    for (int i = 0; i < D / 16; ++i) {
                        o[b][i][0] *= f0, o[b][i][2] *= f0;
                        o[b][i][1] *= f1, o[b][i][3] *= f1;
                    }
                }
                const float b0 = m[b][0] == -INFINITY ? 0.f : m[b][0] - kLift<F16>;
                const float b1 = m[b][1] == -INFINITY ? 0.f : m[b][1] - kLift<F16>;
#pragma unroll
                for (int kg = 0; kg < KG; ++kg)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float e0 = fast_exp2(x[b][kg][2 * h] - b0), e1 = fast_exp2(x[b][kg][2 * h + 1] - b1);
                        l[b][0] += e0;  // (the sums take them unrounded)
                        l[b][1] += e1;
                        pw[b][kg][h] = movmatrix_t(pack16<F16>(e0, e1));
                    }
            }
        };

        const int it0 = (int)(t - t_begin), it = it0 + left - 1;  // the unit's tiles of the run
        // A wait that gives up ends the unit's products, not its barriers: the warps
        // stay together.
        bool ok = true;
        const int codes = left - (has_tree ? 1 : 0);
        for (int k = 0; ok && k < codes; ++k) {
            const int s = (it0 + k) % NS;
            ok = mbar_wait_warp(&bar_full[s], ((it0 + k) / NS) & 1, &s_abort);
            if (!ok) { fail(); break; }
            const int lim = P - (at.tile + k) * kTile - 32 * warp;  // keys of the warp's 32 that exist
            if (lim > 0) {
                const uint32_t ka = smem_u32(base + s * C::STAGE), va = ka + C::KV;
                float x[NB][2][4];
#pragma unroll
                for (int kg = 0; kg < 2; ++kg) {
                    const int key0 = 32 * warp + 16 * kg;
                    const uint32_t m0 = (uint32_t)s_mult[s][0][key0 + gl] * 0x10001u;
                    const uint32_t m1 = (uint32_t)s_mult[s][0][key0 + 8 + gl] * 0x10001u;
#pragma unroll
                    for (int b = 0; b < NB; ++b)
#pragma unroll
                        for (int e = 0; e < 4; ++e) x[b][kg][e] = 0.f;
#pragma unroll
                    for (int i = 0; i < D / 32; ++i) {
                        uint32_t f[4];
                        ldsm_x4(ka + swz8<D>(key0 + (lane & 15), 2 * i + (lane >> 4)), f);
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const uint32_t a[4] = {widen_even<F16>(f[2 * h], m0), widen_even<F16>(f[2 * h + 1], m1),
                                                   widen_odd<F16>(f[2 * h], m0), widen_odd<F16>(f[2 * h + 1], m1)};
#pragma unroll
                            for (int b = 0; b < NB; ++b)
                                mma16816<F16>(x[b][kg], a, q[b][2 * i + h][0], q[b][2 * i + h][1]);
                        }
                    }
                }
#pragma unroll
                for (int b = 0; b < NB; ++b)
#pragma unroll
                    for (int kg = 0; kg < 2; ++kg)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            x[b][kg][e] *= sl2;
                            if (16 * kg + gl + 8 * (e >> 1) >= lim) x[b][kg][e] = -INFINITY;
                        }
                uint32_t pw[NB][2][2];
                weigh(x, pw);
                // (codes past the sequence widen to numbers, whatever they are, and weigh 0)
#pragma unroll
                for (int kg = 0; kg < 2; ++kg) {
                    const int key0 = 32 * warp + 16 * kg;
                    const uint32_t m0 = *(const uint32_t*)&s_mult[s][1][key0 + 2 * cl];
                    const uint32_t m1 = *(const uint32_t*)&s_mult[s][1][key0 + 8 + 2 * cl];
#pragma unroll
                    for (int i = 0; i < D / 32; ++i) {
                        uint32_t f[4];
                        ldsm_x4_t(va + swz8<D>(key0 + (lane & 15), 2 * i + (lane >> 4)), f);
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const uint32_t a[4] = {widen_even<F16>(f[2 * h], m0), widen_odd<F16>(f[2 * h], m0),
                                                   widen_even<F16>(f[2 * h + 1], m1), widen_odd<F16>(f[2 * h + 1], m1)};
#pragma unroll
                            for (int b = 0; b < NB; ++b) mma16816<F16>(o[b][2 * i + h], a, pw[b][kg][0], pw[b][kg][1]);
                        }
                    }
                }
            }
            __syncwarp();
            // (the unit's last stage takes the outputs first)
            if (k < left - 1 && lane == 0) mbar_arrive(&bar_empty[s]);
        }
        if (ok && has_tree) {  // 16-bit rows, one group of 16 keys: the first warp's
            const int s = it % NS;
            ok = mbar_wait_warp(&bar_full[s], (it / NS) & 1, &s_abort);
            if (!ok) fail();
            if (ok && warp == 0) {
                uint8_t* kt = base + s * C::STAGE;
                uint8_t* vt = kt + NH * C::TREE;
                // Rows past the tree may hold anything, and 0 x NaN is NaN.
                for (int i = lane; i < (15 - n) * NH * 8; i += 32) {
                    const int row = n + 1 + i / (NH * 8), h = (i >> 3) % NH;
                    *(uint4*)(vt + h * C::TREE + row * 128 + (i & 7) * 16) = make_uint4(0, 0, 0, 0);
                    *(uint4*)(kt + h * C::TREE + row * 128 + (i & 7) * 16) = make_uint4(0, 0, 0, 0);
                }
                fence_proxy_async_smem();  // (the next copy into the stage comes after)
                __syncwarp();
                float x[NB][1][4];
#pragma unroll
                for (int b = 0; b < NB; ++b)
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[b][0][e] = 0.f;
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    uint32_t a[4];
                    ldsm_x4(smem_u32(kt) + (kk >> 2) * C::TREE + swz(lane & 15, (kk & 3) * 2 + (lane >> 4)), a);
#pragma unroll
                    for (int b = 0; b < NB; ++b) {
                        uint32_t w[2] = {0u, 0u};
                        if (qlive[b]) {
                            w[0] = __ldg((const uint32_t*)(qrow[b] + 16 * kk + 2 * cl));
                            w[1] = __ldg((const uint32_t*)(qrow[b] + 16 * kk + 8 + 2 * cl));
                        }
                        mma16816<F16>(x[b][0], a, w[0], w[1]);
                    }
                }
#pragma unroll
                for (int b = 0; b < NB; ++b)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int u = (8 * b + 2 * cl + (e & 1)) / p.G, key = gl + 8 * (e >> 1);
                        const uint32_t see = u <= n ? __ldg(&p.anc_mask[(size_t)at.b * R + u]) : 0u;  // (one word)
                        x[b][0][e] = key <= n && ((see >> key) & 1u) ? x[b][0][e] * sl2 : -INFINITY;
                    }
                uint32_t pw[NB][1][2];
                weigh(x, pw);
#pragma unroll
                for (int i = 0; i < D / 16; ++i) {
                    uint32_t a[4];
                    ldsm_x4_t(smem_u32(vt) + (i >> 2) * C::TREE +
                                  swz((lane >> 4) * 8 + (lane & 7), (i & 3) * 2 + ((lane >> 3) & 1)),
                              a);
                    // rows gl, gl + 8 of a product are elements 2 gl, 2 gl + 1 of the sums: the
                    // tree's come as gl, gl + 8, so they are summed apart and moved
#pragma unroll
                    for (int b = 0; b < NB; ++b) {
                        float y[4] = {0.f, 0.f, 0.f, 0.f};
                        mma16816<F16>(y, a, pw[b][0][0], pw[b][0][1]);
                        // element 2 gl is row 2 gl (gl < 4) or 2 gl - 8 of the upper half
                        const int from = ((2 * gl) & 7) * 4 + cl, next = from + 4;
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const float lo0 = __shfl_sync(0xffffffffu, y[e], from), hi0 = __shfl_sync(0xffffffffu, y[2 + e], from);
                            const float lo1 = __shfl_sync(0xffffffffu, y[e], next), hi1 = __shfl_sync(0xffffffffu, y[2 + e], next);
                            o[b][i][e] += gl < 4 ? lo0 : hi0;
                            o[b][i][2 + e] += gl < 4 ? lo1 : hi1;
                        }
                    }
                }
            }
        }

        // ---- the warps' shares of the unit, joined in its last stage ----------------
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) l[b][e] += __shfl_xor_sync(0xffffffffu, l[b][e], d);
        float* so = reinterpret_cast<float*>(base + (it % NS) * C::STAGE);
        // element 8 j + e of a warp's row r, its groups of 8 permuted by the row so that the
        // rows that a warp stores at once do not share their banks
        auto so_at = [&](int w, int r, int j, int e) {
            return &so[(w * 8 * NB + r) * D + ((j ^ ((r >> 1) & 3)) << 3) + e];
        };
        // The CTAs that hold its tiles: alone, or this run's piece of several -- slot 1
        // if it is the first, which leaves word of the unit for the second kernel.
        const bool whole_unit = at.tile == 0 && left == at.tiles;
        const bool first = at.tile == 0;
        float* mine = p.part + ((size_t)blockIdx.x * 2 + (first ? 1 : 0)) * p.rows * (D + 4);
        if (tid == 0 && t + left == t_end) {
            const int64_t last_run = (t - at.tile + at.tiles - 1) / chunk;
            p.cut[blockIdx.x] = first && !whole_unit
                                    ? make_int4(at.b, at.g, (int)(last_run - blockIdx.x + 1), n)
                                    : make_int4(0, 0, 0, 0);
        }
        warps_bar();  // every warp has read its keys of the stage
#pragma unroll
        for (int b = 0; b < NB; ++b) {
#pragma unroll
            for (int i = 0; i < D / 16; ++i)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    *(float2*)so_at(warp, 8 * b + 2 * cl + e, 2 * i + (gl >> 2), 2 * (gl & 3)) =
                        make_float2(o[b][i][e], o[b][i][2 + e]);
            if (gl == 0) {
                s_ml[warp][8 * b + 2 * cl] = make_float2(m[b][0], l[b][0]);
                s_ml[warp][8 * b + 2 * cl + 1] = make_float2(m[b][1], l[b][1]);
            }
        }
        warps_bar();
        for (int i = tid; i < p.rows * (D / 4); i += 32 * kWarps) {
            const int r = i / (D / 4), c = i % (D / 4);
            float M = -INFINITY, L = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) M = fmaxf(M, s_ml[w][r].x);
            const float ref = M == -INFINITY ? 0.f : M;
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float f = fast_exp2(s_ml[w][r].x - ref);
                const float4 a = *(const float4*)so_at(w, r, c >> 1, 4 * (c & 1));
                L = fmaf(f, s_ml[w][r].y, L);
                v.x = fmaf(f, a.x, v.x), v.y = fmaf(f, a.y, v.y);
                v.z = fmaf(f, a.z, v.z), v.w = fmaf(f, a.w, v.w);
            }
            if (whole_unit) {
                finish<D, F16>(p, out_row(p, at.b, at.g, r), c, r / p.G <= n, v, M, L);
            } else {
                float* to = mine + r * (D + 4);
                *(float4*)&to[4 * c] = v;
                if (c == 0) *(float2*)&to[D] = make_float2(M, L);
            }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar_empty[it % NS]);
        t += left;
        if (t < t_end) next_unit(at);
    }
    pdl_trigger();
}

template <int D, bool F16, int NB>
cudaError_t launch_rows(const Q8AttnArgs& a, cudaStream_t s) {
    using C = CfgQ<D, NB>;
    static std::once_flag once[64];
    static cudaError_t attr_err[64];
    int dev = 0;
    cudaGetDevice(&dev);
    std::call_once(once[dev & 63], [&] {
        attr_err[dev & 63] = cudaFuncSetAttribute(tree_attn_q8_rows_kernel<D, F16, NB>,
                                                  cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    });
    if (attr_err[dev & 63] != cudaSuccess) return attr_err[dev & 63];
    const Q8Args& c = a.cache;
    const int Hq = a.q.heads, Hkv = c.Hkv, G = Hq / Hkv, R = a.N + 1;
    CUtensorMap mkc, mvc, mkt, mvt;
    const uint64_t tokens = (uint64_t)a.B * R;
    if (!tree_map<D>(&mkt, a.k_tree, tokens, 1, R, F16) || !tree_map<D>(&mvt, a.v_tree, tokens, 1, R, F16) ||
        !code_map<D>(&mkc, c, c.k, kTile, true) || !code_map<D>(&mvc, c, c.v, kTile, true))
        return cudaErrorInvalidValue;
    ParamsQ p{};
    p.prefix_len = a.prefix_len;
    p.n_nodes = a.n_nodes;
    p.table = c.table;
    p.anc_mask = a.anc_mask;
    p.out = (uint16_t*)a.out;
    p.lse = a.lse;
    const int ctas = 2 * num_sms();
    p.cut = (int4*)a.ws;
    p.part = (float*)((char*)a.ws + align_up((size_t)ctas * sizeof(int4), 256));
    p.table_stride = c.table_stride;
    p.cap = (int64_t)c.max_pages * c.page_size;
    p.B = a.B, p.N = a.N, p.Hq = Hq, p.Hkv = Hkv, p.G = G, p.rows = R * G;
    p.num_pages = c.num_pages;
    for (p.ps_log2 = 0; (1 << p.ps_log2) < c.page_size;) ++p.ps_log2;
    p.scale_log2 = a.scale * kLog2e;
    p.err = a.err;
    p.q = (const uint16_t*)a.q.data;
    p.q_ts = a.q.ts, p.q_hs = Hq > 1 ? a.q.hs : D;
    p.k_scales = c.k_scales;
    p.v_scales = c.v_scales;
    for (p.block_log2 = 0; (1 << p.block_log2) < c.block;) ++p.block_log2;
    p.per_page_log2 = p.ps_log2 - p.block_log2;
    if (const cudaError_t e = launch_pdl(tree_attn_q8_rows_kernel<D, F16, NB>, dim3(ctas), dim3(kThreadsR),
                                         (size_t)C::SMEM, s, mkc, mvc, mkt, mvt, p))
        return e;
    return launch_pdl(tree_attn_join_kernel<D, F16>, dim3(ctas, (p.rows + 3) / 4), dim3(2 * D), 0, s, (const ParamsR&)p);
}

template <int D, bool F16>
cudaError_t launch_nb(const Q8AttnArgs& a, cudaStream_t s) {
    const int rows = (a.N + 1) * (a.q.heads / a.cache.Hkv);
    return rows <= 8 ? launch_rows<D, F16, 1>(a, s) : launch_rows<D, F16, 2>(a, s);
}

}  // namespace

bool q8_few_rows(int B, int N, int Hq, int Hkv, int64_t cache_cap) {
    return (int64_t)(N + 1) * (Hq / Hkv) <= 16 && B <= kMaxSeqs && B * (cache_cap / kTile + 2) <= INT32_MAX;
}

cudaError_t launch_tree_attn_q8_rows(const Q8AttnArgs& a, cudaStream_t s) {
    const bool f16 = a.cache.dtype == 2;
    if (a.cache.D == 128) return f16 ? launch_nb<128, true>(a, s) : launch_nb<128, false>(a, s);
    return f16 ? launch_nb<64, true>(a, s) : launch_nb<64, false>(a, s);
}

}  // namespace ddt
