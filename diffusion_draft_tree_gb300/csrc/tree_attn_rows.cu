// tree_attn_rows.cu -- ddtree_tree_attn_paged for few query rows: plain decoding
// (N = 0, the G query heads of a KV head are the rows) and small trees, up to
// kMaxRows = (N + 1) G rows a unit (sequence, KV head).
//
//   out[r] = sum_j 2^(x_rj - m_r) v_j / sum_j 2^(x_rj - m_r),  x = scale log2e q k
//
// HBM-bound: a key and its value are 4 D bytes and 4 rows D flops, far below the
// ridge, so the kernel's job is to keep copies in flight and to give every SM
// the same number of bytes.  All key tiles (64 keys) of all units are one list;
// each CTA takes an equal run of it, whatever the sequences' lengths, reading
// the lengths itself.  A unit cut by a run's end leaves (m, l, O) in 32 bits in
// the workspace, at most two pieces a CTA, and a second kernel, whose launch
// overlaps the first's end, joins each cut unit's pieces in the list's order.
//
// A CTA is one copy warp and four computing warps; two CTAs share an SM.  The
// copy warp runs through the list ahead of them with TMA, pages and unit
// borders included.  A 128-row tcgen05 tile would be 3 to 13 % full here and
// would pass its scores through tensor memory for the privilege; the rows fit
// one m16 operand of mma.sync instead, so a warp keeps its own 16 keys' scores,
// weights, statistics and output in registers and meets the others at a unit's
// end only, in the last tile's stage.
#include "tree_attn_common.cuh"

namespace ddt {

namespace {

using namespace sm100;

constexpr int kTile = 64;       // keys per tile
constexpr int kWarps = 4;       // computing warps
constexpr int kThreadsR = 32 * (kWarps + 1);
constexpr int kMaxSeqs = 1024;  // sequences whose tile counts a CTA adds up
constexpr int kFewRows = 32;    // rows of a unit, at most
// A batch of at most kSmallRuns tiles a CTA is cut at unit borders instead, where
// runs of kMaxRun tiles suffice for that.
constexpr int kSmallRuns = 16, kMinRun = 3, kMaxRun = 24;

template <int D, int MB>
struct CfgR {
    static constexpr int NH = D / 64;                // 128-byte-swizzled slabs of a row
    static constexpr int SLAB = kTile * 128;
    static constexpr int KV = NH * SLAB;             // a tile's K (or V)
    static constexpr int STAGE = 2 * KV;
    static constexpr int NS = D == 128 ? 3 : 6;
    static constexpr int QSLAB = MB * 16 * 128;
    static constexpr int SMEM = 1024 + NS * STAGE + NH * QSLAB;
    static_assert(kWarps / MB * 16 * D * 4 <= STAGE, "a stage holds a row block's outputs");
};

struct ParamsR {
    const int32_t *prefix_len, *n_nodes, *table;
    const uint32_t* anc_mask;
    uint16_t* out;
    float* lse;
    float* part;  // [CTA][2][rows][D + 4]: O, m, l, padding to 16 bytes
    int4* cut;    // [CTA]: the unit that is cut by the end of the CTA's run
    int64_t table_stride, cap;
    int B, N, Hq, Hkv, G, rows, num_pages, ps_log2;
    float scale_log2;
    uint32_t* err;
};

// Named barrier over the computing warps.
DDT_DEV void warps_bar() { asm volatile("bar.sync 1, %0;" ::"n"(32 * kWarps) : "memory"); }

// One output value group: columns [4 c, 4 c + 4) of row r (of `row`, counted over
// the whole output), from the sums over all keys.
template <int D, bool F16>
DDT_DEV void finish(const ParamsR& p, size_t row, int c, bool live, float4 v, float M, float L) {
    live = live && L > 0.f;
    const float inv = live ? 1.f / L : 0.f;
    uint2 w = make_uint2(pack16<F16>(v.x * inv, v.y * inv), pack16<F16>(v.z * inv, v.w * inv));
    if (!live) w = make_uint2(0, 0);
    reinterpret_cast<uint2*>(p.out + row * D)[c] = w;
    if (c == 0 && p.lse) p.lse[row] = live ? (M - kLift<F16> + __log2f(L)) * 0.6931471805599453f : -INFINITY;
}
// Row of the output that is row r of unit (b, g).
DDT_DEV size_t out_row(const ParamsR& p, int b, int g, int r) {
    return ((size_t)b * (p.N + 1) + r / p.G) * p.Hq + g * p.G + r % p.G;
}

// MB: 16-row blocks of query rows (1 or 2).  Warp w computes row block w % MB
// against the 16-key groups w / MB, w / MB + 4 / MB, ... of every tile.
template <int D, bool F16, int MB>
__global__ void __launch_bounds__(kThreadsR, 2)
tree_attn_rows_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_kc,
                      const __grid_constant__ CUtensorMap tm_vc,
                      const __grid_constant__ CUtensorMap tm_kt,
                      const __grid_constant__ CUtensorMap tm_vt, const __grid_constant__ ParamsR p) {
    using C = CfgR<D, MB>;
    constexpr int NS = C::NS, NH = C::NH;
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t bar_full[NS], bar_empty[NS], bar_qfull, bar_qempty;
    __shared__ int s_cum[kMaxSeqs + 1];  // key tiles of a KV head, summed over sequences
    __shared__ uint8_t s_rem[kMaxSeqs];  // keys of a sequence's last prefix tile (64: also none)
    __shared__ uint8_t s_nodes[kMaxSeqs];
    __shared__ uint8_t s_pad[kMaxSeqs];  // tiles added to a unit to make its runs equal
    __shared__ int s_chunk;
    __shared__ float2 s_ml[kWarps][16];
    __shared__ volatile int s_abort;
    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // known to be one number a warp
    const uint32_t base_u32 = (smem_u32(smem_raw) + 1023u) & ~1023u;
    uint8_t* base = smem_raw + (base_u32 - smem_u32(smem_raw));
    uint8_t* sq = base + NS * C::STAGE;

    if (tid == 0) {
        for (int s = 0; s < NS; ++s) {
            mbar_init(&bar_full[s], 1);
            mbar_init(&bar_empty[s], kWarps);
        }
        mbar_init(&bar_qfull, 1);
        mbar_init(&bar_qempty, kWarps);
        s_abort = 0;
        mbar_init_fence();
        tma_prefetch_desc(&tm_q);
        tma_prefetch_desc(&tm_kc);
        tma_prefetch_desc(&tm_vc);
        tma_prefetch_desc(&tm_kt);
        tma_prefetch_desc(&tm_vt);
    }
    pdl_wait();

    // ---- the list: tiles of every sequence, added up ---------------------------
    const int R = p.N + 1;
    for (int b = tid; b < p.B; b += kThreadsR) {
        const int P = p.prefix_len[b], n = p.n_nodes[b];
        int t = 0;
        if (P >= 0 && P <= p.cap && n >= 0 && n <= p.N)
            t = (int)((P + (int64_t)kTile - 1) / kTile) + 1;  // (a tree is one tile)
        else if (blockIdx.x == 0)
            record_error(p.err, ERR_ATTN | (n < 0 || n > p.N ? ERR_BAD_N_NODES : ERR_BAD_PREFIX_LEN));
        s_cum[b + 1] = t;
        s_rem[b] = (uint8_t)((P - 1) % kTile + 1 + (P == 0 ? kTile : 0));
        s_nodes[b] = (uint8_t)n;
    }
    __syncthreads();
    // Each CTA's run is `chunk` tiles.  A large batch is cut anywhere; in a small
    // one, where crossing into another unit costs more than an uneven last run,
    // units are padded to whole runs of the least length, at least kMinRun, for which
    // the grid suffices.
    if (warp == 0) {
        int sum = 0;
        for (int b = lane; b < p.B; b += 32) sum += s_cum[b + 1];
        sum = __reduce_add_sync(0xffffffffu, sum);
        const int64_t all = (int64_t)sum * p.Hkv;
        int c = (int)((all + gridDim.x - 1) / gridDim.x);
        bool small = false;
        if (c <= kSmallRuns) {
            int k = max(c, kMinRun);
            for (; !small && k <= kMaxRun; ++k) {
                int runs = 0;
                for (int b = lane; b < p.B; b += 32) runs += (s_cum[b + 1] + k - 1) / k;
                small = (int64_t)__reduce_add_sync(0xffffffffu, runs) * p.Hkv <= gridDim.x;
            }
            if (small) c = k - 1;
        }
        int carry = 0;
        for (int b0 = 0; b0 < p.B; b0 += 32) {
            const int t = b0 + lane < p.B ? s_cum[b0 + lane + 1] : 0;
            const int pad = small ? (c - t % c) % c : 0;
            int v = t + pad;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int up = __shfl_up_sync(0xffffffffu, v, o);
                if (lane >= o) v += up;
            }
            if (b0 + lane < p.B) {
                s_cum[b0 + lane + 1] = v + carry;
                s_pad[b0 + lane] = (uint8_t)pad;
            }
            carry += __shfl_sync(0xffffffffu, v, 31);
        }
        if (lane == 0) {
            s_cum[0] = 0;
            s_chunk = c;
        }
    }
    __syncthreads();
    const int64_t total = (int64_t)s_cum[p.B] * p.Hkv, chunk = s_chunk;
    const int64_t t_begin = blockIdx.x * chunk;
    int64_t t_end = min(total, t_begin + chunk);
    if (t_begin >= t_end) {
        if (tid == 0) p.cut[blockIdx.x] = make_int4(0, 0, 0, 0);
        return;
    }

    // A place in the list: sequence, KV head, tile of the unit.
    struct Place {
        int b, g;
        int tile, tiles;  // ... of the unit
    };
    auto prefix_of = [&](const Place& x) { return (x.tiles - 2) * kTile + s_rem[x.b]; };
    auto place_of = [&](int64_t t) {
        int lo = 0, hi = p.B - 1;  // the last sequence that starts at or before t
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if ((int64_t)s_cum[mid] * p.Hkv <= t) lo = mid;
            else hi = mid - 1;
        }
        Place x;
        x.b = lo;
        const int span = s_cum[lo + 1] - s_cum[lo];
        const int64_t off = t - (int64_t)s_cum[lo] * p.Hkv;
        x.g = (int)(off / span);
        x.tile = (int)(off - (int64_t)x.g * span);
        x.tiles = span - s_pad[lo];
        return x;
    };
    auto next_unit = [&](Place& x) {
        x.tile = 0;
        if (++x.g == p.Hkv) {
            x.g = 0;
            do ++x.b; while (s_cum[x.b + 1] == s_cum[x.b]);  // (there is one: t < t_end)
            x.tiles = s_cum[x.b + 1] - s_cum[x.b];
        }
    };
    auto fail = [&]() {
        record_error(p.err, ERR_ATTN | ERR_WAIT_TIMEOUT);
        s_abort = 1;
    };
    Place at = place_of(t_begin);
    if (s_pad[at.b]) t_end = min(t_end, t_begin + at.tiles - at.tile);  // (the padding)

    if (warp == kWarps) {
        // ============================= copy warp =============================
        const int ps = 1 << p.ps_log2, box = min(ps, kTile), nb = kTile / box;
        const uint32_t lead = elect_one();
        // Page numbers come 32 boxes at a time, lane l holding box 32 k + l of its
        // unit; the batch after that -- of this unit or the next -- is in flight, and
        // nothing looks at it before a tile of it is due.  From the pool's end a copy
        // reads zeros: pages outside the pool.
        struct Batch {
            Place x;
            int k;
            int64_t left;  // tiles of the run from the unit's first (or the run's) tile on
        };
        auto ids_of = [&](const Batch& y) {
            const int64_t key = ((int64_t)y.k * 32 + lane) * box;
            return key < prefix_of(y.x) ? __ldg(&p.table[y.x.b * p.table_stride + (key >> p.ps_log2)])
                                        : p.num_pages;
        };
        auto checked = [&](int page, const Batch& y) {
            if ((unsigned)page < (unsigned)p.num_pages) return page;
            if (((int64_t)y.k * 32 + lane) * box < prefix_of(y.x))
                record_error(p.err, ERR_ATTN | ERR_BAD_PAGE);
            return p.num_pages;
        };
        auto advance = [&](Batch& y) {
            if (((int64_t)y.k + 1) * 32 * box < prefix_of(y.x)) {
                ++y.k;
            } else {
                y.k = 0;
                y.left -= y.x.tiles - y.x.tile;
                if (y.left > 0) next_unit(y.x);
            }
        };
        Batch ahead{at, (int)((int64_t)at.tile * nb / 32), t_end - t_begin};
        int ids = checked(ids_of(ahead), ahead), next_ids = -1;
        advance(ahead);
        if (ahead.left > 0) next_ids = ids_of(ahead);
        int units = 0, issued = 0;
        for (int64_t t = t_begin; t < t_end; ++t) {
            const int it = (int)(t - t_begin), s = it % NS;
            if (t > t_begin) {
                const bool same = ++at.tile < at.tiles;
                if (!same) next_unit(at);
                if (!same || (at.tile * nb % 32 == 0 && at.tile < at.tiles - 1)) {
                    ids = checked(next_ids, ahead);
                    advance(ahead);
                    if (ahead.left > 0) next_ids = ids_of(ahead);
                }
            }
            const bool first = t == t_begin || at.tile == 0, tree = at.tile == at.tiles - 1;
            const int key0 = at.tile * kTile;
            const int boxes = tree ? 0 : min(nb, (prefix_of(at) - key0 + box - 1) / box);
            bool ok = true;  // (of the warp as a whole)
            if (first) {
                ok = mbar_wait_warp(&bar_qempty, (units & 1) ^ 1, &s_abort);
                if (ok) {
                    if (lane == 0) mbar_arrive_expect_tx(&bar_qfull, NH * p.rows * 128);
                    __syncwarp();
                    for (int h = 0; h < NH; ++h)
                        tma_load_3d_warp(lead, smem_u32(sq) + h * C::QSLAB, &tm_q, &bar_qfull, 64 * h,
                                         at.g * p.G, at.b * R);
                    ++units;
                }
            }
            ok = ok && mbar_wait_warp(&bar_empty[s], ((it / NS) & 1) ^ 1, &s_abort);
            if (!ok) { fail(); break; }
            if (lane == 0)
                mbar_arrive_expect_tx(&bar_full[s], 2 * NH * 128 * (tree ? R : boxes * box));
            __syncwarp();
            uint8_t* dk = base + s * C::STAGE;
            if (tree) {
#pragma unroll
                for (int h = 0; h < NH; ++h) {
                    const uint32_t to = smem_u32(dk) + h * C::SLAB;
                    tma_load_3d_warp(lead, to, &tm_kt, &bar_full[s], 64 * h, at.g, at.b * R);
                    tma_load_3d_warp(lead, to + C::KV, &tm_vt, &bar_full[s], 64 * h, at.g, at.b * R);
                }
            } else {
#pragma unroll 4
                for (int i = 0; i < boxes; ++i) {
                    const int page = __shfl_sync(0xffffffffu, ids, (at.tile * nb + i) & 31);
                    const int row = (key0 + i * box) & (ps - 1);
#pragma unroll
                    for (int h = 0; h < NH; ++h) {
                        const uint32_t to = smem_u32(dk) + h * C::SLAB + i * box * 128;
                        tma_load_4d_warp(lead, to, &tm_kc, &bar_full[s], 64 * h, row, at.g, page);
                        tma_load_4d_warp(lead, to + C::KV, &tm_vc, &bar_full[s], 64 * h, row, at.g, page);
                    }
                }
            }
            issued = it + 1;
        }
        // (where a wait gave up, here or below, no copy may land in memory given back)
        if (units > 0) mbar_wait(&bar_qfull, (units - 1) & 1, nullptr, 100000000ull);
        for (int it = max(0, issued - NS); it < issued; ++it)
            mbar_wait(&bar_full[it % NS], (it / NS) & 1, nullptr, 100000000ull);
        return;
    }

    // ============================ computing warps ============================
    constexpr int KG = kWarps / MB;  // warps along the keys
    const int rb = warp % MB, kg = warp / MB;
    const int r0 = rb * 16 + (lane >> 2), r1 = r0 + 8;  // this thread's two rows
    const int u0 = r0 / p.G, u1 = r1 / p.G;             // ... and their nodes
    const float sl2 = p.scale_log2;
    int units = 0;
    for (int64_t t = t_begin; t < t_end; ++units) {
        // ---- a unit, or the part of it in this CTA's run -------------------------
        const int left = (int)min(t_end - t, (int64_t)(at.tiles - at.tile));
        const bool has_tree = at.tile + left == at.tiles;
        const int P = prefix_of(at), n = s_nodes[at.b];
        uint32_t mask0 = 0u, mask1 = 0u;  // ancestors of the two rows' nodes: R <= 32, one word
        if (has_tree) {
            const uint32_t* m = p.anc_mask + (size_t)at.b * R;
            if (u0 <= n) mask0 = __ldg(&m[u0]);
            if (u1 <= n) mask1 = __ldg(&m[u1]);
        }
        uint32_t qf[D / 16][4];
        // A wait that gives up ends the unit's products, not its barriers: the warps
        // stay together.
        bool ok = mbar_wait_warp(&bar_qfull, units & 1, &s_abort);
        if (!ok) fail();
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
            ldsm_x4(smem_u32(sq) + (kk >> 2) * C::QSLAB +
                        swz(rb * 16 + ((lane >> 3) & 1) * 8 + (lane & 7), (kk & 3) * 2 + (lane >> 4)),
                    qf[kk]);
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar_qempty);
        float o[D / 8][4];
#pragma unroll
        for (int j = 0; j < D / 8; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[j][e] = 0.f;
        float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
        const int it0 = (int)(t - t_begin), it = it0 + left - 1;  // the unit's tiles of the run
        for (int k = 0; ok && k < left; ++k) {
            const int s = (it0 + k) % NS;
            ok = mbar_wait_warp(&bar_full[s], ((it0 + k) / NS) & 1, &s_abort);
            if (!ok) { fail(); break; }
            const bool tree = has_tree && k == left - 1;
            const int lim = tree ? n + 1 : min(kTile, P - (at.tile + k) * kTile);
            uint8_t* vt = base + s * C::STAGE + C::KV;
            const uint32_t ka = smem_u32(base + s * C::STAGE), va = ka + C::KV;
#pragma unroll 1
            for (int kb = kg; kb < kTile / 16; kb += KG) {
                const int key0 = kb * 16;
                if (key0 >= lim) break;  // no keys here or behind
                // ---- scores of 16 keys: two blocks of 8, two chains each -------------
                float x[2][4], y[2][4];
#pragma unroll
                for (int e = 0; e < 4; ++e) x[0][e] = x[1][e] = y[0][e] = y[1][e] = 0.f;
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    uint32_t f[4];
                    ldsm_x4(ka + (kk >> 2) * C::SLAB +
                                swz(key0 + (lane >> 4) * 8 + (lane & 7), (kk & 3) * 2 + ((lane >> 3) & 1)),
                            f);
                    mma16816<F16>(kk & 1 ? y[0] : x[0], qf[kk], f[0], f[1]);
                    mma16816<F16>(kk & 1 ? y[1] : x[1], qf[kk], f[2], f[3]);
                }
                const bool whole = !tree && key0 + 16 <= lim;
                uint32_t see0 = 0xffffu, see1 = 0xffffu;  // keys of the block that the rows see
                if (!whole) {
                    see0 = see1 = key0 + 16 <= lim ? 0xffffu : (1u << (lim - key0)) - 1u;
                    if (tree) {
                        see0 &= mask0 >> key0;
                        see1 &= mask1 >> key0;
                    }
                    // Rows of V past the sequence may hold anything, and 0 x NaN is NaN.
                    if (key0 + 16 > lim) {
                        for (int c = lane; c < (key0 + 16 - lim) * NH * 8; c += 32) {
                            const int row = lim + c / (NH * 8), h = (c >> 3) % NH;
                            *(uint4*)(vt + h * C::SLAB + row * 128 + (c & 7) * 16) = make_uint4(0, 0, 0, 0);
                        }
                        fence_proxy_async_smem();  // (the next copy into the stage comes after)
                        __syncwarp();
                    }
                }
                const int c0 = 2 * (lane & 3);
                float mx0 = -INFINITY, mx1 = -INFINITY;
#pragma unroll
                for (int nbk = 0; nbk < 2; ++nbk)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float v = (x[nbk][e] + y[nbk][e]) * sl2;
                        if (!whole && !(((e < 2 ? see0 : see1) >> (nbk * 8 + c0 + (e & 1))) & 1u)) v = -INFINITY;
                        x[nbk][e] = v;
                        if (e < 2) mx0 = fmaxf(mx0, v);
                        else mx1 = fmaxf(mx1, v);
                    }
#pragma unroll
                for (int d = 1; d < 4; d <<= 1) {
                    mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, d));
                    mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, d));
                }
                // the sums and outputs move to a new maximum only when it is 2^8 larger
                const bool up0 = mx0 > m0 + 8.f, up1 = mx1 > m1 + 8.f;
                if (__any_sync(0xffffffffu, up0 || up1)) {
                    const float f0 = up0 ? fast_exp2(m0 - mx0) : 1.f, f1 = up1 ? fast_exp2(m1 - mx1) : 1.f;
                    m0 = up0 ? mx0 : m0;
                    m1 = up1 ? mx1 : m1;
                    l0 *= f0;
                    l1 *= f1;
#pragma unroll
                    for (int j = 0; j < D / 8; ++j) {
                        o[j][0] *= f0, o[j][1] *= f0;
                        o[j][2] *= f1, o[j][3] *= f1;
                    }
                }
                const float b0 = m0 == -INFINITY ? 0.f : m0 - kLift<F16>, b1 = m1 == -INFINITY ? 0.f : m1 - kLift<F16>;
#pragma unroll
                for (int nbk = 0; nbk < 2; ++nbk) {
                    x[nbk][0] = fast_exp2(x[nbk][0] - b0), x[nbk][1] = fast_exp2(x[nbk][1] - b0);
                    x[nbk][2] = fast_exp2(x[nbk][2] - b1), x[nbk][3] = fast_exp2(x[nbk][3] - b1);
                    l0 += x[nbk][0] + x[nbk][1];
                    l1 += x[nbk][2] + x[nbk][3];
                }
                // ---- the weights, rounded to the cache's type, times V ------------------
                const uint32_t pf[4] = {pack16<F16>(x[0][0], x[0][1]), pack16<F16>(x[0][2], x[0][3]),
                                        pack16<F16>(x[1][0], x[1][1]), pack16<F16>(x[1][2], x[1][3])};
#pragma unroll
                for (int j = 0; j < D / 16; ++j) {
                    uint32_t f[4];
                    ldsm_x4_t(va + (j >> 2) * C::SLAB +
                                  swz(key0 + ((lane >> 3) & 1) * 8 + (lane & 7), (j & 3) * 2 + (lane >> 4)),
                              f);
                    mma16816<F16>(o[2 * j], pf, f[0], f[1]);
                    mma16816<F16>(o[2 * j + 1], pf, f[2], f[3]);
                }
            }
            __syncwarp();
            // (the unit's last stage takes the outputs first)
            if (k < left - 1 && lane == 0) mbar_arrive(&bar_empty[s]);
        }

        // ---- the warps' shares of the unit, joined in its last stage ----------------
        // A row block at a time: [KG][16][D] floats fit a stage for every MB.
#pragma unroll
        for (int d = 1; d < 4; d <<= 1) {
            l0 += __shfl_xor_sync(0xffffffffu, l0, d);
            l1 += __shfl_xor_sync(0xffffffffu, l1, d);
        }
        float* so = reinterpret_cast<float*>(base + (it % NS) * C::STAGE);
        // value (r, 8 j + e) of a warp's 16 rows, its groups of 8 permuted by the row
        // so that the 8 rows a warp stores at once do not share their banks
        auto so_at = [&](int w, int r, int j, int e) { return &so[(w * 16 + r) * D + ((j ^ (r & 7)) << 3) + e]; };
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
#pragma unroll 1
        for (int blk = 0; blk < MB; ++blk) {
            if (rb == blk) {
#pragma unroll
                for (int j = 0; j < D / 8; ++j) {
                    *(float2*)so_at(kg, lane >> 2, j, 2 * (lane & 3)) = make_float2(o[j][0], o[j][1]);
                    *(float2*)so_at(kg, 8 + (lane >> 2), j, 2 * (lane & 3)) = make_float2(o[j][2], o[j][3]);
                }
                if ((lane & 3) == 0) {
                    s_ml[kg][lane >> 2] = make_float2(m0, l0);
                    s_ml[kg][8 + (lane >> 2)] = make_float2(m1, l1);
                }
            }
            warps_bar();
            const int nr = min(16, p.rows - blk * 16);
            for (int i = tid; i < nr * (D / 4); i += 32 * kWarps) {
                const int r = i / (D / 4), c = i % (D / 4);
                float M = -INFINITY, L = 0.f;
#pragma unroll
                for (int w = 0; w < KG; ++w) M = fmaxf(M, s_ml[w][r].x);
                const float ref = M == -INFINITY ? 0.f : M;
                float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int w = 0; w < KG; ++w) {
                    const float f = fast_exp2(s_ml[w][r].x - ref);
                    const float4 a = *(const float4*)so_at(w, r, c >> 1, 4 * (c & 1));
                    L = fmaf(f, s_ml[w][r].y, L);
                    v.x = fmaf(f, a.x, v.x), v.y = fmaf(f, a.y, v.y);
                    v.z = fmaf(f, a.z, v.z), v.w = fmaf(f, a.w, v.w);
                }
                const int row = blk * 16 + r;
                if (whole_unit) {
                    finish<D, F16>(p, out_row(p, at.b, at.g, row), c, row / p.G <= n, v, M, L);
                } else {
                    float* to = mine + row * (D + 4);
                    *(float4*)&to[4 * c] = v;
                    if (c == 0) *(float2*)&to[D] = make_float2(M, L);
                }
            }
            if (blk + 1 < MB) warps_bar();
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar_empty[it % NS]);
        t += left;
        if (t < t_end) next_unit(at);
    }
    pdl_trigger();
}

// Joins the pieces of the units that run ends cut: block (c, y) takes rows 4 y ..
// 4 y + 3 of the unit cut by the end of CTA c's run, whose pieces are slot 1 of c
// and slot 0 of the CTAs after it.  A thread owns 4 columns of a row in every
// second piece, kBatch pieces in flight; the two shares meet in shared memory:
// out = sum_s 2^(m_s - M) O_s / sum_s 2^(m_s - M) l_s.
template <int D, bool F16>
__global__ void __launch_bounds__(2 * D) tree_attn_join_kernel(const __grid_constant__ ParamsR p) {
    constexpr int kBatch = 8, kShares = 2;
    __shared__ float4 s_v[kShares][D];
    __shared__ float2 s_ml[kShares][4];
    pdl_wait();
    const int4 unit = p.cut[blockIdx.x];
    if (unit.z == 0) return;
    const int share = threadIdx.x / D, i = threadIdx.x % D;
    const int r = blockIdx.y * 4 + i / (D / 4), c = i % (D / 4);
    const size_t piece = (size_t)p.rows * (D + 4);
    const float* from = p.part + (size_t)blockIdx.x * 2 * piece + (size_t)min(r, p.rows - 1) * (D + 4);
    float M = -INFINITY, L = 0.f;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k0 = share; k0 < unit.z; k0 += kBatch * kShares) {
        float2 ml[kBatch];
        float4 x[kBatch];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const int s = k0 + k * kShares;
            const float* f = from + (size_t)(2 * s + (s == 0 ? 1 : 0)) * piece;
            ml[k] = s < unit.z ? __ldcg((const float2*)&f[D]) : make_float2(-INFINITY, 0.f);
            x[k] = s < unit.z ? __ldcg((const float4*)&f[4 * c]) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
        float Mn = M;
#pragma unroll
        for (int k = 0; k < kBatch; ++k) Mn = fmaxf(Mn, ml[k].x);
        const float ref = Mn == -INFINITY ? 0.f : Mn, f = fast_exp2(M - ref);
        v.x *= f, v.y *= f, v.z *= f, v.w *= f;
        L *= f;
        M = Mn;
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const float h = fast_exp2(ml[k].x - ref);
            v.x = fmaf(h, x[k].x, v.x), v.y = fmaf(h, x[k].y, v.y);
            v.z = fmaf(h, x[k].z, v.z), v.w = fmaf(h, x[k].w, v.w);
            L = fmaf(h, ml[k].y, L);
        }
    }
    s_v[share][i] = v;
    if (c == 0) s_ml[share][i / (D / 4)] = make_float2(M, L);
    __syncthreads();
    if (share > 0 || r >= p.rows) return;
#pragma unroll
    for (int q = 0; q < kShares; ++q) M = fmaxf(M, s_ml[q][i / (D / 4)].x);
    const float ref = M == -INFINITY ? 0.f : M;
    v = make_float4(0.f, 0.f, 0.f, 0.f);
    L = 0.f;
#pragma unroll
    for (int q = 0; q < kShares; ++q) {
        const float2 ml = s_ml[q][i / (D / 4)];
        const float4 x = s_v[q][i];
        const float h = fast_exp2(ml.x - ref);
        v.x = fmaf(h, x.x, v.x), v.y = fmaf(h, x.y, v.y);
        v.z = fmaf(h, x.z, v.z), v.w = fmaf(h, x.w, v.w);
        L = fmaf(h, ml.y, L);
    }
    finish<D, F16>(p, out_row(p, unit.x, unit.y, r), c, r / p.G <= unit.w, v, M, L);
}

template <int D, bool F16, int MB>
cudaError_t launch_rows(const PagedAttnArgs& a, cudaStream_t s) {
    using C = CfgR<D, MB>;
    static std::once_flag once[64];
    static cudaError_t attr_err[64];
    int dev = 0;
    cudaGetDevice(&dev);
    std::call_once(once[dev & 63], [&] {
        attr_err[dev & 63] = cudaFuncSetAttribute(tree_attn_rows_kernel<D, F16, MB>,
                                                  cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    });
    if (attr_err[dev & 63] != cudaSuccess) return attr_err[dev & 63];
    const int Hq = a.q.heads, Hkv = a.cache.Hkv, G = Hq / Hkv, R = a.N + 1;
    CUtensorMap mq, mkc, mvc, mkt, mvt;
    const PagedArgs& c = a.cache;
    const uint64_t tokens = (uint64_t)a.B * R;
    if (!tree_map<D>(&mq, a.q, tokens, G, R, F16) || !tree_map<D>(&mkt, a.k_tree, tokens, 1, R, F16) ||
        !tree_map<D>(&mvt, a.v_tree, tokens, 1, R, F16) || !page_map<D>(&mkc, c, c.k, kTile, F16) ||
        !page_map<D>(&mvc, c, c.v, kTile, F16))
        return cudaErrorInvalidValue;
    ParamsR p{};
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
    if (const cudaError_t e = launch_pdl(tree_attn_rows_kernel<D, F16, MB>, dim3(ctas), dim3(kThreadsR),
                                         (size_t)C::SMEM, s, mq, mkc, mvc, mkt, mvt, p))
        return e;
    return launch_pdl(tree_attn_join_kernel<D, F16>, dim3(ctas, (p.rows + 3) / 4), dim3(2 * D), 0, s, p);
}

template <int D, bool F16>
cudaError_t launch_mb(const PagedAttnArgs& a, cudaStream_t s) {
    const int rows = (a.N + 1) * (a.q.heads / a.cache.Hkv);
    if (rows <= 16) return launch_rows<D, F16, 1>(a, s);
    return launch_rows<D, F16, 2>(a, s);
}

}  // namespace

// One m16 block of rows (N = 0: G <= 16) always comes here; two do where the units
// alone fill the GPU.  Against the general kernel, D = 128, bf16: 64 sequences of
// 512 to 16384 tokens, 4 to 16 rows 324-331 us against 378-385, 32 rows 345 / 385;
// 256 sequences of 100 to 1000, 4 rows 98 / 182, 32 rows 145 / 183; but 8 units of
// 4096 tokens, 32 rows 15.4 / 12.6 (4 rows 11.7 / 12.5).  (The tile counts are
// added up in 32 bits.)
bool few_rows(int B, int N, int Hq, int Hkv, int64_t cache_cap) {
    const int64_t rows = (int64_t)(N + 1) * (Hq / Hkv);
    return B <= kMaxSeqs && B * (cache_cap / kTile + 2) <= INT32_MAX &&
           (rows <= 16 || (rows <= kFewRows && (int64_t)B * Hkv >= num_sms()));
}

size_t few_rows_workspace_bytes(int N, int Hq, int Hkv, int D) {
    const size_t rows = (size_t)(N + 1) * (Hq / Hkv);
    const size_t ctas = 2 * (size_t)num_sms();
    return align_up(ctas * sizeof(int4), 256) + ctas * 2 * rows * (D + 4) * 4;
}

cudaError_t launch_tree_attn_rows(const PagedAttnArgs& a, cudaStream_t s) {
    const bool f16 = a.cache.dtype == 2;
    if (a.cache.D == 128) return f16 ? launch_mb<128, true>(a, s) : launch_mb<128, false>(a, s);
    return f16 ? launch_mb<64, true>(a, s) : launch_mb<64, false>(a, s);
}

}  // namespace ddt
