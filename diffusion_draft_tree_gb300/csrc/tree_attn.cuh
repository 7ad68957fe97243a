// tree_attn.cuh -- step 3 of a DDTree round: one target layer's attention over
// the draft tree ("Accelerating Speculative Decoding with Block Diffusion Draft
// Trees", abstract and §4.1: every drafted node is verified in one target pass
// with an ancestor-only attention mask; App. B: the pages' runs used a dense
// masked attention because FlashAttention-2 cannot express the pattern).
//
// Work unit = (sequence b, KV head g, pair of query tiles, KV split).  A query
// tile holds 128 rows: 128/G tree nodes x the G query heads that share KV head
// g, so the GQA group turns the tree's (N+1) rows into a real dense
// contraction.  The unit streams its KV range in 128-key tiles: prefix tiles
// from the cache, then (last split only) the tree tiles, where the ancestor
// bitmask is applied.
//
// Per CTA: warp 0 issues TMA loads (Q tiles, K and V tiles, 128-byte swizzled)
// into a 2-3 stage K/V ring; warp 1 owns TMEM and issues tcgen05.mma; two
// groups of four warps (one thread per query row) run the online softmax of
// the two query tiles in the log2 domain, with lazy rescaling (O is rescaled
// only when the row max grows by more than 2^8).  P goes back into TMEM in the
// 16-bit type over the S columns it came from and feeds the P V product directly,
// so shared memory holds only Q, K and V.  The two groups alternate on the tensor
// core: while one exponentiates, the other's products run.  When a unit's
// prefix is split, the splits of few units run as one thread-block cluster and
// merge on chip, those of many units through a workspace.  Every mbarrier wait
// is bounded in wall time; a timeout records an error and the CTA unwinds.
//
// Warps 0 and 1 run their loops whole and issue in one lane, under a predicate:
// addresses and descriptors then stay in uniform registers.  Issued from inside a
// one-lane branch a tile's four products took 3.1 to 3.8 thousand cycles where
// the tensor core needs 2.5; this way they take 2.8 (128-key tiles, D = 128).
//
// The kernel comes in several forms.  kDense reads the prefix from one block per
// sequence.  kPagedBf16 / kPagedFp16 read it from pages: a 128-key tile is
// 128 / page_size copies, one page each, into the same swizzled tile, so nothing
// behind them changes.  These forms also keep a split's partial output in 32 bits
// when splits are merged, sum the unrounded weights (the logsumexp then keeps 32
// bits however few the keys), write -inf over the scores that a row does not see
// instead of masking in the softmax (one code path), take any G <= 128 (a query
// tile holds up to floor(128 / G) nodes) and cut a sequence's tiles by its own
// length rather than by the table's capacity.  kLeftBf16 / kLeftFp16 are those for
// many units with two warps more, for a few rows that whole pairs of tiles leave
// over (left_rows).
#pragma once

#include <mutex>
#include <functional>
#include <algorithm>
#include <vector>
#include <tuple>
#include <type_traits>
#include <map>

#include "tree_attn_common.cuh"

#include "../../include/ddtree.h"

namespace ddt {

namespace {

using namespace sm100;

constexpr int BM = 128;  // query rows per tile
constexpr int BN = 128;  // keys per KV tile
constexpr int kThreads = 320;  // warp 0 TMA, warp 1 MMA, warps 2-9 softmax
constexpr int kHalfBytes = 128 * 128;  // [128 rows][64 bf16], one 128B-swizzled slab
constexpr float kRescaleLog2 = 8.f;
// Column of S_k's TMEM region that holds the bf16 P pairs of keys
// [16 kk, 16 kk + 16): keys 0-95 over the first 48 columns in order, keys
// 96-127 over columns 96-111 (the softmax writes that quarter first, from the
// registers its maximum pass left it in, over its own scores).
DDT_DEV uint32_t p_col(int kk) { return kk < 6 ? (uint32_t)(kk * 8) : (uint32_t)(96 + (kk - 6) * 8); }
constexpr uint32_t kTmemCols = 512;
constexpr int kMaxSplits = 16;  // KV splits of one unit = CTAs of one cluster
constexpr int kMinSplit = 32;       // (many units) key tiles of a split, at least
constexpr int kWays = 3;            // ways of cutting a paged batch's lists that are weighed
constexpr int kRankedSeqs = 96;     // ... sequences, at most
static_assert(kWays * kRankedSeqs <= kThreads, "a thread a sequence and way");
constexpr int kLptMaxItems = 128;  // (sequence, split) items ranked in each CTA, at most
// How the KV splits of a unit combine: a single split stores directly; few
// units run each unit's splits as one cluster and merge on chip; many units
// (clusters would fragment the schedule) merge through a global workspace.
constexpr int kMergeNone = 0, kMergeCluster = 1, kMergeGlobal = 2;

template <int D>
struct Cfg {
    static constexpr int NH = D / 64;
    static constexpr int QT_BYTES = NH * kHalfBytes;  // one 128-row query tile
    static constexpr int KV_BYTES = NH * kHalfBytes;  // one K (or V) tile
    static constexpr int NS = (D == 128) ? 2 : 3;
    static constexpr int SMEM = 1024 + 2 * QT_BYTES + NS * 2 * KV_BYTES;
    // Cluster merge: a split's partial O / l (bf16, both tiles) fills the Q
    // region; its (m, l) rows take the last ML_BYTES of the K/V region, the rest
    // of which receives the peers' slices.
    static constexpr int ML_BYTES = 2 * BM * 8;
    static constexpr int RECV_BYTES = NS * 2 * KV_BYTES - ML_BYTES;
    static_assert(D * 2 * 2 * BM == 2 * QT_BYTES, "partial O fills the Q region");
    // Whether a unit of S splits can receive its slices ...
    static constexpr bool recv_fits(int S) {
        return S * (((D / 8 + S - 1) / S) * 2 * BM * 16 + ML_BYTES) <= RECV_BYTES;
    }
    // ... and every unit of a cluster of S (a short sequence uses fewer splits).
    static constexpr bool recv_fits_upto(int S) {
        for (int s = 2; s <= S; ++s)
            if (!recv_fits(s)) return false;
        return true;
    }
};

// Where the prefix lives, and the 16-bit type of everything; LEFT: with two warps for
// the rows that the query tiles leave over.
constexpr int kDense = 0, kPagedBf16 = 1, kPagedFp16 = 2, kLeftBf16 = 3, kLeftFp16 = 4;
constexpr bool is_left(int mode) { return mode >= kLeftBf16; }
constexpr bool is_f16(int mode) { return mode == kPagedFp16 || mode == kLeftFp16; }
constexpr int threads_of(int mode) { return kThreads + (is_left(mode) ? 64 : 0); }
constexpr int kLeftRows = 8;  // rows left over, at most: the narrow side of mma.sync

struct Params {
    const int32_t* prefix_len;
    const int32_t* n_nodes;
    const uint32_t* anc_mask;
    uint16_t* out;
    float* lse;
    uint32_t* part_o;       // global merge: [B*Hkv*mtiles][smax][D/2][128] bf16 pairs of O / l
    float* part_ml;         // global merge: [B*Hkv*mtiles][smax][2][128]
    unsigned int* tickets;  // global merge: [B*Hkv*mpairs]
    int B, N, Hq, Hkv, G, W, mtiles, mpairs, tps, smax;
    int merge;              // how the KV splits of a unit combine: kMerge*
    int lpt;                // non-cluster plans: CTAs ordered longest split first
    int64_t cache_cap;
    float scale_log2;
    uint32_t* err;
};

struct PagedParams : Params {
    const int32_t* table;  // [B][table_stride] page numbers
    int64_t table_stride;
    int num_pages, ps_log2;  // pages of the pool; log2(positions per page)
    int npt;                 // nodes per query tile, at most BM / G
    int single;              // a unit is one query tile, not a pair
    int share;               // key tiles of a split per 2^16 tiles of the longest list
    int sms;                 // of the device
    // rows left over by the query tiles (LEFT): those of the last nodes, the first of
    // which is mtiles npt
    int left;                // their number
    const uint16_t* q;       // the queries, in rows
    int64_t q_ts, q_hs;
    float* part_left;        // global merge: [B*Hkv][smax][kLeftRows][D + 4] O, m, l
    unsigned int* tickets_left;  // ... [B*Hkv]
};

// Named barrier over the 256 softmax threads (both query tiles).
DDT_DEV void softmax_bar() { asm volatile("bar.sync 1, 256;" ::: "memory"); }
// ... and the AND of `v` over them.
DDT_DEV bool softmax_bar_and(bool v) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
        "bar.red.and.pred q, 1, 256, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)v)
        : "memory");
    return r != 0;
}

// On-chip merge of the paged forms: of the D / 4 four-column chunks, rank o of
// a cluster of S merges [chunk_lo(o), chunk_lo(o + 1)); a split's slice for it is
// chunk_slots chunks of [256 rows][16 bytes], and the (m, l) rows follow the
// slices of all S splits.
template <int D>
__host__ __device__ constexpr int chunk_lo(int o, int S) { return o * (D / 4) / S; }
template <int D>
__host__ __device__ constexpr int chunk_owner(int c, int S) { return ((c + 1) * S - 1) / (D / 4); }
template <int D>
__host__ __device__ constexpr int chunk_slots(int S) { return (D / 4 + S - 1) / S; }
constexpr int kChunk4 = 2 * BM * 16;
template <int D>
constexpr bool merge_fits(int S) {
    return S * (chunk_slots<D>(S) * kChunk4 + Cfg<D>::ML_BYTES) <= Cfg<D>::SMEM - 1024;
}

// A table is as wide as the longest sequence it may ever hold, so a paged batch's
// lists are cut here, where their lengths are known: not at all, at the plan's
// share of the longest one, or at its thirds.  A job -- a piece of a sequence's
// list, for one of its `jobs` units -- costs its tiles and 3, and 8 more for the
// merge if the list is cut; started longest first it begins at (cost of the jobs
// before it) / SMs at the latest.  The way whose latest end comes first is taken.
// Longest first puts the whole pieces before all others, in the sequences' order,
// and then one job of each sequence, its last piece or its list, by length: a
// thread a sequence and way goes over those.
// Against the plan's share alone, cut from a table exactly as wide as the longest
// list (us, 8 KV heads, G = 4, D = 128, bf16): 16 sequences of 1K to 32K, N = 128
// 518 -> 500, N = 127 355 -> 364; 30 of 100 to 16K, N = 100 381 -> 329; 8 of 32K 495 ->
// 500; and under a table 4 times as wide 8 of 32K 624 -> 505.
// Returns the sequence, piece and tiles per piece of the item of rank `rk`, -1 if
// there is none.  `smem` is the kernel's dynamic shared memory, before its first copy
// is issued.  Not inlined: inside the kernel it cost the issuing warps' loops their
// uniform registers (long context 2.56 -> 3.68 ms).
__device__ __noinline__ int3 ranked_item(const int32_t* prefix_len, const int32_t* n_nodes, int B, int N,
                                         int64_t cap, int jobs, int smax, int share, int sms, int rk,
                                         uint8_t* smem) {
    __shared__ int s_end[kWays], s_item[2];
    float* s_cost = reinterpret_cast<float*>(smem);                       // [kWays][kRankedSeqs]
    int* s_whole = reinterpret_cast<int*>(s_cost + kWays * kRankedSeqs);  // [kWays][kRankedSeqs]
    constexpr int kLanes = kRankedSeqs / 32;
    const int tid = threadIdx.x, my_way = tid / kRankedSeqs, i = tid % kRankedSeqs;
    const int ways = smax > 1 ? kWays : 1, Bp = (B + 3) & ~3;
    // every warp reads all lengths, once and at once: this is before everything else
    int P[kLanes], n[kLanes], tot = 0, longest = 1;
#pragma unroll
    for (int k = 0; k < kLanes; ++k) {
        const int at = k * 32 + (tid & 31);
        P[k] = at < B ? prefix_len[at] : -1;
        n[k] = at < B ? n_nodes[at] : -1;
    }
#pragma unroll
    for (int k = 0; k < kLanes; ++k) {
        const bool ok = P[k] >= 0 && P[k] <= cap && n[k] >= 0 && n[k] <= N;
        const int t = ok ? (P[k] + BN - 1) / BN + (n[k] + BN) / BN : 0;
        longest = max(longest, t);
        if (i / 32 == k) tot = t;
    }
    longest = __reduce_max_sync(0xffffffffu, longest);
    auto length = [&](int way) {
        return way == 0 ? longest
                        : max(kMinSplit, way == 1 ? (int)(((int64_t)longest * share + 65535) >> 16) : (longest + 2) / 3);
    };
    const bool mine = my_way < ways && i < Bp;
    const int len = length(my_way);
    // pieces of `len` before the last: no way has more pieces than the plan, at most 4
    const int whole = (tot > len ? 1 : 0) + (tot > 2 * len ? 1 : 0) + (tot > 3 * len ? 1 : 0);
    const float cost = i < B ? (tot > 0 ? (float)(tot - whole * len + (whole ? 11 : 3)) : 0.f) : -1.f;
    if (mine) {
        s_cost[tid] = cost;
        s_whole[tid] = whole;
    }
    if (tid < kWays) s_end[tid] = tid < ways ? 0 : INT32_MAX;
    if (tid < 2) s_item[tid] = -1;
    __syncthreads();
    int rank = 0, wholes = 0, wholes_before = 0;
    if (mine && i < B) {
        float before = 0.f;
        for (int j0 = 0; j0 < Bp; j0 += 4) {
            const float4 c4 = *(const float4*)&s_cost[my_way * kRankedSeqs + j0];
            const int4 w4 = *(const int4*)&s_whole[my_way * kRankedSeqs + j0];
            const float c[4] = {c4.x, c4.y, c4.z, c4.w};
            const int w[4] = {w4.x, w4.y, w4.z, w4.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const bool first = c[k] > cost || (c[k] == cost && j0 + k < i);
                rank += first ? 1 : 0;
                before += first ? c[k] : 0.f;
                wholes += w[k];
                wholes_before += j0 + k < i ? w[k] : 0;
            }
        }
        // (ends times SMs)
        const float one = (float)(len + 11), all = one * wholes;
        float end = (all + before) * jobs + cost * (jobs - 1 + sms);
        if (wholes) end = fmaxf(end, all * jobs + one * (sms - 1));
        atomicMax(&s_end[my_way], __float_as_int(end));  // (not negative: ordered as ints)
    }
    __syncthreads();
    int way = 0;
#pragma unroll
    for (int w = 1; w < kWays; ++w)
        if (s_end[w] < s_end[way]) way = w;
    if (mine && i < B && my_way == way) {
        if (rk >= wholes_before && rk < wholes_before + whole) {
            s_item[0] = i, s_item[1] = rk - wholes_before;
        } else if (rk == wholes + rank) {
            s_item[0] = i, s_item[1] = whole;
        }
    }
    // Copies land in the scratch next, by another proxy: what was stored there comes
    // before them only through this fence, and the barrier for what was read.
    fence_proxy_async_smem();
    __syncthreads();
    return make_int3(s_item[0], s_item[1], length(way));
}

// The rows that a unit's query tiles leave over, at most kLeftRows (N + 1 nodes with N
// a power of two: one node's G rows).  As a query tile of their own, a CTA's lone
// tile, they cost 0.8 of what 256 rows do; here two warps more take them along on
// mma.sync, from the K and V tiles that the pairs read anyway.  The key tiles go round
// the pairs: mma.sync runs beside the pair's tcgen05 products at 32 cycles a product
// and scheduler, so that a tile takes these warps 3.6 thousand cycles where the pair
// needs 2.8 (left out, the products gave 434 us instead of 497 at one pair a unit, the
// shared-memory reads nothing).  Rows are the products' narrow side, S^T = K Q^T and
// O^T += V^T P^T, 8 rows wide instead of 16; 4 warps at an equal share of the
// registers, 128 a thread, spilled (shares moved between warpgroups are untried).
// Warp w takes keys [64 w, 64 w + 64) of a tile, its scores, weights,
// statistics and outputs in registers; K is let go after the scores, V after the
// products, and the copies wait for these warps as for the tensor core.  The two
// meet in shared memory, and the pairs and splits in the workspace: the last of
// them, by an atomic ticket, joins their parts in order.
// us against a lone tile (D = 128, bf16, 8 KV heads, G = 4): 16 sequences of 1K to 32K,
// N = 128 498 -> 421; 8 of 32K 500 -> 412; 16 of 20K, N = 64 428 -> 378; 60 of up to
// 16K, N = 64 622 -> 500.
struct LeftArgs {
    const uint16_t* q;  // row 0 (the first node's first head), and from there by strides
    int64_t q_ts, q_hs;
    const uint32_t* mask;  // its ancestor words
    uint16_t* out;
    float* lse;
    float* part;  // [split][mpair][kLeftRows][D + 4]
    unsigned int* ticket;
    uint64_t *kfull, *kempty, *vfull, *vempty;
    uint8_t *sk, *sv;
    volatile int* abort;
    int W, Hq, G, rows, nodes;  // nodes: live ones among them, may be <= 0
    int n, P, t_begin, nprefix, nt, tree_first, split, splits, mpair, mpairs;
    float sl2;
    uint32_t* err;
};

// Named barrier over the two warps.
DDT_DEV void left_bar() { asm volatile("bar.sync 2, 64;" ::: "memory"); }

template <int D, bool F16>
__device__ __noinline__ void left_rows(const LeftArgs& a) {
    using C = Cfg<D>;
    constexpr int NS = C::NS, NH = C::NH;
    __shared__ __align__(16) float s_o[2][kLeftRows][D + 4];
    __shared__ float2 s_ml[2][kLeftRows];
    __shared__ int s_state;  // bit w: warp w gave up; bit 2: the last part
    const int lane = threadIdx.x & 31, w = (threadIdx.x >> 5) & 1, t = threadIdx.x & 63;
    const int r0 = 2 * (lane & 3), r1 = r0 + 1, u0 = r0 / a.G, u1 = r1 / a.G;  // two rows, their nodes
    const bool live0 = r0 < a.rows && u0 < a.nodes, live1 = r1 < a.rows && u1 < a.nodes;
    if (t == 0) s_state = 0;
    uint32_t q[D / 16][2];  // Q^T, the right operand: row lane / 4
    const int rq = lane >> 2, uq = rq / a.G;
    const uint32_t* row = reinterpret_cast<const uint32_t*>(a.q + uq * a.q_ts + (rq - uq * a.G) * a.q_hs);
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
        for (int e = 0; e < 2; ++e)
            q[kk][e] = rq < a.rows && uq < a.nodes ? __ldg(row + kk * 8 + e * 4 + (lane & 3)) : 0u;
    float o[D / 16][4];  // O^T: columns 16 i + lane / 4 (+ 8), rows r0, r1
#pragma unroll
    for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[i][e] = 0.f;
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
    left_bar();
    bool ok = true;
    int turn = a.t_begin % a.mpairs;
    for (int j = 0; j < a.nt; ++j) {
        const int s = j % NS;
        const bool mine = a.nodes > 0 && turn == a.mpair;
        if (++turn == a.mpairs) turn = 0;
        const bool tree = j >= a.nprefix;
        const int a0 = (a.tree_first + j - a.nprefix) * BN;
        // keys of the warp's 64 that exist, and of those the ones that the rows see
        const int lim = (tree ? a.n + 1 - a0 : a.P - (a.t_begin + j) * BN) - 64 * w;
        if (!mine || lim <= 0) {  // (a tile is let go once it is there: one arrival a copy)
            if (!(ok = mbar_wait_warp(&a.kfull[s], (j / NS) & 1, a.abort))) break;
            if (lane == 0) mbar_arrive(&a.kempty[s]);
            if (!(ok = mbar_wait_warp(&a.vfull[s], (j / NS) & 1, a.abort))) break;
            if (lane == 0) mbar_arrive(&a.vempty[s]);
            continue;
        }
        const bool whole = !tree && lim >= 64;
        uint32_t see0[2], see1[2];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            const int rem = lim - 32 * c;
            see0[c] = see1[c] = rem >= 32 ? ~0u : (rem <= 0 ? 0u : (1u << rem) - 1u);
            if (tree) {
                const int word = a0 / 32 + 2 * w + c;
                see0[c] &= live0 && word < a.W ? __ldg(&a.mask[u0 * a.W + word]) : 0u;
                see1[c] &= live1 && word < a.W ? __ldg(&a.mask[u1 * a.W + word]) : 0u;
            }
        }
        // ---- scores, S^T = K Q^T: 4 blocks of 16 keys --------------------------------------
        if (!(ok = mbar_wait_warp(&a.kfull[s], (j / NS) & 1, a.abort))) break;
        const uint32_t ka = smem_u32(a.sk) + s * C::KV_BYTES, va = smem_u32(a.sv) + s * C::KV_BYTES;
        float x[4][4];
#pragma unroll
        for (int kg = 0; kg < 4; ++kg)
#pragma unroll
            for (int e = 0; e < 4; ++e) x[kg][e] = 0.f;
        {
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                uint32_t f[4][4];
#pragma unroll
                for (int kg = 0; kg < 4; ++kg)
                    ldsm_x4(ka + (kk >> 2) * kHalfBytes +
                                swz(64 * w + kg * 16 + (lane & 15), (kk & 3) * 2 + (lane >> 4)),
                            f[kg]);
#pragma unroll
                for (int kg = 0; kg < 4; ++kg) mma16816<F16>(x[kg], f[kg], q[kk][0], q[kk][1]);
            }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&a.kempty[s]);
        // ---- weights: keys 16 kg + lane / 4 (+ 8) of rows r0, r1 ------------------------------
        float mx0 = -INFINITY, mx1 = -INFINITY;
#pragma unroll
        for (int kg = 0; kg < 4; ++kg)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float v = x[kg][e] * a.sl2;
                const uint32_t see = e & 1 ? see1[kg >> 1] : see0[kg >> 1];
                if (!whole && !((see >> ((kg & 1) * 16 + (lane >> 2) + (e >> 1) * 8)) & 1u)) v = -INFINITY;
                x[kg][e] = v;
                if (e & 1) mx1 = fmaxf(mx1, v);
                else mx0 = fmaxf(mx0, v);
            }
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) {
            mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, d));
            mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, d));
        }
        const bool up0 = mx0 > m0 + kRescaleLog2, up1 = mx1 > m1 + kRescaleLog2;
        if (__any_sync(0xffffffffu, up0 || up1)) {
            const float f0 = up0 ? fast_exp2(m0 - mx0) : 1.f, f1 = up1 ? fast_exp2(m1 - mx1) : 1.f;
            m0 = up0 ? mx0 : m0;
            m1 = up1 ? mx1 : m1;
            l0 *= f0;
            l1 *= f1;
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
                o[i][0] *= f0, o[i][2] *= f0;
                o[i][1] *= f1, o[i][3] *= f1;
            }
        }
        const float b0 = m0 == -INFINITY ? 0.f : m0 - kLift<F16>, b1 = m1 == -INFINITY ? 0.f : m1 - kLift<F16>;
        uint32_t pw[8];  // rounded to the cache's type and turned: keys by twos of row lane / 4
#pragma unroll
        for (int kb = 0; kb < 8; ++kb) {
            const float e0 = fast_exp2(x[kb >> 1][2 * (kb & 1)] - b0), e1 = fast_exp2(x[kb >> 1][2 * (kb & 1) + 1] - b1);
            l0 += e0;  // (the sums take them unrounded)
            l1 += e1;
            pw[kb] = movmatrix_t(pack16<F16>(e0, e1));
        }
        // ---- O^T += V^T P^T ---------------------------------------------------------------------
        if (!(ok = mbar_wait_warp(&a.vfull[s], (j / NS) & 1, a.abort))) break;
        {
            if (lim < 64) {  // rows of V past the sequence may hold anything, and 0 x NaN is NaN
                for (int c = lane; c < (64 - lim) * NH * 8; c += 32) {
                    const int key = 64 * w + lim + c / (NH * 8), h = (c >> 3) % NH;
                    *(uint4*)(a.sv + s * C::KV_BYTES + h * kHalfBytes + key * 128 + (c & 7) * 16) =
                        make_uint4(0, 0, 0, 0);
                }
                fence_proxy_async_smem();  // (the next copy into the stage comes after)
                __syncwarp();
            }
#pragma unroll
            for (int x4 = 0; x4 < 4 * NH; ++x4) {  // keys 16 (x4 / NH) .., columns 64 (x4 % NH) ..
                const int kg = x4 / NH, h = x4 % NH;
                uint32_t f[4][4];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    ldsm_x4_t(va + h * kHalfBytes +
                                  swz(64 * w + kg * 16 + (lane >> 4) * 8 + (lane & 7), i * 2 + ((lane >> 3) & 1)),
                              f[i]);
#pragma unroll
                for (int i = 0; i < 4; ++i) mma16816<F16>(o[4 * h + i], f[i], pw[2 * kg], pw[2 * kg + 1]);
            }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&a.vempty[s]);
    }
    if (!ok && lane == 0) {
        record_error(a.err, ERR_ATTN | ERR_WAIT_TIMEOUT);
        *a.abort = 1;
        atomicOr(&s_state, 1 << w);
    }
    auto finish = [&](int r, int c, float4 v, float M, float L) {
        const bool live = r / a.G < a.nodes && L > 0.f;
        const float inv = live ? 1.f / L : 0.f;
        uint2 y = make_uint2(pack16<F16>(v.x * inv, v.y * inv), pack16<F16>(v.z * inv, v.w * inv));
        if (!live) y = make_uint2(0, 0);
        const size_t at = (size_t)(r / a.G) * a.Hq + r % a.G;
        reinterpret_cast<uint2*>(a.out + at * D)[c] = y;
        if (c == 0 && a.lse) a.lse[at] = live ? (M - kLift<F16> + __log2f(L)) * 0.6931471805599453f : -INFINITY;
    };
    if (a.nodes <= 0) {  // every row is padding: zeros, once
        for (int i = t; a.mpair == 0 && a.split == 0 && i < a.rows * (D / 4); i += 64)
            finish(i / (D / 4), i % (D / 4), make_float4(0.f, 0.f, 0.f, 0.f), 0.f, 0.f);
        return;
    }
    // ---- the two halves of the keys meet --------------------------------------------------------
#pragma unroll
    for (int d = 4; d < 32; d <<= 1) {
        l0 += __shfl_xor_sync(0xffffffffu, l0, d);
        l1 += __shfl_xor_sync(0xffffffffu, l1, d);
    }
#pragma unroll
    for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) s_o[w][e & 1 ? r1 : r0][16 * i + (lane >> 2) + (e >> 1) * 8] = o[i][e];
    if (lane < 4) {
        s_ml[w][r0] = make_float2(m0, l0);
        s_ml[w][r1] = make_float2(m1, l1);
    }
    left_bar();
    const bool fine = (s_state & 3) == 0;
    const int parts = a.splits * a.mpairs, part = a.split * a.mpairs + a.mpair;
    if (fine) {
        for (int i = t; i < a.rows * (D / 4); i += 64) {
            const int r = i / (D / 4), c = i % (D / 4);
            const float2 ml0 = s_ml[0][r], ml1 = s_ml[1][r];
            const float M = fmaxf(ml0.x, ml1.x), ref = M == -INFINITY ? 0.f : M;
            const float f0 = fast_exp2(ml0.x - ref), f1 = fast_exp2(ml1.x - ref);
            const float4 x = *(const float4*)&s_o[0][r][4 * c], y = *(const float4*)&s_o[1][r][4 * c];
            const float4 v = make_float4(f0 * x.x + f1 * y.x, f0 * x.y + f1 * y.y, f0 * x.z + f1 * y.z,
                                         f0 * x.w + f1 * y.w);
            const float L = f0 * ml0.y + f1 * ml1.y;
            if (parts == 1) {
                finish(r, c, v, M, L);
            } else {
                float* to = a.part + ((size_t)part * kLeftRows + r) * (D + 4);
                *(float4*)&to[4 * c] = v;
                if (c == 0) *(float2*)&to[D] = make_float2(M, L);
            }
        }
    }
    if (parts == 1) return;
    __threadfence();
    left_bar();
    // (every part takes its ticket, so that the counter returns to zero)
    if (t == 0 && ticket_is_last(a.ticket, (unsigned)parts)) atomicOr(&s_state, 4);
    left_bar();
    if (!fine || !(s_state & 4)) return;
    for (int i = t; i < a.rows * (D / 4); i += 64) {
        const int r = i / (D / 4), c = i % (D / 4);
        float M = -INFINITY, L = 0.f;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
        for (int s = 0; s < parts; ++s)
            M = fmaxf(M, __ldcg(&a.part[((size_t)s * kLeftRows + r) * (D + 4) + D]));
        const float ref = M == -INFINITY ? 0.f : M;
#pragma unroll 4
        for (int s = 0; s < parts; ++s) {
            const float* from = a.part + ((size_t)s * kLeftRows + r) * (D + 4);
            const float2 ml = __ldcg((const float2*)&from[D]);
            const float4 x = __ldcg((const float4*)&from[4 * c]);
            const float f = fast_exp2(ml.x - ref);
            v.x = fmaf(f, x.x, v.x), v.y = fmaf(f, x.y, v.y);
            v.z = fmaf(f, x.z, v.z), v.w = fmaf(f, x.w, v.w);
            L = fmaf(f, ml.y, L);
        }
        finish(r, c, v, M, L);
    }
}

// One CTA = one (sequence b, KV head g, pair of 128-row query tiles, KV split).
// Warp 0: TMA producer.  Warp 1: TMEM owner and MMA issuer.  Warps 2-5: softmax
// of query tile 0; warps 6-9: softmax of query tile 1.  Per KV tile j the
// tensor core runs S_k = Q_k K_j^T into TMEM columns [128k, 128k+128); softmax
// group k reads S_k, writes P_k (bf16) over the first 64 of those columns, and
// the tensor core runs O_k += P_k V_j with P_k read straight from TMEM.  While
// one group exponentiates, the tensor core works on the other group's tile.
// A unit's key tiles are its prefix tiles followed by its tree tiles; split s
// takes tiles [s tps, (s+1) tps) of that list.
template <int D, int MODE>
__global__ void __launch_bounds__(threads_of(MODE), 1)
tree_attn_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_kc,
                 const __grid_constant__ CUtensorMap tm_vc,
                 const __grid_constant__ CUtensorMap tm_kt,
                 const __grid_constant__ CUtensorMap tm_vt,
                 const std::conditional_t<MODE == kDense, Params, PagedParams> p) {
    using C = Cfg<D>;
    constexpr bool PAGED = MODE != kDense, F16 = is_f16(MODE), LEFT = is_left(MODE);
    constexpr int NS = C::NS;
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t bar_q, bar_kfull[NS], bar_kempty[NS], bar_vfull[NS],
        bar_vempty[NS], bar_sfull[2][2],
        bar_pfull[2][2], bar_odone[2][2], bar_recv, bar_drain;
    __shared__ uint32_t s_tmem;
    __shared__ volatile int s_abort;
    __shared__ bool s_last, s_ok;
    __shared__ float2 s_ml[PAGED ? 2 * BM : 1];  // paged cluster merge: (m, l) of the rows
    __shared__ float2 s_ml1[BM];  // lone tile: (m, l) of the second group's key halves

    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // known to be one number a warp

    // ---- set-up that reads no global memory (overlaps the previous kernel) -------
    if (tid == 0) {
        mbar_init(&bar_q, 1);
        constexpr int readers = LEFT ? 3 : 1;  // the tensor core, and two warps for the rows left over
        for (int s = 0; s < NS; ++s) {
            mbar_init(&bar_kfull[s], 1);
            mbar_init(&bar_kempty[s], readers);
            mbar_init(&bar_vfull[s], 1);
            mbar_init(&bar_vempty[s], readers);
        }
        for (int k = 0; k < 2; ++k) {
            mbar_init(&bar_sfull[k][0], 1);
            mbar_init(&bar_sfull[k][1], 1);
            mbar_init(&bar_pfull[k][0], 128);
            mbar_init(&bar_pfull[k][1], 128);
            mbar_init(&bar_odone[k][0], 1);
            mbar_init(&bar_odone[k][1], 1);
        }
        mbar_init(&bar_recv, 1);
        mbar_init(&bar_drain, 1);
        s_abort = 0;
        mbar_init_fence();
        tma_prefetch_desc(&tm_q);
        tma_prefetch_desc(&tm_kc);
        tma_prefetch_desc(&tm_vc);
        tma_prefetch_desc(&tm_kt);
        tma_prefetch_desc(&tm_vt);
    }
    if (warp == 1) tmem_alloc(&s_tmem, kTmemCols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s_tmem;
    // S_k / P_k at columns 128k; O_k at 256 + D*k
    auto free_tmem = [&]() {  // only on exits where no tcgen05 operation was issued
        if (warp == 1) tmem_dealloc(tmem, kTmemCols);
    };

    // ---- decode the unit.  Cluster plans: a unit's KV splits are consecutive
    // CTAs (one cluster; split == rank in it).  Otherwise the tile pairs that
    // read the same KV range are consecutive CTAs, so they run at the same time
    // and the range comes from DRAM once for all of them.
    // Longest first (p.lpt): the (sequence, split) items are ranked by their key
    // tiles, descending (ties by item), and CTA r * Hkv * mpairs + ... takes the
    // item of rank r, so a ragged batch's long splits start in the first wave
    // and the short ones fill the tail.
    int idx = blockIdx.x;
    int split = 0, mpair, g, b = 0;
    if (p.merge == kMergeCluster) {
        split = idx % p.smax;
        idx /= p.smax;
        mpair = idx % p.mpairs;
        idx /= p.mpairs;
        g = idx % p.Hkv;
        b = idx / p.Hkv;
    } else if (p.lpt) {
        mpair = idx % p.mpairs;
        idx /= p.mpairs;
        g = idx % p.Hkv;  // (idx / Hkv: the item's rank, resolved below)
    } else {
        mpair = idx % p.mpairs;
        idx /= p.mpairs;
        split = idx % p.smax;
        idx /= p.smax;
        g = idx % p.Hkv;
        b = idx / p.Hkv;
    }
    const int R = p.N + 1, G = p.G;
    int tps = p.tps;
    pdl_wait();
    if constexpr (PAGED) {
        if (p.merge != kMergeCluster && p.lpt) {
            const int3 x = ranked_item(p.prefix_len, p.n_nodes, p.B, p.N, p.cache_cap,
                                       p.Hkv * p.mpairs, p.smax, p.share, p.sms, idx / p.Hkv, smem_raw);
            if (x.x < 0) {
                free_tmem();
                return;
            }
            b = x.x, split = x.y, tps = x.z;
        }
    } else if (p.merge != kMergeCluster && p.lpt) {
        // (dynamic shared memory is free until the first copy below is issued)
        int* s_w = reinterpret_cast<int*>(smem_raw);  // [kLptMaxItems] key tiles
        int* s_perm = s_w + kLptMaxItems;              // [kLptMaxItems] item of rank r
        const int items = p.B * p.smax;
        for (int i = tid; i < items; i += kThreads) {
            const int bb = i / p.smax, ss = i - bb * p.smax;
            const int pb = p.prefix_len[bb], nb = p.n_nodes[bb];
            int w = 0;
            if (pb >= 0 && pb <= p.cache_cap && nb >= 0 && nb <= p.N) {
                const int tot = (pb + BN - 1) / BN + (nb + 1 + BN - 1) / BN;
                w = max(0, min(tot, (ss + 1) * p.tps) - ss * p.tps);
            }
            s_w[i] = w;
        }
        __syncthreads();
        for (int i = tid; i < items; i += kThreads) {
            const int wi = s_w[i];
            int rk = 0;
            for (int j = 0; j < items; ++j) {
                const int wj = s_w[j];
                rk += (wj > wi || (wj == wi && j < i)) ? 1 : 0;
            }
            s_perm[rk] = i;
        }
        __syncthreads();
        const int item = s_perm[idx / p.Hkv];
        b = item / p.smax;
        split = item - b * p.smax;
        fence_proxy_async_smem();  // (copies land in the scratch next: see ranked_item)
        __syncthreads();
    }
    if constexpr (PAGED) {
        // One number a warp, which the compiler then keeps in uniform registers: as
        // they were, the 70B-class long context took 2.77 ms, shuffled 2.58, reduced 2.56.
        b = __reduce_max_sync(0xffffffffu, b);
        split = __reduce_max_sync(0xffffffffu, split);
        tps = __reduce_max_sync(0xffffffffu, tps);
    }
    const int P = p.prefix_len[b];
    const int n = p.n_nodes[b];
    if (P < 0 || P > p.cache_cap || n < 0 || n > p.N) {  // (the whole cluster exits here)
        if (tid == 0 && split == 0 && mpair == 0 && g == 0)
            record_error(p.err, ERR_ATTN | (n < 0 || n > p.N ? ERR_BAD_N_NODES : ERR_BAD_PREFIX_LEN));
        free_tmem();
        return;
    }
    const int npt = (P + BN - 1) / BN;      // prefix tiles
    const int ntt = (n + 1 + BN - 1) / BN;  // tree tiles
    int nodes_per_tile = BM / G;
    if constexpr (PAGED) {
        nodes_per_tile = p.npt;
        // the cluster's CTAs share the sequence's own tiles, two or more each
        if (p.merge == kMergeCluster) tps = max(2, (npt + ntt + p.smax - 1) / p.smax);
    }
    const int rows_used = nodes_per_tile * G;  // of a tile's 128 (all of them if dense)
    const int splits = (npt + ntt + tps - 1) / tps;
    int mt0 = 2 * mpair, mt1 = mt0 + 1;
    bool tile1 = mt1 < p.mtiles;                // the second tile exists
    if constexpr (PAGED) {
        if (p.single) mt0 = mpair, mt1 = mt0 + 1, tile1 = false;  // one tile a unit
    }
    const int u00 = mt0 * nodes_per_tile, u01 = mt1 * nodes_per_tile;
    const bool has1 = tile1 && (u01 <= n);      // ... and holds a live node
    // The last query tile of an odd count (R G = 128 m + G r, e.g. N + 1 nodes with
    // N a power of two), unless its few rows are taken along (LEFT), is alone: both softmax groups then work on it, each on
    // one 64-key half of every key tile, and merge their (m, l, O) at the end.
    const bool dual = !LEFT && !tile1;
    const bool two = has1 || dual;              // two S / P / O groups in flight
    // A lone tile's scores take 64 of each group's 128 columns.  The paged forms use
    // the others for the next key tile, whose product then runs while this one is
    // exponentiated.
    const int ahead = PAGED && dual ? 2 : 1;
    auto buffer = [&](int j) { return ahead == 2 ? (uint32_t)(j & 1) * 64u : 0u; };
    // ... and a barrier for each, as either side may then be a tile ahead of the other
    // (a wait tells two phases apart, not three: with one barrier for all tiles, a
    // group at its last tile took the end of the third last for that of its own)
    auto bar_of = [&](int j) { return ahead == 2 ? j & 1 : 0; };
    auto phase_of = [&](int j) { return (uint32_t)(ahead == 2 ? j >> 1 : j) & 1u; };
    if (u00 > n) {  // every query row of both tiles is padding: zeros, once
        if (split == 0) {
            for (int r = tid; r < 2 * BM; r += threads_of(MODE)) {
                int u = u00 + r / G, h = g * G + r % G;
                if constexpr (PAGED) {
                    const int rr = r % BM;
                    u = (r < BM ? u00 : u01) + rr / G, h = g * G + rr % G;
                    if (rr >= rows_used) continue;
                }
                if (u >= R || (r >= BM && !tile1)) continue;
                uint4* o = (uint4*)(p.out + (((size_t)b * R + u) * p.Hq + h) * D);
#pragma unroll
                for (int i = 0; i < D / 8; ++i) o[i] = make_uint4(0, 0, 0, 0);
                if (p.lse) p.lse[((size_t)b * R + u) * p.Hq + h] = -INFINITY;
            }
        }
        free_tmem();
        return;  // (the whole cluster takes this exit: it depends on b and mpair only)
    }
    // (paged) no KV tiles here, but a share of the cluster's merge
    const bool idle = PAGED && p.merge == kMergeCluster && splits > 1 && split >= splits;
    if (split >= splits && !idle) {  // no KV tiles here: only keep the cluster's barrier count
        if (!PAGED && p.merge == kMergeCluster) {
            cluster_sync_relaxed();
            cluster_sync_relaxed();
        }
        free_tmem();
        return;
    }
    const int t_begin = split * tps;
    const int t_end = min(npt + ntt, t_begin + tps);
    const int nprefix = max(0, min(npt, t_end) - t_begin);
    const int tree_first = max(t_begin, npt) - npt;  // first tree tile of this split
    const int nt = t_end - t_begin;                  // >= 1; tiles >= nprefix are tree tiles

    // ---- shared memory carve-up (1024-byte aligned for the 128B swizzle) ----------
    const uint32_t base_u32 = (smem_u32(smem_raw) + 1023u) & ~1023u;
    uint8_t* base = smem_raw + (base_u32 - smem_u32(smem_raw));
    uint8_t* sq = base;                          // two query tiles
    uint8_t* sk = sq + 2 * C::QT_BYTES;          // NS stages of K
    uint8_t* sv = sk + NS * C::KV_BYTES;         // NS stages of V

    auto fail = [&]() {
        record_error(p.err, ERR_ATTN | ERR_WAIT_TIMEOUT);
        s_abort = 1;
    };

    if (idle) {
    } else if (warp == 0) {
        // =========================== TMA producer ===========================
        // The warp keeps together and one lane issues: a lane that polled a barrier for
        // the others, or a lane for each copy, divides the warp, which slowed every
        // warp of its scheduler (long_context_70b over pages 3.2 -> 4.1 ms) and made
        // the copies of 16-row pages the slowest part of the kernel.
        const uint32_t lead = elect_one();
        if (lane == 0) mbar_arrive_expect_tx(&bar_q, (has1 ? 2 : 1) * C::NH * rows_used * 128);
        __syncwarp();
        for (int h = 0; h < C::NH; ++h) {
            tma_load_3d_warp(lead, smem_u32(sq) + h * kHalfBytes, &tm_q, &bar_q, 64 * h, g * G, b * R + u00);
            if (has1)
                tma_load_3d_warp(lead, smem_u32(sq) + C::QT_BYTES + h * kHalfBytes, &tm_q, &bar_q, 64 * h,
                                 g * G, b * R + u01);
        }
        // A paged prefix tile is nb boxes of `box` rows, one page (or part of one)
        // each.  Page numbers come 32 boxes at a time, lane l holding box 32 k + l of
        // the split, the batch after that in flight; nothing looks at them before a
        // tile of theirs is due.  From the pool's end a copy reads zeros: boxes past
        // the prefix, and pages outside the pool.
        int ps = BN, ps_log2 = 0, num_pages = 0;
        const int32_t* table = nullptr;
        if constexpr (PAGED) {
            ps_log2 = p.ps_log2;
            ps = 1 << ps_log2;
            num_pages = p.num_pages;
            table = p.table + b * p.table_stride;
        }
        const int box = min(ps, BN), nb = BN / box;
        auto ids_of = [&](int k) {
            const int x = k * 32 + lane, key = t_begin * BN + x * box;
            return PAGED && x < nprefix * nb && key < P ? __ldg(&table[key >> ps_log2]) : num_pages;
        };
        auto checked = [&](int page, int k) {
            if (!PAGED || (unsigned)page < (unsigned)num_pages) return page;
            const int x = k * 32 + lane;
            if (x < nprefix * nb && t_begin * BN + x * box < P)
                record_error(p.err, ERR_ATTN | ERR_BAD_PAGE);
            return num_pages;
        };
        int ids = checked(ids_of(0), 0), next_ids = ids_of(1);
        int issued[2] = {0, 0};  // tiles of K, of V
        for (int i = 0; i <= nt; ++i) {
            const int ids_v = ids;  // the batch of tile i - 1
            if (PAGED && i > 0 && (i * nb & 31) == 0) {
                ids = checked(next_ids, i * nb / 32);
                next_ids = ids_of(i * nb / 32 + 1);
            }
            // K of tile i, then V of tile i - 1: K and V of a stage come and go
            // separately.  K's half is free again as soon as its tile's scores are
            // formed, so K runs ahead, and the scores wait for half the bytes.
            bool ok = true;
#pragma unroll 1
            for (int v = 0; v < 2; ++v) {
                const int j = i - v, s = j % NS;
                if (j < 0 || j >= nt) continue;
                const CUtensorMap* map = v ? &tm_vc : &tm_kc;
                uint64_t* full = v ? &bar_vfull[s] : &bar_kfull[s];
                const uint32_t to = smem_u32(v ? sv : sk) + s * C::KV_BYTES;
                ok = mbar_wait_warp(v ? &bar_vempty[s] : &bar_kempty[s], ((j / NS) & 1) ^ 1, &s_abort);
                if (!ok) break;
                if (lane == 0) mbar_arrive_expect_tx(full, C::KV_BYTES);
                __syncwarp();
                const int key0 = (t_begin + j) * BN;
                if (j >= nprefix) {
                    const int a0 = (tree_first + j - nprefix) * BN;
#pragma unroll
                    for (int h = 0; h < C::NH; ++h)
                        tma_load_3d_warp(lead, to + h * kHalfBytes, v ? &tm_vt : &tm_kt, full, 64 * h, g,
                                         b * R + a0);
                } else if constexpr (PAGED) {
                    const int mine = v ? ids_v : ids;
#pragma unroll 4
                    for (int x = 0; x < nb; ++x) {
                        const int page = __shfl_sync(0xffffffffu, mine, (j * nb + x) & 31);
                        const int row = (key0 + x * box) & (ps - 1);
#pragma unroll
                        for (int h = 0; h < C::NH; ++h)
                            tma_load_4d_warp(lead, to + h * kHalfBytes + x * box * 128, map, full, 64 * h, row,
                                             g, page);
                    }
                } else {
#pragma unroll
                    for (int h = 0; h < C::NH; ++h)
                        tma_load_3d_warp(lead, to + h * kHalfBytes, map, full, 64 * h, key0, b * p.Hkv + g);
                }
                if (v) issued[1] = j + 1;
                else issued[0] = j + 1;
            }
            if (!ok) { fail(); break; }
        }
        // (where a wait gave up, no copy may land in memory given back)
        mbar_wait(&bar_q, 0, nullptr, 100000000ull);
#pragma unroll
        for (int v = 0; v < 2; ++v)
            for (int j = max(0, issued[v] - NS); j < issued[v]; ++j)
                mbar_wait(v ? &bar_vfull[j % NS] : &bar_kfull[j % NS], (j / NS) & 1, nullptr, 100000000ull);
    } else if (warp == 1) {
        // =========================== MMA issuer =============================
        // The whole warp runs the loop and one lane issues: per key tile j and query
        // tile k, O_k += P_k V_j and then S_k = Q_k K_{j + ahead}^T (which reuses S_k /
        // P_k in that order), each product's descriptors a base plus constants.
        constexpr uint32_t kHalfRows = (BN / 2) * 128;  // bytes of 64 key rows in a slab
        const uint32_t lead = elect_one();
        const uint32_t idesc_qk = idesc_f32<F16>(BM, dual ? BN / 2 : BN, 0, 0);
        constexpr uint32_t idesc_pv = idesc_f32<F16>(BM, D, 0, 1);
        const uint64_t qd = smem_desc_sw128(smem_u32(sq), 16, 1024);
        const uint64_t kd = smem_desc_sw128(smem_u32(sk), 16, 1024);
        const uint64_t vd = smem_desc_sw128(smem_u32(sv), kHalfBytes, 1024);
        const uint32_t k_half = dual ? kHalfRows >> 4 : 0u, q_tile = dual ? 0u : C::QT_BYTES >> 4;
        bool ok = mbar_wait_warp(&bar_q, 0, &s_abort);
#pragma unroll 1
        for (int j = -ahead; ok && j < nt; ++j) {
            const int jq = j + ahead;  // the tile whose scores follow
#pragma unroll 1
            for (int k = 0; ok && k < (two ? 2 : 1); ++k) {
                const uint32_t s_k = tmem + k * BN;
                if (j >= 0) {
                    const int s = j % NS;
                    ok = mbar_wait_warp(&bar_pfull[k][bar_of(j)], phase_of(j), &s_abort);
                    if (k == 0) ok = ok && mbar_wait_warp(&bar_vfull[s], (j / NS) & 1, &s_abort);
                    tc_fence_after();
                    const uint64_t b0 = vd + (uint32_t)(s * (C::KV_BYTES >> 4)) + k * k_half;
                    const uint32_t d0 = tmem + 256 + k * D, a0 = s_k + buffer(j);
#pragma unroll
                    for (int kk = 0; kk < BN / 16; ++kk) {
                        if (dual && kk >= BN / 32) break;  // 64 keys: P columns [0, 32)
                        mma_ts_warp(lead, d0, a0 + p_col(kk), b0 + kk * (2048 >> 4), idesc_pv,
                                    kk > 0 ? 1u : (uint32_t)(j > 0));
                    }
                    mma_commit_warp(lead, &bar_odone[k][bar_of(j)]);
                    if (k == 1 || !two) mma_commit_warp(lead, &bar_vempty[s]);
                }
                if (ok && jq < nt) {
                    const int s = jq % NS;
                    if (k == 0) ok = mbar_wait_warp(&bar_kfull[s], (jq / NS) & 1, &s_abort);
                    tc_fence_after();
                    const uint64_t a0 = qd + k * q_tile;
                    const uint64_t b0 = kd + (uint32_t)(s * (C::KV_BYTES >> 4)) + k * k_half;
                    const uint32_t d0 = s_k + buffer(jq);
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        const uint32_t off = ((kk >> 2) * kHalfBytes + (kk & 3) * 32) >> 4;
                        mma_ss_warp(lead, d0, a0 + off, b0 + off, idesc_qk, kk > 0);
                    }
                    mma_commit_warp(lead, &bar_sfull[k][bar_of(jq)]);
                    if (k == 1 || !two) mma_commit_warp(lead, &bar_kempty[s]);
                }
            }
        }
        if (!ok) fail();
        // (where a wait gave up, here or in another warp, no product may still read
        // memory given back; otherwise the last tile's commit says the same)
        mma_commit_warp(lead, &bar_drain);
        mbar_wait(&bar_drain, 0, nullptr, 100000000ull);
    } else if (LEFT && warp >= 10) {
        if constexpr (LEFT) {
            const int u = p.mtiles * nodes_per_tile;  // the first node left over
            const size_t unit = (size_t)b * p.Hkv + g, row = ((size_t)b * R + u) * p.Hq + g * G;
            LeftArgs a;
            a.q = p.q + ((int64_t)b * R + u) * p.q_ts + (int64_t)g * G * p.q_hs;
            a.q_ts = p.q_ts, a.q_hs = p.q_hs;
            a.mask = p.anc_mask + ((size_t)b * R + u) * p.W;
            a.out = p.out + row * D;
            a.lse = p.lse ? p.lse + row : nullptr;
            a.part = p.part_left + unit * p.smax * p.mpairs * (kLeftRows * (D + 4));
            a.ticket = p.tickets_left + unit;
            a.kfull = bar_kfull, a.kempty = bar_kempty, a.vfull = bar_vfull, a.vempty = bar_vempty;
            a.sk = sk, a.sv = sv;
            a.abort = &s_abort;
            a.W = p.W, a.Hq = p.Hq, a.G = G, a.rows = p.left, a.nodes = n - u + 1;
            a.n = n, a.P = P, a.t_begin = t_begin, a.nprefix = nprefix, a.nt = nt;
            a.tree_first = tree_first, a.split = split, a.splits = splits;
            a.mpair = mpair, a.mpairs = p.mpairs;
            a.sl2 = p.scale_log2;
            a.err = p.err;
            left_rows<D, F16>(a);
        }
    } else {
        // ==================== softmax / epilogue, one thread per query row ====================
        const int k = (warp - 2) >> 2;            // query tile of this group
        const int quarter = warp & 3;
        const int r = quarter * 32 + lane;         // query row == TMEM lane
        const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
        const uint32_t tm_s0 = tmem + lane_off + k * BN;
        const uint32_t tm_o = tmem + lane_off + 256 + k * D;
        const bool mine = (k == 0) || has1;        // this group owns a query tile
        const bool work = mine || dual;            // ... or half of tile 0's keys
        const int key0 = dual ? k * (BN / 2) : 0;  // first key of the group's columns
        const int ncol = dual ? BN / 2 : BN;       // keys per tile of the group
        const int u = (k == 0 || dual ? u00 : u01) + r / G;
        const int hh = g * G + r % G;
        const bool row_used = !PAGED || r < rows_used;
        const bool row_valid = work && (u <= n) && row_used;
        const float sl2 = p.scale_log2;
        // ancestor words of this row for the next tree tile, fetched one tile ahead
        uint32_t am[4] = {0u, 0u, 0u, 0u};
        auto fetch_mask = [&](int tt) {
            const uint32_t* mrow = p.anc_mask + ((size_t)b * R + u) * p.W;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const int wi = tt * (BN / 32) + c;
                am[c] = (row_valid && wi < p.W) ? __ldg(&mrow[wi]) : 0u;
            }
        };
        if (nprefix < nt) fetch_mask(tree_first);
        // O_k *= factor (the running maximum grew by more than 2^8)
        auto rescale_o = [&](float factor) {
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
                uint32_t t[32];
                tmem_ld32(tm_o + c * 32, t);
                tmem_ld_wait(t);
#pragma unroll
                for (int i = 0; i < 32; ++i)
                    t[i] = __float_as_uint(__uint_as_float(t[i]) * factor);
                tmem_st32(tm_o + c * 32, t);
            }
        };
        float m_run = -INFINITY, l = 0.f;          // running max (scaled, log2), sum
        bool ok = true;
        for (int j = 0; work && j < nt; ++j) {
            const int s = j % NS;
            if (!mbar_wait_warp(&bar_sfull[k][bar_of(j)], phase_of(j), &s_abort)) { fail(); ok = false; break; }
            const uint32_t tm_s = tm_s0 + buffer(j);
            tc_fence_after();
            // ---- validity of the tile's keys: one 32-bit mask per 32 columns ----
            // (a whole prefix tile needs none; the last, partial prefix tile keys
            // below the prefix length; a tree tile the row's ancestor bits)
            const bool is_tree = (j >= nprefix);
            const int a0 = (tree_first + j - nprefix) * BN;
            const int lim_t = is_tree ? (n + 1 - a0) : (P - (t_begin + j) * BN);
            const bool key_r_valid = r < lim_t;
            // valid keys among the group's columns (a lone tile's group owns 64: its
            // other columns hold whatever the tensor memory held before)
            const int lim = min(lim_t - key0, ncol);
            bool full = !is_tree && lim >= ncol;
            if constexpr (PAGED) {
                if (!full) {
                    // scores of keys that the row does not see become -inf in place, and
                    // the tile then goes the way of a whole one: one copy of that code
#pragma unroll 1
                    for (int c = 0; c < ncol / 32; ++c) {
                        uint32_t t[32];
                        tmem_ld32(tm_s + 32 * c, t);
                        const int rem = lim - 32 * c, w = c + key0 / 32;
                        uint32_t see = rem >= 32 ? ~0u : (rem <= 0 ? 0u : ((1u << rem) - 1u));
                        if (is_tree) see &= w < 2 ? (w == 0 ? am[0] : am[1]) : (w == 2 ? am[2] : am[3]);
                        tmem_ld_wait(t);
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (!((see >> i) & 1u)) t[i] = 0xff800000u;
                        tmem_st32(tm_s + 32 * c, t);
                    }
                    tmem_st_wait();
                    if (is_tree && j + 1 < nt) fetch_mask(tree_first + j + 1 - nprefix);
                    full = true;
                }
            }
            uint32_t vm[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const int rem = lim - 32 * c;
                vm[c] = rem >= 32 ? ~0u : (rem <= 0 ? 0u : ((1u << rem) - 1u));
            }
            if (!PAGED && is_tree) {
                const bool hi = dual && k == 1;  // keys 64-127: ancestor words 2, 3
#pragma unroll
                for (int c = 0; c < 4; ++c) vm[c] &= (c < 2 && hi) ? am[c + 2] : am[c];
                if (j + 1 < nt) fetch_mask(tree_first + j + 1 - nprefix);
            }
            float sum = 0.f;
            if (PAGED || full) {
                // ---- a whole prefix tile: both passes read S_k in 32-column
                // quarters, the next quarter's TMEM load in flight while the
                // current one is used ----
                uint32_t qa[32], qb[32];
                float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
                auto qmax = [&](const uint32_t (&q)[32]) {
#pragma unroll
                    for (int i = 0; i < 32; ++i) mx[i & 3] = fmaxf(mx[i & 3], __uint_as_float(q[i]));
                };
                tmem_ld32(tm_s, qa);
                tmem_ld_wait(qa);
                tmem_ld32(tm_s + 32, qb);
                qmax(qa);
                tmem_ld_wait(qb);
                if (!dual) {
                    tmem_ld32(tm_s + 64, qa);
                    qmax(qb);
                    tmem_ld_wait(qa);
                    tmem_ld32(tm_s + 96, qb);
                    qmax(qa);
                    tmem_ld_wait(qb);
                }
                qmax(qb);
                const float mt_raw = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
                const float m_new = fmaxf(m_run, mt_raw * sl2);
                const bool resc = m_new > m_run + kRescaleLog2;
                const float m_use = resc ? m_new : m_run;
                const float factor = resc ? fast_exp2(m_run - m_new) : 1.f;
                // O_k is stable here: the commit that signalled S_k covers the
                // previous tile's P_k V product -- unless scores run two tiles ahead.
                if (j >= 1 && __any_sync(0xffffffffu, factor != 1.f)) {
                    if (ahead == 2 && !mbar_wait_warp(&bar_odone[k][bar_of(j - 1)], phase_of(j - 1), &s_abort)) { fail(); ok = false; break; }
                    tc_fence_after();
                    rescale_o(factor);
                }
                l *= factor;
                m_run = m_use;
                // P = 2^(s*scale*log2e - m) as bf16 pairs: quarter c's 32 weights
                // go to columns p_col(2c) .. +16 of S_k, whose scores are read
                // before (the row sum takes the fp32 weights: their bf16 rounding
                // averages out over a whole tile)
                const float neg = (m_use == -INFINITY) ? 0.f : kLift<F16> - m_use;
                float2 acc = make_float2(0.f, 0.f);
                auto qexp = [&](const uint32_t (&q)[32], int c) {
                    uint32_t pk[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const float2 y = ffma2(make_float2(__uint_as_float(q[2 * i]), __uint_as_float(q[2 * i + 1])), sl2, neg);
                        const float2 e = make_float2(fast_exp2(y.x), fast_exp2(y.y));
                        pk[i] = pack16<F16>(e.x, e.y);
                        acc = fadd2(acc, e);
                    }
                    tmem_st16(tm_s + p_col(2 * c), pk);
                };
                if (dual) {  // both quarters are still in registers
                    qexp(qb, 1);
                    qexp(qa, 0);
                } else {
                // the last quarter is still in qb: first, while quarter 0 loads
                tmem_ld32(tm_s, qa);
                qexp(qb, 3);
                tmem_ld_wait(qa);
                tmem_ld32(tm_s + 32, qb);
                qexp(qa, 0);
                tmem_ld_wait(qb);
                tmem_ld32(tm_s + 64, qa);
                qexp(qb, 1);
                tmem_ld_wait(qa);
                qexp(qa, 2);
                }
                sum = acc.x + acc.y;
            } else {
            // ---- pass 1: row max, 64 columns per TMEM wait, four independent chains ----
            float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int c0 = 0; c0 < 4; c0 += 2) {
                uint32_t t[32], t2[32];
                tmem_ld32(tm_s + 32 * c0, t);
                tmem_ld32(tm_s + 32 * c0 + 32, t2);
                tmem_ld_wait(t, t2);
                {
                    const uint32_t m = vm[c0], m2 = vm[c0 + 1];
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        mx[i & 3] = fmaxf(mx[i & 3], ((m >> i) & 1u) ? __uint_as_float(t[i]) : -INFINITY);
                        mx[i & 3] = fmaxf(mx[i & 3], ((m2 >> i) & 1u) ? __uint_as_float(t2[i]) : -INFINITY);
                    }
                }
            }
            const float mt_raw = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
            const float m_new = fmaxf(m_run, mt_raw * sl2);
            const bool resc = m_new > m_run + kRescaleLog2;
            const float m_use = resc ? m_new : m_run;
            const float factor = resc ? fast_exp2(m_run - m_new) : 1.f;
            // O_k is stable here: the commit that signalled S_k covers the
            // previous tile's P_k V product.
            if (j >= 1 && __any_sync(0xffffffffu, factor != 1.f)) rescale_o(factor);
            l *= factor;
            m_run = m_use;

            // ---- pass 2: P = 2^(s*scale*log2e - m) as bf16 pairs, 64 columns at a
            // time, written at the P columns of those keys (p_col), whose scores
            // are all read before they are written
            const float neg = (m_use == -INFINITY) ? 0.f : -m_use;
#pragma unroll 1
            for (int half = 0; half < (dual ? 1 : 2); ++half) {
                uint32_t t0[32], t1[32], pk[32];
                tmem_ld32(tm_s + half * 64, t0);
                tmem_ld32(tm_s + half * 64 + 32, t1);
                tmem_ld_wait(t0, t1);
                // few keys (partial or tree tile): the row sum takes exactly the
                // bf16 weights the P V product sees
                const uint32_t m0 = half ? vm[2] : vm[0], m1 = half ? vm[3] : vm[1];
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const float a = ((m0 >> (2 * i)) & 1u) ? fast_exp2(fmaf(__uint_as_float(t0[2 * i]), sl2, neg)) : 0.f;
                    const float bq = ((m0 >> (2 * i + 1)) & 1u) ? fast_exp2(fmaf(__uint_as_float(t0[2 * i + 1]), sl2, neg)) : 0.f;
                    const float c = ((m1 >> (2 * i)) & 1u) ? fast_exp2(fmaf(__uint_as_float(t1[2 * i]), sl2, neg)) : 0.f;
                    const float d = ((m1 >> (2 * i + 1)) & 1u) ? fast_exp2(fmaf(__uint_as_float(t1[2 * i + 1]), sl2, neg)) : 0.f;
                    pk[i] = pack_bf16x2(a, bq);
                    pk[16 + i] = pack_bf16x2(c, d);
                    sum += (__uint_as_float(pk[i] << 16) + __uint_as_float(pk[i] & 0xffff0000u)) +
                           (__uint_as_float(pk[16 + i] << 16) + __uint_as_float(pk[16 + i] & 0xffff0000u));
                }
                if (half == 0) {
                    tmem_st32(tm_s, pk);
                } else {  // keys 64-95 and 96-127 at their P columns
                    uint32_t lo[16], hi[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        lo[i] = pk[i];
                        hi[i] = pk[16 + i];
                    }
                    tmem_st16(tm_s + p_col(4), lo);
                    tmem_st16(tm_s + p_col(6), hi);
                }
            }
            }
            tmem_st_wait();
            l += sum;
            if (k == 0 && quarter * 32 + 32 > lim_t) {  // (the warp as a whole)
                // key r of this tile is past the sequence: zero its V row so that
                // uninitialised cache memory (possibly NaN) cannot reach O.
                if (!mbar_wait_warp(&bar_vfull[s], (j / NS) & 1, &s_abort)) { fail(); ok = false; break; }
                uint8_t* vrow = sv + s * C::KV_BYTES + r * 128;
                if (!key_r_valid) {
#pragma unroll
                    for (int h = 0; h < C::NH; ++h)
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            *(uint4*)(vrow + h * kHalfBytes + i * 16) = make_uint4(0, 0, 0, 0);
                    fence_proxy_async_smem();
                }
            }
            tc_fence_before();
            mbar_arrive(&bar_pfull[k][bar_of(j)]);
        }

        // ---- epilogue (every softmax thread runs the same barrier sequence) ----
        if (work && ok && !mbar_wait_warp(&bar_odone[k][bar_of(nt - 1)], phase_of(nt - 1), &s_abort)) { fail(); ok = false; }
        // (paged splits in a cluster: everything up to the exchange stays where it is)
        const bool exchange = PAGED && p.merge == kMergeCluster && splits > 1;
        if (exchange) s_ml[k * BM + r] = make_float2(m_run, l);
        else if (dual && k == 1) s_ml1[r] = make_float2(m_run, l);
        const bool all_ok = softmax_bar_and(ok);
        const bool have = all_ok && mine;          // warp-uniform
        tc_fence_after();
        if (dual && have && !exchange) {
            // fold the second group's keys into O_0: O = w0 O_0 + w1 O_1,
            // l = w0 l_0 + w1 l_1, w_k = 2^(m_k - M), 0 for a group without keys
            // (both 0 for a row without keys).  No per-row branch: the TMEM loads
            // and stores are warp-collective.
            const float2 ml1 = s_ml1[r];
            const float M = fmaxf(m_run, ml1.x);
            const float w0 = m_run == -INFINITY ? 0.f : fast_exp2(m_run - M);
            const float w1 = ml1.x == -INFINITY ? 0.f : fast_exp2(ml1.x - M);
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
                uint32_t t0[32], t1[32];
                tmem_ld32(tm_o + c * 32, t0);
                tmem_ld32(tm_o + D + c * 32, t1);
                tmem_ld_wait(t0, t1);
#pragma unroll
                for (int i = 0; i < 32; ++i)
                    t0[i] = __float_as_uint(w0 * __uint_as_float(t0[i]) + w1 * __uint_as_float(t1[i]));
                tmem_st32(tm_o + c * 32, t0);
            }
            tmem_st_wait();
            l = w0 * l + w1 * ml1.y;
            m_run = M;
        }
        const bool row_out = (k == 0 || tile1) && u < R && row_used;
        uint4* dst = (uint4*)(p.out + (((size_t)b * R + u) * p.Hq + hh) * D);
        // writes 32 output columns of this row, scaled by inv
        auto store32 = [&](int c, const float (&v)[32], float inv) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                dst[c * 4 + i] =
                    make_uint4(pack16<F16>(v[8 * i] * inv, v[8 * i + 1] * inv),
                               pack16<F16>(v[8 * i + 2] * inv, v[8 * i + 3] * inv),
                               pack16<F16>(v[8 * i + 4] * inv, v[8 * i + 5] * inv),
                               pack16<F16>(v[8 * i + 6] * inv, v[8 * i + 7] * inv));
        };
        auto store_lse = [&](bool live, float M, float Ls) {
            if (p.lse)
                p.lse[((size_t)b * R + u) * p.Hq + hh] =
                    live ? (M - kLift<F16> + __log2f(Ls)) * 0.6931471805599453f : -INFINITY;
        };
        auto store_zero = [&]() {
            float z[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) z[i] = 0.f;
#pragma unroll
            for (int c = 0; c < D / 32; ++c) store32(c, z, 0.f);
            store_lse(false, 0.f, 0.f);
        };
        if (splits == 1) {
            if (have) {
                const bool live = row_valid && l > 0.f;
                const float inv = live ? 1.f / l : 0.f;
#pragma unroll
                for (int c = 0; c < D / 32; ++c) {
                    uint32_t t[32];
                    tmem_ld32(tm_o + c * 32, t);
                    tmem_ld_wait(t);
                    float v[32];
#pragma unroll
                    for (int i = 0; i < 32; ++i) v[i] = live ? __uint_as_float(t[i]) : 0.f;
                    if (row_out) store32(c, v, inv);
                }
                if (row_out) store_lse(live, m_run, l);
            } else if (all_ok && row_out) {  // a tile of padding rows
                store_zero();
            }
        } else if (exchange) {
            // (the partial stays in TMEM until the peers' shared memory is idle)
            if (tid == 64) s_ok = all_ok;
        } else if (p.merge == kMergeCluster) {
            if (have) {
                // This split's partial into its own shared memory (Q and K/V stages
                // are free: every MMA has completed): O / l as bf16, 8 columns per
                // 16-byte group, [D/8][256 rows]; then (m, l) as float2 [256 rows].
                uint4* part = reinterpret_cast<uint4*>(base);
                const int row2 = k * BM + r;
                const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll 1
                for (int c = 0; c < D / 32; ++c) {
                    uint32_t t[32];
                    tmem_ld32(tm_o + c * 32, t);
                    tmem_ld_wait(t);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        part[(c * 4 + i) * 2 * BM + row2] = make_uint4(
                            pack_bf16x2(__uint_as_float(t[8 * i]) * inv, __uint_as_float(t[8 * i + 1]) * inv),
                            pack_bf16x2(__uint_as_float(t[8 * i + 2]) * inv, __uint_as_float(t[8 * i + 3]) * inv),
                            pack_bf16x2(__uint_as_float(t[8 * i + 4]) * inv, __uint_as_float(t[8 * i + 5]) * inv),
                            pack_bf16x2(__uint_as_float(t[8 * i + 6]) * inv, __uint_as_float(t[8 * i + 7]) * inv));
                }
                reinterpret_cast<float2*>(sk + C::RECV_BYTES)[row2] = make_float2(m_run, l);
            }
            fence_proxy_async_smem();  // the partial leaves by bulk copy (async proxy)
        } else {
            // Global merge (paged: unnormalised O in 32 bits, [D/4][128] float4,
            // rows in use only): partial O / l as bf16 pairs [D/2][128] plus (m, l) in
            // fp32; the last split of the unit (atomic ticket) merges them.
            const size_t tslot = ((size_t)(b * p.Hkv + g) * p.mtiles + mt0 + k) * p.smax;
            if (PAGED && have) {
                float4* po = reinterpret_cast<float4*>(p.part_o) + (tslot + split) * (D / 4) * BM;
#pragma unroll
                for (int c = 0; c < D / 32; ++c) {
                    uint32_t t[32];
                    tmem_ld32(tm_o + c * 32, t);
                    tmem_ld_wait(t);
                    if (row_valid) {
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            po[(c * 8 + i) * BM + r] = make_float4(
                                __uint_as_float(t[4 * i]), __uint_as_float(t[4 * i + 1]),
                                __uint_as_float(t[4 * i + 2]), __uint_as_float(t[4 * i + 3]));
                    }
                }
                p.part_ml[(tslot + split) * 2 * BM + r] = m_run;
                p.part_ml[(tslot + split) * 2 * BM + BM + r] = l;
                __threadfence();
            } else if (have) {
                uint32_t* po = p.part_o + (tslot + split) * (D / 2) * BM;
                const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
                for (int c = 0; c < D / 32; ++c) {
                    uint32_t t[32];
                    tmem_ld32(tm_o + c * 32, t);
                    tmem_ld_wait(t);
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        po[(c * 16 + i) * BM + r] = pack_bf16x2(__uint_as_float(t[2 * i]) * inv,
                                                                __uint_as_float(t[2 * i + 1]) * inv);
                }
                p.part_ml[(tslot + split) * 2 * BM + r] = m_run;
                p.part_ml[(tslot + split) * 2 * BM + BM + r] = l;
                __threadfence();
            }
            softmax_bar();
            if (tid == 64) {
                // every split takes its ticket, also after a timeout, so that the
                // counter returns to zero for the next call
                const bool last = ticket_is_last(&p.tickets[(b * p.Hkv + g) * p.mpairs + mpair],
                                                 (unsigned)splits);
                s_last = all_ok && last;
            }
            softmax_bar();
            if (s_last && mine) {
                // out = sum_s w_s o_s / sum_s w_s, w_s = l_s 2^(m_s - M)
                float M = -INFINITY;
                for (int s2 = 0; s2 < splits; ++s2)
                    M = fmaxf(M, __ldcg(&p.part_ml[(tslot + s2) * 2 * BM + r]));
                const float mref = (M == -INFINITY) ? 0.f : M;
                float Ls = 0.f;
                for (int s2 = 0; s2 < splits; ++s2)
                    Ls += __ldcg(&p.part_ml[(tslot + s2) * 2 * BM + BM + r]) *
                          fast_exp2(__ldcg(&p.part_ml[(tslot + s2) * 2 * BM + r]) - mref);
                const bool live = row_valid && Ls > 0.f;
                const float inv = live ? 1.f / Ls : 0.f;
#pragma unroll 1
                for (int c = 0; c < D / 32; ++c) {
                    float v[32];
#pragma unroll
                    for (int i = 0; i < 32; ++i) v[i] = 0.f;
#pragma unroll 2
                    for (int s2 = 0; live && s2 < splits; ++s2) {
                        const size_t sl = tslot + s2;
                        if constexpr (PAGED) {
                            const float w = fast_exp2(__ldcg(&p.part_ml[sl * 2 * BM + r]) - mref);
                            const float4* q = reinterpret_cast<const float4*>(p.part_o) +
                                              (sl * (D / 4) + c * 8) * BM + r;
                            float4 x[8];
#pragma unroll
                            for (int i = 0; i < 8; ++i) x[i] = __ldcg(&q[i * BM]);
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                v[4 * i] = fmaf(w, x[i].x, v[4 * i]);
                                v[4 * i + 1] = fmaf(w, x[i].y, v[4 * i + 1]);
                                v[4 * i + 2] = fmaf(w, x[i].z, v[4 * i + 2]);
                                v[4 * i + 3] = fmaf(w, x[i].w, v[4 * i + 3]);
                            }
                            continue;
                        }
                        const float w = __ldcg(&p.part_ml[sl * 2 * BM + BM + r]) *
                                        fast_exp2(__ldcg(&p.part_ml[sl * 2 * BM + r]) - mref);
                        const uint32_t* q = p.part_o + sl * (D / 2) * BM + (size_t)(c * 16) * BM + r;
                        uint32_t x[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i) x[i] = __ldcg(&q[i * BM]);
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            v[2 * i] += w * __uint_as_float(x[i] << 16);
                            v[2 * i + 1] += w * __uint_as_float(x[i] & 0xffff0000u);
                        }
                    }
                    if (row_out) store32(c, v, inv);
                }
                if (row_out) store_lse(live, M, Ls);
            }
            if (all_ok && !mine && row_out && split == 0) store_zero();  // padding tile
        }
        tc_fence_before();
    }

    // ---- teardown: every thread arrives here (all waits are bounded) -------------
    tc_fence_before();
    __syncthreads();
    pdl_trigger();
    if constexpr (PAGED && !LEFT) {
        if (p.merge == kMergeCluster && splits > 1) {
            // Every rank of the cluster merges its chunks of the head dimension for
            // all rows, idle ranks too: each split's threads store their rows'
            // unnormalised O, 32 bits a value straight from TMEM, and (m, l) into
            // the owners' shared memory, which no product or copy uses any more;
            // then out = sum_s w_s O_s / sum_s w_s l_s, w_s = 2^(m_s - M).  On a lone
            // tile the two groups fold their halves of the keys on the way out, each
            // for half of the columns, and share the merge.
            const int S = p.smax;
            const uint32_t slot = chunk_slots<D>(S) * kChunk4;
            const uint32_t recv = smem_u32(base), recv_ml = recv + (uint32_t)S * slot;
            const int k = (warp - 2) >> 2, r = (warp & 3) * 32 + lane, tile = dual ? 0 : k;
            const int row2 = tile * BM + r;
            const int u = (tile == 0 ? u00 : u01) + r / G, hh = g * G + r % G;
            const bool mine = tile == 0 || has1;
            const bool row_valid = mine && u <= n && r < rows_used;
            fence_proxy_async_smem();
            cluster_sync();
            if (warp >= 2 && mine && !idle && s_ok) {
                tc_fence_after();
                const uint32_t tm_o = tmem + ((uint32_t)((warp & 3) * 32) << 16) + 256 + tile * D;
                float2 ml = s_ml[row2];
                float w0 = 1.f, w1 = 0.f;
                if (dual) {
                    const float2 ml1 = s_ml[BM + r];
                    const float M = fmaxf(ml.x, ml1.x);
                    w0 = ml.x == -INFINITY ? 0.f : fast_exp2(ml.x - M);
                    w1 = ml1.x == -INFINITY ? 0.f : fast_exp2(ml1.x - M);
                    ml = make_float2(M, w0 * ml.y + w1 * ml1.y);
                }
                const int c_first = dual ? k * (D / 64) : 0, c_last = dual ? c_first + D / 64 : D / 32;
#pragma unroll 1
                for (int c = c_first; c < c_last; ++c) {
                    uint32_t t[32];
                    tmem_ld32(tm_o + c * 32, t);
                    if (dual) {
                        uint32_t t1[32];
                        tmem_ld32(tm_o + D + c * 32, t1);
                        tmem_ld_wait(t, t1);
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            t[i] = __float_as_uint(w0 * __uint_as_float(t[i]) + w1 * __uint_as_float(t1[i]));
                    } else {
                        tmem_ld_wait(t);
                    }
                    if (row_valid) {
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const int cc = c * 8 + i, o = chunk_owner<D>(cc, S);
                            st_dsmem_u32x4(
                                mapa_shared(recv + split * slot + (cc - chunk_lo<D>(o, S)) * kChunk4 +
                                                row2 * 16,
                                            o),
                                make_uint4(t[4 * i], t[4 * i + 1], t[4 * i + 2], t[4 * i + 3]));
                        }
                    }
                }
                if (row_valid && (!dual || k == 0))
                    for (int o = 0; o < S; ++o)
                        st_dsmem_f32x2(mapa_shared(recv_ml + split * C::ML_BYTES + row2 * 8, o), ml);
                tc_fence_before();
            }
            cluster_sync();
            if (warp >= 2 && (tile == 0 || tile1) && u < R && r < rows_used) {
                // (four splits at a time, those past the last with weight 0)
                const float2* ml = reinterpret_cast<const float2*>(base + S * slot) + row2;
                float M = -INFINITY, Ls = 0.f, w[kMaxSplits], ls[kMaxSplits];
#pragma unroll
                for (int s2 = 0; s2 < kMaxSplits; ++s2) {
                    const bool there = row_valid && s2 < splits;
                    const float2 x = there ? ml[s2 * 2 * BM] : make_float2(-INFINITY, 0.f);
                    w[s2] = x.x, ls[s2] = x.y;
                    M = fmaxf(M, x.x);
                }
                const float mref = M == -INFINITY ? 0.f : M;
#pragma unroll
                for (int s2 = 0; s2 < kMaxSplits; ++s2) {
                    w[s2] = fast_exp2(w[s2] - mref);
                    Ls = fmaf(w[s2], ls[s2], Ls);
                }
                const bool live = row_valid && Ls > 0.f;
                const float inv = live ? 1.f / Ls : 0.f;
                uint2* dst = (uint2*)(p.out + (((size_t)b * R + u) * p.Hq + hh) * D);
                const int lo = chunk_lo<D>(split, S), hi = chunk_lo<D>(split + 1, S);
#pragma unroll 1
                for (int c = lo + (dual ? k : 0); c < hi; c += dual ? 2 : 1) {
                    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
                    const float4* x = reinterpret_cast<const float4*>(base + (c - lo) * kChunk4) + row2;
                    if (live) {
#pragma unroll
                        for (int s0 = 0; s0 < kMaxSplits; s0 += 4) {
                            if (s0 < splits) {
                                float4 v[4];
#pragma unroll
                                for (int i = 0; i < 4; ++i) v[i] = x[min(s0 + i, splits - 1) * (slot / 16)];
#pragma unroll
                                for (int i = 0; i < 4; ++i) {
                                    acc.x = fmaf(w[s0 + i], v[i].x, acc.x);
                                    acc.y = fmaf(w[s0 + i], v[i].y, acc.y);
                                    acc.z = fmaf(w[s0 + i], v[i].z, acc.z);
                                    acc.w = fmaf(w[s0 + i], v[i].w, acc.w);
                                }
                            }
                        }
                    }
                    dst[c] = make_uint2(pack16<F16>(acc.x * inv, acc.y * inv),
                                        pack16<F16>(acc.z * inv, acc.w * inv));
                }
                if (split == 0 && p.lse && (!dual || k == 0))
                    p.lse[((size_t)b * R + u) * p.Hq + hh] =
                        live ? (M - kLift<F16> + __log2f(Ls)) * 0.6931471805599453f : -INFINITY;
            }
        }
    } else if (p.merge == kMergeCluster) {
        // Execution order is all that is needed: every split's partial is written
        // and read only by its own copy engine; every K/V stage is idle.
        cluster_sync_relaxed();
        if (splits > 1 && !C::recv_fits(splits)) {  // the plan rules this out
            if (tid == 0 && split == 0) record_error(p.err, ERR_ATTN | ERR_PLAN);
        } else if (splits > 1) {
            // Split o owns head-dimension columns [8 lo(o), 8 hi(o)).  Each CTA's
            // copy engine sends every owner its slice of this CTA's partial and its
            // (m, l) rows, into the owner's (now idle) K/V stages, completing on the
            // owner's bar_recv; the owner then merges from its own shared memory:
            // out = sum_s w_s o_s / sum_s w_s, o_s = O_s / l_s, w_s = l_s 2^(m_s - M).
            constexpr int nch = D / 8;             // 8-column chunks of 256 rows x 16 B
            constexpr uint32_t kChunk = 2 * BM * 16;
            constexpr uint32_t kMl = 2 * BM * 8;
            const int c_lo = split * nch / splits, c_hi = (split + 1) * nch / splits;
            const uint32_t slot = (uint32_t)((nch + splits - 1) / splits) * kChunk;
            const uint32_t part_s = smem_u32(base);
            const uint32_t ml_s = smem_u32(sk + C::RECV_BYTES);
            const uint32_t recv_s = smem_u32(sk);
            const uint32_t recv_ml_s = recv_s + (uint32_t)splits * slot;
            if (tid == 0) {
                mbar_arrive_expect_tx(&bar_recv, (uint32_t)(splits - 1) *
                                                     ((uint32_t)(c_hi - c_lo) * kChunk + kMl));
                for (int i = 1; i < splits; ++i) {
                    const uint32_t o = (uint32_t)((split + i) % splits);
                    const int lo = (int)o * nch / splits, hi = ((int)o + 1) * nch / splits;
                    const uint32_t rbar = mapa_shared(smem_u32(&bar_recv), o);
                    bulk_copy_s2s(mapa_shared(recv_s + (uint32_t)split * slot, o),
                                  part_s + (uint32_t)lo * kChunk, (uint32_t)(hi - lo) * kChunk, rbar);
                    bulk_copy_s2s(mapa_shared(recv_ml_s + (uint32_t)split * kMl, o), ml_s, kMl, rbar);
                }
            }
            if (warp >= 2) {
                const int k = (warp - 2) >> 2;
                const int r = (warp & 3) * 32 + lane;
                const int row2 = k * BM + r;
                const int u = (k == 0 ? u00 : u01) + r / G;
                const int hh = g * G + r % G;
                const bool mine = (k == 0) || has1;
                const bool row_out = (k == 0 || tile1) && u < R;
                const bool row_valid = mine && u <= n;
                if (!mbar_wait_warp(&bar_recv, 0, nullptr) && lane == 0)
                    record_error(p.err, ERR_ATTN | ERR_WAIT_TIMEOUT);
                const float2* mls[kMaxSplits];
                const uint4* prt[kMaxSplits];  // chunk c_lo of each split's slice
#pragma unroll
                for (int s2 = 0; s2 < kMaxSplits; ++s2) {
                    const bool self = s2 == split;
                    mls[s2] = reinterpret_cast<const float2*>(
                        self ? sk + C::RECV_BYTES : sk + splits * slot + s2 * kMl);
                    prt[s2] = reinterpret_cast<const uint4*>(self ? base + c_lo * kChunk
                                                                  : sk + s2 * slot);
                }
                float M = -INFINITY, Ls = 0.f;
                float w[kMaxSplits];
                if (row_valid) {
                    float2 ml[kMaxSplits];
#pragma unroll
                    for (int s2 = 0; s2 < kMaxSplits; ++s2) {
                        ml[s2] = s2 < splits ? mls[s2][row2] : make_float2(-INFINITY, 0.f);
                        M = fmaxf(M, ml[s2].x);
                    }
                    const float mref = (M == -INFINITY) ? 0.f : M;
#pragma unroll
                    for (int s2 = 0; s2 < kMaxSplits; ++s2) {
                        w[s2] = s2 < splits ? ml[s2].y * fast_exp2(ml[s2].x - mref) : 0.f;
                        Ls += w[s2];
                    }
                }
                const bool live = row_valid && Ls > 0.f;
                const float inv = live ? 1.f / Ls : 0.f;
                if (row_out) {
                    uint4* dst = (uint4*)(p.out + (((size_t)b * R + u) * p.Hq + hh) * D);
#pragma unroll 1
                    for (int c = c_lo; c < c_hi; ++c) {
                        float acc[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i) acc[i] = 0.f;
                        if (live) {
#pragma unroll
                            for (int s2 = 0; s2 < kMaxSplits; ++s2) {
                                if (s2 < splits) {
                                    const uint4 x = prt[s2][(c - c_lo) * 2 * BM + row2];
                                    const uint32_t q[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                                    for (int e = 0; e < 4; ++e) {
                                        acc[2 * e] = fmaf(w[s2], __uint_as_float(q[e] << 16), acc[2 * e]);
                                        acc[2 * e + 1] = fmaf(w[s2], __uint_as_float(q[e] & 0xffff0000u), acc[2 * e + 1]);
                                    }
                                }
                            }
                        }
                        dst[c] = make_uint4(pack_bf16x2(acc[0] * inv, acc[1] * inv),
                                            pack_bf16x2(acc[2] * inv, acc[3] * inv),
                                            pack_bf16x2(acc[4] * inv, acc[5] * inv),
                                            pack_bf16x2(acc[6] * inv, acc[7] * inv));
                    }
                    if (split == 0 && p.lse)
                        p.lse[((size_t)b * R + u) * p.Hq + hh] =
                            live ? (M + __log2f(Ls)) * 0.6931471805599453f : -INFINITY;
                }
            }
        }
        cluster_sync_relaxed();  // every copy out of this CTA's shared memory has landed
    }
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

// ------------------------------- host side ---------------------------------------

struct Plan {
    int mtiles, mpairs, tps, smax, merge;
};

// Per-unit tile counts bounding a plan: the longest prefix and the largest tree.
struct Tiles {
    int prefix, tree;
};
Tiles max_tiles(int N, int64_t cache_cap) {
    return {(int)((cache_cap + BN - 1) / BN), (N + 1 + BN - 1) / BN};
}

Plan plan_base(int N, int Hq, int Hkv) {
    Plan pl{};
    const int G = Hq / Hkv;
    const int nodes = BM / G;  // per query tile
    pl.mtiles = (N + 1 + nodes - 1) / nodes;
    pl.mpairs = (pl.mtiles + 1) / 2;
    return pl;
}

long plan_units(const Plan& pl, int B, int Hkv) { return (long)B * Hkv * pl.mpairs; }

// Predicted span of `units` units of T key tiles, each cut into splits of tps
// tiles (the last one shorter), every split a CTA per query-tile pair, the CTAs
// started longest first on `sms` SMs, each costing tiles + 2 (set-up, merge).
long lpt_span(long units, int T, int tps, int sms) {
    std::vector<long> sizes;
    for (int s0 = 0; s0 < T; s0 += tps) sizes.push_back(std::min(T, s0 + tps) - s0 + 2);
    std::sort(sizes.begin(), sizes.end(), std::greater<long>());
    std::map<long, long> sm{{0, sms}};  // load -> SMs that have it: equal pieces go out together
    for (const long z : sizes)
        for (long left = units; left > 0;) {
            const auto [load, idle] = *sm.begin();
            const long take = std::min(idle, left);
            sm.erase(sm.begin());
            if (take < idle) sm[load] = idle - take;
            sm[load + z] += take;
            left -= take;
        }
    return sm.rbegin()->first;
}

// Many units fill the GPU without clusters: split only long tile lists, into
// four pieces merged through the workspace.  The pieces are a quarter of the
// longest list each, unless a longer first three and a short last one pack the
// SMs' waves better: with the CTAs ordered longest first the short ones fill
// the last wave (1152 equal CTAs on 152 SMs leave it 40 % empty).  Every size
// up to just under a third is scored by lpt_span, and the best is taken when
// it beats the quarter by at least 2 %.  The choice assumes every unit as long
// as the longest; it is cached per shape.
// Lists of 64 tiles and fewer stay whole and no piece is shorter than 32: against a
// rule of twice that reach (33 tiles, pieces of 16), us over pages (8 KV heads, G = 4,
// D = 128, bf16): 20 sequences of 8100, N = 63 179 / 186; 24 of 4000, N = 31 and 16 of
// 4000, N = 64 94 / 94 and 92 / 92; 40 of 4000, N = 64 231 / 232; 20 of 100 to 8100,
// N = 63 86 / 95; 40 of 100 to 4000, N = 127 144 / 163.  (A piece's merge costs more
// than the cost model's 8 tiles where pieces are short.)
Plan plan_many(const Plan& base, Tiles t, long units, int sms) {
    Plan pl = base;
    const int T = t.prefix + t.tree;
    pl.tps = T > 64 ? std::max(kMinSplit, (T + 3) / 4) : T;
    if (T > 64 && pl.tps > kMinSplit) {
        static std::mutex mu;
        static std::map<std::tuple<int, long, int>, int> cache;
        std::lock_guard<std::mutex> lock(mu);
        const auto key = std::make_tuple(T, units, sms);
        const auto it = cache.find(key);
        if (it != cache.end()) {
            pl.tps = it->second;
        } else {
            const long quarter = lpt_span(units, T, pl.tps, sms);
            long best = quarter;
            int best_tps = pl.tps;
            for (int tps = pl.tps + 1; (T + tps - 1) / tps == 4; ++tps) {
                const long span = lpt_span(units, T, tps, sms);
                if (span < best) {
                    best = span;
                    best_tps = tps;
                }
            }
            if (best * 100 < quarter * 98) pl.tps = best_tps;  // a clear gain only
            cache[key] = pl.tps;
        }
    }
    pl.smax = (T + pl.tps - 1) / pl.tps;
    pl.merge = pl.smax > 1 ? kMergeGlobal : kMergeNone;
    return pl;
}

// The same over a paged cache, where only the kernel knows how far the lists fall
// short of the table: it takes the plan's share of the longest list (or cuts
// otherwise, see there), and so the plan is made for kPlanTiles tiles at most.
constexpr int kPlanTiles = 2048;
Tiles planned(Tiles t) { return {std::min(t.prefix, kPlanTiles), t.tree}; }

// Few units: split each unit's tiles over a cluster of S CTAs, with the fewest
// tiles per split (at least 2) for which every unit's cluster is resident at
// once: units x S CTAs within one wave, and the device able to co-schedule that
// many clusters of S (active(S) reports how many it can).
template <typename Active>
Plan plan_few(const Plan& base, Tiles t, long units, int sms, Active active) {
    Plan pl = base;
    const int T = t.prefix + t.tree;
    pl.tps = T;
    for (int tps = 2; tps < T; ++tps) {
        const int S = (T + tps - 1) / tps;
        if (S > kMaxSplits || units * S > sms) continue;
        if (active(S) < units) continue;
        pl.tps = tps;
        break;
    }
    pl.smax = (T + pl.tps - 1) / pl.tps;
    pl.merge = pl.smax > 1 ? kMergeCluster : kMergeNone;
    return pl;
}

// Few units, paged: what a CTA's exchange with its cluster costs grows with its
// rows (32-bit partials through distributed shared memory, which passes about 15
// GB/s a CTA: 512 bytes a row of D = 128), so rows are spread over idle SMs too: a unit may be a single query
// tile, and tiles may hold fewer nodes than fit.  Every number of tiles up to
// four times the least and every cluster size that is resident at once is
// scored, in microseconds measured on GB300 (D = 128): a key tile takes a pair
// of query tiles 1.5, a single one 1.2; an exchange 1 and 0.035 a row.  (D = 64, whose
// rows are half as long, goes by the same figures.)
struct PagedPlan : Plan {
    int npt, single;
};
template <typename Active>
PagedPlan plan_paged_few(int B, int N, int G, int Hkv, Tiles t, int sms, Active active) {
    const int R = N + 1, T = t.prefix + t.tree, most = BM / G, least = (R + most - 1) / most;
    PagedPlan best{};
    double best_cost = 1e30;
    for (int tiles = least; tiles <= std::min(R, 4 * least); ++tiles) {
        if (tiles > least && (long)B * Hkv * tiles > sms) break;  // (single from here on)
        const int npt = (R + tiles - 1) / tiles;
        if ((R + npt - 1) / npt != tiles) continue;
        for (int single = tiles == least && tiles > 1 ? 0 : 1; single < 2; ++single) {
            const int per_head = single ? tiles : (tiles + 1) / 2;
            const long units = (long)B * Hkv * per_head;
            for (int S = 1; S <= kMaxSplits && units * S <= sms; ++S) {
                const int per_cta = (T + S - 1) / S;
                if (S > 1 && (per_cta < 2 || active(S) < units)) continue;
                const int rows = npt * G * (single ? 1 : 2);
                const double cost = per_cta * (single ? 1.2 : 1.5) + (S > 1 ? 1.0 + 0.035 * rows : 0.0);
                if (cost >= best_cost) continue;
                best_cost = cost;
                best.mtiles = tiles, best.mpairs = per_head, best.smax = S, best.tps = per_cta;
                best.merge = S > 1 ? kMergeCluster : kMergeNone;
                best.npt = npt, best.single = single;
            }
        }
    }
    return best;
}

// The plan of a paged batch's many units, with the rows that the query tiles leave over
// taken along by the pairs (`left` of them) where that is one operand's worth -- unless
// a unit has one pair, which then takes all of them along, and these units leave a
// good part of the SMs idle while their lists are too short to be cut for them: the
// lone tiles then run on those SMs.  Lone tiles against rows taken along, us (8 KV
// heads, G = 4, N = 64, D = 128, bf16), of lists of 9, 33, 65, 95 and 126 tiles: 10
// sequences (80 units taken along, of 152 SMs) 26 / 35, 59 / 88, 120 / 149, 173 / 176, 220 / 214;
// 12 (96 units) at 65, 95 and 126 tiles 157 / 171, 212 / 179, 266 / 251; 14 (112 units) at 33 and
// 65 tiles 105 / 90, 180 / 175.
constexpr int kLoneTiles = 80;
struct ManyPlan : Plan {
    int left;
};
ManyPlan plan_paged_many(int B, int N, int Hq, int Hkv, Tiles t, int sms) {
    ManyPlan pl{};
    (Plan&)pl = plan_base(N, Hq, Hkv);
    const int G = Hq / Hkv, left = (N + 1 - (pl.mtiles - 1) * (BM / G)) * G;
    if (plan_units(pl, B, Hkv) < sms) return pl;  // few units (smax = 0)
    const long along = (long)B * Hkv * (pl.mpairs - 1);  // units if the pairs take them
    const bool short_wave = pl.mpairs == 2 && along * 10 < sms * 7L && t.prefix + t.tree <= kLoneTiles;
    if (pl.mtiles > 1 && pl.mtiles % 2 && left <= kLeftRows && !short_wave) {
        --pl.mtiles;
        --pl.mpairs;
        pl.left = left;
    }
    (Plan&)pl = plan_many(pl, planned(t), plan_units(pl, B, Hkv), sms);
    return pl;
}

struct WsLayout {
    size_t tickets, part_o, part_ml, tickets_left, part_left, total;
};

// Workspace of the global merge (empty for the other plans); a partial output
// takes `elem` bytes a value.
WsLayout attn_layout(const Plan& pl, int B, int Hkv, int D, int elem, int left = 0) {
    WsLayout w{};
    if (pl.merge != kMergeGlobal && !(left && pl.mpairs > 1)) return w;
    const size_t tiles = (size_t)B * Hkv * pl.mtiles;  // partials per query tile
    if (pl.merge == kMergeGlobal) {
        w.tickets = 0;  // one counter per (sequence, KV head, tile pair)
        w.part_o = align_up((size_t)B * Hkv * pl.mpairs * 4, 256);
        w.part_ml = align_up(w.part_o + tiles * pl.smax * (size_t)D * BM * elem, 256);
        w.total = align_up(w.part_ml + tiles * pl.smax * 2 * BM * 4, 256);
    }
    if (left) {  // (merged over the splits and the pairs)
        const size_t heads = (size_t)B * Hkv;
        w.tickets_left = w.total;
        w.part_left = align_up(w.tickets_left + heads * 4, 256);
        w.total = align_up(w.part_left + heads * pl.smax * pl.mpairs * kLeftRows * (D + 4) * 4, 256);
    }
    return w;
}

// Co-resident clusters of `size` CTAs of tree_attn_kernel<D, MODE> on device `dev`
// (0 if that size cannot launch).  Needs the kernel's attributes set first.
template <int D, int MODE>
int active_clusters(int dev, int size) {
    static std::atomic<int> cached[64][kMaxSplits + 1];  // the number + 1; 0: not asked yet
    if (size < 1 || size > kMaxSplits) return 0;
    int known = cached[dev & 63][size].load(std::memory_order_relaxed);
    if (!known) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)size);
        cfg.blockDim = dim3(kThreads);
        cfg.dynamicSmemBytes = Cfg<D>::SMEM;
        cudaLaunchAttribute at;
        at.id = cudaLaunchAttributeClusterDimension;
        at.val.clusterDim.x = (unsigned)size;
        at.val.clusterDim.y = 1;
        at.val.clusterDim.z = 1;
        cfg.attrs = &at;
        cfg.numAttrs = 1;
        int n = 0;
        if (cudaOccupancyMaxActiveClusters(&n, tree_attn_kernel<D, MODE>, &cfg) != cudaSuccess) {
            n = 0;
            (void)cudaGetLastError();  // a refused size is not an error of the call
        }
        known = n + 1;
        cached[dev & 63][size].store(known, std::memory_order_relaxed);
    }
    return known - 1;
}

// Opts the kernel in to its shared memory and to clusters of 16, once per device.
template <int D, int MODE>
cudaError_t prepare_kernel(int dev) {
    static std::once_flag once[64];
    static cudaError_t attr_err[64];
    std::call_once(once[dev & 63], [&] {
        cudaError_t e = cudaFuncSetAttribute(tree_attn_kernel<D, MODE>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<D>::SMEM);
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(tree_attn_kernel<D, MODE>,
                                     cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        attr_err[dev & 63] = e;
    });
    return attr_err[dev & 63];
}

}  // namespace

}  // namespace ddt
