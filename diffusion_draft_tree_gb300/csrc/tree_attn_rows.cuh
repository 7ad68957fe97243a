// tree_attn_rows.cuh -- what the kernels for few query rows (tree_attn_rows.cu over 16-bit
// pages, tree_attn_q8_rows.cu over 8-bit ones) share: the list of key tiles and its runs,
// a run's pieces in the workspace, and their join.
#pragma once

#include "tree_attn_common.cuh"

namespace ddt {

namespace {

using namespace sm100;

constexpr int kWarps = 4;       // computing warps
constexpr int kThreadsR = 32 * (kWarps + 1);
constexpr int kMaxSeqs = 1024;  // sequences whose tile counts a CTA adds up
// A batch of at most kSmallRuns tiles a CTA is cut at unit borders instead, where
// runs of kMaxRun tiles suffice for that.  Over an 8-bit cache, whose tiles are of 128 keys, the
// rule is kept for want of a clear winner (bf16, 8 KV heads, G = 4; us, cut at unit borders / anywhere):
// N = 0, D = 128, 16 sequences of 500 11.9 / 12.5, 32 of 300 11.7 / 12.9, 4 of 4K 13.9 / 14.0, but one of 500
// 10.3 / 8.7, of 2K 11.3 / 9.7, 64 of 500 25.5 / 22.0; N = 3, 16 of 500 15.8 / 18.5, 4 of 4K 17.9 / 19.1,
// one of 2K 13.2 / 12.1; batches of long lists the same.
constexpr int kSmallRuns = 16, kMinRun = 3, kMaxRun = 24;

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

// The list: all key tiles (TILE keys) of all units, a unit being a sequence and KV head, a
// tree one more tile behind its prefix.
struct RunList {
    int cum[kMaxSeqs + 1];   // key tiles of a KV head, summed over sequences
    uint8_t rem[kMaxSeqs];   // keys of a sequence's last prefix tile (TILE: also none)
    uint8_t nodes[kMaxSeqs];
    uint8_t pad[kMaxSeqs];   // tiles added to a unit to make its runs equal
    int chunk;
};
// A place in the list: sequence, KV head, tile of the unit.
struct Place {
    int b, g;
    int tile, tiles;  // ... of the unit
};
// Fills the list; every thread of the CTA.
template <int TILE>
DDT_DEV void build_list(RunList& l, const ParamsR& p) {
    const int tid = threadIdx.x, lane = tid & 31;
    for (int b = tid; b < p.B; b += kThreadsR) {
        const int P = p.prefix_len[b], n = p.n_nodes[b];
        int t = 0;
        if (P >= 0 && P <= p.cap && n >= 0 && n <= p.N)
            t = (int)((P + (int64_t)TILE - 1) / TILE) + 1;  // (a tree is one tile)
        else if (blockIdx.x == 0)
            record_error(p.err, ERR_ATTN | (n < 0 || n > p.N ? ERR_BAD_N_NODES : ERR_BAD_PREFIX_LEN));
        l.cum[b + 1] = t;
        l.rem[b] = (uint8_t)((P - 1) % TILE + 1 + (P == 0 ? TILE : 0));
        l.nodes[b] = (uint8_t)n;
    }
    __syncthreads();
    // Each CTA's run is `chunk` tiles.  A large batch is cut anywhere; in a small
    // one, where crossing into another unit costs more than an uneven last run,
    // units are padded to whole runs of the least length, at least kMinRun, for which
    // the grid suffices.
    if (tid < 32) {
        int sum = 0;
        for (int b = lane; b < p.B; b += 32) sum += l.cum[b + 1];
        sum = __reduce_add_sync(0xffffffffu, sum);
        const int64_t all = (int64_t)sum * p.Hkv;
        int c = (int)((all + gridDim.x - 1) / gridDim.x);
        bool small = false;
        if (c <= kSmallRuns) {
            int k = max(c, kMinRun);
            for (; !small && k <= kMaxRun; ++k) {
                int runs = 0;
                for (int b = lane; b < p.B; b += 32) runs += (l.cum[b + 1] + k - 1) / k;
                small = (int64_t)__reduce_add_sync(0xffffffffu, runs) * p.Hkv <= gridDim.x;
            }
            if (small) c = k - 1;
        }
        int carry = 0;
        for (int b0 = 0; b0 < p.B; b0 += 32) {
            const int t = b0 + lane < p.B ? l.cum[b0 + lane + 1] : 0;
            const int pad = small ? (c - t % c) % c : 0;
            int v = t + pad;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int up = __shfl_up_sync(0xffffffffu, v, o);
                if (lane >= o) v += up;
            }
            if (b0 + lane < p.B) {
                l.cum[b0 + lane + 1] = v + carry;
                l.pad[b0 + lane] = (uint8_t)pad;
            }
            carry += __shfl_sync(0xffffffffu, v, 31);
        }
        if (lane == 0) {
            l.cum[0] = 0;
            l.chunk = c;
        }
    }
    __syncthreads();
}
template <int TILE>
DDT_DEV int prefix_of(const RunList& l, const Place& x) { return (x.tiles - 2) * TILE + l.rem[x.b]; }
DDT_DEV Place place_of(const RunList& l, const ParamsR& p, int64_t t) {
    int lo = 0, hi = p.B - 1;  // the last sequence that starts at or before t
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if ((int64_t)l.cum[mid] * p.Hkv <= t) lo = mid;
        else hi = mid - 1;
    }
    Place x;
    x.b = lo;
    const int span = l.cum[lo + 1] - l.cum[lo];
    const int64_t off = t - (int64_t)l.cum[lo] * p.Hkv;
    x.g = (int)(off / span);
    x.tile = (int)(off - (int64_t)x.g * span);
    x.tiles = span - l.pad[lo];
    return x;
}
DDT_DEV void next_unit(const RunList& l, const ParamsR& p, Place& x) {
    x.tile = 0;
    if (++x.g == p.Hkv) {
        x.g = 0;
        do ++x.b; while (l.cum[x.b + 1] == l.cum[x.b]);  // (there is one: the run has not ended)
        x.tiles = l.cum[x.b + 1] - l.cum[x.b];
    }
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


}  // namespace

}  // namespace ddt
