// quant.cu -- the 8-bit cache's writers (ddtree_append_q8, ddtree_commit_q8) and its
// reader (ddtree_read_q8); q8.cuh has the format.
//
// Writers.  HBM-bound: rows are read once and stay in registers from their load to their
// codes.  A CTA takes one block of the cache that a run touches (run_block) and some of the
// heads of its tokens: queries, keys, values.  It fills the block's positions' cosine and
// sine table in shared memory once for all of them; a head's rows are then loaded, normed
// and turned in 32 bits -- D / 16 lanes a row, two vectors of 8 elements a lane, as in
// norm_rope.cu -- their largest element found, and rounded to codes under its power of
// two, the next head's loads in flight meanwhile.  A head is one warp's where its rows fit
// the passes that a whole block takes the CTA (a decoding step's single row always does),
// so that warps go on without each other, and the CTA's otherwise, which then meets
// once a head.  18.2K tokens of ragged prompts, normed and turned: 91 us, 67 % of the measured
// HBM rate; one token each of 16 sequences 3.2 us, a launch.  A NaN is found by the maxima (89.5 us
// without that) and recorded.
#include <type_traits>

#include "q8.cuh"
#include "rotary.cuh"

namespace ddt {

namespace {

constexpr int kThreads = 128;  // of the reader; the writers' CTAs have as many or twice
// CTAs per SM that fill the GPU: a block's heads are cut over CTAs up to that.  An append's
// CTAs each fill the block's table (prompts of 18K tokens 98 us at 16, 90 at 3); a commit's
// have none and wait for their rows (128 paths 7.3 us at 3).
constexpr int kFillAppend = 3, kFill = 16, kFillRead = 8;

struct WriteParams {
    RowsArg q, q_out, k, v;
    Q8Args cache;
    const int32_t *first, *at;                                // append
    const int32_t *accept_len, *accepted_nodes, *prefix_len;  // commit
    int32_t* new_len;
    const uint64_t* turns;
    NormArgs norm;
    float scale;
    int T, B, rot, L, N;
    int slots;  // commit: blocks that a path may touch
    int heads, chunk;  // of a token: queries, keys and values; ... that a CTA takes
    int page_log2, block_log2;
    uint32_t* err;
};

// PAIRED: pairs (2j, 2j + 1), else (j, j + rot/2).  kPasses: rows of a lane where a whole
// block is the CTA's, of kWarps warps.
template <typename T, int D, int kWarps, int kPasses, bool PAIRED, bool COMMIT>
__global__ void __launch_bounds__(32 * kWarps, (kPasses == 2 ? 16 : 24) / kWarps) write_kernel(const __grid_constant__ WriteParams p) {
    constexpr int LPR = D / 16, RPW = 32 / LPR;  // lanes a row, rows of a warp's pass
    using Vt = Vec<T, 8>;
    // cos and sin of row r's pair 8 u + e, at [r][e / 4][u][e % 4]
    extern __shared__ __align__(16) float s_cos[];
    __shared__ float s_max[2][kWarps];
    __shared__ int s_node[DDTREE_MAX_L + 1], s_page[DDTREE_MAX_L + 1];  // of a path's rows
    __shared__ int s_bad;
    const Q8Args& c = p.cache;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, S = c.block;
    const int64_t cap = (int64_t)c.max_pages << p.page_log2;
    pdl_wait();
    RunBlock x{};
    if constexpr (COMMIT) {
        // Every CTA of a sequence checks its whole path and its pages, so that all reach
        // the same verdict.
        x.b = blockIdx.x / p.slots;
        const int j = blockIdx.x - x.b * p.slots;
        const int P = p.prefix_len[x.b], a = p.accept_len[x.b];
        if (tid < 32) {
            uint32_t bad = 0;
            if (a < 0 || a > p.L || P < 0 || (int64_t)P + a + 1 > cap) {
                bad = ERR_BAD_PREFIX_LEN;
            } else if (tid <= a) {
                const int node = tid ? p.accepted_nodes[(int64_t)x.b * p.L + tid - 1] : 0;
                const int page = c.table[x.b * c.table_stride + ((P + tid) >> p.page_log2)];
                s_node[tid] = node;
                s_page[tid] = page;
                if (tid && (node < 1 || node > p.N)) bad = ERR_BAD_TREE;
                else if (page < 0 || page >= c.num_pages) bad = ERR_BAD_PAGE;
            }
            bad = __reduce_max_sync(0xffffffffu, bad);
            if (tid == 0) {
                s_bad = (int)bad;
                if (j == 0 && blockIdx.y == 0) {
                    if (bad) record_error(p.err, ERR_COMMIT | bad);
                    if (p.new_len) p.new_len[x.b] = bad ? P : P + a + 1;
                }
            }
        }
        __syncthreads();
        if (s_bad) return;
        x.p0 = (P & -S) + j * S;
        x.lo = max(x.p0, P);
        x.hi = min(x.p0 + S, P + a + 1);
        x.token = x.lo - P;  // (of the path)
        if (x.lo >= x.hi) return;
    } else {
        x = run_block(p.first, p.at, p.B, p.T, p.block_log2, cap, blockIdx.x);
        if (tid == 0 && blockIdx.y == 0)
            check_run(p.first, p.at, p.B, p.T, cap, blockIdx.x, p.err, ERR_APPEND | ERR_BAD_INPUT);
        if (!x.ok) return;
    }
    const int page = COMMIT ? s_page[x.token] : c.table[x.b * c.table_stride + (x.p0 >> p.page_log2)];
    const bool there = page >= 0 && page < c.num_pages;
    const int rows = x.hi - x.lo, slot0 = x.p0 & (c.page_size - 1), least = q8_least(c.dtype == 2);
    const int h_first = blockIdx.y * p.chunk;
    int h_last = min(p.heads, h_first + p.chunk);
    if (!there) {
        if (tid == 0 && h_last > p.q.heads) record_error(p.err, ERR_APPEND | ERR_BAD_PAGE);
        h_last = min(h_last, p.q.heads);  // (queries go on)
    }

    // ---- the block's table, if a head here is turned ---------------------------
    const int pairs = p.rot / 2, ru = p.rot / 16;
    float* s_sin = s_cos + S * pairs;
    if (!COMMIT && pairs && h_first < p.q.heads + c.Hkv) {
        for (int j = tid; j < rows * pairs; j += (32 * kWarps)) {
            const int r = j / pairs, f = j - r * pairs;
            const float2 cs = cos_sin((uint64_t)(uint32_t)(x.lo + r) * p.turns[f]);
            const int at = r * pairs + (((f & 7) >> 2) * ru + (f >> 3)) * 4 + (f & 3);
            s_cos[at] = cs.x * p.scale;
            s_sin[at] = cs.y * p.scale;
        }
        __syncthreads();
    }

    // ---- the heads: of a kind (queries, keys, values) one after another ------------
    const int u = lane & (LPR - 1);  // the lane's two vectors of a row
    const bool in_rot = u < ru;
    const int e0 = in_rot ? (PAIRED ? 16 * u : 8 * u) : p.rot + 16 * (u - ru);
    const int e1 = in_rot && !PAIRED ? e0 + pairs : e0 + 8;
    const bool whole = rows > kPasses * RPW;  // a head is the CTA's
    const int r_first = (whole ? warp * RPW : 0) + lane / LPR, r_step = whole ? kWarps * RPW : RPW;
    const int h_step = whole ? 1 : kWarps, h_off = whole ? 0 : warp;
    int64_t token[kPasses];
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
        const int r = min(r_first + i * r_step, rows - 1);  // (a lane without a row repeats the last)
        token[i] = COMMIT ? (int64_t)x.b * (p.N + 1) + s_node[x.token + r] : x.token + r;
    }
    int turn = 0;
    auto heads = [&](auto kind_, const RowsArg& in, int before, const float* weight) {
        constexpr int kind = decltype(kind_)::value;  // 0 queries, 1 keys, 2 values
        constexpr bool may_turn = !COMMIT && kind != 2;
        const int to = min(h_last - before, in.heads);
        int h = max(h_first - before, 0);
        h += h_off;
        if (h >= to) return;
        struct Rows {
            Vt a[kPasses], b[kPasses];
        };
        const T* src[kPasses];
#pragma unroll
        for (int i = 0; i < kPasses; ++i) src[i] = (const T*)in.data + token[i] * in.ts + h * in.hs;
        const int64_t src_step = h_step * in.hs;
        auto load = [&](Rows& v) {
#pragma unroll
            for (int i = 0; i < kPasses; ++i) {
                v.a[i] = *(const Vt*)(src[i] + e0);
                v.b[i] = *(const Vt*)(src[i] + e1);
                src[i] += src_step;
            }
        };
        Rows ahead;
        load(ahead);
        const bool norm = may_turn && p.norm.on;
        float w[2][8];
        if (norm) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                w[0][e] = weight ? __ldg(&weight[place_of_pair<8, PAIRED>(e0, e1, e, false)]) : 1.f;
                w[1][e] = weight ? __ldg(&weight[place_of_pair<8, PAIRED>(e0, e1, e, true)]) : 1.f;
            }
        }
        for (; h < to; h += h_step) {
            Rows v = ahead;
            if (h + h_step < to) load(ahead);
            uint8_t *scale = nullptr, *codes = nullptr;
            int old = least;
            if constexpr (kind > 0) {
                scale = (kind == 2 ? c.v_scales : c.k_scales) +
                        ((((int64_t)page * c.Hkv + h) << (p.page_log2 - p.block_log2)) + (slot0 >> p.block_log2));
                codes = (kind == 2 ? c.v : c.k) + page * c.page_stride + h * c.head_stride + slot0 * c.slot_stride;
                if (x.lo > x.p0) old = q8_from_byte(*scale, least);
            }
            float ya[kPasses][8], yb[kPasses][8], most = 0.f;  // first and second elements of pairs
#pragma unroll
            for (int i = 0; i < kPasses; ++i) {
                unpack_pairs<T, 8, PAIRED>(v.a[i], v.b[i], ya[i], yb[i]);
                float root = 1.f;  // the norm's factor, which may come last: a rotation is linear
                if (norm) {
                    float s0 = 0.f, s1 = 0.f;
                    add_squares<8>(ya[i], s0, s1);
                    add_squares<8>(yb[i], s0, s1);
                    s0 += s1;
#pragma unroll
                    for (int d = LPR / 2; d; d >>= 1) s0 += __shfl_xor_sync(0xffffffffu, s0, d);
                    root = rsqrtf(fmaf(s0, 1.f / D, p.norm.eps));
                    scale_vec<8>(ya[i], w[0]);
                    scale_vec<8>(yb[i], w[1]);
                }
                if (may_turn && in_rot) {
                    const int at = min(r_first + i * r_step, rows - 1) * pairs + u * 4;
                    float cv[8], sv[8];
#pragma unroll
                    for (int g = 0; g < 2; ++g) {
                        const float4 cc = *(const float4*)&s_cos[at + g * ru * 4], ss = *(const float4*)&s_sin[at + g * ru * 4];
                        cv[4 * g] = cc.x, cv[4 * g + 1] = cc.y, cv[4 * g + 2] = cc.z, cv[4 * g + 3] = cc.w;
                        sv[4 * g] = ss.x, sv[4 * g + 1] = ss.y, sv[4 * g + 2] = ss.z, sv[4 * g + 3] = ss.w;
                    }
                    turn_vec<8>(ya[i], yb[i], cv, sv);
                }
                if (norm) {
                    scale_by<8>(ya[i], root);
                    scale_by<8>(yb[i], root);
                }
                if constexpr (kind > 0) {
                    float m = 0.f;
#pragma unroll
                    for (int e = 0; e < 8; ++e) m = max_nan(m, fabsf(ya[i][e]), fabsf(yb[i][e]));
                    most = max_nan(most, m, m);
                }
            }
            if constexpr (kind == 0) {
#pragma unroll
                for (int i = 0; i < kPasses; ++i)
                    if (r_first + i * r_step < rows) {
                        T* row = (T*)p.q_out.data + token[i] * p.q_out.ts + h * p.q_out.hs;
                        Vt a, b;
                        pack_pairs<T, 8, PAIRED>(ya[i], yb[i], a, b);
                        *(Vt*)(row + e0) = a;
                        *(Vt*)(row + e1) = b;
                    }
            } else {
                uint32_t bits = __reduce_max_sync(0xffffffffu, __float_as_uint(most));  // (not negative; NaN is above inf)
                if (bits > 0x7f800000u) {  // (rare) a NaN, which the scale goes without
                    if (lane == 0) record_error(p.err, (COMMIT ? ERR_COMMIT : ERR_APPEND) | ERR_BAD_INPUT);
                    most = 0.f;
                    for (int i = 0; i < kPasses; ++i)
                        for (int e = 0; e < 8; ++e) most = fmaxf(most, fmaxf(fabsf(ya[i][e]), fabsf(yb[i][e])));
                    bits = __reduce_max_sync(0xffffffffu, __float_as_uint(most));
                }
                most = __uint_as_float(bits);
                if (whole) {
                    if (lane == 0) s_max[turn][warp] = most;
                    __syncthreads();  // (and every thread has read the old scale)
#pragma unroll
                    for (int i = 0; i < kWarps; ++i) most = fmaxf(most, s_max[turn][i]);
                    turn ^= 1;
                }
                const int e = max(q8_exponent(most, least), old);
                if (x.lo > x.p0 && e > old) {  // the block's earlier codes move to its new scale
                    const float f = pow2(old - e);
                    const int n = (x.lo - x.p0) * LPR, step = whole ? 32 * kWarps : 32;
                    for (int i = whole ? tid : lane; i < n; i += step) {
                        uint4* to_ = (uint4*)(codes + (i / LPR) * c.slot_stride + (i & (LPR - 1)) * 16);
                        const uint4 m = *to_;
                        *to_ = make_uint4(q8_moved(m.x, f), q8_moved(m.y, f), q8_moved(m.z, f), q8_moved(m.w, f));
                    }
                }
                const float f = pow2(-e);
#pragma unroll
                for (int i = 0; i < kPasses; ++i) {
                    const int r = r_first + i * r_step;
                    if (r < rows) {
                        uint8_t* row = codes + (x.lo - x.p0 + r) * c.slot_stride;
                        float(&a)[8] = ya[i], (&b)[8] = yb[i];
                        scale_by<8>(a, f);  // (a power of two, and by itself: times a root it may pass the 32-bit range)
                        scale_by<8>(b, f);
                        if constexpr (PAIRED) {
                            *(uint4*)(row + e0) = make_uint4(q8_pack4(a[0], b[0], a[1], b[1]), q8_pack4(a[2], b[2], a[3], b[3]),
                                                             q8_pack4(a[4], b[4], a[5], b[5]), q8_pack4(a[6], b[6], a[7], b[7]));
                        } else {
                            *(uint2*)(row + e0) = make_uint2(q8_pack4(a[0], a[1], a[2], a[3]), q8_pack4(a[4], a[5], a[6], a[7]));
                            *(uint2*)(row + e1) = make_uint2(q8_pack4(b[0], b[1], b[2], b[3]), q8_pack4(b[4], b[5], b[6], b[7]));
                        }
                    }
                }
                __syncwarp();  // (the warp's lanes have read the old scale)
                if ((whole ? tid : lane) == 0) *scale = (uint8_t)(e + 127);
            }
        }
    };
    if constexpr (!COMMIT) heads(std::integral_constant<int, 0>{}, p.q, 0, p.norm.q_weight);
    heads(std::integral_constant<int, 1>{}, p.k, p.q.heads, p.norm.k_weight);
    heads(std::integral_constant<int, 2>{}, p.v, p.q.heads + c.Hkv, nullptr);
    pdl_trigger();
}

struct ReadParams {
    Q8Args cache;
    const int32_t *first, *at;
    RowsArg k_out, v_out;
    int B, T, chunk;
    int page_log2, block_log2;
    uint32_t* err;
};

// Reader.  HBM-bound: a CTA takes one block of the cache that a run touches, for some of its
// (half, head)s; a thread takes 16 codes at a time, several in flight, and stores the 16
// elements that they are.  270K positions back: 296 us, 84 % of the measured HBM rate (eight
// in flight 282, but one prefix of 2K 4.9 us for 4.0).
constexpr int kInFlight = 4;

template <bool F16, int D>
__global__ void __launch_bounds__(kThreads) read_kernel(const __grid_constant__ ReadParams p) {
    constexpr int CH = D / 16;  // 16-byte chunks of a row of codes
    const Q8Args& c = p.cache;
    const int64_t cap = (int64_t)c.max_pages << p.page_log2;
    pdl_wait();
    const RunBlock x = run_block(p.first, p.at, p.B, p.T, p.block_log2, cap, blockIdx.x);
    if (threadIdx.x == 0 && blockIdx.y == 0)
        check_run(p.first, p.at, p.B, p.T, cap, blockIdx.x, p.err, ERR_READ | ERR_BAD_INPUT);
    if (!x.ok) return;
    const int page = c.table[x.b * c.table_stride + (x.p0 >> p.page_log2)];
    if (page < 0 || page >= c.num_pages) {
        if (threadIdx.x == 0) record_error(p.err, ERR_READ | ERR_BAD_PAGE);
        return;
    }
    const int slot0 = x.p0 & (c.page_size - 1), r_lo = x.lo - x.p0, r_hi = x.hi - x.p0;
    const int t_first = blockIdx.y * p.chunk, t_last = min(2 * c.Hkv, t_first + p.chunk);
    // items: (half, head), slot of the block, chunk of the row
    const int items = ((t_last - t_first) << p.block_log2) * CH;
    for (int i0 = threadIdx.x; i0 < items; i0 += kInFlight * kThreads) {
        uint4 w[kInFlight];
        uint32_t f[kInFlight];
#pragma unroll
        for (int k = 0; k < kInFlight; ++k) {
            const int i = i0 + k * kThreads, r = i / CH & (c.block - 1), t = t_first + ((i / CH) >> p.block_log2);
            if (i < items && r >= r_lo && r < r_hi) {
                const bool is_v = t >= c.Hkv;
                const int head = is_v ? t - c.Hkv : t;
                const uint8_t* row = (is_v ? c.v : c.k) + page * c.page_stride + head * c.head_stride +
                                     (slot0 + r) * c.slot_stride;
                w[k] = ld_stream_v4(row + (i & (CH - 1)) * 16);
                f[k] = __ldg((is_v ? c.v_scales : c.k_scales) +
                             ((((int64_t)page * c.Hkv + head) << (p.page_log2 - p.block_log2)) + (slot0 >> p.block_log2)));
            }
        }
#pragma unroll
        for (int k = 0; k < kInFlight; ++k) {
            const int i = i0 + k * kThreads, r = i / CH & (c.block - 1), t = t_first + ((i / CH) >> p.block_log2);
            if (i < items && r >= r_lo && r < r_hi) {
                const bool is_v = t >= c.Hkv;
                const RowsArg& out = is_v ? p.v_out : p.k_out;
                uint16_t* row = (uint16_t*)out.data + (int64_t)(x.token + r - r_lo) * out.ts +
                                (is_v ? t - c.Hkv : t) * out.hs + (i & (CH - 1)) * 16;
                const uint32_t m = widen_factor<F16>(f[k]) * 0x10001u;
                *(uint4*)row = make_uint4(widen_lo<F16>(w[k].x, m), widen_hi<F16>(w[k].x, m),
                                          widen_lo<F16>(w[k].y, m), widen_hi<F16>(w[k].y, m));
                *(uint4*)(row + 8) = make_uint4(widen_lo<F16>(w[k].z, m), widen_hi<F16>(w[k].z, m),
                                                widen_lo<F16>(w[k].w, m), widen_hi<F16>(w[k].w, m));
            }
        }
    }
    pdl_trigger();
}

int log2_of(int x) {
    int n = 0;
    while ((1 << n) < x) ++n;
    return n;
}

// Heads of a CTA: as many as leave per_sm CTAs an SM, at least `least` of them.
int heads_of(int heads, int64_t slots, int least, int per_sm) {
    const int64_t fill = (int64_t)num_sms() * per_sm, cuts = std::max<int64_t>(1, (fill + slots - 1) / slots);
    return (int)std::max<int64_t>(std::min(least, heads), (heads + cuts - 1) / cuts);
}

template <typename T, int D, int WARPS, int PASSES, bool PAIRED, bool COMMIT>
cudaError_t launch_passes(WriteParams& p, int64_t blocks, cudaStream_t s) {
    p.page_log2 = log2_of(p.cache.page_size);
    p.block_log2 = log2_of(p.cache.block);
    p.heads = p.q.heads + 2 * p.cache.Hkv;
    p.chunk = heads_of(p.heads, blocks, WARPS, COMMIT ? kFill : kFillAppend);
    if (blocks > INT32_MAX) return cudaErrorInvalidValue;
    const dim3 grid((unsigned)blocks, (unsigned)((p.heads + p.chunk - 1) / p.chunk));
    return launch_pdl(write_kernel<T, D, WARPS, PASSES, PAIRED, COMMIT>, grid, dim3(32 * WARPS),
                      (size_t)p.cache.block * p.rot * sizeof(float), s, p);
}
// The fewest registers that hold a block's rows: one row a lane, two, or two of twice the
// lanes (64 rows of D = 128; four a lane spilled).
template <typename T, int D, bool PAIRED, bool COMMIT>
cudaError_t launch_write(WriteParams& p, int64_t blocks, cudaStream_t s) {
    constexpr int rows = 4 * 32 / (D / 16);  // of a pass of four warps
    static_assert(DDTREE_MAX_Q8_BLOCK <= 4 * rows, "two passes of eight warps");
    if constexpr (DDTREE_MAX_Q8_BLOCK > 2 * rows)
        if (p.cache.block > 2 * rows) return launch_passes<T, D, 8, 2, PAIRED, COMMIT>(p, blocks, s);
    if constexpr (DDTREE_MAX_Q8_BLOCK > rows)
        if (p.cache.block > rows) return launch_passes<T, D, 4, 2, PAIRED, COMMIT>(p, blocks, s);
    return launch_passes<T, D, 4, 1, PAIRED, COMMIT>(p, blocks, s);
}
template <typename T, int D>
cudaError_t launch_append(WriteParams& p, int64_t blocks, bool paired, cudaStream_t s) {
    return paired ? launch_write<T, D, true, false>(p, blocks, s) : launch_write<T, D, false, false>(p, blocks, s);
}

}  // namespace

cudaError_t launch_append_q8(const AppendQ8Args& a, cudaStream_t s) {
    WriteParams p{};
    p.q = a.q, p.q_out = a.q_out, p.k = a.k, p.v = a.v, p.cache = a.cache;
    p.first = a.first, p.at = a.at, p.turns = a.turns, p.norm = a.norm, p.scale = a.scale;
    p.T = a.T, p.B = a.B, p.rot = a.rot, p.err = a.err;
    const int64_t blocks = run_slots(a.B, a.T, a.cache.block);
    const bool f16 = a.cache.dtype == 2;
    if (a.cache.D == 128)
        return f16 ? launch_append<__half, 128>(p, blocks, a.interleaved, s)
                   : launch_append<__nv_bfloat16, 128>(p, blocks, a.interleaved, s);
    return f16 ? launch_append<__half, 64>(p, blocks, a.interleaved, s)
               : launch_append<__nv_bfloat16, 64>(p, blocks, a.interleaved, s);
}

cudaError_t launch_commit_q8(const CommitQ8Args& a, cudaStream_t s) {
    WriteParams p{};
    p.k = a.k_tree, p.v = a.v_tree, p.cache = a.cache;
    p.accept_len = a.accept_len, p.accepted_nodes = a.accepted_nodes, p.prefix_len = a.prefix_len;
    p.new_len = a.new_len, p.B = a.B, p.L = a.L, p.N = a.N, p.err = a.err;
    p.slots = (a.L - 1 + a.cache.block) / a.cache.block + 1;  // blocks that L + 1 positions touch
    const int64_t blocks = (int64_t)a.B * p.slots;
    const bool f16 = a.cache.dtype == 2;
    if (a.cache.D == 128)
        return f16 ? launch_write<__half, 128, true, true>(p, blocks, s)
                   : launch_write<__nv_bfloat16, 128, true, true>(p, blocks, s);
    return f16 ? launch_write<__half, 64, true, true>(p, blocks, s)
               : launch_write<__nv_bfloat16, 64, true, true>(p, blocks, s);
}

cudaError_t launch_read_q8(const ReadQ8Args& a, cudaStream_t s) {
    ReadParams p{};
    p.cache = a.cache, p.first = a.first, p.at = a.at, p.k_out = a.k_out, p.v_out = a.v_out;
    p.B = a.B, p.T = a.T, p.err = a.err;
    p.page_log2 = log2_of(a.cache.page_size);
    p.block_log2 = log2_of(a.cache.block);
    const int64_t blocks = run_slots(a.B, a.T, a.cache.block);
    if (blocks > INT32_MAX) return cudaErrorInvalidValue;
    // (at least one round of a CTA's threads)
    const int tasks = 2 * a.cache.Hkv, one = a.cache.block * a.cache.D / 16;
    p.chunk = heads_of(tasks, blocks, std::max(1, kThreads / one), kFillRead);
    const dim3 grid((unsigned)blocks, (unsigned)((tasks + p.chunk - 1) / p.chunk));
    const bool f16 = a.cache.dtype == 2;
    if (a.cache.D == 128)
        return f16 ? launch_pdl(read_kernel<true, 128>, grid, dim3(kThreads), 0, s, p)
                   : launch_pdl(read_kernel<false, 128>, grid, dim3(kThreads), 0, s, p);
    return f16 ? launch_pdl(read_kernel<true, 64>, grid, dim3(kThreads), 0, s, p)
               : launch_pdl(read_kernel<false, 64>, grid, dim3(kThreads), 0, s, p);
}

}  // namespace ddt
