// norm_rope.cu -- ddtree_norm_rope: the norm of every head of queries and keys and the
// rotation behind it in one pass.
//
//   y = x / sqrt(mean x^2 + eps) * w,  then pairs of y turned as in rotary.cu
//
// HBM-bound: every row is read and written once.  As in rotary.cu a CTA takes some tokens
// (few tokens are cut by heads over more CTAs), fills their cosine / sine table in shared
// memory and goes over their rows, the next row's loads in flight while one is worked on.
// A row belongs to LPR neighbouring lanes, a power of two, so that its sum of squares is
// log2(LPR) shuffles; a lane holds E units of two vectors, 16 elements at most, worked on by
// two an instruction, and reads cosines, sines and weights of its places from tables.
// 8209 tokens of 72 heads, D = 128: 62 us, 72 % of the measured HBM rate (the rotation alone
// 51); warps that go on from run to run of rows 81 to 83, two rows ahead 68 to 74.
#include <algorithm>

#include "rotary.cuh"

namespace ddt {

namespace {

constexpr int kThreads = 128;
constexpr int kMaxTok = 16;   // tokens per CTA, at most
constexpr int kTable = 2048;  // pairs of a CTA's tokens, at most
constexpr int kPasses = 8;    // rounds of a CTA's threads over its rows, about
constexpr int kFill = 16;     // CTAs per SM that fill the GPU

// Place of float e of V of unit u among `units`: [e / 4][u][e % 4] (for V < 4: [u][e]), so that a
// warp's 16-byte reads fall on different banks; and a unit's V floats from there.
template <int V>
DDT_DEV int float_at(int u, int e, int units) {
    return V < 4 ? u * V + e : ((e >> 2) * units + u) * 4 + (e & 3);
}
template <int V>
DDT_DEV void lane_floats(const float* from, int u, int units, float (&y)[V]) {
    if constexpr (V >= 4) {
#pragma unroll
        for (int e = 0; e < V; e += 4) {
            const float4 x = *(const float4*)&from[((e >> 2) * units + u) * 4];
            y[e] = x.x, y[e + 1] = x.y, y[e + 2] = x.z, y[e + 3] = x.w;
        }
    } else {
#pragma unroll
        for (int e = 0; e < V; ++e) y[e] = from[u * V + e];
    }
}

struct Params {
    RowsArg q, q_out, k, k_out;
    const int32_t* pos;
    const uint64_t* turns;
    NormArgs norm;
    float scale;
    int T, D, rot, tok;
    int units;    // two-vector units per head
    int ru;       // ... of which rotated
    int heads;    // q and k heads of a token
    int chunk;    // ... of which a CTA takes
    int inplace;  // bit 0: q, bit 1: k (untouched rows are skipped)
};

// V: elements per vector, E: units a lane.  PAIRED: pairs (2j, 2j + 1), else (j, j + rot/2).
// FULL: every lane has all of its units.
template <typename T, int V, int E, bool PAIRED, bool FULL>
__global__ void __launch_bounds__(kThreads, FULL ? 8 : 5) norm_rope_kernel(const __grid_constant__ Params p, int lpr_log2) {
    using Vt = Vec<T, V>;
    // cos and sin of token t's pairs, at [t][their place]
    extern __shared__ __align__(16) float s_cos[];
    float* s_sin = s_cos + p.tok * (p.rot / 2);
    __shared__ __align__(16) float s_w[2][2][E * V * 32];  // weights: of q, k; first, second of a unit's pairs
    __shared__ int32_t s_pos[kMaxTok];
    const int tid = threadIdx.x, lpr = 1 << lpr_log2, l = tid & (lpr - 1);
    const int t0 = blockIdx.x * p.tok, nt = min(p.tok, p.T - t0);
    const int per_pass = kThreads >> lpr_log2;  // rows of a pass
    const int h_first = blockIdx.y * p.chunk, heads = min(p.chunk, p.heads - h_first);
    // a unit's two vectors, D where there is none
    auto first_of = [&](int u) {
        return u >= p.units ? p.D : u < p.ru ? (PAIRED ? 2 * V * u : V * u) : p.rot + 2 * V * (u - p.ru);
    };
    auto second_of = [&](int u, int first) {
        return u >= p.units ? p.D : u < p.ru && !PAIRED ? first + p.rot / 2 : first + V;
    };
    int e0[E], e1[E];
#pragma unroll
    for (int i = 0; i < E; ++i) {
        e0[i] = first_of(l + i * lpr);
        e1[i] = second_of(l + i * lpr, e0[i]);
    }
    pdl_wait();

    // a row's token and head, kept as a pair: no division a step
    struct At {
        int t, h;
    };
    auto step = [&](At& x) {
        for (x.h += per_pass; x.h >= h_first + heads; x.h -= heads) ++x.t;
    };
    struct Row {
        Vt a[E], b[E];
    };
    auto load = [&](const At& x, Row& v) {
        const int64_t tok = t0 + x.t;
        const int hk = x.h - p.q.heads;
        const T* s = hk < 0 ? (const T*)p.q.data + tok * p.q.ts + x.h * p.q.hs
                            : (const T*)p.k.data + tok * p.k.ts + hk * p.k.hs;
#pragma unroll
        for (int i = 0; i < E; ++i) {
            if (FULL || e0[i] < p.D) v.a[i] = *(const Vt*)(s + e0[i]);
            if (FULL || e1[i] < p.D) v.b[i] = *(const Vt*)(s + e1[i]);
        }
    };
    At next{0, h_first + (tid >> lpr_log2)};
    while (next.h >= h_first + heads) next.h -= heads, ++next.t;
    Row ahead;
    if (next.t < nt) load(next, ahead);

    // ---- the tokens' tables ----------------------------------------------------
    if (tid < nt) s_pos[tid] = p.pos[t0 + tid];
    const int pairs = p.rot / 2;
    for (int j = tid; j < nt * pairs; j += kThreads) {
        const int t = j / pairs, f = j - t * pairs;
        const int pos = p.pos[t0 + t];
        const float2 cs = cos_sin((uint64_t)(uint32_t)max(pos, 0) * p.turns[f]);
        const int at = t * pairs + float_at<V>(f / V, f % V, p.ru);
        s_cos[at] = cs.x * p.scale;
        s_sin[at] = cs.y * p.scale;
    }
    for (int j = tid; j < 4 * E * V << lpr_log2; j += kThreads) {
        const int e = j % V, second = j / V & 1, u = j / (2 * V) & (E * lpr - 1), kind = j / (2 * V) / E >> lpr_log2;
        const float* from = kind ? p.norm.k_weight : p.norm.q_weight;
        const int a0 = first_of(u), at = place_of_pair<V, PAIRED>(a0, second_of(u, a0), e, second);
        s_w[kind][second][float_at<V>(u, e, E * lpr)] = from && (FULL || at < p.D) ? __ldg(&from[at]) : 1.f;
    }
    __syncthreads();

    // ---- the rows: the warps go on together, for the shuffles ---------------------
    const float inv_D = 1.f / p.D;
    const int rows = nt * heads;
    for (int r0 = tid >> 5 << (5 - lpr_log2); r0 < rows; r0 += per_pass) {
        Row x = ahead;
        const At at = next;
        step(next);
        if (next.t < nt) load(next, ahead);
        float a[E][V], b[E][V], s0 = 0.f, s1 = 0.f;
#pragma unroll
        for (int i = 0; i < E; ++i) {
            if (!FULL && e0[i] >= p.D) x.a[i] = Vt{};
            if (!FULL && e1[i] >= p.D) x.b[i] = Vt{};
            unpack_pairs<T, V, PAIRED>(x.a[i], x.b[i], a[i], b[i]);
            add_squares<V>(a[i], s0, s1);
            add_squares<V>(b[i], s0, s1);
        }
        s0 += s1;
        for (int d = lpr >> 1; d; d >>= 1) s0 += __shfl_xor_sync(0xffffffffu, s0, d);
        if (at.t >= nt) continue;
        const int hk = at.h - p.q.heads, kind = hk >= 0;
        const bool norm = s_pos[at.t] >= 0;
        if (norm) {
            const float f = rsqrtf(fmaf(s0, inv_D, p.norm.eps));
            const float* tc = s_cos + at.t * pairs;
            const float* ts = s_sin + at.t * pairs;
#pragma unroll
            for (int i = 0; i < E; ++i) {
                const int u = l + i * lpr;
                float w[V], c[V], s[V];
                scale_by<V>(a[i], f);
                scale_by<V>(b[i], f);
                lane_floats<V>(s_w[kind][0], u, E * lpr, w);
                scale_vec<V>(a[i], w);
                lane_floats<V>(s_w[kind][1], u, E * lpr, w);
                scale_vec<V>(b[i], w);
                if (u < p.ru) {
                    lane_floats<V>(tc, u, p.ru, c);
                    lane_floats<V>(ts, u, p.ru, s);
                    turn_vec<V>(a[i], b[i], c, s);
                }
                pack_pairs<T, V, PAIRED>(a[i], b[i], x.a[i], x.b[i]);
            }
        } else if ((p.inplace >> kind) & 1) {
            continue;
        }
        const int64_t tok = t0 + at.t;
        T* dst = kind ? (T*)p.k_out.data + tok * p.k_out.ts + hk * p.k_out.hs
                      : (T*)p.q_out.data + tok * p.q_out.ts + at.h * p.q_out.hs;
#pragma unroll
        for (int i = 0; i < E; ++i) {
            if (FULL || e0[i] < p.D) *(Vt*)(dst + e0[i]) = x.a[i];
            if (FULL || e1[i] < p.D) *(Vt*)(dst + e1[i]) = x.b[i];
        }
    }
    pdl_trigger();
}

template <typename T, int V, int E, bool PAIRED>
cudaError_t launch_e(Params& p, cudaStream_t s) {
    int lpr_log2 = 0;
    while ((E << lpr_log2) < p.units) ++lpr_log2;
    // Tokens of a CTA: enough for kPasses rounds of its threads, as long as the CTAs
    // still fill the GPU; few tokens are cut by heads instead.
    const int64_t fill = (int64_t)num_sms() * kFill, lanes = (int64_t)p.heads << lpr_log2;
    p.tok = 1;
    while (p.tok < kMaxTok && p.tok * lanes < kPasses * kThreads && 2 * p.tok * (p.rot / 2) <= kTable &&
           p.T / (2 * p.tok) >= fill)
        p.tok *= 2;
    const int64_t cuts = std::min((lanes + kThreads - 1) / kThreads, std::max<int64_t>(1, fill / p.T));
    p.chunk = (int)((p.heads + cuts - 1) / cuts);
    const dim3 grid((unsigned)((p.T + p.tok - 1) / p.tok), (unsigned)((p.heads + p.chunk - 1) / p.chunk));
    const size_t smem = (size_t)p.tok * p.rot * sizeof(float);
    // (in the general form 8209 tokens of 72 heads, D = 128, took 65 us, in this one 62)
    if constexpr (E == 1 && V * sizeof(T) == 16)
        if (p.units == 1 << lpr_log2 && (p.D - p.rot) % (2 * V) == 0)
            return launch_pdl(norm_rope_kernel<T, V, E, PAIRED, true>, grid, dim3(kThreads), smem, s, p, lpr_log2);
    return launch_pdl(norm_rope_kernel<T, V, E, PAIRED, false>, grid, dim3(kThreads), smem, s, p, lpr_log2);
}

template <typename T, int V>
cudaError_t launch_v(Params& p, bool paired, cudaStream_t s) {
    constexpr int most = 8 / V;  // units a lane: D is at most 512
    p.ru = p.rot / (2 * V);
    p.units = p.ru + (p.D - p.rot + 2 * V - 1) / (2 * V);
    if constexpr (most > 1)
        if (p.units > 32) return paired ? launch_e<T, V, most, true>(p, s) : launch_e<T, V, most, false>(p, s);
    return paired ? launch_e<T, V, 1, true>(p, s) : launch_e<T, V, 1, false>(p, s);
}

// The widest vectors that sizes, strides and addresses allow: 16 bytes, 8, or
// single elements.
template <typename T>
cudaError_t launch(Params& p, bool paired, cudaStream_t s) {
    constexpr int V16 = 16 / (int)sizeof(T), V8 = 8 / (int)sizeof(T);
    auto fits = [&](int V) {
        bool ok = p.rot / 2 % V == 0 && p.D % V == 0;
        for (const RowsArg* r : {&p.q, &p.q_out, &p.k, &p.k_out})
            if (r->heads) ok = ok && on_grid(r->data, r->ts, r->hs, 0, sizeof(T), V);
        return ok;
    };
    if (fits(V16)) return launch_v<T, V16>(p, paired, s);
    if (fits(V8)) return launch_v<T, V8>(p, paired, s);
    return launch_v<T, 1>(p, paired, s);
}

}  // namespace

cudaError_t launch_norm_rope(const NormRopeArgs& a, cudaStream_t s) {
    Params p{};
    p.q = a.q, p.q_out = a.q_out, p.k = a.k, p.k_out = a.k_out;
    p.pos = a.pos, p.turns = a.turns, p.norm = a.norm, p.scale = a.scale;
    p.T = a.T, p.D = a.D, p.rot = a.rot;
    p.heads = a.q.heads + a.k.heads;
    p.inplace = (a.q.data == a.q_out.data ? 1 : 0) | (a.k.data == a.k_out.data ? 2 : 0);
    if (a.dtype == 0) return launch<__nv_bfloat16>(p, a.interleaved, s);
    if (a.dtype == 1) return launch<float>(p, a.interleaved, s);
    return launch<__half>(p, a.interleaved, s);
}

}  // namespace ddt
