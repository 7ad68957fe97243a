// norm_rope.cu -- ddtree_norm_rope: the norm of every head of queries and keys and the
// rotation behind it in one pass.
//
//   y = x / sqrt(mean x^2 + eps) * w,  then pairs of y turned as in rotary.cu
//
// HBM-bound: every row is read and written once.  As in rotary.cu a CTA takes some tokens
// (few tokens are cut by heads over more CTAs), fills their cosine / sine table in shared
// memory and goes over their rows, the next row's loads in flight while one is worked on.
// A row belongs to LPR neighbouring lanes, a power of two, so that its sum of squares is
// log2(LPR) shuffles; a lane holds E units of two vectors, 16 elements at most, and the
// weights of the same places, which change only between queries and keys.
#include <algorithm>

#include "rotary.cuh"

namespace ddt {

namespace {

constexpr int kThreads = 128;
constexpr int kMaxTok = 16;   // tokens per CTA, at most
constexpr int kTable = 2048;  // pairs of a CTA's tokens, at most
constexpr int kPasses = 8;    // rounds of a CTA's threads over its rows, about
constexpr int kFill = 16;     // CTAs per SM that fill the GPU

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

// V: elements per vector, E: units a lane, LPR: lanes a row.  PAIRED: pairs (2j, 2j + 1), else
// (j, j + rot/2).
template <typename T, int V, int E, bool PAIRED>
__global__ void __launch_bounds__(kThreads, 5) norm_rope_kernel(const __grid_constant__ Params p, int lpr_log2) {
    using Vt = Vec<T, V>;
    // cos and sin of token t's pair V * u + e, at [t][e / 4][u][e % 4] (for V < 4: [t][u][e])
    extern __shared__ __align__(16) float s_cos[];
    float* s_sin = s_cos + p.tok * (p.rot / 2);
    __shared__ int32_t s_pos[kMaxTok];
    const int tid = threadIdx.x, lpr = 1 << lpr_log2, l = tid & (lpr - 1);
    const int t0 = blockIdx.x * p.tok, nt = min(p.tok, p.T - t0);
    const int per_pass = kThreads >> lpr_log2;  // rows of a pass
    const int h_first = blockIdx.y * p.chunk, heads = min(p.chunk, p.heads - h_first);
    int e0[E], e1[E];  // a unit's two vectors, D where there is none
#pragma unroll
    for (int i = 0; i < E; ++i) {
        const int u = l + i * lpr;
        e0[i] = u >= p.units ? p.D : u < p.ru ? (PAIRED ? 2 * V * u : V * u) : p.rot + 2 * V * (u - p.ru);
        e1[i] = u >= p.units ? p.D : u < p.ru && !PAIRED ? e0[i] + p.rot / 2 : e0[i] + V;
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
            if (e0[i] < p.D) v.a[i] = *(const Vt*)(s + e0[i]);
            if (e1[i] < p.D) v.b[i] = *(const Vt*)(s + e1[i]);
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
        const int un = f / V, e = f - un * V;
        const int at = t * pairs + (V < 4 ? un * V + e : ((e >> 2) * p.ru + un) * 4 + (e & 3));
        s_cos[at] = cs.x * p.scale;
        s_sin[at] = cs.y * p.scale;
    }
    __syncthreads();

    // ---- the rows: the warps go on together, for the shuffles ---------------------
    float wa[E][V], wb[E][V];
    int kind = -1;  // whose weights these are
    const float inv_D = 1.f / p.D;
    const int rows = nt * heads;
    for (int r0 = tid >> 5 << (5 - lpr_log2); r0 < rows; r0 += per_pass) {
        Row x = ahead;
        const At at = next;
        step(next);
        if (next.t < nt) load(next, ahead);
        const bool live = at.t < nt;
        const bool is_k = at.h >= p.q.heads;
        const bool norm = live && s_pos[live ? at.t : 0] >= 0;
        float a[E][V], b[E][V], sum = 0.f;
#pragma unroll
        for (int i = 0; i < E; ++i)
#pragma unroll
            for (int e = 0; e < V; ++e) {
                a[i][e] = e0[i] < p.D ? to_f(x.a[i].e[e]) : 0.f;
                b[i][e] = e1[i] < p.D ? to_f(x.b[i].e[e]) : 0.f;
                sum = fmaf(a[i][e], a[i][e], sum);
                sum = fmaf(b[i][e], b[i][e], sum);
            }
        for (int d = lpr >> 1; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
        if (!live) continue;
        const int hh = is_k ? at.h - p.q.heads : at.h;
        const int64_t tok = t0 + at.t;
        T* dst = is_k ? (T*)p.k_out.data + tok * p.k_out.ts + hh * p.k_out.hs
                      : (T*)p.q_out.data + tok * p.q_out.ts + hh * p.q_out.hs;
        if (norm) {
            if (kind != (int)is_k) {
                kind = is_k;
                const float* w = is_k ? p.norm.k_weight : p.norm.q_weight;
#pragma unroll
                for (int i = 0; i < E; ++i)
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        wa[i][e] = w && e0[i] < p.D ? __ldg(&w[e0[i] + e]) : 1.f;
                        wb[i][e] = w && e1[i] < p.D ? __ldg(&w[e1[i] + e]) : 1.f;
                    }
            }
            const float f = rsqrtf(fmaf(sum, inv_D, p.norm.eps));
            const float* tc = s_cos + at.t * pairs;
            const float* ts = s_sin + at.t * pairs;
#pragma unroll
            for (int i = 0; i < E; ++i) {
                float ya[V], yb[V];
#pragma unroll
                for (int e = 0; e < V; ++e) ya[e] = a[i][e] * f * wa[i][e], yb[e] = b[i][e] * f * wb[i][e];
                const int u = l + i * lpr;
                if (u < p.ru) {
                    float c[V], s[V];
                    if constexpr (V >= 4) {
#pragma unroll
                        for (int e = 0; e < V; e += 4) {
                            const float4 cc = *(const float4*)&tc[((e >> 2) * p.ru + u) * 4];
                            const float4 ss = *(const float4*)&ts[((e >> 2) * p.ru + u) * 4];
                            c[e] = cc.x, c[e + 1] = cc.y, c[e + 2] = cc.z, c[e + 3] = cc.w;
                            s[e] = ss.x, s[e + 1] = ss.y, s[e + 2] = ss.z, s[e + 3] = ss.w;
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < V; ++e) c[e] = tc[u * V + e], s[e] = ts[u * V + e];
                    }
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        float& m = PAIRED ? (2 * e < V ? ya[2 * e % V] : yb[2 * e % V]) : ya[e];
                        float& n = PAIRED ? (2 * e + 1 < V ? ya[(2 * e + 1) % V] : yb[(2 * e + 1) % V]) : yb[e];
                        const float2 z = turned(m, n, c[e], s[e]);
                        m = z.x, n = z.y;
                    }
                }
                pack_vec<T, V>(ya, x.a[i]);
                pack_vec<T, V>(yb, x.b[i]);
            }
        } else if ((p.inplace >> (int)is_k) & 1) {
            continue;
        }
#pragma unroll
        for (int i = 0; i < E; ++i) {
            if (e0[i] < p.D) *(Vt*)(dst + e0[i]) = x.a[i];
            if (e1[i] < p.D) *(Vt*)(dst + e1[i]) = x.b[i];
        }
    }
    pdl_trigger();
}

template <typename T, int V, int E>
cudaError_t launch_e(Params& p, bool paired, cudaStream_t s) {
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
    return paired ? launch_pdl(norm_rope_kernel<T, V, E, true>, grid, dim3(kThreads), smem, s, p, lpr_log2)
                  : launch_pdl(norm_rope_kernel<T, V, E, false>, grid, dim3(kThreads), smem, s, p, lpr_log2);
}

template <typename T, int V>
cudaError_t launch_v(Params& p, bool paired, cudaStream_t s) {
    constexpr int most = 8 / V;  // units a lane: D is at most 512
    p.ru = p.rot / (2 * V);
    p.units = p.ru + (p.D - p.rot + 2 * V - 1) / (2 * V);
    if constexpr (most > 1)
        if (p.units > 32) return launch_e<T, V, most>(p, paired, s);
    return launch_e<T, V, 1>(p, paired, s);
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
