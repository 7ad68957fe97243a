// rotary.cu -- rotary positions (ddtree_rope) and the append of new tokens to a
// paged KV cache with the rotation applied on the way (ddtree_append_paged).
//
// Rotation of pair j of a token at position p: (a + i b) -> (a + i b) e^{i p f_j} s,
// j in [0, rot/2), the pair being elements (j, j + rot/2) or (2j, 2j + 1).  The
// frequency is held in turns per position, as a 64-bit fraction F_j = f_j / 2pi
// * 2^64: p * F_j modulo 2^64 is then the angle's fraction of a turn exactly
// as an integer product leaves it, at any 32-bit position, with no range
// reduction in floating point (a 32-bit product p f_j is off by 0.06 rad at a
// million).  The top bits give the octant-centred remainder, sincospif the rest.
//
// HBM-bound: every row is read and written once.  A CTA takes some tokens: it
// fills their cosine / sine table (rot/2 entries each) in shared memory, so an
// angle is computed once a token and serves every head, then its threads go over
// (token, head, unit) items, a unit being two vectors -- the two halves of a
// group of pairs, or neighbours -- of the widest type that the sizes and
// addresses allow, the next item's loads in flight while one is turned.  Each
// thread's first item is loaded before the table is built, which takes the table
// off a small call's critical path; few tokens are cut by heads over more CTAs.
// CTAs are small (128 threads, 8 an SM) because each one's table and barrier
// leave it idle for a while: 256 threads and one token a CTA took 81 us for 16384
// tokens of 40 heads, D = 128, bf16, and 3.4 us for 65 tokens.  Issue slots came
// next (61 % busy): an item's token and head are stepped, not divided out, and
// 16-bit elements are taken and rounded in pairs, 63 -> 58 us (86 % of measured
// HBM), 2.5 us for 65 tokens.  A warp a token with its angles in registers and no
// table took 68 us (the angles are then computed once every 4 heads), two items
// in flight 70 (registers, so fewer CTAs).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "common.cuh"
#include "internal.h"

namespace ddt {

namespace {

constexpr int kThreads = 128;
constexpr int kMaxTok = 16;        // tokens per CTA, at most
constexpr int kTable = 2048;       // pairs of a CTA's tokens, at most
constexpr int kPasses = 8;         // rounds of a CTA's threads over its items, about
constexpr int kFill = 16;          // CTAs per SM that fill the GPU

template <typename T> DDT_DEV float to_f(T x);
template <> DDT_DEV float to_f<float>(float x) { return x; }
template <> DDT_DEV float to_f<__half>(__half x) { return __half2float(x); }
template <> DDT_DEV float to_f<__nv_bfloat16>(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T> DDT_DEV T from_f(float x);
template <> DDT_DEV float from_f<float>(float x) { return x; }
template <> DDT_DEV __half from_f<__half>(float x) { return __float2half_rn(x); }
template <> DDT_DEV __nv_bfloat16 from_f<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

// Two neighbours of a 16-bit type, in one word.
template <typename T> DDT_DEV float2 unpack2(uint32_t w);
template <> DDT_DEV float2 unpack2<__nv_bfloat16>(uint32_t w) { return make_float2(bf16lo(w), bf16hi(w)); }
template <> DDT_DEV float2 unpack2<__half>(uint32_t w) { return __half22float2(*(const __half2*)&w); }
template <typename T> DDT_DEV uint32_t pack2(float lo, float hi);
template <> DDT_DEV uint32_t pack2<__nv_bfloat16>(float lo, float hi) { return pack_bf16x2(lo, hi); }
template <> DDT_DEV uint32_t pack2<__half>(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *(const uint32_t*)&h;
}

template <typename T, int V>
struct alignas(sizeof(T) * V) Vec {
    T e[V];
};

// Turns the V pairs of two vectors: pairs (a.e[i], b.e[i]), or PAIRED neighbours,
// a's before b's.  In 32 bits, one rounding each.
DDT_DEV float2 turned(float a, float b, float c, float s) {
    return make_float2(fmaf(a, c, -(b * s)), fmaf(a, s, b * c));
}
template <typename T, int V, bool PAIRED>
DDT_DEV void turn_pairs(Vec<T, V>& a, Vec<T, V>& b, const float (&c)[V], const float (&s)[V]) {
    if constexpr (sizeof(T) == 2 && V > 1) {
        uint32_t* wa = reinterpret_cast<uint32_t*>(a.e);
        uint32_t* wb = reinterpret_cast<uint32_t*>(b.e);
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
            const float2 x = unpack2<T>(wa[i]), y = unpack2<T>(wb[i]);
            if constexpr (PAIRED) {
                const float2 p = turned(x.x, x.y, c[i], s[i]), q = turned(y.x, y.y, c[V / 2 + i], s[V / 2 + i]);
                wa[i] = pack2<T>(p.x, p.y);
                wb[i] = pack2<T>(q.x, q.y);
            } else {
                const float2 p = turned(x.x, y.x, c[2 * i], s[2 * i]);
                const float2 q = turned(x.y, y.y, c[2 * i + 1], s[2 * i + 1]);
                wa[i] = pack2<T>(p.x, q.x);
                wb[i] = pack2<T>(p.y, q.y);
            }
        }
    } else {
#pragma unroll
        for (int e = 0; e < V; ++e) {
            T& ra = PAIRED ? (2 * e < V ? a.e[2 * e] : b.e[2 * e - V]) : a.e[e];
            T& rb = PAIRED ? (2 * e + 1 < V ? a.e[2 * e + 1] : b.e[2 * e + 1 - V]) : b.e[e];
            const float2 p = turned(to_f(ra), to_f(rb), c[e], s[e]);
            ra = from_f<T>(p.x);
            rb = from_f<T>(p.y);
        }
    }
}

struct Params {
    RowsArg q, q_out, k, k_out, v;  // unused parts have 0 heads
    PagedArgs cache;                // append: where k and v go
    const int32_t* seq;             // append only
    const int32_t* pos;
    const uint64_t* turns;
    float scale;
    int T, D, rot, tok, B;
    int units;    // two-vector units per head
    int ru;       // ... of which rotated
    int heads;    // q, k and v heads of a token
    int chunk;    // ... of which a CTA takes
    int inplace;  // bit 0: q, bit 1: k (untouched parts are skipped)
    int inverse;
    uint32_t* err;
};

// cos and sin of `phase` / 2^64 turns.  |x| <= 1/4, so its rounding and
// sincospif's are relative to a small angle.
DDT_DEV float2 cos_sin(uint64_t phase) {
    const uint32_t top = (uint32_t)(phase >> 32);
    const uint32_t quad = (top + 0x20000000u) >> 30;
    const int32_t r = (int32_t)(top - (quad << 30));
    float s, c;
    sincospif((float)r * 0x1p-31f, &s, &c);
    if (quad & 1) {
        const float t = c;
        c = -s;
        s = t;
    }
    return (quad & 2) ? make_float2(-c, -s) : make_float2(c, s);
}

// V: elements per vector.  PAIRED: pairs (2j, 2j + 1), else (j, j + rot/2).
template <typename T, int V, bool PAIRED, bool APPEND>
__global__ void __launch_bounds__(kThreads, 8) rotary_kernel(const __grid_constant__ Params p) {
    using Vt = Vec<T, V>;
    // cos and sin of token t's pair V * u + e, at [t][e / 4][u][e % 4] (for V < 4:
    // [t][u][e]), so that a warp's 16-byte reads fall on different banks
    extern __shared__ __align__(16) float s_cos[];
    float* s_sin = s_cos + p.tok * (p.rot / 2);
    __shared__ int64_t s_dst[kMaxTok];  // page * page_stride + slot * slot_stride, or -1
    __shared__ int32_t s_pos[kMaxTok];
    const int tid = threadIdx.x;
    const int t0 = blockIdx.x * p.tok;
    const int nt = min(p.tok, p.T - t0);
    // (a head of more units than threads is cut along blockIdx.z)
    const int per = min(p.units, kThreads), per_pass = kThreads / per;  // heads of a pass
    const int u = blockIdx.z * kThreads + tid % per;
    const int h_first = blockIdx.y * p.chunk, heads = min(p.chunk, p.heads - h_first);
    const bool rotated = u < p.ru;
    // the unit's two vectors (the second may lie past an odd tail)
    const int e0 = rotated ? (PAIRED ? 2 * V * u : V * u) : p.rot + 2 * V * (u - p.ru);
    const int e1 = rotated && !PAIRED ? e0 + p.rot / 2 : e0 + V;
    const bool two = e1 < p.D;
    pdl_wait();

    struct Item {
        Vt a, b;
    };
    // an item's token and head, kept as a pair: no division a step
    struct At {
        int t, h;
    };
    auto step = [&](At& x) {
        for (x.h += per_pass; x.h >= h_first + heads; x.h -= heads) ++x.t;
    };
    auto load = [&](const At& x, Item& v) {
        const int64_t tok = t0 + x.t;
        const int hk = x.h - p.q.heads, hv = hk - p.k.heads;
        const T* s = hk < 0   ? (const T*)p.q.data + tok * p.q.ts + x.h * p.q.hs
                     : hv < 0 ? (const T*)p.k.data + tok * p.k.ts + hk * p.k.hs
                              : (const T*)p.v.data + tok * p.v.ts + hv * p.v.hs;
        v.a = *(const Vt*)(s + e0);
        if (two) v.b = *(const Vt*)(s + e1);
    };
    At next{tid / per < per_pass && u < p.units ? 0 : nt, h_first + tid / per};
    while (next.h >= h_first + heads) next.h -= heads, ++next.t;
    Item ahead;
    if (next.t < nt) load(next, ahead);

    // ---- the tokens' tables ----------------------------------------------------
    if (tid < nt) {
        const int pos = p.pos[t0 + tid];
        s_pos[tid] = pos;
        if constexpr (APPEND) {
            int64_t dst = -1;
            if (pos >= 0) {
                const int b = p.seq[t0 + tid];
                const int pg = pos / p.cache.page_size;
                if (b < 0 || b >= p.B || pg >= p.cache.max_pages) {
                    record_error(p.err, ERR_APPEND | ERR_BAD_INPUT);
                } else {
                    const int page = p.cache.table[b * p.cache.table_stride + pg];
                    if (page < 0 || page >= p.cache.num_pages)
                        record_error(p.err, ERR_APPEND | ERR_BAD_PAGE);
                    else
                        dst = page * p.cache.page_stride +
                              (pos - pg * p.cache.page_size) * p.cache.slot_stride;
                }
            }
            s_dst[tid] = dst;
        }
    }
    const int pairs = p.rot / 2;
    for (int j = tid; j < nt * pairs; j += kThreads) {
        const int t = j / pairs, f = j - t * pairs;
        const int pos = p.pos[t0 + t];
        const float2 cs = cos_sin((uint64_t)(uint32_t)max(pos, 0) * p.turns[f]);
        const int un = f / V, e = f - un * V;
        const int at = t * pairs + (V < 4 ? un * V + e : ((e >> 2) * p.ru + un) * 4 + (e & 3));
        s_cos[at] = cs.x * p.scale;
        s_sin[at] = (p.inverse ? -cs.y : cs.y) * p.scale;
    }
    __syncthreads();

    // ---- the items -------------------------------------------------------------
    while (next.t < nt) {
        Item x = ahead;
        const At at = next;
        step(next);
        if (next.t < nt) load(next, ahead);
        const int t = at.t, h = at.h;
        const int64_t tok = t0 + t;
        const int hk = h - p.q.heads, hv = hk - p.k.heads;
        T* dst;
        const bool turn = rotated && s_pos[t] >= 0 && (!APPEND || hv < 0);
        if (hk < 0) {
            if ((p.inplace & 1) && !turn) continue;
            dst = (T*)p.q_out.data + tok * p.q_out.ts + h * p.q_out.hs;
        } else if constexpr (APPEND) {
            if (s_dst[t] < 0) continue;
            dst = hv < 0 ? (T*)p.cache.k + s_dst[t] + hk * p.cache.head_stride
                         : (T*)p.cache.v + s_dst[t] + hv * p.cache.head_stride;
        } else {
            if ((p.inplace & 2) && !turn) continue;
            dst = (T*)p.k_out.data + tok * p.k_out.ts + hk * p.k_out.hs;
        }
        if (turn) {
            float c[V], s[V];
            const float* tc = s_cos + t * pairs;
            const float* ts = s_sin + t * pairs;
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
            turn_pairs<T, V, PAIRED>(x.a, x.b, c, s);
        }
        *(Vt*)(dst + e0) = x.a;
        if (two) *(Vt*)(dst + e1) = x.b;
    }
    pdl_trigger();
}

bool on_grid(const void* p, int64_t a, int64_t b, int64_t c, size_t es, int V) {
    return (uintptr_t)p % (es * V) == 0 && a % V == 0 && b % V == 0 && c % V == 0;
}

template <typename T, int V, bool APPEND>
cudaError_t launch_v(Params& p, bool paired, cudaStream_t s) {
    p.ru = p.rot / (2 * V);
    p.units = p.ru + (p.D - p.rot + 2 * V - 1) / (2 * V);
    // Tokens of a CTA: enough for kPasses rounds of its threads, as long as the CTAs
    // still fill the GPU; few tokens are cut by heads instead.
    const int64_t fill = (int64_t)num_sms() * kFill, units = (int64_t)p.heads * p.units;
    p.tok = 1;
    while (p.tok < kMaxTok && p.tok * units < kPasses * kThreads && 2 * p.tok * (p.rot / 2) <= kTable &&
           p.T / (2 * p.tok) >= fill)
        p.tok *= 2;
    const int64_t cuts = std::min((units + kThreads - 1) / kThreads, std::max<int64_t>(1, fill / p.T));
    p.chunk = (int)((p.heads + cuts - 1) / cuts);
    const dim3 grid((unsigned)((p.T + p.tok - 1) / p.tok), (unsigned)((p.heads + p.chunk - 1) / p.chunk),
                    (unsigned)((p.units + kThreads - 1) / kThreads));
    const size_t smem = (size_t)p.tok * p.rot * sizeof(float);
    return paired ? launch_pdl(rotary_kernel<T, V, true, APPEND>, grid, dim3(kThreads), smem, s, p)
                  : launch_pdl(rotary_kernel<T, V, false, APPEND>, grid, dim3(kThreads), smem, s, p);
}

// The widest vectors that sizes, strides and addresses allow: 16 bytes, 8, or
// single elements.
template <typename T, bool APPEND>
cudaError_t launch_t(Params& p, bool paired, cudaStream_t s) {
    constexpr int V16 = 16 / (int)sizeof(T), V8 = 8 / (int)sizeof(T);
    auto fits = [&](int V) {
        bool ok = p.rot / 2 % V == 0 && p.D % V == 0;
        for (const RowsArg* r : {&p.q, &p.q_out, &p.k, &p.k_out, &p.v})
            if (r->heads) ok = ok && on_grid(r->data, r->ts, r->hs, 0, sizeof(T), V);
        if (APPEND)
            for (const void* c : {p.cache.k, p.cache.v})
                ok = ok && on_grid(c, p.cache.page_stride, p.cache.head_stride,
                                   p.cache.slot_stride, sizeof(T), V);
        return ok;
    };
    if (fits(V16)) return launch_v<T, V16, APPEND>(p, paired, s);
    if (fits(V8)) return launch_v<T, V8, APPEND>(p, paired, s);
    return launch_v<T, 1, APPEND>(p, paired, s);
}

template <bool APPEND>
cudaError_t launch(Params& p, int dtype, bool paired, cudaStream_t s) {
    if (dtype == 0) return launch_t<__nv_bfloat16, APPEND>(p, paired, s);
    if constexpr (!APPEND)  // a cache has no 32-bit form
        if (dtype == 1) return launch_t<float, APPEND>(p, paired, s);
    return launch_t<__half, APPEND>(p, paired, s);
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& a, cudaStream_t s) {
    Params p{};
    p.q = a.q, p.q_out = a.q_out, p.k = a.k, p.k_out = a.k_out;
    p.pos = a.pos, p.turns = a.turns, p.scale = a.scale;
    p.T = a.T, p.D = a.D, p.rot = a.rot, p.inverse = a.inverse;
    p.heads = a.q.heads + a.k.heads;
    p.inplace = (a.q.data == a.q_out.data ? 1 : 0) | (a.k.data == a.k_out.data ? 2 : 0);
    return launch<false>(p, a.dtype, a.interleaved, s);
}

cudaError_t launch_append_paged(const AppendArgs& a, cudaStream_t s) {
    Params p{};
    p.q = a.q, p.q_out = a.q_out, p.k = a.k, p.v = a.v;
    p.cache = a.cache, p.seq = a.seq, p.pos = a.pos, p.turns = a.turns, p.scale = a.scale;
    p.T = a.T, p.D = a.cache.D, p.rot = a.rot, p.B = a.B;
    p.heads = a.q.heads + a.k.heads + a.v.heads;
    p.inplace = a.q.heads && a.q.data == a.q_out.data ? 1 : 0;
    p.err = a.err;
    return launch<true>(p, a.cache.dtype, a.interleaved, s);
}

}  // namespace ddt
