// rotary.cuh -- what the kernels that rotate share: element types, vectors, cosine
// and sine of a position's turn (rotary.cu has the mathematics).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"
#include "internal.h"

namespace ddt {

namespace {

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

// A lane's share of a head in 32 bits: the first and the second elements of V pairs, whose
// places are two vectors -- one each, or PAIRED neighbours, the first vector's before
// the second's -- so that two pairs are worked on by an instruction, however they lie.
//
// Where the first (second) element of pair e is, in a head whose vectors are at e0 and e1.
template <int V, bool PAIRED>
DDT_DEV int place_of_pair(int e0, int e1, int e, bool second) {
    if constexpr (!PAIRED) return (second ? e1 : e0) + e;
    const int i = 2 * e + (second ? 1 : 0);
    return i < V ? e0 + i : e1 + i - V;
}
template <typename T, int V, bool PAIRED>
DDT_DEV void unpack_pairs(const Vec<T, V>& va, const Vec<T, V>& vb, float (&a)[V], float (&b)[V]) {
    if constexpr (sizeof(T) == 2 && V > 1) {
        const uint32_t* wa = reinterpret_cast<const uint32_t*>(va.e);
        const uint32_t* wb = reinterpret_cast<const uint32_t*>(vb.e);
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
            const float2 x = unpack2<T>(wa[i]), y = unpack2<T>(wb[i]);
            if constexpr (PAIRED) {
                a[i] = x.x, b[i] = x.y;
                a[V / 2 + i] = y.x, b[V / 2 + i] = y.y;
            } else {
                a[2 * i] = x.x, a[2 * i + 1] = x.y;
                b[2 * i] = y.x, b[2 * i + 1] = y.y;
            }
        }
    } else {
#pragma unroll
        for (int e = 0; e < V; ++e) {
            a[e] = to_f(PAIRED ? (2 * e < V ? va.e[2 * e % V] : vb.e[2 * e % V]) : va.e[e]);
            b[e] = to_f(PAIRED ? (2 * e + 1 < V ? va.e[(2 * e + 1) % V] : vb.e[(2 * e + 1) % V]) : vb.e[e]);
        }
    }
}
template <typename T, int V, bool PAIRED>
DDT_DEV void pack_pairs(const float (&a)[V], const float (&b)[V], Vec<T, V>& va, Vec<T, V>& vb) {
    if constexpr (sizeof(T) == 2 && V > 1) {
        uint32_t* wa = reinterpret_cast<uint32_t*>(va.e);
        uint32_t* wb = reinterpret_cast<uint32_t*>(vb.e);
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
            wa[i] = PAIRED ? pack2<T>(a[i], b[i]) : pack2<T>(a[2 * i], a[2 * i + 1]);
            wb[i] = PAIRED ? pack2<T>(a[V / 2 + i], b[V / 2 + i]) : pack2<T>(b[2 * i], b[2 * i + 1]);
        }
    } else {
#pragma unroll
        for (int e = 0; e < V; ++e) {
            (PAIRED ? (2 * e < V ? va.e[2 * e % V] : vb.e[2 * e % V]) : va.e[e]) = from_f<T>(a[e]);
            (PAIRED ? (2 * e + 1 < V ? va.e[(2 * e + 1) % V] : vb.e[(2 * e + 1) % V]) : vb.e[e]) = from_f<T>(b[e]);
        }
    }
}
template <int V>
DDT_DEV void scale_vec(float (&y)[V], const float (&s)[V]) {
    if constexpr (V > 1) {
#pragma unroll
        for (int i = 0; i < V; i += 2) mul2(y[i], y[i + 1], s[i], s[i + 1]);
    } else {
        y[0] *= s[0];
    }
}
template <int V>
DDT_DEV void scale_by(float (&y)[V], float s) {
    if constexpr (V > 1) {
#pragma unroll
        for (int i = 0; i < V; i += 2) mul2(y[i], y[i + 1], s, s);
    } else {
        y[0] *= s;
    }
}
// Sums of squares, even and odd elements apart.
template <int V>
DDT_DEV void add_squares(const float (&y)[V], float& s0, float& s1) {
    if constexpr (V > 1) {
#pragma unroll
        for (int i = 0; i < V; i += 2) fma2(s0, s1, y[i], y[i + 1], y[i], y[i + 1]);
    } else {
        s0 = fmaf(y[0], y[0], s0);
    }
}
template <int V>
DDT_DEV void turn_vec(float (&a)[V], float (&b)[V], const float (&c)[V], const float (&s)[V]) {
    if constexpr (V > 1) {
#pragma unroll
        for (int i = 0; i < V; i += 2) {
            const float x0 = a[i], x1 = a[i + 1];
            float t0 = b[i], t1 = b[i + 1];
            mul2(t0, t1, s[i], s[i + 1]);
            a[i] = fmaf(x0, c[i], -t0), a[i + 1] = fmaf(x1, c[i + 1], -t1);
            mul2(b[i], b[i + 1], c[i], c[i + 1]);
            fma2(b[i], b[i + 1], x0, x1, s[i], s[i + 1]);
        }
    } else {
        const float x = a[0];
        a[0] = fmaf(x, c[0], -(b[0] * s[0]));
        b[0] = fmaf(x, s[0], b[0] * c[0]);
    }
}

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

inline bool on_grid(const void* p, int64_t a, int64_t b, int64_t c, size_t es, int V) {
    return (uintptr_t)p % (es * V) == 0 && a % V == 0 && b % V == 0 && c % V == 0;
}

}  // namespace

}  // namespace ddt
