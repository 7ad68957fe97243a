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

// Elements in 32 bits into a vector, rounded once.
template <typename T, int V>
DDT_DEV void pack_vec(const float (&y)[V], Vec<T, V>& v) {
    if constexpr (sizeof(T) == 2 && V > 1) {
        uint32_t* w = reinterpret_cast<uint32_t*>(v.e);
#pragma unroll
        for (int i = 0; i < V / 2; ++i) w[i] = pack2<T>(y[2 * i], y[2 * i + 1]);
    } else {
#pragma unroll
        for (int e = 0; e < V; ++e) v.e[e] = from_f<T>(y[e]);
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
