// q8.cuh -- the 8-bit cache's format: e4m3 codes under a power of two for each block of
// positions of a page and head, and where a run's blocks lie.
//
// A code c stands for c * 2^e, also the two that e4m3 itself has for no number: 480 and -480, as
// their bits say.  The exponent of a block is the least e at which its
// largest element is at most 448 * 2^e (448 = 1.75 * 2^8 is the largest code), so that its
// significand is found by a power of two alone: x * 2^-e is exact, the one rounding is to
// the code, and c * 2^e is exact in bf16 always and in fp16 from e = -15 (the smallest
// code's step is then fp16's own, 2^-24) to 7 (448 * 2^7 = 57344).  bf16 stops at 7 too:
// its codes are widened by a product with 2^(120 + e), which has to be a bf16 number.
#pragma once

#include <algorithm>

#include "common.cuh"
#include "internal.h"

namespace ddt {

namespace {

constexpr int kQ8Most = 7;
__host__ __device__ constexpr int q8_least(bool f16) { return f16 ? -15 : -96; }

// The largest of three numbers, NaN if one of them is.
DDT_DEV float max_nan(float a, float b, float c) {
    float r;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
DDT_DEV float pow2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }  // -126 <= e <= 127
// The exponent of a block whose largest element is amax >= 0.
DDT_DEV int q8_exponent(float amax, int least) {
    const uint32_t b = __float_as_uint(amax);
    const int e = (int)(b >> 23) - 135 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);
    return min(max(e, least), kQ8Most);
}
DDT_DEV int q8_from_byte(uint32_t x, int least) { return min(max((int)x - 127, least), kQ8Most); }

// Two elements as codes, lo in the low byte: to the nearest, ties to even, at most 448.
DDT_DEV uint32_t q8_pack2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}
DDT_DEV uint32_t q8_pack4(float a, float b, float c, float d) {
    return __byte_perm(q8_pack2(a, b), q8_pack2(c, d), 0x5410);
}
// Four codes moved to a scale 2^-shift as large: rounded once more where they fall below
// the normal codes.
DDT_DEV uint32_t q8_moved(uint32_t w, float factor) {
    float v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t c = w >> (8 * i);
        v[i] = __uint_as_float((c & 0x80u) << 24 | (c & 0x7fu) << 20) * 0x1p120f * factor;
    }
    return q8_pack4(v[0], v[1], v[2], v[3]);
}
// Codes as elements of the tokens' type.  Each code's exponent and significand bits move to the
// type's places and its sign bit to the top, which is a number 2^-8 (fp16) or 2^-120
// (bf16) of the code's, subnormal codes included; one packed product with the block's scale
// and that power gives the value, exactly.  (bf16's product takes and gives subnormal
// numbers as they are.)  Four instructions a pair: a byte permute puts a code under a
// byte of its sign bit eight times, a shift brings both to their places, a mask
// takes the sign bits between them away.
// All 256 codes are numbers here, 0x7F and 0xFF +-480 as their bits say.  (fp16 has a conversion
// of pairs of codes, which takes those two for NaN and forgets their signs; it left the product
// alone to do: tree attention over fp16 then took 2.86 ms for 2.99 (70B-class long context) and
// 490 us for 533 (ragged serving).)
//
// What that product takes for a block's scale byte, as the type's bits.
template <bool F16>
DDT_DEV uint32_t widen_factor(uint32_t byte) {
    const int e = q8_from_byte(byte, q8_least(F16));
    return F16 ? (uint32_t)(23 + e) << 10 : (uint32_t)(247 + e) << 7;
}
// Two codes of a word, by a permutation that gives (code, its sign, code, its sign).
template <bool F16, uint32_t SEL>
DDT_DEV uint32_t widen(uint32_t w, uint32_t factors) {
    uint32_t t;
    asm("prmt.b32 %0, %1, 0, %2;" : "=r"(t) : "r"(w), "n"(SEL));
    uint32_t r = F16 ? (t << 7) & 0xbf80bf80u : (t << 4) & 0x87f087f0u;
    if constexpr (F16) asm("mul.rn.f16x2 %0, %0, %1;" : "+r"(r) : "r"(factors));
    else asm("mul.rn.bf16x2 %0, %0, %1;" : "+r"(r) : "r"(factors));
    return r;
}
template <bool F16>
DDT_DEV uint32_t widen_even(uint32_t w, uint32_t factors) { return widen<F16, 0xa280>(w, factors); }
template <bool F16>
DDT_DEV uint32_t widen_odd(uint32_t w, uint32_t factors) { return widen<F16, 0xb391>(w, factors); }
// Codes 0, 1 and codes 2, 3 of a word as pairs in their order.
template <bool F16>
DDT_DEV uint32_t widen_lo(uint32_t w, uint32_t factors) { return widen<F16, 0x9180>(w, factors); }
template <bool F16>
DDT_DEV uint32_t widen_hi(uint32_t w, uint32_t factors) { return widen<F16, 0xb3a2>(w, factors); }

// Attention's copy warps hold a box of positions (a page, or as much of it as a key tile takes) a
// lane: its page number and the up to 16 bytes of its scales, a power of two of them.  `from`:
// the scale of the box's first position.
DDT_DEV uint4 box_scales(const uint8_t* from, int per_box) {
    uint4 y = make_uint4(0u, 0u, 0u, 0u);
    if (per_box == 1) y.x = __ldg(from);
    else if (per_box == 2) y.x = __ldg((const uint16_t*)from);
    else if (per_box == 4) y.x = __ldg((const uint32_t*)from);
    else if (per_box == 8) *(uint2*)&y = __ldg((const uint2*)from);
    else y = __ldg((const uint4*)from);
    return y;
}
// The scale byte of keys 4 l .. 4 l + 3 of a tile for lane l (a block is 8 keys or more), the tile's
// boxes held by the lanes from `first` on; warp-collective.
DDT_DEV uint32_t tile_scale(const uint4& y, int first, int box_log2, int block_log2, int per_box, int lane) {
    const int src = (first + (4 * lane >> box_log2)) & 31, byte = (4 * lane & ((1 << box_log2) - 1)) >> block_log2;
    uint32_t word = __shfl_sync(0xffffffffu, y.x, src);
    if (per_box > 4) {
        const uint32_t w1 = __shfl_sync(0xffffffffu, y.y, src), w2 = __shfl_sync(0xffffffffu, y.z, src),
                       w3 = __shfl_sync(0xffffffffu, y.w, src);
        word = byte < 4 ? word : byte < 8 ? w1 : byte < 12 ? w2 : w3;
    }
    return (word >> (8 * (byte & 3))) & 0xffu;
}

// A run's tokens first[b] .. first[b + 1] - 1 become positions at[b] .. of sequence b.  Whether
// it is one that no call may carry out: outside the T tokens or the table's positions.
DDT_DEV bool run_bad(int f, int n, int p, int T, int64_t cap) {
    return n != 0 && (f < 0 || n < 0 || (int64_t)f + n > T || p < 0 || (int64_t)p + n > cap);
}
// One block of a run: positions [p0, p0 + S) of the sequence, of which [lo, hi) are the run's.
struct RunBlock {
    int b, lo, hi, p0;
    int token;  // of position lo
    bool ok;    // there is such a block, and its run is not a bad one
};
// Runs cover their blocks by slots: sequence b has slots first[b] / S + 2 b and up, two more
// than its tokens fill, as n tokens touch at most (n - 2) / S + 2 blocks.  The slots'
// starts are known without adding up the runs before, so a CTA finds its own by halving.  Where
// `first` descends the starts do too, and halving may miss some of a run's slots: the starts it
// meets on its way to a run are the same from every slot, so each CTA of the run sees from
// them whether all of its slots get here, and none takes it up otherwise.
DDT_DEV RunBlock run_block(const int32_t* first, const int32_t* at, int B, int T, int block_log2, int64_t cap,
                           int slot) {
    const int S = 1 << block_log2;
    int lo = 0, hi = B - 1;  // the last sequence whose slots start at or before this one
    auto start_of = [&](int f, int b) { return (min(f, T) >> block_log2) + 2 * b; };  // (at most run_slots)
    int before = INT32_MIN, after = INT32_MAX;  // starts met on the way: the last and the first
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        const int start = start_of(first[mid], mid);
        const bool here = start <= slot;
        lo = here ? mid : lo;
        hi = here ? hi : mid - 1;
        before = max(before, here ? start : INT32_MIN);
        after = min(after, here ? INT32_MAX : start);
    }
    RunBlock x{};
    x.b = lo;
    const int f = first[lo], n = first[lo + 1] - f, p = at[lo];
    const int start = start_of(f, lo);
    const int64_t j = (int64_t)slot - start;
    if (j < 0 || n == 0 || run_bad(f, n, p, T, cap)) return x;
    const int last = ((p + n - 1) >> block_log2) - (p >> block_log2);  // its last slot
    if (before > start || (int64_t)start + last >= after) return x;
    x.p0 = (int)min((int64_t)(p & -S) + j * S, (int64_t)INT32_MAX - S);
    x.lo = max(x.p0, p);
    x.hi = min(x.p0 + S, p + n);
    x.ok = x.lo < x.hi;
    x.token = f + (x.lo - p);
    return x;
}
// Records a bad run; every run has a slot of its own number.
DDT_DEV void check_run(const int32_t* first, const int32_t* at, int B, int T, int64_t cap, int64_t slot,
                       uint32_t* err, uint32_t code) {
    if (slot < B && run_bad(first[slot], first[slot + 1] - first[slot], at[slot], T, cap)) record_error(err, code);
}
inline int64_t run_slots(int B, int T, int S) { return (int64_t)T / S + 2 * (int64_t)B; }

}  // namespace

}  // namespace ddt
