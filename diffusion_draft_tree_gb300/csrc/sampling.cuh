// sampling.cuh -- the target's temperature-T decoding rule, shared by the
// full-tree and path-only accept kernels: one Philox4x64-10 uniform per node.
#pragma once

#include "common.cuh"

namespace ddt {

// Philox4x64-10 (Salmon, Moraes, Dror, Shaw, SC'11): ten rounds of two 64x64
// multiplies with the Weyl key schedule.
DDT_DEV void philox4x64_10(uint64_t c[4], uint64_t k0, uint64_t k1) {
#pragma unroll
    for (int r = 0; r < 10; ++r) {
        const uint64_t lo0 = 0xD2E7470EE14C6C93ull * c[0], hi0 = __umul64hi(0xD2E7470EE14C6C93ull, c[0]);
        const uint64_t lo1 = 0xCA5A826395121157ull * c[2], hi1 = __umul64hi(0xCA5A826395121157ull, c[2]);
        const uint64_t x0 = hi1 ^ c[1] ^ k0, x2 = hi0 ^ c[3] ^ k1;
        c[0] = x0; c[1] = lo1; c[2] = x2; c[3] = lo0;
        k0 += 0x9E3779B97F4A7C15ull;
        k1 += 0xBB67AE8584CAA73Bull;
    }
}

DDT_DEV float node_uniform(uint64_t seed, uint64_t step, uint64_t seq, uint64_t node) {
    uint64_t c[4] = {seq, node, 0ull, 0ull};
    philox4x64_10(c, seed, step);
    return (float)(c[0] >> 40) * (1.0f / 16777216.0f);
}

}  // namespace ddt
