// tree_attn_q8.cu -- ddtree_tree_attn_q8: tree attention over an 8-bit paged cache.
//
//   out[r] = sum_j w_rj v_j / sum_j w_rj,  w_rj = 2^(x_rj - m_r),  x = scale log2e q k
//
// A CTA takes kRows query rows (node-major, the G heads of a node together) of a KV head
// of a sequence, and goes over its keys kKeys at a time, widened to 32 bits in shared
// memory, with the running maximum and sum of each row.
#include "q8.cuh"
#include "rotary.cuh"

namespace ddt {

namespace {

constexpr int kThreads = 256, kRows = 16, kKeys = 32;

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) tree_attn_q8_kernel(const __grid_constant__ Q8AttnArgs a, int tiles) {
    __shared__ float s_q[kRows][D], s_k[kKeys][D + 1], s_v[kKeys][D], s_p[kRows][kKeys + 1];
    const Q8Args& c = a.cache;
    const int tid = threadIdx.x, R = a.N + 1, Hq = a.q.heads, G = Hq / c.Hkv, W = (R + 31) / 32, S = c.block;
    const int tile = blockIdx.x % tiles, g = blockIdx.x / tiles % c.Hkv, b = blockIdx.x / tiles / c.Hkv;
    pdl_wait();
    const int P = a.prefix_len[b], n = a.n_nodes[b];
    if (P < 0 || P > (int64_t)c.max_pages * c.page_size || n < 0 || n > a.N) {
        if (tid == 0 && tile == 0 && g == 0)
            record_error(a.err, ERR_ATTN | (n < 0 || n > a.N ? ERR_BAD_N_NODES : ERR_BAD_PREFIX_LEN));
        return;
    }
    const int row0 = tile * kRows, least = q8_least(c.dtype == 2);
    for (int i = tid; i < kRows * D; i += kThreads) {
        const int r = row0 + i / D, u = r / G;
        s_q[i / D][i % D] = u <= n ? to_f(((const T*)a.q.data + ((int64_t)b * R + u) * a.q.ts + (g * G + r % G) * a.q.hs)[i % D])
                                   : 0.f;
    }
    constexpr int C = D / 16;
    const int r = tid / 16, l = tid % 16, u = (row0 + r) / G;
    const uint32_t* mask = a.anc_mask + ((int64_t)b * R + min(u, a.N)) * W;
    const float sl2 = a.scale * kLog2e;
    float m = -INFINITY, sum = 0.f, o[C] = {};
    const int keys = P + n + 1;
    for (int j0 = 0; j0 < keys; j0 += kKeys) {
        __syncthreads();
        for (int i = tid; i < kKeys * D; i += kThreads) {
            const int j = j0 + i / D, d = i % D;
            float kx = 0.f, vx = 0.f;
            if (j < P) {
                const int page = c.table[b * c.table_stride + j / c.page_size], slot = j % c.page_size;
                if (page < 0 || page >= c.num_pages) {
                    record_error(a.err, ERR_ATTN | ERR_BAD_PAGE);
                } else {
                    const int64_t at = page * c.page_stride + g * c.head_stride + slot * c.slot_stride + d;
                    const int64_t sc = ((int64_t)page * c.Hkv + g) * (c.page_size / S) + slot / S;
                    kx = q8_value(c.k[at]) * pow2(q8_from_byte(c.k_scales[sc], least));
                    vx = q8_value(c.v[at]) * pow2(q8_from_byte(c.v_scales[sc], least));
                }
            } else if (j < keys) {
                const int64_t t = (int64_t)b * R + j - P;
                kx = to_f(((const T*)a.k_tree.data + t * a.k_tree.ts + g * a.k_tree.hs)[d]);
                vx = to_f(((const T*)a.v_tree.data + t * a.v_tree.ts + g * a.v_tree.hs)[d]);
            }
            s_k[i / D][d] = kx;
            s_v[i / D][d] = vx;
        }
        __syncthreads();
        float x[2], most = -INFINITY;
        for (int e = 0; e < 2; ++e) {
            const int k = l + 16 * e, j = j0 + k;
            float dot = 0.f;
            for (int d = 0; d < D; ++d) dot = fmaf(s_q[r][d], s_k[k][d], dot);
            bool see = u <= n && j < keys;
            if (see && j >= P) see = (mask[(j - P) / 32] >> ((j - P) % 32)) & 1u;
            x[e] = see ? dot * sl2 : -INFINITY;
            most = fmaxf(most, x[e]);
        }
        for (int d = 8; d; d >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, d, 16));
        const float m2 = fmaxf(m, most), ref = m2 == -INFINITY ? 0.f : m2, f = exp2f(m - ref);
        m = m2;
        sum *= f;
        for (int e = 0; e < 2; ++e) {
            const float w = exp2f(x[e] - ref);
            sum += w;
            s_p[r][l + 16 * e] = w;
        }
        __syncwarp();
        for (int i = 0; i < C; ++i) {
            float acc = o[i] * f;
            for (int k = 0; k < kKeys; ++k) acc = fmaf(s_p[r][k], s_v[k][l + 16 * i], acc);
            o[i] = acc;
        }
    }
    for (int d = 8; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d, 16);
    if (u >= R) return;
    const int64_t at = ((int64_t)b * R + u) * Hq + g * G + (row0 + r) % G;
    const bool live = u <= n && sum > 0.f;
    for (int i = 0; i < C; ++i) ((T*)a.out)[at * D + l + 16 * i] = from_f<T>(live ? o[i] / sum : 0.f);
    if (l == 0 && a.lse) a.lse[at] = live ? (m + log2f(sum)) * 0.6931471805599453f : -INFINITY;
}

template <typename T, int D>
cudaError_t launch(const Q8AttnArgs& a, cudaStream_t s) {
    const int64_t rows = (int64_t)(a.N + 1) * (a.q.heads / a.cache.Hkv);
    const int tiles = (int)((rows + kRows - 1) / kRows);
    const int64_t grid = (int64_t)tiles * a.B * a.cache.Hkv;
    if (grid > INT32_MAX) return cudaErrorInvalidValue;
    return launch_pdl(tree_attn_q8_kernel<T, D>, dim3((unsigned)grid), dim3(kThreads), 0, s, a, tiles);
}

}  // namespace

size_t q8_attn_workspace_bytes(int, int, int, int, int, int64_t) { return 0; }

cudaError_t launch_tree_attn_q8(const Q8AttnArgs& a, cudaStream_t s) {
    if (a.cache.D == 128) return a.cache.dtype == 2 ? launch<__half, 128>(a, s) : launch<__nv_bfloat16, 128>(a, s);
    return a.cache.dtype == 2 ? launch<__half, 64>(a, s) : launch<__nv_bfloat16, 64>(a, s);
}

}  // namespace ddt
