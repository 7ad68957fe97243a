// quant.cu -- the 8-bit cache's writers (ddtree_append_q8, ddtree_commit_q8) and its
// reader (ddtree_read_q8); q8.cuh has the format.
//
// Writers.  A CTA takes one block of the cache that a run touches, for one head of the
// keys or values (or of the queries, which only pass through): its rows in 32 bits in
// shared memory, normed and turned, their largest element, the exponent, the codes.
#include "q8.cuh"
#include "rotary.cuh"

namespace ddt {

namespace {

constexpr int kThreads = 128;
constexpr int kMaxBlock = DDTREE_MAX_Q8_BLOCK, kMaxD = 128;

struct WriteParams {
    RowsArg q, q_out, k, v;
    Q8Args cache;
    const int32_t *first, *at;                              // append
    const int32_t *accept_len, *accepted_nodes, *prefix_len;  // commit
    int32_t* new_len;
    const uint64_t* turns;
    NormArgs norm;
    float scale;
    int T, B, rot, L, N, slots;
    bool interleaved;
    uint32_t* err;
};

template <typename T, bool COMMIT>
__global__ void __launch_bounds__(kThreads) write_kernel(const __grid_constant__ WriteParams p) {
    __shared__ float s_x[kMaxBlock][kMaxD];
    __shared__ float s_max[kThreads / 32];
    __shared__ int s_node[DDTREE_MAX_L + 1];
    __shared__ int s_bad;
    const Q8Args& c = p.cache;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, S = c.block, D = c.D;
    const int64_t cap = (int64_t)c.max_pages * c.page_size;
    pdl_wait();
    RunBlock x;
    if constexpr (COMMIT) {
        x.b = blockIdx.x / p.slots;
        const int j = blockIdx.x % p.slots;
        const int P = p.prefix_len[x.b], a = p.accept_len[x.b];
        if (tid == 0) s_bad = 0;
        __syncthreads();
        if (a < 0 || a > p.L || P < 0 || (int64_t)P + a + 1 > cap) {
            if (tid == 0) s_bad = ERR_BAD_PREFIX_LEN;
        } else if (tid <= a) {
            const int node = tid ? p.accepted_nodes[(int64_t)x.b * p.L + tid - 1] : 0;
            const int page = c.table[x.b * c.table_stride + (P + tid) / c.page_size];
            s_node[tid] = node;
            if (tid && (node < 1 || node > p.N)) atomicMax(&s_bad, (int)ERR_BAD_TREE);
            else if (page < 0 || page >= c.num_pages) atomicMax(&s_bad, (int)ERR_BAD_PAGE);
        }
        __syncthreads();
        if (j == 0 && blockIdx.y == 0 && tid == 0) {
            if (s_bad) record_error(p.err, ERR_COMMIT | (uint32_t)s_bad);
            if (p.new_len) p.new_len[x.b] = s_bad ? P : P + a + 1;
        }
        if (s_bad) return;
        x.p0 = P / S * S + j * S;
        x.lo = max(x.p0, P);
        x.hi = min(x.p0 + S, P + a + 1);
        x.token = x.lo - P;  // (of the path)
        if (x.lo >= x.hi) return;
    } else {
        x = run_block(p.first, p.at, p.B, p.T, S, cap, blockIdx.x);
        if (tid == 0 && blockIdx.y == 0)
            check_run(p.first, p.at, p.B, p.T, cap, blockIdx.x, p.err, ERR_APPEND | ERR_BAD_INPUT);
        if (!x.ok) return;
    }
    const int h = blockIdx.y, hk = h - p.q.heads, hv = hk - c.Hkv;
    const bool is_q = hk < 0, is_v = hv >= 0;
    const int head = is_q ? h : (is_v ? hv : hk);
    const RowsArg& in = is_q ? p.q : (is_v ? p.v : p.k);
    const int page = c.table[x.b * c.table_stride + x.p0 / c.page_size];
    const bool there = page >= 0 && page < c.num_pages;
    if (!there && !is_q) {
        if (tid == 0) record_error(p.err, ERR_APPEND | ERR_BAD_PAGE);
        return;
    }
    const int rows = x.hi - x.lo;
    const bool norm = !is_v && p.norm.on;
    const float* w = is_q ? p.norm.q_weight : p.norm.k_weight;
    float most = 0.f;
    for (int r = warp; r < rows; r += kThreads / 32) {
        const int64_t token = COMMIT ? (int64_t)x.b * (p.N + 1) + s_node[x.token + r] : x.token + r;
        const T* row = (const T*)in.data + token * in.ts + head * in.hs;
        float* y = s_x[r];
        float sum = 0.f;
        for (int i = lane; i < D; i += 32) {
            y[i] = to_f(row[i]);
            sum = fmaf(y[i], y[i], sum);
        }
        if (norm) {
            for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
            const float f = rsqrtf(sum / D + p.norm.eps);
            for (int i = lane; i < D; i += 32) y[i] = y[i] * f * (w ? w[i] : 1.f);
        }
        __syncwarp();
        if (!is_v)
            for (int j = lane; j < p.rot / 2; j += 32) {
                const int a = p.interleaved ? 2 * j : j, b = p.interleaved ? 2 * j + 1 : j + p.rot / 2;
                const float2 cs = cos_sin((uint64_t)(uint32_t)(x.lo + r) * p.turns[j]);
                const float2 z = turned(y[a], y[b], cs.x * p.scale, cs.y * p.scale);
                y[a] = z.x;
                y[b] = z.y;
            }
        __syncwarp();
        for (int i = lane; i < D; i += 32) {
            most = fmaxf(most, fabsf(y[i]));
            if (is_q) ((T*)p.q_out.data + token * p.q_out.ts + head * p.q_out.hs)[i] = from_f<T>(y[i]);
        }
    }
    if (is_q) return;
    for (int d = 16; d; d >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, d));
    if (lane == 0) s_max[warp] = most;
    __syncthreads();
    most = fmaxf(fmaxf(s_max[0], s_max[1]), fmaxf(s_max[2], s_max[3]));
    const int slot0 = x.p0 % c.page_size, least = q8_least(c.dtype == 2);
    uint8_t* scale = (is_v ? c.v_scales : c.k_scales) +
                     ((int64_t)page * c.Hkv + head) * (c.page_size / S) + slot0 / S;
    uint8_t* codes = (is_v ? c.v : c.k) + page * c.page_stride + head * c.head_stride;
    int e = q8_exponent(most, least);
    if (x.lo > x.p0) {
        const int old = q8_from_byte(*scale, least);
        e = max(e, old);
        if (e > old)
            for (int i = tid; i < (x.lo - x.p0) * D; i += kThreads) {
                uint8_t* at = codes + (slot0 + i / D) * c.slot_stride + i % D;
                *at = (uint8_t)q8_pack2(q8_value(*at) * pow2(old - e), 0.f);
            }
    }
    const float f = pow2(-e);
    for (int i = tid; i < rows * D; i += kThreads)
        codes[(slot0 + x.lo - x.p0 + i / D) * c.slot_stride + i % D] = (uint8_t)q8_pack2(s_x[i / D][i % D] * f, 0.f);
    __syncthreads();  // (every thread has read the old scale)
    if (tid == 0) *scale = (uint8_t)(e + 127);
}

struct ReadParams {
    Q8Args cache;
    const int32_t *first, *at;
    RowsArg k_out, v_out;
    int B, T;
    uint32_t* err;
};

template <typename T>
__global__ void __launch_bounds__(kThreads) read_kernel(const __grid_constant__ ReadParams p) {
    const Q8Args& c = p.cache;
    const int S = c.block, D = c.D, head = blockIdx.y, half = blockIdx.z;
    pdl_wait();
    const int64_t cap = (int64_t)c.max_pages * c.page_size;
    const RunBlock x = run_block(p.first, p.at, p.B, p.T, S, cap, blockIdx.x);
    if (threadIdx.x == 0 && head == 0 && half == 0)
        check_run(p.first, p.at, p.B, p.T, cap, blockIdx.x, p.err, ERR_READ | ERR_BAD_INPUT);
    if (!x.ok) return;
    const int page = c.table[x.b * c.table_stride + x.p0 / c.page_size];
    if (page < 0 || page >= c.num_pages) {
        if (threadIdx.x == 0) record_error(p.err, ERR_READ | ERR_BAD_PAGE);
        return;
    }
    const int slot0 = x.p0 % c.page_size;
    const uint8_t* scales = half ? c.v_scales : c.k_scales;
    const float f = pow2(q8_from_byte(scales[((int64_t)page * c.Hkv + head) * (c.page_size / S) + slot0 / S],
                                      q8_least(c.dtype == 2)));
    const uint8_t* codes = (half ? c.v : c.k) + page * c.page_stride + head * c.head_stride;
    const RowsArg& out = half ? p.v_out : p.k_out;
    for (int i = threadIdx.x; i < (x.hi - x.lo) * D; i += kThreads) {
        const int r = i / D, d = i % D;
        const float y = q8_value(codes[(slot0 + x.lo - x.p0 + r) * c.slot_stride + d]) * f;
        ((T*)out.data + (int64_t)(x.token + r) * out.ts + head * out.hs)[d] = from_f<T>(y);
    }
}

}  // namespace

cudaError_t launch_append_q8(const AppendQ8Args& a, cudaStream_t s) {
    WriteParams p{};
    p.q = a.q, p.q_out = a.q_out, p.k = a.k, p.v = a.v, p.cache = a.cache;
    p.first = a.first, p.at = a.at, p.turns = a.turns, p.norm = a.norm, p.scale = a.scale;
    p.T = a.T, p.B = a.B, p.rot = a.rot, p.interleaved = a.interleaved, p.err = a.err;
    const int64_t slots = run_slots(a.B, a.T, a.cache.block);
    if (slots > INT32_MAX) return cudaErrorInvalidValue;
    const dim3 grid((unsigned)slots, (unsigned)(a.q.heads + 2 * a.cache.Hkv));
    return a.cache.dtype == 2 ? launch_pdl(write_kernel<__half, false>, grid, dim3(kThreads), 0, s, p)
                              : launch_pdl(write_kernel<__nv_bfloat16, false>, grid, dim3(kThreads), 0, s, p);
}

cudaError_t launch_commit_q8(const CommitQ8Args& a, cudaStream_t s) {
    WriteParams p{};
    p.k = a.k_tree, p.v = a.v_tree, p.cache = a.cache;
    p.accept_len = a.accept_len, p.accepted_nodes = a.accepted_nodes, p.prefix_len = a.prefix_len;
    p.new_len = a.new_len, p.B = a.B, p.L = a.L, p.N = a.N, p.err = a.err;
    p.slots = (a.L + 1 - 2 + a.cache.block) / a.cache.block + 1;  // blocks that L + 1 positions touch
    const dim3 grid((unsigned)(a.B * p.slots), (unsigned)(2 * a.cache.Hkv));
    return a.cache.dtype == 2 ? launch_pdl(write_kernel<__half, true>, grid, dim3(kThreads), 0, s, p)
                              : launch_pdl(write_kernel<__nv_bfloat16, true>, grid, dim3(kThreads), 0, s, p);
}

cudaError_t launch_read_q8(const ReadQ8Args& a, cudaStream_t s) {
    ReadParams p{a.cache, a.first, a.at, a.k_out, a.v_out, a.B, a.T, a.err};
    const int64_t slots = run_slots(a.B, a.T, a.cache.block);
    if (slots > INT32_MAX) return cudaErrorInvalidValue;
    const dim3 grid((unsigned)slots, (unsigned)a.cache.Hkv, 2);
    return a.cache.dtype == 2 ? launch_pdl(read_kernel<__half>, grid, dim3(kThreads), 0, s, p)
                              : launch_pdl(read_kernel<__nv_bfloat16>, grid, dim3(kThreads), 0, s, p);
}

}  // namespace ddt
