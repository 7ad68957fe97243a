// commit.cu -- after the walk: the accepted path joins the KV cache
// ("Accelerating Speculative Decoding with Block Diffusion Draft Trees", §3 and
// §4.1: the bonus token that rooted the tree and the accepted tokens are
// verified, so they become part of the prefix the next round attends to).
//
// One CTA per sequence.  The path rows are node 0 (the root) followed by the
// a = accept_len accepted nodes; row i of the path holds its tokens' keys and
// values for every KV head in the tree K/V and moves to cache position P + i
// (its depth is i, and tree keys were computed at position P + depth).  The
// CTA reads P and the path once, copies (a+1) x Hkv rows of D bf16 for K and
// V with 16-byte accesses, then advances prefix_len[b] to P + a + 1 -- in
// place, which is safe because only this CTA touches sequence b.  HBM-bound;
// algorithmic bytes per sequence 8 (a+1) Hkv D (K and V, read and written).
#include "common.cuh"
#include "internal.h"

#include "../../include/ddtree.h"

namespace ddt {

namespace {

constexpr int kThreads = 256;

__global__ void __launch_bounds__(kThreads)
commit_kernel(uint4* __restrict__ k_cache, uint4* __restrict__ v_cache, int64_t cache_cap,
              const uint4* __restrict__ k_tree, const uint4* __restrict__ v_tree,
              const int32_t* __restrict__ accept_len, const int32_t* __restrict__ accepted_nodes,
              int32_t* __restrict__ prefix_len, int L, int N, int Hkv, int D, uint32_t* err) {
    __shared__ int s_rows[DDTREE_MAX_L + 1];
    __shared__ int s_ok;
    __shared__ int64_t s_P;
    __shared__ int s_a;
    const int b = blockIdx.x, tid = threadIdx.x;
    pdl_wait();
    if (tid == 0) {
        const int64_t P = prefix_len[b];
        const int a = accept_len[b];
        s_P = P;
        s_a = a;
        s_ok = (a >= 0 && a <= L && P >= 0 && P + a + 1 <= cache_cap) ? 1 : 0;
        s_rows[0] = 0;
        if (!s_ok) record_error(err, ERR_COMMIT | ERR_BAD_PREFIX_LEN);
    }
    __syncthreads();
    const int a = s_a;
    if (s_ok && tid < a) {
        const int u = accepted_nodes[(size_t)b * L + tid];
        s_rows[tid + 1] = u;
        if (u < 1 || u > N) {
            s_ok = 0;
            record_error(err, ERR_COMMIT | ERR_BAD_TREE);
        }
    }
    __syncthreads();
    pdl_trigger();
    if (!s_ok) return;
    const int64_t P = s_P;
    const int vd = D / 8;                 // 16-byte vectors per row
    const int per_row = Hkv * vd;
    const int R = N + 1;
    const int total = (a + 1) * per_row;
    for (int i = tid; i < total; i += kThreads) {
        const int r = i / per_row, rem = i - r * per_row;
        const int g = rem / vd, c = rem - g * vd;
        const size_t src = (((size_t)b * R + s_rows[r]) * Hkv + g) * vd + c;
        const size_t dst = (((size_t)b * Hkv + g) * (size_t)cache_cap + (size_t)(P + r)) * vd + c;
        k_cache[dst] = __ldg(&k_tree[src]);
        v_cache[dst] = __ldg(&v_tree[src]);
    }
    __syncthreads();
    if (tid == 0) prefix_len[b] = (int32_t)(P + a + 1);
}

// The same commit into a paged cache.  One CTA per (path row, sequence): each
// checks the whole path and its pages with one warp -- lane i row i, L + 1 <= 17
// rows -- so that all of a sequence's CTAs reach the same verdict without
// talking to each other, then copies its row's Hkv heads of K and V, 16 bytes a
// thread.  A row of a few KB is latency, not bandwidth: three dependent round
// trips (lengths, nodes and pages, the row).  With a CTA a row every copy is in
// flight at once, where one CTA a sequence would take up to 17 turns, and with
// 128 threads a CTA all rows of 128 sequences are resident at once (4.2 us; 256
// threads 4.8, 64 threads 4.5).
constexpr int kPagedThreads = 128, kAhead = 2;

__global__ void __launch_bounds__(kPagedThreads)
commit_paged_kernel(const __grid_constant__ PagedArgs c, const RowsArg kt, const RowsArg vt,
                    const int32_t* __restrict__ accept_len,
                    const int32_t* __restrict__ accepted_nodes,
                    const int32_t* __restrict__ prefix_len, int32_t* __restrict__ new_len, int L,
                    int N, uint32_t* err) {
    __shared__ int s_ok, s_node, s_page;
    const int b = blockIdx.y, row = blockIdx.x, tid = threadIdx.x;
    pdl_wait();
    const int P = prefix_len[b], a = accept_len[b];
    if (tid < 32) {
        // what is wrong with path row `tid`, the first kind found over the warp
        uint32_t bad = 0;
        int node = 0, page = 0;
        if (a < 0 || a > L || P < 0 || (int64_t)P + a + 1 > (int64_t)c.max_pages * c.page_size) {
            bad = ERR_BAD_PREFIX_LEN;
        } else if (tid <= a) {
            if (tid > 0) node = accepted_nodes[(size_t)b * L + tid - 1];
            page = c.table[b * c.table_stride + (P + tid) / c.page_size];
            if (tid > 0 && (node < 1 || node > N)) bad = ERR_BAD_TREE;
            else if (page < 0 || page >= c.num_pages) bad = ERR_BAD_PAGE;
        }
        const uint32_t worst = __reduce_max_sync(0xffffffffu, bad);
        if (tid == 0) {
            s_ok = worst == 0;
            if (worst && row == 0) record_error(err, ERR_COMMIT | worst);
        }
        if (tid == row) {
            s_node = node;
            s_page = page;
        }
    }
    __syncthreads();
    pdl_trigger();
    if (row == 0 && tid == 0 && new_len) new_len[b] = s_ok ? P + a + 1 : P;
    if (!s_ok || row > a) return;
    const int vd = c.D / 8;
    const int64_t tok = (int64_t)b * (N + 1) + s_node;
    const int64_t dst = s_page * c.page_stride + (P + row) % c.page_size * c.slot_stride;
    const int total = 2 * c.Hkv * vd;  // vectors, K's then V's
    auto place = [&](const RowsArg& src, int j) {
        const int g = j / vd, e = (j - g * vd) * 8;
        return (const uint4*)((const uint16_t*)src.data + tok * src.ts + g * src.hs + e);
    };
    for (int i0 = tid; i0 < total; i0 += kAhead * kPagedThreads) {
        uint4 x[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int i = i0 + k * kPagedThreads, j = i < total / 2 ? i : i - total / 2;
            if (i < total) x[k] = __ldg(place(i < total / 2 ? kt : vt, j));
        }
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int i = i0 + k * kPagedThreads, j = i < total / 2 ? i : i - total / 2;
            const int g = j / vd, e = (j - g * vd) * 8;
            if (i < total)
                *(uint4*)((uint16_t*)(i < total / 2 ? c.k : c.v) + dst + g * c.head_stride + e) = x[k];
        }
    }
}

}  // namespace

cudaError_t launch_commit_paged(const CommitPagedArgs& a, cudaStream_t s) {
    return launch_pdl(commit_paged_kernel, dim3(a.L + 1, a.B), dim3(kPagedThreads), 0, s, a.cache,
                      a.k_tree, a.v_tree, a.accept_len, a.accepted_nodes, a.prefix_len, a.new_len,
                      a.L, a.N, a.err);
}

cudaError_t launch_commit(const CommitArgs& a, cudaStream_t s) {
    return launch_pdl(commit_kernel, dim3(a.B), dim3(kThreads), 0, s, (uint4*)a.k_cache,
                      (uint4*)a.v_cache, a.cache_cap, (const uint4*)a.k_tree,
                      (const uint4*)a.v_tree, a.accept_len, a.accepted_nodes, a.prefix_len, a.L,
                      a.N, a.Hkv, a.D, a.err);
}

}  // namespace ddt
