// api.cu -- the C ABI (include/ddtree.h): host-side validation, the per-device
// error word, and dispatch to the kernel launchers.  No allocation, no
// synchronisation except in ddtree_device_check().
#include <algorithm>
#include <cmath>
#include <initializer_list>
#include <mutex>
#include <new>

#include "common.cuh"
#include "internal.h"
#include "sm100.cuh"

#include "../../include/ddtree.h"

namespace {

constexpr int kMaxDevices = 64;
uint32_t* g_err_ptr[kMaxDevices];
std::mutex g_err_mu;

}  // namespace

// One error word per device; kernels record the first inconsistency they meet.
static __device__ uint32_t g_ddtree_error_word;

namespace ddt {

// Device address of this device's error word (looked up once per device).
uint32_t* error_word() {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return nullptr;
    std::lock_guard<std::mutex> g(g_err_mu);
    if (!g_err_ptr[dev]) {
        void* p = nullptr;
        if (cudaGetSymbolAddress(&p, g_ddtree_error_word) != cudaSuccess) return nullptr;
        g_err_ptr[dev] = (uint32_t*)p;
    }
    return g_err_ptr[dev];
}

}  // namespace ddt

namespace {

using ddt::error_word;

inline bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }
// Every pointer of 4-byte elements (int32, uint32, float) on its grid; null
// entries (optional outputs) pass.
inline bool aligned4(std::initializer_list<const void*> ps) {
    for (const void* p : ps)
        if (p && !aligned(p, 4)) return false;
    return true;
}

thread_local const char* t_last_cuda_error = "no error";

ddtree_status launched(cudaError_t e) {
    if (e == cudaSuccess) return DDTREE_OK;
    t_last_cuda_error = cudaGetErrorName(e);
    return DDTREE_ERR_CUDA;
}

}  // namespace

namespace ddt {
int launch_status(cudaError_t e) { return (int)launched(e); }
// For the handler around a C entry, out of which no C++ exception goes: the host's
// memory has run out, or a lock failed.
ddtree_status caught() {
    try {
        throw;
    } catch (const std::bad_alloc&) {
        return launched(cudaErrorMemoryAllocation);
    } catch (...) {
        return launched(cudaErrorUnknown);
    }
}
}  // namespace ddt

extern "C" {

const char* ddtree_last_cuda_error(void) { return t_last_cuda_error; }

const char* ddtree_status_str(ddtree_status s) {
    switch (s) {
        case DDTREE_OK: return "ok";
        case DDTREE_ERR_INVALID_ARG: return "invalid argument";
        case DDTREE_ERR_UNSUPPORTED: return "unsupported shape";
        case DDTREE_ERR_CUDA: return "CUDA error";
        case DDTREE_ERR_DEVICE: return "kernel recorded bad device data or a timeout";
    }
    return "unknown status";
}

size_t ddtree_workspace_size(ddtree_op op, int B, int L, int N, int V, int K, int dtype, int Hq,
                             int Hkv, int D, int64_t cache_cap) try {
    switch (op) {
        case DDTREE_OP_TOPK:
            if (B <= 0 || V <= 0 || (dtype != DDTREE_BF16 && dtype != DDTREE_FP32)) return 0;
            return ddt::topk_workspace_bytes(B * (L > 0 ? L : 1), V, dtype, K);
        case DDTREE_OP_TREE_ATTN:
            if (B <= 0 || N < 0 || Hq <= 0 || Hkv <= 0 || D <= 0 || cache_cap < 0) return 0;
            return ddt::attn_workspace_bytes(B, N, Hq, Hkv, D, cache_cap);
        case DDTREE_OP_ACCEPT:
            if (B <= 0 || N < 0 || V <= 0 || (dtype != DDTREE_BF16 && dtype != DDTREE_FP32))
                return 0;
            return ddt::accept_workspace_bytes(B, N, V, dtype);
        case DDTREE_OP_TREE_ATTN_PAGED:
            if (B <= 0 || N < 0 || Hkv <= 0 || Hq < Hkv || Hq % Hkv || Hq / Hkv > 128 || D <= 0 ||
                cache_cap < 0 || cache_cap > (1 << 30))
                return 0;
            return ddt::paged_attn_workspace_bytes(B, N, Hq, Hkv, D, cache_cap);
        case DDTREE_OP_TREE_ATTN_Q8:
            if (B <= 0 || N < 0 || Hkv <= 0 || Hq < Hkv || Hq % Hkv || Hq / Hkv > 128 || D <= 0 ||
                cache_cap < 0 || cache_cap > (1 << 30))
                return 0;
            return ddt::q8_attn_workspace_bytes(B, N, Hq, Hkv, D, cache_cap);
    }
    return 0;
} catch (...) {
    return 0;
}

ddtree_status ddtree_topk(const void* draft_logits, int dtype, int rows, int V,
                          int64_t row_stride, int K, int32_t* topk_idx, float* topk_logp,
                          float* lse, void* workspace, size_t ws_bytes, void* stream) try {
    if (!draft_logits || !topk_idx || !topk_logp) return DDTREE_ERR_INVALID_ARG;
    if (dtype != DDTREE_BF16 && dtype != DDTREE_FP32) return DDTREE_ERR_INVALID_ARG;
    if (rows <= 0 || rows > 65535 || V <= 0 || row_stride < V || K < 1 || K > V)
        return DDTREE_ERR_INVALID_ARG;
    if (K > DDTREE_MAX_K || !ddt::topk_supported(V, dtype, K)) return DDTREE_ERR_UNSUPPORTED;
    if (!aligned(draft_logits, dtype == DDTREE_BF16 ? 2 : 4)) return DDTREE_ERR_INVALID_ARG;
    if (!aligned4({topk_idx, topk_logp, lse})) return DDTREE_ERR_INVALID_ARG;
    const size_t need = ddt::topk_workspace_bytes(rows, V, dtype, K);
    if (need && (!workspace || ws_bytes < need || !aligned(workspace, 256)))
        return DDTREE_ERR_INVALID_ARG;
    ddt::TopkArgs a{draft_logits, dtype, rows, V, row_stride, K, topk_idx, topk_logp, lse,
                    workspace, error_word()};
    return launched(ddt::launch_topk(a, (cudaStream_t)stream));
} catch (...) {
    return ddt::caught();
}

namespace {
ddtree_status build_common(bool heap, const float* topk_logp, const int32_t* topk_idx,
                           const int32_t* bonus, const int32_t* prefix_len, int B, int L, int K,
                           int N, int32_t* parent, int32_t* depth, int32_t* rank, int32_t* token,
                           int32_t* pos_id, float* score, int32_t* child_count,
                           uint32_t* anc_mask, int32_t* n_nodes, void* stream) {
    if (!topk_logp || !topk_idx || !bonus || !prefix_len || !parent || !depth || !rank ||
        !token || !pos_id || !score || !child_count || !anc_mask || !n_nodes)
        return DDTREE_ERR_INVALID_ARG;
    if (B <= 0 || B > 65535 || L <= 0 || K <= 0 || N < 0) return DDTREE_ERR_INVALID_ARG;
    if (!aligned4({topk_logp, topk_idx, bonus, prefix_len, parent, depth, rank, token, pos_id,
                   score, child_count, anc_mask, n_nodes}))
        return DDTREE_ERR_INVALID_ARG;
    if (L > DDTREE_MAX_L || K > DDTREE_MAX_K || N > DDTREE_MAX_N) return DDTREE_ERR_UNSUPPORTED;
    ddt::BuildArgs a{topk_logp, topk_idx, bonus, prefix_len, B, L, K, N, parent, depth, rank,
                     token, pos_id, score, child_count, anc_mask, n_nodes, error_word()};
    return launched(heap ? ddt::launch_build(a, (cudaStream_t)stream)
                         : ddt::launch_build_level(a, (cudaStream_t)stream));
}
}  // namespace

ddtree_status ddtree_build(const float* topk_logp, const int32_t* topk_idx, const int32_t* bonus,
                           const int32_t* prefix_len, int B, int L, int K, int N,
                           int32_t* parent, int32_t* depth, int32_t* rank, int32_t* token,
                           int32_t* pos_id, float* score, int32_t* child_count,
                           uint32_t* anc_mask, int32_t* n_nodes, void* stream) try {
    return build_common(false, topk_logp, topk_idx, bonus, prefix_len, B, L, K, N, parent, depth,
                        rank, token, pos_id, score, child_count, anc_mask, n_nodes, stream);
} catch (...) {
    return ddt::caught();
}

ddtree_status ddtree_build_heap(const float* topk_logp, const int32_t* topk_idx,
                                const int32_t* bonus, const int32_t* prefix_len, int B, int L,
                                int K, int N, int32_t* parent, int32_t* depth, int32_t* rank,
                                int32_t* token, int32_t* pos_id, float* score,
                                int32_t* child_count, uint32_t* anc_mask, int32_t* n_nodes,
                                void* stream) try {
    return build_common(true, topk_logp, topk_idx, bonus, prefix_len, B, L, K, N, parent, depth,
                        rank, token, pos_id, score, child_count, anc_mask, n_nodes, stream);
} catch (...) {
    return ddt::caught();
}

ddtree_status ddtree_tree_attn(const void* q, const void* k_cache, const void* v_cache,
                               int64_t cache_cap, const void* k_tree, const void* v_tree,
                               const int32_t* prefix_len, const int32_t* n_nodes,
                               const uint32_t* anc_mask, int B, int N, int Hq, int Hkv, int D,
                               float scale, void* out, float* lse, void* workspace,
                               size_t ws_bytes, void* stream) try {
    if (!q || !k_cache || !v_cache || !k_tree || !v_tree || !prefix_len || !n_nodes ||
        !anc_mask || !out)
        return DDTREE_ERR_INVALID_ARG;
    if (B <= 0 || N < 0 || Hq <= 0 || Hkv <= 0 || Hq % Hkv || cache_cap < 0 || !(scale > 0.f))
        return DDTREE_ERR_INVALID_ARG;
    const int G = Hq / Hkv;
    if (N > DDTREE_MAX_N || (D != 64 && D != 128) || (G & (G - 1)) || G > 128)
        return DDTREE_ERR_UNSUPPORTED;
    for (const void* p : {q, k_cache, v_cache, k_tree, v_tree, (const void*)out})
        if (!aligned(p, 16)) return DDTREE_ERR_INVALID_ARG;
    if (!aligned4({prefix_len, n_nodes, anc_mask, lse})) return DDTREE_ERR_INVALID_ARG;
    const size_t need = ddt::attn_workspace_bytes(B, N, Hq, Hkv, D, cache_cap);
    if (need && (!workspace || ws_bytes < need || !aligned(workspace, 256)))
        return DDTREE_ERR_INVALID_ARG;
    ddt::AttnArgs a{q, k_cache, v_cache, cache_cap, k_tree, v_tree, prefix_len, n_nodes, anc_mask,
                    B, N, Hq, Hkv, D, scale, out, lse, workspace, error_word()};
    return launched(ddt::launch_tree_attn(a, (cudaStream_t)stream));
} catch (...) {
    return ddt::caught();
}

ddtree_status ddtree_accept(const void* target_logits, int dtype, int64_t row_stride,
                            const int32_t* parent, const int32_t* token, const int32_t* n_nodes,
                            int B, int L, int N, int V, float temperature, uint64_t seed,
                            uint64_t step, int32_t* target_token, int32_t* accept_len,
                            int32_t* accepted_nodes, int32_t* out_tokens, int32_t* next_bonus,
                            void* workspace, size_t ws_bytes, void* stream) try {
    if (!target_logits || !parent || !token || !n_nodes || !accept_len || !accepted_nodes ||
        !out_tokens || !next_bonus)
        return DDTREE_ERR_INVALID_ARG;
    if (dtype != DDTREE_BF16 && dtype != DDTREE_FP32) return DDTREE_ERR_INVALID_ARG;
    if (B <= 0 || B > 65535 || L <= 0 || N < 0 || V <= 0 || row_stride < V ||
        !(temperature >= 0.f) || temperature > 1e30f)
        return DDTREE_ERR_INVALID_ARG;
    if (N > DDTREE_MAX_N || L > DDTREE_MAX_L || !ddt::accept_supported(V, dtype))
        return DDTREE_ERR_UNSUPPORTED;
    if (!aligned(target_logits, dtype == DDTREE_BF16 ? 2 : 4)) return DDTREE_ERR_INVALID_ARG;
    if (!aligned4({parent, token, n_nodes, target_token, accept_len, accepted_nodes, out_tokens,
                   next_bonus}))
        return DDTREE_ERR_INVALID_ARG;
    const size_t need = ddt::accept_workspace_bytes(B, N, V, dtype);
    if (!workspace || ws_bytes < need || !aligned(workspace, 256)) return DDTREE_ERR_INVALID_ARG;
    ddt::AcceptArgs a{target_logits, dtype, row_stride, parent, token, n_nodes, B, L, N, V,
                      temperature, seed, step, target_token, accept_len, accepted_nodes,
                      out_tokens, next_bonus, workspace, error_word()};
    return launched(ddt::launch_accept(a, (cudaStream_t)stream));
} catch (...) {
    return ddt::caught();
}

ddtree_status ddtree_accept_path(const void* target_logits, int dtype, int64_t row_stride,
                                 const int32_t* parent, const int32_t* token,
                                 const int32_t* n_nodes, int B, int L, int N, int V,
                                 float temperature, uint64_t seed, uint64_t step,
                                 int32_t* target_token, int32_t* accept_len,
                                 int32_t* accepted_nodes, int32_t* out_tokens,
                                 int32_t* next_bonus, void* stream) try {
    if (!target_logits || !parent || !token || !n_nodes || !accept_len || !accepted_nodes ||
        !out_tokens || !next_bonus)
        return DDTREE_ERR_INVALID_ARG;
    if (dtype != DDTREE_BF16 && dtype != DDTREE_FP32) return DDTREE_ERR_INVALID_ARG;
    if (B <= 0 || B > 65535 || L <= 0 || N < 0 || V <= 0 || row_stride < V ||
        !(temperature >= 0.f) || temperature > 1e30f)
        return DDTREE_ERR_INVALID_ARG;
    if (N > DDTREE_MAX_N || L > DDTREE_MAX_L || !ddt::accept_path_supported(V, dtype))
        return DDTREE_ERR_UNSUPPORTED;
    if (!aligned(target_logits, dtype == DDTREE_BF16 ? 2 : 4)) return DDTREE_ERR_INVALID_ARG;
    if (!aligned4({parent, token, n_nodes, target_token, accept_len, accepted_nodes, out_tokens,
                   next_bonus}))
        return DDTREE_ERR_INVALID_ARG;
    ddt::AcceptArgs a{target_logits, dtype, row_stride, parent, token, n_nodes, B, L, N, V,
                      temperature, seed, step, target_token, accept_len, accepted_nodes,
                      out_tokens, next_bonus, nullptr, error_word()};
    return launched(ddt::launch_accept_path(a, (cudaStream_t)stream));
} catch (...) {
    return ddt::caught();
}

ddtree_status ddtree_commit(void* k_cache, void* v_cache, int64_t cache_cap, const void* k_tree,
                            const void* v_tree, const int32_t* accept_len,
                            const int32_t* accepted_nodes, int32_t* prefix_len, int B, int L,
                            int N, int Hkv, int D, void* stream) try {
    if (!k_cache || !v_cache || !k_tree || !v_tree || !accept_len || !accepted_nodes ||
        !prefix_len)
        return DDTREE_ERR_INVALID_ARG;
    if (B <= 0 || B > 65535 || L <= 0 || N < 0 || Hkv <= 0 || D <= 0 || cache_cap <= 0)
        return DDTREE_ERR_INVALID_ARG;
    if (L > DDTREE_MAX_L || N > DDTREE_MAX_N || D % 8 != 0) return DDTREE_ERR_UNSUPPORTED;
    if (!aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(k_tree, 16) ||
        !aligned(v_tree, 16) || !aligned(accept_len, 4) || !aligned(accepted_nodes, 4) ||
        !aligned(prefix_len, 4))
        return DDTREE_ERR_INVALID_ARG;
    ddt::CommitArgs a{k_cache, v_cache, cache_cap, k_tree, v_tree, accept_len, accepted_nodes,
                      prefix_len, B, L, N, Hkv, D, error_word()};
    return launched(ddt::launch_commit(a, (cudaStream_t)stream));
} catch (...) {
    return ddt::caught();
}

// ---- the round over a paged cache ----------------------------------------------

namespace {

int esize(int dtype) { return dtype == DDTREE_FP32 ? 4 : 2; }
bool dtype16(int dtype) { return dtype == DDTREE_BF16 || dtype == DDTREE_FP16; }

// A ddtree_rows that can be read (out: written) as rows of D elements: not null,
// on the element grid, strides sane.
bool rows_ok(const ddtree_rows* r, int dtype, int D, bool out) {
    if (!r || !r->data || r->heads <= 0 || !aligned(r->data, esize(dtype))) return false;
    const int64_t least = out ? D : 0;
    return r->token_stride >= least && (r->heads == 1 || r->head_stride >= least);
}
// ... and also by 16-byte accesses.
bool rows16(const ddtree_rows* r) {
    return aligned(r->data, 16) && r->token_stride % 8 == 0 && r->head_stride % 8 == 0;
}
// q_out: as many heads as q; the same tensor only with the same strides.
bool pair_ok(const ddtree_rows* in, const ddtree_rows* out, int dtype, int D) {
    if (!rows_ok(in, dtype, D, false) || !rows_ok(out, dtype, D, true)) return false;
    if (in->heads != out->heads) return false;
    return in->data != out->data || (in->token_stride == out->token_stride &&
                                     (in->heads == 1 || in->head_stride == out->head_stride));
}
// Neither output is the other, nor the other's input.
bool apart(const ddtree_rows* q, const ddtree_rows* q_out, const ddtree_rows* k,
           const ddtree_rows* k_out) {
    return q_out->data != k->data && (!k_out || (k_out->data != q->data && k_out->data != q_out->data));
}
ddt::RowsArg rows_arg(const ddtree_rows* r) {
    return r ? ddt::RowsArg{r->data, r->heads, r->token_stride, r->head_stride} : ddt::RowsArg{};
}

ddtree_status cache_status(const ddtree_paged_cache* c) {
    if (!c || !c->k_pages || !c->v_pages || !c->page_table) return DDTREE_ERR_INVALID_ARG;
    if (!dtype16(c->dtype) || c->num_pages <= 0 || c->page_size <= 0 || c->Hkv <= 0 || c->D <= 0 ||
        c->max_pages <= 0 || c->table_stride < c->max_pages ||
        (int64_t)c->max_pages * c->page_size > (1 << 30))
        return DDTREE_ERR_INVALID_ARG;
    if ((c->num_pages > 1 && c->page_stride < c->D) || (c->Hkv > 1 && c->head_stride < c->D) ||
        (c->page_size > 1 && c->slot_stride < c->D))
        return DDTREE_ERR_INVALID_ARG;
    if (c->page_stride < 0 || c->head_stride < 0 || c->slot_stride < 0)
        return DDTREE_ERR_INVALID_ARG;
    if (!aligned(c->k_pages, 2) || !aligned(c->v_pages, 2) || !aligned(c->page_table, 4))
        return DDTREE_ERR_INVALID_ARG;
    return DDTREE_OK;
}
bool cache16(const ddtree_paged_cache* c) {
    return aligned(c->k_pages, 16) && aligned(c->v_pages, 16) && c->page_stride % 8 == 0 &&
           c->head_stride % 8 == 0 && c->slot_stride % 8 == 0;
}
ddt::PagedArgs cache_arg(const ddtree_paged_cache* c) {
    return {c->k_pages, c->v_pages, c->dtype, c->num_pages, c->page_size, c->Hkv, c->D,
            c->page_stride, c->head_stride, c->slot_stride, c->page_table, c->max_pages,
            c->table_stride};
}

bool rotary_ok(const ddtree_rotary* r, int D) {
    return r && r->turns && aligned(r->turns, 8) && r->rot_dim >= 2 && r->rot_dim % 2 == 0 &&
           r->rot_dim <= D && std::isfinite(r->scale);
}

}  // namespace

ddtree_status ddtree_rope_frequencies(int rot_dim, double base, int scaling, double factor,
                                      double orig_len, double low, double high,
                                      double* inv_freq, float* scale) {
    if (!inv_freq || !scale || rot_dim < 2 || rot_dim % 2) return DDTREE_ERR_INVALID_ARG;
    if (rot_dim > DDTREE_MAX_ROPE_D) return DDTREE_ERR_UNSUPPORTED;
    if (scaling < DDTREE_ROPE_NONE || scaling > DDTREE_ROPE_YARN || !(base > 0) ||
        !std::isfinite(base) || (scaling != DDTREE_ROPE_NONE && !(factor > 0 && std::isfinite(factor))))
        return DDTREE_ERR_INVALID_ARG;
    if (scaling >= DDTREE_ROPE_BANDED &&
        !(orig_len > 0 && std::isfinite(orig_len) && low > 0 && high > low && std::isfinite(high)))
        return DDTREE_ERR_INVALID_ARG;
    if (scaling == DDTREE_ROPE_YARN && !(base > 1)) return DDTREE_ERR_INVALID_ARG;
    if (scaling == DDTREE_ROPE_NTK) {
        if (rot_dim < 4) return DDTREE_ERR_INVALID_ARG;
        base *= std::pow(factor, (double)rot_dim / (rot_dim - 2));
    }
    constexpr double kTwoPi = 6.283185307179586476925;
    double lo = 0, hi = 0;
    if (scaling == DDTREE_ROPE_YARN) {
        auto dim = [&](double t) {
            return rot_dim * std::log(orig_len / (kTwoPi * t)) / (2 * std::log(base));
        };
        lo = std::max(std::floor(dim(high)), 0.0);
        hi = std::min(std::ceil(dim(low)), (double)rot_dim - 1);
    }
    *scale = scaling == DDTREE_ROPE_YARN && factor > 1 ? (float)(0.1 * std::log(factor) + 1) : 1.f;
    for (int j = 0; j < rot_dim / 2; ++j) {
        const double f = std::pow(base, -2.0 * j / rot_dim);
        double s = 1;  // share of the unscaled frequency
        if (scaling == DDTREE_ROPE_LINEAR) s = 0;
        if (scaling == DDTREE_ROPE_BANDED) s = (orig_len * f / kTwoPi - low) / (high - low);
        if (scaling == DDTREE_ROPE_YARN) s = 1 - (j - lo) / std::max(hi - lo, 1e-3);
        s = std::min(std::max(s, 0.0), 1.0);
        inv_freq[j] = s == 1 ? f : (1 - s) * (f / factor) + s * f;
    }
    return DDTREE_OK;
}

ddtree_status ddtree_rope_turns(const double* inv_freq, int n, uint64_t* turns) {
    if (!inv_freq || !turns || n < 1) return DDTREE_ERR_INVALID_ARG;
    for (int j = 0; j < n; ++j)
        if (!std::isfinite(inv_freq[j])) return DDTREE_ERR_INVALID_ARG;
    for (int j = 0; j < n; ++j) {
        const double t = inv_freq[j] / 6.283185307179586476925;
        const double frac = t - std::floor(t);  // [0, 1], 1 only for a tiny negative t
        turns[j] = frac < 1 ? (uint64_t)std::ldexp(frac, 64) : 0;
    }
    return DDTREE_OK;
}

ddtree_status ddtree_rope(const ddtree_rows* q, const ddtree_rows* q_out, const ddtree_rows* k,
                          const ddtree_rows* k_out, int dtype, int T, int D, const int32_t* pos,
                          const ddtree_rotary* rot, int inverse, void* stream) try {
    if ((dtype != DDTREE_FP32 && !dtype16(dtype)) || T < 0 || D < 1 ||
        (inverse != 0 && inverse != 1))
        return DDTREE_ERR_INVALID_ARG;
    if (D > DDTREE_MAX_ROPE_D) return DDTREE_ERR_UNSUPPORTED;
    if (T == 0) return DDTREE_OK;
    if (!pos || !aligned(pos, 4) || !pair_ok(q, q_out, dtype, D) || (k || k_out ? !pair_ok(k, k_out, dtype, D) : false) ||
        !rotary_ok(rot, D) || (k && !apart(q, q_out, k, k_out)))
        return DDTREE_ERR_INVALID_ARG;
    if ((int64_t)q->heads + (k ? k->heads : 0) > 65535) return DDTREE_ERR_UNSUPPORTED;
    ddt::RopeArgs a{rows_arg(q), rows_arg(q_out), rows_arg(k), rows_arg(k_out), dtype, T, D, pos,
                    rot->turns, rot->rot_dim, rot->interleaved != 0, rot->scale, inverse};
    return launched(ddt::launch_rope(a, (cudaStream_t)stream));
} catch (...) {
    return ddt::caught();
}

ddtree_status ddtree_append_paged(const ddtree_rows* k, const ddtree_rows* v, int T,
                                  const int32_t* seq, const int32_t* pos, int B,
                                  const ddtree_paged_cache* cache, const ddtree_rotary* rot,
                                  const ddtree_rows* q, const ddtree_rows* q_out, void* stream) try {
    if (ddtree_status st = cache_status(cache)) return st;
    const int dt = cache->dtype, D = cache->D;
    if (T < 0 || B <= 0) return DDTREE_ERR_INVALID_ARG;
    if (D > DDTREE_MAX_ROPE_D) return DDTREE_ERR_UNSUPPORTED;
    if (T == 0) return DDTREE_OK;
    if (!seq || !pos || !aligned4({seq, pos})) return DDTREE_ERR_INVALID_ARG;
    if (!rows_ok(k, dt, D, false) || !rows_ok(v, dt, D, false) || k->heads != cache->Hkv ||
        v->heads != cache->Hkv || (q || q_out ? !pair_ok(q, q_out, dt, D) : false) ||
        (rot && !rotary_ok(rot, D)) || k->data == cache->k_pages || v->data == cache->v_pages ||
        (q && !(apart(q, q_out, k, nullptr) && apart(q, q_out, v, nullptr))))
        return DDTREE_ERR_INVALID_ARG;
    if (2 * (int64_t)cache->Hkv + (q ? q->heads : 0) > 65535) return DDTREE_ERR_UNSUPPORTED;
    ddt::AppendArgs a{rows_arg(q), rows_arg(q_out), rows_arg(k), rows_arg(v), T, B, seq, pos,
                      cache_arg(cache), rot ? rot->turns : nullptr, rot ? rot->rot_dim : 0,
                      rot && rot->interleaved, rot ? rot->scale : 1.f, error_word()};
    return launched(ddt::launch_append_paged(a, (cudaStream_t)stream));
} catch (...) {
    return ddt::caught();
}

ddtree_status ddtree_tree_attn_paged(const ddtree_rows* q, const ddtree_paged_cache* cache,
                                     const ddtree_rows* k_tree, const ddtree_rows* v_tree,
                                     const int32_t* prefix_len, const int32_t* n_nodes,
                                     const uint32_t* anc_mask, int B, int N, float scale,
                                     void* out, float* lse, void* workspace, size_t ws_bytes,
                                     void* stream) try {
    if (ddtree_status st = cache_status(cache)) return st;
    const int dt = cache->dtype, D = cache->D, Hkv = cache->Hkv, ps = cache->page_size;
    if (!prefix_len || !n_nodes || !anc_mask || !out || B <= 0 || N < 0 || !(scale > 0.f) ||
        !std::isfinite(scale))
        return DDTREE_ERR_INVALID_ARG;
    if (!rows_ok(q, dt, D, true) || !rows_ok(k_tree, dt, D, true) ||
        !rows_ok(v_tree, dt, D, true) || k_tree->heads != Hkv || v_tree->heads != Hkv ||
        q->heads % Hkv || out == q->data || out == k_tree->data || out == v_tree->data)
        return DDTREE_ERR_INVALID_ARG;
    if (N > DDTREE_MAX_N || (D != 64 && D != 128) || q->heads / Hkv > 128 || ps < 8 ||
        (ps & (ps - 1)) || (int64_t)B * (N + 1) > INT32_MAX)
        return DDTREE_ERR_UNSUPPORTED;
    if (!rows16(q) || !rows16(k_tree) || !rows16(v_tree) || !cache16(cache) || !aligned(out, 16) ||
        !aligned4({prefix_len, n_nodes, anc_mask, lse}))
        return DDTREE_ERR_INVALID_ARG;
    const size_t need = ddt::paged_attn_workspace_bytes(B, N, q->heads, Hkv, D,
                                                        (int64_t)cache->max_pages * ps);
    if (need && (!workspace || ws_bytes < need || !aligned(workspace, 256)))
        return DDTREE_ERR_INVALID_ARG;
    ddt::PagedAttnArgs a{rows_arg(q), rows_arg(k_tree), rows_arg(v_tree), cache_arg(cache),
                         prefix_len, n_nodes, anc_mask, B, N, scale, out, lse, workspace,
                         error_word()};
    return launched(ddt::launch_tree_attn_paged(a, (cudaStream_t)stream));
} catch (...) {
    return ddt::caught();
}

ddtree_status ddtree_commit_paged(const ddtree_paged_cache* cache, const ddtree_rows* k_tree,
                                  const ddtree_rows* v_tree, const int32_t* accept_len,
                                  const int32_t* accepted_nodes, const int32_t* prefix_len,
                                  int32_t* new_len, int B, int L, int N, void* stream) try {
    if (ddtree_status st = cache_status(cache)) return st;
    const int dt = cache->dtype, D = cache->D;
    if (!accept_len || !accepted_nodes || !prefix_len || B <= 0 || B > 65535 || L <= 0 || N < 0)
        return DDTREE_ERR_INVALID_ARG;
    if (!rows_ok(k_tree, dt, D, false) || !rows_ok(v_tree, dt, D, false) ||
        k_tree->heads != cache->Hkv || v_tree->heads != cache->Hkv ||
        !aligned4({accept_len, accepted_nodes, prefix_len, new_len}) ||
        (new_len && (new_len == prefix_len || new_len == accept_len || new_len == accepted_nodes)))
        return DDTREE_ERR_INVALID_ARG;
    if (L > DDTREE_MAX_L || N > DDTREE_MAX_N || D % 8 != 0) return DDTREE_ERR_UNSUPPORTED;
    if (!rows16(k_tree) || !rows16(v_tree) || !cache16(cache)) return DDTREE_ERR_INVALID_ARG;
    ddt::CommitPagedArgs a{cache_arg(cache), rows_arg(k_tree), rows_arg(v_tree), accept_len,
                           accepted_nodes, prefix_len, new_len, B, L, N, error_word()};
    return launched(ddt::launch_commit_paged(a, (cudaStream_t)stream));
} catch (...) {
    return ddt::caught();
}

// ---- the round over an 8-bit paged cache ----------------------------------------

namespace {

// Whether a norm can be used; NULL is none.
bool norm_ok(const ddtree_head_norm* n) {
    return !n || (n->eps > 0.f && std::isfinite(n->eps) && aligned4({n->q_weight, n->k_weight}));
}
ddt::NormArgs norm_arg(const ddtree_head_norm* n) {
    return n ? ddt::NormArgs{n->q_weight, n->k_weight, n->eps, true} : ddt::NormArgs{};
}

ddtree_status q8_status(const ddtree_q8_cache* c) {
    if (!c || !c->k_pages || !c->v_pages || !c->k_scales || !c->v_scales || !c->page_table ||
        c->k_pages == c->v_pages || c->k_scales == c->v_scales)
        return DDTREE_ERR_INVALID_ARG;
    if (!dtype16(c->dtype) || c->num_pages <= 0 || c->page_size <= 0 || c->block <= 0 || c->Hkv <= 0 ||
        c->D <= 0 || c->max_pages <= 0 || c->table_stride < c->max_pages ||
        (int64_t)c->max_pages * c->page_size > (1 << 30))
        return DDTREE_ERR_INVALID_ARG;
    for (const int64_t st : {c->page_stride, c->head_stride, c->slot_stride})
        if (st < 0 || st % 16) return DDTREE_ERR_INVALID_ARG;
    if ((c->num_pages > 1 && c->page_stride < c->D) || (c->Hkv > 1 && c->head_stride < c->D) ||
        (c->page_size > 1 && c->slot_stride < c->D))
        return DDTREE_ERR_INVALID_ARG;
    for (const void* p : {(const void*)c->k_pages, (const void*)c->v_pages, (const void*)c->k_scales,
                          (const void*)c->v_scales})
        if (!aligned(p, 16)) return DDTREE_ERR_INVALID_ARG;
    if (!aligned(c->page_table, 4)) return DDTREE_ERR_INVALID_ARG;
    if ((c->D != 64 && c->D != 128) || c->page_size < 8 || (c->page_size & (c->page_size - 1)) ||
        c->block < 8 || (c->block & (c->block - 1)) || c->block > c->page_size ||
        c->block > DDTREE_MAX_Q8_BLOCK)
        return DDTREE_ERR_UNSUPPORTED;
    return DDTREE_OK;
}
ddt::Q8Args q8_arg(const ddtree_q8_cache* c) {
    return {(uint8_t*)c->k_pages, (uint8_t*)c->v_pages, c->k_scales, c->v_scales, c->dtype,
            c->num_pages, c->page_size, c->block, c->Hkv, c->D, c->page_stride, c->head_stride,
            c->slot_stride, c->page_table, c->max_pages, c->table_stride};
}
// Rows of a call over an 8-bit cache: 16-byte accesses, one row a KV head.
bool q8_rows_ok(const ddtree_rows* r, const ddtree_q8_cache* c, bool out) {
    return rows_ok(r, c->dtype, c->D, out) && rows16(r) && r->heads == c->Hkv;
}

}  // namespace

ddtree_status ddtree_norm_rope(const ddtree_rows* q, const ddtree_rows* q_out,
                               const ddtree_rows* k, const ddtree_rows* k_out, int dtype, int T,
                               int D, const int32_t* pos, const ddtree_head_norm* norm,
                               const ddtree_rotary* rot, void* stream) try {
    if ((dtype != DDTREE_FP32 && !dtype16(dtype)) || T < 0 || D < 1) return DDTREE_ERR_INVALID_ARG;
    if (D > DDTREE_MAX_ROPE_D) return DDTREE_ERR_UNSUPPORTED;
    if (T == 0) return DDTREE_OK;
    if (!pos || !aligned(pos, 4) || !norm || !norm_ok(norm) || !pair_ok(q, q_out, dtype, D) ||
        (k || k_out ? !pair_ok(k, k_out, dtype, D) : false) || (rot && !rotary_ok(rot, D)) ||
        (k && !apart(q, q_out, k, k_out)))
        return DDTREE_ERR_INVALID_ARG;
    if ((int64_t)q->heads + (k ? k->heads : 0) > 65535) return DDTREE_ERR_UNSUPPORTED;
    ddt::NormRopeArgs a{rows_arg(q), rows_arg(q_out), rows_arg(k), rows_arg(k_out), dtype, T, D, pos,
                        rot ? rot->turns : nullptr, rot ? rot->rot_dim : 0, rot && rot->interleaved,
                        rot ? rot->scale : 1.f, norm_arg(norm)};
    return launched(ddt::launch_norm_rope(a, (cudaStream_t)stream));
} catch (...) {
    return ddt::caught();
}

ddtree_status ddtree_append_q8(const ddtree_rows* k, const ddtree_rows* v, int T,
                               const int32_t* first, const int32_t* at, int B,
                               const ddtree_q8_cache* cache, const ddtree_rotary* rot,
                               const ddtree_head_norm* norm, const ddtree_rows* q,
                               const ddtree_rows* q_out, void* stream) try {
    if (ddtree_status st = q8_status(cache)) return st;
    const int dt = cache->dtype, D = cache->D;
    if (T < 0 || B <= 0) return DDTREE_ERR_INVALID_ARG;
    if (T == 0) return DDTREE_OK;
    if (!first || !at || !aligned4({first, at}) || !q8_rows_ok(k, cache, false) ||
        !q8_rows_ok(v, cache, false) || !norm_ok(norm) || (rot && !rotary_ok(rot, D)) ||
        (q || q_out ? !(pair_ok(q, q_out, dt, D) && rows16(q) && rows16(q_out)) : false) ||
        (q && !(apart(q, q_out, k, nullptr) && apart(q, q_out, v, nullptr))))
        return DDTREE_ERR_INVALID_ARG;
    if ((rot && rot->rot_dim % 16) || 2 * (int64_t)cache->Hkv + (q ? q->heads : 0) > 65535)
        return DDTREE_ERR_UNSUPPORTED;
    ddt::AppendQ8Args a{rows_arg(q), rows_arg(q_out), rows_arg(k), rows_arg(v), T, B, first, at,
                        q8_arg(cache), rot ? rot->turns : nullptr, rot ? rot->rot_dim : 0,
                        rot && rot->interleaved, rot ? rot->scale : 1.f, norm_arg(norm), error_word()};
    return launched(ddt::launch_append_q8(a, (cudaStream_t)stream));
} catch (...) {
    return ddt::caught();
}

ddtree_status ddtree_commit_q8(const ddtree_q8_cache* cache, const ddtree_rows* k_tree,
                               const ddtree_rows* v_tree, const int32_t* accept_len,
                               const int32_t* accepted_nodes, const int32_t* prefix_len,
                               int32_t* new_len, int B, int L, int N, void* stream) try {
    if (ddtree_status st = q8_status(cache)) return st;
    if (!accept_len || !accepted_nodes || !prefix_len || B <= 0 || B > 65535 || L <= 0 || N < 0)
        return DDTREE_ERR_INVALID_ARG;
    if (!q8_rows_ok(k_tree, cache, false) || !q8_rows_ok(v_tree, cache, false) ||
        !aligned4({accept_len, accepted_nodes, prefix_len, new_len}) ||
        (new_len && (new_len == prefix_len || new_len == accept_len || new_len == accepted_nodes)))
        return DDTREE_ERR_INVALID_ARG;
    if (L > DDTREE_MAX_L || N > DDTREE_MAX_N || cache->Hkv > 65535) return DDTREE_ERR_UNSUPPORTED;
    ddt::CommitQ8Args a{q8_arg(cache), rows_arg(k_tree), rows_arg(v_tree), accept_len,
                        accepted_nodes, prefix_len, new_len, B, L, N, error_word()};
    return launched(ddt::launch_commit_q8(a, (cudaStream_t)stream));
} catch (...) {
    return ddt::caught();
}

ddtree_status ddtree_read_q8(const ddtree_q8_cache* cache, const int32_t* first,
                             const int32_t* at, int B, const ddtree_rows* k_out,
                             const ddtree_rows* v_out, int T, void* stream) try {
    if (ddtree_status st = q8_status(cache)) return st;
    if (T < 0 || B <= 0) return DDTREE_ERR_INVALID_ARG;
    if (T == 0) return DDTREE_OK;
    if (!first || !at || !aligned4({first, at}) || !q8_rows_ok(k_out, cache, true) ||
        !q8_rows_ok(v_out, cache, true) || k_out->data == v_out->data)
        return DDTREE_ERR_INVALID_ARG;
    if (cache->Hkv > 65535) return DDTREE_ERR_UNSUPPORTED;
    ddt::ReadQ8Args a{q8_arg(cache), first, at, rows_arg(k_out), rows_arg(v_out), B, T, error_word()};
    return launched(ddt::launch_read_q8(a, (cudaStream_t)stream));
} catch (...) {
    return ddt::caught();
}

ddtree_status ddtree_tree_attn_q8(const ddtree_rows* q, const ddtree_q8_cache* cache,
                                  const ddtree_rows* k_tree, const ddtree_rows* v_tree,
                                  const int32_t* prefix_len, const int32_t* n_nodes,
                                  const uint32_t* anc_mask, int B, int N, float scale, void* out,
                                  float* lse, void* workspace, size_t ws_bytes, void* stream) try {
    if (ddtree_status st = q8_status(cache)) return st;
    const int dt = cache->dtype, D = cache->D, Hkv = cache->Hkv;
    if (!prefix_len || !n_nodes || !anc_mask || !out || B <= 0 || N < 0 || !(scale > 0.f) ||
        !std::isfinite(scale))
        return DDTREE_ERR_INVALID_ARG;
    if (!rows_ok(q, dt, D, true) || !rows16(q) || !q8_rows_ok(k_tree, cache, true) ||
        !q8_rows_ok(v_tree, cache, true) || q->heads % Hkv || out == q->data ||
        out == k_tree->data || out == v_tree->data || !aligned(out, 16) ||
        !aligned4({prefix_len, n_nodes, anc_mask, lse}))
        return DDTREE_ERR_INVALID_ARG;
    if (N > DDTREE_MAX_N || q->heads / Hkv > 128 || (int64_t)B * (N + 1) > INT32_MAX)
        return DDTREE_ERR_UNSUPPORTED;
    const size_t need = ddt::q8_attn_workspace_bytes(B, N, q->heads, Hkv, D,
                                                     (int64_t)cache->max_pages * cache->page_size);
    if (need && (!workspace || ws_bytes < need || !aligned(workspace, 256)))
        return DDTREE_ERR_INVALID_ARG;
    ddt::Q8AttnArgs a{rows_arg(q), rows_arg(k_tree), rows_arg(v_tree), q8_arg(cache),
                      prefix_len, n_nodes, anc_mask, B, N, scale, out, lse, workspace,
                      error_word()};
    return launched(ddt::launch_tree_attn_q8(a, (cudaStream_t)stream));
} catch (...) {
    return ddt::caught();
}

namespace {

// Two warps wait, through the bounded wait every kernel of the library uses, on
// an mbarrier that nothing arrives on.  When the first one's bound passes it sets
// the abort flag, which ends the second one's wait, and both leave as whole warps,
// as a kernel whose copy never landed does; the timeout is recorded in the error
// word.
__global__ void selftest_wait_kernel(uint64_t limit_ns, uint32_t* err) {
    __shared__ __align__(8) uint64_t bar;
    __shared__ volatile int s_abort;
    if (threadIdx.x == 0) {
        ddt::sm100::mbar_init(&bar, 1);
        ddt::sm100::mbar_init_fence();
        s_abort = 0;
    }
    __syncthreads();
    const bool first = threadIdx.x < 32;
    const bool ok = first ? ddt::sm100::mbar_wait_warp(&bar, 0, &s_abort, limit_ns)
                          : ddt::sm100::mbar_wait_warp(&bar, 0, &s_abort);
    if (first && !ok) s_abort = 1;
    const int gave_up = __syncthreads_count(!ok);
    if (threadIdx.x == 0 && gave_up == (int)blockDim.x)
        ddt::record_error(err, ddt::ERR_SELFTEST | ddt::ERR_WAIT_TIMEOUT);
}

}  // namespace

ddtree_status ddtree_selftest_wait(uint32_t limit_us, void* stream) try {
    if (limit_us < 1 || limit_us > 1000000) return DDTREE_ERR_INVALID_ARG;
    uint32_t* err = error_word();
    if (!err) return DDTREE_ERR_CUDA;
    selftest_wait_kernel<<<1, 64, 0, (cudaStream_t)stream>>>((uint64_t)limit_us * 1000ull, err);
    return launched(cudaGetLastError());
} catch (...) {
    return ddt::caught();
}

ddtree_status ddtree_device_check(void* stream, uint32_t* detail) try {
    uint32_t* p = error_word();
    if (!p) return DDTREE_ERR_CUDA;
    cudaStream_t s = (cudaStream_t)stream;
    uint32_t v = 0, zero = 0;
    if (cudaMemcpyAsync(&v, p, sizeof v, cudaMemcpyDeviceToHost, s) != cudaSuccess)
        return DDTREE_ERR_CUDA;
    if (cudaMemcpyAsync(p, &zero, sizeof zero, cudaMemcpyHostToDevice, s) != cudaSuccess)
        return DDTREE_ERR_CUDA;
    if (cudaStreamSynchronize(s) != cudaSuccess) return DDTREE_ERR_CUDA;
    if (detail) *detail = v;
    return v ? DDTREE_ERR_DEVICE : DDTREE_OK;
} catch (...) {
    return ddt::caught();
}

}  // extern "C"
