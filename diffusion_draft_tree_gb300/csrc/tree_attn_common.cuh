// tree_attn_common.cuh -- what the tree-attention kernels share: rounding to the
// 16-bit types, tensor maps, the device's size.
#pragma once

#include <algorithm>
#include <mutex>

#include <cudaTypedefs.h>

#include "internal.h"
#include "sm100.cuh"

namespace ddt {

namespace {

// A pair of weights or outputs rounded to the kernel's 16-bit type.
template <bool F16>
DDT_DEV uint32_t pack16(float lo, float hi) {
    if constexpr (F16) {
        uint32_t r;
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
        return r;
    } else {
        return pack_bf16x2(lo, hi);
    }
}

// Softmax weights are rounded to the 16-bit type for the product with V: the tensor
// core takes both factors in one type, and 32-bit weights as two such halves would
// double that product.  In bf16 that is up to 2^-8 of a weight: outputs are 0.0023 of
// their size off, where rounding the output alone makes 0.0017 (fp16 0.00022, 0.00020).
// fp16 has no numbers below 2^-24, and a weight below that is dropped where the sum counts it; so
// its weights are taken 2^kLift larger.  The largest is then 2^(8 + 7) -- a maximum may
// be 2^8 behind -- and a weight keeps half a step down to 2^-21 of the row's largest
// one and is dropped at 2^-32.  Sums and outputs carry the factor alike; only the
// logsumexp takes it off.
template <bool F16>
constexpr float kLift = F16 ? 7.f : 0.f;

// mma.sync and its operands from shared memory, for few query rows.
DDT_DEV void ldsm_x4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
DDT_DEV void ldsm_x4_t(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
template <bool F16>
DDT_DEV void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (F16)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
            "{%8, %9}, {%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
            "{%8, %9}, {%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Transposes an 8 x 8 matrix of 16-bit elements that a warp holds by twos.
DDT_DEV uint32_t movmatrix_t(uint32_t x) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}
// 16-byte chunk c of row r of a 128-byte-swizzled slab.
DDT_DEV uint32_t swz(int r, int c) { return (uint32_t)(r * 128 + ((c ^ (r & 7)) << 4)); }

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault,
                                             &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = (PFN_cuTensorMapEncodeTiled_v12000)f;
    });
    return fn;
}

struct MapDim {
    uint64_t size, stride_bytes;  // (the innermost stride is the element's)
    uint32_t box;
};
// A 128-byte-swizzled map of 16-bit elements, rank 3 or 4.
template <int RANK>
bool make_map(CUtensorMap* m, const void* ptr, const MapDim (&d)[RANK], bool f16 = false) {
    auto fn = encode_fn();
    if (!fn) return false;
    cuuint64_t dims[RANK], strides[RANK - 1];
    cuuint32_t box[RANK], estr[RANK];
    for (int i = 0; i < RANK; ++i) {
        dims[i] = d[i].size ? d[i].size : 1;
        if (i) strides[i - 1] = d[i].stride_bytes;
        box[i] = d[i].box;
        estr[i] = 1;
    }
    return fn(m, f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, RANK,
              const_cast<void*>(ptr), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The stride of a dimension of one entry is never used; its map needs a legal one.
inline uint64_t stride_bytes(int64_t elements, uint64_t size, uint64_t rowb) {
    return size > 1 ? (uint64_t)elements * 2 : rowb;
}

// Tree queries, keys or values: boxes of 64 columns, `heads` heads, `nodes` nodes.
template <int D>
bool tree_map(CUtensorMap* m, const RowsArg& r, uint64_t tokens, uint32_t heads, uint32_t nodes,
              bool f16) {
    const uint64_t rowb = (uint64_t)D * 2;
    const MapDim d[3] = {{(uint64_t)D, 0, 64},
                         {(uint64_t)r.heads, stride_bytes(r.hs, r.heads, rowb), heads},
                         {tokens, stride_bytes(r.ts, tokens, rowb), nodes}};
    return make_map(m, r.data, d, f16);
}

// Pages: boxes of 64 columns and at most `rows` slots of one head of one page.
template <int D>
bool page_map(CUtensorMap* m, const PagedArgs& c, const void* pages, int rows, bool f16) {
    const uint64_t rowb = (uint64_t)D * 2;
    const MapDim d[4] = {{(uint64_t)D, 0, 64},
                         {(uint64_t)c.page_size, stride_bytes(c.slot_stride, c.page_size, rowb),
                          (uint32_t)std::min(c.page_size, rows)},
                         {(uint64_t)c.Hkv, stride_bytes(c.head_stride, c.Hkv, rowb), 1},
                         {(uint64_t)c.num_pages, stride_bytes(c.page_stride, c.num_pages, rowb), 1}};
    return make_map(m, pages, d, f16);
}

// Pages of an 8-bit cache: boxes of a head's whole rows, swizzled over the row's length or not
// at all.
template <int D>
bool code_map(CUtensorMap* m, const Q8Args& c, const void* pages, int rows, bool swizzled = false) {
    auto fn = encode_fn();
    if (!fn) return false;
    auto stride = [](int64_t bytes, int size) { return size > 1 ? (cuuint64_t)bytes : (cuuint64_t)D; };
    const cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)c.page_size, (cuuint64_t)c.Hkv, (cuuint64_t)c.num_pages};
    const cuuint64_t strides[3] = {stride(c.slot_stride, c.page_size), stride(c.head_stride, c.Hkv),
                                   stride(c.page_stride, c.num_pages)};
    const cuuint32_t box[4] = {(cuuint32_t)D, (cuuint32_t)std::min(c.page_size, rows), 1, 1}, estr[4] = {1, 1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<void*>(pages), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE,
              !swizzled ? CU_TENSOR_MAP_SWIZZLE_NONE : D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

// The kernel for few query rows (tree_attn_rows.cu): whether it takes a shape,
// its workspace, its launch.
bool few_rows(int B, int N, int Hq, int Hkv, int64_t cache_cap);
size_t few_rows_workspace_bytes(int N, int Hq, int Hkv, int D);
cudaError_t launch_tree_attn_rows(const PagedAttnArgs& a, cudaStream_t s);
// ... over an 8-bit cache (tree_attn_q8_rows.cu), in a workspace of the same size.
bool q8_few_rows(int B, int N, int Hq, int Hkv, int64_t cache_cap);
cudaError_t launch_tree_attn_q8_rows(const Q8AttnArgs& a, cudaStream_t s);

}  // namespace ddt
