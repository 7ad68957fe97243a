// norm_rope.cu -- ddtree_norm_rope: the norm of every head of queries and keys and the
// rotation behind it in one pass.
//
//   y = x / sqrt(mean x^2 + eps) * w,  then pairs of y turned as in rotary.cu
//
// A warp takes a row: its sum of squares by shuffles, then its pairs, whose cosine and
// sine it computes itself.
#include "rotary.cuh"

namespace ddt {

namespace {

constexpr int kThreads = 128;

struct Params {
    RowsArg q, q_out, k, k_out;
    const int32_t* pos;
    const uint64_t* turns;
    NormArgs norm;
    float scale;
    int T, D, rot;
    bool interleaved;
};

template <typename T>
__global__ void __launch_bounds__(kThreads) norm_rope_kernel(const __grid_constant__ Params p) {
    const int lane = threadIdx.x & 31, heads = p.q.heads + p.k.heads;
    pdl_wait();
    const int64_t row = (int64_t)blockIdx.x * (kThreads / 32) + threadIdx.x / 32;
    const int64_t t = row / heads;
    const int h = (int)(row - t * heads);
    if (t >= p.T) return;
    const bool is_q = h < p.q.heads;
    const RowsArg &in = is_q ? p.q : p.k, &out = is_q ? p.q_out : p.k_out;
    const int hh = is_q ? h : h - p.q.heads;
    const T* x = (const T*)in.data + t * in.ts + hh * in.hs;
    T* y = (T*)out.data + t * out.ts + hh * out.hs;
    const int pos = p.pos[t];
    if (pos < 0) {
        if (x != y)
            for (int i = lane; i < p.D; i += 32) y[i] = x[i];
        return;
    }
    const float* w = is_q ? p.norm.q_weight : p.norm.k_weight;
    float sum = 0.f;
    for (int i = lane; i < p.D; i += 32) sum = fmaf(to_f(x[i]), to_f(x[i]), sum);
    for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    const float r = rsqrtf(sum / p.D + p.norm.eps);
    auto normed = [&](int i) { return to_f(x[i]) * r * (w ? w[i] : 1.f); };
    for (int j = lane; j < p.rot / 2; j += 32) {
        const int a = p.interleaved ? 2 * j : j, b = p.interleaved ? 2 * j + 1 : j + p.rot / 2;
        const float2 cs = cos_sin((uint64_t)(uint32_t)pos * p.turns[j]);
        const float2 z = turned(normed(a), normed(b), cs.x * p.scale, cs.y * p.scale);
        y[a] = from_f<T>(z.x);
        y[b] = from_f<T>(z.y);
    }
    for (int i = p.rot + lane; i < p.D; i += 32) y[i] = from_f<T>(normed(i));
}

template <typename T>
cudaError_t launch(const Params& p, cudaStream_t s) {
    const int64_t rows = (int64_t)p.T * (p.q.heads + p.k.heads), per = kThreads / 32;
    if ((rows + per - 1) / per > INT32_MAX) return cudaErrorInvalidValue;
    return launch_pdl(norm_rope_kernel<T>, dim3((unsigned)((rows + per - 1) / per)), dim3(kThreads), 0, s, p);
}

}  // namespace

cudaError_t launch_norm_rope(const NormRopeArgs& a, cudaStream_t s) {
    Params p{a.q, a.q_out, a.k, a.k_out, a.pos, a.turns, a.norm, a.scale, a.T, a.D, a.rot, a.interleaved};
    if (a.dtype == 0) return launch<__nv_bfloat16>(p, s);
    if (a.dtype == 1) return launch<float>(p, s);
    return launch<__half>(p, s);
}

}  // namespace ddt
