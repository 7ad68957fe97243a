// binding.cpp -- the paged-cache calls' argument marshalling for ops.py.
//
// These calls run once a layer and more, most of them a few microseconds on the
// GPU, and describe up to four strided tensors each.  Reading a tensor's shape,
// strides, type and address through Python attributes cost 8 us a call (11 for
// attention), three times the launch; here it is a few field reads.  Every check
// of an argument is made on this side; what the library checks itself
// (include/ddtree.h) is left to it.  Each function returns the library's
// status; a tensor that does not fit raises ValueError.
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <ATen/core/grad_mode.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <cmath>
#include <cstring>
#include <stdexcept>
#include <string>

#include "../../include/ddtree.h"

namespace {

using at::Tensor;

[[noreturn]] void bad(const std::string& what) { throw std::invalid_argument(what); }

std::string list(c10::IntArrayRef v) {
    std::string s = "[";
    for (size_t i = 0; i < v.size(); ++i) s += (i ? ", " : "") + std::to_string(v[i]);
    return s + "]";
}
std::string about(const Tensor& t) {
    return std::string(c10::toString(t.scalar_type())) + " " + list(t.sizes()) + " on " +
           t.device().str();
}

const Tensor& tensor(PyObject* o, const char* name) {
    if (!THPVariable_Check(o)) bad(std::string(name) + " must be a tensor");
    return THPVariable_Unpack(o);
}

int code(at::ScalarType t) {
    switch (t) {
        case at::kBFloat16: return DDTREE_BF16;
        case at::kHalf: return DDTREE_FP16;
        case at::kFloat: return DDTREE_FP32;
        default: return -1;
    }
}

// What every tensor of a call has in common.
struct Common {
    int index;
    int64_t D;
    at::ScalarType dtype;
};

// ddtree_rows of a [tokens][heads][D] or [B][nodes][heads][D] tensor, and its
// number of tokens.
struct Rows {
    ddtree_rows r;
    int64_t tokens;
};
Rows rows(const Tensor& t, const char* name, const Common& c) {
    const auto n = t.sizes(), st = t.strides();
    if (!t.is_cuda() || t.get_device() != c.index || t.scalar_type() != c.dtype)
        bad(std::string(name) + " must be a " + c10::toString(c.dtype) + " tensor on cuda:" +
            std::to_string(c.index) + ", got " + about(t));
    if (n.size() != 3 && n.size() != 4)
        bad(std::string(name) + " must be [tokens][heads][D] or [B][nodes][heads][D]");
    const size_t h = n.size() - 2;  // the heads' dimension
    int64_t tokens = n[h - 1], ts = st[h - 1];
    if (h == 2) {
        if (n[1] == 1)
            ts = st[0];
        else if (n[0] > 1 && st[0] != n[1] * st[1])
            bad(std::string(name) + ": the strides of its first two dimensions do not merge");
        tokens = n[0] * n[1];
    }
    if (n[h + 1] != c.D || (st[h + 1] != 1 && c.D > 1))
        bad(std::string(name) + " must end in " + std::to_string(c.D) + " contiguous elements");
    if (tokens > INT32_MAX || n[h] > INT32_MAX) bad(std::string(name) + " is too large");
    // (the stride of a dimension of one entry says nothing)
    const int64_t hs = n[h] == 1 ? c.D : st[h];
    if (tokens == 1) ts = std::max(n[h] * hs, c.D);
    return {{t.data_ptr(), (int32_t)n[h], ts, hs}, tokens};
}
Rows rows(PyObject* o, const char* name, const Common& c) { return rows(tensor(o, name), name, c); }

// Device pointer of a contiguous tensor of the given type and shape.
void* dense(PyObject* o, const char* name, at::ScalarType dtype, c10::IntArrayRef shape, int index) {
    const Tensor& t = tensor(o, name);
    if (t.scalar_type() != dtype || t.sizes() != shape || !t.is_cuda() || t.get_device() != index ||
        !t.is_contiguous())
        bad(std::string(name) + " must be a contiguous " + c10::toString(dtype) + " tensor " +
            list(shape) + " on cuda:" + std::to_string(index) + ", got " + about(t));
    return t.data_ptr();
}
int32_t* ints(PyObject* o, const char* name, c10::IntArrayRef shape, int index) {
    return (int32_t*)dense(o, name, at::kInt, shape, index);
}
// ... of `tokens` entries: [tokens], or the leading dimensions of `like`.
int32_t* token_ints(PyObject* o, const char* name, const Tensor& like, int64_t tokens, int index) {
    const Tensor& t = tensor(o, name);
    if (t.dim() == 1) return ints(o, name, {tokens}, index);
    return ints(o, name, like.sizes().slice(0, like.dim() - 2), index);
}

// The tensors that a call writes, behind autograd's back.  One that it differentiates
// is refused, as torch refuses it for its own in-place and out= calls; the others'
// versions go up, so that a backward pass that saved one of them notices.
struct Written {
    const Tensor* t[5] = {};
    int n = 0;
    void add(const Tensor& x, const char* name) {
        if (x.requires_grad() && at::GradMode::is_enabled())
            bad(std::string(name) + " requires grad and would be written without a graph: call under "
                                    "torch.no_grad(), or on a detached tensor");
        t[n++] = &x;
    }
    int done(int status) const {
        for (int i = 0; i < n && status == DDTREE_OK; ++i)
            if (!t[i]->is_inference()) t[i]->unsafeGetTensorImpl()->bump_version();
        return status;
    }
};

template <typename T>
T packed(PyObject* o, const char* name) {
    T v;
    if (!PyBytes_Check(o) || PyBytes_GET_SIZE(o) != (Py_ssize_t)sizeof(T))
        bad(std::string(name) + " is not one of ops' handles");
    std::memcpy(&v, PyBytes_AS_STRING(o), sizeof(T));
    return v;
}

// `index` made the current device while the call is enqueued on `stream` (None:
// that device's current stream).
struct Launch {
    c10::cuda::CUDAGuard guard;
    void* stream;
    Launch(int index, PyObject* o) : guard((c10::DeviceIndex)index) {
        if (o == Py_None) {
            stream = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)index).stream();
        } else {
            stream = PyLong_AsVoidPtr(o);
            if (!stream && PyErr_Occurred()) bad("stream must be a torch.cuda.Stream");
        }
    }
};

// A rotation, or none.
struct Turn {
    ddtree_rotary r;
    bool on;
    const ddtree_rotary* p() const { return on ? &r : nullptr; }
};
Turn turn_of(PyObject* o, PyObject* index, const Common& c, const char* other) {
    Turn t{};
    if (o == Py_None) return t;
    if (PyLong_AsLong(index) != c.index) bad(std::string("rotary is on another device than ") + other);
    t.r = packed<ddtree_rotary>(o, "rotary");
    t.on = true;
    return t;
}
// A norm of heads of D elements from (packed struct, device index, D), or none.
struct Norm {
    ddtree_head_norm n;
    bool on;
    const ddtree_head_norm* p() const { return on ? &n : nullptr; }
};
Norm norm_of(PyObject* const* a, const Common& c, const char* other) {
    Norm x{};
    if (a[0] == Py_None) return x;
    const long index = PyLong_AsLong(a[1]), D = PyLong_AsLong(a[2]);
    if (index >= 0 && index != c.index) bad(std::string("norm is on another device than ") + other);
    if (D >= 0 && D != c.D)
        bad("norm has weights of " + std::to_string(D) + " elements, a head " + std::to_string(c.D));
    x.n = packed<ddtree_head_norm>(a[0], "norm");
    x.on = true;
    return x;
}

// Queries and, unless k is None, keys of a call that turns them: rows in and out.
struct Pair {
    Rows q, qo, k, ko;
    bool with_k;
};
Pair pair_of(PyObject* oq, PyObject* ok, PyObject* oqo, PyObject* oko, const Common& c, Written& w) {
    Pair x{};
    const Tensor& q = tensor(oq, "q");
    x.qo = x.q = rows(q, "q", c);
    if (oqo != Py_None) {
        x.qo = rows(oqo, "q_out", c);
        if (tensor(oqo, "q_out").sizes() != q.sizes()) bad("q_out must have q's shape");
    }
    x.with_k = ok != Py_None;
    if (x.with_k) {
        const Tensor& k = tensor(ok, "k");
        x.ko = x.k = rows(k, "k", c);
        if (x.k.tokens != x.q.tokens)
            bad("k has " + std::to_string(x.k.tokens) + " tokens, q " + std::to_string(x.q.tokens));
        if (oko != Py_None) {
            x.ko = rows(oko, "k_out", c);
            if (tensor(oko, "k_out").sizes() != k.sizes()) bad("k_out must have k's shape");
        }
    } else if (oko != Py_None) {
        bad("k_out without k");
    }
    w.add(oqo == Py_None ? q : tensor(oqo, "q_out"), oqo == Py_None ? "q" : "q_out");
    if (x.with_k) w.add(tensor(oko == Py_None ? ok : oko, "k"), oko == Py_None ? "k" : "k_out");
    return x;
}

// norm_rope(q, k, pos, norm x 3, rotary, rotary_index, q_out, k_out, stream)
int norm_rope(PyObject* const* a) {
    const Tensor& q = tensor(a[0], "q");
    if (!q.is_cuda() || q.dim() < 1 || code(q.scalar_type()) < 0)
        bad("q must be a bfloat16, float16 or float32 CUDA tensor, got " + about(q));
    const Common c{(int)q.get_device(), q.size(-1), q.scalar_type()};
    const Norm norm = norm_of(a + 3, c, "q");
    if (!norm.on) bad("norm must be an ops.HeadNorm");
    const Turn turn = turn_of(a[6], a[7], c, "q");
    Written w;
    const Pair x = pair_of(a[0], a[1], a[8], a[9], c, w);
    const int32_t* pos = token_ints(a[2], "pos", q, x.q.tokens, c.index);
    const Launch l(c.index, a[10]);
    return w.done(ddtree_norm_rope(&x.q.r, &x.qo.r, x.with_k ? &x.k.r : nullptr,
                                   x.with_k ? &x.ko.r : nullptr, code(c.dtype), (int)x.q.tokens,
                                   (int)std::min<int64_t>(c.D, INT32_MAX), pos, norm.p(), turn.p(),
                                   l.stream));
}

// rope(q, k, pos, rotary, rotary_index, q_out, k_out, inverse, stream)
int rope(PyObject* const* a) {
    const Tensor& q = tensor(a[0], "q");
    if (!q.is_cuda() || q.dim() < 1 || code(q.scalar_type()) < 0)
        bad("q must be a bfloat16, float16 or float32 CUDA tensor, got " + about(q));
    const Common c{(int)q.get_device(), q.size(-1), q.scalar_type()};
    if (PyLong_AsLong(a[4]) != c.index) bad("rotary is on another device than q");
    const ddtree_rotary rot = packed<ddtree_rotary>(a[3], "rotary");
    Written w;
    const Pair x = pair_of(a[0], a[1], a[5], a[6], c, w);
    const int32_t* pos = token_ints(a[2], "pos", q, x.q.tokens, c.index);
    const Launch l(c.index, a[8]);
    return w.done(ddtree_rope(&x.q.r, &x.qo.r, x.with_k ? &x.k.r : nullptr, x.with_k ? &x.ko.r : nullptr,
                              code(c.dtype), (int)x.q.tokens, (int)std::min<int64_t>(c.D, INT32_MAX), pos, &rot,
                              PyObject_IsTrue(a[7]), l.stream));
}

// The cache of a call and its pages' device and type.
struct Cache {
    ddtree_paged_cache s;
    Common c;
    int64_t B;
};
// ... from (packed struct, device index, sequences).
Cache cache(PyObject* const* a) {
    Cache x{packed<ddtree_paged_cache>(a[0], "cache"), {}, PyLong_AsLong(a[2])};
    x.c = {(int)PyLong_AsLong(a[1]), x.s.D, x.s.dtype == DDTREE_FP16 ? at::kHalf : at::kBFloat16};
    return x;
}

// append(cache x 3, k, v, seq, pos, rotary, rotary_index, q, q_out, stream, k_pages, v_pages)
int append(PyObject* const* a) {
    const Cache x = cache(a);
    a += 3;
    const Tensor& k = tensor(a[0], "k");
    const Rows kr = rows(k, "k", x.c), vr = rows(a[1], "v", x.c);
    if (vr.tokens != kr.tokens)
        bad("v has " + std::to_string(vr.tokens) + " tokens, k " + std::to_string(kr.tokens));
    const bool turn = a[4] != Py_None, with_q = a[6] != Py_None;
    ddtree_rotary rot{};
    if (turn) {
        if (PyLong_AsLong(a[5]) != x.c.index) bad("rotary is on another device than the cache");
        rot = packed<ddtree_rotary>(a[4], "rotary");
    }
    Rows qr{}, qo{};
    if (with_q) {
        const Tensor& q = tensor(a[6], "q");
        qo = qr = rows(q, "q", x.c);
        if (qr.tokens != kr.tokens)
            bad("q has " + std::to_string(qr.tokens) + " tokens, k " + std::to_string(kr.tokens));
        if (a[7] != Py_None) {
            qo = rows(a[7], "q_out", x.c);
            if (tensor(a[7], "q_out").sizes() != q.sizes()) bad("q_out must have q's shape");
        }
    } else if (a[7] != Py_None) {
        bad("q_out without q");
    }
    const int32_t* seq = token_ints(a[2], "seq", k, kr.tokens, x.c.index);
    const int32_t* pos = token_ints(a[3], "pos", k, kr.tokens, x.c.index);
    Written w;
    w.add(tensor(a[9], "k_pages"), "k_pages");
    w.add(tensor(a[10], "v_pages"), "v_pages");
    if (with_q) w.add(tensor(a[7] == Py_None ? a[6] : a[7], "q"), a[7] == Py_None ? "q" : "q_out");
    const Launch l(x.c.index, a[8]);
    return w.done(ddtree_append_paged(&kr.r, &vr.r, (int)kr.tokens, seq, pos, (int)x.B, &x.s,
                                      turn ? &rot : nullptr, with_q ? &qr.r : nullptr,
                                      with_q ? &qo.r : nullptr, l.stream));
}

// The tree attention of one cache or the other: its status for the arguments.
using AttnOf = int (*)(const void* cache, const ddtree_rows* q, const ddtree_rows* k, const ddtree_rows* v,
                       const int32_t* P, const int32_t* n, const uint32_t* mask, int B, int N, float scale,
                       void* out, float* lse, void* ws, size_t bytes, void* stream);
// (cache), then (q, k_tree, v_tree, prefix_len, n_nodes, anc_mask, out, lse, scale, workspace,
// stream)
template <typename C>
int attn_of(const C& x, PyObject* const* a, AttnOf call) {
    const int dev = x.c.index;
    const Tensor &q = tensor(a[0], "q"), &kt = tensor(a[1], "k_tree"), &vt = tensor(a[2], "v_tree");
    if (q.dim() != 4 || kt.dim() != 4 || vt.dim() != 4)
        bad("q, k_tree and v_tree must be [B][nodes][heads][D]");
    const int64_t B = q.size(0), R = q.size(1), Hq = q.size(2);
    if (kt.size(0) != B || vt.size(0) != B || kt.size(1) != R || vt.size(1) != R || x.B != B)
        bad("q, k_tree, v_tree and the page table must agree in B and nodes");
    const Rows qr = rows(q, "q", x.c), kr = rows(kt, "k_tree", x.c), vr = rows(vt, "v_tree", x.c);
    void* out = dense(a[6], "out", x.c.dtype, q.sizes(), dev);
    float* lse = a[7] == Py_None ? nullptr : (float*)dense(a[7], "lse", at::kFloat, {B, R, Hq}, dev);
    void* ws = nullptr;
    size_t bytes = 0;
    if (a[9] != Py_None) {
        const Tensor& w = tensor(a[9], "workspace");
        bytes = (size_t)w.numel();
        ws = dense(a[9], "workspace", at::kByte, w.sizes(), dev);
    }
    const int32_t *P = ints(a[3], "prefix_len", {B}, dev), *n = ints(a[4], "n_nodes", {B}, dev);
    const auto* mask = (const uint32_t*)ints(a[5], "anc_mask", {B, R, (R + 31) / 32}, dev);
    const double scale = a[8] == Py_None ? 1.0 / std::sqrt((double)x.c.D) : PyFloat_AsDouble(a[8]);
    if (PyErr_Occurred()) bad("scale must be a number");
    Written w;
    w.add(tensor(a[6], "out"), "out");
    if (lse) w.add(tensor(a[7], "lse"), "lse");
    const Launch l(dev, a[10]);
    return w.done(call(&x.s, &qr.r, &kr.r, &vr.r, P, n, mask, (int)B, (int)(R - 1), (float)scale, out, lse,
                       ws, bytes, l.stream));
}
// attn(cache x 3, and as attn_of)
int attn(PyObject* const* a) {
    return attn_of(cache(a), a + 3, [](const void* cache, const ddtree_rows* q, const ddtree_rows* k,
                                       const ddtree_rows* v, const int32_t* P, const int32_t* n,
                                       const uint32_t* mask, int B, int N, float scale, void* out, float* lse,
                                       void* ws, size_t bytes, void* stream) -> int {
        return ddtree_tree_attn_paged(q, (const ddtree_paged_cache*)cache, k, v, P, n, mask, B, N, scale, out,
                                      lse, ws, bytes, stream);
    });
}

// The commit into one cache or the other.
using CommitOf = int (*)(const void* cache, const ddtree_rows* k, const ddtree_rows* v, const int32_t* alen,
                         const int32_t* nodes, const int32_t* P, int32_t* to, int B, int L, int N, void* stream);
// (cache), then (k_tree, v_tree, accept_len, accepted_nodes, prefix_len, new_len, stream);
// `w` has the cache's own tensors
template <typename C>
int commit_of(const C& x, PyObject* const* a, Written w, CommitOf call) {
    const int dev = x.c.index;
    const Tensor &kt = tensor(a[0], "k_tree"), &vt = tensor(a[1], "v_tree");
    const Tensor& nodes = tensor(a[3], "accepted_nodes");
    if (kt.dim() != 4 || kt.size(0) != x.B || vt.sizes() != kt.sizes())
        bad("k_tree and v_tree must be [B][nodes][Hkv][D], B as the page table's");
    if (nodes.dim() != 2) bad("accepted_nodes must be [B][L]");
    const Rows kr = rows(kt, "k_tree", x.c), vr = rows(vt, "v_tree", x.c);
    const int64_t L = nodes.size(1);
    const int32_t* alen = ints(a[2], "accept_len", {x.B}, dev);
    const int32_t* acc = ints(a[3], "accepted_nodes", {x.B, L}, dev);
    const int32_t* P = ints(a[4], "prefix_len", {x.B}, dev);
    int32_t* to = a[5] == Py_None ? nullptr : ints(a[5], "new_len", {x.B}, dev);
    if (to) w.add(tensor(a[5], "new_len"), "new_len");
    const Launch l(dev, a[6]);
    return w.done(call(&x.s, &kr.r, &vr.r, alen, acc, P, to, (int)x.B, (int)std::min<int64_t>(L, INT32_MAX),
                       (int)(kt.size(1) - 1), l.stream));
}
// commit(cache x 3, as commit_of, k_pages, v_pages)
int commit(PyObject* const* a) {
    Written w;
    w.add(tensor(a[10], "k_pages"), "k_pages");
    w.add(tensor(a[11], "v_pages"), "v_pages");
    return commit_of(cache(a), a + 3, w, [](const void* cache, const ddtree_rows* k, const ddtree_rows* v,
                                            const int32_t* alen, const int32_t* nodes, const int32_t* P,
                                            int32_t* to, int B, int L, int N, void* stream) -> int {
        return ddtree_commit_paged((const ddtree_paged_cache*)cache, k, v, alen, nodes, P, to, B, L, N, stream);
    });
}

// An 8-bit cache of a call, its pages' device and its tokens' type, from (packed struct,
// device index, sequences).
struct Q8Cache {
    ddtree_q8_cache s;
    Common c;
    int64_t B;
};
Q8Cache q8_cache(PyObject* const* a) {
    Q8Cache x{packed<ddtree_q8_cache>(a[0], "cache"), {}, PyLong_AsLong(a[2])};
    x.c = {(int)PyLong_AsLong(a[1]), x.s.D, x.s.dtype == DDTREE_FP16 ? at::kHalf : at::kBFloat16};
    return x;
}
// The codes and scales of a cache that a call writes: four tensors.
void add_pages(Written& w, PyObject* const* a) {
    static const char* const names[4] = {"k_pages", "v_pages", "k_scales", "v_scales"};
    for (int i = 0; i < 4; ++i) w.add(tensor(a[i], names[i]), names[i]);
}

// tree_attn_q8(cache x 3, and as attn_of)
int attn_q8(PyObject* const* a) {
    return attn_of(q8_cache(a), a + 3, [](const void* cache, const ddtree_rows* q, const ddtree_rows* k,
                                          const ddtree_rows* v, const int32_t* P, const int32_t* n,
                                          const uint32_t* mask, int B, int N, float scale, void* out, float* lse,
                                          void* ws, size_t bytes, void* stream) -> int {
        return ddtree_tree_attn_q8(q, (const ddtree_q8_cache*)cache, k, v, P, n, mask, B, N, scale, out, lse, ws,
                                   bytes, stream);
    });
}

// commit_q8(cache x 3, as commit_of, k_pages, v_pages, k_scales, v_scales)
int commit_q8(PyObject* const* a) {
    Written w;
    add_pages(w, a + 10);
    return commit_of(q8_cache(a), a + 3, w, [](const void* cache, const ddtree_rows* k, const ddtree_rows* v,
                                               const int32_t* alen, const int32_t* nodes, const int32_t* P,
                                               int32_t* to, int B, int L, int N, void* stream) -> int {
        return ddtree_commit_q8((const ddtree_q8_cache*)cache, k, v, alen, nodes, P, to, B, L, N, stream);
    });
}

// append_q8(cache x 3, k, v, first, at, rotary, rotary_index, norm x 3, q, q_out, stream,
//           k_pages, v_pages, k_scales, v_scales)
int append_q8(PyObject* const* a) {
    const Q8Cache x = q8_cache(a);
    a += 3;
    const Rows kr = rows(a[0], "k", x.c), vr = rows(a[1], "v", x.c);
    if (vr.tokens != kr.tokens)
        bad("v has " + std::to_string(vr.tokens) + " tokens, k " + std::to_string(kr.tokens));
    const int32_t *first = ints(a[2], "first", {x.B + 1}, x.c.index), *at = ints(a[3], "at", {x.B}, x.c.index);
    const Turn turn = turn_of(a[4], a[5], x.c, "the cache");
    const Norm norm = norm_of(a + 6, x.c, "the cache");
    const bool with_q = a[9] != Py_None;
    Written w;
    Pair y{};
    if (with_q) {
        y = pair_of(a[9], Py_None, a[10], Py_None, x.c, w);
        if (y.q.tokens != kr.tokens)
            bad("q has " + std::to_string(y.q.tokens) + " tokens, k " + std::to_string(kr.tokens));
    } else if (a[10] != Py_None) {
        bad("q_out without q");
    }
    add_pages(w, a + 12);
    const Launch l(x.c.index, a[11]);
    return w.done(ddtree_append_q8(&kr.r, &vr.r, (int)kr.tokens, first, at, (int)x.B, &x.s, turn.p(),
                                   norm.p(), with_q ? &y.q.r : nullptr, with_q ? &y.qo.r : nullptr,
                                   l.stream));
}

// read_q8(cache x 3, first, at, k_out, v_out, stream)
int read_q8(PyObject* const* a) {
    const Q8Cache x = q8_cache(a);
    a += 3;
    const int32_t *first = ints(a[0], "first", {x.B + 1}, x.c.index), *at = ints(a[1], "at", {x.B}, x.c.index);
    const Rows kr = rows(a[2], "k_out", x.c), vr = rows(a[3], "v_out", x.c);
    if (vr.tokens != kr.tokens)
        bad("v_out has " + std::to_string(vr.tokens) + " tokens, k_out " + std::to_string(kr.tokens));
    Written w;
    w.add(tensor(a[2], "k_out"), "k_out");
    w.add(tensor(a[3], "v_out"), "v_out");
    const Launch l(x.c.index, a[4]);
    return w.done(ddtree_read_q8(&x.s, first, at, (int)x.B, &kr.r, &vr.r, (int)kr.tokens, l.stream));
}

// The Python entry of one of these, `N` arguments; no C++ exception leaves it.
template <int (*F)(PyObject* const*), int N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
    if (n != N) {
        PyErr_Format(PyExc_TypeError, "%d arguments expected, got %zd", N, n);
        return nullptr;
    }
    try {
        const int status = F(args);
        return PyErr_Occurred() ? nullptr : PyLong_FromLong(status);
    } catch (const std::invalid_argument& e) {
        PyErr_SetString(PyExc_ValueError, e.what());
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

template <int (*F)(PyObject* const*), int N>
PyMethodDef method(const char* name) {
    return {name, (PyCFunction)(void (*)(void))entry<F, N>, METH_FASTCALL, nullptr};
}

PyMethodDef g_methods[] = {method<rope, 9>("rope"), method<append, 14>("append_paged"),
                           method<attn, 14>("tree_attn_paged"), method<commit, 12>("commit_paged"),
                           method<norm_rope, 11>("norm_rope"), method<append_q8, 19>("append_q8"),
                           method<commit_q8, 14>("commit_q8"), method<read_q8, 8>("read_q8"),
                           method<attn_q8, 14>("tree_attn_q8"), {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_ddtree", nullptr, -1, g_methods,
                        nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__ddtree(void) {
    PyObject* m = PyModule_Create(&g_module);
    // (the torch and interpreter whose headers it was compiled with: ops checks)
    if (m && PyModule_AddStringConstant(m, "built_for", DDTREE_BUILT_FOR)) {
        Py_DECREF(m);
        return nullptr;
    }
    return m;
}
