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
    const Tensor* t[3] = {};
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

// rope(q, k, pos, rotary, rotary_index, q_out, k_out, inverse, stream)
int rope(PyObject* const* a) {
    const Tensor& q = tensor(a[0], "q");
    if (!q.is_cuda() || q.dim() < 1 || code(q.scalar_type()) < 0)
        bad("q must be a bfloat16, float16 or float32 CUDA tensor, got " + about(q));
    const Common c{(int)q.get_device(), q.size(-1), q.scalar_type()};
    if (PyLong_AsLong(a[4]) != c.index) bad("rotary is on another device than q");
    const ddtree_rotary rot = packed<ddtree_rotary>(a[3], "rotary");
    const Rows qr = rows(q, "q", c);
    Rows qo = qr, kr{}, ko{};
    if (a[5] != Py_None) {
        qo = rows(a[5], "q_out", c);
        if (tensor(a[5], "q_out").sizes() != q.sizes()) bad("q_out must have q's shape");
    }
    const bool with_k = a[1] != Py_None;
    if (with_k) {
        const Tensor& k = tensor(a[1], "k");
        ko = kr = rows(k, "k", c);
        if (kr.tokens != qr.tokens)
            bad("k has " + std::to_string(kr.tokens) + " tokens, q " + std::to_string(qr.tokens));
        if (a[6] != Py_None) {
            ko = rows(a[6], "k_out", c);
            if (tensor(a[6], "k_out").sizes() != k.sizes()) bad("k_out must have k's shape");
        }
    } else if (a[6] != Py_None) {
        bad("k_out without k");
    }
    const int32_t* pos = token_ints(a[2], "pos", q, qr.tokens, c.index);
    Written w;
    w.add(a[5] == Py_None ? q : tensor(a[5], "q_out"), a[5] == Py_None ? "q" : "q_out");
    if (with_k) w.add(tensor(a[6] == Py_None ? a[1] : a[6], "k"), a[6] == Py_None ? "k" : "k_out");
    const Launch l(c.index, a[8]);
    return w.done(ddtree_rope(&qr.r, &qo.r, with_k ? &kr.r : nullptr, with_k ? &ko.r : nullptr,
                              code(c.dtype), (int)qr.tokens,
                              (int)std::min<int64_t>(c.D, INT32_MAX), pos, &rot,
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

// attn(cache x 3, q, k_tree, v_tree, prefix_len, n_nodes, anc_mask, out, lse, scale,
//      workspace, stream)
int attn(PyObject* const* a) {
    const Cache x = cache(a);
    a += 3;
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
    return w.done(ddtree_tree_attn_paged(&qr.r, &x.s, &kr.r, &vr.r, P, n, mask, (int)B, (int)(R - 1),
                                         (float)scale, out, lse, ws, bytes, l.stream));
}

// commit(cache x 3, k_tree, v_tree, accept_len, accepted_nodes, prefix_len, new_len, stream,
//        k_pages, v_pages)
int commit(PyObject* const* a) {
    const Cache x = cache(a);
    a += 3;
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
    Written w;
    w.add(tensor(a[7], "k_pages"), "k_pages");
    w.add(tensor(a[8], "v_pages"), "v_pages");
    if (to) w.add(tensor(a[5], "new_len"), "new_len");
    const Launch l(dev, a[6]);
    return w.done(ddtree_commit_paged(&x.s, &kr.r, &vr.r, alen, acc, P, to, (int)x.B,
                                      (int)std::min<int64_t>(L, INT32_MAX), (int)(kt.size(1) - 1),
                                      l.stream));
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
                           {nullptr, nullptr, 0, nullptr}};
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
