// paged_binding.cpp -- the hot side of vsa.PagedCache: checks the tensors of
// a call, allocates its outputs and passes their pointers on to the C entry
// points, for the decode step whose kernels take a few microseconds. The same
// in Python (checks, two torch.empty, a ctypes call) took 12.7 us for
// vsa_paged_attn on a GB300's CPU; here 4.7 us, most of it the launch.
//
// Module paged_binding, type Calls(desc, k, v, k_mean, workspace,
// workspace_bytes, functions, fail), the cache's tensors apart: desc is the address of a vsa_paged_desc
// (copied), k .. workspace device addresses (0: none), functions the
// addresses of vsa_paged_append, vsa_page_select and vsa_paged_attn, fail a
// callable (name, status) that raises. The tensors behind the addresses are
// kept alive by the owner. Calls run on the current stream of the cache's
// device, with that device current.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/core/grad_mode.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>
#include <sstream>
#include <stdexcept>
#include <utility>

#include "vsa.h"

namespace {

struct Calls {
    PyObject_HEAD;
    vsa_paged_desc d;
    void *k, *v, *mean, *ws;
    size_t ws_bytes;
    decltype(&vsa_paged_append) append;
    decltype(&vsa_page_select) select;
    decltype(&vsa_paged_attn) attn;
    PyObject *fail;
    int device;  // CUDA device index, -1: the cache is not on a GPU
    bool shared;  // k and v share memory: attended to, but not appended to
    at::ScalarType dtype() const { return d.dtype == VSA_DTYPE_BF16 ? at::kBFloat16 : at::kHalf; }
};

// A refused argument: ValueError.
struct Refused : std::invalid_argument {
    using std::invalid_argument::invalid_argument;
};
struct Raised {};  // the Python error is set

template <typename... A> [[noreturn]] void refuse(const A &...a) {
    std::ostringstream s;
    (s << ... << a);
    throw Refused(s.str());
}

const at::Tensor *optional(PyObject *o, const char *name) {
    if (o == Py_None) return nullptr;
    if (!THPVariable_Check(o)) refuse(name, ": expected a tensor");
    return &THPVariable_Unpack(o);
}
const at::Tensor &tensor(PyObject *o, const char *name) {
    const at::Tensor *t = optional(o, name);
    if (!t) refuse(name, ": expected a tensor");
    return *t;
}
long integer(PyObject *o, const char *name) {
    const long v = PyLong_AsLong(o);
    if (v == -1 && PyErr_Occurred()) throw Raised();
    if (v < INT32_MIN || v > INT32_MAX) refuse(name, ": out of range");
    return v;
}

void check_kind(const Calls &c, const char *name, const at::Tensor &t, at::ScalarType dtype) {
    const bool here = c.device < 0 ? t.is_cpu() : t.is_cuda() && t.get_device() == c.device;
    if (t.scalar_type() != dtype || !here || t.layout() != at::kStrided)
        refuse(name, ": expected ", dtype, " on the cache's device (", c.device < 0 ? "cpu" : "cuda:",
               c.device < 0 ? std::string() : std::to_string(c.device), "), got ", t.scalar_type(), " on ",
               t.device());
    if (t.requires_grad() && at::GradMode::is_enabled())
        refuse(name, ": the paged calls give no gradient; detach it, or call them under torch.no_grad()");
}
void check_dense(const Calls &c, const char *name, const at::Tensor &t, at::ScalarType dtype, at::IntArrayRef shape) {
    check_kind(c, name, t, dtype);
    if (t.sizes() != shape) refuse(name, ": expected ", shape, ", got ", t.sizes());
    if (!t.is_contiguous()) refuse(name, ": must be contiguous");
}
// Elements from one token of t [tokens, heads, D] to the next (heads and dims
// dense; 0 where there is only one token).
int64_t row_stride(const Calls &c, const char *name, const at::Tensor &t, int64_t heads) {
    check_kind(c, name, t, c.dtype());
    if (t.dim() != 3 || t.size(1) != heads || t.size(2) != c.d.D)
        refuse(name, ": expected [tokens, ", heads, ", ", c.d.D, "], got ", t.sizes());
    if (t.size(0) > 0 && (t.stride(2) != 1 || (heads > 1 && t.stride(1) != c.d.D)))
        refuse(name, ": heads and dims must be dense");
    if (t.size(0) < 2) return 0;
    if (t.stride(0) < heads * c.d.D) refuse(name, ": tokens must not share memory");  // 0 means dense further on
    return t.stride(0);
}
at::Tensor output(const Calls &c, at::IntArrayRef shape, at::ScalarType dtype) {
    const at::Device device = c.device < 0 ? at::Device(at::kCPU) : at::Device(at::kCUDA, c.device);
    return at::empty(shape, at::TensorOptions().dtype(dtype).device(device));
}
PyObject *pair(at::Tensor a, at::Tensor b) {
    PyObject *t = PyTuple_New(2);
    if (!t) throw Raised();
    PyTuple_SET_ITEM(t, 0, THPVariable_Wrap(std::move(a)));
    PyTuple_SET_ITEM(t, 1, THPVariable_Wrap(std::move(b)));
    return t;
}
// Equal pieces of memory, `pitch` bytes from one to the next: the rows of a
// part of a projection's output, the pages of one half of a buffer.
struct Pieces {
    const char *name;
    uintptr_t at;
    int64_t count, bytes, pitch;
};
// t, whose entries along its first dimension are dense.
Pieces pieces(const char *name, const at::Tensor &t) {
    const int64_t n = t.numel() > 0 ? t.size(0) : 0, size = t.element_size();
    return {name, (uintptr_t)t.data_ptr(), n, n ? t.numel() / n * size : 0, n ? t.stride(0) * size : 0};
}
Pieces whole(const char *name, const void *at, int64_t bytes) { return {name, (uintptr_t)at, at ? 1 : 0, bytes, 0}; }
bool meet(Pieces a, Pieces b) {
    if (a.count > b.count) std::swap(a, b);
    if (a.count == 0 || a.bytes == 0 || b.bytes == 0) return false;
    auto end = [](const Pieces &p) { return p.at + (p.count - 1) * p.pitch + p.bytes; };
    if (end(a) <= b.at || end(b) <= a.at) return false;
    for (int64_t i = 0; i < a.count; ++i) {
        const int64_t from = (int64_t)(a.at - b.at) + i * a.pitch;  // of this piece, behind b's first
        // b's first piece that ends behind it
        const int64_t j = from < b.bytes ? 0 : b.count == 1 ? 1 : (from - b.bytes) / b.pitch + 1;
        if (j < b.count && j * b.pitch < from + a.bytes) return true;
    }
    return false;
}
// Refuses memory that a call writes and that others of its tensors share:
// some CTAs still read the one while others write the other.
void apart(const Pieces &one, std::initializer_list<Pieces> others) {
    for (const Pieces &o : others)
        if (meet(one, o)) refuse(one.name, ": shares memory with ", o.name);
}
Pieces opt(const char *name, const at::Tensor *t) { return t ? pieces(name, *t) : Pieces{name, 0, 0, 0, 0}; }
// The cache's own memory.
Pieces cache_pages(const Calls &c, const char *name, const void *at) {
    const int64_t dense = (int64_t)c.d.page * c.d.Hkv * c.d.D * 2;
    return {name, (uintptr_t)at, at ? c.d.num_pages : 0, dense, c.d.page_stride ? c.d.page_stride * 2 : dense};
}
Pieces cache_k(const Calls &c) { return cache_pages(c, "the cache's k", c.k); }
Pieces cache_v(const Calls &c) { return cache_pages(c, "the cache's v", c.v); }
Pieces cache_mean(const Calls &c) {
    return whole("the cache's k_mean", c.mean, (int64_t)c.d.num_pages * c.d.Hkv * c.d.D * 4);
}
Pieces cache_table(const Calls &c) { return whole("page_table", c.d.page_table, (int64_t)c.d.B * c.d.max_pages * 4); }
Pieces cache_lens(const Calls &c) { return whole("seq_lens", c.d.seq_lens, (int64_t)c.d.B * 4); }
Pieces cache_ws(const Calls &c) { return whole("the workspace", c.ws, (int64_t)c.ws_bytes); }

template <typename T> T *ptr(const at::Tensor *t) { return t ? static_cast<T *>(t->data_ptr()) : nullptr; }

// The call itself: f(stream) with the cache's device current.
template <typename F> void run(const Calls &c, const char *name, F f) {
    if (c.device < 0) refuse("the cache is on cpu: the calls run on a GPU only");
    const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(c.device));
    const vsa_status st = f(static_cast<vsa_stream_t>(c10::cuda::getCurrentCUDAStream(c.device).stream()));
    if (st != VSA_OK) {
        PyObject *r = PyObject_CallFunction(c.fail, "si", name, (int)st);
        Py_XDECREF(r);
        if (!PyErr_Occurred()) PyErr_Format(PyExc_RuntimeError, "%s failed: %d", name, (int)st);
        throw Raised();
    }
}

// Runs a method body; refused arguments become ValueError, torch's errors
// what torch makes of them. No exception leaves.
template <typename F> PyObject *guarded(PyObject *self, Py_ssize_t given, Py_ssize_t wanted, F f) {
    HANDLE_TH_ERRORS
    if (given != wanted) {
        PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", wanted, given);
        return nullptr;
    }
    try {
        return f(*reinterpret_cast<Calls *>(self));
    } catch (const Refused &e) {
        PyErr_SetString(PyExc_ValueError, e.what());
        return nullptr;
    } catch (const Raised &) {
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

// append(k, v, q, cu_seqlens, cos, sin, positions, interleaved, q_out)
PyObject *calls_append(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    return guarded(self, n, 9, [&](Calls &c) -> PyObject * {
        if (!c.k) refuse("this cache has no k and v");
        if (c.shared) refuse("the cache's k and v share memory");
        const at::Tensor &k = tensor(a[0], "k"), &v = tensor(a[1], "v");
        const at::Tensor *q = optional(a[2], "q"), *cu = optional(a[3], "cu_seqlens"), *cos = optional(a[4], "cos"),
                         *sin = optional(a[5], "sin"), *pos = optional(a[6], "positions"),
                         *given = optional(a[8], "q_out");
        const int inter = PyObject_IsTrue(a[7]);
        if (inter < 0) throw Raised();
        const int64_t ks = row_stride(c, "k", k, c.d.Hkv), vs = row_stride(c, "v", v, c.d.Hkv), T = k.size(0);
        const int64_t qs = q ? row_stride(c, "q", *q, c.d.Hq) : 0;
        if (v.size(0) != T || (q && q->size(0) != T)) refuse("k, v and q must have the same number of tokens");
        if (T > INT32_MAX) refuse("k: too many tokens");
        if (cu)
            check_dense(c, "cu_seqlens", *cu, at::kInt, {c.d.B + 1});
        else if (T != c.d.B)
            refuse("without cu_seqlens there is one token per sequence");
        if (!cos != !sin) refuse("give both cos and sin, or neither");
        if (cos) {
            if (cos->dim() != 2 || cos->size(0) > INT32_MAX || cos->size(1) > c.d.D)
                refuse("cos and sin: expected [rows, rot_dim / 2], got ", cos->sizes());
            check_dense(c, "cos", *cos, at::kFloat, cos->sizes());
            check_dense(c, "sin", *sin, at::kFloat, cos->sizes());
        }
        if (pos) check_dense(c, "positions", *pos, at::kInt, {T});
        at::Tensor q_out;
        if (given) {
            if (!q) refuse("q_out without q");
            check_dense(c, "q_out", *given, c.dtype(), {T, c.d.Hq, c.d.D});
            if (T > 0 && given->data_ptr() == q->data_ptr()) refuse("q_out: must not be q");
            apart(pieces("q_out", *given),
                  {pieces("k", k), pieces("v", v), pieces("q", *q), opt("cu_seqlens", cu), opt("cos", cos),
                   opt("sin", sin), opt("positions", pos), cache_k(c), cache_v(c), cache_mean(c), cache_table(c),
                   cache_lens(c)});
            q_out = *given;
        } else if (q) {
            q_out = output(c, {T, c.d.Hq, c.d.D}, c.dtype());
        }
        for (const Pieces &written : {cache_k(c), cache_v(c), cache_mean(c)})
            apart(written, {pieces("k", k), pieces("v", v), opt("q", q), opt("cu_seqlens", cu), opt("cos", cos),
                            opt("sin", sin), opt("positions", pos)});
        if (T > 0 || c.device < 0)
            run(c, "vsa_paged_append", [&](vsa_stream_t s) {
                return c.append(&c.d, (int)T, k.data_ptr(), ks, v.data_ptr(), vs, ptr<void>(q), qs,
                                q ? q_out.data_ptr() : nullptr, ptr<int32_t>(cu), ptr<int32_t>(pos), ptr<float>(cos),
                                ptr<float>(sin), cos ? (int)cos->size(0) : 0, cos ? 2 * (int)cos->size(1) : 0, inter,
                                c.k, c.v, static_cast<float *>(c.mean), s);
            });
        if (!q) Py_RETURN_NONE;
        return THPVariable_Wrap(std::move(q_out));
    });
}

// Checks the queries of one token per sequence; their row stride.
int64_t query_rows(const Calls &c, const at::Tensor &q) {
    const int64_t qs = row_stride(c, "q", q, c.d.Hq);
    if (q.size(0) != c.d.B) refuse("q: expected one token for each of ", c.d.B, " sequences");
    return qs;
}

// select(q, topk, keep_first, keep_last, page_idx, page_cnt)
PyObject *calls_select(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    return guarded(self, n, 6, [&](Calls &c) -> PyObject * {
        if (!c.mean) refuse("this cache has no k_mean");
        const at::Tensor &q = tensor(a[0], "q");
        const long topk = integer(a[1], "topk"), first = integer(a[2], "keep_first"), last = integer(a[3], "keep_last");
        const at::Tensor *gi = optional(a[4], "page_idx"), *gc = optional(a[5], "page_cnt");
        const int64_t qs = query_rows(c, q);
        if (topk < 1) refuse("topk: at least one page");
        if (gi) check_dense(c, "page_idx", *gi, at::kInt, {c.d.B, c.d.Hkv, topk});
        if (gc) check_dense(c, "page_cnt", *gc, at::kInt, {c.d.B, c.d.Hkv});
        const Pieces pi = opt("page_idx", gi), pc = opt("page_cnt", gc);
        for (const Pieces &written : {pi, pc})
            apart(written, {pieces("q", q), cache_mean(c), cache_table(c), cache_lens(c), cache_ws(c)});
        apart(pi, {pc});
        at::Tensor idx = gi ? *gi : output(c, {c.d.B, c.d.Hkv, topk}, at::kInt);
        at::Tensor cnt = gc ? *gc : output(c, {c.d.B, c.d.Hkv}, at::kInt);
        run(c, "vsa_page_select", [&](vsa_stream_t s) {
            return c.select(&c.d, q.data_ptr(), qs, static_cast<float *>(c.mean), (int)topk, (int)first, (int)last,
                            ptr<int32_t>(&idx), ptr<int32_t>(&cnt), c.ws, c.ws_bytes, s);
        });
        return pair(std::move(idx), std::move(cnt));
    });
}

// attend(q, pages, out, lse)
PyObject *calls_attend(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    return guarded(self, n, 4, [&](Calls &c) -> PyObject * {
        if (!c.k) refuse("this cache has no k and v");
        const at::Tensor &q = tensor(a[0], "q");
        const int64_t qs = query_rows(c, q);
        const at::Tensor *idx = nullptr, *cnt = nullptr;
        if (a[1] != Py_None) {
            if (!PyTuple_Check(a[1]) || PyTuple_GET_SIZE(a[1]) != 2) refuse("pages: expected (page_idx, page_cnt)");
            idx = &tensor(PyTuple_GET_ITEM(a[1], 0), "page_idx");
            cnt = &tensor(PyTuple_GET_ITEM(a[1], 1), "page_cnt");
            if (idx->dim() != 3 || idx->size(2) > INT32_MAX) refuse("page_idx: expected [B, Hkv, cap]");
            check_dense(c, "page_idx", *idx, at::kInt, {c.d.B, c.d.Hkv, idx->size(2)});
            check_dense(c, "page_cnt", *cnt, at::kInt, {c.d.B, c.d.Hkv});
        }
        const at::Tensor *go = optional(a[2], "out"), *gl = optional(a[3], "lse");
        if (go) check_dense(c, "out", *go, c.dtype(), {c.d.B, c.d.Hq, c.d.D});
        if (go && go->data_ptr() == q.data_ptr()) refuse("out: must not be q");
        if (gl) check_dense(c, "lse", *gl, at::kFloat, {c.d.B, c.d.Hq});
        const Pieces po = opt("out", go), pl = opt("lse", gl);
        for (const Pieces &written : {po, pl})
            apart(written, {pieces("q", q), opt("page_idx", idx), opt("page_cnt", cnt), cache_k(c), cache_v(c),
                            cache_table(c), cache_lens(c), cache_ws(c)});
        apart(po, {pl});
        at::Tensor out = go ? *go : output(c, {c.d.B, c.d.Hq, c.d.D}, c.dtype());
        at::Tensor lse = gl ? *gl : output(c, {c.d.B, c.d.Hq}, at::kFloat);
        run(c, "vsa_paged_attn", [&](vsa_stream_t s) {
            return c.attn(&c.d, q.data_ptr(), qs, c.k, c.v, ptr<int32_t>(idx), ptr<int32_t>(cnt),
                          idx ? (int)idx->size(2) : 0, out.data_ptr(), ptr<float>(&lse), c.ws, c.ws_bytes, s);
        });
        return pair(std::move(out), std::move(lse));
    });
}

// Calls(desc, device, k, v, k_mean, workspace, workspace_bytes, append, select, attn, fail)
PyObject *calls_new(PyTypeObject *type, PyObject *args, PyObject *) {
    unsigned long long desc, k, v, mean, ws, bytes, append, select, attn;
    int device;
    PyObject *fail;
    if (!PyArg_ParseTuple(args, "KiKKKKKKKKO", &desc, &device, &k, &v, &mean, &ws, &bytes, &append, &select, &attn,
                          &fail))
        return nullptr;
    PyObject *self = type->tp_alloc(type, 0);
    if (!self) return nullptr;
    Calls *c = reinterpret_cast<Calls *>(self);
    c->d = *reinterpret_cast<const vsa_paged_desc *>(desc);
    c->device = device;
    c->k = reinterpret_cast<void *>(k);
    c->v = reinterpret_cast<void *>(v);
    c->mean = reinterpret_cast<void *>(mean);
    c->ws = reinterpret_cast<void *>(ws);
    c->ws_bytes = (size_t)bytes;
    c->append = reinterpret_cast<decltype(c->append)>(append);
    c->select = reinterpret_cast<decltype(c->select)>(select);
    c->attn = reinterpret_cast<decltype(c->attn)>(attn);
    Py_INCREF(fail);
    c->fail = fail;
    c->shared = meet(cache_k(*c), cache_v(*c));
    try {
        apart(cache_mean(*c), {cache_k(*c), cache_v(*c)});
        apart(cache_ws(*c), {cache_k(*c), cache_v(*c), cache_mean(*c)});
        for (const Pieces &read : {cache_table(*c), cache_lens(*c)})
            apart(read, {cache_k(*c), cache_v(*c), cache_mean(*c), cache_ws(*c)});
    } catch (const Refused &e) {
        PyErr_SetString(PyExc_ValueError, e.what());
        Py_DECREF(self);
        return nullptr;
    }
    return self;
}
void calls_dealloc(PyObject *self) {
    PyTypeObject *type = Py_TYPE(self);
    Py_XDECREF(reinterpret_cast<Calls *>(self)->fail);
    type->tp_free(self);
    Py_DECREF(type);
}

PyCFunction fast(PyObject *(*f)(PyObject *, PyObject *const *, Py_ssize_t)) {
    return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(f));
}
PyMethodDef methods[] = {
    {"append", fast(calls_append), METH_FASTCALL, "vsa_paged_append"},
    {"select", fast(calls_select), METH_FASTCALL, "vsa_page_select"},
    {"attend", fast(calls_attend), METH_FASTCALL, "vsa_paged_attn"},
    {nullptr, nullptr, 0, nullptr},
};
PyType_Slot slots[] = {
    {Py_tp_new, reinterpret_cast<void *>(calls_new)},
    {Py_tp_dealloc, reinterpret_cast<void *>(calls_dealloc)},
    {Py_tp_methods, methods},
    {0, nullptr},
};
PyType_Spec spec = {"paged_binding.Calls", sizeof(Calls), 0, Py_TPFLAGS_DEFAULT, slots};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "paged_binding", nullptr, -1, nullptr, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_paged_binding() {
    PyObject *m = PyModule_Create(&module);
    if (!m) return nullptr;
    PyObject *t = PyType_FromSpec(&spec);
    if (!t || PyModule_AddObject(m, "Calls", t) < 0) {
        Py_XDECREF(t);
        Py_DECREF(m);
        return nullptr;
    }
    return m;
}
