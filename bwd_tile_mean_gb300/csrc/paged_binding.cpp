// paged_binding.cpp -- the hot side of vsa.PagedCache and vsa.AxialRope: checks the tensors of
// a call, allocates its outputs and passes their pointers on to the C entry
// points, for the decode step whose kernels take a few microseconds. The same
// in Python (checks, two torch.empty, a ctypes call) took 12.7 us for
// vsa_paged_attn on a GB300's CPU; here 4.0 to 4.5 us, most of it the launch.
//
// Module paged_binding, type Calls(desc, device, eight, k, v, k_scale, v_scale, k_mean, workspace,
// workspace_bytes, weigh_bytes, functions, fail), the cache's tensors apart: desc is the address of a vsa_paged_desc
// (copied), eight whether the cache is in 8 bits, k .. workspace device addresses (0: none), weigh_bytes the workspace's
// for page weights (0: too small), functions the
// addresses of the paged entry points in the order of their members below, fail a
// callable (name, status) that raises. The tensors behind the addresses are
// kept alive by the owner. Calls run on the current stream of the cache's
// device, with that device current. Type Rope(rope, functions, fail): rope is
// the address of a vsa_rope (copied), functions those of vsa_rope_apply and
// vsa_rope_table; calls run on the device of their tensors.
#include <Python.h>

#include <ATen/Context.h>
#include <ATen/core/Tensor.h>
#include <ATen/core/grad_mode.h>
#include <ATen/cuda/EmptyTensor.h>
#include <ATen/ops/empty.h>
#include <ATen/record_function.h>
#include <c10/core/InferenceMode.h>
#include <c10/core/impl/TorchDispatchModeTLS.h>
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
    float *kscale, *vscale;
    size_t ws_bytes, weigh_bytes;
    decltype(&vsa_paged_append) append;
    decltype(&vsa_page_select) select;
    decltype(&vsa_paged_attn) attn;
    decltype(&vsa_paged8_append) append8;
    decltype(&vsa_paged8_attn) attn8;
    decltype(&vsa_paged_read) read;
    decltype(&vsa_paged_attn_weigh) weigh;
    decltype(&vsa_page_evict) evict;
    PyObject *fail;
    int device;  // CUDA device index, -1: the cache is not on a GPU
    bool eight;   // the cache is in 8 bits
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
// Whether at::empty does more than allocate: inference tensors, torch.use_deterministic_algorithms' NaN in uninitialised
// memory, dispatch modes and the profiler that are to see it.
bool empty_is_more() {
    const at::Context &torch = at::globalContext();
    return c10::InferenceMode::is_enabled() ||
           (torch.deterministicAlgorithms() && torch.deterministicFillUninitializedMemory()) ||
           c10::impl::dispatch_mode_enabled() || at::hasCallbacks();
}
// Dense tensors for a call's outputs, uninitialised: straight from the GPU's allocator where at::empty would come to that (two
// of them cost a call 3.4 us through the dispatcher, more than its launch; the question costs some 0.1).
struct Outputs {
    const bool more = empty_is_more();
    at::Tensor dense(at::IntArrayRef shape, at::ScalarType dtype, at::Device device) const {
        if (device.is_cuda() && !more) return at::Tensor(at::detail::empty_cuda(shape, dtype, device, std::nullopt));
        return at::empty(shape, at::TensorOptions().dtype(dtype).device(device));
    }
    at::Tensor dense(at::IntArrayRef shape, at::ScalarType dtype, const Calls &c) const {
        return dense(shape, dtype, c.device < 0 ? at::Device(at::kCPU) : at::Device(at::kCUDA, c.device));
    }
};
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
    const int64_t size = c.eight ? 1 : 2, dense = (int64_t)c.d.page * c.d.Hkv * c.d.D * size;
    return {name, (uintptr_t)at, at ? c.d.num_pages : 0, dense, c.d.page_stride ? c.d.page_stride * size : dense};
}
Pieces cache_k(const Calls &c) { return cache_pages(c, "the cache's k", c.k); }
Pieces cache_v(const Calls &c) { return cache_pages(c, "the cache's v", c.v); }
Pieces cache_mean(const Calls &c) {
    return whole("the cache's k_mean", c.mean, (int64_t)c.d.num_pages * c.d.Hkv * c.d.D * 4);
}
Pieces cache_scale(const Calls &c, const char *name, const float *at) {
    return whole(name, at, (int64_t)c.d.num_pages * c.d.Hkv * (c.d.page / 16) * 4);
}
Pieces cache_ks(const Calls &c) { return cache_scale(c, "the cache's k_scale", c.kscale); }
Pieces cache_vs(const Calls &c) { return cache_scale(c, "the cache's v_scale", c.vscale); }
Pieces cache_table(const Calls &c) { return whole("page_table", c.d.page_table, (int64_t)c.d.B * c.d.max_pages * 4); }
Pieces cache_lens(const Calls &c) { return whole("seq_lens", c.d.seq_lens, (int64_t)c.d.B * 4); }
Pieces cache_ws(const Calls &c, bool weigh = false) {
    return whole("the workspace", c.ws, (int64_t)(weigh ? c.weigh_bytes : c.ws_bytes));
}

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
template <typename C = Calls, typename F> PyObject *guarded(PyObject *self, Py_ssize_t given, Py_ssize_t wanted, F f) {
    HANDLE_TH_ERRORS
    if (given != wanted) {
        PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", wanted, given);
        return nullptr;
    }
    try {
        return f(*reinterpret_cast<C *>(self));
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
        const Outputs made;
        at::Tensor q_out;
        if (given) {
            if (!q) refuse("q_out without q");
            check_dense(c, "q_out", *given, c.dtype(), {T, c.d.Hq, c.d.D});
            if (T > 0 && given->data_ptr() == q->data_ptr()) refuse("q_out: must not be q");
            apart(pieces("q_out", *given),
                  {pieces("k", k), pieces("v", v), pieces("q", *q), opt("cu_seqlens", cu), opt("cos", cos),
                   opt("sin", sin), opt("positions", pos), cache_k(c), cache_v(c), cache_ks(c), cache_vs(c),
                   cache_mean(c), cache_table(c), cache_lens(c)});
            q_out = *given;
        } else if (q) {
            q_out = made.dense({T, c.d.Hq, c.d.D}, c.dtype(), c);
        }
        for (const Pieces &written : {cache_k(c), cache_v(c), cache_ks(c), cache_vs(c), cache_mean(c)})
            apart(written, {pieces("k", k), pieces("v", v), opt("q", q), opt("cu_seqlens", cu), opt("cos", cos),
                            opt("sin", sin), opt("positions", pos)});
        if (T > 0 || c.device < 0)
            run(c, c.eight ? "vsa_paged8_append" : "vsa_paged_append", [&](vsa_stream_t s) {
                if (c.eight)
                    return c.append8(&c.d, (int)T, k.data_ptr(), ks, v.data_ptr(), vs, ptr<void>(q), qs,
                                     q ? q_out.data_ptr() : nullptr, ptr<int32_t>(cu), ptr<int32_t>(pos), ptr<float>(cos),
                                     ptr<float>(sin), cos ? (int)cos->size(0) : 0, cos ? 2 * (int)cos->size(1) : 0, inter,
                                     c.k, c.v, c.kscale, c.vscale, static_cast<float *>(c.mean), s);
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
        const Outputs made;
        at::Tensor idx = gi ? *gi : made.dense({c.d.B, c.d.Hkv, topk}, at::kInt, c);
        at::Tensor cnt = gc ? *gc : made.dense({c.d.B, c.d.Hkv}, at::kInt, c);
        run(c, "vsa_page_select", [&](vsa_stream_t s) {
            return c.select(&c.d, q.data_ptr(), qs, static_cast<float *>(c.mean), (int)topk, (int)first, (int)last,
                            ptr<int32_t>(&idx), ptr<int32_t>(&cnt), c.ws, c.ws_bytes, s);
        });
        return pair(std::move(idx), std::move(cnt));
    });
}

double number(PyObject *o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw Raised();
    return v;
}

// attend(q, pages, out, lse, page_weight, weight_out, decay)
PyObject *calls_attend(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    return guarded(self, n, 7, [&](Calls &c) -> PyObject * {
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
        const at::Tensor *pw = optional(a[4], "page_weight"), *wo = optional(a[5], "weight_out");
        const double decay = number(a[6]);
        if (go) check_dense(c, "out", *go, c.dtype(), {c.d.B, c.d.Hq, c.d.D});
        if (go && go->data_ptr() == q.data_ptr()) refuse("out: must not be q");
        if (gl) check_dense(c, "lse", *gl, at::kFloat, {c.d.B, c.d.Hq});
        if (!pw && (wo || decay != 1.0)) refuse("weight_out and decay belong to page_weight");
        if (pw) {
            check_dense(c, "page_weight", *pw, at::kFloat, {c.d.B, c.d.Hkv, c.d.max_pages});
            if (wo) check_dense(c, "weight_out", *wo, at::kFloat, pw->sizes());
            if (!(decay >= 0.0 && decay <= 1.0)) refuse("decay: from 0 to 1, not ", decay);
            if (idx && idx->size(2) > c.d.max_pages) refuse("page_idx: no longer than the table where pages are weighed");
            if (!c.weigh_bytes) refuse("the workspace is too small for page weights: make the cache with weigh=True");
        }
        const at::Tensor *to = pw && !wo ? pw : wo;
        const Pieces po = opt("out", go), pl = opt("lse", gl), pt = opt("weight_out", to), pp = opt("page_weight", pw);
        for (const Pieces &written : {po, pl, pt})
            apart(written, {pieces("q", q), opt("page_idx", idx), opt("page_cnt", cnt), cache_k(c), cache_v(c), cache_ks(c),
                            cache_vs(c), cache_table(c), cache_lens(c), cache_ws(c, pw != nullptr)});
        apart(po, {pl, pt, pp});
        apart(pl, {pt, pp});
        if (pw && pt.at != pp.at) apart(pt, {pp});
        if (pw)  // the part behind the plain calls' may be a tensor of the cache, as long as pages are not weighed
            apart(cache_ws(c, true), {pp, cache_k(c), cache_v(c), cache_ks(c), cache_vs(c), cache_mean(c), cache_table(c),
                                      cache_lens(c)});
        const Outputs made;
        at::Tensor out = go ? *go : made.dense({c.d.B, c.d.Hq, c.d.D}, c.dtype(), c);
        at::Tensor lse = gl ? *gl : made.dense({c.d.B, c.d.Hq}, at::kFloat, c);
        const int cap = idx ? (int)idx->size(2) : 0;
        run(c, pw ? "vsa_paged_attn_weigh" : c.eight ? "vsa_paged8_attn" : "vsa_paged_attn", [&](vsa_stream_t s) {
            if (pw)
                return c.weigh(&c.d, q.data_ptr(), qs, c.k, c.v, c.kscale, c.vscale, ptr<int32_t>(idx), ptr<int32_t>(cnt), cap,
                               out.data_ptr(), ptr<float>(&lse), ptr<float>(pw), ptr<float>(to), (float)decay, c.ws,
                               c.weigh_bytes, s);
            if (c.eight)
                return c.attn8(&c.d, q.data_ptr(), qs, c.k, c.v, c.kscale, c.vscale, ptr<int32_t>(idx), ptr<int32_t>(cnt), cap,
                               out.data_ptr(), ptr<float>(&lse), c.ws, c.ws_bytes, s);
            return c.attn(&c.d, q.data_ptr(), qs, c.k, c.v, ptr<int32_t>(idx), ptr<int32_t>(cnt), cap, out.data_ptr(),
                          ptr<float>(&lse), c.ws, c.ws_bytes, s);
        });
        return pair(std::move(out), std::move(lse));
    });
}

// read(tokens, cu_seqlens, k_out, v_out)
PyObject *calls_read(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    return guarded(self, n, 4, [&](Calls &c) -> PyObject * {
        if (!c.k) refuse("this cache has no k and v");
        const long T = integer(a[0], "tokens");
        const at::Tensor *cu = optional(a[1], "cu_seqlens"), *gk = optional(a[2], "k_out"), *gv = optional(a[3], "v_out");
        if (T < 0) refuse("tokens: out of range");
        if (cu)
            check_dense(c, "cu_seqlens", *cu, at::kInt, {c.d.B + 1});
        else if (T != c.d.B)
            refuse("without cu_seqlens there is one token per sequence");
        if (gk) check_dense(c, "k_out", *gk, c.dtype(), {T, c.d.Hkv, c.d.D});
        if (gv) check_dense(c, "v_out", *gv, c.dtype(), {T, c.d.Hkv, c.d.D});
        const Pieces pk = opt("k_out", gk), pv = opt("v_out", gv);
        for (const Pieces &written : {pk, pv})
            apart(written, {opt("cu_seqlens", cu), cache_k(c), cache_v(c), cache_ks(c), cache_vs(c), cache_table(c),
                            cache_lens(c)});
        apart(pk, {pv});
        const Outputs made;
        at::Tensor k = gk ? *gk : made.dense({T, c.d.Hkv, c.d.D}, c.dtype(), c);
        at::Tensor v = gv ? *gv : made.dense({T, c.d.Hkv, c.d.D}, c.dtype(), c);
        if (T > 0 || c.device < 0)
            run(c, "vsa_paged_read", [&](vsa_stream_t s) {
                return c.read(&c.d, (int)T, ptr<int32_t>(cu), c.k, c.v, c.kscale, c.vscale, k.data_ptr(), v.data_ptr(), s);
            });
        return pair(std::move(k), std::move(v));
    });
}

// evict(page_weight, keep, keep_first, keep_last, freed, freed_cnt, out)
PyObject *calls_evict(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    return guarded(self, n, 7, [&](Calls &c) -> PyObject * {
        const at::Tensor &w = tensor(a[0], "page_weight");
        const long keep = integer(a[1], "keep"), first = integer(a[2], "keep_first"), last = integer(a[3], "keep_last");
        const at::Tensor *gf = optional(a[4], "freed"), *gc = optional(a[5], "freed_cnt");
        check_dense(c, "page_weight", w, at::kFloat, {c.d.B, c.d.Hkv, c.d.max_pages});
        if (first < 0 || last < 1 || keep < first + last)
            refuse("keep: at least keep_first (0 or more) and keep_last (1 or more), not ", keep, " of ", first, " and ", last);
        const int64_t cap = keep < c.d.max_pages ? c.d.max_pages - keep : 1;
        if (gf) check_dense(c, "freed", *gf, at::kInt, {c.d.B, cap});
        if (gc) check_dense(c, "freed_cnt", *gc, at::kInt, {c.d.B});
        // in place, or into the three tensors of `out`
        void *table = const_cast<int32_t *>(c.d.page_table), *lens = const_cast<int32_t *>(c.d.seq_lens), *to = w.data_ptr();
        if (a[6] != Py_None) {
            if (!PyTuple_Check(a[6]) || PyTuple_GET_SIZE(a[6]) != 3)
                refuse("out: expected (page_table, seq_lens, page_weight)");
            const at::Tensor &t = tensor(PyTuple_GET_ITEM(a[6], 0), "out: page_table"),
                             &l = tensor(PyTuple_GET_ITEM(a[6], 1), "out: seq_lens"),
                             &o = tensor(PyTuple_GET_ITEM(a[6], 2), "out: page_weight");
            check_dense(c, "out: page_table", t, at::kInt, {c.d.B, c.d.max_pages});
            check_dense(c, "out: seq_lens", l, at::kInt, {c.d.B});
            check_dense(c, "out: page_weight", o, at::kFloat, w.sizes());
            table = t.data_ptr();
            lens = l.data_ptr();
            to = o.data_ptr();
        }
        const Pieces in[3] = {cache_table(c), cache_lens(c), pieces("page_weight", w)};
        Pieces outs[5] = {in[0], in[1], in[2], opt("freed", gf), opt("freed_cnt", gc)};
        const void *at[3] = {table, lens, to};
        const char *names[3] = {"the evicted page_table", "the evicted seq_lens", "the evicted page_weight"};
        for (int i = 0; i < 3; ++i) outs[i].at = (uintptr_t)at[i], outs[i].name = names[i];
        for (int i = 0; i < 5; ++i) {
            apart(outs[i], {cache_k(c), cache_v(c), cache_ks(c), cache_vs(c), cache_mean(c), cache_ws(c)});
            for (int j = 0; j < 3; ++j)
                if (i != j || outs[i].at != in[j].at) apart(outs[i], {in[j]});
            for (int j = 0; j < i; ++j) apart(outs[i], {outs[j]});
        }
        apart(cache_ws(c), {in[2]});
        const Outputs made;
        at::Tensor freed = gf ? *gf : made.dense({c.d.B, cap}, at::kInt, c);
        at::Tensor count = gc ? *gc : made.dense({c.d.B}, at::kInt, c);
        run(c, "vsa_page_evict", [&](vsa_stream_t s) {
            return c.evict(&c.d, ptr<float>(&w), (int)keep, (int)first, (int)last, static_cast<int32_t *>(table),
                           static_cast<int32_t *>(lens), static_cast<float *>(to), ptr<int32_t>(&freed), ptr<int32_t>(&count),
                           c.ws, c.ws_bytes, s);
        });
        return pair(std::move(freed), std::move(count));
    });
}

// Calls(desc, device, eight, k, v, k_scale, v_scale, k_mean, workspace, workspace_bytes, weigh_bytes, functions, fail)
PyObject *calls_new(PyTypeObject *type, PyObject *args, PyObject *) {
    unsigned long long desc, k, v, ks, vs, mean, ws, bytes, weigh_bytes, f[8];
    int device, eight;
    PyObject *fail;
    if (!PyArg_ParseTuple(args, "KipKKKKKKKK(KKKKKKKK)O", &desc, &device, &eight, &k, &v, &ks, &vs, &mean, &ws, &bytes,
                          &weigh_bytes, &f[0], &f[1], &f[2], &f[3], &f[4], &f[5], &f[6], &f[7], &fail))
        return nullptr;
    PyObject *self = type->tp_alloc(type, 0);
    if (!self) return nullptr;
    Calls *c = reinterpret_cast<Calls *>(self);
    c->d = *reinterpret_cast<const vsa_paged_desc *>(desc);
    c->device = device;
    c->eight = eight != 0;
    c->k = reinterpret_cast<void *>(k);
    c->v = reinterpret_cast<void *>(v);
    c->kscale = reinterpret_cast<float *>(ks);
    c->vscale = reinterpret_cast<float *>(vs);
    c->mean = reinterpret_cast<void *>(mean);
    c->ws = reinterpret_cast<void *>(ws);
    c->ws_bytes = (size_t)bytes;
    c->weigh_bytes = (size_t)weigh_bytes;
    c->append = reinterpret_cast<decltype(c->append)>(f[0]);
    c->select = reinterpret_cast<decltype(c->select)>(f[1]);
    c->attn = reinterpret_cast<decltype(c->attn)>(f[2]);
    c->append8 = reinterpret_cast<decltype(c->append8)>(f[3]);
    c->attn8 = reinterpret_cast<decltype(c->attn8)>(f[4]);
    c->read = reinterpret_cast<decltype(c->read)>(f[5]);
    c->weigh = reinterpret_cast<decltype(c->weigh)>(f[6]);
    c->evict = reinterpret_cast<decltype(c->evict)>(f[7]);
    Py_INCREF(fail);
    c->fail = fail;
    c->shared = meet(cache_k(*c), cache_v(*c));
    try {
        apart(cache_mean(*c), {cache_k(*c), cache_v(*c)});
        apart(cache_ws(*c), {cache_k(*c), cache_v(*c), cache_mean(*c)});
        apart(cache_ks(*c), {cache_vs(*c)});
        for (const Pieces &scale : {cache_ks(*c), cache_vs(*c)})
            apart(scale, {cache_k(*c), cache_v(*c), cache_mean(*c), cache_ws(*c)});
        for (const Pieces &read : {cache_table(*c), cache_lens(*c)})
            apart(read, {cache_k(*c), cache_v(*c), cache_ks(*c), cache_vs(*c), cache_mean(*c), cache_ws(*c)});
    } catch (const Refused &e) {
        PyErr_SetString(PyExc_ValueError, e.what());
        Py_DECREF(self);
        return nullptr;
    }
    return self;
}
struct Rope {
    PyObject_HEAD;
    vsa_rope r;
    decltype(&vsa_rope_apply) apply;
    decltype(&vsa_rope_table) table;
    PyObject *fail;
};

// A tensor of tokens as vsa_rope_apply takes it: sizes and strides of batch
// entries, tokens and heads (strides of dimensions of one entry are 0).
struct Tokens {
    const char *name;
    char *at;
    int64_t size, n[3], stride[3];  // element size; batch, tokens, heads
    int64_t last() const {          // bytes from the first element to behind the last
        int64_t e = 128;
        for (int i = 0; i < 3; ++i) e += (n[i] - 1) * stride[i];
        return e * size;
    }
};
enum { kBhsd = 0, kBshd = 1, kTnd = 2 };
Tokens tokens(const char *name, const at::Tensor &t, int layout) {
    const int64_t dims = layout == kTnd ? 3 : 4;
    if (t.dim() != dims || t.size(dims - 1) != 128)
        refuse(name, ": expected ", layout == kTnd ? "[T, H, 128]" : layout == kBshd ? "[B, S, H, 128]" : "[B, H, S, 128]",
               ", got ", t.sizes());
    const int64_t order[3][3] = {{0, 2, 1}, {0, 1, 2}, {-1, 0, 1}};
    Tokens k{name, static_cast<char *>(t.data_ptr()), (int64_t)t.element_size(), {}, {}};
    if (t.numel() > 0 && t.stride(dims - 1) != 1) refuse(name, ": the last dimension must be dense");
    for (int i = 0; i < 3; ++i) {
        const int64_t d = order[layout][i];
        k.n[i] = d < 0 ? 1 : t.size(d);
        k.stride[i] = k.n[i] > 1 ? t.stride(d) : 0;
        if (k.stride[i] % 8 != 0) refuse(name, ": strides must be multiples of 8 elements");
    }
    return k;
}
bool empty(const Tokens &t) { return t.n[0] == 0 || t.n[1] == 0 || t.n[2] == 0; }
bool same_place(const Tokens &a, const Tokens &b) {
    bool same = a.at == b.at;
    for (int i = 0; i < 3; ++i) same = same && a.n[i] == b.n[i] && a.stride[i] == b.stride[i];
    return same;
}
// Whether the rows of `t` are known to be apart from each other.
bool rows_apart(const Tokens &t) {
    int at[3] = {0, 1, 2};
    for (int i = 0; i < 3; ++i)
        for (int j = i + 1; j < 3; ++j)
            if (t.stride[at[j]] < t.stride[at[i]]) std::swap(at[i], at[j]);
    int64_t reach = 128;  // elements of the dimensions so far
    for (int i : at) {
        if (t.n[i] < 2) continue;
        if (t.stride[i] < reach) return false;
        reach = (t.n[i] - 1) * t.stride[i] + reach;
    }
    return true;
}
// Whether a and b are known to share no memory: apart as a whole, or heads
// side by side in the same rows of one buffer, as the parts of a projection's
// output are.
bool are_apart(const Tokens &a, const Tokens &b) {
    if (empty(a) || empty(b) || a.at + a.last() <= b.at || b.at + b.last() <= a.at) return true;
    auto dense = [](const Tokens &t) { return t.n[2] < 2 || t.stride[2] == 128; };
    const int64_t row = a.n[1] > 1 ? a.stride[1] : a.stride[0];
    if (!dense(a) || !dense(b) || row <= 0 || a.n[0] != b.n[0] || a.n[1] != b.n[1] || a.stride[0] != b.stride[0] ||
        a.stride[1] != b.stride[1] || a.stride[0] % row != 0)
        return false;
    const int64_t pitch = row * a.size;
    int64_t rel = (b.at - a.at) % pitch;
    if (rel < 0) rel += pitch;
    return rel >= a.n[2] * 128 * a.size && rel + b.n[2] * 128 * b.size <= pitch;
}
void same_device(const at::Tensor &first, const char *name, const at::Tensor &t, at::ScalarType dtype) {
    if (t.scalar_type() != dtype || t.device() != first.device() || t.layout() != at::kStrided)
        refuse(name, ": expected ", dtype, " on ", first.device(), ", got ", t.scalar_type(), " on ", t.device());
    if (t.requires_grad() && at::GradMode::is_enabled())
        refuse(name, ": the call records no gradient; use backward() for it, and call both under torch.no_grad()");
}
// The call itself, with the tensors' device current.
template <typename F> void run_at(const Rope &r, const at::Tensor &first, const char *name, F f) {
    if (!first.is_cuda()) refuse("the tensors are on ", first.device(), ": the calls run on a GPU only");
    const c10::cuda::CUDAGuard guard(first.device());
    const vsa_status st = f(static_cast<vsa_stream_t>(c10::cuda::getCurrentCUDAStream(first.get_device()).stream()));
    if (st != VSA_OK) {
        PyObject *x = PyObject_CallFunction(r.fail, "si", name, (int)st);
        Py_XDECREF(x);
        if (!PyErr_Occurred()) PyErr_Format(PyExc_RuntimeError, "%s failed: %d", name, (int)st);
        throw Raised();
    }
}
// Positions [S, axes] or [B, S, axes]: strides between batch entries and tokens.
struct Positions {
    const int32_t *at;
    int64_t batch, token;
};
Positions positions_of(const Rope &r, const at::Tensor &t, int64_t B, int64_t S, bool batched) {
    const int64_t d = t.dim();
    if (!(d == 2 || (batched && d == 3)) || t.size(d - 1) != r.r.n_axes || t.size(d - 2) != S || (d == 3 && t.size(0) != B))
        refuse("positions: expected ", batched ? "[S, axes] or [B, S, axes]" : "[T, axes]", " of ", B, " x ", S,
               " tokens and ", r.r.n_axes, " axes, got ", t.sizes());
    if (t.numel() > 0 && r.r.n_axes > 1 && t.stride(d - 1) != 1) refuse("positions: a token's must be dense");
    return {static_cast<int32_t *>(t.data_ptr()), d == 3 && B > 1 ? t.stride(0) : 0, S > 1 ? t.stride(d - 2) : 0};
}
Tokens as_tokens(const at::Tensor &t, const char *name) {  // a dense or strided small tensor as one piece of memory
    int64_t last = t.numel() > 0 ? 1 : 0;
    for (int64_t i = 0; i < t.dim() && last; ++i) last += (t.size(i) - 1) * t.stride(i);
    Tokens k{name, static_cast<char *>(t.data_ptr()), 1, {last ? 1 : 0, 1, 1}, {}};
    k.n[1] = last * (int64_t)t.element_size();  // bytes as tokens one byte apart
    k.stride[1] = 1;
    return k;
}

// apply(q, k, positions, layout, q_out, k_out, inverse)
PyObject *rope_apply(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    return guarded<Rope>(self, n, 7, [&](Rope &r) -> PyObject * {
        const at::Tensor &q = tensor(a[0], "q"), &pos = tensor(a[2], "positions");
        const at::Tensor *k = optional(a[1], "k"), *qo = optional(a[4], "q_out"), *ko = optional(a[5], "k_out");
        const long layout = integer(a[3], "layout");
        const int inverse = PyObject_IsTrue(a[6]);
        if (inverse < 0) throw Raised();
        if (layout < 0 || layout > 2) refuse("layout: bshd, bhsd or tnd");
        if (ko && !k) refuse("k_out without k");
        if (q.scalar_type() != at::kBFloat16 && q.scalar_type() != at::kHalf)
            refuse("q: expected bfloat16 or float16, got ", q.scalar_type());
        const at::ScalarType dtype = q.scalar_type();
        same_device(q, "q", q, dtype);
        same_device(q, "positions", pos, at::kInt);
        Tokens x[2] = {tokens("q", q, layout)};
        const int64_t B = x[0].n[0], S = x[0].n[1];
        if (k) {
            same_device(q, "k", *k, dtype);
            x[1] = tokens("k", *k, layout);
            if (x[1].n[0] != B || x[1].n[1] != S) refuse("k: expected as many tokens as q, got ", k->sizes());
        }
        for (int i = 0; i < (k ? 2 : 1); ++i)
            if (B > INT32_MAX || S > INT32_MAX || x[i].n[2] > INT32_MAX) refuse(x[i].name, ": too large");
        const Positions p = positions_of(r, pos, B, S, layout != kTnd);
        const int count = k ? 2 : 1;
        const Outputs made;
        at::Tensor out[2];
        Tokens y[2];
        const at::Tensor *in[2] = {&q, k}, *given[2] = {qo, ko};
        for (int i = 0; i < count; ++i) {
            const char *name = i ? "k_out" : "q_out";
            if (given[i]) {
                same_device(q, name, *given[i], dtype);
                if (given[i]->sizes() != in[i]->sizes())
                    refuse(name, ": expected ", in[i]->sizes(), ", got ", given[i]->sizes());
                out[i] = *given[i];
            } else {
                out[i] = made.dense(in[i]->sizes(), dtype, q.device());
            }
            y[i] = tokens(name, out[i], layout);
            if (!given[i]) continue;
            if (!empty(y[i]) && !rows_apart(y[i])) refuse(name, ": its rows share memory");
            for (int j = 0; j < count; ++j)
                if (!(i == j && same_place(y[i], x[j])) && !are_apart(y[i], x[j]))
                    refuse(name, ": shares memory with ", x[j].name);
            const char *first = y[i].at, *end = first + (empty(y[i]) ? 0 : y[i].last());
            const Tokens m = as_tokens(pos, "positions");
            if (!empty(m) && !empty(y[i]) && m.at < end && first < m.at + m.n[1]) refuse(name, ": shares memory with positions");
        }
        if (count == 2 && !are_apart(y[0], y[1])) refuse("q_out: shares memory with k_out");
        // a tensor without heads has no part in the call
        vsa_rope_tensor t[2];
        int used = 0;
        for (int i = 0; i < count; ++i)
            if (!empty(x[i]))
                t[used++] = {x[i].at,        y[i].at,        (int32_t)x[i].n[2], x[i].stride[0], x[i].stride[1],
                             x[i].stride[2], y[i].stride[0], y[i].stride[1],     y[i].stride[2]};
        if (used)
            run_at(r, q, "vsa_rope_apply", [&](vsa_stream_t s) {
                return r.apply(&r.r, dtype == at::kBFloat16 ? VSA_DTYPE_BF16 : VSA_DTYPE_FP16, (int)B, (int)S, 128, t, used,
                               p.at, p.batch, p.token, inverse, s);
            });
        if (!k) return THPVariable_Wrap(std::move(out[0]));
        return pair(std::move(out[0]), std::move(out[1]));
    });
}

// table(positions, cos, sin)
PyObject *rope_table(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    return guarded<Rope>(self, n, 3, [&](Rope &r) -> PyObject * {
        const at::Tensor &pos = tensor(a[0], "positions");
        const at::Tensor *gc = optional(a[1], "cos"), *gs = optional(a[2], "sin");
        same_device(pos, "positions", pos, at::kInt);
        const int64_t T = pos.dim() == 2 ? pos.size(0) : 0, pairs = r.r.rot_dim / 2;
        const Positions p = positions_of(r, pos, 1, T, false);
        if (T > INT32_MAX) refuse("positions: too many tokens");
        const Outputs made;
        at::Tensor out[2];
        const at::Tensor *given[2] = {gc, gs};
        for (int i = 0; i < 2; ++i) {
            const char *name = i ? "sin" : "cos";
            if (given[i]) {
                same_device(pos, name, *given[i], at::kFloat);
                if (given[i]->sizes() != at::IntArrayRef({T, pairs}) || !given[i]->is_contiguous())
                    refuse(name, ": expected a contiguous [", T, ", ", pairs, "], got ", given[i]->sizes());
                out[i] = *given[i];
            } else {
                out[i] = made.dense({T, pairs}, at::kFloat, pos.device());
            }
        }
        const Tokens m = as_tokens(pos, "positions");
        const Pieces mine = whole("positions", m.at, m.n[0] ? m.n[1] : 0);
        apart(pieces("cos", out[0]), {mine, pieces("sin", out[1])});
        apart(pieces("sin", out[1]), {mine});
        if (T > 0)
            run_at(r, pos, "vsa_rope_table", [&](vsa_stream_t s) {
                return r.table(&r.r, (int)T, p.at, p.token, static_cast<float *>(out[0].data_ptr()),
                               static_cast<float *>(out[1].data_ptr()), s);
            });
        return pair(std::move(out[0]), std::move(out[1]));
    });
}

// Rope(rope, apply, table, fail)
PyObject *rope_new(PyTypeObject *type, PyObject *args, PyObject *) {
    unsigned long long rope, apply, table;
    PyObject *fail;
    if (!PyArg_ParseTuple(args, "KKKO", &rope, &apply, &table, &fail)) return nullptr;
    PyObject *self = type->tp_alloc(type, 0);
    if (!self) return nullptr;
    Rope *r = reinterpret_cast<Rope *>(self);
    r->r = *reinterpret_cast<const vsa_rope *>(rope);
    r->apply = reinterpret_cast<decltype(r->apply)>(apply);
    r->table = reinterpret_cast<decltype(r->table)>(table);
    Py_INCREF(fail);
    r->fail = fail;
    return self;
}
template <typename C> void drop(PyObject *self) {
    PyTypeObject *type = Py_TYPE(self);
    Py_XDECREF(reinterpret_cast<C *>(self)->fail);
    type->tp_free(self);
    Py_DECREF(type);
}

PyCFunction fast(PyObject *(*f)(PyObject *, PyObject *const *, Py_ssize_t)) {
    return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(f));
}
PyMethodDef methods[] = {
    {"append", fast(calls_append), METH_FASTCALL, "vsa_paged_append, vsa_paged8_append"},
    {"select", fast(calls_select), METH_FASTCALL, "vsa_page_select"},
    {"attend", fast(calls_attend), METH_FASTCALL, "vsa_paged_attn, vsa_paged8_attn, vsa_paged_attn_weigh"},
    {"read", fast(calls_read), METH_FASTCALL, "vsa_paged_read"},
    {"evict", fast(calls_evict), METH_FASTCALL, "vsa_page_evict"},
    {nullptr, nullptr, 0, nullptr},
};
PyType_Slot slots[] = {
    {Py_tp_new, reinterpret_cast<void *>(calls_new)},
    {Py_tp_dealloc, reinterpret_cast<void *>(drop<Calls>)},
    {Py_tp_methods, methods},
    {0, nullptr},
};
PyType_Spec spec = {"paged_binding.Calls", sizeof(Calls), 0, Py_TPFLAGS_DEFAULT, slots};
PyMethodDef rope_methods[] = {
    {"apply", fast(rope_apply), METH_FASTCALL, "vsa_rope_apply"},
    {"table", fast(rope_table), METH_FASTCALL, "vsa_rope_table"},
    {nullptr, nullptr, 0, nullptr},
};
PyType_Slot rope_slots[] = {
    {Py_tp_new, reinterpret_cast<void *>(rope_new)},
    {Py_tp_dealloc, reinterpret_cast<void *>(drop<Rope>)},
    {Py_tp_methods, rope_methods},
    {0, nullptr},
};
PyType_Spec rope_spec = {"paged_binding.Rope", sizeof(Rope), 0, Py_TPFLAGS_DEFAULT, rope_slots};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "paged_binding", nullptr, -1, nullptr, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_paged_binding() {
    PyObject *m = PyModule_Create(&module);
    if (!m) return nullptr;
    for (auto [name, from] : {std::pair{"Calls", &spec}, std::pair{"Rope", &rope_spec}}) {
        PyObject *t = PyType_FromSpec(from);
        if (!t || PyModule_AddObject(m, name, t) < 0) {
            Py_XDECREF(t);
            Py_DECREF(m);
            return nullptr;
        }
    }
    return m;
}
