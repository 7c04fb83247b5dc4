// The torch side of the paged cache's calls: checks of the tensors, allocation of what a call returns, the current
// stream, and attention's and selection's workspaces. A decode step's calls are small, and in Python these steps
// took longer than the kernels (15 to 17 us a call against 4 to 8); here they take about 4.
//
// Functions of a CPython module over the C ABI of libpolykv; pages.py wraps them and documents the arguments.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <algorithm>
#include <map>
#include <vector>
#include <string>
#include <utility>

#include <ATen/core/grad_mode.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "polykv.h"

namespace {

PyObject* g_error = nullptr;   // PolyKVError(status, message)

struct Failure {};             // a Python exception is set

[[noreturn]] void value_error(const std::string& msg) {
    PyErr_SetString(PyExc_ValueError, msg.c_str());
    throw Failure{};
}
void check(polykv_status st) {
    if (st == POLYKV_OK) return;
    PyObject* e = PyObject_CallFunction(g_error, "is", (int)st, polykv_last_error());
    if (e) {
        PyErr_SetObject(g_error, e);
        Py_DECREF(e);
    }
    throw Failure{};
}

// Where a call's tensors have to be, and whose device that is.
struct Owner {
    c10::Device device{c10::DeviceType::CPU};
    const char* name = "the cache";
    bool plural = false;
};
// A cache as these calls see it.
struct Cache : Owner {
    polykv_pages* handle;
    int64_t H, d;
    c10::ScalarType dtype;   // of rows
    std::map<std::pair<cudaStream_t, int>, at::Tensor> attend_ws;   // by stream and query heads
    std::map<cudaStream_t, at::Tensor> select_ws, joint_ws, rows_ws;
};
// Block tables as these calls see them.
struct Tables : Owner {
    polykv_page_tables t;
    std::vector<at::Tensor> kept;   // what t points into
};
Cache* cache_of(PyObject* o) {
    void* p = PyCapsule_GetPointer(o, "polykv.pages");
    if (!p) throw Failure{};
    return static_cast<Cache*>(p);
}
void cache_free(PyObject* o) { delete static_cast<Cache*>(PyCapsule_GetPointer(o, "polykv.pages")); }
Tables* tables_of(PyObject* o) {
    void* p = PyCapsule_GetPointer(o, "polykv.tables");
    if (!p) throw Failure{};
    return static_cast<Tables*>(p);
}
void tables_free(PyObject* o) { delete static_cast<Tables*>(PyCapsule_GetPointer(o, "polykv.tables")); }

const at::Tensor& tensor(PyObject* o, const char* name) {
    if (!THPVariable_Check(o)) value_error(std::string(name) + " must be a tensor");
    return THPVariable_Unpack(o);
}

std::string shape_text(c10::IntArrayRef s) {
    std::string t = "(";
    for (size_t i = 0; i < s.size(); ++i) t += (i ? ", " : "") + std::to_string(s[i]);
    return t + ")";
}
void check_shape(const at::Tensor& t, const char* name, c10::IntArrayRef want) {
    if (!t.sizes().equals(want))
        value_error(std::string(name) + " has shape " + shape_text(t.sizes()) + ", expected " + shape_text(want));
}
void check_kind(const at::Tensor& t, const char* name, c10::ScalarType dtype, const Owner& c) {
    if (t.scalar_type() != dtype)
        value_error(std::string(name) + " must be " + c10::toString(dtype) + ", got " + c10::toString(t.scalar_type()));
    if (t.device() != c.device)
        value_error(std::string(name) + " is on " + t.device().str() + ", " + c.name + " on " + c.device.str());
}
// These calls have no backward pass and their results no history: a tensor that would need one is refused, not detached.
void check_no_grad(const at::Tensor& t, const char* name) {
    if (at::GradMode::is_enabled() && t.requires_grad())
        value_error(std::string(name) + " requires a gradient, which this call does not give: detach it or call under torch.no_grad()");
}
// A contiguous tensor of exactly this shape and type on the cache's device.
const at::Tensor& exactly(PyObject* o, const char* name, c10::IntArrayRef shape, c10::ScalarType dtype, const Owner& c) {
    const at::Tensor& t = tensor(o, name);
    check_shape(t, name, shape);
    check_kind(t, name, dtype, c);
    if (!t.is_contiguous()) value_error(std::string(name) + " must be contiguous");
    return t;
}
const at::Tensor& four(PyObject* o, const char* name, const char* dims) {
    const at::Tensor& t = tensor(o, name);
    if (t.dim() != 4) value_error(std::string(name) + " must be " + dims + ", got shape " + shape_text(t.sizes()));
    return t;
}
// [layers][rows][heads][d] with a contiguous last dimension.
polykv_row_strides rows_of(const at::Tensor& t, const char* name, c10::IntArrayRef shape, const Cache& c) {
    check_shape(t, name, shape);
    check_kind(t, name, c.dtype, c);
    if (t.stride(3) != 1) value_error(std::string(name) + "'s last dimension must be contiguous");
    // the stride of a dimension of one element says nothing
    return {shape[0] > 1 ? t.stride(0) : 0, shape[1] > 1 ? t.stride(1) : 0, shape[2] > 1 ? t.stride(2) : 0};
}
// A result whose elements stand in places of their own: sorted by stride, each dimension steps over those before it.
void check_places(const at::Tensor& t, const char* name) {
    int dims[4] = {0, 1, 2, 3};
    std::sort(dims, dims + 4, [&](int a, int b) { return t.stride(a) < t.stride(b); });
    int64_t reach = 1;
    for (int i : dims) {
        if (t.size(i) < 2) continue;
        if (t.stride(i) < reach) value_error(std::string(name) + "'s rows overlap");
        reach = t.stride(i) * (t.size(i) - 1) + reach;
    }
}
// A contiguous result that shares no memory with an input that is read again after parts of the result are written.
void check_apart(const at::Tensor& out, const char* name, const at::Tensor& in, const char* of) {
    if (out.numel() == 0 || in.numel() == 0) return;
    int64_t reach = 1;
    for (int64_t i = 0; i < in.dim(); ++i) reach += (in.size(i) - 1) * in.stride(i);
    const char *o = static_cast<const char*>(out.data_ptr()), *p = static_cast<const char*>(in.data_ptr());
    if (o < p + reach * in.element_size() && p < o + out.nbytes()) value_error(std::string(name) + " overlaps " + of);
}
polykv_pages_seqs seqs_of(PyObject* table, PyObject* lens, int64_t A, int64_t layer, int64_t L, const Cache& c) {
    const at::Tensor& t = tensor(table, "block_table");
    if (t.dim() != 2) value_error("block_table must be [A][max_pages], got shape " + shape_text(t.sizes()));
    exactly(table, "block_table", {A, t.size(1)}, at::kInt, c);
    const at::Tensor& n = exactly(lens, "lens", {A}, at::kInt, c);
    if (layer < INT32_MIN || layer > INT32_MAX || A > INT32_MAX || L > INT32_MAX) value_error("layer is out of range");
    polykv_pages_seqs s;
    s.block_table = static_cast<const int32_t*>(t.data_ptr());
    s.lens = static_cast<const int32_t*>(n.data_ptr());
    s.max_pages = t.size(1);
    s.n_seqs = (int32_t)A;
    s.layer0 = (int32_t)layer;
    s.n_layers = (int32_t)L;
    return s;
}
const int32_t* selected_of(PyObject* o, int64_t L, int64_t A, const Cache& c, int64_t* n) {
    *n = -1;
    if (o == Py_None) return nullptr;
    const at::Tensor& t = four(o, "selected", "[L][A][H][n]");
    *n = t.size(3);
    exactly(o, "selected", {L, A, c.H, *n}, at::kInt, c);
    if (*n < 1) value_error("selected names no pages");   // its data pointer is null, which the C calls take for all pages
    return static_cast<const int32_t*>(t.data_ptr());
}
int64_t integer(PyObject* o) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw Failure{};
    return v;
}
double real(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw Failure{};
    return v;
}
int32_t heads_of(int64_t n) { return n > INT32_MAX ? INT32_MAX : (int32_t)n; }

// The cache's device current and its current stream, once all arguments are checked.
struct Here {
    c10::cuda::OptionalCUDAGuard guard;
    cudaStream_t stream = nullptr;
    explicit Here(const Owner& c) {
        if (!c.device.is_cuda()) value_error(std::string(c.name) + (c.plural ? " are on " : " is on ") + c.device.str() + ", not on a CUDA device");
        if (c10::cuda::current_device() != c.device.index()) guard.set_index(c.device.index());
        stream = c10::cuda::getCurrentCUDAStream(c.device.index()).stream();
    }
};
at::Tensor empty(c10::IntArrayRef shape, c10::ScalarType dtype, const Owner& c) {
    return at::detail::empty_cuda(shape, dtype, c.device, std::nullopt);
}
bool capturing(cudaStream_t st) {
    cudaStreamCaptureStatus s = cudaStreamCaptureStatusNone;
    return cudaStreamIsCapturing(st, &s) == cudaSuccess && s != cudaStreamCaptureStatusNone;
}
at::Tensor cleared(int64_t bytes, const Cache& c, cudaStream_t st) {
    at::Tensor t = empty({bytes}, at::kByte, c);
    const cudaError_t e = cudaMemsetAsync(t.data_ptr(), 0, bytes < 4096 ? bytes : 4096, st);
    if (e != cudaSuccess) {
        PyErr_Format(PyExc_RuntimeError, "clearing a workspace: %s", cudaGetErrorString(e));
        throw Failure{};
    }
    return t;
}
// A workspace whose arrival counts are zero. Calls on one stream are ordered and share one; a graph under capture
// gets its own, which it clears itself.
template <class Map, class Key>
at::Tensor workspace(Map& kept, const Key& key, int64_t need, const Cache& c, cudaStream_t st) {
    if (capturing(st)) return cleared(need, c, st);
    at::Tensor& t = kept[key];
    if (!t.defined() || t.numel() < need) t = cleared(need, c, st);
    return t;
}
at::Tensor given_workspace(PyObject* o, const Cache& c) {
    const at::Tensor& t = tensor(o, "workspace");
    if (t.device() != c.device || !t.is_contiguous()) value_error("workspace must be contiguous and on " + c.device.str());
    return t;
}

template <class F>
PyObject* guarded(F f) {
    try {
        return f();
    } catch (const Failure&) {
    } catch (...) {   // torch's own: out of memory and the like
        torch::translate_exception_to_python(std::current_exception());
    }
    return nullptr;
}
bool want_args(Py_ssize_t n, Py_ssize_t want) {
    if (n == want) return true;
    PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, n);
    return false;
}

// (PolyKVError)
PyObject* init(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (!want_args(n, 1)) return nullptr;
    Py_INCREF(a[0]);
    Py_XSETREF(g_error, a[0]);
    Py_RETURN_NONE;
}

// (handle, k_pages, rows): rows 1 for bf16, 0 for f16
PyObject* cache(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (!want_args(n, 3)) return nullptr;
    return guarded([&]() -> PyObject* {
        const at::Tensor& k = tensor(a[1], "k_pages");
        Cache* c = new Cache;
        c->handle = reinterpret_cast<polykv_pages*>(integer(a[0]));
        c->H = k.size(2);
        c->d = k.size(4);
        c->dtype = integer(a[2]) ? at::kBFloat16 : at::kHalf;
        c->device = k.device();
        return PyCapsule_New(c, "polykv.pages", cache_free);
    });
}

// (cache, k, v, block_table, lens, starts, q, q_out, turns, rotary_dim, interleaved, mscale, positions, pos_offset, layer)
PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
    if (!want_args(n_args, 15)) return nullptr;
    return guarded([&]() -> PyObject* {
        Cache& c = *cache_of(a[0]);
        const at::Tensor &k = four(a[1], "k", "[L][n][H][d]"), &v = four(a[2], "v", "[L][n][H][d]");
        const at::Tensor& lens = tensor(a[4], "lens");
        const int64_t L = k.size(0), n = k.size(1), A = lens.dim() == 1 ? lens.size(0) : -1;
        polykv_pages_append_args x = {};
        x.k_strides = rows_of(k, "k", {L, n, c.H, c.d}, c);
        x.v_strides = rows_of(v, "v", {L, n, c.H, c.d}, c);
        check_no_grad(k, "k");
        check_no_grad(v, "v");
        x.k = k.data_ptr();
        x.v = v.data_ptr();
        x.n_rows = n;
        const polykv_pages_seqs s = seqs_of(a[3], a[4], A, integer(a[14]), L, c);
        if (a[5] != Py_None)
            x.starts = static_cast<const int32_t*>(exactly(a[5], "starts", {A + 1}, at::kInt, c).data_ptr());
        if (a[12] != Py_None)
            x.positions = static_cast<const int64_t*>(exactly(a[12], "positions", {n}, at::kLong, c).data_ptr());
        x.pos_offset = integer(a[13]);
        if (a[8] != Py_None) {
            const at::Tensor& turns = tensor(a[8], "rope");
            check_kind(turns, "rope", at::kLong, c);
            x.turns = static_cast<const uint64_t*>(turns.data_ptr());
            x.rotary_dim = (int32_t)integer(a[9]);
            x.interleaved = a[10] == Py_True;
            x.mscale = (float)real(a[11]);
        }
        at::Tensor made;
        if (a[6] != Py_None) {
            const at::Tensor& q = four(a[6], "q", "[L][n][Hq][d]");
            const int64_t shape[4] = {L, n, q.size(2), c.d};
            x.q_strides = rows_of(q, "q", shape, c);
            check_no_grad(q, "q");
            x.q = q.data_ptr();
            x.n_q_heads = heads_of(q.size(2));
            if (a[7] != Py_None) {
                const at::Tensor& out = four(a[7], "q_out", "[L][n][Hq][d]");
                x.q_out_strides = rows_of(out, "q_out", shape, c);
                check_places(out, "q_out");
                check_no_grad(out, "q_out");
                x.q_out = out.data_ptr();
            }
        } else if (a[7] != Py_None) {
            value_error("q_out without q");
        }
        Here here(c);
        if (a[6] != Py_None && a[7] == Py_None) {
            const int64_t hq = tensor(a[6], "q").size(2);
            made = empty({L, n, hq, c.d}, c.dtype, c);
            x.q_out = made.data_ptr();
            x.q_out_strides = {n * hq * c.d, hq * c.d, c.d};
        }
        check(polykv_pages_append(c.handle, &s, &x, here.stream));
        if (made.defined()) return THPVariable_Wrap(made);
        PyObject* r = a[6] != Py_None ? a[7] : Py_None;
        Py_INCREF(r);
        return r;
    });
}

// (cache, q, block_table, lens, selected, out, out_kind, softmax_scale, layer, workspace, window, sinks); out_kind: 0 fp32,
// 1 the cache's type, -1 whatever `out` has
PyObject* attend(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
    if (!want_args(n_args, 12)) return nullptr;
    return guarded([&]() -> PyObject* {
        Cache& c = *cache_of(a[0]);
        const at::Tensor& q = four(a[1], "q", "[L][A][Hq][d]");
        const int64_t L = q.size(0), A = q.size(1), Hq = q.size(2);
        const int64_t shape[4] = {L, A, Hq, c.d};
        const polykv_row_strides qs = rows_of(q, "q", shape, c);
        check_no_grad(q, "q");
        const polykv_pages_seqs s = seqs_of(a[2], a[3], A, integer(a[8]), L, c);
        int64_t n_sel;
        const int32_t* sel = selected_of(a[4], L, A, c, &n_sel);
        const int64_t kind = integer(a[6]);
        at::Tensor out;
        bool f32 = kind != 1;
        if (a[5] != Py_None) {
            const at::Tensor& t = tensor(a[5], "out");
            if (kind < 0) {
                f32 = t.scalar_type() == at::kFloat;
                if (!f32 && t.scalar_type() != c.dtype)
                    value_error(std::string("out must be Float or ") + c10::toString(c.dtype) + ", got " + c10::toString(t.scalar_type()));
            }
            out = exactly(a[5], "out", shape, f32 ? at::kFloat : c.dtype, c);
            check_no_grad(out, "out");
        }
        const float scale = (float)real(a[7]);
        const int64_t window = integer(a[10]), sinks = integer(a[11]);
        if (sel && (window != 0 || sinks != 0)) value_error("selected and a window exclude each other");
        Here here(c);
        if (!out.defined()) out = empty(shape, f32 ? at::kFloat : c.dtype, c);
        at::Tensor ws;
        if (a[9] != Py_None) {
            ws = given_workspace(a[9], c);
        } else {
            size_t need = 0;
            check(polykv_pages_attend_workspace_size(c.handle, heads_of(Hq), &need));
            ws = workspace(c.attend_ws, std::make_pair(here.stream, (int)Hq), (int64_t)need, c, here.stream);
        }
        if (window != 0 || sinks != 0)
            check(polykv_pages_attend_window(c.handle, &s, q.data_ptr(), &qs, heads_of(Hq), window, sinks, scale, out.data_ptr(), f32,
                                             ws.data_ptr(), ws.nbytes(), here.stream));
        else
            check(polykv_pages_attend(c.handle, &s, q.data_ptr(), &qs, heads_of(Hq), sel, n_sel, scale, out.data_ptr(), f32,
                                      ws.data_ptr(), ws.nbytes(), here.stream));
        return THPVariable_Wrap(out);
    });
}

// (cache, q, block_table, lens, starts, window, sinks, out, softmax_scale, layer, workspace)
PyObject* attend_rows(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
    if (!want_args(n_args, 11)) return nullptr;
    return guarded([&]() -> PyObject* {
        Cache& c = *cache_of(a[0]);
        const at::Tensor &q = four(a[1], "q", "[L][n][Hq][d]"), &lens = tensor(a[3], "lens");
        const int64_t L = q.size(0), n = q.size(1), Hq = q.size(2), A = lens.dim() == 1 ? lens.size(0) : -1;
        const int64_t shape[4] = {L, n, Hq, c.d};
        const polykv_row_strides qs = rows_of(q, "q", shape, c);
        check_no_grad(q, "q");
        const polykv_pages_seqs s = seqs_of(a[2], a[3], A, integer(a[9]), L, c);
        const int32_t* starts = static_cast<const int32_t*>(exactly(a[4], "starts", {A + 1}, at::kInt, c).data_ptr());
        const int64_t window = integer(a[5]), sinks = integer(a[6]);
        at::Tensor out, ws;
        if (a[7] != Py_None) {
            out = exactly(a[7], "out", shape, c.dtype, c);
            check_no_grad(out, "out");
            check_apart(out, "out", q, "q");
        }
        const float scale = (float)real(a[8]);
        Here here(c);
        if (!out.defined()) out = empty(shape, c.dtype, c);
        if (a[10] != Py_None) {
            ws = given_workspace(a[10], c);
        } else {
            size_t need = 0;
            check(polykv_pages_attend_rows_workspace_size(c.handle, &s, heads_of(Hq), n, window, sinks, &need));
            if (need) ws = workspace(c.rows_ws, here.stream, (int64_t)need, c, here.stream);
        }
        check(polykv_pages_attend_rows(c.handle, &s, q.data_ptr(), &qs, heads_of(Hq), n, starts, window, sinks, scale, out.data_ptr(),
                                       ws.defined() ? ws.data_ptr() : nullptr, ws.defined() ? ws.nbytes() : 0, here.stream));
        return THPVariable_Wrap(out);
    });
}

// (cache, block_table, lens, starts, n_rows, layers, k, v, layer)
PyObject* gather(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
    if (!want_args(n_args, 9)) return nullptr;
    return guarded([&]() -> PyObject* {
        Cache& c = *cache_of(a[0]);
        const at::Tensor& lens = tensor(a[2], "lens");
        const int64_t A = lens.dim() == 1 ? lens.size(0) : -1, n = integer(a[4]), L = integer(a[5]);
        const polykv_pages_seqs s = seqs_of(a[1], a[2], A, integer(a[8]), L, c);
        const int32_t* starts = static_cast<const int32_t*>(exactly(a[3], "starts", {A + 1}, at::kInt, c).data_ptr());
        if (n < 0 || n > INT32_MAX) value_error("n_rows must be between 0 and 2^31 - 1");
        const int64_t shape[4] = {L, n, c.H, c.d};
        at::Tensor k, v;
        if (a[6] != Py_None) k = exactly(a[6], "k", shape, c.dtype, c);
        if (a[7] != Py_None) v = exactly(a[7], "v", shape, c.dtype, c);
        if (k.defined()) check_no_grad(k, "k");
        if (v.defined()) check_no_grad(v, "v");
        Here here(c);
        if (L < 1) value_error("layers must be at least 1");
        if (!k.defined()) k = empty(shape, c.dtype, c);
        if (!v.defined()) v = empty(shape, c.dtype, c);
        check(polykv_pages_gather(c.handle, &s, n, starts, k.data_ptr(), v.data_ptr(), here.stream));
        PyObject* pk = THPVariable_Wrap(k);
        PyObject* pv = THPVariable_Wrap(v);
        return Py_BuildValue("(NN)", pk, pv);
    });
}

// (block_table, lens, first, ring, counts, arrivals, status, page_tokens, window, sinks)
PyObject* tables(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (!want_args(n, 10)) return nullptr;
    return guarded([&]() -> PyObject* {
        const at::Tensor& table = tensor(a[0], "block_table");
        if (table.dim() != 2) value_error("block_table must be [A][max_pages], got shape " + shape_text(table.sizes()));
        Owner o;
        o.name = "the tables";
        o.plural = true;
        o.device = table.device();
        const int64_t A = table.size(0), P = tensor(a[3], "ring").numel();
        if (A > INT32_MAX) value_error("n_seqs is out of range");
        Tables t;
        static_cast<Owner&>(t) = o;
        t.t.block_table = static_cast<int32_t*>(exactly(a[0], "block_table", {A, table.size(1)}, at::kInt, o).data_ptr());
        t.t.lens = static_cast<int32_t*>(exactly(a[1], "lens", {A}, at::kInt, o).data_ptr());
        t.t.first = static_cast<int32_t*>(exactly(a[2], "first", {A}, at::kInt, o).data_ptr());
        t.t.ring = static_cast<int32_t*>(exactly(a[3], "ring", {P}, at::kInt, o).data_ptr());
        t.t.counts = static_cast<int64_t*>(exactly(a[4], "counts", {2}, at::kLong, o).data_ptr());
        t.t.arrivals = static_cast<uint32_t*>(exactly(a[5], "arrivals", {1}, at::kInt, o).data_ptr());
        t.t.status = static_cast<uint32_t*>(exactly(a[6], "status", {1}, at::kInt, o).data_ptr());
        t.t.max_pages = table.size(1);
        t.t.n_pages = P;
        t.t.n_seqs = (int32_t)A;
        const int64_t page = integer(a[7]);
        t.t.page_tokens = page < 0 || page > INT32_MAX ? 0 : (int32_t)page;
        t.t.window = integer(a[8]);
        t.t.sinks = integer(a[9]);
        for (int i = 0; i < 7; ++i) t.kept.push_back(tensor(a[i], "tensor"));
        return PyCapsule_New(new Tables(t), "polykv.tables", tables_free);
    });
}

// (tables, new_tokens, n_rows) -> (starts, before, after, slots, positions)
PyObject* tables_plan(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
    if (!want_args(n_args, 3)) return nullptr;
    return guarded([&]() -> PyObject* {
        const Tables& t = *tables_of(a[0]);
        const int64_t A = t.t.n_seqs, n = integer(a[2]);
        const at::Tensor& fresh = exactly(a[1], "new", {A}, at::kInt, t);
        if (n < 0 || n > INT32_MAX) value_error("n_rows must be between 0 and 2^31 - 1");
        Here here(t);
        at::Tensor starts = empty({A + 1}, at::kInt, t), before = empty({A}, at::kInt, t), after = empty({A}, at::kInt, t),
                   slots = empty({n}, at::kLong, t), positions = empty({n}, at::kLong, t);
        check(polykv_tables_plan(&t.t, static_cast<const int32_t*>(fresh.data_ptr()), n, static_cast<int32_t*>(starts.data_ptr()),
                                 static_cast<int32_t*>(before.data_ptr()), static_cast<int32_t*>(after.data_ptr()),
                                 static_cast<int64_t*>(slots.data_ptr()), static_cast<int64_t*>(positions.data_ptr()), here.stream));
        return Py_BuildValue("(NNNNN)", THPVariable_Wrap(starts), THPVariable_Wrap(before), THPVariable_Wrap(after),
                             THPVariable_Wrap(slots), THPVariable_Wrap(positions));
    });
}

// (tables, keep)
PyObject* tables_cut(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
    if (!want_args(n_args, 2)) return nullptr;
    return guarded([&]() -> PyObject* {
        const Tables& t = *tables_of(a[0]);
        const at::Tensor& keep = exactly(a[1], "keep", {t.t.n_seqs}, at::kInt, t);
        Here here(t);
        check(polykv_tables_cut(&t.t, static_cast<const int32_t*>(keep.data_ptr()), here.stream));
        Py_RETURN_NONE;
    });
}

// (tables)
PyObject* tables_status(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
    if (!want_args(n_args, 1)) return nullptr;
    return guarded([&]() -> PyObject* {
        const Tables& t = *tables_of(a[0]);
        Here here(t);
        uint32_t flags = 0;
        polykv_status st;
        Py_BEGIN_ALLOW_THREADS;
        st = polykv_tables_status(&t.t, here.stream, &flags);
        Py_END_ALLOW_THREADS;
        check(st);
        return PyLong_FromUnsignedLong(flags);
    });
}

// (cache, q, block_table, lens, n_selected, keep_first, keep_last, out, layer, workspace)
PyObject* select(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
    if (!want_args(n_args, 10)) return nullptr;
    return guarded([&]() -> PyObject* {
        Cache& c = *cache_of(a[0]);
        const at::Tensor& q = four(a[1], "q", "[L][A][Hq][d]");
        const int64_t L = q.size(0), A = q.size(1), Hq = q.size(2), n = integer(a[4]);
        const polykv_row_strides qs = rows_of(q, "q", {L, A, Hq, c.d}, c);
        const polykv_pages_seqs s = seqs_of(a[2], a[3], A, integer(a[8]), L, c);
        const int64_t first = integer(a[5]), last = integer(a[6]);
        const int64_t shape[4] = {L, A, c.H, n};
        at::Tensor out;
        if (a[7] != Py_None) out = exactly(a[7], "out", shape, at::kInt, c);
        Here here(c);
        at::Tensor ws;
        if (a[9] != Py_None) {
            ws = given_workspace(a[9], c);
        } else {
            size_t need = 0;
            check(polykv_pages_select_workspace_size(c.handle, &s, &need));
            if (need) ws = workspace(c.select_ws, here.stream, (int64_t)need, c, here.stream);
        }
        if (!out.defined()) {
            if (n < 1 || n > (1 << 20)) value_error("n_selected must be between 1 and 2^20");
            out = empty(shape, at::kInt, c);
        }
        check(polykv_pages_select(c.handle, &s, q.data_ptr(), &qs, heads_of(Hq), n, first, last,
                                  static_cast<int32_t*>(out.data_ptr()), ws.defined() ? ws.data_ptr() : nullptr,
                                  ws.defined() ? ws.nbytes() : 0, here.stream));
        return THPVariable_Wrap(out);
    });
}

// (cache, pool handle, pool buffer, pool layers, pool head_dim, q, n_ctx, block_table, lens, selected, out, softmax_scale, workspace)
PyObject* attend_with_pool(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
    if (!want_args(n_args, 13)) return nullptr;
    return guarded([&]() -> PyObject* {
        Cache& c = *cache_of(a[0]);
        const polykv_pool* pool = reinterpret_cast<const polykv_pool*>(integer(a[1]));
        const at::Tensor &buf = tensor(a[2], "pool"), &q = four(a[5], "q", "[L][A][Hq][d]");
        const int64_t A = q.size(1), Hq = q.size(2), L = integer(a[3]);
        const int64_t shape[4] = {L, A, Hq, integer(a[4])};
        check_shape(q, "q", shape);
        if (q.element_size() != 2 || (q.is_floating_point() && q.scalar_type() != c.dtype))
            value_error(std::string("q must be ") + c10::toString(c.dtype) + " or its bits in 2-byte integers, got " +
                        c10::toString(q.scalar_type()));
        if (q.device() != c.device) value_error("q is on " + q.device().str() + ", the cache on " + c.device.str());
        if (!q.is_contiguous()) value_error("q must be contiguous");
        check_no_grad(q, "q");
        if (buf.device() != c.device) value_error("the pool is on " + buf.device().str() + ", the cache on " + c.device.str());
        const polykv_pages_seqs s = seqs_of(a[7], a[8], A, 0, L, c);
        int64_t n_sel;
        const int32_t* sel = selected_of(a[9], L, A, c, &n_sel);
        const int64_t n_ctx = integer(a[6]);
        const float scale = (float)real(a[11]);
        at::Tensor out, ws;
        if (a[10] != Py_None) {
            out = exactly(a[10], "out", shape, at::kFloat, c);
            check_no_grad(out, "out");
        }
        Here here(c);
        if (a[12] != Py_None) {
            ws = given_workspace(a[12], c);
        } else {
            size_t need = 0;
            check(polykv_attend_pages_workspace_size(pool, c.handle, &s, heads_of(Hq), n_ctx, &need));
            ws = workspace(c.joint_ws, here.stream, (int64_t)need, c, here.stream);
        }
        if (!out.defined()) out = empty(shape, at::kFloat, c);
        check(polykv_attend_pages(pool, c.handle, &s, q.data_ptr(), static_cast<float*>(out.data_ptr()), heads_of(Hq), n_ctx,
                                  scale, sel, n_sel, ws.data_ptr(), ws.nbytes(), here.stream));
        return THPVariable_Wrap(out);
    });
}

// (cache)
PyObject* status(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
    if (!want_args(n_args, 1)) return nullptr;
    return guarded([&]() -> PyObject* {
        Cache& c = *cache_of(a[0]);
        Here here(c);
        uint32_t flags = 0;
        polykv_status st;
        Py_BEGIN_ALLOW_THREADS;
        st = polykv_pages_status(c.handle, here.stream, &flags);
        Py_END_ALLOW_THREADS;
        if (st == POLYKV_E_TIMEOUT) c.rows_ws.clear();   // a call that gave up may have left arrivals uncounted
        check(st);
        return PyLong_FromUnsignedLong(flags);
    });
}

PyMethodDef methods[] = {
    {"init", (PyCFunction)(void (*)(void))init, METH_FASTCALL, nullptr},
    {"cache", (PyCFunction)(void (*)(void))cache, METH_FASTCALL, nullptr},
    {"append", (PyCFunction)(void (*)(void))append, METH_FASTCALL, nullptr},
    {"attend", (PyCFunction)(void (*)(void))attend, METH_FASTCALL, nullptr},
    {"attend_rows", (PyCFunction)(void (*)(void))attend_rows, METH_FASTCALL, nullptr},
    {"gather", (PyCFunction)(void (*)(void))gather, METH_FASTCALL, nullptr},
    {"tables", (PyCFunction)(void (*)(void))tables, METH_FASTCALL, nullptr},
    {"tables_plan", (PyCFunction)(void (*)(void))tables_plan, METH_FASTCALL, nullptr},
    {"tables_cut", (PyCFunction)(void (*)(void))tables_cut, METH_FASTCALL, nullptr},
    {"tables_status", (PyCFunction)(void (*)(void))tables_status, METH_FASTCALL, nullptr},
    {"select", (PyCFunction)(void (*)(void))select, METH_FASTCALL, nullptr},
    {"attend_with_pool", (PyCFunction)(void (*)(void))attend_with_pool, METH_FASTCALL, nullptr},
    {"status", (PyCFunction)(void (*)(void))status, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_pages", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__pages(void) { return PyModule_Create(&module); }
