// fa_binding.cpp -- the Python binding's marshalling of the calls around
// attention (norm and rotation, paged append, paged attention): checks torch
// tensors, allocates what the caller left out, and calls the C ABI of fa.h on
// the tensors' device and torch's current stream there.
//
// A server makes these calls once per layer and token, when a kernel takes a
// few microseconds: checked attribute by attribute and passed through ctypes
// the append of one token took 23 us of host time, from here it takes 8.
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>
#include <string>

#include "fa.h"

namespace {

PyObject* g_status_error = nullptr;  // raised as error(status, where)

[[noreturn]] void fail(PyObject* type, const char* name, const std::string& what) {
    PyErr_Format(type, "%s: %s", name, what.c_str());
    throw python_error();
}

void check(fa_status st, const char* where) {
    if (st == FA_OK) return;
    PyObject* e = PyObject_CallFunction(g_status_error, "is", static_cast<int>(st), where);
    if (e) {
        PyErr_SetObject(g_status_error, e);
        Py_DECREF(e);
    }
    throw python_error();
}

std::string text(at::IntArrayRef sizes) {
    std::string s = "(";
    for (size_t i = 0; i < sizes.size(); ++i) s += (i ? ", " : "") + std::to_string(sizes[i]);
    return s + (sizes.size() == 1 ? ",)" : ")");
}

const at::Tensor& tensor(PyObject* o, const char* name) {
    if (!THPVariable_Check(o)) fail(PyExc_TypeError, name, "expected a tensor");
    return THPVariable_Unpack(o);
}

long long integer(PyObject* o, const char* name) {
    const long long x = PyLong_AsLongLong(o);
    if (x == -1 && PyErr_Occurred()) throw python_error();
    if (x < -0x7fffffffll || x > 0x7fffffffll) fail(PyExc_ValueError, name, "out of range");
    return x;
}

double number(PyObject* o) {
    const double x = PyFloat_AsDouble(o);
    if (x == -1.0 && PyErr_Occurred()) throw python_error();
    return x;
}

int truth(PyObject* o) {
    const int x = PyObject_IsTrue(o);
    if (x < 0) throw python_error();
    return x;
}

// Sizes are 32-bit in the C ABI.
int size_of(const at::Tensor& t, int dim, const char* name) {
    const int64_t n = t.size(dim);
    if (n > 0x7fffffffll) fail(PyExc_ValueError, name, "a dimension exceeds 2^31 - 1");
    return static_cast<int>(n);
}

at::Device cuda_device(const at::Tensor& t, const char* name) {
    if (!t.is_cuda()) fail(PyExc_ValueError, name, "expected a CUDA tensor");
    return t.device();
}

void same(const at::Tensor& t, const char* name, at::IntArrayRef shape, at::ScalarType type,
          at::Device dev) {
    if (t.scalar_type() != type)
        fail(PyExc_TypeError, name,
             std::string("expected ") + c10::toString(type) + ", got " +
                 c10::toString(t.scalar_type()));
    if (t.device() != dev)
        fail(PyExc_ValueError, name, "expected device " + dev.str() + ", got " + t.device().str());
    if (t.sizes() != shape)
        fail(PyExc_ValueError, name, "expected shape " + text(shape) + ", got " + text(t.sizes()));
}

// Data of a contiguous tensor of exactly this shape and type.
void* exact(const at::Tensor& t, const char* name, at::IntArrayRef shape, at::ScalarType type,
            at::Device dev) {
    same(t, name, shape, type, dev);
    if (!t.is_contiguous()) fail(PyExc_ValueError, name, "must be contiguous");
    return t.data_ptr();
}

// Data of a bf16 tensor whose rows are contiguous, and its other strides (a
// dimension of one element gets stride 0).
void* rows(const at::Tensor& t, const char* name, at::IntArrayRef shape, at::Device dev,
           long long* strides) {
    same(t, name, shape, at::kBFloat16, dev);
    const int last = static_cast<int>(shape.size()) - 1;
    if (t.stride(last) != 1)
        fail(PyExc_ValueError, name, "the last dimension must be contiguous");
    for (int i = 0; i < last; ++i) strides[i] = shape[i] > 1 ? t.stride(i) : 0;
    return t.data_ptr();
}

at::Tensor empty(at::IntArrayRef shape, at::ScalarType type, at::Device dev) {
    return at::detail::empty_cuda(shape, type, dev, std::nullopt);
}

// The caller's output, or a new one.
at::Tensor output(PyObject* o, const char* name, at::IntArrayRef shape, at::ScalarType type,
                  at::Device dev) {
    if (o == Py_None) return empty(shape, type, dev);
    const at::Tensor& t = tensor(o, name);
    exact(t, name, shape, type, dev);
    return t;
}

void* workspace_of(const at::Tensor& t, at::Device dev, size_t* bytes) {
    if (t.device() != dev)
        fail(PyExc_ValueError, "workspace",
             "expected device " + dev.str() + ", got " + t.device().str());
    if (!t.is_contiguous()) fail(PyExc_ValueError, "workspace", "must be contiguous");
    *bytes = static_cast<size_t>(t.numel()) * t.element_size();
    return t.data_ptr();
}

// The device made current for a call, and torch's current stream on it.
struct Place {
    c10::cuda::CUDAGuard guard;
    void* stream;
    explicit Place(at::Device dev)
        : guard(dev.index()), stream(c10::cuda::getCurrentCUDAStream(dev.index()).stream()) {}
};

struct NormRope {
    void *wq = nullptr, *wk = nullptr;
    int w_f32 = 0;
    float* table = nullptr;
    long long rows = 0;
    int width = 0;

    NormRope(PyObject* q_weight, PyObject* k_weight, PyObject* rope, int64_t d, at::Device dev) {
        if ((q_weight == Py_None) != (k_weight == Py_None))
            fail(PyExc_ValueError, "q_weight and k_weight", "give both or neither");
        if (q_weight != Py_None) {
            const at::Tensor& q = tensor(q_weight, "q_weight");
            const at::ScalarType type = q.scalar_type();
            if (type != at::kBFloat16 && type != at::kFloat)
                fail(PyExc_TypeError, "q_weight",
                     std::string("expected BFloat16 or Float, got ") + c10::toString(type));
            wq = exact(q, "q_weight", {d}, type, dev);
            wk = exact(tensor(k_weight, "k_weight"), "k_weight", {d}, type, dev);
            w_f32 = type == at::kFloat;
        }
        if (rope == Py_None) return;
        const at::Tensor& t = tensor(rope, "rope");
        if (t.dim() != 3 || t.size(2) != 2)
            fail(PyExc_ValueError, "rope", "expected a [positions, rope_dim / 2, 2] table");
        // Its pointer would be null, which the C ABI takes for no rotation.
        if (t.numel() == 0) fail(PyExc_ValueError, "rope", "the table is empty");
        table = static_cast<float*>(exact(t, "rope", t.sizes(), at::kFloat, dev));
        rows = t.size(0);
        width = static_cast<int>(std::min<int64_t>(2 * t.size(1), 1 << 20));
    }
};

PyObject* wrap(const at::Tensor& t) {
    if (!t.defined()) Py_RETURN_NONE;
    return THPVariable_Wrap(t);
}

PyObject* tuple_of(std::initializer_list<at::Tensor> ts) {
    PyObject* out = PyTuple_New(static_cast<Py_ssize_t>(ts.size()));
    if (!out) throw python_error();
    Py_ssize_t i = 0;
    for (const at::Tensor& t : ts) {
        PyObject* x = wrap(t);
        if (!x) {
            Py_DECREF(out);
            throw python_error();
        }
        PyTuple_SET_ITEM(out, i++, x);
    }
    return out;
}

void arity(Py_ssize_t n, Py_ssize_t want) {
    if (n == want) return;
    PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, n);
    throw python_error();
}

// q, k, v, q_weight, k_weight, eps, rope, positions, interleaved, q_out, k_out, v_out
PyObject* qk_norm_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    arity(n, 12);
    const at::Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k");
    if (q.dim() != 4 || k.dim() != 4)
        fail(PyExc_ValueError, "q, k", "expected [B, N, H, d] tensors");
    const at::Device dev = cuda_device(q, "q");
    const int B = size_of(q, 0, "q"), N = size_of(q, 1, "q"), Hq = size_of(q, 2, "q"),
              d = size_of(q, 3, "q"), Hkv = size_of(k, 2, "k");
    long long strides[9] = {};
    void* qp = rows(q, "q", {B, N, Hq, d}, dev, strides);
    void* kp = rows(k, "k", {B, N, Hkv, d}, dev, strides + 3);
    void* vp = nullptr;
    if (a[2] != Py_None)
        vp = rows(tensor(a[2], "v"), "v", {B, N, Hkv, d}, dev, strides + 6);
    else if (a[11] != Py_None)
        fail(PyExc_ValueError, "v_out", "given without v");
    const NormRope nr(a[3], a[4], a[6], d, dev);
    const int* pos = nullptr;
    if (a[7] != Py_None)
        pos = static_cast<int*>(
            exact(tensor(a[7], "positions"), "positions", {B, N}, at::kInt, dev));
    const Place place(dev);
    const at::Tensor qo = output(a[9], "q_out", {B, Hq, N, d}, at::kBFloat16, dev);
    const at::Tensor ko = output(a[10], "k_out", {B, Hkv, N, d}, at::kBFloat16, dev);
    at::Tensor vo;
    if (a[2] != Py_None) vo = output(a[11], "v_out", {B, Hkv, N, d}, at::kBFloat16, dev);
    check(fa_qk_norm_rope(qp, kp, vp, strides, nr.wq, nr.wk, nr.w_f32,
                          static_cast<float>(number(a[5])), nr.table, nr.rows, nr.width,
                          truth(a[8]), pos, qo.data_ptr(), ko.data_ptr(),
                          vo.defined() ? vo.data_ptr() : nullptr, B, N, Hq, Hkv, d, place.stream),
          "fa_qk_norm_rope");
    return tuple_of({qo, ko, vo});
    END_HANDLE_TH_ERRORS
}

// dq_out, dk_out, dv_out, q, k, q_weight, k_weight, eps, rope, positions, interleaved, dq, dk, dv,
// workspace
PyObject* qk_norm_rope_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    arity(n, 15);
    const at::Tensor &gq = tensor(a[0], "dq_out"), &gk = tensor(a[1], "dk_out");
    if (gq.dim() != 4 || gk.dim() != 4)
        fail(PyExc_ValueError, "dq_out, dk_out", "expected [B, H, N, d] gradients");
    const at::Device dev = cuda_device(gq, "dq_out");
    const int B = size_of(gq, 0, "dq_out"), Hq = size_of(gq, 1, "dq_out"),
              N = size_of(gq, 2, "dq_out"), d = size_of(gq, 3, "dq_out"),
              Hkv = size_of(gk, 1, "dk_out");
    void* gqp = exact(gq, "dq_out", {B, Hq, N, d}, at::kBFloat16, dev);
    void* gkp = exact(gk, "dk_out", {B, Hkv, N, d}, at::kBFloat16, dev);
    void* gvp = nullptr;
    if (a[2] != Py_None)
        gvp = exact(tensor(a[2], "dv_out"), "dv_out", {B, Hkv, N, d}, at::kBFloat16, dev);
    else if (a[13] != Py_None)
        fail(PyExc_ValueError, "dv", "given without dv_out");
    const NormRope nr(a[5], a[6], a[8], d, dev);
    long long strides[6] = {}, grads[9] = {};
    void *qp = nullptr, *kp = nullptr;
    if (nr.wq) {
        if (a[3] == Py_None || a[4] == Py_None)
            fail(PyExc_ValueError, "q and k", "needed for the gradients of a norm");
        qp = rows(tensor(a[3], "q"), "q", {B, N, Hq, d}, dev, strides);
        kp = rows(tensor(a[4], "k"), "k", {B, N, Hkv, d}, dev, strides + 3);
    }
    const int* pos = nullptr;
    if (a[9] != Py_None)
        pos = static_cast<int*>(
            exact(tensor(a[9], "positions"), "positions", {B, N}, at::kInt, dev));
    const Place place(dev);
    auto grad = [&](PyObject* o, const char* name, int H, long long* st) {
        at::Tensor t = o == Py_None ? empty({B, N, H, d}, at::kBFloat16, dev) : tensor(o, name);
        rows(t, name, {B, N, H, d}, dev, st);
        return t;
    };
    const at::Tensor dq = grad(a[11], "dq", Hq, grads), dk = grad(a[12], "dk", Hkv, grads + 3);
    at::Tensor dv, dwq, dwk, ws;
    if (gvp) dv = grad(a[13], "dv", Hkv, grads + 6);
    size_t ws_bytes = 0;
    void* wsp = nullptr;
    if (a[14] != Py_None) ws = tensor(a[14], "workspace");
    if (nr.wq) {
        dwq = empty({d}, at::kFloat, dev);
        dwk = empty({d}, at::kFloat, dev);
        if (!ws.defined())
            ws = empty({static_cast<int64_t>(fa_qk_norm_rope_bwd_workspace_size(d))}, at::kByte,
                       dev);
    }
    if (ws.defined()) wsp = workspace_of(ws, dev, &ws_bytes);
    check(fa_qk_norm_rope_bwd(
              gqp, gkp, gvp, qp, kp, strides, nr.wq, nr.wk, nr.w_f32,
              static_cast<float>(number(a[7])), nr.table, nr.rows, nr.width, truth(a[10]), pos,
              dq.data_ptr(), dk.data_ptr(), dv.defined() ? dv.data_ptr() : nullptr, grads,
              nr.wq ? dwq.data_ptr<float>() : nullptr, nr.wq ? dwk.data_ptr<float>() : nullptr, B,
              N, Hq, Hkv, d, wsp, ws_bytes, place.stream),
          "fa_qk_norm_rope_bwd");
    return tuple_of({dq, dk, dv, dwq, dwk});
    END_HANDLE_TH_ERRORS
}

// The paged cache that two calls take.
struct Cache {
    int pages, heads, page_size, S, max_pages;
    void *k, *v;
    int *table, *starts, *lens;

    Cache(PyObject* k_pages, PyObject* v_pages, PyObject* block_table, PyObject* seq_start,
          PyObject* len, const char* len_name, int64_t d, at::Device dev) {
        const at::Tensor &kt = tensor(k_pages, "k_pages"), &bt = tensor(block_table, "block_table");
        if (kt.dim() != 4)
            fail(PyExc_ValueError, "k_pages", "expected [num_pages, Hkv, page_size, d]");
        if (bt.dim() != 2) fail(PyExc_ValueError, "block_table", "expected [S, max_pages]");
        pages = size_of(kt, 0, "k_pages");
        heads = size_of(kt, 1, "k_pages");
        page_size = size_of(kt, 2, "k_pages");
        S = size_of(bt, 0, "block_table");
        max_pages = size_of(bt, 1, "block_table");
        k = exact(kt, "k_pages", {pages, heads, page_size, d}, at::kBFloat16, dev);
        v = exact(tensor(v_pages, "v_pages"), "v_pages", {pages, heads, page_size, d},
                  at::kBFloat16, dev);
        table = static_cast<int*>(exact(bt, "block_table", {S, max_pages}, at::kInt, dev));
        starts = static_cast<int*>(
            exact(tensor(seq_start, "seq_start"), "seq_start", {S + 1ll}, at::kInt, dev));
        lens = static_cast<int*>(exact(tensor(len, len_name), len_name, {S}, at::kInt, dev));
    }
};

// q, k, v, k_pages, v_pages, block_table, seq_start, cache_len, rope, pos_offset, q_weight,
// k_weight, eps, interleaved, q_out
PyObject* paged_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    arity(n, 15);
    const at::Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k");
    if (q.dim() != 3 || k.dim() != 3) fail(PyExc_ValueError, "q, k", "expected [T, H, d] tensors");
    const at::Device dev = cuda_device(q, "q");
    const int T = size_of(q, 0, "q"), Hq = size_of(q, 1, "q"), d = size_of(q, 2, "q"),
              Hkv = size_of(k, 1, "k");
    long long strides[6];
    void* qp = rows(q, "q", {T, Hq, d}, dev, strides);
    void* kp = rows(k, "k", {T, Hkv, d}, dev, strides + 2);
    void* vp = rows(tensor(a[2], "v"), "v", {T, Hkv, d}, dev, strides + 4);
    const Cache c(a[3], a[4], a[5], a[6], a[7], "cache_len", d, dev);
    if (c.heads != Hkv)
        fail(PyExc_ValueError, "k_pages",
             "expected " + std::to_string(Hkv) + " heads, got " + std::to_string(c.heads));
    const NormRope nr(a[10], a[11], a[8], d, dev);
    const Place place(dev);
    const at::Tensor out = output(a[14], "q_out", {T, Hq, d}, at::kBFloat16, dev);
    if (T > 0)
        check(fa_paged_append(qp, kp, vp, strides, nr.wq, nr.wk, nr.w_f32,
                              static_cast<float>(number(a[12])), nr.table, nr.rows, nr.width,
                              truth(a[13]), static_cast<int>(integer(a[9], "pos_offset")),
                              c.starts, c.lens, c.table, out.data_ptr(), c.k, c.v, c.S, T, Hq, Hkv,
                              d, c.page_size, c.pages, c.max_pages, place.stream),
              "fa_paged_append");
    return wrap(out);
    END_HANDLE_TH_ERRORS
}

// q, k_pages, v_pages, block_table, seq_start, kv_len, scale, prefix_pages, prefix_len, max_new,
// out, lse, workspace
PyObject* attention_paged(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    arity(n, 13);
    const at::Tensor& q = tensor(a[0], "q");
    if (q.dim() != 3) fail(PyExc_ValueError, "q", "expected [T, Hq, d]");
    const at::Device dev = cuda_device(q, "q");
    const int T = size_of(q, 0, "q"), Hq = size_of(q, 1, "q"), d = size_of(q, 2, "q");
    void* qp = exact(q, "q", {T, Hq, d}, at::kBFloat16, dev);
    const Cache c(a[1], a[2], a[3], a[4], a[5], "kv_len", d, dev);
    const int P = static_cast<int>(integer(a[8], "prefix_len"));
    const int* prefix = nullptr;
    if (P != 0) {
        if (a[7] == Py_None) fail(PyExc_ValueError, "prefix_len", "given without prefix_pages");
        const at::Tensor& t = tensor(a[7], "prefix_pages");
        prefix = static_cast<int*>(exact(t, "prefix_pages", {t.numel()}, at::kInt, dev));
        if (t.numel() * c.page_size < P)
            fail(PyExc_ValueError, "prefix_pages",
                 std::to_string(t.numel()) + " pages do not hold " + std::to_string(P) + " keys");
    }
    const int most = a[9] == Py_None ? T : static_cast<int>(integer(a[9], "max_new"));
    const Place place(dev);
    const at::Tensor out = output(a[10], "out", {T, Hq, d}, at::kBFloat16, dev);
    const at::Tensor lse = output(a[11], "lse", {T, Hq}, at::kFloat, dev);
    if (T > 0) {
        at::Tensor ws;
        if (a[12] != Py_None)
            ws = tensor(a[12], "workspace");
        else
            ws = empty({static_cast<int64_t>(fa_paged_workspace_size(
                           c.S, T, Hq, c.heads, d, c.page_size, c.max_pages, P, most))},
                       at::kByte, dev);
        size_t ws_bytes = 0;
        void* wsp = workspace_of(ws, dev, &ws_bytes);
        check(fa_fwd_paged(qp, c.k, c.v, c.table, c.starts, c.lens, prefix, P, out.data_ptr(),
                           lse.data_ptr<float>(), c.S, T, Hq, c.heads, d, c.page_size, c.pages,
                           c.max_pages, most, static_cast<float>(number(a[6])), wsp, ws_bytes,
                           place.stream),
              "fa_fwd_paged");
    }
    return tuple_of({out, lse});
    END_HANDLE_TH_ERRORS
}

// The class that a status other than FA_OK is raised as.
PyObject* set_status_error(PyObject*, PyObject* type) {
    Py_INCREF(type);
    Py_XSETREF(g_status_error, type);
    Py_RETURN_NONE;
}

#define FAST(f) \
    {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef g_methods[] = {FAST(qk_norm_rope), FAST(qk_norm_rope_backward), FAST(paged_append),
                           FAST(attention_paged),
                           {"set_status_error", set_status_error, METH_O, nullptr},
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_fa_binding", nullptr, -1, g_methods,
                        nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fa_binding() { return PyModule_Create(&g_module); }
