// attention_bind.cpp -- Python entry of the attention block (module _attention).
//
// Marshalling only, as in binding.py: torch tensors become pointers and strides,
// the current stream of the tensors' device becomes the HIP stream, and status
// codes become exceptions; the arithmetic is behind the C ABI of libw4a8.so.  It
// is compiled because a decode step's calls are small: with the same checks in
// Python, the head norms of one token took 16.5 us a call, of which the kernel
// runs 4.
//
// Every function takes all of its arguments by position; the signatures,
// defaults and documentation are in attention.py.
#include <Python.h>

#include <cmath>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/core/DeviceGuard.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "w4a8.h"

namespace {

struct Refused {};   // a Python exception is set

template <typename... A>
[[noreturn]] void refuse(PyObject* kind, const char* format, A... a) {
    PyErr_Format(kind, format, a...);
    throw Refused();
}

const char* type_name(at::ScalarType t) {
    switch (t) {
        case at::kByte: return "uint8";
        case at::kInt: return "int32";
        case at::kLong: return "int64";
        case at::kFloat: return "float32";
        case at::kHalf: return "float16";
        case at::kBFloat16: return "bfloat16";
        default: return "16-bit float";
    }
}

const at::Tensor& tensor(PyObject* o, const char* name) {
    if (!THPVariable_Check(o)) refuse(PyExc_TypeError, "%s must be a torch tensor", name);
    return THPVariable_Unpack(o);
}
const at::Tensor& tensor(PyObject* o, const char* name, at::ScalarType type, at::Device dev) {
    const at::Tensor& t = tensor(o, name);
    if (t.scalar_type() != type) refuse(PyExc_TypeError, "%s must be a %s tensor", name, type_name(type));
    if (t.device() != dev)
        refuse(PyExc_ValueError, "%s is on %s, expected %s", name, t.device().str().c_str(), dev.str().c_str());
    return t;
}
const at::Tensor& vector(PyObject* o, const char* name, at::ScalarType type, at::Device dev, int64_t n) {
    const at::Tensor& t = tensor(o, name, type, dev);
    if (t.dim() != 1 || t.size(0) != n || !t.is_contiguous())
        refuse(PyExc_ValueError, "%s must be a contiguous vector of %lld", name, (long long)n);
    return t;
}

bool known_dim(int64_t d) { return d == 64 || d == 128 || d == 256; }

// bf16 or fp16 [tokens, heads, head_dim] with contiguous heads
w4a8_float float_kind(const at::Tensor& t, const char* name) {
    if (t.scalar_type() == at::kBFloat16) return W4A8_BF16;
    if (t.scalar_type() == at::kHalf) return W4A8_FP16;
    refuse(PyExc_TypeError, "%s must be a bfloat16 or float16 tensor", name);
}
struct Heads {
    const uint16_t* p = nullptr;
    int64_t st = 0, sh = 0;
    int n = 0;
};
Heads heads(const at::Tensor& t, const char* name, int64_t tokens, int64_t count, int64_t d) {
    if (t.dim() != 3 || t.size(2) != d || (tokens >= 0 && t.size(0) != tokens) || (count >= 0 && t.size(1) != count))
        refuse(PyExc_ValueError, "%s must be [tokens, heads, head_dim = %lld]%s", name, (long long)d,
               tokens >= 0 || count >= 0 ? ", with the tokens and heads of the other tensors" : "");
    if (t.stride(2) != 1) refuse(PyExc_ValueError, "%s must have contiguous heads (unit last stride)", name);
    if (t.size(1) > 1024) refuse(PyExc_ValueError, "%s has more than 1024 heads", name);
    return {static_cast<const uint16_t*>(t.const_data_ptr()), t.stride(0), t.stride(1), (int)t.size(1)};
}

void on_gpu(const at::Tensor& t, const char* name) {
    if (!t.is_cuda()) refuse(PyExc_ValueError, "%s must be on a GPU", name);
}

// the caller's output, or a new contiguous tensor
at::Tensor output(PyObject* o, const char* name, const at::Tensor& like, at::IntArrayRef shape, bool gpu) {
    if (o == Py_None) {
        if (!gpu) refuse(PyExc_ValueError, "%s needs a GPU", name);
        return at::empty(shape, like.options());
    }
    const at::Tensor& t = tensor(o, name, like.scalar_type(), like.device());
    if (t.sizes() != shape || !t.is_contiguous())
        refuse(PyExc_ValueError, "%s must be a contiguous tensor of the input's shape", name);
    return t;
}

struct Turn {
    const float* table = nullptr;
    int64_t rows = 0;
    const int64_t* positions = nullptr;
    int rot = 0;
};
Turn turn(PyObject* table, PyObject* positions, at::Device dev, int64_t tokens, int64_t d) {
    Turn r;
    if (table == Py_None) return r;
    const at::Tensor& t = tensor(table, "cos_sin", at::kFloat, dev);
    if (t.dim() != 2 || !t.is_contiguous() || t.size(0) < 1)
        refuse(PyExc_ValueError, "cos_sin must be a contiguous [positions, rot] tensor");
    if (t.size(1) < 16 || t.size(1) % 16 || t.size(1) > d)
        refuse(PyExc_ValueError, "cos_sin: rot must be a multiple of 16 up to head_dim = %lld, got %lld", (long long)d,
               (long long)t.size(1));
    if (positions == Py_None) refuse(PyExc_ValueError, "a rotation needs positions");
    r.table = t.const_data_ptr<float>();
    r.rows = t.size(0);
    r.rot = (int)t.size(1);
    r.positions = vector(positions, "positions", at::kLong, dev, tokens).const_data_ptr<int64_t>();
    return r;
}
const float* weight(PyObject* o, const char* name, at::Device dev, int64_t d) {
    return o == Py_None ? nullptr : vector(o, name, at::kFloat, dev, d).const_data_ptr<float>();
}

double number(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw Refused();
    return v;
}
int64_t integer(PyObject* o, const char* name, int64_t lo, int64_t hi) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw Refused();
    if (v < lo || v > hi) refuse(PyExc_ValueError, "%s must be from %lld to %lld", name, (long long)lo, (long long)hi);
    return v;
}
bool truth(PyObject* o) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw Refused();
    return v != 0;
}
void arguments(Py_ssize_t got, Py_ssize_t want) {
    if (got != want) refuse(PyExc_TypeError, "%zd arguments, expected %zd", got, want);
}

void* stream(at::Device dev) { return (void*)c10::hip::getCurrentHIPStream(dev.index()).stream(); }

PyObject* hip_error;   // W4A8Error of binding.py, set by attention.py

void check(w4a8_status s, const char* what) {
    if (s == W4A8_OK) return;
    if (s == W4A8_ERR_HIP && hip_error) {
        PyObject* e = PyObject_CallFunction(hip_error, "is", (int)s, what);
        if (e) {
            PyErr_SetObject(hip_error, e);
            Py_DECREF(e);
        }
        throw Refused();
    }
    refuse(s == W4A8_ERR_HIP ? PyExc_RuntimeError : PyExc_ValueError, "%s: %s (status %d)", what, w4a8_status_string(s),
           (int)s);
}

// ---- the cache: its four tensors, held ----
struct Cache {
    at::Tensor t[4];
    at::Device dev;
    w4a8_kv_cache view() const {
        w4a8_kv_cache c;
        c.k_codes = static_cast<uint8_t*>(t[0].data_ptr());
        c.k_e8m0 = static_cast<uint8_t*>(t[1].data_ptr());
        c.v_codes = static_cast<uint8_t*>(t[2].data_ptr());
        c.v_e8m0 = static_cast<uint8_t*>(t[3].data_ptr());
        c.pages = t[0].size(0);
        c.kv_heads = (int)t[0].size(1);
        c.page = (int)t[0].size(2);
        c.head_dim = (int)(2 * t[0].size(3));
        return c;
    }
};
const char kCache[] = "w4a8_kv_cache";
void drop_cache(PyObject* o) { delete static_cast<Cache*>(PyCapsule_GetPointer(o, kCache)); }
const Cache& cache_of(PyObject* o) {
    if (!PyCapsule_IsValid(o, kCache)) refuse(PyExc_TypeError, "cache must be a KVCacheMXFP4");
    return *static_cast<const Cache*>(PyCapsule_GetPointer(o, kCache));
}

PyObject* make_cache(PyObject* const* a, Py_ssize_t n) {
    arguments(n, 4);
    static const char* names[4] = {"k_codes", "k_e8m0", "v_codes", "v_e8m0"};
    const at::Device dev = tensor(a[0], names[0]).device();
    const at::Tensor* t[4];
    for (int i = 0; i < 4; ++i) {
        t[i] = &tensor(a[i], names[i], at::kByte, dev);
        if (t[i]->dim() != 4 || !t[i]->is_contiguous())
            refuse(PyExc_ValueError, "%s must be a contiguous 4-D tensor", names[i]);
    }
    const int64_t pages = t[0]->size(0), hk = t[0]->size(1), page = t[0]->size(2), d = 2 * t[0]->size(3);
    if (!known_dim(d)) refuse(PyExc_ValueError, "head_dim must be 64, 128 or 256, got %lld", (long long)d);
    if (page < 16 || page > 1024 || (page & (page - 1)))
        refuse(PyExc_ValueError, "page must be a power of two from 16 to 1024, got %lld", (long long)page);
    if (pages < 1 || hk < 1 || hk > 1024)
        refuse(PyExc_ValueError, "a cache needs at least one page, and from 1 to 1024 heads");
    const int64_t codes[4] = {pages, hk, page, d / 2}, exps[4] = {pages, hk, d / 32, page};
    if (t[2]->sizes() != at::IntArrayRef(codes, 4) || t[1]->sizes() != at::IntArrayRef(exps, 4) ||
        t[3]->sizes() != at::IntArrayRef(exps, 4))
        refuse(PyExc_ValueError,
               "codes must be [pages, kv_heads, page, head_dim / 2], exponents [pages, kv_heads, head_dim / 32, page], "
               "the same for keys and values");
    return PyCapsule_New(new Cache{{*t[0], *t[1], *t[2], *t[3]}, dev}, kCache, drop_cache);
}

// q, k, cos_sin, positions, q_weight, k_weight, eps, interleaved, q_out, k_out
PyObject* norm_rope(PyObject* const* a, Py_ssize_t n) {
    arguments(n, 10);
    const bool has_q = a[0] != Py_None, has_k = a[1] != Py_None;
    const char* name = has_q ? "q" : "k";
    const at::Tensor& x = tensor(has_q ? a[0] : a[1], name);
    const w4a8_float type = float_kind(x, name);
    const at::Device dev = x.device();
    if (x.dim() != 3 || !known_dim(x.size(2)))
        refuse(PyExc_ValueError, "%s must be [tokens, heads, head_dim] with head_dim 64, 128 or 256", name);
    const int64_t tokens = x.size(0), d = x.size(2);
    const Turn t = turn(a[2], a[3], dev, tokens, d);
    Heads q, k;
    at::Tensor qo, ko;
    if (has_q) q = heads(x, "q", tokens, -1, d);
    if (has_k) k = heads(tensor(a[1], "k", x.scalar_type(), dev), "k", tokens, -1, d);
    const float *qw = weight(a[4], "q_weight", dev, d), *kw = weight(a[5], "k_weight", dev, d);
    const double eps = number(a[6]);
    const bool inter = truth(a[7]);
    on_gpu(x, name);
    if (has_q) qo = output(a[8], "q_out", x, x.sizes(), true);
    if (has_k) ko = output(a[9], "k_out", x, THPVariable_Unpack(a[1]).sizes(), true);
    const c10::DeviceGuard guard(dev);
    if (tokens && q.n + k.n)
        check(w4a8_qk_norm_rope(type, q.n ? q.p : nullptr, q.st, q.sh, q.n, k.n ? k.p : nullptr, k.st, k.sh, k.n, tokens,
                                (int)d, qw, kw, (float)eps, t.table, t.rows, t.positions, t.rot, inter,
                                q.n ? static_cast<uint16_t*>(qo.data_ptr()) : nullptr,
                                k.n ? static_cast<uint16_t*>(ko.data_ptr()) : nullptr, stream(dev)),
              "w4a8_qk_norm_rope");
    PyObject* r = PyTuple_New(2);
    PyTuple_SET_ITEM(r, 0, has_q ? THPVariable_Wrap(qo) : Py_NewRef(Py_None));
    PyTuple_SET_ITEM(r, 1, has_k ? THPVariable_Wrap(ko) : Py_NewRef(Py_None));
    return r;
}

// cache, k, v, slots, mode, cos_sin, positions, k_weight, eps, interleaved, q, q_weight, q_out
PyObject* append(PyObject* const* a, Py_ssize_t n) {
    arguments(n, 13);
    const Cache& c = cache_of(a[0]);
    const w4a8_kv_cache view = c.view();
    const int64_t d = view.head_dim;
    const at::Tensor& kt = tensor(a[1], "k");
    const w4a8_float type = float_kind(kt, "k");
    tensor(a[1], "k", kt.scalar_type(), c.dev);
    const int64_t tokens = kt.dim() ? kt.size(0) : 0;
    const Heads k = heads(kt, "k", tokens, view.kv_heads, d);
    const Heads v = heads(tensor(a[2], "v", kt.scalar_type(), c.dev), "v", tokens, view.kv_heads, d);
    const int64_t* slots = vector(a[3], "slots", at::kLong, c.dev, tokens).const_data_ptr<int64_t>();
    const w4a8_exp_mode mode = (w4a8_exp_mode)integer(a[4], "mode", W4A8_EXP_OCP, W4A8_EXP_NOCLIP);
    const Turn t = turn(a[5], a[6], c.dev, tokens, d);
    const float* kw = weight(a[7], "k_weight", c.dev, d);
    const double eps = number(a[8]);
    const bool inter = truth(a[9]);
    Heads q;
    at::Tensor qo;
    const bool has_q = a[10] != Py_None;
    const float* qw = weight(a[11], "q_weight", c.dev, d);
    if (has_q) q = heads(tensor(a[10], "q", kt.scalar_type(), c.dev), "q", tokens, -1, d);
    on_gpu(kt, "k");
    if (has_q) qo = output(a[12], "q_out", kt, THPVariable_Unpack(a[10]).sizes(), true);
    const c10::DeviceGuard guard(c.dev);
    if (tokens)
        check(w4a8_kv_append_mxfp4(&view, type, k.p, k.st, k.sh, v.p, v.st, v.sh, tokens, slots, mode, kw, (float)eps,
                                   t.table, t.rows, t.positions, t.rot, inter, q.n ? q.p : nullptr, q.st, q.sh, q.n, qw,
                                   q.n ? static_cast<uint16_t*>(qo.data_ptr()) : nullptr, stream(c.dev)),
              "w4a8_kv_append_mxfp4");
    return has_q ? THPVariable_Wrap(qo) : Py_NewRef(Py_None);
}

// cache, slots
PyObject* read(PyObject* const* a, Py_ssize_t n) {
    arguments(n, 2);
    const Cache& c = cache_of(a[0]);
    const w4a8_kv_cache view = c.view();
    const at::Tensor& s = tensor(a[1], "slots");
    const int64_t tokens = s.dim() == 1 ? s.size(0) : -1;
    const int64_t* slots = vector(a[1], "slots", at::kLong, c.dev, tokens).const_data_ptr<int64_t>();
    on_gpu(s, "slots");
    const int64_t shape[3] = {tokens, view.kv_heads, view.head_dim};
    const auto options = s.options().dtype(at::kBFloat16);
    const at::Tensor k = at::empty(at::IntArrayRef(shape, 3), options), v = at::empty(at::IntArrayRef(shape, 3), options);
    const c10::DeviceGuard guard(c.dev);
    if (tokens)
        check(w4a8_kv_read_mxfp4(&view, tokens, slots, static_cast<uint16_t*>(k.data_ptr()),
                                 static_cast<uint16_t*>(v.data_ptr()), stream(c.dev)),
              "w4a8_kv_read_mxfp4");
    PyObject* r = PyTuple_New(2);
    PyTuple_SET_ITEM(r, 0, THPVariable_Wrap(k));
    PyTuple_SET_ITEM(r, 1, THPVariable_Wrap(v));
    return r;
}

// q, cache, block_table, context_lens, cu_q, max_q, scale, causal, window, workspace (uint8 tensor or None), out
PyObject* attention(PyObject* const* a, Py_ssize_t n) {
    arguments(n, 11);
    const at::Tensor& qt = tensor(a[0], "q");
    const w4a8_float type = float_kind(qt, "q");
    const Cache& c = cache_of(a[1]);
    const w4a8_kv_cache view = c.view();
    tensor(a[0], "q", qt.scalar_type(), c.dev);
    const Heads q = heads(qt, "q", -1, -1, view.head_dim);
    const int64_t tokens = qt.size(0);
    if (q.n == 0 || q.n % view.kv_heads)
        refuse(PyExc_ValueError, "q_heads = %d must be a multiple of kv_heads = %d", q.n, view.kv_heads);
    const at::Tensor& ct = tensor(a[3], "context_lens", at::kInt, c.dev);
    const int64_t seqs = ct.dim() == 1 ? ct.size(0) : -1;
    vector(a[3], "context_lens", at::kInt, c.dev, seqs);
    const at::Tensor& table = tensor(a[2], "block_table", at::kInt, c.dev);
    if (table.dim() != 2 || table.size(0) != seqs || (table.size(1) > 1 && table.stride(1) != 1) ||
        (seqs > 1 && table.stride(0) < table.size(1)))
        refuse(PyExc_ValueError, "block_table must be [seqs, width] with contiguous rows");
    const int64_t max_q = integer(a[5], "max_q", 1, INT32_MAX);
    const int32_t* cu = nullptr;
    if (a[4] != Py_None) cu = vector(a[4], "cu_q", at::kInt, c.dev, seqs + 1).const_data_ptr<int32_t>();
    else if (tokens != seqs || max_q != 1)
        refuse(PyExc_ValueError,
               "without cu_q every sequence has one query token: %lld tokens, %lld sequences, max_q = %lld",
               (long long)tokens, (long long)seqs, (long long)max_q);
    const double scale = a[6] == Py_None ? 1.0 / std::sqrt((double)view.head_dim) : number(a[6]);
    const bool causal = truth(a[7]);
    const int64_t window = integer(a[8], "window", 0, INT32_MAX);
    if (window && !causal) refuse(PyExc_ValueError, "a window needs a causal mask");
    const int64_t width = table.size(1);
    if (width < 1 && seqs > 0) refuse(PyExc_ValueError, "block_table needs at least one column");
    on_gpu(qt, "q");
    at::Tensor out = output(a[10], "out", qt, qt.sizes(), true);
    if (tokens == 0 || seqs == 0) return THPVariable_Wrap(out);
    const c10::DeviceGuard guard(c.dev);
    at::Tensor ws;
    if (a[9] != Py_None) {
        ws = tensor(a[9], "workspace", at::kByte, c.dev);
    } else {
        const size_t need = w4a8_attention_workspace_bytes(seqs, max_q, q.n, view.kv_heads, view.head_dim);
        ws = at::empty({(int64_t)need}, qt.options().dtype(at::kByte));
        check(w4a8_workspace_init(ws.data_ptr(), w4a8_attention_counter_bytes(), stream(c.dev)), "w4a8_workspace_init");
    }
    check(w4a8_attention_mxfp4(&view, type, q.p, q.st, q.sh, q.n, tokens, seqs, cu, max_q, table.const_data_ptr<int32_t>(),
                               seqs > 1 ? table.stride(0) : width, width, ct.const_data_ptr<int32_t>(), (float)scale, causal,
                               (int)window, static_cast<uint16_t*>(out.data_ptr()), ws.data_ptr(), (size_t)ws.numel(),
                               stream(c.dev)),
          "w4a8_attention_mxfp4");
    return THPVariable_Wrap(out);
}

PyObject* set_error(PyObject* const* a, Py_ssize_t n) {
    arguments(n, 1);
    Py_XDECREF(hip_error);
    hip_error = Py_NewRef(a[0]);
    return Py_NewRef(Py_None);
}

// no exception leaves an entry: torch's become Python's
template <PyObject* (*F)(PyObject* const*, Py_ssize_t)>
PyObject* entry(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    try {
        return F(a, n);
    } catch (const Refused&) {
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}
template <PyObject* (*F)(PyObject* const*, Py_ssize_t)>
PyMethodDef method(const char* name) {
    return {name, (PyCFunction)(void (*)(void))entry<F>, METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {method<make_cache>("cache"), method<norm_rope>("norm_rope"), method<append>("append"),
                         method<read>("read"), method<attention>("attention"), method<set_error>("set_error"),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_attention", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__attention() { return PyModule_Create(&module); }
