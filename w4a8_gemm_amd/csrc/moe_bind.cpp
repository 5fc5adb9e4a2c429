// moe_bind.cpp -- Python entry of the expert half of a layer (module _moe).
//
// Marshalling only, as attention_bind.cpp: checks that a pointer cannot carry,
// pointers, strides and the current stream, status codes as exceptions.  Every
// function takes all of its arguments by position; the signatures, defaults and
// documentation are in moe.py.
#include <optional>

#include <ATen/hip/EmptyTensor.h>

#include "bind.h"

namespace {

PyObject* or_none(const at::Tensor& t) { return t.defined() ? THPVariable_Wrap(t) : Py_NewRef(Py_None); }

// [rows, cols] with contiguous rows
void matrix(const at::Tensor& t, const char* name, int64_t rows, int64_t cols) {
    if (t.dim() != 2 || t.size(0) != rows || t.size(1) != cols)
        refuse(PyExc_ValueError, "%s must be [%lld, %lld]", name, (long long)rows, (long long)cols);
    if (cols > 1 && t.stride(1) != 1) refuse(PyExc_ValueError, "%s must have contiguous rows (unit last stride)", name);
}
// a new contiguous tensor, past the dispatcher
at::Tensor fresh(at::Device dev, at::ScalarType type, at::IntArrayRef shape) {
    return at::Tensor(at::detail::empty_cuda(shape, type, dev, std::nullopt));
}
// the caller's contiguous output, or a new one
at::Tensor target(PyObject* o, const char* name, const at::Tensor& like, at::ScalarType type, at::IntArrayRef shape) {
    if (o == Py_None) return fresh(like.device(), type, shape);
    const at::Tensor& t = tensor(o, name, type, like.device());
    if (t.sizes() != shape || !t.is_contiguous())
        refuse(PyExc_ValueError, "%s must be a contiguous tensor of the result's shape", name);
    return t;
}

// y, residual, weight, post_weight, gate, scale, eps, values, fp8, residual_out, out, x_fp8, x_scale
PyObject* residual_norm(PyObject* const* a, Py_ssize_t n) {
    arguments(n, 13);
    const at::Tensor& y = tensor(a[0], "y");
    const w4a8_float type = float_kind(y, "y");
    const at::Device dev = y.device();
    if (y.dim() != 2 || y.size(1) < 1) refuse(PyExc_ValueError, "y must be [tokens, hidden]");
    const int64_t tokens = y.size(0), hidden = y.size(1);
    matrix(y, "y", tokens, hidden);
    const at::Tensor* r = nullptr;
    if (a[1] != Py_None) {
        r = &tensor(a[1], "residual");
        if (r->scalar_type() != at::kFloat && r->scalar_type() != y.scalar_type())
            refuse(PyExc_TypeError, "residual must be of y's type or float32");
        tensor(a[1], "residual", r->scalar_type(), dev);
        matrix(*r, "residual", tokens, hidden);
    }
    const float *w = weight(a[2], "weight", dev, hidden), *pw = weight(a[3], "post_weight", dev, hidden);
    const at::Tensor* g = nullptr;
    int64_t gs[2] = {0, 0};
    if (a[4] != Py_None) {
        g = &tensor(a[4], "gate", y.scalar_type(), dev);
        const bool fits = g->dim() == 2 && (g->size(0) == tokens || g->size(0) == 1) && (g->size(1) == hidden || g->size(1) == 1);
        if (!fits) refuse(PyExc_ValueError, "gate must be [tokens or 1, hidden or 1]");
        gs[0] = g->size(0) == 1 ? 0 : g->stride(0);
        gs[1] = g->size(1) == 1 ? 0 : g->stride(1);
        if (gs[1] > 1) refuse(PyExc_ValueError, "gate must have contiguous rows, or one value for a row");
    }
    const double scale = number(a[5]), eps = number(a[6]);
    const bool values = truth(a[7]), fp8 = truth(a[8]);
    if (!values && !fp8 && !r && a[9] == Py_None) refuse(PyExc_ValueError, "nothing to compute: values, fp8 or a residual");
    if (!values && a[10] != Py_None) refuse(PyExc_ValueError, "out needs values=True");
    if (!fp8 && (a[11] != Py_None || a[12] != Py_None)) refuse(PyExc_ValueError, "x_fp8 and x_scale need fp8=True");
    on_gpu(y, "y");
    const c10::DeviceGuard guard(dev);
    at::Tensor ro, out, x8, xs;
    if (r || a[9] != Py_None) {
        const at::ScalarType rt = r ? r->scalar_type() : y.scalar_type();
        if (a[9] == Py_None) {
            ro = fresh(dev, rt, {tokens, hidden});
        } else {
            ro = tensor(a[9], "residual_out", rt, dev);
            matrix(ro, "residual_out", tokens, hidden);
            if (tokens > 1 && ro.stride(0) < hidden) refuse(PyExc_ValueError, "residual_out's rows overlap");
        }
    }
    const int64_t shape[2] = {tokens, hidden};
    if (values) out = target(a[10], "out", y, y.scalar_type(), at::IntArrayRef(shape, 2));
    if (fp8) {
        x8 = target(a[11], "x_fp8", y, at::kByte, at::IntArrayRef(shape, 2));
        xs = target(a[12], "x_scale", y, at::kFloat, at::IntArrayRef(shape, 1));
    }
    if (tokens)
        check(w4a8_residual_norm(type, static_cast<const uint16_t*>(y.const_data_ptr()), y.stride(0), tokens, hidden, pw,
                                 g ? static_cast<const uint16_t*>(g->const_data_ptr()) : nullptr, gs[0], gs[1], (float)scale,
                                 r ? r->const_data_ptr() : nullptr, r && r->scalar_type() == at::kFloat, r ? r->stride(0) : 0,
                                 ro.defined() ? ro.data_ptr() : nullptr, ro.defined() ? ro.stride(0) : 0, w, (float)eps,
                                 values ? static_cast<uint16_t*>(out.data_ptr()) : nullptr,
                                 fp8 ? static_cast<uint8_t*>(x8.data_ptr()) : nullptr,
                                 fp8 ? static_cast<float*>(xs.data_ptr()) : nullptr, stream(dev)),
              "w4a8_residual_norm");
    PyObject* t = PyTuple_New(4);
    PyTuple_SET_ITEM(t, 0, or_none(ro));
    PyTuple_SET_ITEM(t, 1, or_none(out));
    PyTuple_SET_ITEM(t, 2, or_none(x8));
    PyTuple_SET_ITEM(t, 3, or_none(xs));
    return t;
}

// logits, top_k, score, bias, groups, groups_kept, group_top, renormalize, scale, weights, ids
PyObject* route(PyObject* const* a, Py_ssize_t n) {
    arguments(n, 11);
    const at::Tensor& x = tensor(a[0], "logits");
    const at::Device dev = x.device();
    w4a8_float type = W4A8_FP32;
    if (x.scalar_type() == at::kBFloat16) type = W4A8_BF16;
    else if (x.scalar_type() == at::kHalf) type = W4A8_FP16;
    else if (x.scalar_type() != at::kFloat) refuse(PyExc_TypeError, "logits must be a float32, bfloat16 or float16 tensor");
    if (x.dim() != 2 || x.size(1) < 1 || x.size(1) > 1024) refuse(PyExc_ValueError, "logits must be [tokens, 1 to 1024 experts]");
    const int64_t tokens = x.size(0), experts = x.size(1);
    matrix(x, "logits", tokens, experts);
    const int64_t k = integer(a[1], "top_k", 1, experts < 32 ? experts : 32);
    const w4a8_score score = (w4a8_score)integer(a[2], "score", 0, 1);
    const float* bias = weight(a[3], "bias", dev, experts);
    const int64_t groups = integer(a[4], "groups", 1, experts < 64 ? experts : 64);
    if (experts % groups) refuse(PyExc_ValueError, "groups must divide the %lld experts", (long long)experts);
    const int64_t kept = integer(a[5], "groups_kept", 1, groups), top = integer(a[6], "group_top", 1, 2);
    const bool renormalize = truth(a[7]);
    const double scale = number(a[8]);
    on_gpu(x, "logits");
    const c10::DeviceGuard guard(dev);
    const int64_t shape[2] = {tokens, k};
    at::Tensor w = target(a[9], "weights", x, at::kFloat, at::IntArrayRef(shape, 2));
    at::Tensor ids = target(a[10], "ids", x, at::kInt, at::IntArrayRef(shape, 2));
    if (tokens)
        check(w4a8_moe_route(type, x.const_data_ptr(), x.stride(0), tokens, (int)experts, (int)k, score, bias, (int)groups,
                             (int)kept, (int)top, renormalize, (float)scale, static_cast<int32_t*>(ids.data_ptr()),
                             static_cast<float*>(w.data_ptr()), stream(dev)),
              "w4a8_moe_route");
    PyObject* t = PyTuple_New(2);
    PyTuple_SET_ITEM(t, 0, THPVariable_Wrap(w));
    PyTuple_SET_ITEM(t, 1, THPVariable_Wrap(ids));
    return t;
}

// ---- the experts: their four tensors, held ----
struct Experts {
    at::Tensor t[4];
    at::Device dev;
    w4a8_experts_mxfp4 view;
};
const char kExperts[] = "w4a8_experts_mxfp4";
void drop_experts(PyObject* o) { delete static_cast<Experts*>(PyCapsule_GetPointer(o, kExperts)); }

// up_w, up_s, down_w, down_s, experts, hidden, inter
PyObject* make_experts(PyObject* const* a, Py_ssize_t n) {
    arguments(n, 7);
    static const char* names[4] = {"up.w", "up.s", "down.w", "down.s"};
    const at::Device dev = tensor(a[0], names[0]).device();
    const int64_t e = integer(a[4], "experts", 1, 1024), hidden = integer(a[5], "hidden", 128, 65536),
                  inter = integer(a[6], "inter", 128, 65536);
    if (hidden % 128 || inter % 128) refuse(PyExc_ValueError, "hidden and inter must be multiples of 128");
    size_t need[4];
    check(w4a8_mxfp4_prepared_bytes(e * 2 * inter, hidden, &need[0], &need[1]), "w4a8_mxfp4_prepared_bytes");
    check(w4a8_mxfp4_prepared_bytes(e * hidden, inter, &need[2], &need[3]), "w4a8_mxfp4_prepared_bytes");
    const at::Tensor* t[4];
    for (int i = 0; i < 4; ++i) {
        t[i] = &tensor(a[i], names[i], at::kByte, dev);
        if (!t[i]->is_contiguous() || t[i]->numel() < (int64_t)need[i])
            refuse(PyExc_ValueError, "%s holds fewer than the %lld contiguous bytes of this weight", names[i], (long long)need[i]);
    }
    const auto p = [&](int i) { return static_cast<const uint8_t*>(t[i]->const_data_ptr()); };
    return PyCapsule_New(new Experts{{*t[0], *t[1], *t[2], *t[3]}, dev, {p(0), p(1), p(2), p(3), (int)e, hidden, inter}},
                         kExperts, drop_experts);
}

// x_fp8, x_scale, ids, weights, experts, act, workspace (uint8 tensor or None), out
PyObject* moe(PyObject* const* a, Py_ssize_t n) {
    arguments(n, 8);
    if (!PyCapsule_IsValid(a[4], kExperts)) refuse(PyExc_TypeError, "experts must be an ExpertsMXFP4");
    const Experts& e = *static_cast<const Experts*>(PyCapsule_GetPointer(a[4], kExperts));
    const at::Tensor& x = tensor(a[0], "x_fp8", at::kByte, e.dev);
    const int64_t tokens = x.dim() == 2 ? x.size(0) : -1;
    matrix(x, "x_fp8", tokens, e.view.hidden);
    if (!x.is_contiguous()) refuse(PyExc_ValueError, "x_fp8 must be contiguous");
    const float* xs = vector(a[1], "x_scale", at::kFloat, e.dev, tokens).const_data_ptr<float>();
    const at::Tensor& ids = tensor(a[2], "ids", at::kInt, e.dev);
    const int64_t k = ids.dim() == 2 ? ids.size(1) : 0;
    if (k < 1 || k > 32 || k > e.view.experts) refuse(PyExc_ValueError, "ids must be [tokens, 1 to 32, and to the experts]");
    const at::Tensor& w = tensor(a[3], "weights", at::kFloat, e.dev);
    matrix(ids, "ids", tokens, k);
    matrix(w, "weights", tokens, k);
    if (!ids.is_contiguous() || !w.is_contiguous()) refuse(PyExc_ValueError, "ids and weights must be contiguous");
    const w4a8_act act = (w4a8_act)integer(a[5], "act", 0, 1);
    on_gpu(x, "x_fp8");
    const c10::DeviceGuard guard(e.dev);
    const int64_t shape[2] = {tokens, e.view.hidden};
    at::Tensor out = target(a[7], "out", x, at::kBFloat16, at::IntArrayRef(shape, 2));
    if (tokens == 0) return THPVariable_Wrap(out);
    const at::Tensor ws = a[6] != Py_None ? tensor(a[6], "workspace", at::kByte, e.dev)
                                          : fresh(e.dev, at::kByte, {(int64_t)w4a8_moe_workspace_bytes(tokens, (int)k, e.view.hidden, e.view.inter)});
    check(w4a8_moe_mxfp4(&e.view, static_cast<const uint8_t*>(x.const_data_ptr()), xs, tokens, ids.const_data_ptr<int32_t>(),
                         w.const_data_ptr<float>(), (int)k, act, static_cast<uint16_t*>(out.data_ptr()), ws.data_ptr(),
                         (size_t)ws.numel(), stream(e.dev)),
          "w4a8_moe_mxfp4");
    return THPVariable_Wrap(out);
}

PyMethodDef methods[] = {method<residual_norm>("residual_norm"), method<route>("route"), method<make_experts>("experts"),
                         method<moe>("moe"), method<set_error>("set_error"), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_moe", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__moe() { return PyModule_Create(&module); }
