// ff_binding.cpp -- the Python side of the feed-forward operators' C ABI as a CPython extension.
// feedforward.py has the signatures and documentation; every function here takes all arguments by
// position, the stream (or None) last.
#include "binding.hpp"

#include "../../include/ddpm_ff.h"

namespace {

int activation_of(PyObject *o) {
    const char *s = PyUnicode_Check(o) ? PyUnicode_AsUTF8(o) : nullptr;
    if (s == nullptr) {
        PyErr_Clear();
        throw c10::TypeError({__func__, __FILE__, __LINE__}, "activation must be a str");
    }
    const char *names[] = {"none", "relu", "silu", "gelu"};
    for (int k = 0; k < 4; ++k)
        if (std::strcmp(s, names[k]) == 0) return k;
    refuse("activation must be none, relu, silu or gelu (got ", s, ")");
}

// [..., C] with its last axis replaced.
c10::SmallVector<int64_t, 6> with_last(const Tensor &x, int64_t last) {
    c10::SmallVector<int64_t, 6> s(x.sizes().begin(), x.sizes().end());
    s.back() = last;
    return s;
}

// A tensor of the call's type, with rows as x has them.
Rows rows_like(const Call &c, PyObject *o, const char *name, at::IntArrayRef sizes) {
    const Tensor &t = tensor(o, name);
    c.same(t, name, c.x.scalar_type(), sizes);
    return rows_of(t, name);
}

// weight [halves * N, C], contiguous: its N.
struct Weight {
    const void *data;
    int64_t N, width;
};
Weight weight_of(const Call &c, PyObject *o, int64_t C, int64_t halves) {
    const Tensor &w = tensor(o, "weight");
    if (w.dim() != 2 || w.size(1) != C || w.size(0) < 1 || w.size(0) % halves != 0)
        refuse("weight must have shape (", halves == 2 ? "2 * N, " : "N, ", C, ") (got ", w.sizes(), ")");
    return {c.like(o, "weight", {w.size(0), C}), w.size(0) / halves, w.size(0)};
}

Tensor room(const Call &c, int64_t bytes) { return bytes > 0 ? c.bytes(bytes) : Tensor(); }

// Floats of what the forward saves.
int64_t saved_of(const Call &c, const Rows &r, const Weight &w, int act, bool gated) {
    return gated ? ddpm_gated_linear_saved(r.rows, r.C, w.N, c.dtype) : ddpm_linear_saved(r.rows, r.C, w.N, act, c.dtype);
}

PyObject *forward(PyObject *const *a, bool gated) {
    PyObject *residual = gated ? Py_None : a[3];
    PyObject *const *rest = a + (gated ? 3 : 4);  // activation save stream
    Call c(a[0], "x", rest[2]);
    const Rows r = rows_of(c.x, "x");
    const Weight w = weight_of(c, a[1], r.C, gated ? 2 : 1);
    const void *bias = c.maybe(a[2], "bias", c.x.scalar_type(), {w.width});
    const int act = activation_of(rest[0]);
    const auto out = with_last(c.x, w.N);
    Rows rr = {0, 0, 0};
    const void *res = nullptr;
    if (residual != Py_None) {
        rr = rows_like(c, residual, "residual", out);
        res = tensor(residual, "residual").data_ptr();
    }
    const Tensor y = c.empty(out);
    Tensor saved;
    if (truth(rest[1]) && (gated || act != DDPM_ACT_NONE)) saved = c.empty({saved_of(c, r, w, act, gated)}, at::kFloat);
    const Tensor work = room(c, gated ? ddpm_gated_linear_fwd_workspace(r.rows, r.C, w.N, c.dtype)
                                      : ddpm_linear_fwd_workspace(r.rows, r.C, w.N, c.dtype));
    if (gated)
        done("ddpm_gated_linear_fwd",
             ddpm_gated_linear_fwd(c.x.data_ptr(), w.data, bias, y.data_ptr(), (float *)at_of(saved), at_of(work), r.rows, r.C, w.N,
                                   r.stride, act, c.dtype, c.stream));
    else
        done("ddpm_linear_fwd", ddpm_linear_fwd(c.x.data_ptr(), w.data, bias, res, y.data_ptr(), (float *)at_of(saved), at_of(work),
                                                r.rows, r.C, w.N, r.stride, rr.stride, act, c.dtype, c.stream));
    return tuple({y, saved});
}

PyObject *backward(PyObject *const *a, bool gated) {
    // grad x weight saved activation need_x need_weight stream
    Call c(a[1], "x", a[7]);
    const Rows r = rows_of(c.x, "x");
    const Weight w = weight_of(c, a[2], r.C, gated ? 2 : 1);
    const Rows gr = rows_like(c, a[0], "grad", with_last(c.x, w.N));
    const Tensor &grad = tensor(a[0], "grad");
    const int act = activation_of(a[4]);
    const float *saved = nullptr;
    if (gated || act != DDPM_ACT_NONE) saved = (const float *)c.like(a[3], "saved", at::kFloat, {saved_of(c, r, w, act, gated)});
    else if (a[3] != Py_None) refuse("saved must be None without an activation");
    Tensor gx, gw, gb;
    if (truth(a[5])) gx = c.empty(c.x.sizes());
    if (truth(a[6])) {
        gw = c.empty({w.width, r.C});
        gb = c.empty({w.width});
    }
    const Tensor work = room(c, gated ? ddpm_gated_linear_bwd_workspace(r.rows, r.C, w.N, c.dtype)
                                      : ddpm_linear_bwd_workspace(r.rows, r.C, w.N, act, c.dtype));
    done(gated ? "ddpm_gated_linear_bwd" : "ddpm_linear_bwd",
         (gated ? ddpm_gated_linear_bwd : ddpm_linear_bwd)(grad.data_ptr(), c.x.data_ptr(), w.data, saved, at_of(gx), at_of(gw),
                                                           at_of(gb), at_of(work), r.rows, r.C, w.N, r.stride, gr.stride, act,
                                                           c.dtype, c.stream));
    return tuple({gx, gw, gb});
}

PyObject *linear_fwd(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    count(n, 7);  // x weight bias residual activation save stream
    return forward(a, false);
    END_HANDLE_TH_ERRORS
}
PyObject *gated_linear_fwd(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    count(n, 6);  // x weight bias activation save stream
    return forward(a, true);
    END_HANDLE_TH_ERRORS
}
PyObject *linear_bwd(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    count(n, 8);
    return backward(a, false);
    END_HANDLE_TH_ERRORS
}
PyObject *gated_linear_bwd(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    count(n, 8);
    return backward(a, true);
    END_HANDLE_TH_ERRORS
}

#define DDPM_FF_METHOD(name) {#name, (PyCFunction)(void (*)(void))name, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {DDPM_FF_METHOD(linear_fwd), DDPM_FF_METHOD(linear_bwd), DDPM_FF_METHOD(gated_linear_fwd),
                         DDPM_FF_METHOD(gated_linear_bwd), {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_feedforward", "Binding of ddpm_ff.h.", -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__feedforward(void) { return PyModule_Create(&module); }
