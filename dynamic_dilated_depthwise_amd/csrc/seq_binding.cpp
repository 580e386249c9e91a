// seq_binding.cpp -- the Python side of the sequence operators' C ABI as a CPython extension:
// argument checks, outputs and workspaces from torch's allocator, the call on the current
// stream.  The single-token forms take 3 us on the GPU; the same checks and allocations in
// Python take 12 us and more, here 3.  sequence.py has the signatures and documentation;
// every function here takes all arguments by position, the stream (or None) last.
#include "binding.hpp"

#include "../../include/ddpm_seq.h"

namespace {

// A state that a step writes in place, as torch's own in-place forms treat it: not where autograd
// would have to follow the write, and counted, so that a backward pass that has kept it raises.
void writable(const Tensor &t, const char *name) {
    if (t.requires_grad() && c10::GradMode::is_enabled())
        refuse(name, " requires grad and a step writes it in place; call it under torch.no_grad()");
}
// slots, or none: the places 0, 1, ... must then be there.
const void *slots_of(const Call &c, PyObject *o, int64_t batch, int64_t S) {
    if (o == Py_None && S < batch) refuse("state has ", S, " places for ", batch, " sequences without slots");
    return c.maybe(o, "slots", at::kInt, {batch});
}
void written(const Tensor &t) {
    if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

// ------------------------------------------------------------------------- layer norm
PyObject *layer_norm_fwd(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    count(n, 6);  // x weight bias eps stats stream
    Call c(a[0], "x", a[5]);
    const Rows r = rows_of(c.x, "x");
    const void *w = c.like(a[1], "weight", {r.C}), *b = c.like(a[2], "bias", {r.C});
    const double eps = PyFloat_AsDouble(a[3]);
    if (eps == -1. && PyErr_Occurred()) throw python_error();
    Tensor y = c.empty(c.x.sizes()), mean, rstd;
    if (truth(a[4])) {
        const at::IntArrayRef lead = c.x.sizes().slice(0, c.x.dim() - 1);
        mean = c.empty(lead, at::kFloat);
        rstd = c.empty(lead, at::kFloat);
    }
    done("ddpm_layer_norm_fwd", ddpm_layer_norm_fwd(c.x.data_ptr(), w, b, y.data_ptr(), (float *)at_of(mean), (float *)at_of(rstd),
                                                    r.rows, r.C, r.stride, (float)eps, c.dtype, c.stream));
    return tuple({y, mean, rstd});
    END_HANDLE_TH_ERRORS
}

PyObject *layer_norm_bwd(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    count(n, 6);  // grad x weight mean rstd stream
    Call c(a[1], "x", a[5]);
    const Rows r = rows_of(c.x, "x");
    const Tensor &grad = tensor(a[0], "grad");
    c.same(grad, "grad", c.x.scalar_type(), c.x.sizes());
    const Rows gr = rows_of(grad, "grad");
    const at::IntArrayRef lead = c.x.sizes().slice(0, c.x.dim() - 1);
    const void *w = c.like(a[2], "weight", {r.C}), *m = c.like(a[3], "mean", at::kFloat, lead),
               *s = c.like(a[4], "rstd", at::kFloat, lead);
    const Tensor gx = c.empty(c.x.sizes()), gw = c.empty({r.C}), gb = c.empty({r.C});
    const Tensor work = c.bytes(ddpm_layer_norm_bwd_workspace(r.rows, r.C, c.dtype));
    done("ddpm_layer_norm_bwd",
         ddpm_layer_norm_bwd(grad.data_ptr(), c.x.data_ptr(), w, (const float *)m, (const float *)s, gx.data_ptr(), gw.data_ptr(),
                             gb.data_ptr(), work.data_ptr(), r.rows, r.C, r.stride, gr.stride, c.dtype, c.stream));
    return tuple({gx, gw, gb});
    END_HANDLE_TH_ERRORS
}

// -------------------------------------------------------------------- causal convolution
struct Taps {
    int64_t W;
    const void *weight, *bias;
};
Taps taps(const Call &c, PyObject *ow, PyObject *ob, int64_t D) {
    const Tensor &w = tensor(ow, "weight");
    if (w.dim() != 2 || w.size(0) != D || w.size(1) < 1) refuse("weight must have shape (", D, ", width) (got ", w.sizes(), ")");
    if (w.size(1) > 0x7fffffff) refuse("weight is too wide");
    return {w.size(1), c.like(ow, "weight", {D, w.size(1)}), c.like(ob, "bias", {D})};
}

void *conv_state(const Call &c, PyObject *o, const char *name, int64_t batch, int64_t W, int64_t D) {
    if (o != Py_None && W == 1) refuse(name, " must be None with one tap");
    return c.maybe(o, name, c.x.scalar_type(), {batch, W - 1, D});
}

PyObject *causal_conv_fwd(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    count(n, 7);  // x weight bias initial_state lengths return_state stream
    Call c(a[0], "x", a[6]);
    shaped(c.x, "x", 3);
    const int64_t batch = c.x.size(0), L = c.x.size(1), D = c.x.size(2);
    c.view(a[0], "x", c.x.sizes(), 2);
    const Taps t = taps(c, a[1], a[2], D);
    const void *init = conv_state(c, a[3], "initial_state", batch, t.W, D), *len = c.maybe(a[4], "lengths", at::kInt, {batch});
    const Tensor y = c.empty({batch, L, D});
    Tensor last;
    if (truth(a[5])) last = c.empty({batch, t.W - 1, D});
    done("ddpm_causal_conv_fwd",
         ddpm_causal_conv_fwd(c.x.data_ptr(), t.weight, t.bias, init, (const int32_t *)len, y.data_ptr(),
                              t.W > 1 ? at_of(last) : nullptr, batch, L, D, (int)t.W, c.x.stride(0), c.x.stride(1), c.dtype,
                              c.stream));
    return tuple({y, last});
    END_HANDLE_TH_ERRORS
}

PyObject *causal_conv_bwd(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    count(n, 8);  // grad x weight bias initial_state lengths grad_state stream
    Call c(a[1], "x", a[7]);
    shaped(c.x, "x", 3);
    const int64_t batch = c.x.size(0), L = c.x.size(1), D = c.x.size(2);
    c.view(a[1], "x", c.x.sizes(), 2);
    const Tensor &grad = c.view(a[0], "grad", c.x.sizes(), 2);
    const Taps t = taps(c, a[2], a[3], D);
    const void *init = conv_state(c, a[4], "initial_state", batch, t.W, D), *len = c.maybe(a[5], "lengths", at::kInt, {batch}),
               *gs = conv_state(c, a[6], "grad_state", batch, t.W, D);
    const Tensor gx = c.empty({batch, L, D}), gw = c.empty({D, t.W}), gb = c.empty({D});
    Tensor gi;
    if (init != nullptr) gi = c.empty({batch, t.W - 1, D});
    const Tensor work = c.bytes(ddpm_causal_conv_bwd_workspace(batch, L, D, (int)t.W, c.dtype));
    done("ddpm_causal_conv_bwd",
         ddpm_causal_conv_bwd(grad.data_ptr(), c.x.data_ptr(), t.weight, t.bias, init, (const int32_t *)len, gs, gx.data_ptr(),
                              gw.data_ptr(), gb.data_ptr(), at_of(gi), work.data_ptr(), batch, L, D, (int)t.W, c.x.stride(0),
                              c.x.stride(1), grad.stride(0), grad.stride(1), c.dtype, c.stream));
    return tuple({gx, gw, gb, gi});
    END_HANDLE_TH_ERRORS
}

PyObject *causal_conv_step(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    count(n, 6);  // x weight bias state slots stream
    Call c(a[0], "x", a[5]);
    shaped(c.x, "x", 2);
    const int64_t batch = c.x.size(0), D = c.x.size(1);
    c.view(a[0], "x", c.x.sizes(), 1);
    const Taps t = taps(c, a[1], a[2], D);
    const Tensor &state = tensor(a[3], "state");
    const int64_t S = state.dim() == 3 ? state.size(0) : 0;
    void *st = c.like(a[3], "state", {S, t.W - 1, D});
    writable(state, "state");
    const void *slots = slots_of(c, a[4], batch, S);
    const Tensor y = c.empty({batch, D});
    done("ddpm_causal_conv_step",
         ddpm_causal_conv_step(c.x.data_ptr(), t.weight, t.bias, t.W > 1 ? st : nullptr, (const int32_t *)slots, y.data_ptr(),
                               batch, S, D, (int)t.W, c.x.stride(0), c.dtype, c.stream));
    written(state);
    return wrap(y);
    END_HANDLE_TH_ERRORS
}

// ----------------------------------------------------------------------- selective scan
// The scan's struct from x dt A B C D dt_bias (a[0] .. a[6]); `lead` axes before the heads.
ddpm_scan scan_of(const Call &c, PyObject *const *a, int64_t lead, PyObject *initial, PyObject *lengths) {
    shaped(c.x, "x", lead + 2);
    const Tensor &B = tensor(a[3], "B");
    shaped(B, "B", lead + 2);
    const int64_t batch = c.x.size(0), L = lead == 2 ? c.x.size(1) : 1, H = c.x.size(lead), P = c.x.size(lead + 1);
    const int64_t G = B.size(lead), N = B.size(lead + 1);
    if (H % G) refuse(H, " heads do not divide into ", G, " groups");
    for (int64_t v : {H, P, G, N})
        if (v > 0x7fffffff) refuse("heads, groups and their sizes must be below 2^31");
    const auto view = [&](int k, const char *name, int64_t p, int64_t q) -> const Tensor & {
        int64_t s[4] = {batch, L, p, q};
        if (lead == 1) { s[1] = p; s[2] = q; }
        return c.view(a[k], name, at::IntArrayRef(s, (size_t)(lead + (q ? 2 : 1))), lead);
    };
    const Tensor &x = view(0, "x", H, P), &dt = view(1, "dt", H, 0), &b = view(3, "B", G, N), &cc = view(4, "C", G, N);
    const auto token = [&](const Tensor &t) { return lead == 2 ? t.stride(1) : 0; };
    ddpm_scan s;
    s.x = x.data_ptr();
    s.dt = dt.data_ptr();
    s.B = b.data_ptr();
    s.C = cc.data_ptr();
    s.A = (const float *)c.like(a[2], "A", at::kFloat, {H});
    s.D = (const float *)c.like(a[5], "D", at::kFloat, {H});
    s.dt_bias = (const float *)c.like(a[6], "dt_bias", at::kFloat, {H});
    s.initial_state = (const float *)c.maybe(initial, "initial_state", at::kFloat, {batch, H, P, N});
    s.lengths = (const int32_t *)c.maybe(lengths, "lengths", at::kInt, {batch});
    s.batch = batch;
    s.length = L;
    s.x_batch = x.stride(0);
    s.x_token = token(x);
    s.dt_batch = dt.stride(0);
    s.dt_token = token(dt);
    s.B_batch = b.stride(0);
    s.B_token = token(b);
    s.C_batch = cc.stride(0);
    s.C_token = token(cc);
    s.heads = (int32_t)H;
    s.P = (int32_t)P;
    s.groups = (int32_t)G;
    s.N = (int32_t)N;
    s.dtype = c.dtype;
    return s;
}

PyObject *selective_scan_fwd(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    count(n, 12);  // x dt A B C D dt_bias initial_state lengths return_state save stream
    Call c(a[0], "x", a[11]);
    const ddpm_scan s = scan_of(c, a, 2, a[7], a[8]);
    const bool save = truth(a[10]);
    const Tensor y = c.empty(c.x.sizes());
    Tensor last;
    if (truth(a[9])) last = c.empty({s.batch, s.heads, s.P, s.N}, at::kFloat);
    const Tensor work = c.bytes(ddpm_selective_scan_fwd_workspace(&s));
    done("ddpm_selective_scan_fwd",
         ddpm_selective_scan_fwd(&s, y.data_ptr(), (float *)at_of(last), save ? 1 : 0, work.data_ptr(), c.stream));
    return tuple({y, last, save ? work : Tensor()});
    END_HANDLE_TH_ERRORS
}

PyObject *selective_scan_bwd(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    count(n, 13);  // grad x dt A B C D dt_bias saved initial_state lengths grad_state stream
    Call c(a[1], "x", a[12]);
    const ddpm_scan s = scan_of(c, a + 1, 2, a[9], a[10]);
    const Tensor &grad = c.view(a[0], "grad", c.x.sizes(), 2);
    const void *saved = c.like(a[8], "saved", at::kByte, {ddpm_selective_scan_fwd_workspace(&s)});
    const float *gs = (const float *)c.maybe(a[11], "grad_state", at::kFloat, {s.batch, s.heads, s.P, s.N});
    const Tensor gx = c.empty(c.x.sizes()), gdt = c.empty({s.batch, s.length, s.heads}),
                 gB = c.empty({s.batch, s.length, s.groups, s.N}), gC = c.empty({s.batch, s.length, s.groups, s.N}),
                 gA = c.empty({s.heads}, at::kFloat), gD = c.empty({s.heads}, at::kFloat), gbias = c.empty({s.heads}, at::kFloat);
    Tensor gi;
    if (s.initial_state != nullptr) gi = c.empty({s.batch, s.heads, s.P, s.N}, at::kFloat);
    const Tensor work = c.bytes(ddpm_selective_scan_bwd_workspace(&s));
    done("ddpm_selective_scan_bwd",
         ddpm_selective_scan_bwd(&s, saved, grad.data_ptr(), grad.stride(0), grad.stride(1), gs, gx.data_ptr(), gdt.data_ptr(),
                                 (float *)gA.data_ptr(), gB.data_ptr(), gC.data_ptr(), (float *)gD.data_ptr(),
                                 (float *)gbias.data_ptr(), (float *)at_of(gi), work.data_ptr(), c.stream));
    return tuple({gx, gdt, gA, gB, gC, gD, gbias, gi});
    END_HANDLE_TH_ERRORS
}

PyObject *selective_scan_step(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    count(n, 10);  // x dt A B C D dt_bias state slots stream
    Call c(a[0], "x", a[9]);
    const ddpm_scan s = scan_of(c, a, 1, Py_None, Py_None);
    const Tensor &state = tensor(a[7], "state");
    const int64_t S = state.dim() == 4 ? state.size(0) : 0;
    float *st = (float *)c.like(a[7], "state", at::kFloat, {S, s.heads, s.P, s.N});
    writable(state, "state");
    const void *slots = slots_of(c, a[8], s.batch, S);
    const Tensor y = c.empty(c.x.sizes());
    done("ddpm_selective_scan_step", ddpm_selective_scan_step(&s, st, (const int32_t *)slots, S, y.data_ptr(), c.stream));
    written(state);
    return wrap(y);
    END_HANDLE_TH_ERRORS
}

#define DDPM_SEQ_METHOD(name) {#name, (PyCFunction)(void (*)(void))name, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {
    DDPM_SEQ_METHOD(layer_norm_fwd),     DDPM_SEQ_METHOD(layer_norm_bwd),     DDPM_SEQ_METHOD(causal_conv_fwd),
    DDPM_SEQ_METHOD(causal_conv_bwd),    DDPM_SEQ_METHOD(causal_conv_step),   DDPM_SEQ_METHOD(selective_scan_fwd),
    DDPM_SEQ_METHOD(selective_scan_bwd), DDPM_SEQ_METHOD(selective_scan_step), {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_sequence", "Binding of ddpm_seq.h.", -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__sequence(void) { return PyModule_Create(&module); }
