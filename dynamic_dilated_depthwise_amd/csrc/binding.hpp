// binding.hpp -- what the CPython extensions of the operators' C ABI share: argument checks, outputs
// and workspaces from torch's allocator, the stream of a call, errors.  Everything here is local to
// the source that includes it.
#pragma once

#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/hip/EmptyTensor.h>
#include <c10/core/DeviceGuard.h>
#include <c10/core/GradMode.h>
#include <c10/core/StreamGuard.h>
#include <c10/hip/HIPCachingAllocator.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/Stream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstring>
#include <initializer_list>
#include <optional>
#include <sstream>

#include "../../include/ddpm.h"

namespace {

using at::Tensor;
typedef std::initializer_list<int64_t> Sizes;

template <typename... A>
[[noreturn]] void refuse(const A &...a) {
    std::ostringstream s;
    (s << ... << a);
    throw c10::ValueError({__func__, __FILE__, __LINE__}, s.str());
}

const Tensor &tensor(PyObject *o, const char *name) {
    if (!THPVariable_Check(o)) throw c10::TypeError({__func__, __FILE__, __LINE__}, std::string(name) + " must be a torch.Tensor");
    const Tensor &t = THPVariable_Unpack(o);
    if (!t.is_cuda()) refuse(name, " must be a device tensor (got ", t.device(), ")");
    return t;
}

// What every call starts with: its first tensor, the device and stream that it runs on.
struct Call {
    const Tensor &x;
    std::optional<c10::StreamGuard> on;
    std::optional<c10::DeviceGuard> at_device;
    int dtype = 0;
    hipStream_t stream = nullptr;
    bool given = false;  // a stream other than the current one

    Call(PyObject *ox, const char *name, PyObject *stream_or_none) : x(tensor(ox, name)) {
        if (stream_or_none != Py_None) {
            if (!PyObject_IsInstance(stream_or_none, (PyObject *)THPStreamClass))
                throw c10::TypeError({__func__, __FILE__, __LINE__}, "stream must be a torch.cuda.Stream");
            auto *s = (THPStream *)stream_or_none;
            given = c10::hip::getCurrentHIPStream(x.device().index()).id() != s->stream_id;
            on.emplace(c10::Stream::unpack3(s->stream_id, (c10::DeviceIndex)s->device_index, (c10::DeviceType)s->device_type));
            if (s->device_index != x.device().index()) refuse("stream must be on ", x.device());
        } else if (x.device().index() != c10::hip::current_device()) {
            at_device.emplace(x.device());
        }
        if (x.scalar_type() == at::kFloat) dtype = DDPM_F32;
        else if (x.scalar_type() == at::kBFloat16) dtype = DDPM_BF16;
        else refuse("unsupported dtype ", x.scalar_type(), "; use float32 or bfloat16");
        stream = c10::hip::getCurrentHIPStream(x.device().index()).stream();
        use(x);
    }

    // On a given stream an argument's memory must not go to another tensor before the work is
    // done, whenever its owner lets go of it; outputs and workspaces come from that stream.
    void use(const Tensor &t) const {
        if (given) c10::hip::HIPCachingAllocator::recordStream(t.storage().data_ptr(), c10::hip::getCurrentHIPStream(x.device().index()));
    }

    Tensor empty(at::IntArrayRef sizes, at::ScalarType t) const {
        return Tensor(at::detail::empty_cuda(sizes, t, x.device(), std::nullopt));
    }
    Tensor empty(at::IntArrayRef sizes) const { return empty(sizes, x.scalar_type()); }
    Tensor bytes(int64_t n) const { return empty({n}, at::kByte); }

    void same(const Tensor &t, const char *name, at::ScalarType type, at::IntArrayRef sizes) const {
        if (t.scalar_type() != type) refuse(name, " must be ", type, " (got ", t.scalar_type(), ")");
        if (t.sizes() != sizes) refuse(name, " must have shape ", sizes, " (got ", t.sizes(), ")");
        if (t.device() != x.device()) refuse(name, " must be on ", x.device(), " (got ", t.device(), ")");
        use(t);
    }
    // A contiguous tensor of this type and shape.
    void *like(PyObject *o, const char *name, at::ScalarType type, at::IntArrayRef sizes) const {
        const Tensor &t = tensor(o, name);
        same(t, name, type, sizes);
        if (!t.is_contiguous()) refuse(name, " must be contiguous");
        return t.data_ptr();
    }
    void *like(PyObject *o, const char *name, at::IntArrayRef sizes) const { return like(o, name, x.scalar_type(), sizes); }
    void *maybe(PyObject *o, const char *name, at::ScalarType type, at::IntArrayRef sizes) const {
        return o == Py_None ? nullptr : like(o, name, type, sizes);
    }
    // One whose axes after the first `axes` are contiguous.
    const Tensor &view(PyObject *o, const char *name, at::IntArrayRef sizes, int64_t axes) const {
        const Tensor &t = tensor(o, name);
        same(t, name, x.scalar_type(), sizes);
        int64_t want = 1;
        for (int64_t k = t.dim() - 1; k >= axes; --k) {
            if (t.size(k) != 1 && t.stride(k) != want)
                refuse(name, " must be contiguous after its first ", axes, " axes (got strides ", t.strides(), ")");
            want *= t.size(k);
        }
        return t;
    }
};

void shaped(const Tensor &t, const char *name, int64_t axes) {
    if (t.dim() != axes) refuse(name, " must have ", axes, " axes (got shape ", t.sizes(), ")");
    if (t.numel() == 0) refuse(name, " must not be empty (got shape ", t.sizes(), ")");
}

void done(const char *fn, int status) {
    if (status == DDPM_OK) return;
    PyObject *module = PyImport_ImportModule("dynamic_dilated_depthwise_amd");
    PyObject *type = module != nullptr ? PyObject_GetAttrString(module, "DDPMError") : nullptr;
    PyObject *error = type != nullptr ? PyObject_CallFunction(type, "si", fn, status) : nullptr;
    if (error != nullptr) PyErr_SetObject(type, error);
    Py_XDECREF(error);
    Py_XDECREF(type);
    Py_XDECREF(module);
    throw python_error();
}

PyObject *wrap(const Tensor &t) {
    if (!t.defined()) Py_RETURN_NONE;
    return THPVariable_Wrap(t);
}

PyObject *tuple(std::initializer_list<Tensor> ts) {
    PyObject *r = PyTuple_New((Py_ssize_t)ts.size());
    Py_ssize_t k = 0;
    for (const Tensor &t : ts) PyTuple_SET_ITEM(r, k++, wrap(t));
    return r;
}

void *at_of(const Tensor &t) { return t.defined() ? t.data_ptr() : nullptr; }

void count(Py_ssize_t n, Py_ssize_t want) {
    if (n != want) throw c10::TypeError({__func__, __FILE__, __LINE__}, "wrong number of arguments");
}

bool truth(PyObject *o) {
    const int r = PyObject_IsTrue(o);
    if (r < 0) throw python_error();
    return r != 0;
}

struct Rows {
    int64_t rows, C, stride;
};
// [..., C]: contiguous, or two axes with contiguous rows.
Rows rows_of(const Tensor &x, const char *name) {
    if (x.dim() < 1 || x.numel() == 0) refuse(name, " must have a last axis and not be empty (got shape ", x.sizes(), ")");
    const int64_t C = x.size(-1);
    if (x.is_contiguous()) return {x.numel() / C, C, C};
    if (x.dim() == 2 && (x.stride(1) == 1 || C == 1)) return {x.size(0), C, x.stride(0)};
    refuse(name, " must be contiguous, or have two axes with contiguous rows (got strides ", x.strides(), ")");
}

}  // namespace
