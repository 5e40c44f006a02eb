// CPython extension that calls the large products of libsgmv: it turns torch
// tensors into descriptors and passes torch's current stream, nothing else.
// A decode step calls these entry points for every layer; marshalled field by
// field through ctypes a call took 23 us of host time, longer than its kernels.
//
// init() receives the addresses of the library's functions, so the extension
// does not link against libsgmv.so.
#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "sgmv.h"

namespace {

using LoraFn = decltype(&sgmv_lora_linear);
using GroupedFn = decltype(&sgmv_grouped_gemm);   // sgmv_grouped_wgrad has the same type
LoraFn g_lora = nullptr;
GroupedFn g_gemm = nullptr, g_wgrad = nullptr;

int dtype_of(const at::Tensor& t) {
    switch (t.scalar_type()) {
        case at::kHalf: return SGMV_F16;
        case at::kBFloat16: return SGMV_BF16;
        case at::kFloat: return SGMV_F32;
        case at::kInt: return SGMV_I32;
        case at::kLong: return SGMV_I64;
        default: return -1;
    }
}

// Fills d from a tensor on `device`; false with a Python error set, or *rc < 0.
bool describe(PyObject* o, const c10::Device& device, sgmv_tensor* d, int* rc) {
    if (!THPVariable_Check(o)) {
        PyErr_SetString(PyExc_TypeError, "expected a torch.Tensor");
        return false;
    }
    const at::Tensor& t = THPVariable_Unpack(o);
    if (t.device() != device) {
        PyErr_SetString(PyExc_ValueError, "all tensors must be CUDA tensors on the same device");
        return false;
    }
    d->dtype = dtype_of(t);
    if (d->dtype < 0) {
        PyErr_Format(PyExc_TypeError, "unsupported dtype %s", c10::toString(t.scalar_type()));
        return false;
    }
    if (t.dim() < 1 || t.dim() > 4) {
        *rc = SGMV_ERR_NDIM;
        return false;
    }
    d->data = t.data_ptr();
    d->ndim = (int32_t)t.dim();
    for (int i = 0; i < d->ndim; ++i) {
        d->shape[i] = t.size(i);
        d->stride[i] = t.stride(i);
    }
    return true;
}

bool number(PyObject* o, int64_t* v) {
    PyObject* i = PyNumber_Index(o);
    if (!i) return false;
    *v = PyLong_AsLongLong(i);
    Py_DECREF(i);
    return !(*v == -1 && PyErr_Occurred());
}

// The device of the output; false with a Python error set.
bool device_of(PyObject* o, c10::Device* device) {
    if (!THPVariable_Check(o)) {
        PyErr_SetString(PyExc_TypeError, "expected a torch.Tensor");
        return false;
    }
    *device = THPVariable_Unpack(o).device();
    if (!device->is_cuda()) {
        PyErr_SetString(PyExc_ValueError, "all tensors must be CUDA tensors on the same device");
        return false;
    }
    return true;
}

// lora_linear(inputs, weight, bias | None, lora_a, lora_b, out, start, len, idx, batches, max_len, workspace | None) -> status
PyObject* lora_linear(PyObject*, PyObject* const* args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != 12) {
        PyErr_SetString(PyExc_TypeError, "lora_linear takes 12 arguments");
        return nullptr;
    }
    c10::Device device(c10::kCPU);
    if (!device_of(args[5], &device)) return nullptr;
    sgmv_tensor d[9];
    int rc = 0;
    const bool bias = args[2] != Py_None;
    for (int i = 0; i < 9; ++i) {
        if (i == 2 && !bias) continue;
        if (!describe(args[i], device, &d[i], &rc)) return rc < 0 ? PyLong_FromLong(rc) : nullptr;
    }
    int64_t batches = 0, max_len = 0;
    if (!number(args[9], &batches) || !number(args[10], &max_len)) return nullptr;
    void* ws = nullptr;
    size_t ws_bytes = 0;
    if (args[11] != Py_None) {
        if (!THPVariable_Check(args[11])) {
            PyErr_SetString(PyExc_TypeError, "workspace must be a torch.Tensor");
            return nullptr;
        }
        const at::Tensor& t = THPVariable_Unpack(args[11]);
        if (t.device() != device || !t.is_contiguous()) {
            PyErr_SetString(PyExc_ValueError, "workspace must be a contiguous CUDA tensor on the same device");
            return nullptr;
        }
        ws = t.data_ptr();
        ws_bytes = t.nbytes();
    }
    const c10::cuda::CUDAGuard guard(device);
    void* stream = c10::cuda::getCurrentCUDAStream(device.index()).stream();
    // a launch waits where the stream's queue is full: other Python threads run meanwhile
    Py_BEGIN_ALLOW_THREADS
    rc = g_lora(&d[0], &d[1], bias ? &d[2] : nullptr, &d[3], &d[4], &d[5], &d[6], &d[7], &d[8], batches, max_len, ws,
                ws_bytes, stream);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(rc);
    END_HANDLE_TH_ERRORS
}

// grouped_gemm / grouped_wgrad(a, b, out, start, len, idx, batches, max_len, add) -> status
PyObject* grouped(GroupedFn fn, PyObject* const* args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != 9) {
        PyErr_SetString(PyExc_TypeError, "a grouped product takes 9 arguments");
        return nullptr;
    }
    c10::Device device(c10::kCPU);
    if (!device_of(args[2], &device)) return nullptr;
    sgmv_tensor d[6];
    int rc = 0;
    for (int i = 0; i < 6; ++i)
        if (!describe(args[i], device, &d[i], &rc)) return rc < 0 ? PyLong_FromLong(rc) : nullptr;
    int64_t batches = 0, max_len = 0;
    if (!number(args[6], &batches) || !number(args[7], &max_len)) return nullptr;
    const int add = PyObject_IsTrue(args[8]);
    if (add < 0) return nullptr;
    const c10::cuda::CUDAGuard guard(device);
    void* stream = c10::cuda::getCurrentCUDAStream(device.index()).stream();
    Py_BEGIN_ALLOW_THREADS
    rc = fn(&d[0], &d[1], &d[2], &d[3], &d[4], &d[5], batches, max_len, add, stream);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(rc);
    END_HANDLE_TH_ERRORS
}

PyObject* grouped_gemm(PyObject*, PyObject* const* args, Py_ssize_t n) { return grouped(g_gemm, args, n); }
PyObject* grouped_wgrad(PyObject*, PyObject* const* args, Py_ssize_t n) { return grouped(g_wgrad, args, n); }

PyObject* init(PyObject*, PyObject* args) {
    unsigned long long lora, gemm, wgrad;
    if (!PyArg_ParseTuple(args, "KKK", &lora, &gemm, &wgrad)) return nullptr;
    g_lora = reinterpret_cast<LoraFn>(lora);
    g_gemm = reinterpret_cast<GroupedFn>(gemm);
    g_wgrad = reinterpret_cast<GroupedFn>(wgrad);
    Py_RETURN_NONE;
}

PyMethodDef g_methods[] = {
    {"init", init, METH_VARARGS, "addresses of sgmv_lora_linear, sgmv_grouped_gemm and sgmv_grouped_wgrad"},
    {"lora_linear", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(lora_linear)), METH_FASTCALL, nullptr},
    {"grouped_gemm", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(grouped_gemm)), METH_FASTCALL, nullptr},
    {"grouped_wgrad", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(grouped_wgrad)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

// What the extension was compiled for; the build and the loader compare it with what they run on.
PyMODINIT_FUNC PyInit__binding() {
    PyObject* m = PyModule_Create(&g_module);
    if (m && PyModule_AddStringConstant(m, "built_for", BUILT_FOR) < 0) {
        Py_DECREF(m);
        return nullptr;
    }
    return m;
}
