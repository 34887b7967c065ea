// Argument marshalling of the Python binding, natively: tensors to the C ABI's
// descriptors, their common device, and the stream a call goes to.  No
// computation happens here; the entry points are called through ctypes.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstring>
#include <exception>

#include "sdattn.h"

namespace {

constexpr long kNoTensor = -1, kNotCuda = -2, kMixed = -3;

int code_of(c10::ScalarType t)
{
    switch (t) {
    case c10::ScalarType::BFloat16: return SDA_DTYPE_BF16;
    case c10::ScalarType::Float8_e4m3fn: return SDA_DTYPE_FP8_E4M3;
    case c10::ScalarType::Byte: return SDA_DTYPE_UINT8;
    case c10::ScalarType::Int: return SDA_DTYPE_INT32;
    case c10::ScalarType::Bool: return SDA_DTYPE_BOOL;
    case c10::ScalarType::Float: return SDA_DTYPE_FP32;
    case c10::ScalarType::Long: return SDA_DTYPE_INT64;
    default: return 0;
    }
}

// False with a Python error set where `t` cannot be described.
bool describe(const at::Tensor &t, sda_tensor &d)
{
    std::memset(&d, 0, sizeof d);
    const int code = code_of(t.scalar_type());
    if (!code) {
        PyErr_Format(PyExc_TypeError, "unsupported dtype %s", c10::toString(t.scalar_type()));
        return false;
    }
    if (t.dim() > 4) {
        PyErr_SetString(PyExc_ValueError, "at most 4 dimensions");
        return false;
    }
    d.data = t.numel() ? t.data_ptr() : nullptr;
    d.dtype = code;
    d.ndim = static_cast<int32_t>(t.dim());
    for (int64_t i = 0; i < t.dim(); ++i) {
        d.shape[i] = t.size(i);
        d.stride[i] = t.stride(i);
    }
    return true;
}

// pack(*tensors or None) -> (memory, addresses, device, on_current_device, stream,
// capturing: whether the stream is being captured)
// The descriptors lie in `memory`, which the caller keeps until its call has
// returned; None has address None.  device < 0: no CUDA device in common.
PyObject *pack(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    PyObject *memory = PyBytes_FromStringAndSize(nullptr, n * static_cast<Py_ssize_t>(sizeof(sda_tensor)));
    PyObject *where = memory ? PyTuple_New(n) : nullptr;
    if (!where) {
        Py_XDECREF(memory);
        return nullptr;
    }
    sda_tensor *out = reinterpret_cast<sda_tensor *>(PyBytes_AS_STRING(memory));
    long device = kNoTensor, current = 0, capturing = 0;
    unsigned long long stream = 0;
    try {
        for (Py_ssize_t i = 0; i < n; ++i) {
            PyObject *slot = Py_None;
            if (args[i] == Py_None) {
                Py_INCREF(slot);
            } else {
                if (!THPVariable_Check(args[i])) {
                    PyErr_SetString(PyExc_TypeError, "a tensor or None is expected");
                    throw std::exception();
                }
                const at::Tensor &t = THPVariable_Unpack(args[i]);
                const long dev = t.is_cuda() ? static_cast<long>(t.get_device()) : kNotCuda;
                device = device == kNoTensor || device == dev ? dev : kMixed;
                if (dev >= 0 && !describe(t, out[i]))
                    throw std::exception();
                slot = PyLong_FromVoidPtr(out + i);
                if (!slot)
                    throw std::exception();
            }
            PyTuple_SET_ITEM(where, i, slot);
        }
        if (device >= 0) {
            const cudaStream_t s = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(device)).stream();
            stream = reinterpret_cast<unsigned long long>(s);
            cudaStreamCaptureStatus status = cudaStreamCaptureStatusNone;
            capturing = cudaStreamIsCapturing(s, &status) != cudaSuccess || status != cudaStreamCaptureStatusNone;
            current = c10::cuda::current_device() == device;
        }
    } catch (const std::exception &e) {
        if (!PyErr_Occurred())
            PyErr_SetString(PyExc_RuntimeError, e.what());
        Py_DECREF(where);
        Py_DECREF(memory);
        return nullptr;
    }
    return Py_BuildValue("(NNllKl)", memory, where, device, current, stream, capturing);
}

// scalar(tensor, device) -> address of a one-element float32 tensor on that device.
PyObject *scalar(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    if (n != 2 || !THPVariable_Check(args[0])) {
        PyErr_SetString(PyExc_TypeError, "scalar(tensor, device)");
        return nullptr;
    }
    const long device = PyLong_AsLong(args[1]);
    if (device == -1 && PyErr_Occurred())
        return nullptr;
    try {
        const at::Tensor &t = THPVariable_Unpack(args[0]);
        if (t.scalar_type() != c10::ScalarType::Float || t.numel() != 1 || !t.is_cuda() || t.get_device() != device) {
            PyErr_SetString(PyExc_ValueError,
                            "k_scale / v_scale must be one-element float32 tensors on the query's device");
            return nullptr;
        }
        return PyLong_FromVoidPtr(t.data_ptr());
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}

PyMethodDef methods[] = {
    {"pack", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(pack)), METH_FASTCALL, nullptr},
    {"scalar", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(scalar)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal(void)
{
    return PyModule_Create(&module);
}
