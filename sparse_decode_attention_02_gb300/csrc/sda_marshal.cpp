// Argument marshalling of the Python binding, natively: tensors to the C ABI's
// descriptors, their common device, and the stream a call goes to.  No
// computation happens here.  The serving-step entries (plan_step and those below it) make
// the plain calls from here (all on the current device, a workspace at hand); where
// the binding has to see to something first they answer None, and the call goes
// through ctypes.
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
    case c10::ScalarType::Char: return SDA_DTYPE_INT8;
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

// A plain call's descriptors, workspace and stream.
class Plain {
public:
    sda_tensor *at[11];                         // of the tensors; null: None
    void *workspace = nullptr, *stream = nullptr;
    size_t bytes = 0;

    Plain() = default;
    Plain(const Plain &) = delete;
    ~Plain() { Py_XDECREF(keep_); }

    // args: the entry point's address, the default workspaces by (device, stream),
    // the bytes that the call needs, a workspace or None, then n tensors or None.
    // False: not a plain call, or a Python error is set.
    bool read(PyObject *const *args, int n)
    {
        for (int i = 0; i < n; ++i) {
            PyObject *x = args[4 + i];
            at[i] = nullptr;
            if (x == Py_None)
                continue;
            if (!THPVariable_Check(x)) {
                PyErr_SetString(PyExc_TypeError, "a tensor or None is expected");
                return false;
            }
            const at::Tensor &t = THPVariable_Unpack(x);
            if (!t.is_cuda() || (device_ >= 0 && device_ != t.get_device()))
                return false;
            device_ = t.get_device();
            if (!describe(t, d_[i]))
                return false;
            at[i] = &d_[i];
        }
        if (device_ < 0 || c10::cuda::current_device() != device_)
            return false;
        const cudaStream_t s = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(device_)).stream();
        stream = s;
        if (args[3] != Py_None) {
            if (!THPVariable_Check(args[3])) {
                PyErr_SetString(PyExc_TypeError, "workspace: a tensor or None is expected");
                return false;
            }
            const at::Tensor &w = THPVariable_Unpack(args[3]);
            if (!w.is_cuda() || w.get_device() != device_ || !w.is_contiguous())
                return false;                   // the binding refuses it
            workspace = w.data_ptr();
            bytes = w.nbytes();
            return true;
        }
        cudaStreamCaptureStatus status = cudaStreamCaptureStatusNone;
        if (cudaStreamIsCapturing(s, &status) != cudaSuccess || status != cudaStreamCaptureStatusNone)
            return false;
        PyObject *key = Py_BuildValue("(lK)", static_cast<long>(device_), reinterpret_cast<unsigned long long>(s));
        PyObject *have = key ? PyDict_GetItemWithError(args[1], key) : nullptr;     // (tensor, address, bytes)
        Py_XDECREF(key);
        if (!have || !PyTuple_Check(have) || PyTuple_GET_SIZE(have) != 3)
            return false;
        Py_INCREF(keep_ = have);                // another thread may put a larger one in its place meanwhile
        workspace = PyLong_AsVoidPtr(PyTuple_GET_ITEM(have, 1));
        bytes = PyLong_AsSize_t(PyTuple_GET_ITEM(have, 2));
        const size_t need = PyLong_AsSize_t(args[2]);
        return !PyErr_Occurred() && bytes >= need;
    }

    // A scale: None or a tensor (a number has to be uploaded, and scalar() refuses the rest).
    bool scale(PyObject *x, const float *&out) const
    {
        out = nullptr;
        if (x == Py_None)
            return true;
        if (!THPVariable_Check(x))
            return false;
        const at::Tensor &t = THPVariable_Unpack(x);
        if (t.scalar_type() != c10::ScalarType::Float || t.numel() != 1 || !t.is_cuda() || t.get_device() != device_)
            return false;
        out = static_cast<const float *>(t.data_ptr());
        return true;
    }

private:
    sda_tensor d_[11];
    int device_ = -1;
    PyObject *keep_ = nullptr;
};

bool as_int(PyObject *x, int &out)
{
    const long v = PyLong_AsLong(x);
    out = static_cast<int>(v);
    if (v == -1 && PyErr_Occurred())
        return false;
    if (v != out) {
        PyErr_SetString(PyExc_OverflowError, "an argument does not fit 32 bits");
        return false;
    }
    return true;
}

bool as_float(PyObject *x, float &out)
{
    out = static_cast<float>(PyFloat_AsDouble(x));
    return !PyErr_Occurred();
}

// entry(args) with `count` arguments, or None where `run` says that it is not a plain call.
template <class Run>
PyObject *plain_call(PyObject *const *args, Py_ssize_t n, Py_ssize_t count, Run run)
{
    if (n != count || !PyDict_Check(args[1])) {
        PyErr_SetString(PyExc_TypeError, "entry point, default workspaces, bytes, workspace, tensors, scalars");
        return nullptr;
    }
    void *entry = PyLong_AsVoidPtr(args[0]);
    if (!entry) {
        if (!PyErr_Occurred())
            PyErr_SetString(PyExc_ValueError, "no entry point");
        return nullptr;
    }
    sda_status status = SDA_OK;
    try {
        if (!run(entry, status)) {
            if (PyErr_Occurred())
                return nullptr;
            Py_RETURN_NONE;
        }
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
    return PyLong_FromLong(status);
}

// The entry point at `entry`, called without the interpreter's lock.
template <class Entry, class... Args>
sda_status call(void *entry, Args... args)
{
    PyThreadState *state = PyEval_SaveThread();
    const sda_status status = reinterpret_cast<Entry *>(entry)(args...);
    PyEval_RestoreThread(state);
    return status;
}

// tensors: context_lens, new_lens, free_pages, free_state, free_next, block_table,
// seq_lens, token_starts, slots, positions, requests; block_size, rows_per_request
PyObject *plan_step(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    return plain_call(args, n, 17, [&](void *entry, sda_status &status) {
        Plain c;
        int block, per_request;
        if (!c.read(args, 11) || !as_int(args[15], block) || !as_int(args[16], per_request))
            return false;
        status = call<decltype(sparse_decode_plan_step)>(entry, c.at[0], c.at[1], block, per_request, c.at[2], c.at[3], c.at[4],
                      c.at[5], c.at[6], c.at[7], c.at[8], c.at[9], c.at[10], c.workspace, c.bytes, c.stream);
        return true;
    });
}

// tensors: query, query_out, key, value, positions, inv_freq, slots, cache; sections
// (None or up to four), interleaved_axes, adjacent_pairs, amplitude, k_scale, v_scale
PyObject *rope_append(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    return plain_call(args, n, 18, [&](void *entry, sda_status &status) {
        Plain c;
        int32_t sections[4] = {0, 0, 0, 0};
        float amplitude;
        const float *ks, *vs;
        if (!c.read(args, 8) || !c.scale(args[16], ks) || !c.scale(args[17], vs) || !as_float(args[15], amplitude))
            return false;
        if (args[12] != Py_None) {
            const Py_ssize_t axes = PySequence_Size(args[12]);
            if (axes < 0 || axes > 4)
                return false;
            for (Py_ssize_t i = 0; i < axes; ++i) {
                PyObject *x = PySequence_GetItem(args[12], i);
                const bool ok = x && as_int(x, sections[i]);
                Py_XDECREF(x);
                if (!ok)
                    return false;
            }
        }
        const int interleaved = PyObject_IsTrue(args[13]), adjacent = PyObject_IsTrue(args[14]);
        if (interleaved < 0 || adjacent < 0)
            return false;
        status = call<decltype(sparse_decode_rope_append)>(entry, c.at[0], c.at[1], c.at[2], c.at[3], c.at[4], c.at[5],
                      args[12] == Py_None ? nullptr : sections, interleaved, adjacent, amplitude, c.at[6], c.at[7], ks, vs,
                      c.workspace, c.bytes, c.stream);
        return true;
    });
}

// tensors: query, cache, block_table, seq_lens, output, lse, gate; scale, query_len,
// k_scale, v_scale
PyObject *paged_attention(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    return plain_call(args, n, 15, [&](void *entry, sda_status &status) {
        Plain c;
        float scale;
        int query_len;
        const float *ks, *vs;
        if (!c.read(args, 7) || !c.scale(args[13], ks) || !c.scale(args[14], vs) || !as_float(args[11], scale) ||
            !as_int(args[12], query_len))
            return false;
        status = call<decltype(sparse_decode_paged_attention)>(entry, c.at[0], c.at[1], c.at[2], c.at[3], c.at[4], c.at[5], scale,
                      query_len, ks, vs, c.at[6], c.workspace, c.bytes, c.stream);
        return true;
    });
}

// tensors: key, value, slots, cache, scales
PyObject *quantised_append(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    return plain_call(args, n, 9, [&](void *entry, sda_status &status) {
        Plain c;
        if (!c.read(args, 5))
            return false;
        status = call<decltype(sparse_decode_quantised_append)>(entry, c.at[0], c.at[1], c.at[2], c.at[3], c.at[4], c.workspace,
                      c.bytes, c.stream);
        return true;
    });
}

// tensors: cache, scales, block_table, token_starts, first_tokens, key, value
PyObject *quantised_read(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    return plain_call(args, n, 11, [&](void *entry, sda_status &status) {
        Plain c;
        if (!c.read(args, 7))
            return false;
        status = call<decltype(sparse_decode_quantised_read)>(entry, c.at[0], c.at[1], c.at[2], c.at[3], c.at[4], c.at[5], c.at[6],
                      c.workspace, c.bytes, c.stream);
        return true;
    });
}

// tensors: query, cache, scales, block_table, seq_lens, output, lse, gate; scale, query_len
PyObject *quantised_paged_attention(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    return plain_call(args, n, 14, [&](void *entry, sda_status &status) {
        Plain c;
        float scale;
        int query_len;
        if (!c.read(args, 8) || !as_float(args[12], scale) || !as_int(args[13], query_len))
            return false;
        status = call<decltype(sparse_decode_quantised_paged_attention)>(entry, c.at[0], c.at[1], c.at[2], c.at[3], c.at[4],
                      c.at[5], c.at[6], scale, query_len, c.at[7], c.workspace, c.bytes, c.stream);
        return true;
    });
}

// tensors: query, cache, scales, regions, block_table, positions, active, output, lse, gate;
// scale, query_len, clear_inactive, region_tokens
PyObject *quantised_attention(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    return plain_call(args, n, 18, [&](void *entry, sda_status &status) {
        Plain c;
        float scale;
        int query_len, region_tokens;
        if (!c.read(args, 10) || !as_float(args[14], scale) || !as_int(args[15], query_len) || !as_int(args[17], region_tokens))
            return false;
        const int clear = PyObject_IsTrue(args[16]);
        if (clear < 0)
            return false;
        status = call<decltype(sparse_decode_quantised_attention)>(entry, c.at[0], c.at[1], c.at[2], c.at[3], c.at[4], c.at[5],
                      c.at[6], c.at[7], c.at[8], scale, query_len, c.at[9], clear, region_tokens, c.workspace, c.bytes, c.stream);
        return true;
    });
}

PyMethodDef methods[] = {
    {"pack", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(pack)), METH_FASTCALL, nullptr},
    {"scalar", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(scalar)), METH_FASTCALL, nullptr},
    {"plan_step", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(plan_step)), METH_FASTCALL, nullptr},
    {"rope_append", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(rope_append)), METH_FASTCALL, nullptr},
    {"paged_attention", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(paged_attention)), METH_FASTCALL, nullptr},
    {"quantised_append", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(quantised_append)), METH_FASTCALL, nullptr},
    {"quantised_read", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(quantised_read)), METH_FASTCALL, nullptr},
    {"quantised_paged_attention", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(quantised_paged_attention)),
     METH_FASTCALL, nullptr},
    {"quantised_attention", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(quantised_attention)), METH_FASTCALL,
     nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal(void)
{
    return PyModule_Create(&module);
}
