// ecmd_binding.cpp -- the part of the Python binding that is worth compiling:
// torch tensors to cmd_arg structures (a Python extension module, _binding).
//
//   pack(ranks, *tensors) -> (cmd_args, device, stream)
//   scratch(bytes, device) -> (pointer, owner)
//   wrote(*tensors)
//
// cmd_args holds one structure for each tensor, in order: the tensor of the
// rank that its byte of `ranks` says; another rank is packed with sizes that the
// library refuses; None gives kind 0.  device is the GPU that holds every tensor
// if that is the current one, else -1; stream its current stream's handle (0
// without one).  Reading four attributes of each tensor from Python takes
// about 1 us a tensor, as long as the kernels of a small call; this takes 0.1.
// scratch is an uninitialised tensor of that many bytes on that GPU and its address.
// wrote advances the tensors' version counters (None: nothing), as torch's own
// in-place operations do, so that a backward pass that saved one of them notices.
#include <Python.h>

#include <c10/hip/HIPFunctions.h>
#include <ATen/ATen.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/ecmd_serving.h"

namespace {

int32_t code(at::ScalarType t)
{
    switch (t) {
    case at::kHalf: return CMD_F16;
    case at::kFloat: return CMD_F32;
    case at::kInt: return CMD_I32;
    case at::kBFloat16: return CMD_BF16;
    case at::kDouble: return CMD_F64;
    default: return 0;
    }
}

PyObject *pack_tensors(PyObject *const *args, Py_ssize_t n)
{
    if (n < 1 || !PyBytes_Check(args[0]) || PyBytes_GET_SIZE(args[0]) != n - 1) {
        PyErr_SetString(PyExc_TypeError, "pack(ranks, *tensors): one byte of ranks for each tensor");
        return nullptr;
    }
    const char *ranks = PyBytes_AS_STRING(args[0]);
    PyObject *out = PyBytes_FromStringAndSize(nullptr, (n - 1) * (Py_ssize_t)sizeof(cmd_arg));
    if (!out) return nullptr;
    cmd_arg *a = (cmd_arg *)PyBytes_AS_STRING(out);
    memset(static_cast<void *>(a), 0, (n - 1) * sizeof(cmd_arg));
    int64_t device = -2;   // none seen yet
    for (Py_ssize_t i = 1; i < n; ++i, ++a, ++ranks) {
        if (args[i] == Py_None) continue;
        if (!THPVariable_Check(args[i])) {
            Py_DECREF(out);
            PyErr_Format(PyExc_TypeError, "a torch.Tensor expected, got %s", Py_TYPE(args[i])->tp_name);
            return nullptr;
        }
        const at::Tensor &t = THPVariable_Unpack(args[i]);
        if (t.layout() != at::kStrided) {
            Py_DECREF(out);
            PyErr_SetString(PyExc_TypeError, "a strided tensor expected");
            return nullptr;
        }
        if (t.is_neg()) {   // its memory holds the opposite numbers
            Py_DECREF(out);
            PyErr_SetString(PyExc_TypeError, "a tensor with the negative bit set (resolve_neg() makes one without)");
            return nullptr;
        }
        const int64_t on = t.is_cuda() ? t.get_device() : -1;
        device = device == -2 || device == on ? on : -1;
        a->kind = CMD_ARG_TENSOR;
        a->dtype = code(t.scalar_type());
        a->ptr = t.mutable_data_ptr();
        if (t.dim() == *ranks) {
            for (int k = 0; k < *ranks; ++k) {
                a->size[k] = t.size(k);
                a->stride[k] = t.stride(k);
            }
        } else {
            for (int k = 0; k < 4; ++k) a->size[k] = -1;
        }
    }
    void *stream = nullptr;
    if (device >= 0) {
        if (device == c10::hip::current_device()) stream = c10::hip::getCurrentHIPStream((c10::DeviceIndex)device).stream();
        else device = -1;
    } else {
        device = -1;
    }
    return Py_BuildValue("(NLK)", out, (long long)device, (unsigned long long)(uintptr_t)stream);
}

PyObject *pack(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    try {
        return pack_tensors(args, n);
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}

PyObject *scratch(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    try {
        if (n != 2) {
            PyErr_SetString(PyExc_TypeError, "scratch(bytes, device)");
            return nullptr;
        }
        const long long size = PyLong_AsLongLong(args[0]), device = PyLong_AsLongLong(args[1]);
        if (PyErr_Occurred()) return nullptr;
        at::Tensor t = at::empty({(int64_t)size},
                                 at::TensorOptions().dtype(at::kByte).device(at::kCUDA, (c10::DeviceIndex)device));
        const unsigned long long at = (unsigned long long)(uintptr_t)t.mutable_data_ptr();
        return Py_BuildValue("(KN)", at, THPVariable_Wrap(std::move(t)));
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}

PyObject *wrote(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    try {
        for (Py_ssize_t i = 0; i < n; ++i) {
            if (args[i] == Py_None) continue;
            if (!THPVariable_Check(args[i])) {
                PyErr_Format(PyExc_TypeError, "a torch.Tensor expected, got %s", Py_TYPE(args[i])->tp_name);
                return nullptr;
            }
            const at::Tensor &t = THPVariable_Unpack(args[i]);
            if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();   // inference tensors have none
        }
        Py_RETURN_NONE;
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}

PyMethodDef methods[] = {
    {"scratch", (PyCFunction)(void (*)(void))scratch, METH_FASTCALL, "scratch(bytes, device) -> (pointer, owner)"},
    {"wrote", (PyCFunction)(void (*)(void))wrote, METH_FASTCALL, "wrote(*tensors): advances their version counters"},
    {"pack", (PyCFunction)(void (*)(void))pack, METH_FASTCALL, "pack(ranks, *tensors) -> (cmd_args, device, stream)"},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", "torch tensors to cmd_arg structures", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding(void) { return PyModule_Create(&module); }
