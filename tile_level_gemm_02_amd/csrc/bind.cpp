// Marshalling of tg_clip_grads for Python: reads the tensors of a list (their
// types, sizes, devices and pointers) in C++.  Read one attribute at a time
// from Python they take about 0.5 us each tensor, 72 us for 56 gradients with
// their outputs, several times the kernels of a small call.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <torch/csrc/autograd/python_variable.h>

#include <vector>

#include "tg_ops.h"

namespace {

typedef tg_status (*clip_fn)(int64_t, const void* const*, void* const*, const int64_t*, const int32_t*, float, float, float*,
                             void*, int64_t, void*);

PyObject* refuse(const char* what)
{
    PyErr_SetString(PyExc_ValueError, what);
    return nullptr;
}

// the tensor in `o` if it is a contiguous one on GPU `dev`, else null with an error set
const at::Tensor* contiguous_on(PyObject* o, int64_t dev, const char* what)
{
    if (!THPVariable_Check(o)) {
        PyErr_Format(PyExc_ValueError, "%s must be tensors", what);
        return nullptr;
    }
    const at::Tensor& t = THPVariable_Unpack(o);
    if (!t.is_contiguous()) {
        PyErr_Format(PyExc_ValueError, "%s must be contiguous", what);
        return nullptr;
    }
    if (!t.is_cuda() || t.get_device() != dev) {
        PyErr_Format(PyExc_ValueError, "every tensor must be on the current GPU, one of %s is not", what);
        return nullptr;
    }
    return &t;
}

// clip_grads(function address, grads list, outs list or None, max_norm, eps, norm or None, device index,
//            workspace address, workspace bytes, stream) -> status
PyObject* clip_grads(PyObject*, PyObject* args)
{
    unsigned long long fn, ws, stream;
    PyObject *grads, *outs, *norm;
    float max_norm, eps;
    long long dev, ws_bytes;
    if (!PyArg_ParseTuple(args, "KO!OffOLKLK", &fn, &PyList_Type, &grads, &outs, &max_norm, &eps, &norm, &dev, &ws, &ws_bytes,
                          &stream))
        return nullptr;
    const Py_ssize_t n = PyList_GET_SIZE(grads);
    if (outs != Py_None && (!PyList_Check(outs) || PyList_GET_SIZE(outs) != n))
        return refuse("out must hold a tensor for each gradient");
    try {
        std::vector<const void*> in(n);
        std::vector<void*> out(n);
        std::vector<int64_t> size(n);
        std::vector<int32_t> type(n);
        for (Py_ssize_t i = 0; i < n; ++i) {
            const at::Tensor* g = contiguous_on(PyList_GET_ITEM(grads, i), dev, "gradients");
            if (g == nullptr)
                return nullptr;
            const auto t = g->scalar_type();
            if (t != at::kFloat && t != at::kHalf && t != at::kBFloat16)
                return refuse("gradients must be float32, float16 or bfloat16");
            type[i] = t == at::kFloat ? TG_F32 : t == at::kHalf ? TG_F16 : TG_BF16;
            size[i] = g->numel();
            in[i] = out[i] = g->data_ptr();
            if (outs != Py_None) {
                const at::Tensor* o = contiguous_on(PyList_GET_ITEM(outs, i), dev, "outputs");
                if (o == nullptr)
                    return nullptr;
                if (o->scalar_type() != t || o->sizes() != g->sizes())
                    return refuse("each out must be a tensor like its gradient");
                out[i] = o->data_ptr();
            }
        }
        float* pn = nullptr;
        if (norm != Py_None) {
            const at::Tensor* t = contiguous_on(norm, dev, "the norm");
            if (t == nullptr)
                return nullptr;
            if (t->scalar_type() != at::kFloat || t->numel() != 1)
                return refuse("norm must be a float32 tensor of one element");
            pn = (float*)t->data_ptr();
        }
        const tg_status st = ((clip_fn)(uintptr_t)fn)(n, in.data(), out.data(), size.data(), type.data(), max_norm, eps, pn,
                                                      (void*)(uintptr_t)ws, ws_bytes, (void*)(uintptr_t)stream);
        return PyLong_FromLong((long)st);
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}

PyMethodDef methods[] = {{"clip_grads", clip_grads, METH_VARARGS, "Marshals a tg_clip_grads call; returns its status."},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_tgbind", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__tgbind(void) { return PyModule_Create(&module); }
