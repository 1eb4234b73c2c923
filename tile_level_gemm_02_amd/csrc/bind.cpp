// Marshalling of tg_clip_grads, tg_adamw and the int8 layers for Python: reads
// the tensors (their types, sizes, devices and pointers) in C++.  Read one
// attribute at a time from Python they take about 0.5 us each tensor, 72 us for
// 56 gradients with their outputs, several times the kernels of a small call; a
// token through an int8 layer is 8 us of kernels and was 14 of marshalling.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <torch/csrc/autograd/python_variable.h>

#include <vector>

#include "tg_int8.h"
#include "tg_ops.h"
#include "tg_train.h"

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

// tg_dtype of an element type, or -1
int c_dtype(at::ScalarType s) { return s == at::kFloat ? TG_F32 : s == at::kHalf ? TG_F16 : s == at::kBFloat16 ? TG_BF16 : -1; }

// a tensor of one element of type `type` on GPU `dev`: its pointer, else null with an error set
const void* scalar_on(PyObject* o, int64_t dev, at::ScalarType type, const char* what)
{
    const at::Tensor* t = contiguous_on(o, dev, what);
    if (t == nullptr)
        return nullptr;
    if (t->scalar_type() != type || t->numel() != 1) {
        PyErr_Format(PyExc_ValueError, "%s must be a %s tensor of one element", what, type == at::kLong ? "int64" : "float32");
        return nullptr;
    }
    return t->data_ptr();
}

typedef tg_status (*adamw_fn)(int64_t, const tg_adamw_tensor*, int64_t, double, double, double, double, double, const float*, float,
                              const int64_t*, const float*, void*);

// adamw(function address, params, grads, exp_avg, exp_avg_sq, masters or None, their scales or None twice, step, lr, beta1,
//       beta2, eps, weight decay, norm or None, max_norm, device index, stream) -> status
PyObject* adamw(PyObject*, PyObject* args)
{
    unsigned long long fn, stream;
    PyObject *list[7], *step_o, *lr_o, *norm;
    double beta1, beta2, eps, decay;
    float max_norm;
    long long dev;
    if (!PyArg_ParseTuple(args, "KO!O!O!O!OOOOOddddOfLK", &fn, &PyList_Type, &list[0], &PyList_Type, &list[1], &PyList_Type, &list[2],
                          &PyList_Type, &list[3], &list[4], &list[5], &list[6], &step_o, &lr_o, &beta1, &beta2, &eps, &decay, &norm,
                          &max_norm, &dev, &stream))
        return nullptr;
    const Py_ssize_t n = PyList_GET_SIZE(list[0]);
    for (int k = 1; k < 7; ++k)
        if (list[k] != Py_None && (!PyList_Check(list[k]) || PyList_GET_SIZE(list[k]) != n))
            return refuse("every list must hold a tensor for each parameter");
    if ((list[5] == Py_None) != (list[6] == Py_None))
        return refuse("exp_avg_scales and exp_avg_sq_scales come together");
    const bool eight = list[5] != Py_None;
    try {
        std::vector<tg_adamw_tensor> t(n);
        for (Py_ssize_t i = 0; i < n; ++i) {
            static const char* const names[7] = {"params", "grads", "exp_avg", "exp_avg_sq", "masters", "exp_avg_scales", "exp_avg_sq_scales"};
            void* at[7] = {};
            int type[2] = {};
            int64_t size = 0;
            for (int k = 0; k < 7; ++k) {
                if (list[k] == Py_None)
                    continue;
                const at::Tensor* x = contiguous_on(PyList_GET_ITEM(list[k], i), dev, names[k]);
                if (x == nullptr)
                    return nullptr;
                if (k < 2) {
                    type[k] = c_dtype(x->scalar_type());
                    if (type[k] < 0)
                        return refuse("params and grads must be float32, float16 or bfloat16");
                } else if (x->scalar_type() != (eight && k < 4 ? at::kFloat8_e4m3fn : at::kFloat)) {
                    PyErr_Format(PyExc_ValueError, "%s must be %s", names[k], eight && k < 4 ? "float8_e4m3fn beside scales" : "float32");
                    return nullptr;
                }
                if (k == 0)
                    size = x->numel();
                if (x->numel() != (k < 5 ? size : (size + 255) / 256)) {
                    PyErr_Format(PyExc_ValueError, "%s must match the parameter's size", names[k]);
                    return nullptr;
                }
                at[k] = x->data_ptr();
            }
            if (at[4] != nullptr && type[0] == TG_F32)
                return refuse("masters go with 16-bit params");
            t[i] = tg_adamw_tensor{at[0], (float*)at[4], at[1], at[2], at[3], (float*)at[5], (float*)at[6], size, type[0], type[1]};
        }
        const void *pn = nullptr, *ps = nullptr, *pl = nullptr;
        long long step = 1;
        double lr = 0.0;
        if (norm != Py_None && (pn = scalar_on(norm, dev, at::kFloat, "the norm")) == nullptr)
            return nullptr;
        if (THPVariable_Check(step_o)) {
            if ((ps = scalar_on(step_o, dev, at::kLong, "step")) == nullptr)
                return nullptr;
        } else {
            step = PyLong_AsLongLong(step_o);
            if (step == -1 && PyErr_Occurred())
                return nullptr;
        }
        if (THPVariable_Check(lr_o)) {
            if ((pl = scalar_on(lr_o, dev, at::kFloat, "lr")) == nullptr)
                return nullptr;
        } else {
            lr = PyFloat_AsDouble(lr_o);
            if (lr == -1.0 && PyErr_Occurred())
                return nullptr;
        }
        const tg_status st = ((adamw_fn)(uintptr_t)fn)(n, t.data(), step, lr, beta1, beta2, eps, decay, (const float*)pn, max_norm,
                                                       (const int64_t*)ps, (const float*)pl, (void*)(uintptr_t)stream);
        return PyLong_FromLong((long)st);
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}

// A matrix argument: the strides and devices that ops.py's _mat takes
struct Mat {
    void* p = nullptr;
    int64_t rows = 0, cols = 0, ld = 0;
    at::ScalarType type = at::kFloat;
};

bool matrix(PyObject* o, const char* name, int64_t dev, Mat& m)
{
    if (!THPVariable_Check(o)) {
        PyErr_Format(PyExc_ValueError, "%s must be a tensor", name);
        return false;
    }
    const at::Tensor& t = THPVariable_Unpack(o);
    if (t.dim() != 2) {
        PyErr_Format(PyExc_ValueError, "%s must be 2-D", name);
        return false;
    }
    m.rows = t.size(0);
    m.cols = t.size(1);
    m.type = t.scalar_type();
    if (t.stride(1) != 1 && m.cols > 1) {
        PyErr_Format(PyExc_ValueError, "%s must have unit stride along its last dimension", name);
        return false;
    }
    if (!t.is_cuda() || t.get_device() != dev) {
        PyErr_Format(PyExc_ValueError, "every tensor must be on the current GPU, %s is not", name);
        return false;
    }
    // one row has no second one: its stride is not looked at, an aligned one stands for it
    m.ld = m.rows > 1 ? t.stride(0) : (m.cols + 15) & -16;
    m.p = t.data_ptr();
    return true;
}

bool shaped(const Mat& m, const char* name, int64_t rows, int64_t cols)
{
    if (m.rows == rows && m.cols == cols)
        return true;
    PyErr_Format(PyExc_ValueError, "%s must be %lldx%lld, got %lldx%lld", name, (long long)rows, (long long)cols, (long long)m.rows,
                 (long long)m.cols);
    return false;
}

bool typed(const Mat& m, const char* name, at::ScalarType type, const char* what)
{
    if (m.type == type)
        return true;
    PyErr_Format(PyExc_ValueError, "%s must be %s", name, what);
    return false;
}

// a contiguous float32 vector of n
bool vector(PyObject* o, const char* name, int64_t n, int64_t dev, float*& p)
{
    if (THPVariable_Check(o)) {
        const at::Tensor& t = THPVariable_Unpack(o);
        if (t.scalar_type() == at::kFloat && t.dim() == 1 && t.size(0) == n && t.is_contiguous()) {
            if (!t.is_cuda() || t.get_device() != dev) {
                PyErr_Format(PyExc_ValueError, "every tensor must be on the current GPU, %s is not", name);
                return false;
            }
            p = (float*)t.data_ptr();
            return true;
        }
    }
    PyErr_Format(PyExc_ValueError, "%s must be a contiguous float32 vector of %lld", name, (long long)n);
    return false;
}

typedef tg_status (*quantize_fn)(int, int64_t, int64_t, const void*, int64_t, int8_t*, int64_t, float*, void*);

// quantize_i8(function address, x, q, scale, device index, stream) -> status
PyObject* quantize_i8(PyObject*, PyObject* args)
{
    unsigned long long fn, stream;
    PyObject *x_o, *q_o, *scale_o;
    long long dev;
    if (!PyArg_ParseTuple(args, "KOOOLK", &fn, &x_o, &q_o, &scale_o, &dev, &stream))
        return nullptr;
    try {
        Mat x, q;
        float* scale = nullptr;
        if (!matrix(x_o, "x", dev, x))
            return nullptr;
        if (c_dtype(x.type) < 0)
            return refuse("x must be float32, float16 or bfloat16");
        if (!matrix(q_o, "q", dev, q) || !typed(q, "q", at::kChar, "int8") || !shaped(q, "q", x.rows, x.cols) ||
            !vector(scale_o, "scale", x.rows, dev, scale))
            return nullptr;
        return PyLong_FromLong((long)((quantize_fn)(uintptr_t)fn)(c_dtype(x.type), x.rows, x.cols, x.p, x.ld, (int8_t*)q.p, q.ld, scale,
                                                                  (void*)(uintptr_t)stream));
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}

typedef tg_status (*linear_i8_fn)(int64_t, int64_t, int64_t, const int8_t*, int64_t, const int8_t*, int64_t, const float*, const float*,
                                  const float*, int, const void*, int64_t, void*, int64_t, int, void*, int64_t, void*);

// linear_i8(function address, x, W, Y, scale_x, scale_w, bias or None, act, residual or None, workspace or None, device index,
//           stream) -> status
PyObject* linear_i8(PyObject*, PyObject* args)
{
    unsigned long long fn, stream;
    PyObject *x_o, *w_o, *y_o, *sx_o, *sw_o, *b_o, *r_o, *ws_o;
    int act;
    long long dev;
    if (!PyArg_ParseTuple(args, "KOOOOOOiOOLK", &fn, &x_o, &w_o, &y_o, &sx_o, &sw_o, &b_o, &act, &r_o, &ws_o, &dev, &stream))
        return nullptr;
    try {
        Mat x, w, y, r;
        float *sx = nullptr, *sw = nullptr, *b = nullptr;
        if (!matrix(x_o, "x", dev, x) || !typed(x, "x", at::kChar, "int8") || !matrix(w_o, "W", dev, w) ||
            !typed(w, "W", at::kChar, "int8") || !shaped(w, "W", w.rows, x.cols) || !matrix(y_o, "Y", dev, y) ||
            !shaped(y, "Y", x.rows, w.rows))
            return nullptr;
        if (c_dtype(y.type) < 0)
            return refuse("Y must be float32, float16 or bfloat16");
        if (!vector(sx_o, "scale_x", x.rows, dev, sx) || !vector(sw_o, "scale_w", w.rows, dev, sw) ||
            (b_o != Py_None && !vector(b_o, "bias", w.rows, dev, b)))
            return nullptr;
        if (r_o != Py_None && (!matrix(r_o, "residual", dev, r) || !typed(r, "residual", y.type, "of Y's type") ||
                               !shaped(r, "residual", x.rows, w.rows)))
            return nullptr;
        void* ws = nullptr;
        int64_t ws_bytes = 0;
        if (ws_o != Py_None) {
            const at::Tensor* t = contiguous_on(ws_o, dev, "the workspace");
            if (t == nullptr)
                return nullptr;
            ws = t->data_ptr();
            ws_bytes = (int64_t)t->nbytes();
        }
        return PyLong_FromLong((long)((linear_i8_fn)(uintptr_t)fn)(x.rows, w.rows, x.cols, (const int8_t*)x.p, x.ld, (const int8_t*)w.p, w.ld,
                                                                   sx, sw, b, act, r.p, r.ld, y.p, y.ld, c_dtype(y.type), ws, ws_bytes,
                                                                   (void*)(uintptr_t)stream));
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}

PyMethodDef methods[] = {{"clip_grads", clip_grads, METH_VARARGS, "Marshals a tg_clip_grads call; returns its status."},
                         {"adamw", adamw, METH_VARARGS, "Marshals a tg_adamw call; returns its status."},
                         {"quantize_i8", quantize_i8, METH_VARARGS, "Marshals a tg_quantize_i8 call; returns its status."},
                         {"linear_i8", linear_i8, METH_VARARGS, "Marshals a tg_linear_i8 call; returns its status."},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_tgbind", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__tgbind(void) { return PyModule_Create(&module); }
