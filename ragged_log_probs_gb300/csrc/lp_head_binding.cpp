// Python binding of the head operators (include/lp_head.h): checks of the tensors, and the
// call. Compiled, because these calls are made once a token: the same checks in Python took
// 6 us of a call of 8 (a norm of one token), a launch takes under 2.
//
// The functions take their arguments by position (ragged_log_probs_gb300/head.py has the
// signatures) and launch on the current stream of the current device.
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/DynamicTypes.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>
#include <string>

#include "lp_head.h"

namespace {

PyObject* g_failed = nullptr;  // called with (code, function name); raises

struct Refused {};  // a Python error has been set

[[noreturn]] void refuse(PyObject* type, const std::string& text) {
    PyErr_SetString(type, text.c_str());
    throw Refused();
}

uint32_t dtype_code(c10::ScalarType t) {
    switch (t) {
        case c10::ScalarType::Float: return LP_F32;
        case c10::ScalarType::BFloat16: return LP_BF16;
        case c10::ScalarType::Half: return LP_F16;
        case c10::ScalarType::Float8_e4m3fn: return LP_E4M3;
        default: return 99;  // refused by the library
    }
}
std::string dims(const at::Tensor& t) {
    std::string s = "[";
    for (int64_t i = 0; i < t.dim(); ++i) s += (i ? ", " : "") + std::to_string(t.size(i));
    return s + "]";
}

struct Call {
    mutable int current = -1;
    int device() const {  // (asked once a call, and not before a tensor is known to be on a GPU)
        if (current < 0) current = c10::cuda::current_device();
        return current;
    }

    const at::Tensor& tensor(PyObject* o, const char* name) const {
        if (!THPVariable_Check(o)) refuse(PyExc_TypeError, std::string(name) + " must be a CUDA tensor");
        const at::Tensor& t = THPVariable_Unpack(o);
        if (!t.is_cuda()) refuse(PyExc_TypeError, std::string(name) + " must be a CUDA tensor");
        if (t.get_device() != device())
            refuse(PyExc_ValueError, std::string(name) + " is on cuda:" + std::to_string(t.get_device()) +
                                         ", the current device is cuda:" + std::to_string(device()));
        return t;
    }
    const at::Tensor& two_dims(PyObject* o, const char* name) const {
        const at::Tensor& t = tensor(o, name);
        if (t.dim() != 2)
            refuse(PyExc_ValueError, std::string(name) + " must be 2-D, has " + std::to_string(t.dim()) + " dimensions");
        return t;
    }

    // A 2-D tensor whose last dimension is contiguous: its pointer and row stride.
    struct Matrix {
        void* ptr = nullptr;
        uint64_t stride = 0;
    };
    Matrix matrix(const at::Tensor& t, const char* name, int64_t rows, int64_t cols, c10::ScalarType type) const {
        if (t.dim() != 2 || t.size(0) != rows || t.size(1) != cols)
            refuse(PyExc_ValueError, std::string(name) + " must be [" + std::to_string(rows) + ", " +
                                         std::to_string(cols) + "], is " + dims(t));
        if (t.scalar_type() != type)
            refuse(PyExc_TypeError, std::string(name) + " must be " + c10::toString(type) + ", is " +
                                        c10::toString(t.scalar_type()));
        if (t.stride(1) != 1 && cols > 1)
            refuse(PyExc_ValueError, std::string(name) + "'s last dimension must be contiguous");
        return {t.data_ptr(), static_cast<uint64_t>(rows > 1 ? t.stride(0) : cols)};
    }
    Matrix matrix(PyObject* o, const char* name, int64_t rows, int64_t cols, c10::ScalarType type) const {
        return matrix(tensor(o, name), name, rows, cols, type);
    }

    // A contiguous 1-D tensor of n elements (n < 0: any number) and one of two types.
    const at::Tensor& vector(PyObject* o, const char* name, int64_t n, c10::ScalarType a, c10::ScalarType b) const {
        const at::Tensor& t = tensor(o, name);
        if (t.scalar_type() != a && t.scalar_type() != b)
            refuse(PyExc_TypeError, std::string(name) + " must be " + c10::toString(a) +
                                        (a == b ? "" : std::string(" or ") + c10::toString(b)) + ", is " +
                                        c10::toString(t.scalar_type()));
        if (t.dim() != 1 || !t.is_contiguous() || (n >= 0 && t.size(0) != n))
            refuse(PyExc_ValueError, std::string(name) + " must be contiguous 1-D" +
                                         (n < 0 ? "" : " with " + std::to_string(n) + " elements") + ", is " + dims(t));
        return t;
    }
    const uint32_t* ints(PyObject* o, const char* name, int64_t n) const {
        if (o == Py_None) return nullptr;
        return static_cast<const uint32_t*>(vector(o, name, n, c10::ScalarType::Int, c10::ScalarType::UInt32).data_ptr());
    }
    float* floats(PyObject* o, const char* name, int64_t n) const {
        if (o == Py_None) return nullptr;
        return static_cast<float*>(vector(o, name, n, c10::ScalarType::Float, c10::ScalarType::Float).data_ptr());
    }

    struct Scratch {
        void* ptr = nullptr;
        size_t bytes = 0;
    };
    Scratch scratch(PyObject* o) const {
        if (o == Py_None) return {};
        const at::Tensor& t = tensor(o, "workspace");
        if (!t.is_contiguous()) refuse(PyExc_TypeError, "workspace must be contiguous (see new_head_workspace)");
        return {t.data_ptr(), static_cast<size_t>(t.nbytes())};
    }

    // The given output, or a new one; `type` as asked for by the caller, or none.
    at::Tensor output(PyObject* out, PyObject* type, c10::ScalarType otherwise, int64_t rows, int64_t cols,
                      const at::Tensor& like) const {
        const bool asked = type != Py_None;
        if (asked && !THPDtype_Check(type)) refuse(PyExc_TypeError, "out_dtype must be a torch.dtype");
        const c10::ScalarType want = asked ? reinterpret_cast<THPDtype*>(type)->scalar_type : otherwise;
        if (out == Py_None) return at::empty({rows, cols}, like.options().dtype(want));
        const at::Tensor& t = tensor(out, "out");
        if (asked && t.scalar_type() != want)
            refuse(PyExc_TypeError, std::string("out must be ") + c10::toString(want) + ", is " +
                                        c10::toString(t.scalar_type()));
        return t;
    }
    lp_stream_t stream() const {
        return reinterpret_cast<lp_stream_t>(c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(device())).stream());
    }
};

uint32_t size32(int64_t n, const char* name) {
    if (n < 0 || n > 0xFFFFFFFFll) refuse(PyExc_ValueError, std::string(name) + " is too large");
    return static_cast<uint32_t>(n);
}

void check(lp_status rc, const char* what) {
    if (rc == LP_OK) return;
    PyObject* r = PyObject_CallFunction(g_failed, "is", static_cast<int>(rc), what);
    Py_XDECREF(r);
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, what);
    throw Refused();
}

// C++ exceptions (an allocation that fails, for one) become Python errors.
template <typename F>
PyObject* guarded(Py_ssize_t given, Py_ssize_t wanted, F body) {
    if (given != wanted) {
        PyErr_Format(PyExc_TypeError, "%zd arguments expected, %zd given", wanted, given);
        return nullptr;
    }
    try {
        return body();
    } catch (const Refused&) {
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    } catch (...) {
        PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
    }
    return nullptr;
}

// (x, weight, eps, residual, rows, out_dtype, out, out_scale, residual_out, workspace)
PyObject* rms_norm(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
    return guarded(n_args, 10, [&]() -> PyObject* {
        const Call c;
        const at::Tensor& x = c.two_dims(a[0], "x");
        const int64_t T = x.size(0), H = x.size(1);
        const c10::ScalarType type = x.scalar_type();
        const double eps = PyFloat_AsDouble(a[2]);
        if (eps == -1.0 && PyErr_Occurred()) throw Refused();
        const Call::Matrix xm = c.matrix(x, "x", T, H, type);
        Call::Matrix rm, km;
        if (a[3] != Py_None) rm = c.matrix(a[3], "residual", T, H, type);
        int64_t n = T;
        const uint32_t* rows = nullptr;
        if (a[4] != Py_None) {
            rows = c.ints(a[4], "rows", -1);
            n = THPVariable_Unpack(a[4]).size(0);
        }
        const at::Tensor out = c.output(a[6], a[5], type, n, H, x);
        const Call::Matrix om = c.matrix(out, "out", n, H, out.scalar_type());
        const bool quant = out.scalar_type() == c10::ScalarType::Float8_e4m3fn;
        at::Tensor scale;
        float* scale_ptr = c.floats(a[7], "out_scale", n);
        if (quant && !scale_ptr) {
            scale = at::empty({n}, x.options().dtype(c10::ScalarType::Float));
            scale_ptr = static_cast<float*>(scale.data_ptr());
        }
        if (a[8] != Py_None) km = c.matrix(a[8], "residual_out", n, H, type);
        const at::Tensor& w = c.vector(a[1], "weight", H, type, c10::ScalarType::Float);
        const Call::Scratch ws = c.scratch(a[9]);
        check(lp_head_norm(xm.ptr, rm.ptr, w.data_ptr(), dtype_code(type), dtype_code(w.scalar_type()), size32(T, "x"),
                           size32(H, "x"), xm.stride, rm.stride, rows, size32(n, "rows"), static_cast<float>(eps), om.ptr,
                           dtype_code(out.scalar_type()), om.stride, scale_ptr, km.ptr, km.stride, ws.ptr, ws.bytes,
                           c.stream()),
              "lp_head_norm");
        PyObject* result = THPVariable_Wrap(out);
        if (!quant) return result;
        PyObject* s = a[7];
        if (scale.defined()) s = THPVariable_Wrap(scale);
        else Py_INCREF(s);
        PyObject* both = PyTuple_Pack(2, result, s);
        Py_DECREF(result);
        Py_DECREF(s);
        return both;
    });
}

// (x, weight, x_scale, weight_scale, lora_a, lora_b, adapter_scale, adapter_ids, row_offsets,
//  out, out_dtype, workspace)
PyObject* project(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
    return guarded(n_args, 12, [&]() -> PyObject* {
        const Call c;
        const at::Tensor& x = c.two_dims(a[0], "x");
        const int64_t T = x.size(0), H = x.size(1);
        const c10::ScalarType type = x.scalar_type();
        const Call::Matrix xm = c.matrix(x, "x", T, H, type);
        const at::Tensor& w = c.two_dims(a[1], "weight");
        const int64_t V = w.size(0);
        const Call::Matrix wm = c.matrix(w, "weight", V, H, type);
        const void *la = nullptr, *lb = nullptr;
        int64_t A = 0, rank = 0, B = 0;
        c10::ScalarType lora = type;
        const float* adapter_scale = nullptr;
        const int32_t* ids = nullptr;
        const uint32_t* offsets = nullptr;
        if (a[4] != Py_None) {
            if (a[5] == Py_None || a[7] == Py_None) refuse(PyExc_ValueError, "lora_a needs lora_b and adapter_ids");
            const at::Tensor &ta = c.tensor(a[4], "lora_a"), &tb = c.tensor(a[5], "lora_b");
            lora = ta.scalar_type();
            if (ta.dim() != 3 || ta.size(2) != H || !ta.is_contiguous())
                refuse(PyExc_ValueError, "lora_a must be contiguous [adapters, rank, " + std::to_string(H) + "], is " + dims(ta));
            A = ta.size(0);
            rank = ta.size(1);
            if (tb.dim() != 3 || tb.size(0) != A || tb.size(1) != V || tb.size(2) != rank || !tb.is_contiguous())
                refuse(PyExc_ValueError, "lora_b must be contiguous [" + std::to_string(A) + ", " + std::to_string(V) + ", " +
                                             std::to_string(rank) + "], is " + dims(tb));
            if (tb.scalar_type() != lora) refuse(PyExc_TypeError, "lora_a and lora_b must have one type");
            if (A == 0) refuse(PyExc_ValueError, "lora_a has no adapters");
            B = T;
            if (a[8] != Py_None) {
                offsets = c.ints(a[8], "row_offsets", -1);
                B = THPVariable_Unpack(a[8]).size(0) - 1;
            }
            ids = static_cast<const int32_t*>(
                c.vector(a[7], "adapter_ids", B, c10::ScalarType::Int, c10::ScalarType::Int).data_ptr());
            adapter_scale = c.floats(a[6], "adapter_scale", A);
            la = ta.data_ptr();
            lb = tb.data_ptr();
        } else if (a[5] != Py_None || a[6] != Py_None || a[7] != Py_None) {
            refuse(PyExc_ValueError, "lora_b, adapter_ids and adapter_scale need lora_a");
        }
        const at::Tensor out = c.output(a[9], a[10], c10::ScalarType::Float, T, V, x);
        const Call::Matrix om = c.matrix(out, "out", T, V, out.scalar_type());
        const Call::Scratch ws = c.scratch(a[11]);
        check(lp_head_project(xm.ptr, dtype_code(type), size32(T, "x"), size32(H, "x"), xm.stride,
                              c.floats(a[2], "x_scale", T), wm.ptr, size32(V, "weight"), wm.stride,
                              c.floats(a[3], "weight_scale", V), la, lb, dtype_code(lora), size32(A, "lora_a"),
                              size32(rank, "lora_a"), adapter_scale, ids, offsets, size32(B, "row_offsets"), om.ptr,
                              dtype_code(out.scalar_type()), om.stride, ws.ptr, ws.bytes, c.stream()),
              "lp_head_project");
        return THPVariable_Wrap(out);
    });
}

// (logits, row_offsets, history, history_offsets, prompt_lens, repetition, frequency, presence,
//  bias_tokens, bias_values, bias_offsets, mask, mask_index, out, workspace)
PyObject* process_logits(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
    return guarded(n_args, 15, [&]() -> PyObject* {
        const Call c;
        const at::Tensor& x = c.two_dims(a[0], "logits");
        const int64_t T = x.size(0), V = x.size(1);
        const Call::Matrix xm = c.matrix(x, "logits", T, V, x.scalar_type());
        int64_t B = T, n_history = 0, n_bias = 0, mask_rows = 0;
        const uint32_t* offsets = nullptr;
        if (a[1] != Py_None) {
            offsets = c.ints(a[1], "row_offsets", -1);
            B = THPVariable_Unpack(a[1]).size(0) - 1;
            if (B < 0) refuse(PyExc_ValueError, "row_offsets must have an element more than there are requests");
        }
        if ((a[2] == Py_None) != (a[3] == Py_None)) refuse(PyExc_ValueError, "history and history_offsets come together");
        const uint32_t* history = c.ints(a[2], "history", -1);
        if (a[2] != Py_None) n_history = THPVariable_Unpack(a[2]).size(0);
        if ((a[8] == Py_None) != (a[9] == Py_None) || (a[8] == Py_None) != (a[10] == Py_None))
            refuse(PyExc_ValueError, "bias_tokens, bias_values and bias_offsets come together");
        const uint32_t* bias_tokens = c.ints(a[8], "bias_tokens", -1);
        if (a[8] != Py_None) n_bias = THPVariable_Unpack(a[8]).size(0);
        Call::Matrix mm;
        if (a[11] != Py_None) {
            const at::Tensor& m = c.two_dims(a[11], "mask");
            mask_rows = m.size(0);
            if ((m.scalar_type() != c10::ScalarType::Int && m.scalar_type() != c10::ScalarType::UInt32) ||
                m.size(1) < (V + 31) / 32)
                refuse(PyExc_ValueError, "mask must be int32 [rows, " + std::to_string((V + 31) / 32) + " or more]");
            mm = c.matrix(m, "mask", mask_rows, m.size(1), m.scalar_type());
        } else if (a[12] != Py_None) {
            refuse(PyExc_ValueError, "mask_index needs a mask");
        }
        const at::Tensor out = c.output(a[13], Py_None, c10::ScalarType::Float, T, V, x);
        const Call::Matrix om = c.matrix(out, "out", T, V, c10::ScalarType::Float);
        const Call::Scratch ws = c.scratch(a[14]);
        check(lp_head_process(xm.ptr, dtype_code(x.scalar_type()), size32(T, "logits"), size32(V, "logits"), xm.stride,
                              offsets, size32(B, "row_offsets"), history, c.ints(a[3], "history_offsets", B + 1),
                              size32(n_history, "history"), c.ints(a[4], "prompt_lens", B),
                              c.floats(a[5], "repetition", B), c.floats(a[6], "frequency", B),
                              c.floats(a[7], "presence", B), bias_tokens, c.floats(a[9], "bias_values", n_bias),
                              c.ints(a[10], "bias_offsets", B + 1), size32(n_bias, "bias_tokens"),
                              static_cast<const uint32_t*>(mm.ptr), mm.stride, size32(mask_rows, "mask"),
                              reinterpret_cast<const int32_t*>(c.ints(a[12], "mask_index", T)),
                              static_cast<float*>(om.ptr), om.stride, ws.ptr, ws.bytes, c.stream()),
              "lp_head_process");
        return THPVariable_Wrap(out);
    });
}

// (workspace,)
PyObject* clear_status(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
    return guarded(n_args, 1, [&]() -> PyObject* {
        const Call c;
        const Call::Scratch ws = c.scratch(a[0]);
        check(lp_head_clear_status(ws.ptr, c.stream()), "lp_head_clear_status");
        Py_RETURN_NONE;
    });
}

PyObject* on_failure(PyObject*, PyObject* callable) {
    Py_XDECREF(g_failed);
    Py_INCREF(callable);
    g_failed = callable;
    Py_RETURN_NONE;
}

using Fast = PyObject* (*)(PyObject*, PyObject* const*, Py_ssize_t);
PyCFunction fast(Fast f) { return reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(f)); }

PyMethodDef g_methods[] = {{"rms_norm", fast(rms_norm), METH_FASTCALL, nullptr},
                           {"project", fast(project), METH_FASTCALL, nullptr},
                           {"process_logits", fast(process_logits), METH_FASTCALL, nullptr},
                           {"clear_status", fast(clear_status), METH_FASTCALL, nullptr},
                           {"on_failure", on_failure, METH_O, nullptr},
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "lp_head_binding", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_lp_head_binding(void) { return PyModule_Create(&g_module); }
