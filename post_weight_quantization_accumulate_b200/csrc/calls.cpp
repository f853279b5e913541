// calls.cpp -- the host side of w8a8.py as a CPython module: takes tensors,
// checks them, allocates the outputs and calls libgptq.so on the device's
// current torch stream.  A call of a few tokens takes the GPU 2 to 4 us; the
// same steps in Python took 12 to 20 us a call, here 5 to 8.
//
// Nothing is computed here.  Wrong types raise TypeError, wrong shapes, rows
// that are not contiguous and mixed devices ValueError; a status of the
// library goes to the function that set_check() was given.
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "gptq.h"

namespace {

PyObject* g_check = nullptr;   // check(function name, status): raises

// Messages are put together as strings, not by streams.
void need_type(bool ok, const std::string& text) { TORCH_CHECK_TYPE(ok, text); }
void need_value(bool ok, const std::string& text) { TORCH_CHECK_VALUE(ok, text); }
std::string size_text(int64_t n) { return std::to_string(n); }

int type_code(at::ScalarType t, const char* name)
{
    switch (t) {
        case at::kBFloat16: return GPTQ_BF16;
        case at::kHalf: return GPTQ_F16;
        case at::kFloat: return GPTQ_F32;
        default: break;
    }
    need_type(false, std::string(name) + " must be a bfloat16, float16 or float32 tensor");
    return -1;
}

const at::Tensor& tensor(PyObject* o, const char* name)
{
    if (!THPVariable_Check(o)) need_type(false, std::string(name) + " must be a tensor");
    return THPVariable_Unpack(o);
}

const at::Tensor& matrix(PyObject* o, const char* name)
{
    const at::Tensor& t = tensor(o, name);
    if (t.dim() != 2) need_value(false, std::string(name) + " must be a matrix");
    if (!t.is_cuda()) need_value(false, "tensor arguments must be on a CUDA device");
    return t;
}

struct Rows {
    void* p = nullptr;
    int64_t ld = 0;
};

// 8-bit rows and single rows have pitches that the library accepts.
int64_t code_pitch(int64_t cols) { return (cols + 15) / 16 * 16; }

// A matrix of contiguous rows; None gives none.
Rows rows(PyObject* o, at::ScalarType type, int64_t m, int64_t k, at::Device dev, const char* name)
{
    if (o == Py_None) return {};
    const at::Tensor& t = tensor(o, name);
    if (t.scalar_type() != type) need_type(false, std::string(name) + " must be a " + c10::toString(type) + " tensor");
    if (t.dim() != 2 || t.size(0) != m || t.size(1) != k)
        need_value(false, std::string(name) + " must be [" + size_text(m) + ", " + size_text(k) + "]");
    if (t.device() != dev) need_value(false, "tensor arguments must be on one device");
    if (k > 1 && t.stride(1) != 1) need_value(false, std::string("the rows of ") + name + " must be contiguous");
    return {t.data_ptr(), m > 1 ? t.stride(0) : code_pitch(k)};
}

void* vec(PyObject* o, at::ScalarType type, int64_t n, at::Device dev, const char* name)
{
    if (o == Py_None) return nullptr;
    const at::Tensor& t = tensor(o, name);
    if (t.scalar_type() != type) need_type(false, std::string(name) + " must be a " + c10::toString(type) + " tensor");
    if (t.dim() != 1 || t.size(0) != n) need_value(false, std::string(name) + " must be [" + size_text(n) + "]");
    if (t.device() != dev) need_value(false, "tensor arguments must be on one device");
    if (!t.is_contiguous()) need_value(false, std::string(name) + " must be contiguous");
    return t.data_ptr();
}

at::Tensor empty(at::IntArrayRef shape, at::ScalarType type, at::Device dev)
{
    return at::empty(shape, at::TensorOptions().dtype(type).device(dev));
}

struct Codes {
    at::Tensor codes, scales, sums;
    Rows rows;

    Codes() = default;
    Codes(int64_t m, int64_t k, at::Device dev, bool with_codes)
    {
        const int64_t pitch = code_pitch(k);
        if (with_codes) {
            codes = empty({m, pitch}, at::kChar, dev);
            rows = {codes.data_ptr(), pitch};
            if (pitch != k) codes = codes.narrow(1, 0, k);
        }
        scales = empty({m}, at::kFloat, dev);
        sums = empty({m}, at::kInt, dev);
    }
};

PyObject* wrap(const at::Tensor& t)
{
    if (!t.defined()) Py_RETURN_NONE;
    return THPVariable_Wrap(t);
}

PyObject* tuple(std::initializer_list<at::Tensor> tensors)
{
    PyObject* r = PyTuple_New(static_cast<Py_ssize_t>(tensors.size()));
    if (!r) return nullptr;
    Py_ssize_t i = 0;
    for (const at::Tensor& t : tensors) {
        PyObject* o = wrap(t);
        if (!o) {
            Py_DECREF(r);
            return nullptr;
        }
        PyTuple_SET_ITEM(r, i++, o);
    }
    return r;
}

// Whether the library took the call; else the Python error is set.
bool taken(const char* fn, int status)
{
    if (status == GPTQ_OK) return true;
    PyObject* r = PyObject_CallFunction(g_check, "si", fn, status);
    Py_XDECREF(r);
    if (r) PyErr_Format(PyExc_RuntimeError, "%s -> %d", fn, status);
    return false;
}

// The device made current, and its current torch stream.
struct On {
    c10::cuda::CUDAGuard guard;
    void* stream;
    explicit On(at::Device dev) : guard(dev), stream(c10::cuda::getCurrentCUDAStream(dev.index()).stream()) {}
};

// Lets other Python threads run while the outputs are allocated and the kernel
// is launched: both can wait, for memory or for room in the stream's queue.
struct Released {
    PyThreadState* state = PyEval_SaveThread();
    ~Released() { PyEval_RestoreThread(state); }
};

bool counted(const char* fn, Py_ssize_t got, Py_ssize_t want)
{
    if (got == want) return true;
    PyErr_Format(PyExc_TypeError, "%s takes %zd arguments", fn, want);
    return false;
}

// quantize_tokens(x, gate, codes, hat) -> (codes, scales, sums, hat)
PyObject* quantize_tokens(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    if (!counted("quantize_tokens", n, 4)) return nullptr;
    const at::Tensor& x = matrix(a[0], "x");
    const at::ScalarType type = x.scalar_type();
    const int code = type_code(type, "x");
    const int64_t m = x.size(0), k = x.size(1);
    const at::Device dev = x.device();
    const Rows xr = rows(a[0], type, m, k, dev, "x"), gr = rows(a[1], type, m, k, dev, "gate");
    const bool with_codes = PyObject_IsTrue(a[2]) == 1, with_hat = PyObject_IsTrue(a[3]) == 1;
    Codes q;
    at::Tensor hat;
    int status = 0;
    {
        const Released released;
        const On on(dev);
        q = Codes(m, k, dev, with_codes);
        if (with_hat) hat = empty({m, k}, type, dev);
        status = gptq_quantize_tokens(static_cast<int8_t*>(q.rows.p), q.rows.ld, q.scales.data_ptr<float>(),
                                      q.sums.data_ptr<int32_t>(), hat.defined() ? hat.data_ptr() : nullptr, k, xr.p, xr.ld, gr.p,
                                      gr.ld, code, m, k, on.stream);
    }
    if (!taken("gptq_quantize_tokens", status)) return nullptr;
    return tuple({q.codes, q.scales, q.sums, hat});
    END_HANDLE_TH_ERRORS
}

// block_norm(block, residual, pre_weight, post_norm, post_weight, gate,
// gate_rows, scale, eps, quantize, keep_stream, keep_out)
//     -> (stream, out, codes, scales, sums)
PyObject* block_norm(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    if (!counted("block_norm", n, 12)) return nullptr;
    const at::Tensor& t = a[0] != Py_None ? matrix(a[0], "block") : matrix(a[1], "residual");
    const at::ScalarType type = t.scalar_type();
    const int code = type_code(type, a[0] != Py_None ? "block" : "residual");
    const int64_t m = t.size(0), d = t.size(1);
    const at::Device dev = t.device();
    const int64_t gate_rows = PyLong_AsLongLong(a[6]);
    const double scale = PyFloat_AsDouble(a[7]), eps = PyFloat_AsDouble(a[8]);
    if (PyErr_Occurred()) return nullptr;
    need_value(a[5] == Py_None || gate_rows >= 1, "gate_rows must be positive");
    const Rows block = rows(a[0], type, m, d, dev, "block"), residual = rows(a[1], type, m, d, dev, "residual");
    const Rows gate = rows(a[5], type, m > 0 && gate_rows >= 1 ? (m - 1) / gate_rows + 1 : 0, d, dev, "gate");
    const void* pre = vec(a[2], at::kFloat, d, dev, "pre_weight");
    const void* post = vec(a[4], at::kFloat, d, dev, "post_weight");
    const bool post_norm = PyObject_IsTrue(a[3]) == 1, quantize = PyObject_IsTrue(a[9]) == 1;
    const bool keep_stream = PyObject_IsTrue(a[10]) == 1, keep_out = PyObject_IsTrue(a[11]) == 1;
    at::Tensor stream, out;
    Codes q;
    int status = 0;
    {
        const Released released;
        const On on(dev);
        if (keep_stream) stream = empty({m, d}, type, dev);
        if (keep_out && quantize)
            q = Codes(m, d, dev, true);
        else if (keep_out)
            out = empty({m, d}, type, dev);
        const bool codes = q.codes.defined();
        status = gptq_block_norm(stream.defined() ? stream.data_ptr() : nullptr, d, out.defined() ? out.data_ptr() : nullptr, d,
                                 static_cast<int8_t*>(q.rows.p), q.rows.ld, codes ? q.scales.data_ptr<float>() : nullptr,
                                 codes ? q.sums.data_ptr<int32_t>() : nullptr, block.p, block.ld, residual.p, residual.ld, gate.p,
                                 gate.ld, gate_rows, static_cast<const float*>(post), static_cast<const float*>(pre), post_norm,
                                 static_cast<float>(scale), static_cast<float>(eps), code, m, d, on.stream);
    }
    if (!taken("gptq_block_norm", status)) return nullptr;
    return tuple({stream, out, q.codes, q.scales, q.sums});
    END_HANDLE_TH_ERRORS
}

// linear(x codes, x scales, x sums, w codes, w scales, w zeros, bias, dtype) -> y
PyObject* linear(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    if (!counted("linear", n, 8)) return nullptr;
    const at::Tensor& x = matrix(a[0], "the tokens' codes");
    const at::Tensor& w = matrix(a[3], "the weight's codes");
    need_type(THPDtype_Check(a[7]), "dtype must be a torch.dtype");
    const at::ScalarType type = reinterpret_cast<THPDtype*>(a[7])->scalar_type;
    const int code = type_code(type, "the result");
    const int64_t m = x.size(0), k = x.size(1), rows_w = w.size(0);
    const at::Device dev = x.device();
    need_value(a[5] == Py_None || a[2] != Py_None, "weights with a zero point need the tokens' sums");
    const Rows xr = rows(a[0], at::kChar, m, k, dev, "the tokens' codes"), wr = rows(a[3], at::kChar, rows_w, k, dev, "the weight's codes");
    const void* xs = vec(a[1], at::kFloat, m, dev, "the tokens' scales");
    const void* sums = vec(a[2], at::kInt, m, dev, "the tokens' sums");
    const void* ws = vec(a[4], at::kFloat, rows_w, dev, "the weight's scales");
    const void* zeros = vec(a[5], at::kInt, rows_w, dev, "the weight's zeros");
    const void* bias = vec(a[6], at::kFloat, rows_w, dev, "bias");
    at::Tensor y;
    int status = 0;
    {
        const Released released;
        const On on(dev);
        y = empty({m, rows_w}, type, dev);
        status = gptq_w8a8_gemm(y.data_ptr(), rows_w, code, static_cast<const int8_t*>(xr.p), xr.ld, static_cast<const float*>(xs),
                                static_cast<const int32_t*>(sums), static_cast<const int8_t*>(wr.p), wr.ld,
                                static_cast<const float*>(ws), static_cast<const int32_t*>(zeros), static_cast<const float*>(bias),
                                m, rows_w, k, on.stream);
    }
    if (!taken("gptq_w8a8_gemm", status)) return nullptr;
    return wrap(y);
    END_HANDLE_TH_ERRORS
}

PyObject* set_check(PyObject*, PyObject* f)
{
    Py_XDECREF(g_check);
    Py_INCREF(f);
    g_check = f;
    Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"quantize_tokens", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(quantize_tokens)), METH_FASTCALL, nullptr},
    {"block_norm", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(block_norm)), METH_FASTCALL, nullptr},
    {"linear", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(linear)), METH_FASTCALL, nullptr},
    {"set_check", set_check, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls(void) { return PyModule_Create(&module); }
