// Argument marshalling of the operators around the adapters, compiled: the same
// checks and calls as the ctypes functions of _binding.py, at the cost of about a
// microsecond instead of eight, which is more than the small calls' kernels take.
//
// Each function takes its arguments by position (tensors, None or numbers; the
// last is the stream as an integer), raises TypeError or ValueError for a tensor
// that does not fit, and returns the C entry point's status.
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/lora_det.h"

namespace {

// The C entry points, taken from the library that _binding.py has loaded.
decltype(&lora_mx4_quantize) quantize_fn;
decltype(&lora_mx4_dequantize) dequantize_fn;
decltype(&lora_mx4_linear) linear_fn;
decltype(&lora_mx4_linear_q) linear_q_fn;
decltype(&lora_block_norm) norm_fn;
decltype(&lora_sample) sample_fn;

struct Refused {};                           // a Python exception is set

[[noreturn]] void refuse(PyObject* type, const char* format, ...)
{
    va_list args;
    va_start(args, format);
    PyErr_FormatV(type, format, args);
    va_end(args);
    throw Refused();
}

constexpr at::ScalarType kBf16 = at::kBFloat16;

// A GPU tensor of one type, or nothing where `arg` is None and may be.
const at::Tensor* tensor(PyObject* arg, at::ScalarType type, const char* name, bool optional = false)
{
    if (optional && arg == Py_None)
        return nullptr;
    if (!THPVariable_Check(arg))
        refuse(PyExc_TypeError, "%s must be a tensor", name);
    const at::Tensor& t = THPVariable_Unpack(arg);
    if (t.scalar_type() != type)
        refuse(PyExc_TypeError, "%s must be %s, got %s", name, c10::toString(type), c10::toString(t.scalar_type()));
    if (!t.is_cuda())
        refuse(PyExc_ValueError, "%s must be a GPU tensor", name);
    return &t;
}

struct Matrix {
    void* p = nullptr;
    int64_t rows = 0, cols = 0, ld = 0;
};

Matrix matrix(PyObject* arg, at::ScalarType type, const char* name, bool optional = false)
{
    const at::Tensor* t = tensor(arg, type, name, optional);
    if (!t)
        return {};
    if (t->dim() != 2)
        refuse(PyExc_ValueError, "%s must be 2-D", name);
    if (t->stride(1) != 1)
        refuse(PyExc_ValueError, "%s rows must be contiguous (stride(1) == 1)", name);
    const int64_t rows = t->size(0), cols = t->size(1), ld = t->stride(0);
    // a single row's stride means nothing (a transposed column's is 1): where it does
    // not suit the entry points' rules, the width, to a whole word of scales, does
    const bool as_it_is = rows > 1 || (ld >= cols && ld % 16 == 0);
    return {t->data_ptr(), rows, cols, as_it_is ? ld : (cols + 3) / 4 * 4};
}

void* vector(PyObject* arg, int64_t n, at::ScalarType type, const char* name, bool optional = true)
{
    const at::Tensor* t = tensor(arg, type, name, optional);
    if (!t)
        return nullptr;
    if (t->dim() != 1 || t->size(0) != n || !t->is_contiguous())
        refuse(PyExc_ValueError, "%s must be a contiguous vector of %lld elements", name, (long long)n);
    return t->data_ptr();
}

int64_t integer(PyObject* arg)
{
    const int64_t v = PyLong_AsLongLong(arg);
    if (v == -1 && PyErr_Occurred())
        throw Refused();
    return v;
}

double number(PyObject* arg)
{
    const double v = PyFloat_AsDouble(arg);
    if (v == -1.0 && PyErr_Occurred())
        throw Refused();
    return v;
}

void* address(PyObject* arg)
{
    void* p = PyLong_AsVoidPtr(arg);
    if (!p && PyErr_Occurred())
        throw Refused();
    return p;
}

void same_rows(int64_t rows, const Matrix& m, const char* name)
{
    if (m.rows != rows)
        refuse(PyExc_ValueError, "%s must have %lld rows, got %lld", name, (long long)rows, (long long)m.rows);
}

// Codes [rows, K / 2] and scales [rows, >= K / 32].
struct Mx4 {
    Matrix q, s;
};

Mx4 mx4(PyObject* q, PyObject* s, int64_t K, const char* name)
{
    Mx4 m{matrix(q, at::kByte, name), matrix(s, at::kByte, name)};
    if (m.q.cols * 2 != K || m.s.cols * 32 < K)
        refuse(PyExc_ValueError, "%s: codes must be [rows, %lld] and scales [rows, at least %lld]", name,
               (long long)(K / 2), (long long)(K / 32));
    same_rows(m.q.rows, m.s, name);
    return m;
}

// A status of 32 bits per call that the library does not take more of.
int32_t narrow(int64_t v)
{
    return v > INT32_MAX || v < INT32_MIN ? INT32_MIN : (int32_t)v;
}

template <class F>
PyObject* call(Py_ssize_t given, Py_ssize_t wanted, F f)
{
    if (given != wanted) {
        PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
        return nullptr;
    }
    try {
        return PyLong_FromLong(f());
    } catch (const Refused&) {
        return nullptr;
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}

uint8_t* u8(void* p) { return static_cast<uint8_t*>(p); }
uint16_t* u16(void* p) { return static_cast<uint16_t*>(p); }
float* f32(void* p) { return static_cast<float*>(p); }
int32_t* i32(void* p) { return static_cast<int32_t*>(p); }

// x, q, scales, stream
template <bool BACK>
PyObject* convert(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return call(n, 4, [&] {
        const Matrix x = matrix(a[0], kBf16, "x");
        const Mx4 m = mx4(a[1], a[2], x.cols, "q, scales");
        same_rows(x.rows, m.q, "q");
        if (BACK)
            return dequantize_fn(u8(m.q.p), m.q.ld, u8(m.s.p), m.s.ld, u16(x.p), x.ld, x.rows, x.cols, address(a[3]));
        return quantize_fn(u16(x.p), x.ld, u8(m.q.p), m.q.ld, u8(m.s.p), m.s.ld, x.rows, x.cols, address(a[3]));
    });
}

struct Workspace {
    void* p = nullptr;
    size_t bytes = 0;
};

Workspace workspace(PyObject* arg)
{
    if (arg == Py_None)
        return {};
    if (!THPVariable_Check(arg))
        refuse(PyExc_TypeError, "workspace must be a tensor");
    const at::Tensor& t = THPVariable_Unpack(arg);
    if (!t.is_cuda() || !t.is_contiguous())
        refuse(PyExc_ValueError, "workspace must be a contiguous GPU tensor");
    return {t.data_ptr(), (size_t)t.nbytes()};
}

// x, wq, ws, y, split_k, workspace, stream
PyObject* linear(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return call(n, 7, [&] {
        const Matrix x = matrix(a[0], kBf16, "x"), y = matrix(a[3], kBf16, "y");
        const Mx4 w = mx4(a[1], a[2], x.cols, "W");
        same_rows(x.rows, y, "y");
        same_rows(y.cols, w.q, "W");
        const Workspace s = workspace(a[5]);
        return linear_fn(u16(x.p), x.ld, u8(w.q.p), w.q.ld, u8(w.s.p), w.s.ld, u16(y.p), y.ld, x.rows, x.cols, y.cols,
                         narrow(integer(a[4])), s.p, s.bytes, address(a[6]));
    });
}

// xq, xs, wq, ws, y, split_k, workspace, stream
PyObject* linear_q(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return call(n, 8, [&] {
        const Matrix y = matrix(a[4], kBf16, "y");
        const int64_t K = 2 * matrix(a[0], at::kByte, "x").cols;
        const Mx4 x = mx4(a[0], a[1], K, "x"), w = mx4(a[2], a[3], K, "W");
        same_rows(x.q.rows, y, "y");
        same_rows(y.cols, w.q, "W");
        const Workspace s = workspace(a[6]);
        return linear_q_fn(u8(x.q.p), x.q.ld, u8(x.s.p), x.s.ld, u8(w.q.p), w.q.ld, u8(w.s.p), w.s.ld, u16(y.p), y.ld,
                           x.q.rows, K, y.cols, narrow(integer(a[5])), s.p, s.bytes, address(a[7]));
    });
}

Matrix like(const Matrix& r, PyObject* arg, const char* name, bool optional)
{
    const Matrix m = matrix(arg, kBf16, name, optional);
    if (m.p && (m.rows != r.rows || m.cols != r.cols))
        refuse(PyExc_ValueError, "%s must be [%lld, %lld]", name, (long long)r.rows, (long long)r.cols);
    return m;
}

// y, post, post_w, post_b, gate, gate_group (None: by the gate's rows), r, res_scale,
// r_out, pre, pre_w, pre_b, x_out, eps, stream
PyObject* block_norm(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return call(n, 15, [&] {
        const Matrix r = matrix(a[6], kBf16, "r");
        const int64_t M = r.rows, C = r.cols;
        const Matrix y = like(r, a[0], "y", true), r_out = like(r, a[8], "r_out", false);
        const Matrix x_out = like(r, a[12], "x_out", true);
        const Matrix gate = matrix(a[4], kBf16, "gate", true);
        int64_t group = 1;
        if (a[4] != Py_None) {
            if (gate.cols != C || gate.rows < 1)
                refuse(PyExc_ValueError, "gate must be [rows, %lld]", (long long)C);
            group = a[5] != Py_None ? integer(a[5]) : M > 0 ? (M + gate.rows - 1) / gate.rows : 1;
            if (group < 1 || (M + group - 1) / group > gate.rows)
                refuse(PyExc_ValueError, "gate has %lld rows for groups of %lld: %lld rows need more",
                       (long long)gate.rows, (long long)group, (long long)M);
        }
        return norm_fn(u16(y.p), y.ld, narrow(integer(a[1])), u16(vector(a[2], C, kBf16, "post_w")),
                       u16(vector(a[3], C, kBf16, "post_b")), u16(gate.p), gate.ld, group, u16(r.p), r.ld,
                       (float)number(a[7]), u16(r_out.p), r_out.ld, narrow(integer(a[9])),
                       u16(vector(a[10], C, kBf16, "pre_w")), u16(vector(a[11], C, kBf16, "pre_b")), u16(x_out.p),
                       x_out.ld, M, C, (float)number(a[13]), address(a[14]));
    });
}

// logits, temperature, top_k, top_p, min_p, u, tokens, logprobs, stream
PyObject* sample(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return call(n, 9, [&] {
        if (!THPVariable_Check(a[0]))
            refuse(PyExc_TypeError, "logits must be a tensor");
        const at::ScalarType type = THPVariable_Unpack(a[0]).scalar_type();
        if (type != kBf16 && type != at::kFloat)
            refuse(PyExc_TypeError, "logits must be bfloat16 or float32, got %s", c10::toString(type));
        const Matrix l = matrix(a[0], type, "logits");
        const int64_t B = l.rows;
        return sample_fn(l.p, type == kBf16 ? LORA_LOGITS_BF16 : LORA_LOGITS_F32, l.ld, B, l.cols,
                         f32(vector(a[1], B, at::kFloat, "temperature")), i32(vector(a[2], B, at::kInt, "top_k")),
                         f32(vector(a[3], B, at::kFloat, "top_p")), f32(vector(a[4], B, at::kFloat, "min_p")),
                         f32(vector(a[5], B, at::kFloat, "u", false)), i32(vector(a[6], B, at::kInt, "tokens", false)),
                         f32(vector(a[7], B, at::kFloat, "logprobs")), address(a[8]));
    });
}

// The addresses of the entry points, in the order above.
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return call(n, 6, [&] {
        quantize_fn = reinterpret_cast<decltype(quantize_fn)>(address(a[0]));
        dequantize_fn = reinterpret_cast<decltype(dequantize_fn)>(address(a[1]));
        linear_fn = reinterpret_cast<decltype(linear_fn)>(address(a[2]));
        linear_q_fn = reinterpret_cast<decltype(linear_q_fn)>(address(a[3]));
        norm_fn = reinterpret_cast<decltype(norm_fn)>(address(a[4]));
        sample_fn = reinterpret_cast<decltype(sample_fn)>(address(a[5]));
        return 0;
    });
}

template <class F>
PyCFunction fast(F f)
{
    return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}

PyMethodDef methods[] = {
    {"bind", fast(bind), METH_FASTCALL, nullptr},
    {"mx4_quantize", fast(convert<false>), METH_FASTCALL, nullptr},
    {"mx4_dequantize", fast(convert<true>), METH_FASTCALL, nullptr},
    {"mx4_linear", fast(linear), METH_FASTCALL, nullptr},
    {"mx4_linear_q", fast(linear_q), METH_FASTCALL, nullptr},
    {"block_norm", fast(block_norm), METH_FASTCALL, nullptr},
    {"sample", fast(sample), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_native", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__native()
{
    PyObject* m = PyModule_Create(&module);
    // the torch whose objects' layout is compiled in; _binding.py compares it
    if (m && PyModule_AddStringConstant(m, "torch_version", LORA_TORCH_VERSION) != 0) {
        Py_DECREF(m);
        return nullptr;
    }
    return m;
}
