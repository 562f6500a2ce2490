// The 8-bit linear path's calls from Python, compiled: each function tests its
// tensors as the binding does and makes the C call on the current stream.  It
// returns the call's status, or -1 where the tensors are not what the call takes
// as they stand; the binding then looks for what is wrong and says it.
//
// A call of few rows is 2 to 6 us on the GPU.  The same tests in Python with ctypes
// behind them take the host 4.4 us (quantize_fp8) to 6.0 (gemm_fp8), so that an eager decode
// step waits for the host; here they take 1.9 to 2.2 with the launch.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <exception>

#include "bi.h"

namespace {

struct Calls {
    decltype(&bi_quantize_fp8) quantize;
    decltype(&bi_fp8_read) read;
    decltype(&bi_rmsnorm_fp8) rmsnorm;
    decltype(&bi_add_rmsnorm_fp8) add_rmsnorm;
    decltype(&bi_gemm_fp8) gemm;
    decltype(&bi_gemm_fp8_swiglu) gemm_swiglu;
};
Calls calls = {};  // libbi.so's, given once by bind()

constexpr auto kBf16 = at::ScalarType::BFloat16;
constexpr auto kFp8 = at::ScalarType::Float8_e4m3fn;
constexpr auto kByte = at::ScalarType::Byte;

// Thrown by the readers below for what is not a plain argument; never leaves this file.
struct NotPlain {};

struct Rows {
    void* p;
    int64_t rows, cols, ld;
};

const at::Tensor& tensor(PyObject* o, at::ScalarType type, int dev) {
    if (!THPVariable_Check(o)) throw NotPlain{};
    const at::Tensor& t = THPVariable_Unpack(o);
    if (t.layout() != at::kStrided || !t.is_cuda() || t.get_device() != dev || t.scalar_type() != type)
        throw NotPlain{};
    return t;
}

// A matrix, each row in one run, its leading dimension (one row's is the least there is
// for the type: a row's own stride says nothing).
Rows rows_of(PyObject* o, at::ScalarType type, int dev) {
    const at::Tensor& t = tensor(o, type, dev);
    if (t.dim() != 2 || t.stride(1) != 1) throw NotPlain{};
    const int64_t step = type == kFp8 ? 16 : 8, cols = t.size(1);
    return {t.data_ptr(), t.size(0), cols, t.size(0) > 1 ? t.stride(0) : (cols + step - 1) / step * step};
}
Rows rows_of(PyObject* o, at::ScalarType type, int dev, int64_t rows, int64_t cols) {
    const Rows r = rows_of(o, type, dev);
    if (r.rows != rows || r.cols != cols) throw NotPlain{};
    return r;
}

void* scales_of(PyObject* o, int dev, int64_t rows, int64_t K) {
    const at::Tensor& t = tensor(o, kByte, dev);
    if (t.dim() != 3 || t.size(0) != (rows + 127) / 128 || t.size(1) != (K + 511) / 512 ||
        t.size(2) != BI_FP8_TILE_BYTES || !t.is_contiguous())
        throw NotPlain{};
    return t.data_ptr();
}

void* vector_of(PyObject* o, int dev, int64_t n) {
    const at::Tensor& t = tensor(o, kBf16, dev);
    if (t.dim() != 1 || t.size(0) != n || !t.is_contiguous()) throw NotPlain{};
    return t.data_ptr();
}

int32_t int_of(int64_t v) {
    if (v > 0x7fffffff) throw NotPlain{};
    return static_cast<int32_t>(v);
}

float float_of(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) {
        PyErr_Clear();
        throw NotPlain{};
    }
    return static_cast<float>(v);
}

// f(args, device, stream) -> status, its tensors on the current device and its stream that one's.
template <Py_ssize_t N, typename F>
PyObject* call(PyObject* const* a, Py_ssize_t n, const F& f) {
    long status = -1;
    try {
        if (n == N && calls.gemm && THPVariable_Check(a[0]) && THPVariable_Unpack(a[0]).is_cuda()) {
            const int dev = c10::cuda::current_device();
            status = f(a, dev, c10::cuda::getCurrentCUDAStream(dev).stream());
        }
    } catch (const NotPlain&) {
        status = -1;
    } catch (const std::exception&) {  // torch's: a tensor without storage or strides
        PyErr_Clear();
        status = -1;
    }  // no other: where the interpreter ends meanwhile, the C library unwinds this thread to its end
    return PyLong_FromLong(status);
}

// the C call without the interpreter's lock, which a full launch queue could hold for long
template <typename F>
long unlocked(const F& f) {
    PyThreadState* const state = PyEval_SaveThread();
    const bi_status st = f();
    PyEval_RestoreThread(state);
    return st;
}

PyObject* quantize(PyObject*, PyObject* const* a, Py_ssize_t n) {  // x, out, scales
    return call<3>(a, n, [](PyObject* const* a, int dev, cudaStream_t s) {
        const Rows x = rows_of(a[0], kBf16, dev), q = rows_of(a[1], kFp8, dev, x.rows, x.cols);
        void* const scales = scales_of(a[2], dev, x.rows, x.cols);
        const int32_t K = int_of(x.cols);
        return unlocked([&] { return calls.quantize(x.p, x.ld, x.rows, K, q.p, q.ld, scales, s); });
    });
}

PyObject* read(PyObject*, PyObject* const* a, Py_ssize_t n) {  // q, scales, out
    return call<3>(a, n, [](PyObject* const* a, int dev, cudaStream_t s) {
        const Rows q = rows_of(a[0], kFp8, dev), y = rows_of(a[2], kBf16, dev, q.rows, q.cols);
        void* const scales = scales_of(a[1], dev, q.rows, q.cols);
        const int32_t K = int_of(q.cols);
        return unlocked([&] { return calls.read(q.p, q.ld, scales, q.rows, K, y.p, y.ld, s); });
    });
}

PyObject* rmsnorm(PyObject*, PyObject* const* a, Py_ssize_t n) {  // x, w, eps, out, scales
    return call<5>(a, n, [](PyObject* const* a, int dev, cudaStream_t s) {
        const Rows x = rows_of(a[0], kBf16, dev), q = rows_of(a[3], kFp8, dev, x.rows, x.cols);
        void* const w = vector_of(a[1], dev, x.cols);
        void* const scales = scales_of(a[4], dev, x.rows, x.cols);
        const float eps = float_of(a[2]);
        const int32_t K = int_of(x.cols);
        return unlocked([&] { return calls.rmsnorm(x.p, w, q.p, scales, x.rows, K, x.ld, q.ld, eps, s); });
    });
}

PyObject* add_rmsnorm(PyObject*, PyObject* const* a, Py_ssize_t n) {
    // x, residual, w, eps, residual_out, out, scales
    return call<7>(a, n, [](PyObject* const* a, int dev, cudaStream_t s) {
        const Rows x = rows_of(a[0], kBf16, dev);
        const Rows res = rows_of(a[1], kBf16, dev, x.rows, x.cols), sum = rows_of(a[4], kBf16, dev, x.rows, x.cols);
        const Rows q = rows_of(a[5], kFp8, dev, x.rows, x.cols);
        void* const w = vector_of(a[2], dev, x.cols);
        void* const scales = scales_of(a[6], dev, x.rows, x.cols);
        const float eps = float_of(a[3]);
        const int32_t K = int_of(x.cols);
        return unlocked([&] {
            return calls.add_rmsnorm(x.p, res.p, sum.p, w, q.p, scales, x.rows, K, x.ld, res.ld, sum.ld, q.ld, eps, s);
        });
    });
}

PyObject* gemm(PyObject*, PyObject* const* a, Py_ssize_t n) {  // x, x_scales, W, W_scales, out
    return call<5>(a, n, [](PyObject* const* a, int dev, cudaStream_t s) {
        const Rows x = rows_of(a[0], kFp8, dev), W = rows_of(a[2], kFp8, dev);
        if (W.cols != x.cols) throw NotPlain{};
        const Rows y = rows_of(a[4], kBf16, dev, x.rows, W.rows);
        void* const xs = scales_of(a[1], dev, x.rows, x.cols);
        void* const ws = scales_of(a[3], dev, W.rows, W.cols);
        const int32_t M = int_of(x.rows), N = int_of(W.rows), K = int_of(x.cols);
        return unlocked([&] { return calls.gemm(x.p, xs, W.p, ws, y.p, M, N, K, x.ld, W.ld, y.ld, s); });
    });
}

PyObject* gemm_swiglu(PyObject*, PyObject* const* a, Py_ssize_t n) {
    // x, x_scales, W_gu, W_gu_scales, out, scales
    return call<6>(a, n, [](PyObject* const* a, int dev, cudaStream_t s) {
        const Rows x = rows_of(a[0], kFp8, dev), W = rows_of(a[2], kFp8, dev);
        if (W.cols != x.cols || W.rows % 32) throw NotPlain{};
        const Rows h = rows_of(a[4], kFp8, dev, x.rows, W.rows / 2);
        void* const xs = scales_of(a[1], dev, x.rows, x.cols);
        void* const ws = scales_of(a[3], dev, W.rows, W.cols);
        void* const hs = scales_of(a[5], dev, h.rows, h.cols);
        const int32_t M = int_of(x.rows), F = int_of(h.cols), K = int_of(x.cols);
        return unlocked([&] { return calls.gemm_swiglu(x.p, xs, W.p, ws, h.p, hs, M, F, K, x.ld, W.ld, h.ld, s); });
    });
}

PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {  // the addresses of libbi.so's six entries
    if (n != 6) {
        PyErr_SetString(PyExc_TypeError, "bind: six addresses expected");
        return nullptr;
    }
    void* p[6];
    for (int i = 0; i < 6; ++i)
        if (!(p[i] = PyLong_AsVoidPtr(a[i]))) {
            if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "bind: a null address");
            return nullptr;
        }
    calls = {reinterpret_cast<decltype(calls.quantize)>(p[0]),    reinterpret_cast<decltype(calls.read)>(p[1]),
             reinterpret_cast<decltype(calls.rmsnorm)>(p[2]),     reinterpret_cast<decltype(calls.add_rmsnorm)>(p[3]),
             reinterpret_cast<decltype(calls.gemm)>(p[4]),        reinterpret_cast<decltype(calls.gemm_swiglu)>(p[5])};
    Py_RETURN_NONE;
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyMethodDef method(const char* name, const char* doc) {
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(F)), METH_FASTCALL, doc};
}

PyMethodDef methods[] = {
    method<bind>("bind", "bind(addresses of the six entries)"),
    method<quantize>("quantize_fp8", "quantize_fp8(x, out, scales) -> status or -1"),
    method<read>("fp8_read", "fp8_read(q, scales, out) -> status or -1"),
    method<rmsnorm>("rmsnorm_fp8", "rmsnorm_fp8(x, w, eps, out, scales) -> status or -1"),
    method<add_rmsnorm>("add_rmsnorm_fp8",
                        "add_rmsnorm_fp8(x, residual, w, eps, residual_out, out, scales) -> status or -1"),
    method<gemm>("gemm_fp8", "gemm_fp8(x, x_scales, W, W_scales, out) -> status or -1"),
    method<gemm_swiglu>("gemm_fp8_swiglu",
                        "gemm_fp8_swiglu(x, x_scales, W_gu, W_gu_scales, out, scales) -> status or -1"),
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_call_fp8", "The 8-bit linear path's calls, compiled.", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

// `built_for`: the torch whose objects are read here, by their layout then.
PyMODINIT_FUNC PyInit__call_fp8() {
    PyObject* const m = PyModule_Create(&module);
    if (m && PyModule_AddStringConstant(m, "built_for", BUILT_FOR) < 0) {
        Py_DECREF(m);
        return nullptr;
    }
    return m;
}
