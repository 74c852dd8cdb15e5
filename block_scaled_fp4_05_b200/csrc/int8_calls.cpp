// Python calls of the INT8 entry points: checks of the tensors and argument
// marshalling in one step.  A call of a small product costs the host more than
// the GPU; the same checks written in Python take 2.5 us of it, and ctypes 1.2.
//
// Module _int8_calls.  set_entry_points(quantize, gemm, grouped) takes the
// addresses of fp4_quantize_int8, fp4_gemm_int8 and fp4_gemm_int8_grouped in
// libfp4.so.  quantize / gemm / grouped(tensors..., stream) return the call's
// status, or -1 without a call where a tensor does not fit (the caller finds
// out which); the *_args functions return the C arguments as a tuple, or None.
// stream is None for the current stream, else a handle as an integer.
// built_for names the torch and the Python whose headers it was compiled with.

#include <torch/csrc/autograd/python_variable.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>

#include <cstdint>
#include <initializer_list>

#include "../../include/fp4.h"

namespace {

decltype(&fp4_quantize_int8) g_quantize;
decltype(&fp4_gemm_int8) g_gemm;
decltype(&fp4_gemm_int8_grouped) g_grouped;

const at::Tensor* tensor(PyObject* o) { return THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr; }

bool on(const at::Tensor& t, int device) { return t.is_cuda() && t.get_device() == device; }

bool dtype16(const at::Tensor& t, fp4_dtype* out)
{
    const auto s = t.scalar_type();
    *out = s == at::kHalf ? FP4_FP16 : FP4_BF16;
    return s == at::kHalf || s == at::kBFloat16;
}

// Leading dimension of a matrix (the last two dimensions of t) with unit
// column stride.  That of a single row, or of rows without elements, is never
// used: it counts as the next multiple of `unit`.
bool leading(const at::Tensor& t, int64_t unit, int64_t* ld)
{
    const auto n = t.dim();
    const int64_t rows = t.size(n - 2), cols = t.size(n - 1);
    if (cols > 1 && t.stride(n - 1) != 1) return false;
    *ld = rows > 1 && cols > 0 ? t.stride(n - 2) : (cols + unit - 1) / unit * unit;
    return true;
}

bool vector(const at::Tensor& t, int device, at::ScalarType type, at::IntArrayRef shape)
{
    return t.scalar_type() == type && t.sizes() == shape && t.is_contiguous() && on(t, device);
}

// The handle in o, or the current stream of the device.
bool stream_of(PyObject* o, int device, fp4_stream_t* out)
{
    if (o == Py_None) {
        *out = reinterpret_cast<fp4_stream_t>(c10::cuda::getCurrentCUDAStream(device).stream());
        return true;
    }
    *out = static_cast<fp4_stream_t>(PyLong_AsVoidPtr(o));
    return !PyErr_Occurred();
}

struct Quantize {
    const void* in;
    fp4_dtype dtype;
    int64_t rows_in, cols, ld;
    const int32_t* index;
    int64_t rows;
    void* codes;
    int64_t ldc;
    float* scales;
    fp4_stream_t stream;

    static constexpr int kArgs = 5;   // x, codes, scales, row_index, stream
    bool parse(PyObject* const* a)
    {
        const at::Tensor *x = tensor(a[0]), *c = tensor(a[1]), *s = tensor(a[2]), *r = tensor(a[3]);
        if (!x || !c || !s || (!r && a[3] != Py_None) || x->dim() != 2 || c->dim() != 2) return false;
        const int device = c10::cuda::current_device();
        rows_in = x->size(0);
        cols = x->size(1);
        rows = c->size(0);
        if (c->size(1) != cols || (r ? false : rows != rows_in) || !dtype16(*x, &dtype) || c->scalar_type() != at::kChar ||
            !on(*x, device) || !on(*c, device) || !leading(*x, 8, &ld) || !leading(*c, 16, &ldc) ||
            !vector(*s, device, at::kFloat, {rows}) || (r && !vector(*r, device, at::kInt, {rows})))
            return false;
        in = x->data_ptr();
        index = r ? static_cast<const int32_t*>(r->data_ptr()) : nullptr;
        codes = c->data_ptr();
        scales = static_cast<float*>(s->data_ptr());
        return stream_of(a[4], device, &stream);
    }
    fp4_status call() const
    {
        return g_quantize(in, dtype, rows_in, cols, ld, index, rows, codes, ldc, scales, stream);
    }
    PyObject* tuple() const
    {
        return Py_BuildValue("(NiLLLNLNLNN)", PyLong_FromVoidPtr(const_cast<void*>(in)), (int)dtype, rows_in, cols, ld,
                             PyLong_FromVoidPtr(const_cast<int32_t*>(index)), rows, PyLong_FromVoidPtr(codes), ldc,
                             PyLong_FromVoidPtr(scales), PyLong_FromVoidPtr(stream));
    }
};

struct Gemm {
    const void *A, *B;
    const float *sA, *sB, *bias;
    const int32_t* offsets;
    void* D;
    int64_t lda, ldb, stride_b, ldd, E, M, N, K;
    fp4_dtype dtype;
    int kernel;
    fp4_stream_t stream;

    // A, sA, B, sB, offsets or NULL (dense), D, bias, kernel, stream
    bool parse(PyObject* pA, PyObject* psA, PyObject* pB, PyObject* psB, PyObject* po, PyObject* pD, PyObject* pbias,
               PyObject* pkernel, PyObject* pstream)
    {
        const at::Tensor *a = tensor(pA), *sa = tensor(psA), *b = tensor(pB), *sb = tensor(psB), *d = tensor(pD),
                         *c = tensor(pbias), *o = po ? tensor(po) : nullptr;
        const int grouped = po ? 1 : 0;
        if (!a || !sa || !b || !sb || !d || (!c && pbias != Py_None) || (po && !o) || a->dim() != 2 ||
            b->dim() != 2 + grouped || d->dim() != 2)
            return false;
        const int device = c10::cuda::current_device();
        M = a->size(0);
        K = a->size(1);
        E = grouped ? b->size(0) : 1;
        N = b->size(grouped);
        if (b->size(1 + grouped) != K || d->size(0) != M || d->size(1) != N || a->scalar_type() != at::kChar ||
            b->scalar_type() != at::kChar || !dtype16(*d, &dtype) || !on(*a, device) || !on(*b, device) ||
            !on(*d, device) || !leading(*a, 16, &lda) || !leading(*b, 16, &ldb) || !leading(*d, 8, &ldd) ||
            !vector(*sa, device, at::kFloat, {M}))
            return false;
        const int64_t shape[2] = {E, N};
        const at::IntArrayRef channels(shape + 1 - grouped, 1 + grouped);
        if (!vector(*sb, device, at::kFloat, channels) || (c && !vector(*c, device, at::kFloat, channels)) ||
            (o && !vector(*o, device, at::kInt, {E + 1})))
            return false;
        stride_b = grouped && E > 1 && K > 0 ? b->stride(0) : N * ldb;
        A = a->data_ptr();
        B = b->data_ptr();
        D = d->data_ptr();
        sA = static_cast<const float*>(sa->data_ptr());
        sB = static_cast<const float*>(sb->data_ptr());
        bias = c ? static_cast<const float*>(c->data_ptr()) : nullptr;
        offsets = o ? static_cast<const int32_t*>(o->data_ptr()) : nullptr;
        const long choice = PyLong_AsLong(pkernel);
        kernel = choice == (int)choice ? (int)choice : -1;   // (which the call refuses)
        return !PyErr_Occurred() && stream_of(pstream, device, &stream);
    }
};

struct Dense : Gemm {
    static constexpr int kArgs = 8;   // A, sA, B, sB, D, bias, kernel, stream
    bool parse(PyObject* const* a) { return Gemm::parse(a[0], a[1], a[2], a[3], nullptr, a[4], a[5], a[6], a[7]); }
    fp4_status call() const
    {
        return g_gemm(A, lda, sA, B, ldb, sB, M, N, K, bias, dtype, D, ldd, (fp4_gemm_kernel)kernel, stream);
    }
    PyObject* tuple() const
    {
        return Py_BuildValue("(NLNNLNLLLNiNLiN)", PyLong_FromVoidPtr(const_cast<void*>(A)), lda,
                             PyLong_FromVoidPtr(const_cast<float*>(sA)), PyLong_FromVoidPtr(const_cast<void*>(B)), ldb,
                             PyLong_FromVoidPtr(const_cast<float*>(sB)), M, N, K,
                             PyLong_FromVoidPtr(const_cast<float*>(bias)), (int)dtype, PyLong_FromVoidPtr(D), ldd, kernel,
                             PyLong_FromVoidPtr(stream));
    }
};

struct Grouped : Gemm {
    static constexpr int kArgs = 9;   // A, sA, B, sB, offsets, D, bias, kernel, stream
    bool parse(PyObject* const* a) { return Gemm::parse(a[0], a[1], a[2], a[3], a[4], a[5], a[6], a[7], a[8]); }
    fp4_status call() const
    {
        return g_grouped(A, lda, sA, B, ldb, stride_b, sB, offsets, E, M, N, K, bias, dtype, D, ldd,
                         (fp4_gemm_kernel)kernel, stream);
    }
    PyObject* tuple() const
    {
        return Py_BuildValue("(NLNNLLNNLLLLNiNLiN)", PyLong_FromVoidPtr(const_cast<void*>(A)), lda,
                             PyLong_FromVoidPtr(const_cast<float*>(sA)), PyLong_FromVoidPtr(const_cast<void*>(B)), ldb,
                             stride_b, PyLong_FromVoidPtr(const_cast<float*>(sB)),
                             PyLong_FromVoidPtr(const_cast<int32_t*>(offsets)), E, M, N, K,
                             PyLong_FromVoidPtr(const_cast<float*>(bias)), (int)dtype, PyLong_FromVoidPtr(D), ldd, kernel,
                             PyLong_FromVoidPtr(stream));
    }
};

// Parses into `call`; false where the tensors do not fit (what torch throws
// about them counts as that: the caller names the fault).
template <class Call>
bool parsed(Call& call, PyObject* const* args, Py_ssize_t n)
{
    if (n != Call::kArgs) return false;
    try {
        const bool ok = call.parse(args);
        if (!ok) PyErr_Clear();
        return ok;
    } catch (...) {
        PyErr_Clear();
        return false;
    }
}

template <class Call>
PyObject* run(PyObject*, PyObject* const* args, Py_ssize_t n)
{
    if (!g_quantize) {
        PyErr_SetString(PyExc_RuntimeError, "set_entry_points has not been called");
        return nullptr;
    }
    Call call;
    if (!parsed(call, args, n)) return PyLong_FromLong(-1);
    fp4_status st;
    Py_BEGIN_ALLOW_THREADS st = call.call();
    Py_END_ALLOW_THREADS return PyLong_FromLong((long)st);
}

template <class Call>
PyObject* arguments(PyObject*, PyObject* const* args, Py_ssize_t n)
{
    Call call;
    if (!parsed(call, args, n)) Py_RETURN_NONE;
    return call.tuple();
}

PyObject* set_entry_points(PyObject*, PyObject* const* args, Py_ssize_t n)
{
    if (n != 3) {
        PyErr_SetString(PyExc_TypeError, "three addresses");
        return nullptr;
    }
    void* p[3];
    for (int i = 0; i < 3; ++i) {
        p[i] = PyLong_AsVoidPtr(args[i]);
        if (PyErr_Occurred()) return nullptr;
    }
    g_gemm = reinterpret_cast<decltype(g_gemm)>(p[1]);
    g_grouped = reinterpret_cast<decltype(g_grouped)>(p[2]);
    g_quantize = reinterpret_cast<decltype(g_quantize)>(p[0]);
    Py_RETURN_NONE;
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
constexpr PyMethodDef method(const char* name)
{
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(F)), METH_FASTCALL, nullptr};
}

PyMethodDef g_methods[] = {
    method<set_entry_points>("set_entry_points"),
    method<run<Quantize>>("quantize"),
    method<run<Dense>>("gemm"),
    method<run<Grouped>>("grouped"),
    method<arguments<Quantize>>("quantize_args"),
    method<arguments<Dense>>("gemm_args"),
    method<arguments<Grouped>>("grouped_args"),
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_int8_calls", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__int8_calls(void)
{
    PyObject* m = PyModule_Create(&g_module);
    if (m && PyModule_AddStringConstant(m, "built_for", FP4_BUILT_FOR) < 0) {
        Py_DECREF(m);
        return nullptr;
    }
    return m;
}
