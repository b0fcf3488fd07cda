// Native half of the Python binding for the operators that write a product's
// operand and for the products that take it (dense_gemm_packer_amd's
// __init__.py): argument checks, allocation of the outputs and the call of the
// C ABI, in one step.  A decode step makes many of these calls on a few rows
// each, where the kernel takes 2-4 us: with the checks and allocations in
// Python a call cost 7-9 us on the host.  Here quantize takes 4.0 us and the
// norm, with its three outputs, 4.6, of which the launch is 2.9.
//
// The C ABI is called through addresses that bind() receives, so the module
// follows a switch of the active library, and its status codes go to the
// Python function that raises DgpError.
#include <Python.h>

#include <ATen/EmptyTensor.h>
#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/core/DeviceGuard.h>
#include <c10/core/StreamGuard.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/Stream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <optional>
#include <sstream>
#include <string>

#include "../../include/dgp.h"

namespace {

struct Abi {
    decltype(&dgp_quantize_workspace_bytes) workspace_bytes;
    decltype(&dgp_quantize) quantize;
    decltype(&dgp_quantize_b) quantize_b;
    decltype(&dgp_rmsnorm_quantize) rmsnorm;
    decltype(&dgp_swiglu_quantize) swiglu;
    decltype(&dgp_gemm_preshuffle_grouped) grouped;
    decltype(&dgp_gemm_preshuffle) gemm;
};
Abi abi;
PyObject *raise_status;     // raises DgpError for a status code
PyObject *refuse_mode;      // raises DgpError for a scale mode
PyObject *current_stream;   // device index -> stream handle

using at::ScalarType;
using at::Tensor;

[[noreturn]] void bad_value(const std::string &msg)
{
    PyErr_SetString(PyExc_ValueError, msg.c_str());
    throw python_error();
}

template <class... Ts>
std::string text(const Ts &...parts)
{
    std::ostringstream s;
    (s << ... << parts);
    return s.str();
}

const Tensor &tensor(PyObject *o, const char *what)
{
    if (!THPVariable_Check(o)) {
        PyErr_Format(PyExc_TypeError, "%s must be a tensor (got %s)", what, Py_TYPE(o)->tp_name);
        throw python_error();
    }
    return THPVariable_Unpack(o);
}

// An optional tensor argument: undefined for None.
Tensor maybe(PyObject *o, const char *what)
{
    return o == Py_None ? Tensor() : tensor(o, what);
}

void *ptr(const Tensor &t) { return t.defined() ? t.data_ptr() : nullptr; }

// The C ABI's code of a quantising operator's input type.
int input_code(const Tensor &t)
{
    switch (t.scalar_type()) {
    case ScalarType::BFloat16: return DGP_BF16;
    case ScalarType::Half: return DGP_F16;
    case ScalarType::Float: return DGP_F32;
    default: break;
    }
    PyErr_SetString(PyExc_TypeError, text("unsupported input type ", t.scalar_type(), " (bfloat16, float16 or float32)").c_str());
    throw python_error();
}

int operand_code(const Tensor &t)
{
    switch (t.scalar_type()) {
    case ScalarType::BFloat16: return DGP_BF16;
    case ScalarType::Float8_e4m3fn: return DGP_FP8_E4M3;
    case ScalarType::Float4_e2m1fn_x2: return DGP_FP4_E2M1;
    default: break;
    }
    PyErr_SetString(PyExc_TypeError, text("unsupported element type ", t.scalar_type(),
                                          " (bfloat16, float8_e4m3fn or float4_e2m1fn_x2)").c_str());
    throw python_error();
}

void on_device(const Tensor &t, const char *what)
{
    if (!t.is_cuda())
        bad_value(text(what, " must be a device tensor"));
}

void same_device(const Tensor &t, const char *what, const Tensor &X)
{
    if (t.device() != X.device())
        bad_value(text(what, " is on ", t.device(), ", the input on ", X.device()));
}

// A strided [M][K] input: the row stride in elements.
int64_t row_stride(const Tensor &t, const char *what)
{
    if (t.dim() != 2)
        bad_value(text(what, " must be 2-D (got ", t.dim(), "-D)"));
    const int64_t M = t.size(0), K = t.size(1);
    if (K > 1 && t.stride(1) != 1)
        bad_value(text(what, ": the elements of a row must be contiguous"));
    if (M <= 1)
        return K;
    if (t.stride(0) < K)
        bad_value(text(what, ": rows overlap (stride ", t.stride(0), ", ", K, " elements)"));
    return t.stride(0);
}

int64_t row_stride_like(const Tensor &t, const char *what, const Tensor &X)
{
    if (t.sizes() != X.sizes())
        bad_value(text(what, " must be ", X.sizes(), " (got ", t.sizes(), ")"));
    if (t.scalar_type() != X.scalar_type() || t.device() != X.device())
        bad_value(text(what, " is ", t.scalar_type(), " on ", t.device(), ", the input ", X.scalar_type(), " on ", X.device()));
    return row_stride(t, what);
}

// A dense tensor of the given type and shape on the input's device.
void dense(const Tensor &t, ScalarType dtype, at::IntArrayRef shape, const Tensor &X, const char *what)
{
    if (t.scalar_type() != dtype || t.sizes() != shape)
        bad_value(text(what, " must be a ", shape, " ", dtype, " tensor (got ", t.sizes(), " ", t.scalar_type(), ")"));
    if (!t.is_contiguous())
        bad_value(text(what, " must be contiguous"));
    same_device(t, what, X);
}

int scale_mode(PyObject *o, bool allow_none)
{
    const long mode = PyLong_AsLong(o);
    if (mode == -1 && PyErr_Occurred())
        throw python_error();
    if (mode < (allow_none ? DGP_SCALE_NONE : DGP_SCALE_TENSOR) || mode > DGP_SCALE_MX32) {
        PyObject *r = PyObject_CallFunction(refuse_mode, "l", mode);
        Py_XDECREF(r);
        throw python_error();
    }
    return (int)mode;
}

ScalarType code_type(int mode)
{
    return mode == DGP_SCALE_NONE ? ScalarType::BFloat16 : mode == DGP_SCALE_MX32 ? ScalarType::Float4_e2m1fn_x2
                                                                                  : ScalarType::Float8_e4m3fn;
}
ScalarType scale_type(int mode)
{
    return mode == DGP_SCALE_TENSOR || mode == DGP_SCALE_BLOCK128 ? ScalarType::Float : ScalarType::Byte;
}

// Where a call runs: the given stream, or the current one of X's device; X's
// device is current, and outputs are allocated on that stream, while this lives.
// A call that allocates nothing also takes any object with a cuda_stream handle.
class Place {
public:
    Place(const Tensor &X, PyObject *stream, bool allocates = true)
    {
        if (stream == Py_None) {
            device_.emplace(X.device());
            PyObject *h = PyObject_CallFunction(current_stream, "i", (int)X.device().index());
            handle_ = take(h);
        } else if (!allocates && !THPStream_Check(stream)) {
            device_.emplace(X.device());
            handle_ = take(PyObject_GetAttrString(stream, "cuda_stream"));
        } else {
            if (!THPStream_Check(stream)) {
                PyErr_SetString(PyExc_TypeError, "stream must be a torch stream");
                throw python_error();
            }
            const auto *s = reinterpret_cast<THPStream *>(stream);
            const c10::Stream native = c10::Stream::unpack3(s->stream_id, (c10::DeviceIndex)s->device_index,
                                                            (c10::DeviceType)s->device_type);
            if (native.device() != X.device())
                bad_value(text("stream is on ", native.device(), ", the input on ", X.device()));
            stream_.emplace(native);
            handle_ = take(PyObject_GetAttrString(stream, "cuda_stream"));
        }
    }
    void *handle() const { return handle_; }

private:
    static void *take(PyObject *h)
    {
        if (!h)
            throw python_error();
        void *p = PyLong_AsVoidPtr(h);
        Py_DECREF(h);
        if (!p && PyErr_Occurred())
            throw python_error();
        return p;
    }
    std::optional<c10::DeviceGuard> device_;
    std::optional<c10::StreamGuard> stream_;
    void *handle_ = nullptr;
};

// From the allocator that at::empty takes for this kind of device, without the
// dispatcher's way to it: 0.2 us an output, not 0.6 (the device and stream are
// those Place has made current).
Tensor empty(at::IntArrayRef shape, ScalarType dtype, const Tensor &X)
{
    static c10::Allocator *const allocator =
        at::empty({1}, at::TensorOptions().dtype(ScalarType::Byte).device(X.device())).storage().allocator();
    return at::detail::empty_generic(shape, allocator, c10::DispatchKeySet(c10::DispatchKey::CUDA), dtype, std::nullopt);
}

template <class Fn, class... Args>
void call(Fn fn, Args... args)
{
    dgp_status status;
    Py_BEGIN_ALLOW_THREADS
    status = fn(args...);
    Py_END_ALLOW_THREADS
    if (status != DGP_OK) {
        PyObject *r = PyObject_CallFunction(raise_status, "i", (int)status);
        Py_XDECREF(r);
        throw python_error();
    }
}

PyObject *pair(const Tensor &Q, const Tensor &S)
{
    PyObject *s = S.defined() ? THPVariable_Wrap(S) : Py_NewRef(Py_None);
    return Py_BuildValue("(NN)", THPVariable_Wrap(Q), s);
}

// Codes and scales of an [M][K] operand, given or to be allocated.
struct Operand {
    Tensor Q, S, scale;   // scale: the given per-tensor scale
    int64_t shape_q[2], shape_s[2];
    int dim_s;

    Operand(const Tensor &X, int64_t M, int64_t K, int mode, PyObject *scale_o, PyObject *out_o, PyObject *scales_o)
        : Q(maybe(out_o, "out")), S(maybe(scales_o, "scales")), scale(maybe(scale_o, "scale"))
    {
        shape_q[0] = shape_s[0] = M;
        shape_q[1] = mode == DGP_SCALE_MX32 ? K / 2 : K;
        shape_s[1] = mode == DGP_SCALE_MX32 ? K / 32 : K / 128;
        dim_s = 2;
        if (mode == DGP_SCALE_TENSOR)
            shape_s[0] = 1, dim_s = 1;
        if (Q.defined())
            dense(Q, code_type(mode), at::IntArrayRef(shape_q, 2), X, "out");
        if (scale.defined()) {
            if (mode != DGP_SCALE_TENSOR)
                bad_value("a given scale goes with SCALE_TENSOR only");
            if (S.defined())
                bad_value("scale is given: there are no scales to write");
            if (scale.numel() != 1)
                bad_value(text("scale must hold one value (got ", scale.numel(), ")"));
            dense(scale, ScalarType::Float, scale.sizes(), X, "scale");
        } else if (S.defined()) {
            if (mode == DGP_SCALE_NONE)
                bad_value("SCALE_NONE writes no scales");
            dense(S, scale_type(mode), at::IntArrayRef(shape_s, dim_s), X, "scales");
        }
    }

    void allocate(const Tensor &X, int mode)
    {
        if (!Q.defined())
            Q = empty(at::IntArrayRef(shape_q, 2), code_type(mode), X);
        if (!S.defined() && !scale.defined() && mode != DGP_SCALE_NONE)
            S = empty(at::IntArrayRef(shape_s, dim_s), scale_type(mode), X);
    }

    const Tensor &scales() const { return scale.defined() ? scale : S; }
};

Tensor workspace(const Tensor &X, int64_t E, int mode, size_t *bytes)
{
    *bytes = abi.workspace_bytes(E, mode);
    return *bytes ? empty({(int64_t)(*bytes / 4)}, ScalarType::Float, X) : Tensor();
}

void arity(Py_ssize_t got, Py_ssize_t want)
{
    if (got != want) {
        PyErr_Format(PyExc_TypeError, "%zd arguments, %zd expected", got, want);
        throw python_error();
    }
}

// quantize(X, mode, scale, out, scales, stream)
PyObject *quantize(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    arity(n, 6);
    const Tensor &X = tensor(a[0], "X");
    const int64_t ld = row_stride(X, "X");
    const int mode = scale_mode(a[1], false), code = input_code(X);
    const int64_t M = X.size(0), K = X.size(1);
    Operand o(X, M, K, mode, a[2], a[3], a[4]);
    on_device(X, "X");
    Place place(X, a[5]);
    o.allocate(X, mode);
    size_t ws_bytes = 0;
    Tensor ws;
    if (!o.scale.defined())
        ws = workspace(X, 1, mode, &ws_bytes);
    call(abi.quantize, (const void *)X.data_ptr(), ld, code, o.Q.data_ptr(), ptr(o.S), (const float *)ptr(o.scale), M, K,
         mode, (float *)ptr(ws), ws_bytes, place.handle());
    return pair(o.Q, o.scales());
    END_HANDLE_TH_ERRORS
}

// quantize_b(B, mode, out, scales, stream)
PyObject *quantize_b(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    arity(n, 5);
    const Tensor &B = tensor(a[0], "B");
    if (B.dim() != 2 && B.dim() != 3)
        bad_value(text("B must be 2-D or 3-D (got ", B.dim(), "-D)"));
    if (!B.is_contiguous())
        bad_value("B must be contiguous");
    const int mode = scale_mode(a[1], false), code = input_code(B);
    const bool stack = B.dim() == 3;
    const int64_t E = stack ? B.size(0) : 1, N = B.size(-2), K = B.size(-1);
    c10::SmallVector<int64_t, 3> shape_q, shape_s;
    if (stack)
        shape_q.push_back(E), shape_s.push_back(E);
    shape_q.push_back(N), shape_q.push_back(mode == DGP_SCALE_MX32 ? K / 2 : K);
    if (mode == DGP_SCALE_TENSOR) {
        if (!stack)
            shape_s.push_back(1);
    } else {
        shape_s.push_back(mode == DGP_SCALE_BLOCK128 ? N / 128 : N);
        shape_s.push_back(mode == DGP_SCALE_MX32 ? K / 32 : K / 128);
    }
    Tensor Q = maybe(a[2], "out"), S = maybe(a[3], "scales");
    if (Q.defined())
        dense(Q, code_type(mode), shape_q, B, "out");
    if (S.defined())
        dense(S, scale_type(mode), shape_s, B, "scales");
    on_device(B, "B");
    Place place(B, a[4]);
    if (!Q.defined())
        Q = empty(shape_q, code_type(mode), B);
    if (!S.defined())
        S = empty(shape_s, scale_type(mode), B);
    size_t ws_bytes = 0;
    const Tensor ws = workspace(B, E, mode, &ws_bytes);
    call(abi.quantize_b, (const void *)B.data_ptr(), code, Q.data_ptr(), S.data_ptr(), E, N, K, mode, (float *)ptr(ws),
         ws_bytes, place.handle());
    return pair(Q, S);
    END_HANDLE_TH_ERRORS
}

// rmsnorm_quantize(X, weight, mode, residual, eps, scale, out, scales, residual_out, stream)
PyObject *rmsnorm_quantize(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    arity(n, 10);
    const Tensor &X = tensor(a[0], "X"), &W = tensor(a[1], "weight");
    const int64_t ldx = row_stride(X, "X");
    const int mode = scale_mode(a[2], true), code = input_code(X);
    const int64_t M = X.size(0), K = X.size(1);
    const Tensor R = maybe(a[3], "residual");
    const double eps = PyFloat_AsDouble(a[4]);
    if (eps == -1.0 && PyErr_Occurred())
        throw python_error();
    const int64_t ldr = R.defined() ? row_stride_like(R, "residual", X) : 0;
    if (W.dim() != 1 || W.size(0) != K || (W.scalar_type() != X.scalar_type() && W.scalar_type() != ScalarType::Float))
        bad_value(text("weight must hold ", K, " values of ", X.scalar_type(), " or float32 (got ", W.sizes(), " ",
                       W.scalar_type(), ")"));
    if (!W.is_contiguous())
        bad_value("weight must be contiguous");
    same_device(W, "weight", X);
    Operand o(X, M, K, mode, a[5], a[6], a[7]);
    Tensor H = maybe(a[8], "residual_out");
    if (H.defined()) {
        if (!R.defined())
            bad_value("residual_out needs a residual");
        dense(H, X.scalar_type(), X.sizes(), X, "residual_out");
    }
    on_device(X, "X");
    Place place(X, a[9]);
    o.allocate(X, mode);
    if (R.defined() && !H.defined())
        H = empty(X.sizes(), X.scalar_type(), X);
    call(abi.rmsnorm, (const void *)X.data_ptr(), ldx, (const void *)ptr(R), ldr, code, (const void *)W.data_ptr(),
         input_code(W), (float)eps, o.Q.data_ptr(), ptr(o.S), (const float *)ptr(o.scale), ptr(H), M, K, mode,
         place.handle());
    if (!R.defined())
        return pair(o.Q, o.scales());
    const Tensor &S = o.scales();
    PyObject *s = S.defined() ? THPVariable_Wrap(S) : Py_NewRef(Py_None);
    return Py_BuildValue("(NNN)", THPVariable_Wrap(o.Q), s, THPVariable_Wrap(H));
    END_HANDLE_TH_ERRORS
}

// swiglu_quantize(gate, up, mode, scale, out, scales, stream)
PyObject *swiglu_quantize(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    arity(n, 7);
    const Tensor &G = tensor(a[0], "gate"), &U = tensor(a[1], "up");
    const int64_t ldg = row_stride(G, "gate"), ldu = row_stride_like(U, "up", G);
    const int mode = scale_mode(a[2], true), code = input_code(G);
    const int64_t M = G.size(0), K = G.size(1);
    Operand o(G, M, K, mode, a[3], a[4], a[5]);
    on_device(G, "gate");
    Place place(G, a[6]);
    o.allocate(G, mode);
    call(abi.swiglu, (const void *)G.data_ptr(), ldg, (const void *)U.data_ptr(), ldu, code, o.Q.data_ptr(), ptr(o.S),
         (const float *)ptr(o.scale), M, K, mode, place.handle());
    return pair(o.Q, o.scales());
    END_HANDLE_TH_ERRORS
}

// A scale tensor of a grouped product: undefined (the C ABI's DGP_ERR_NULL) or
// n values of its mode's type.
void check_scales(const Tensor &t, const char *what, int mode, int64_t n, const Tensor &A)
{
    if (!t.defined())
        return;
    if (t.scalar_type() != scale_type(mode) || t.numel() != n)
        bad_value(text(what, " must hold ", n, " ", scale_type(mode), " values for this scale mode and shape (got ",
                       t.numel(), " ", t.scalar_type(), ")"));
    dense(t, t.scalar_type(), t.sizes(), A, what);
}

// The scales of a product's operands, `stack` weights of N rows.  (K or N
// that break a mode's divisibility rule are the C ABI's to refuse.)
void check_all_scales(const Tensor &sA, const Tensor &sB, int mode, int64_t a_rows, int64_t stack, int64_t N, int64_t K,
                      const Tensor &A)
{
    if (mode == DGP_SCALE_TENSOR) {
        check_scales(sA, "sA", mode, 1, A);
        check_scales(sB, "sB", mode, stack, A);
    } else if (mode == DGP_SCALE_BLOCK128 && K % 128 == 0 && N % 128 == 0) {
        check_scales(sA, "sA", mode, a_rows * (K / 128), A);
        check_scales(sB, "sB", mode, stack * (N / 128) * (K / 128), A);
    } else if (mode == DGP_SCALE_MX128 && K % 128 == 0) {
        check_scales(sA, "sA", mode, a_rows * (K / 128), A);
        check_scales(sB, "sB", mode, stack * N * (K / 128), A);
    } else if (mode == DGP_SCALE_MX32 && K % 32 == 0) {
        check_scales(sA, "sA", mode, a_rows * (K / 32), A);
        check_scales(sB, "sB", mode, stack * N * (K / 32), A);
    }
}

long product_mode(PyObject *o)
{
    const long mode = PyLong_AsLong(o);
    if (mode == -1 && PyErr_Occurred())
        throw python_error();
    return mode;
}

const dgp_config *config_at(PyObject *o)
{
    if (o == Py_None)
        return nullptr;
    const void *p = PyLong_AsVoidPtr(o);
    if (PyErr_Occurred())
        throw python_error();
    return (const dgp_config *)p;
}

// gemm(A, Bs, sA, sB, mode, out, config address, stream)
PyObject *gemm(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    arity(n, 8);
    const Tensor &A = tensor(a[0], "A"), &Bs = tensor(a[1], "Bs");
    const Tensor sA = maybe(a[2], "sA"), sB = maybe(a[3], "sB");
    const long mode = product_mode(a[4]);
    Tensor C = maybe(a[5], "out");
    const dgp_config *cfg = config_at(a[6]);
    if (A.dim() != 2 || Bs.dim() != 2)
        bad_value(text("A and Bs must be 2-D (got ", A.dim(), "-D and ", Bs.dim(), "-D)"));
    on_device(A, "A");
    const int dtype = operand_code(A);
    if (Bs.scalar_type() != A.scalar_type())
        bad_value(text("Bs is ", Bs.scalar_type(), ", A is ", A.scalar_type(), ": both operands take one element type"));
    const int64_t per = dtype == DGP_FP4_E2M1 ? 2 : 1;
    const int64_t M = A.size(0), N = Bs.size(0), K = A.size(1) * per;
    if (Bs.size(1) != A.size(1))
        bad_value(text("Bs holds ", Bs.size(1) * per, " elements per row, A ", K));
    if (!A.is_contiguous() || !Bs.is_contiguous())
        bad_value("A and Bs must be contiguous");
    same_device(Bs, "Bs", A);
    const int64_t shape_c[2] = {M, N};
    if (C.defined())
        dense(C, ScalarType::BFloat16, shape_c, A, "out");
    check_all_scales(sA, sB, (int)mode, M, 1, N, K, A);
    Place place(A, a[7], !C.defined());
    if (!C.defined())
        C = empty(shape_c, ScalarType::BFloat16, A);
    call(abi.gemm, (const void *)A.data_ptr(), (const void *)Bs.data_ptr(), C.data_ptr(), M, N, K, dtype, (int)mode,
         (const void *)ptr(sA), (const void *)ptr(sB), cfg, place.handle());
    return THPVariable_Wrap(C);
    END_HANDLE_TH_ERRORS
}

// grouped(A, Bs, offsets, sA, sB, mode, rows, out, config address, stream)
PyObject *grouped(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    arity(n, 10);
    const Tensor &A = tensor(a[0], "A"), &Bs = tensor(a[1], "Bs"), &off = tensor(a[2], "offsets");
    const Tensor sA = maybe(a[3], "sA"), sB = maybe(a[4], "sB"), rows = maybe(a[6], "rows");
    Tensor C = maybe(a[7], "out");
    const long mode = product_mode(a[5]);
    const dgp_config *cfg = config_at(a[8]);
    if (A.dim() != 2 || Bs.dim() != 3)
        bad_value(text("A must be 2-D and Bs 3-D (got ", A.dim(), "-D and ", Bs.dim(), "-D)"));
    const int dtype = operand_code(A);
    if (Bs.scalar_type() != A.scalar_type())
        bad_value(text("Bs is ", Bs.scalar_type(), ", A is ", A.scalar_type(), ": both operands take one element type"));
    const int64_t per = dtype == DGP_FP4_E2M1 ? 2 : 1;   // elements per stored value
    const int64_t E = Bs.size(0), N = Bs.size(1), K = A.size(1) * per;
    if (Bs.size(2) != A.size(1))
        bad_value(text("Bs holds ", Bs.size(2) * per, " elements per row, A ", K));
    if (!A.is_contiguous() || !Bs.is_contiguous())
        bad_value("A and Bs must be contiguous");
    same_device(Bs, "Bs", A);
    if (off.scalar_type() != ScalarType::Int || off.dim() != 1 || off.size(0) != E + 1)
        bad_value(text("offsets must be ", E + 1, " int32 values (got ", off.sizes(), " ", off.scalar_type(), ")"));
    dense(off, ScalarType::Int, off.sizes(), A, "offsets");
    if (rows.defined()) {
        if (rows.scalar_type() != ScalarType::Int || rows.dim() != 1)
            bad_value(text("rows must be a 1-D int32 tensor (got ", rows.sizes(), " ", rows.scalar_type(), ")"));
        dense(rows, ScalarType::Int, rows.sizes(), A, "rows");
    }
    const int64_t M = rows.defined() ? rows.size(0) : A.size(0);
    const int64_t shape_c[2] = {M, N};
    if (C.defined())
        dense(C, ScalarType::BFloat16, shape_c, A, "out");
    check_all_scales(sA, sB, (int)mode, A.size(0), E, N, K, A);
    on_device(A, "A");
    Place place(A, a[9]);
    if (!C.defined())
        C = empty(shape_c, ScalarType::BFloat16, A);
    call(abi.grouped, (const void *)A.data_ptr(), A.size(0), (const void *)Bs.data_ptr(), C.data_ptr(), M, N, K, E,
         (const int32_t *)off.data_ptr(), (const int32_t *)ptr(rows), dtype, (int)mode, (const void *)ptr(sA),
         (const void *)ptr(sB), cfg, place.handle());
    return THPVariable_Wrap(C);
    END_HANDLE_TH_ERRORS
}

// bind(addresses, raise_status, refuse_mode, current_stream): addresses of the
// entry points in Abi's order.
PyObject *bind(PyObject *, PyObject *args)
{
    PyObject *addr, *rs, *rm, *cs;
    if (!PyArg_ParseTuple(args, "O!OOO", &PyTuple_Type, &addr, &rs, &rm, &cs))
        return nullptr;
    constexpr int kEntries = sizeof(Abi) / sizeof(void *);
    void *p[kEntries];
    if (PyTuple_GET_SIZE(addr) != kEntries) {
        PyErr_Format(PyExc_ValueError, "%d addresses expected", kEntries);
        return nullptr;
    }
    for (int i = 0; i < kEntries; ++i) {
        p[i] = PyLong_AsVoidPtr(PyTuple_GET_ITEM(addr, i));
        if (!p[i]) {
            if (!PyErr_Occurred())
                PyErr_SetString(PyExc_ValueError, "null address");
            return nullptr;
        }
    }
    abi = Abi{(decltype(Abi::workspace_bytes))p[0], (decltype(Abi::quantize))p[1], (decltype(Abi::quantize_b))p[2],
              (decltype(Abi::rmsnorm))p[3], (decltype(Abi::swiglu))p[4], (decltype(Abi::grouped))p[5],
              (decltype(Abi::gemm))p[6]};
    Py_XSETREF(raise_status, Py_NewRef(rs));
    Py_XSETREF(refuse_mode, Py_NewRef(rm));
    Py_XSETREF(current_stream, Py_NewRef(cs));
    Py_RETURN_NONE;
}

#define FAST(f) {#f, (PyCFunction)(void (*)(void))f, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FAST(quantize), FAST(quantize_b), FAST(rmsnorm_quantize), FAST(swiglu_quantize), FAST(grouped), FAST(gemm),
                         {"bind", bind, METH_VARARGS, nullptr}, {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding(void) { return PyModule_Create(&module); }
