// Torch binding of the feed-forward entry points: checks the tensors,
// allocates results and workspaces from torch's allocator, and calls the C ABI
// (include/tlg.h) on the current stream. A compiled binding because a call
// that reads a few hundred kilobytes takes the GPU 3 us: checked and marshalled
// in Python (ctypes) it took the host 9.5 us, here it takes 4.
#include <ATen/ATen.h>
#include <ATen/DeviceGuard.h>
#include <ATen/EmptyTensor.h>
#include <ATen/hip/impl/HIPCachingAllocatorMasqueradingAsCUDA.h>
#include <c10/core/GradMode.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/utils/pybind.h>

#include <string>

#include "tlg.h"

namespace py = pybind11;
using at::Tensor;
using OptTensor = std::optional<Tensor>;

namespace {

// dict of a device's index to the package's Handle, its filler, the error class
PyObject *g_handles, *g_handle_for, *g_error;

[[noreturn]] void value_error(const std::string &s) { throw py::value_error(s); }

std::string shape_of(const Tensor &t) {
    std::string s = "(";
    for (int64_t i = 0; i < t.dim(); ++i) s += (i ? ", " : "") + std::to_string(t.size(i));
    return s + (t.dim() == 1 ? ",)" : ")");
}
const char *name_of(at::ScalarType t) {
    switch (t) {
        case at::kHalf: return "torch.float16";
        case at::kBFloat16: return "torch.bfloat16";
        case at::kFloat: return "torch.float32";
        case at::kChar: return "torch.int8";
        default: return at::toString(t);
    }
}
[[noreturn]] void type_error(const char *name, const std::string &want, at::ScalarType got) {
    throw py::type_error(std::string(name) + " must be " + want + ", got " + name_of(got));
}
std::string device_of(const at::Device &d) { return d.str(); }

int32_t dtype_of(at::ScalarType t) {
    return t == at::kHalf ? TLG_F16 : t == at::kBFloat16 ? TLG_BF16 : t == at::kFloat ? TLG_F32 : 0;
}

// Raised rather than an answer without the derivative that was asked for.
[[noreturn]] void no_derivative(const char *name, const char *what) {
    PyErr_SetString(PyExc_NotImplementedError, (std::string(name) + what).c_str());
    throw py::error_already_set();
}
// Results carry no forward-mode derivative, and a transform's wrapper of a
// tensor (torch.func) would come out unwrapped.
void check_plain(const Tensor &t, const char *name) {
    const c10::TensorImpl *impl = t.unsafeGetTensorImpl();
    if (impl->key_set().has_any(c10::DispatchKeySet({c10::DispatchKey::FuncTorchBatched,
                                                     c10::DispatchKey::FuncTorchGradWrapper})))
        no_derivative(name, " belongs to a torch.func transform, which this operator has no rule for");
    if (impl->_fw_grad(0, t).defined())
        no_derivative(name, " carries a forward-mode derivative, which this operator does not compute");
}
// Scales take no gradient.
void check_scale_grad(const Tensor &t, const char *name) {
    if (t.requires_grad() && c10::GradMode::is_enabled())
        no_derivative(name, " requires a gradient, which this operator does not compute (detach it, or call "
                            "under torch.no_grad())");
}

// The operand that names the call's device and sizes.
void check_first(const Tensor &t, const char *name, bool type_ok, const char *types) {
    check_plain(t, name);
    if (!type_ok) type_error(name, types, t.scalar_type());
    if (t.dim() != 2) value_error(std::string(name) + " must be 2-D");
    if (!t.is_cuda()) value_error(std::string(name) + " must be on a GPU");
}

// Leading dimension of a row-major (rows, cols) matrix of one type on one device.
int64_t ld_of(const Tensor &t, const char *name, at::ScalarType dtype, int64_t rows, int64_t cols,
              const at::Device &device) {
    check_plain(t, name);
    if (t.scalar_type() != dtype) type_error(name, name_of(dtype), t.scalar_type());
    if (t.dim() != 2) value_error(std::string(name) + " must be 2-D");
    if (t.size(0) != rows || t.size(1) != cols)
        value_error(std::string(name) + " must be (" + std::to_string(rows) + ", " + std::to_string(cols) + "), got " +
                    shape_of(t));
    if (t.device() != device)
        value_error(std::string(name) + " is on " + device_of(t.device()) + ", expected " + device_of(device));
    if (rows && cols > 1 && t.stride(1) != 1)
        value_error(std::string(name) + " must have unit stride along its rows (row-major)");
    if (rows <= 1 || cols == 0) return cols ? cols : 1;
    if (t.stride(0) < cols) value_error(std::string(name) + " rows overlap");
    return t.stride(0);
}

float *scales_of(const Tensor &t, const char *name, int64_t n, const at::Device &device) {
    check_plain(t, name);
    if (t.scalar_type() != at::kFloat) type_error(name, "torch.float32", t.scalar_type());
    if (t.dim() != 1 || t.size(0) != n)
        value_error(std::string(name) + " must have " + std::to_string(n) + " elements, got " + shape_of(t));
    if (t.device() != device)
        value_error(std::string(name) + " is on " + device_of(t.device()) + ", expected " + device_of(device));
    if (n > 1 && t.stride(0) != 1) value_error(std::string(name) + " must be contiguous");
    return (float *)t.data_ptr();
}

// torch's allocator of GPU memory; it allocates on the current device, for the
// current stream (a Call's, which every allocation here comes after).
c10::Allocator *allocator() {
    static c10::Allocator *a = c10::hip::HIPCachingAllocatorMasqueradingAsCUDA::get();
    return a;
}
// A new tensor straight from the allocator: at::empty's way through the
// dispatcher takes as long again (quantising one token, two results: 4.8 us a
// call with it, 4.1 this way).
Tensor empty(at::IntArrayRef size, at::ScalarType dtype) {
    return Tensor(at::detail::empty_generic(size, allocator(), c10::DispatchKeySet(c10::DispatchKey::CUDA), dtype,
                                            std::nullopt));
}
Tensor empty2(int64_t rows, int64_t cols, at::ScalarType dtype) { return empty({rows, cols}, dtype); }

// A result matrix and its leading dimension: the caller's, or a new one.
Tensor result(const OptTensor &out, int64_t rows, int64_t cols, at::ScalarType dtype, const at::Device &device,
              int64_t *ld) {
    if (!out) {
        *ld = cols ? cols : 1;
        return empty2(rows, cols, dtype);
    }
    *ld = ld_of(*out, "out", dtype, rows, cols, device);
    return *out;
}

// The workspace that a call of these sizes can use; a forced kernel may take
// up to what the largest split sum or aligned copy needs. One that only makes
// the call faster (a forward call's) is left out where memory does not allow
// it: copies of unaligned operands may be as large as they are.
constexpr int64_t kForcedWorkspace = 64ll << 20;
struct Workspace {
    c10::DataPtr memory;
    void *p = nullptr;
    int64_t bytes = 0;
    explicit Workspace(int64_t size, bool needed = false) : bytes(size) {
        if (!size) return;
        try {
            memory = allocator()->allocate((size_t)size);
        } catch (const c10::OutOfMemoryError &) {
            if (needed) throw;
            bytes = 0;
        }
        p = memory.get();
    }
};

// A call's device made current, its handle and stream.
struct Call {
    at::DeviceGuard guard;
    tlg_handle h;
    hipStream_t stream;
    Call(const at::Device &device, const py::object &handle)
        : guard(device), stream(c10::hip::getCurrentHIPStream(device.index()).stream()) {
        py::object own = handle;
        if (own.is_none()) {
            py::int_ index(device.index());
            PyObject *found = PyDict_GetItem(g_handles, index.ptr());
            own = found ? py::reinterpret_borrow<py::object>(found)
                        : py::reinterpret_borrow<py::object>(g_handle_for)(py::cast(device));
        }
        static PyObject *name = PyUnicode_InternFromString("ptr");
        py::object ptr = py::reinterpret_steal<py::object>(PyObject_GetAttr(own.ptr(), name));
        if (!ptr) throw py::error_already_set();
        h = ptr.is_none() ? nullptr : (tlg_handle)PyLong_AsVoidPtr(ptr.ptr());
    }
    void check(tlg_status st, const char *what) const {
        if (st == TLG_SUCCESS) return;
        py::object e = py::reinterpret_borrow<py::object>(g_error)((int)st, what);
        PyErr_SetObject(g_error, e.ptr());
        throw py::error_already_set();
    }
};

bool is16(const Tensor &t) { return t.scalar_type() == at::kHalf || t.scalar_type() == at::kBFloat16; }
constexpr const char *k16 = "torch.float16 or torch.bfloat16";

void need_weight(const Tensor &t, const char *name) {
    if (t.dim() != 2) value_error(std::string(name) + " must be 2-D");
}

py::object gated_ffn(const Tensor &X, const Tensor &Wg, const Tensor &Wu, int32_t act, bool save, const OptTensor &out,
                     int32_t config, const py::object &handle) {
    HANDLE_TH_ERRORS
    check_first(X, "X", is16(X), k16);
    need_weight(Wg, "Wg");
    const auto dt = X.scalar_type();
    const at::Device dev = X.device();
    const int64_t M = X.size(0), K = X.size(1), N = Wg.size(0);
    tlg_gated_ffn_desc d = {};
    d.M = M;
    d.N = N;
    d.K = K;
    d.ldx = ld_of(X, "X", dt, M, K, dev);
    d.ldwg = ld_of(Wg, "Wg", dt, N, K, dev);
    d.ldwu = ld_of(Wu, "Wu", dt, N, K, dev);
    const Call call(dev, handle);
    Tensor H = result(out, M, N, dt, dev, &d.ldh), G, U;
    if (save) {
        G = empty2(M, N, dt);
        U = empty2(M, N, dt);
        d.G = G.data_ptr();
        d.U = U.data_ptr();
    }
    d.ldg = d.ldu = N ? N : 1;
    d.X = X.data_ptr();
    d.Wg = Wg.data_ptr();
    d.Wu = Wu.data_ptr();
    d.H = H.data_ptr();
    const Workspace ws(config < 0 ? tlg_gated_ffn_workspace(M, N, K) : kForcedWorkspace);
    call.check(tlg_gated_ffn_variant(call.h, config, dtype_of(dt), act, &d, ws.p, ws.bytes, call.stream),
               "tlg_gated_ffn");
    if (save) return py::make_tuple(H, G, U);
    return py::cast(H);
    END_HANDLE_TH_ERRORS_PYBIND
}

py::tuple gated_ffn_backward(const Tensor &dH, const Tensor &X, const Tensor &Wg, const Tensor &Wu, const Tensor &G,
                             const Tensor &U, int32_t act, bool need_x, bool need_w, int32_t config,
                             const py::object &handle) {
    HANDLE_TH_ERRORS
    check_first(X, "X", is16(X), k16);
    need_weight(Wg, "Wg");
    const auto dt = X.scalar_type();
    const at::Device dev = X.device();
    const int64_t M = X.size(0), K = X.size(1), N = Wg.size(0);
    tlg_gated_ffn_grad_desc d = {};
    d.M = M;
    d.N = N;
    d.K = K;
    d.lddh = ld_of(dH, "dH", dt, M, N, dev);
    d.ldx = ld_of(X, "X", dt, M, K, dev);
    d.ldwg = ld_of(Wg, "Wg", dt, N, K, dev);
    d.ldwu = ld_of(Wu, "Wu", dt, N, K, dev);
    d.ldg = ld_of(G, "G", dt, M, N, dev);
    d.ldu = ld_of(U, "U", dt, M, N, dev);
    d.dH = dH.data_ptr();
    d.X = X.data_ptr();
    d.Wg = Wg.data_ptr();
    d.Wu = Wu.data_ptr();
    d.G = G.data_ptr();
    d.U = U.data_ptr();
    const Call call(dev, handle);
    Tensor dX, dWg, dWu;
    d.lddx = d.lddwg = d.lddwu = K ? K : 1;
    if (need_x) {
        dX = empty2(M, K, dt);
        d.dX = dX.data_ptr();
    }
    if (need_w) {
        dWg = empty2(N, K, dt);
        dWu = empty2(N, K, dt);
        d.dWg = dWg.data_ptr();
        d.dWu = dWu.data_ptr();
    }
    int64_t size = need_x || need_w ? tlg_gated_ffn_backward_workspace(M, N, K) : 0;
    if (size && config >= 0) size += kForcedWorkspace;
    const Workspace ws(size, true);
    call.check(tlg_gated_ffn_backward_variant(call.h, config, dtype_of(dt), act, &d, ws.p, ws.bytes, call.stream),
               "tlg_gated_ffn_backward");
    const auto some = [](bool need, const Tensor &t) { return need ? py::cast(t) : py::object(py::none()); };
    return py::make_tuple(some(need_x, dX), some(need_w, dWg), some(need_w, dWu));
    END_HANDLE_TH_ERRORS_PYBIND
}

py::tuple quantize_i8(const Tensor &X, const OptTensor &out, const OptTensor &scale, const py::object &handle) {
    HANDLE_TH_ERRORS
    const auto dt = X.scalar_type();
    check_first(X, "X", dtype_of(dt) != 0, "torch.float16, torch.bfloat16 or torch.float32");
    const at::Device dev = X.device();
    const int64_t M = X.size(0), K = X.size(1), ldx = ld_of(X, "X", dt, M, K, dev);
    const Call call(dev, handle);
    int64_t ldq;
    Tensor Q = result(out, M, K, at::kChar, dev, &ldq);
    Tensor S = scale ? *scale : empty({M}, at::kFloat);
    float *s = scales_of(S, "scale", M, dev);
    call.check(tlg_quantize_i8(call.h, dtype_of(dt), M, K, X.data_ptr(), ldx, (int8_t *)Q.data_ptr(), ldq, s,
                               call.stream),
               "tlg_quantize_i8");
    return py::make_tuple(Q, S);
    END_HANDLE_TH_ERRORS_PYBIND
}

// The type of a result: `out`'s, or the one asked for.
at::ScalarType result_type(const OptTensor &out, const py::object &out_dtype, bool fp32) {
    at::ScalarType t;
    if (out) {
        t = out->scalar_type();
    } else {
        if (!THPDtype_Check(out_dtype.ptr())) throw py::type_error("out_dtype must be a torch.dtype");
        t = reinterpret_cast<THPDtype *>(out_dtype.ptr())->scalar_type;
    }
    if (t != at::kHalf && t != at::kBFloat16 && !(fp32 && t == at::kFloat))
        type_error("out_dtype", fp32 ? "torch.float16, torch.bfloat16 or torch.float32" : k16, t);
    return t;
}

Tensor gemm_i8(const Tensor &A, const Tensor &SA, const Tensor &B, const Tensor &SB, bool relu, const OptTensor &out,
               const py::object &out_dtype, int32_t config, const py::object &handle) {
    HANDLE_TH_ERRORS
    check_first(A, "A", A.scalar_type() == at::kChar, "torch.int8");
    need_weight(B, "B");
    const at::Device dev = A.device();
    const int64_t M = A.size(0), K = A.size(1), N = B.size(0);
    const int64_t lda = ld_of(A, "A", at::kChar, M, K, dev), ldb = ld_of(B, "B", at::kChar, N, K, dev);
    const float *sa = scales_of(SA, "SA", M, dev), *sb = scales_of(SB, "SB", N, dev);
    check_scale_grad(SA, "SA");
    check_scale_grad(SB, "SB");
    const auto dt = result_type(out, out_dtype, true);
    const Call call(dev, handle);
    int64_t ldc;
    Tensor C = result(out, M, N, dt, dev, &ldc);
    const Workspace ws(config < 0 ? tlg_gemm_i8_workspace(M, N, K) : kForcedWorkspace);
    call.check(tlg_gemm_i8_variant(call.h, config, dtype_of(dt), relu, M, N, K, (const int8_t *)A.data_ptr(), lda, sa,
                                   (const int8_t *)B.data_ptr(), ldb, sb, C.data_ptr(), ldc, ws.p, ws.bytes,
                                   call.stream),
               "tlg_gemm_i8");
    return C;
    END_HANDLE_TH_ERRORS_PYBIND
}

Tensor gated_ffn_i8(const Tensor &X, const Tensor &SX, const Tensor &Wg, const Tensor &SG, const Tensor &Wu,
                    const Tensor &SU, int32_t act, const OptTensor &out, const py::object &out_dtype, int32_t config,
                    const py::object &handle) {
    HANDLE_TH_ERRORS
    check_first(X, "X", X.scalar_type() == at::kChar, "torch.int8");
    need_weight(Wg, "Wg");
    const at::Device dev = X.device();
    const int64_t M = X.size(0), K = X.size(1), N = Wg.size(0);
    tlg_gated_ffn_desc d = {};
    d.M = M;
    d.N = N;
    d.K = K;
    d.ldx = ld_of(X, "X", at::kChar, M, K, dev);
    d.ldwg = ld_of(Wg, "Wg", at::kChar, N, K, dev);
    d.ldwu = ld_of(Wu, "Wu", at::kChar, N, K, dev);
    d.ldg = d.ldu = N ? N : 1;
    const float *sx = scales_of(SX, "SX", M, dev), *sg = scales_of(SG, "SG", N, dev),
                *su = scales_of(SU, "SU", N, dev);
    check_scale_grad(SX, "SX");
    check_scale_grad(SG, "SG");
    check_scale_grad(SU, "SU");
    const auto dt = result_type(out, out_dtype, false);
    const Call call(dev, handle);
    Tensor H = result(out, M, N, dt, dev, &d.ldh);
    d.X = X.data_ptr();
    d.Wg = Wg.data_ptr();
    d.Wu = Wu.data_ptr();
    d.H = H.data_ptr();
    const Workspace ws(config < 0 ? tlg_gated_ffn_i8_workspace(M, N, K) : kForcedWorkspace);
    call.check(tlg_gated_ffn_i8_variant(call.h, config, dtype_of(dt), act, &d, sx, sg, su, ws.p, ws.bytes,
                                        call.stream),
               "tlg_gated_ffn_i8");
    return H;
    END_HANDLE_TH_ERRORS_PYBIND
}

}  // namespace

PYBIND11_MODULE(_ffn_torch, m) {
    // the package's objects that calls need: {index: Handle}, handle_for, TlgError
    m.def("setup", [](py::dict handles, py::object handle_for, py::object error) {
        g_handles = handles.release().ptr();
        g_handle_for = handle_for.release().ptr();
        g_error = error.release().ptr();
    });
    m.def("gated_ffn", &gated_ffn);
    m.def("gated_ffn_backward", &gated_ffn_backward);
    m.def("quantize_i8", &quantize_i8);
    m.def("gemm_i8", &gemm_i8);
    m.def("gated_ffn_i8", &gated_ffn_i8);
}
