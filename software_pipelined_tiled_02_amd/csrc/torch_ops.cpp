// torch_ops.cpp -- the 8-bit and the feed-forward operators on torch tensors: argument checks,
// output allocation and the call of the C ABI, as a CPython module
// (_torch_ops) that `binding` wraps.
//
// Why not ctypes, as for the rest of the binding: single-token calls are
// bound by the host.  A kernel launch takes 3.7 us; with the checks, the
// allocations and the call in Python a product took 8.4 us and a norm 12.6.
//
// Every function takes positional arguments only (binding fills in the
// defaults) and runs on the current stream of its tensors' device.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/hip/EmptyTensor.h>
#include <c10/hip/HIPGraphsC10Utils.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <limits>
#include <mutex>
#include <string>

#include "linear_rows.h"
#include "pipegemm.h"

namespace {

// An argument error: ValueError.
struct BadArgument {
    std::string text;
};

constexpr int64_t kBlock = 128;
constexpr int kMaxDevices = 64;

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Elements from one row of an 8-bit matrix to the next: rows start on 16
// bytes; wide ones on 128, the caches' lines, so that the product's loads of
// 128 bytes touch one line each, not two (8192 x 8192 x 8200: 447 us, 505 with
// rows on 16; 512 x 4096 x 4100: 17.2 and 22.0; at K = 520 no difference).
int64_t pitch(int64_t n) { return n < 1024 ? (n + 15) / 16 * 16 : (n + 127) / 128 * 128; }

std::mutex g_mutex;
gemm_handle_t g_handles[kMaxDevices];

// Raises binding.GemmError; returns NULL.
PyObject* gemm_error(int status, const char* where) {
    PyObject* module = PyImport_ImportModule("software_pipelined_tiled_02_amd.binding");
    PyObject* cls = module ? PyObject_GetAttrString(module, "GemmError") : nullptr;
    PyObject* error = cls ? PyObject_CallFunction(cls, "is", status, where) : nullptr;
    if (error) PyErr_SetObject(cls, error);
    Py_XDECREF(error);
    Py_XDECREF(cls);
    Py_XDECREF(module);
    return nullptr;
}

// The handle of a device, made on first use: that waits for the device, so
// it cannot be part of a graph capture.
gemm_handle_t handle_of(int index) {
    TORCH_CHECK(index >= 0 && index < kMaxDevices, "device number ", index);
    std::lock_guard<std::mutex> lock(g_mutex);
    if (g_handles[index] == nullptr) {
        TORCH_CHECK(c10::hip::currentStreamCaptureStatusMayInitCtx() == c10::hip::CaptureStatus::None,
                    "the first call on a device sets it up: make one before the graph capture");
        const int rc = gemm_create(&g_handles[index], index);
        TORCH_CHECK(rc == GEMM_OK, "gemm_create: ", gemm_status_string(rc));
    }
    return g_handles[index];
}

int float_type(at::ScalarType t) {
    switch (t) {
    case at::kBFloat16: return GEMM_BF16;
    case at::kHalf: return GEMM_F16;
    case at::kFloat: return GEMM_F32;
    default: return -1;
    }
}
int fp8_type(at::ScalarType t) {
    return t == at::kFloat8_e4m3fn ? GEMM_E4M3 : t == at::kFloat8_e5m2 ? GEMM_E5M2 : -1;
}
at::ScalarType fp8_scalar(int64_t t) { return t == GEMM_E5M2 ? at::kFloat8_e5m2 : at::kFloat8_e4m3fn; }

const at::Tensor& tensor(PyObject* o, const char* what) {
    if (!THPVariable_Check(o)) throw BadArgument{std::string(what) + " must be a torch tensor"};
    return THPVariable_Unpack(o);
}

std::string shape_of(const at::Tensor& t) {
    std::string s = "(";
    for (int64_t i = 0; i < t.dim(); ++i) s += (i ? ", " : "") + std::to_string(t.size(i));
    return s + ")";
}

struct Matrix {
    char* p = nullptr;
    int64_t rows = 0, cols = 0, ld = 0;
    int type = -1;      // GEMM_*
    int device = -1;
};

enum Kinds { kFloats, kFp8 };

// A 2-D CUDA tensor of a kind (and, where given, of one type, on one device,
// of one shape) with unit stride along its last axis and rows that do not
// overlap.  A single row's leading dimension is free: the next multiple of 16.
Matrix matrix(const at::Tensor& t, const char* what, Kinds kind, int device = -1, int type = -1, int64_t rows = -1,
              int64_t cols = -1) {
    const std::string name(what);
    if (t.dim() != 2) throw BadArgument{name + " must have two dimensions (got " + shape_of(t) + ")"};
    Matrix m;
    m.type = kind == kFp8 ? fp8_type(t.scalar_type()) : float_type(t.scalar_type());
    if (m.type < 0)
        throw BadArgument{name + (kind == kFp8 ? " must be float8_e4m3fn or float8_e5m2"
                                               : " must be bfloat16, float16 or float32") +
                          " (got " + c10::toString(t.scalar_type()) + ")"};
    if (type >= 0 && m.type != type) throw BadArgument{name + " has another type than the tensor it goes with"};
    if (!t.is_cuda() || t.layout() != c10::kStrided || (device >= 0 && t.get_device() != device))
        throw BadArgument{"all tensors must be CUDA tensors on one device (" + name + " is on " + t.device().str() + ")"};
    m.device = t.get_device();
    m.rows = t.size(0);
    m.cols = t.size(1);
    if (rows >= 0 && (m.rows != rows || m.cols != cols))
        throw BadArgument{name + " must be " + std::to_string(rows) + " x " + std::to_string(cols) + " (got " +
                          shape_of(t) + ")"};
    m.ld = m.rows > 1 ? t.stride(0) : (m.cols + 15) / 16 * 16;
    if ((m.cols > 1 && t.stride(1) != 1) || m.ld < m.cols)
        throw BadArgument{name + " must have unit stride along its last axis, and rows that do not overlap"};
    m.p = (char*)t.data_ptr();
    return m;
}

struct Scales {
    float* p;
    int64_t rows, blocks, row, blk;
};
Scales scales(const at::Tensor& t, const char* what, int device) {
    if (t.scalar_type() != at::kFloat || t.dim() != 2 || !t.is_cuda() || t.layout() != c10::kStrided ||
        t.get_device() != device)
        throw BadArgument{std::string(what) + " must be a 2-D float32 tensor on the matrices' device"};
    return Scales{(float*)t.data_ptr(), t.size(0), t.size(1), t.stride(0), t.stride(1)};
}

// n contiguous values, of fp32 or (type >= 0) that type; returns GEMM_*.
int vector(const at::Tensor& t, const char* what, int64_t n, int device, int type) {
    const int got = float_type(t.scalar_type());
    if (got < 0 || (got != GEMM_F32 && got != type) || t.dim() != 1 || t.size(0) != n || !t.is_cuda() ||
        t.layout() != c10::kStrided || t.get_device() != device || (n > 1 && t.stride(0) != 1))
        throw BadArgument{std::string(what) + " must be " + std::to_string(n) +
                          " contiguous values of float32 (a weight: or of the matrices' type) on their device"};
    return got;
}

at::Tensor empty(at::IntArrayRef size, at::IntArrayRef stride, at::ScalarType type, int device) {
    return at::detail::empty_strided_cuda(size, stride, type, c10::Device(c10::kCUDA, (c10::DeviceIndex)device));
}
// rows x cols of 8-bit values, rows `pitch` apart.
at::Tensor empty_fp8(int64_t rows, int64_t cols, at::ScalarType type, int device) {
    return empty({rows, cols}, {pitch(cols), 1}, type, device);
}
// rows x blocks scales, one block's after another (the order the product reads them in).
at::Tensor empty_scales(int64_t rows, int64_t blocks, int device) {
    return empty({rows, blocks}, {1, rows}, at::kFloat, device);
}
void* raw_stream(int device) { return c10::hip::getCurrentHIPStream((c10::DeviceIndex)device).stream(); }

// The C call without the GIL (a full queue makes a launch wait).
template <typename F>
int enqueue(F call) {
    PyThreadState* state = PyEval_SaveThread();
    const int rc = call();
    PyEval_RestoreThread(state);
    return rc;
}

PyObject* tuple_of(std::initializer_list<at::Tensor> list) {
    PyObject* t = PyTuple_New((Py_ssize_t)list.size());
    if (t == nullptr) return nullptr;
    Py_ssize_t i = 0;
    for (const at::Tensor& x : list) PyTuple_SET_ITEM(t, i++, THPVariable_Wrap(x));
    return t;
}

bool none(PyObject* o) { return o == Py_None; }
bool truth(PyObject* o) {
    const int r = PyObject_IsTrue(o);
    if (r < 0) throw python_error();
    return r != 0;
}
int64_t integer(PyObject* o) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw python_error();
    return v;
}
void arguments(Py_ssize_t got, Py_ssize_t wanted) {
    TORCH_CHECK(got == wanted, "takes ", wanted, " arguments, got ", got);
}

// A caller's tensor was written: autograd counts such writes, and refuses a backward
// pass that needs what was there.  (Tensors of inference mode have no count.)
void written(const at::Tensor& t) {
    if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

// run_fp8(a, sa, b, sb, out, out_dtype, accumulate, tile)
PyObject* run_fp8_(PyObject* const* arg, Py_ssize_t n) {
    arguments(n, 8);
    const Matrix a = matrix(tensor(arg[0], "a"), "a", kFp8);
    const Matrix b = matrix(tensor(arg[2], "b"), "b", kFp8, a.device);
    if (b.cols != a.cols)
        throw BadArgument{"inner dimensions differ: a has K = " + std::to_string(a.cols) + ", b has " +
                          std::to_string(b.cols)};
    const int64_t blocks = ceil_div(a.cols, kBlock);
    const Scales sa = scales(tensor(arg[1], "sa"), "sa", a.device), sb = scales(tensor(arg[3], "sb"), "sb", a.device);
    if (sa.rows != a.rows || sa.blocks != blocks)
        throw BadArgument{"sa must be M x ceil(K / 128) = " + std::to_string(a.rows) + " x " + std::to_string(blocks)};
    const int sb_rows = sb.rows == ceil_div(b.rows, kBlock) ? (int)kBlock : 1;
    if ((sb_rows == 1 && sb.rows != b.rows) || sb.blocks != blocks)
        throw BadArgument{"sb must be ceil(N / 128) or N rows of ceil(K / 128) = " + std::to_string(blocks) + " scales"};
    const bool accumulate = truth(arg[6]);
    const int64_t tile = integer(arg[7]);
    at::ScalarType type = at::kBFloat16;
    if (!none(arg[5])) {
        if (!THPDtype_Check(arg[5])) throw BadArgument{"out_dtype must be a torch dtype"};
        type = ((THPDtype*)arg[5])->scalar_type;
    }
    at::Tensor made;
    Matrix c;
    if (none(arg[4])) {
        if (accumulate) throw BadArgument{"accumulate needs out"};
        c.type = float_type(type);
        if (c.type < 0) throw BadArgument{"out_dtype must be bfloat16, float16 or float32"};
    } else {
        c = matrix(tensor(arg[4], "out"), "out", kFloats, a.device, -1, a.rows, b.rows);
        if (!none(arg[5]) && float_type(type) != c.type) throw BadArgument{"out has another type than out_dtype"};
        if (accumulate && c.type != GEMM_F32) throw BadArgument{"accumulate needs a float32 out"};
    }
    const gemm_handle_t h = handle_of(a.device);
    if (none(arg[4])) {
        made = empty({a.rows, b.rows}, {b.rows, 1}, type, a.device);
        c.p = (char*)made.data_ptr();
        c.ld = a.rows > 1 ? b.rows : (b.rows + 15) / 16 * 16;
    }
    void* const stream = raw_stream(a.device);
    const int rc = enqueue([&] {
        return gemm_run_fp8(h, a.rows, b.rows, a.cols, a.type, b.type, c.type, sb_rows, accumulate, (int)tile, a.p, a.ld,
                            sa.p, sa.row, sa.blk, b.p, b.ld, sb.p, sb.row, sb.blk, c.p, c.ld, stream);
    });
    if (rc != GEMM_OK) return gemm_error(rc, "gemm_run_fp8");
    if (none(arg[4])) return THPVariable_Wrap(std::move(made));
    written(THPVariable_Unpack(arg[4]));
    Py_INCREF(arg[4]);
    return arg[4];
}

// quantize_fp8(x, block_rows, fp8, pow2, rows, transpose)
PyObject* quantize_fp8_(PyObject* const* arg, Py_ssize_t n) {
    arguments(n, 6);
    const Matrix x = matrix(tensor(arg[0], "x"), "x", kFloats);
    const int64_t block_rows = integer(arg[1]), fp8 = integer(arg[2]);
    const bool pow2 = truth(arg[3]), rows = truth(arg[4]), transpose = truth(arg[5]);
    if (!rows && !transpose) throw BadArgument{"rows or transpose must be asked for"};
    const gemm_handle_t h = handle_of(x.device);
    const int64_t M = x.rows, K = x.cols, m = ceil_div(M, block_rows), k = ceil_div(K, block_rows);
    at::Tensor q, s, qt, st;
    if (rows) {
        q = empty_fp8(M, K, fp8_scalar(fp8), x.device);
        s = empty_scales(m, ceil_div(K, kBlock), x.device);
    }
    if (transpose) {
        qt = empty_fp8(K, M, fp8_scalar(fp8), x.device);
        st = empty_scales(k, ceil_div(M, kBlock), x.device);
    }
    void* const stream = raw_stream(x.device);
    const int rc = enqueue([&] {
        return gemm_quantize_fp8(h, M, K, x.type, (int)fp8, (int)block_rows, pow2, x.p, x.ld,
                                 rows ? q.data_ptr() : nullptr, pitch(K), rows ? (float*)s.data_ptr() : nullptr, 1, m,
                                 transpose ? qt.data_ptr() : nullptr, pitch(M),
                                 transpose ? (float*)st.data_ptr() : nullptr, 1, k, stream);
    });
    if (rc != GEMM_OK) return gemm_error(rc, "gemm_quantize_fp8");
    return !transpose ? tuple_of({q, s}) : !rows ? tuple_of({qt, st}) : tuple_of({q, s, qt, st});
}

// rms_fp8(x, weight, residual, eps, fp8, pow2, norm, h_out)
PyObject* rms_fp8_(PyObject* const* arg, Py_ssize_t n) {
    arguments(n, 8);
    const at::Tensor& xt = tensor(arg[0], "x");
    const Matrix x = matrix(xt, "x", kFloats);
    const int64_t M = x.rows, D = x.cols, fp8 = integer(arg[4]);
    const at::Tensor& w = tensor(arg[1], "weight");
    const int w_type = vector(w, "weight", D, x.device, x.type);
    Matrix r, ho;
    if (!none(arg[2])) r = matrix(tensor(arg[2], "residual"), "residual", kFloats, x.device, x.type, M, D);
    if (!none(arg[7])) ho = matrix(tensor(arg[7], "h_out"), "h_out", kFloats, x.device, x.type, M, D);
    const double eps = PyFloat_AsDouble(arg[3]);
    if (eps == -1.0 && PyErr_Occurred()) throw python_error();
    const bool pow2 = truth(arg[5]), norm = truth(arg[6]);
    const gemm_handle_t h = handle_of(x.device);
    const at::Tensor q = empty_fp8(M, D, fp8_scalar(fp8), x.device), s = empty_scales(M, ceil_div(D, kBlock), x.device);
    const at::Tensor rstd = empty({M}, {1}, at::kFloat, x.device);
    at::Tensor made, y, ht = xt;
    if (!none(arg[7])) {
        ht = THPVariable_Unpack(arg[7]);
    } else if (!none(arg[2])) {
        ht = empty({M, D}, {D, 1}, xt.scalar_type(), x.device);
        ho.p = (char*)ht.data_ptr();
        ho.ld = D;
    }
    if (norm) y = empty({M, D}, {D, 1}, xt.scalar_type(), x.device);
    if (D == 0) rstd.fill_(std::numeric_limits<double>::quiet_NaN());     // the mean of no values; the kernel writes nothing
    void* const stream = raw_stream(x.device);
    const int rc = enqueue([&] {
        return gemm_rms_fp8(h, M, D, x.type, w_type, (int)fp8, pow2, (float)eps, x.p, x.ld, r.p, r.ld, w.data_ptr(),
                            ho.p, ho.ld, norm ? y.data_ptr() : nullptr, D, q.data_ptr(), pitch(D),
                            (float*)s.data_ptr(), 1, M, (float*)rstd.data_ptr(), stream);
    });
    if (rc != GEMM_OK) return gemm_error(rc, "gemm_rms_fp8");
    if (!none(arg[7])) written(ht);
    return norm ? tuple_of({q, s, ht, rstd, y}) : tuple_of({q, s, ht, rstd});
}

// rms_backward(dy, h, weight, rstd, dh, dx_out)
PyObject* rms_backward_(PyObject* const* arg, Py_ssize_t n) {
    arguments(n, 6);
    const at::Tensor& ht = tensor(arg[1], "h");
    const Matrix hm = matrix(ht, "h", kFloats);
    const int64_t M = hm.rows, D = hm.cols;
    const Matrix dy = matrix(tensor(arg[0], "dy"), "dy", kFloats, hm.device, hm.type, M, D);
    const at::Tensor& w = tensor(arg[2], "weight");
    const int w_type = vector(w, "weight", D, hm.device, hm.type);
    const at::Tensor& rstd = tensor(arg[3], "rstd");
    vector(rstd, "rstd", M, hm.device, -1);
    Matrix dh, dx;
    if (!none(arg[4])) dh = matrix(tensor(arg[4], "dh"), "dh", kFloats, hm.device, hm.type, M, D);
    if (!none(arg[5])) dx = matrix(tensor(arg[5], "dx_out"), "dx_out", kFloats, hm.device, hm.type, M, D);
    const gemm_handle_t h = handle_of(hm.device);
    at::Tensor dxt;
    if (none(arg[5])) {
        dxt = empty({M, D}, {D, 1}, ht.scalar_type(), hm.device);
        dx.p = (char*)dxt.data_ptr();
        dx.ld = D;
    } else {
        dxt = THPVariable_Unpack(arg[5]);
    }
    const at::Tensor dw = empty({D}, {1}, at::kFloat, hm.device);
    // a workspace of this call's own: it belongs to the stream (and, under capture, to the graph)
    const int64_t bytes = gemm_rms_backward_workspace(M, D);
    at::Tensor ws;
    if (bytes > 0) ws = empty({bytes}, {1}, at::kByte, hm.device);
    void* const stream = raw_stream(hm.device);
    const int rc = enqueue([&] {
        return gemm_rms_backward(h, M, D, hm.type, w_type, dy.p, dy.ld, hm.p, hm.ld, w.data_ptr(),
                                 (const float*)rstd.data_ptr(), dh.p, dh.ld, dx.p, dx.ld, (float*)dw.data_ptr(),
                                 bytes > 0 ? ws.data_ptr() : nullptr, bytes, stream);
    });
    if (rc != GEMM_OK) return gemm_error(rc, "gemm_rms_backward");
    if (!none(arg[5])) written(dxt);
    return tuple_of({dxt, dw});
}

// ---- a feed-forward block in 16 bits ------------------------------------------

// A matrix of bfloat16 or float16 (of one type, where given).
Matrix halves(const at::Tensor& t, const char* what, int device = -1, int type = -1, int64_t rows = -1, int64_t cols = -1) {
    const Matrix m = matrix(t, what, kFloats, device, type, rows, cols);
    if (m.type == GEMM_F32) throw BadArgument{std::string(what) + " must be bfloat16 or float16"};
    return m;
}
Matrix halves_or_none(PyObject* o, const char* what, const Matrix& like, int64_t rows, int64_t cols) {
    return none(o) ? Matrix() : halves(tensor(o, what), what, like.device, like.type, rows, cols);
}
const void* bias_of(PyObject* o, const char* what, int64_t n, const Matrix& like, int* type) {
    if (none(o)) return nullptr;
    const at::Tensor& t = tensor(o, what);
    *type = vector(t, what, n, like.device, like.type);
    return t.data_ptr();
}
// A new M x N matrix, its rows one after another.
at::Tensor made_like(const at::Tensor& t, int64_t rows, int64_t cols, Matrix* m) {
    const at::Tensor made = empty({rows, cols}, {cols, 1}, t.scalar_type(), t.get_device());
    m->p = (char*)made.data_ptr();
    m->ld = cols;
    return made;
}
void same_k(const Matrix& a, int64_t k, const char* what) {
    if (a.cols != k)
        throw BadArgument{"inner dimensions differ: " + std::to_string(a.cols) + ", and " + std::to_string(k) + " of " + what};
}

Matrix row_of(const void* p, int64_t cols, int type) {
    Matrix m;
    m.p = (char*)p;
    m.rows = 1;
    m.cols = m.ld = cols;
    m.type = type;
    return m;
}
// Whether two matrices have a byte in common.
bool touch(const Matrix& x, const Matrix& y) {
    if (x.p == nullptr || y.p == nullptr) return false;
    const auto bytes = [](const Matrix& m) {
        const int64_t size = m.type == GEMM_F32 ? 4 : 2;
        return pg::ByteRows{(int64_t)m.p, m.rows, m.cols * size, m.ld * size};
    };
    return pg::rows_meet(bytes(x), bytes(y));
}
// What is written lies apart from everything else.
void apart(const Matrix& written, const char* what, std::initializer_list<Matrix> others) {
    for (const Matrix& o : others)
        if (touch(written, o)) throw BadArgument{std::string(what) + " overlaps another operand"};
}

// linear(a, b, layout, bias, activation, residual, a2, b2, keep, out, tile)
PyObject* linear_(PyObject* const* arg, Py_ssize_t n) {
    arguments(n, 11);
    const at::Tensor& at = tensor(arg[0], "a");
    const Matrix a = halves(at, "a");
    const Matrix b = halves(tensor(arg[1], "b"), "b", a.device, a.type);
    const int64_t layout = integer(arg[2]), act = integer(arg[4]), tile = integer(arg[10]);
    const bool rr = layout == GEMM_LAYOUT_RR, keep = truth(arg[8]);
    const int64_t M = a.rows, K = a.cols, N = rr ? b.cols : b.rows;
    same_k(a, rr ? b.rows : b.cols, "b");
    int bias_type = GEMM_F32;
    const void* const bias = bias_of(arg[3], "bias", N, a, &bias_type);
    const Matrix r = halves_or_none(arg[5], "residual", a, M, N);
    const Matrix a2 = halves_or_none(arg[6], "pair's a", a, M, K), b2 = halves_or_none(arg[7], "pair's b", a, b.rows, b.cols);
    // (an empty matrix has no address, which would read as none given)
    const bool second = a2.p != nullptr && b2.p != nullptr;
    Matrix c = halves_or_none(arg[9], "out", a, M, N), z;
    apart(c, "out", {a, b, a2, b2, row_of(bias, N, bias_type)});
    if (r.p != c.p || (r.ld != c.ld && M > 1)) apart(c, "out", {r});
    const gemm_handle_t h = handle_of(a.device);
    at::Tensor ct, zt;
    if (none(arg[9])) ct = made_like(at, M, N, &c);
    else ct = THPVariable_Unpack(arg[9]);
    if (keep) zt = made_like(at, M, N, &z);
    void* const stream = raw_stream(a.device);
    const int rc = enqueue([&] {
        return gemm_linear(h, M, N, K, a.type, (int)layout, (int)act, bias_type, (int)tile, a.p, a.ld, b.p, b.ld, second ? a2.p : nullptr,
                           a2.ld, second ? b2.p : nullptr, b2.ld, bias, r.p, r.ld, z.p, z.ld, c.p, c.ld, stream);
    });
    if (rc != GEMM_OK) return gemm_error(rc, "gemm_linear");
    if (!none(arg[9])) written(ct);
    return keep ? tuple_of({ct, zt}) : THPVariable_Wrap(std::move(ct));
}

// gated(x, gate, up, gate_bias, up_bias, activation, keep, out, tile)
PyObject* gated_(PyObject* const* arg, Py_ssize_t n) {
    arguments(n, 9);
    const at::Tensor& xt = tensor(arg[0], "x");
    const Matrix x = halves(xt, "x");
    const Matrix wg = halves(tensor(arg[1], "gate"), "gate", x.device, x.type);
    same_k(x, wg.cols, "gate");
    const int64_t M = x.rows, K = x.cols, N = wg.rows;
    const Matrix wu = halves(tensor(arg[2], "up"), "up", x.device, x.type, N, K);
    int type = GEMM_F32, type_u = GEMM_F32;
    const void* const bg = bias_of(arg[3], "gate_bias", N, x, &type);
    const void* const bu = bias_of(arg[4], "up_bias", N, x, &type_u);
    if (bg != nullptr && bu != nullptr && type != type_u) throw BadArgument{"the biases must be of one type"};
    if (bg == nullptr) type = type_u;
    const int64_t act = integer(arg[5]), tile = integer(arg[8]);
    const bool keep = truth(arg[6]);
    Matrix ho = halves_or_none(arg[7], "out", x, M, N), g, u;
    apart(ho, "out", {x, wg, wu, row_of(bg, N, type), row_of(bu, N, type)});
    const gemm_handle_t h = handle_of(x.device);
    at::Tensor ht, gt, ut;
    if (none(arg[7])) ht = made_like(xt, M, N, &ho);
    else ht = THPVariable_Unpack(arg[7]);
    if (keep) {
        gt = made_like(xt, M, N, &g);
        ut = made_like(xt, M, N, &u);
    }
    void* const stream = raw_stream(x.device);
    const int rc = enqueue([&] {
        return gemm_gated(h, M, N, K, x.type, (int)act, type, (int)tile, x.p, x.ld, wg.p, wg.ld, wu.p, wu.ld, bg, bu, g.p, g.ld,
                          u.p, u.ld, ho.p, ho.ld, stream);
    });
    if (rc != GEMM_OK) return gemm_error(rc, "gemm_gated");
    if (!none(arg[7])) written(ht);
    return keep ? tuple_of({ht, gt, ut}) : THPVariable_Wrap(std::move(ht));
}

// gated_backward(dy, w, g, u, activation, keep, tile)
PyObject* gated_backward_(PyObject* const* arg, Py_ssize_t n) {
    arguments(n, 7);
    const at::Tensor& dyt = tensor(arg[0], "dy");
    const Matrix dy = halves(dyt, "dy");
    const Matrix w = halves(tensor(arg[1], "w"), "w", dy.device, dy.type);
    same_k(dy, w.rows, "w");
    const int64_t M = dy.rows, K = dy.cols, N = w.cols, act = integer(arg[4]), tile = integer(arg[6]);
    const Matrix g = halves(tensor(arg[2], "g"), "g", dy.device, dy.type, M, N), u = halves_or_none(arg[3], "u", dy, M, N);
    const bool gate = !none(arg[3]), keep = truth(arg[5]);
    const gemm_handle_t h = handle_of(dy.device);
    Matrix dg, du, hm;
    at::Tensor dut, ht;
    at::Tensor dgt = made_like(dyt, M, N, &dg);
    if (gate) dut = made_like(dyt, M, N, &du);
    if (keep) ht = made_like(dyt, M, N, &hm);
    void* const stream = raw_stream(dy.device);
    const int rc = enqueue([&] {
        return gemm_gated_backward(h, M, N, K, dy.type, (int)act, (int)tile, dy.p, dy.ld, w.p, w.ld, g.p, g.ld, u.p, u.ld, dg.p,
                                   dg.ld, du.p, du.ld, hm.p, hm.ld, stream);
    });
    if (rc != GEMM_OK) return gemm_error(rc, "gemm_gated_backward");
    if (gate) return keep ? tuple_of({dgt, dut, ht}) : tuple_of({dgt, dut});
    return keep ? tuple_of({dgt, ht}) : THPVariable_Wrap(std::move(dgt));
}

// weight_gradient(dc, a, out, bias, bias_out, accumulate, tile)
PyObject* weight_gradient_(PyObject* const* arg, Py_ssize_t n) {
    arguments(n, 7);
    const Matrix dc = halves(tensor(arg[0], "dc"), "dc");
    const Matrix a = halves(tensor(arg[1], "a"), "a", dc.device, dc.type);
    if (a.rows != dc.rows)
        throw BadArgument{"dc and a must have as many rows (got " + std::to_string(dc.rows) + " and " + std::to_string(a.rows) + ")"};
    const int64_t M = dc.rows, N = dc.cols, K = a.cols, tile = integer(arg[6]);
    const bool bias = truth(arg[3]) || !none(arg[4]), accumulate = truth(arg[5]);
    if (accumulate && (none(arg[2]) || (bias && none(arg[4])))) throw BadArgument{"accumulate needs out (and bias_out for the bias)"};
    if (bias && K == 0 && N > 0) throw BadArgument{"the bias's gradient needs an input with columns"};
    Matrix dw;
    at::Tensor dwt, dbt;
    if (!none(arg[2])) {
        dwt = tensor(arg[2], "out");
        dw = matrix(dwt, "out", kFloats, dc.device, GEMM_F32, N, K);
    }
    if (!none(arg[4])) {
        dbt = tensor(arg[4], "bias_out");
        if (vector(dbt, "bias_out", N, dc.device, -1) != GEMM_F32) throw BadArgument{"bias_out must be float32"};
        apart(row_of(dbt.data_ptr(), N, GEMM_F32), "bias_out", {dc, a, dw});
    }
    apart(dw, "out", {dc, a});
    const gemm_handle_t h = handle_of(dc.device);
    if (none(arg[2])) {
        dwt = empty({N, K}, {K, 1}, at::kFloat, dc.device);
        dw.p = (char*)dwt.data_ptr();
        dw.ld = K;
    }
    if (bias && none(arg[4])) dbt = empty({N}, {1}, at::kFloat, dc.device);
    void* const stream = raw_stream(dc.device);
    const int rc = enqueue([&] {
        return gemm_weight_gradient(h, M, N, K, dc.type, accumulate, (int)tile, dc.p, dc.ld, a.p, a.ld, (float*)dw.p, dw.ld,
                                    bias ? (float*)dbt.data_ptr() : nullptr, stream);
    });
    if (rc != GEMM_OK) return gemm_error(rc, "gemm_weight_gradient");
    if (!none(arg[2])) written(dwt);
    if (!none(arg[4])) written(dbt);
    return bias ? tuple_of({dwt, dbt}) : THPVariable_Wrap(std::move(dwt));
}

// C++ errors as Python's.
template <PyObject* (*F)(PyObject* const*, Py_ssize_t)>
PyObject* guarded(PyObject*, PyObject* const* arg, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    try {
        return F(arg, n);
    } catch (const BadArgument& e) {
        PyErr_SetString(PyExc_ValueError, e.text.c_str());
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

PyMethodDef g_methods[] = {
    {"run_fp8", (PyCFunction)(void (*)())&guarded<run_fp8_>, METH_FASTCALL, nullptr},
    {"quantize_fp8", (PyCFunction)(void (*)())&guarded<quantize_fp8_>, METH_FASTCALL, nullptr},
    {"rms_fp8", (PyCFunction)(void (*)())&guarded<rms_fp8_>, METH_FASTCALL, nullptr},
    {"rms_backward", (PyCFunction)(void (*)())&guarded<rms_backward_>, METH_FASTCALL, nullptr},
    {"linear", (PyCFunction)(void (*)())&guarded<linear_>, METH_FASTCALL, nullptr},
    {"gated", (PyCFunction)(void (*)())&guarded<gated_>, METH_FASTCALL, nullptr},
    {"gated_backward", (PyCFunction)(void (*)())&guarded<gated_backward_>, METH_FASTCALL, nullptr},
    {"weight_gradient", (PyCFunction)(void (*)())&guarded<weight_gradient_>, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_torch_ops", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__torch_ops(void) { return PyModule_Create(&g_module); }
