// The operators' calls from Python: checks of tensors, outputs and workspaces from torch's allocator,
// and one call of the C ABI each, on the current stream of the tensors' device.
//
// A call of a few microseconds of GPU time is bound by what surrounds it on the host.  With the same steps
// in Python and ctypes a layer norm of one row takes 10.1 us, of which the launch is 3.1; here 5.3.
// Arguments come by position (the functions that users call, with their documentation, are in __init__.py).
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/core/DeviceGuard.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include <sstream>
#include <stdexcept>
#include <string>

#include "../../include/tsgemm.h"
#include "limits.hpp"

namespace {

using at::ScalarType;
using at::Tensor;

PyObject* g_error = nullptr;   // the package's TsError

struct Refusal : std::runtime_error {   // ValueError
    using std::runtime_error::runtime_error;
};
struct WrongType : std::runtime_error {   // TypeError
    using std::runtime_error::runtime_error;
};
struct Failed {   // TsError
    int64_t status;
};
struct Raised {};   // Python's own error, already set

// ---- arguments ---------------------------------------------------------------------------

const Tensor& tensor(PyObject* o, const char* what) {
    if (!THPVariable_Check(o)) throw WrongType(std::string(what) + " must be a tensor");
    return THPVariable_Unpack(o);
}
// A tensor, or null for None.
const Tensor* maybe(PyObject* o, const char* what) { return o == Py_None ? nullptr : &tensor(o, what); }
int64_t number(PyObject* o) {
    const int64_t v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) {
        PyErr_Clear();
        throw WrongType("an integer is required");
    }
    return v;
}
float real(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) {
        PyErr_Clear();
        throw WrongType("eps must be a number");
    }
    return (float)v;
}
bool flag(PyObject* o) {
    const int truth = PyObject_IsTrue(o);
    if (truth < 0) throw Raised();
    return truth == 1;
}
// A dtype, or `none` for None.
ScalarType dtype(PyObject* o, ScalarType none) {
    if (o == Py_None) return none;
    if (!THPDtype_Check(o)) throw WrongType("a torch.dtype is required");
    return reinterpret_cast<THPDtype*>(o)->scalar_type;
}

int32_t code(ScalarType t) {
    switch (t) {
        case at::kHalf: return TS_F16;
        case at::kBFloat16: return TS_BF16;
        case at::kFloat: return TS_F32;
        case at::kFloat8_e4m3fn: return TS_E4M3;
        case at::kChar: return TS_I8;
        default: return 0;   // refused by the library
    }
}
int32_t row_code(ScalarType t) {
    const int32_t c = code(t);
    return c <= TS_F32 ? c : 0;
}
bool eight_bit(ScalarType t) { return t == at::kFloat8_e4m3fn || t == at::kChar; }
std::string name(ScalarType t) {
    switch (t) {
        case at::kHalf: return "torch.float16";
        case at::kBFloat16: return "torch.bfloat16";
        case at::kFloat: return "torch.float32";
        case at::kDouble: return "torch.float64";
        case at::kFloat8_e4m3fn: return "torch.float8_e4m3fn";
        case at::kChar: return "torch.int8";
        case at::kByte: return "torch.uint8";
        default: return c10::toString(t);
    }
}
std::string shape(at::IntArrayRef s) {
    std::ostringstream o;
    o << "(";
    for (size_t i = 0; i < s.size(); ++i) o << (i ? ", " : "") << s[i];
    o << (s.size() == 1 ? ",)" : ")");
    return o.str();
}

constexpr ScalarType kAny = ScalarType::Undefined;

// Row stride of an M x N matrix with unit column stride, after its checks.
int64_t rows(const Tensor& t, int64_t M, int64_t N, const char* what, ScalarType type = kAny) {
    if (t.dim() != 2 || t.size(0) != M || t.size(1) != N)
        throw Refusal(std::string(what) + " has shape " + shape(t.sizes()) + ", expected " + shape({M, N}));
    if (type != kAny && t.scalar_type() != type)
        throw Refusal(std::string(what) + " is " + name(t.scalar_type()) + ", expected " + name(type));
    if (N > 1 && t.stride(1) != 1) throw Refusal(std::string(what) + " must have unit stride along its rows");
    return t.stride(0);
}
// What a Checkpoint's constructor has seen may have been changed since: whether its data still holds n columns a row.
// (Rows that are not 16-byte aligned are refused by the library.)
void kept_data(const Tensor& data, int64_t n) {
    if (data.dim() != 2 || data.scalar_type() != at::kByte || (data.size(1) > 1 && data.stride(1) != 1) || n < 0 ||
        n > INT32_MAX || data.size(1) < 33 * ((n + 31) / 32))
        throw Refusal("a checkpoint's data " + name(data.scalar_type()) + " " + shape(data.sizes()) + " does not hold rows of " +
                      std::to_string(n) + " columns");
}
// A checkpoint's rows: its bytes and the number of columns that they hold.
int64_t kept_rows(const Tensor& data, int64_t n, int64_t M, int64_t N, const char* what) {
    kept_data(data, n);
    if (data.size(0) != M || n != N)
        throw Refusal(std::string(what) + " has shape " + shape({data.size(0), n}) + ", expected " + shape({M, N}));
    return data.stride(0);
}
void vector(const Tensor& t, int64_t n, const char* what, ScalarType type = kAny) {
    if (t.dim() != 1 || t.size(0) != n || (n > 1 && t.stride(0) != 1))
        throw Refusal(std::string(what) + " must be a contiguous vector of " + std::to_string(n));
    if (type != kAny && t.scalar_type() != type)
        throw Refusal(std::string(what) + " is " + name(t.scalar_type()) + ", expected " + name(type));
    if (!row_code(t.scalar_type())) throw Refusal(std::string(what) + " is " + name(t.scalar_type()));
}
void matrix_of_rows(const Tensor& t, const char* what) {
    if (t.dim() != 2) throw Refusal(std::string(what) + " must be a matrix of rows");
}
void* ptr(const Tensor* t) { return t ? t->data_ptr() : nullptr; }

// The one GPU that every given tensor is on.
template <class... T>
c10::Device device_of(const Tensor& first, const T*... others) {
    const auto index = first.get_device();
    for (const Tensor* t : {others...})
        if (t && t->get_device() != index) throw Refusal("all tensors must be on the same GPU");
    if (index < 0) throw Refusal("tensors must be on a GPU");
    return first.device();
}
// That device, current for one call, and its current stream.
struct Launch {
    c10::DeviceGuard guard;
    void* stream;
    explicit Launch(c10::Device d) : guard(d), stream(c10::hip::getCurrentHIPStream(d.index()).stream()) {}
};
// One call of the library, other Python threads running meanwhile (a full queue makes a launch wait).
template <class F>
void run(F&& f) {
    PyThreadState* state = PyEval_SaveThread();
    const ts_status status = f();
    PyEval_RestoreThread(state);
    if (status != TS_OK) throw Failed{status};
}
Tensor empty(at::IntArrayRef size, ScalarType type, const Tensor& like) { return at::empty(size, like.options().dtype(type)); }
// A workspace of the call's own, from torch's allocator: calls on other streams, and graphs
// captured one after the other, never share one.
struct Scratch {
    Tensor t;
    int64_t bytes;
    Scratch(int64_t need, const Tensor& like) : bytes(need) {
        if (need < 0) throw Failed{need};
        if (need) t = empty({need}, at::kByte, like);
    }
    void* ptr() const { return bytes ? t.data_ptr() : nullptr; }
};

PyObject* wrap(const Tensor& t) { return THPVariable_Wrap(t); }
PyObject* same(PyObject* o) {
    Py_INCREF(o);
    return o;
}
PyObject* wrap_or_none(const Tensor& t) { return t.defined() ? wrap(t) : same(Py_None); }
PyObject* tuple(std::initializer_list<PyObject*> v) {
    PyObject* r = PyTuple_New((Py_ssize_t)v.size());
    Py_ssize_t i = 0;
    for (PyObject* o : v) PyTuple_SET_ITEM(r, i++, o);
    return r;
}

// A call: `n` arguments by position, errors as Python's.
template <int N, PyObject* (*F)(PyObject* const*)>
PyObject* call(PyObject*, PyObject* const* a, Py_ssize_t n) {
    try {
        if (n != N) throw WrongType("wrong number of arguments");
        at::AutoDispatchBelowADInplaceOrView below;   // autograd does not see these calls
        return F(a);
    } catch (const Raised&) {
    } catch (const Failed& e) {
        PyObject* status = PyLong_FromLongLong(e.status);
        PyObject* error = PyObject_CallFunctionObjArgs(g_error, status, nullptr);
        Py_DECREF(status);
        if (error) {
            PyErr_SetObject(g_error, error);
            Py_DECREF(error);
        }
    } catch (const Refusal& e) {
        PyErr_SetString(PyExc_ValueError, e.what());
    } catch (const WrongType& e) {
        PyErr_SetString(PyExc_TypeError, e.what());
    } catch (const c10::OutOfMemoryError& e) {
        PyObject* torch = PyImport_ImportModule("torch");
        PyObject* oom = torch ? PyObject_GetAttrString(torch, "OutOfMemoryError") : nullptr;
        PyErr_SetString(oom ? oom : PyExc_MemoryError, e.what_without_backtrace());
        Py_XDECREF(oom);
        Py_XDECREF(torch);
    } catch (const c10::Error& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what_without_backtrace());
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

// ---- products ----------------------------------------------------------------------------

// a, b, out, out_dtype, activation, grad, schedule (address or 0), residual, preact, columns of a checkpoint's
// preact (-1: a tensor), bias, scale_a, scale_b
PyObject* product(PyObject* const* p) {
    const Tensor &a = tensor(p[0], "A"), &b = tensor(p[1], "B");
    if (a.dim() != 2 || b.dim() != 2 || a.size(1) != b.size(0))
        throw Refusal("shapes " + shape(a.sizes()) + " @ " + shape(b.sizes()) + " do not multiply");
    if (a.scalar_type() != b.scalar_type())
        throw Refusal("A is " + name(a.scalar_type()) + ", B is " + name(b.scalar_type()));
    const Tensor *out = maybe(p[2], "out"), *residual = maybe(p[7], "residual"), *preact = maybe(p[8], "preact"),
                 *bias = maybe(p[10], "bias"), *scale_a = maybe(p[11], "scale_a"), *scale_b = maybe(p[12], "scale_b");
    const int64_t kept_n = number(p[9]), M = a.size(0), K = a.size(1), N = b.size(1);
    if (preact && kept_n >= 0) kept_data(*preact, kept_n);
    const c10::Device dev = device_of(a, &b, out, bias, residual, preact, scale_a, scale_b);
    const ScalarType type = dtype(p[3], a.scalar_type());
    if (out && (out->dim() != 2 || out->size(0) != M || out->size(1) != N || out->scalar_type() != type))
        throw Refusal("out has the wrong shape or type");
    ts_epilogue e = {};
    e.activation = (int32_t)number(p[4]);
    e.grad = (int32_t)number(p[5]);
    if (residual) {
        e.stride_rm = rows(*residual, M, N, "residual", type);
        e.residual = residual->data_ptr();
    }
    if (preact) {
        if (kept_n >= 0) e.preact_dtype = TS_Q8;
        e.stride_pm = kept_n >= 0 ? kept_rows(*preact, kept_n, M, N, "preact") : rows(*preact, M, N, "preact", type);
        e.preact = preact->data_ptr();
    }
    if (bias) {
        vector(*bias, N, "bias");
        e.bias = bias->data_ptr();
        e.bias_dtype = code(bias->scalar_type());
    }
    if (scale_a) {
        vector(*scale_a, M, "scale_a", at::kFloat);
        e.scale_a = static_cast<const float*>(scale_a->data_ptr());
    }
    if (scale_b) {
        vector(*scale_b, N, "scale_b", at::kFloat);
        e.scale_b = static_cast<const float*>(scale_b->data_ptr());
    }
    const ts_schedule* s = reinterpret_cast<const ts_schedule*>((uintptr_t)number(p[6]));
    const void *pa = a.data_ptr(), *pb = b.data_ptr();
    const bool work = M && N && K;
    if (work && out && (out->data_ptr() == pa || out->data_ptr() == pb))
        throw Refusal("out must not be an operand of the product");
    if (work && e.preact && !e.grad && (e.preact == pa || e.preact == pb))
        throw Refusal("preact must not be an operand of the product");
    Launch l(dev);
    const Tensor made = out ? Tensor() : empty({M, N}, type, a);
    const Tensor& c = out ? *out : made;
    const int32_t ab_t = code(a.scalar_type()), c_t = code(type);
    const Scratch ws(ts_gemm_epilogue_workspace(pa, pb, M, N, K, a.stride(0), a.stride(1), b.stride(0), b.stride(1), ab_t,
                                                c_t, s), a);
    run([&] {
        return ts_gemm_epilogue(pa, pb, c.data_ptr(), M, N, K, a.stride(0), a.stride(1), b.stride(0), b.stride(1),
                                c.stride(0), c.stride(1), ab_t, c_t, &e, s, l.stream, ws.ptr(), ws.bytes);
    });
    return out ? same(p[2]) : wrap(made);
}

// dc, preact, columns of a checkpoint's preact (-1: a tensor), activation, out, out_dtype, dbias, dbias_dtype, act_out
PyObject* act_grad(PyObject* const* p) {
    const Tensor& dc = tensor(p[0], "dC");
    if (dc.dim() != 2) throw Refusal("dC must be a matrix");
    const int64_t M = dc.size(0), N = dc.size(1), kept_n = number(p[2]);
    const int32_t act = (int32_t)number(p[3]);
    const Tensor *out = maybe(p[4], "out"), *value = maybe(p[8], "act_out"), *preact = maybe(p[1], "preact");
    const bool reads = act || value, dbias = flag(p[6]);
    if (reads && !preact) throw Refusal("preact is needed for this activation");
    if (!reads) preact = nullptr;
    const bool kept = preact && kept_n >= 0;
    const ScalarType in = dc.scalar_type();
    const int64_t ldc = rows(dc, M, N, "dC");
    const int64_t ldz = kept ? kept_rows(*preact, kept_n, M, N, "preact") : preact ? rows(*preact, M, N, "preact", in) : N;
    const bool make = !out && (act || dtype(p[5], in) != in);
    const c10::Device dev = device_of(dc, preact, out, value);
    const ScalarType dz_t = out ? out->scalar_type() : make ? dtype(p[5], in) : in;
    const ScalarType out_t = out || make ? dz_t : value ? value->scalar_type() : in;
    const int64_t ldo = out ? rows(*out, M, N, "out", dtype(p[5], kAny)) : N;
    const int64_t ldv = value ? rows(*value, M, N, "act_out", out || make ? dz_t : kAny) : N;
    if (!out && !make && !dbias && !value) return tuple({same(p[0]), same(Py_None)});
    Launch l(dev);
    const Tensor made = make ? empty({M, N}, dz_t, dc) : Tensor();
    const ScalarType db_t = dtype(p[7], at::kFloat);
    const Tensor db = dbias ? empty({N}, db_t, dc) : Tensor();
    const Scratch ws(dbias ? ts_act_grad_workspace(M, N) : 0, dc);
    void* dz = out ? out->data_ptr() : make ? made.data_ptr() : nullptr;
    run([&] {
        return ts_act_grad_value(dc.data_ptr(), ptr(preact), dz, ptr(value), dbias ? db.data_ptr() : nullptr, M, N,
                                 ldc, ldz, ldo, ldv, row_code(in), kept ? TS_Q8 : row_code(in), row_code(out_t),
                                 row_code(db_t), act, l.stream, ws.ptr(), ws.bytes);
    });
    return tuple({out ? same(p[4]) : make ? wrap(made) : same(p[0]), wrap_or_none(db)});
}

// ---- rows --------------------------------------------------------------------------------

// What the two norms have in common: the outputs of a forward pass.
struct Norm {
    const Tensor &x, *residual, *out, *h;
    int64_t M, N, ldx, ldy, ldr, ldh;
    ScalarType type, y_t;
    Tensor made_y, made_h, scale;
    void* y;
    PyObject *po, *ph, *px;
    Norm(PyObject* x_, PyObject* residual_, PyObject* out_dtype, PyObject* out_, PyObject* h_)
        : x(tensor(x_, "x")), residual(maybe(residual_, "residual")), out(maybe(out_, "out")), h(maybe(h_, "h")),
          po(out_), ph(h_), px(x_) {
        matrix_of_rows(x, "x");
        if (h && !residual) throw Refusal("h is written only with a residual");
        M = x.size(0);
        N = x.size(1);
        type = x.scalar_type();
        y_t = dtype(out_dtype, out ? out->scalar_type() : type);
        ldx = rows(x, M, N, "x");
        ldy = out ? rows(*out, M, N, "out", y_t) : N;
        ldr = residual ? rows(*residual, M, N, "residual", type) : N;
        ldh = h ? rows(*h, M, N, "h", type) : N;
    }
    void make() {
        if (!out) made_y = empty({M, N}, y_t, x);
        if (residual && !h) made_h = empty({M, N}, type, x);
        if (eight_bit(y_t)) scale = empty({M}, at::kFloat, x);
        y = out ? out->data_ptr() : made_y.data_ptr();
    }
    void* h_ptr() const { return h ? h->data_ptr() : residual ? made_h.data_ptr() : nullptr; }
    float* scale_ptr() const { return scale.defined() ? static_cast<float*>(scale.data_ptr()) : nullptr; }
    PyObject* result() const {
        return tuple({out ? same(po) : wrap(made_y), wrap_or_none(scale), h ? same(ph) : residual ? wrap(made_h) : same(px)});
    }
};

// x, weight, residual, eps, out_dtype, out, h
PyObject* rmsnorm(PyObject* const* p) {
    Norm n(p[0], p[2], p[4], p[5], p[6]);
    const Tensor* w = maybe(p[1], "weight");
    if (w) vector(*w, n.N, "weight");
    const float eps = real(p[3]);
    Launch l(device_of(n.x, w, n.residual, n.out, n.h));
    n.make();
    run([&] {
        return ts_rmsnorm(n.x.data_ptr(), ptr(n.residual), ptr(w), n.y, n.h_ptr(), n.scale_ptr(), n.M, n.N, n.ldx,
                          n.ldr, n.ldy, n.ldh, row_code(n.type), w ? code(w->scalar_type()) : TS_F32, code(n.y_t),
                          eps, l.stream);
    });
    return n.result();
}

// x, weight, bias, residual, eps, out_dtype, out, h, checkpoint's data, its columns
PyObject* layernorm(PyObject* const* p) {
    Norm n(p[0], p[3], p[5], p[6], p[7]);
    const Tensor *w = maybe(p[1], "weight"), *b = maybe(p[2], "bias"), *keep = maybe(p[8], "keep");
    if (w) vector(*w, n.N, "weight");
    if (b) vector(*b, n.N, "bias", w ? w->scalar_type() : kAny);
    const float eps = real(p[4]);
    const int64_t ldk = keep ? kept_rows(*keep, number(p[9]), n.M, n.N, "keep") : n.N;
    Launch l(device_of(n.x, w, b, n.residual, n.out, n.h, keep));
    n.make();
    run([&] {
        return ts_layernorm(n.x.data_ptr(), ptr(n.residual), ptr(w), ptr(b), n.y, n.h_ptr(), n.scale_ptr(),
                            ptr(keep), n.M, n.N, n.ldx, n.ldr, n.ldy, n.ldh, ldk, row_code(n.type), w ?
                            code(w->scalar_type()) : b ? code(b->scalar_type()) : TS_F32, code(n.y_t), eps,
                            l.stream);
    });
    return n.result();
}

// What the gradients of the two norms have in common.
struct NormGrad {
    const Tensor &dy, &h, *weight, *dh, *out;
    bool kept;
    int64_t M, N, ldy, ldh, lds, ldx;
    ScalarType type;
    Tensor made;
    PyObject* po;
    NormGrad(PyObject* dy_, PyObject* h_, int64_t kept_n, PyObject* weight_, PyObject* dh_, PyObject* out_)
        : dy(tensor(dy_, "dy")), h(tensor(h_, "h")), weight(maybe(weight_, "weight")), dh(maybe(dh_, "dh")),
          out(maybe(out_, "out")), kept(kept_n >= 0), po(out_) {
        matrix_of_rows(dy, "dy");
        M = dy.size(0);
        N = dy.size(1);
        type = dy.scalar_type();
        ldy = rows(dy, M, N, "dy");
        ldh = kept ? kept_rows(h, kept_n, M, N, "h") : rows(h, M, N, "h", type);
        ldx = out ? rows(*out, M, N, "out", type) : N;
        lds = dh ? rows(*dh, M, N, "dh", type) : N;
        if (weight) vector(*weight, N, "weight");
    }
    void* dx() {
        if (!out) made = empty({M, N}, type, dy);
        return out ? out->data_ptr() : made.data_ptr();
    }
    PyObject* dx_object() const { return out ? same(po) : wrap(made); }
};

// dy, h, weight, eps, dh, dweight, out
PyObject* rmsnorm_backward(PyObject* const* p) {
    NormGrad n(p[0], p[1], -1, p[2], p[4], p[6]);
    const float eps = real(p[3]);
    const bool dweight = flag(p[5]);
    Launch l(device_of(n.dy, &n.h, n.weight, n.dh, n.out));
    void* dx = n.dx();
    const Tensor dw = n.weight && dweight ? empty({n.N}, n.weight->scalar_type(), n.dy) : Tensor();
    const Scratch ws(dw.defined() || n.N > ts::kRmsGradRow ? ts_rmsnorm_backward_workspace(n.M, n.N) : 0, n.dy);
    run([&] {
        return ts_rmsnorm_backward(n.dy.data_ptr(), n.h.data_ptr(), ptr(n.weight), ptr(n.dh), dx, dw.defined() ?
                                   dw.data_ptr() : nullptr, n.M, n.N, n.ldy, n.ldh, n.lds, n.ldx, row_code(n.type),
                                   n.weight ? code(n.weight->scalar_type()) : TS_F32, eps, l.stream, ws.ptr(),
                                   ws.bytes);
    });
    return tuple({n.dx_object(), wrap_or_none(dw)});
}

// dy, h, columns of a checkpoint's h (-1: a tensor), weight, eps, dh, dweight, dbias, dbias_dtype, out
PyObject* layernorm_backward(PyObject* const* p) {
    NormGrad n(p[0], p[1], number(p[2]), p[3], p[5], p[9]);
    const float eps = real(p[4]);
    const bool dweight = flag(p[6]), dbias = flag(p[7]);
    const ScalarType asked = dtype(p[8], kAny), sums = n.weight ? n.weight->scalar_type() : asked == kAny ? at::kFloat : asked;
    if (n.weight && asked != kAny && asked != sums) throw Refusal("dbias has weight's type");
    Launch l(device_of(n.dy, &n.h, n.weight, n.dh, n.out));
    void* dx = n.dx();
    const Tensor dw = n.weight && dweight ? empty({n.N}, sums, n.dy) : Tensor(), db = dbias ? empty({n.N}, sums, n.dy) : Tensor();
    const Scratch ws(dw.defined() || db.defined() || n.N > ts::kLayerGradRow ? ts_layernorm_backward_workspace(n.M, n.N) : 0, n.dy);
    run([&] {
        return ts_layernorm_backward(n.dy.data_ptr(), n.h.data_ptr(), ptr(n.weight), ptr(n.dh), dx, dw.defined() ?
                                     dw.data_ptr() : nullptr, db.defined() ? db.data_ptr() : nullptr, n.M, n.N,
                                     n.ldy, n.ldh, n.lds, n.ldx, row_code(n.type), n.kept ? TS_Q8 :
                                     row_code(n.type), row_code(sums), eps, l.stream, ws.ptr(), ws.bytes);
    });
    return tuple({n.dx_object(), wrap_or_none(dw), wrap_or_none(db)});
}

// x, out_dtype, out
PyObject* quantize_rows(PyObject* const* p) {
    const Tensor &x = tensor(p[0], "x"), *out = maybe(p[2], "out");
    matrix_of_rows(x, "x");
    const int64_t M = x.size(0), N = x.size(1);
    const ScalarType to = dtype(p[1], at::kChar);
    const int64_t ldx = rows(x, M, N, "x"), ldy = out ? rows(*out, M, N, "out", to) : N;
    Launch l(device_of(x, out));
    const Tensor made = out ? Tensor() : empty({M, N}, to, x), scale = empty({M}, at::kFloat, x);
    run([&] {
        return ts_quantize_rows(x.data_ptr(), out ? out->data_ptr() : made.data_ptr(),
                                static_cast<float*>(scale.data_ptr()), M, N, ldx, ldy, row_code(x.scalar_type()),
                                code(to), l.stream);
    });
    return tuple({out ? same(p[2]) : wrap(made), wrap(scale)});
}

int64_t kept_pitch(int64_t n) { return (33 * ((n + 31) / 32) + 63) / 64 * 64; }

// x, checkpoint's data or None, its columns; returns the data
PyObject* checkpoint_pack(PyObject* const* p) {
    const Tensor &x = tensor(p[0], "x"), *out = maybe(p[1], "out");
    matrix_of_rows(x, "x");
    const int64_t M = x.size(0), N = x.size(1), ldx = rows(x, M, N, "x");
    if (out) kept_rows(*out, number(p[2]), M, N, "out");
    Launch l(device_of(x, out));
    const Tensor made = out ? Tensor() : empty({M, kept_pitch(N)}, at::kByte, x);
    const Tensor& d = out ? *out : made;
    run([&] {
        return ts_checkpoint_pack(x.data_ptr(), d.data_ptr(), M, N, ldx, d.stride(0), row_code(x.scalar_type()),
                                  l.stream);
    });
    return out ? same(p[1]) : wrap(made);
}

// checkpoint's data, its columns, activation, out, out_dtype
PyObject* checkpoint_unpack(PyObject* const* p) {
    const Tensor &d = tensor(p[0], "kept"), *out = maybe(p[3], "out");
    const int64_t N = number(p[1]);
    kept_data(d, N);
    const int64_t M = d.size(0);
    const int32_t act = (int32_t)number(p[2]);
    const ScalarType to = dtype(p[4], out ? out->scalar_type() : at::kFloat);
    const int64_t ldo = out ? rows(*out, M, N, "out", to) : N;
    Launch l(device_of(d, out));
    const Tensor made = out ? Tensor() : empty({M, N}, to, d);
    run([&] {
        return ts_checkpoint_unpack(d.data_ptr(), out ? out->data_ptr() : made.data_ptr(), M, N, d.stride(0), ldo,
                                    row_code(to), act, l.stream);
    });
    return out ? same(p[3]) : wrap(made);
}

PyObject* set_error(PyObject*, PyObject* type) {
    Py_INCREF(type);
    Py_XSETREF(g_error, type);
    Py_RETURN_NONE;
}

#define TS_CALL(F, N) {#F, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&call<N, F>)), METH_FASTCALL, nullptr}
PyMethodDef kMethods[] = {
    {"set_error", set_error, METH_O, nullptr},
    TS_CALL(product, 13), TS_CALL(act_grad, 9), TS_CALL(rmsnorm, 7), TS_CALL(layernorm, 10), TS_CALL(rmsnorm_backward, 7),
    TS_CALL(layernorm_backward, 10), TS_CALL(quantize_rows, 3), TS_CALL(checkpoint_pack, 3), TS_CALL(checkpoint_unpack, 5),
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() {
    PyObject* module = PyModule_Create(&kModule);
    if (module && PyModule_AddStringConstant(module, "built_for", TS_BUILT_FOR) < 0) {   // the package compares it with what runs
        Py_DECREF(module);
        return nullptr;
    }
    return module;
}
