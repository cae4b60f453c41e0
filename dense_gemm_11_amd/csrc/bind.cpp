// Marshalling of the calls around an expert layer's products (run_route to
// run_grouped_act_grad): checks torch tensors and makes the C calls of
// include/dense_gemm.h with their pointers.  A decoding loop makes these calls per
// token, where their kernels take 3 to 6 us and the same checks in Python, with
// ctypes' conversions, took 4 to 5.  Called positionally by the package, which
// documents the arguments; a call returns the library's status or raises
// TypeError (dtypes) or ValueError (shapes, strides, devices).
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <torch/csrc/autograd/python_variable.h>

#include <exception>
#include <string>

#include "dense_gemm.h"

namespace {

struct Failure : std::exception {
    PyObject* type;
    std::string text;
    Failure(PyObject* t, std::string s) : type(t), text(std::move(s)) {}
    const char* what() const noexcept override { return text.c_str(); }
};
[[noreturn]] void wrong_value(std::string s) { throw Failure(PyExc_ValueError, std::move(s)); }
[[noreturn]] void wrong_type(std::string s) { throw Failure(PyExc_TypeError, std::move(s)); }
// A conversion has set Python's error already.
struct Raised {};

const at::Tensor& tensor(PyObject* o, const char* name)
{
    if (!THPVariable_Check(o)) wrong_type(std::string(name) + " must be a tensor");
    return THPVariable_Unpack(o);
}
const at::Tensor* maybe(PyObject* o, const char* name) { return o == Py_None ? nullptr : &tensor(o, name); }

int64_t integer(PyObject* o)
{
    const int64_t v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw Raised();
    return v;
}
// ... that fits an int: others become -1, which the library refuses.
int small(PyObject* o)
{
    const int64_t v = integer(o);
    return v < INT32_MIN || v > INT32_MAX ? -1 : (int)v;
}
float number(PyObject* o)
{
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw Raised();
    return (float)v;
}
bool truth(PyObject* o)
{
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw Raised();
    return v != 0;
}
void* pointer(PyObject* o)  // an address, or None
{
    if (o == Py_None) return nullptr;
    void* p = PyLong_AsVoidPtr(o);
    if (!p && PyErr_Occurred()) throw Raised();
    return p;
}

// The device that a call's tensors share.
struct Device {
    int index;
    explicit Device(const at::Tensor& t) : index(t.is_cuda() ? t.get_device() : -1)
    {
        if (index < 0) wrong_value("the tensors must be on a GPU");
    }
    void holds(const at::Tensor& t, const char* name) const
    {
        if (!t.is_cuda() || t.get_device() != index)
            wrong_value(std::string(name) + " must be on the other tensors' device");
    }
};

struct Matrix {
    void* p;
    int64_t rows, cols, ld;
};
// A 2-D tensor with unit stride in its last axis.  (A single row has no stride of
// its own; too small a one, of an expanded tensor, is refused by the library.)
Matrix matrix(const at::Tensor& t, const char* name)
{
    if (t.dim() != 2 || (t.size(1) > 1 && t.stride(1) != 1))
        wrong_value(std::string(name) + " must be a 2-D tensor with unit stride in its last axis");
    const int64_t rows = t.size(0), cols = t.size(1);
    return {t.data_ptr(), rows, cols, rows > 1 ? t.stride(0) : cols > 1 ? cols : 1};
}
// ... of this shape and dtype on the device, or absent.
Matrix shaped(const at::Tensor* t, at::ScalarType type, int64_t rows, int64_t cols, const Device& device,
              const char* name)
{
    if (!t) return {nullptr, rows, cols, cols > 1 ? cols : 1};
    if (t->scalar_type() != type) wrong_type(std::string(name) + " has the wrong dtype");
    const Matrix m = matrix(*t, name);
    if (m.rows != rows || m.cols != cols)
        wrong_value(std::string(name) + " must be " + std::to_string(rows) + " x " + std::to_string(cols));
    device.holds(*t, name);
    return m;
}
// Address of a packed tensor of this shape (cols < 0: a vector), dtype and device,
// or of none.
void* packed(const at::Tensor* t, at::ScalarType type, int64_t rows, int64_t cols, const Device& device,
             const char* name)
{
    if (!t) return nullptr;
    const bool fits = cols < 0 ? t->dim() == 1 && t->size(0) == rows
                               : t->dim() == 2 && t->size(0) == rows && t->size(1) == cols;
    if (!fits || t->scalar_type() != type || !t->is_contiguous())
        wrong_value(std::string(name) + " must be a contiguous " +
                    (type == at::kInt ? "int32" : "float32") + " tensor of " + std::to_string(rows) +
                    (cols < 0 ? "" : " x " + std::to_string(cols)));
    device.holds(*t, name);
    return t->data_ptr();
}
template <typename T>
T* packed_as(PyObject* o, int64_t rows, int64_t cols, const Device& device, const char* name)
{
    return static_cast<T*>(packed(maybe(o, name), sizeof(T) == sizeof(int32_t) && std::is_integral_v<T>
                                                      ? at::kInt : at::kFloat,
                                  rows, cols, device, name));
}

// The types of operands and outputs.
gemm_dtype_t two_types(at::ScalarType in, at::ScalarType out)
{
    if (in == at::kFloat && out == at::kFloat) return GEMM_DTYPE_F32;
    if (in == at::kBFloat16 && out == at::kBFloat16) return GEMM_DTYPE_BF16_BF16;
    if (in == at::kBFloat16 && out == at::kFloat) return GEMM_DTYPE_BF16_F32;
    wrong_type("operands must be float32, or bfloat16 with float32 or bfloat16 outputs");
}
gemm_dtype_t logits_type(const at::Tensor& t)
{
    if (t.scalar_type() == at::kFloat) return GEMM_DTYPE_F32;
    if (t.scalar_type() == at::kBFloat16) return GEMM_DTYPE_BF16_BF16;
    wrong_type("logits must be float32 or bfloat16");
}
void same_type(const at::Tensor& a, const at::Tensor* b, const char* text)
{
    if (b && a.scalar_type() != b->scalar_type()) wrong_type(text);
}
int64_t columns(PyObject* o, const char* name)
{
    const at::Tensor& t = tensor(o, name);
    if (t.dim() != 2) wrong_value(std::string(name) + " must be tokens x top");
    return t.size(1);
}
int as_int(int64_t v) { return v > INT32_MAX ? -1 : (int)v; }

// A workspace, whose bytes count from its first one.
struct Workspace {
    const at::Tensor* t;
    explicit Workspace(PyObject* o) : t(maybe(o, "workspace"))
    {
        if (t && !t->is_contiguous()) wrong_value("the workspace must be contiguous");
    }
    void* on(const Device& device) const
    {
        if (t) device.holds(*t, "the workspace");
        return t ? t->data_ptr() : nullptr;
    }
    size_t bytes() const { return t ? t->nbytes() : 0; }
};

// GROUPS: offsets of `groups` groups (None: no groups) and their scales.
struct Groups : gemm_groups_t {
    bool any;
    Groups(PyObject* offsets, PyObject* scales, int64_t count, const Device& device)
        : gemm_groups_t{as_int(count), nullptr, nullptr}, any(offsets != Py_None)
    {
        if (!any) {
            if (scales != Py_None) wrong_value("scales are the groups': without offsets, use alpha");
            return;
        }
        this->offsets = packed_as<int32_t>(offsets, count + 1, -1, device, "offsets");
        this->scales = packed_as<float>(scales, count, -1, device, "scales");
    }
    const gemm_groups_t* get() const { return any ? this : nullptr; }
};

// Every function takes the stream and the handle first.
#define STREAM static_cast<hipStream_t>(pointer(a[0]))
#define HANDLE static_cast<gemm_handle_t>(pointer(a[1]))

// logits, ids, weights, offsets, order, position, workspace, scores, bias, groups,
// top_groups, group_top, renormalize, scale
int route(PyObject* const* a)
{
    const at::Tensor& x = tensor(a[2], "logits");
    const gemm_dtype_t dtype = logits_type(x);
    const Matrix m = matrix(x, "logits");
    const int64_t top = columns(a[3], "ids"), T = m.rows, E = m.cols;
    const Workspace ws(a[8]);
    const Device device(x);
    if ((a[5] == Py_None) != (a[6] == Py_None) || (a[6] == Py_None) != (a[7] == Py_None))
        wrong_value("offsets, order and position come together");
    const gemm_routing_t r{as_int(E), as_int(top), (gemm_scores_t)small(a[9]), small(a[11]), small(a[12]),
                           small(a[13]), packed_as<float>(a[10], E, -1, device, "bias"), truth(a[14]),
                           number(a[15])};
    return gemm_route(HANDLE, T, m.p, m.ld, dtype, &r, packed_as<int32_t>(a[3], T, top, device, "ids"),
                      packed_as<float>(a[4], T, top, device, "weights"),
                      packed_as<int32_t>(a[5], E + 1, -1, device, "offsets"),
                      packed_as<int32_t>(a[6], T * top, -1, device, "order"),
                      packed_as<int32_t>(a[7], T, top, device, "position"), ws.on(device), ws.bytes(), STREAM);
}

// logits, ids, dweights, dlogits, scores, renormalize, scale
int route_grad(PyObject* const* a)
{
    const at::Tensor &x = tensor(a[2], "logits"), &dx = tensor(a[5], "dlogits");
    const gemm_dtype_t dtype = logits_type(x);
    const Matrix m = matrix(x, "logits");
    const int64_t top = columns(a[3], "ids"), T = m.rows, E = m.cols;
    if (dx.sizes() != x.sizes()) wrong_value("dlogits must have the logits' shape");
    const Device device(x);
    const Matrix d = shaped(&dx, x.scalar_type(), T, E, device, "dlogits");
    const gemm_routing_t r{as_int(E), as_int(top), (gemm_scores_t)small(a[6]), 1, 1, 1, nullptr, truth(a[7]),
                           number(a[8])};
    return gemm_route_grad(HANDLE, T, m.p, m.ld, dtype, &r,
                           packed_as<int32_t>(a[3], T, top, device, "ids"),
                           packed_as<float>(a[4], T, top, device, "dweights"), d.p, d.ld, STREAM);
}

// X, D, order, top, weights
int gather_rows(PyObject* const* a)
{
    const at::Tensor &x = tensor(a[2], "X"), &d = tensor(a[3], "D");
    const gemm_dtype_t dtype = two_types(x.scalar_type(), d.scalar_type());
    const Matrix mx = matrix(x, "X"), md = matrix(d, "D");
    const int top = small(a[5]);
    if (mx.cols != md.cols) wrong_value("X and D must have the same columns");
    const Device device(d);
    device.holds(x, "X");
    return gemm_gather_rows(HANDLE, mx.rows, mx.cols, top, mx.p, mx.ld, md.rows,
                            packed_as<int32_t>(a[4], md.rows, -1, device, "order"),
                            packed_as<float>(a[6], mx.rows, top, device, "weights"), md.p, md.ld, dtype,
                            STREAM);
}

// Y, D, position, weights, C, beta
int combine_rows(PyObject* const* a)
{
    const at::Tensor &y = tensor(a[2], "Y"), &d = tensor(a[3], "D");
    const at::Tensor* c = maybe(a[6], "C");
    same_type(d, c, "C must have D's dtype");
    const gemm_dtype_t dtype = two_types(y.scalar_type(), d.scalar_type());
    const Matrix my = matrix(y, "Y"), md = matrix(d, "D");
    const int64_t top = columns(a[4], "position"), T = md.rows;
    if (my.cols != md.cols || (c && c->sizes() != d.sizes())) wrong_value("inconsistent shapes of Y, C and D");
    const Device device(d);
    device.holds(y, "Y");
    const Matrix mc = shaped(c, d.scalar_type(), T, md.cols, device, "C");
    return gemm_combine_rows(HANDLE, T, md.cols, as_int(top), my.p, my.ld, my.rows,
                             packed_as<int32_t>(a[4], T, top, device, "position"),
                             packed_as<float>(a[5], T, top, device, "weights"), number(a[7]), mc.p, mc.ld,
                             md.p, md.ld, dtype, STREAM);
}

// Y, dD, dY, dweights, position, weights
int combine_rows_grad(PyObject* const* a)
{
    const at::Tensor &y = tensor(a[2], "Y"), &dd = tensor(a[3], "dD"), &dy = tensor(a[4], "dY");
    same_type(y, &dy, "dY must have Y's dtype");
    const gemm_dtype_t dtype = two_types(y.scalar_type(), dd.scalar_type());
    const Matrix my = matrix(y, "Y"), md = matrix(dd, "dD");
    const int64_t top = columns(a[6], "position"), T = md.rows;
    if (my.cols != md.cols || dy.sizes() != y.sizes()) wrong_value("inconsistent shapes of Y, dY and dD");
    const Device device(y);
    device.holds(dd, "dD");
    const Matrix mdy = shaped(&dy, y.scalar_type(), my.rows, my.cols, device, "dY");
    return gemm_combine_rows_grad(HANDLE, T, md.cols, as_int(top), my.p, my.ld, my.rows,
                                  packed_as<int32_t>(a[6], T, top, device, "position"),
                                  packed_as<float>(a[7], T, top, device, "weights"), md.p, md.ld, mdy.p,
                                  mdy.ld, packed_as<float>(a[5], T, top, device, "dweights"), dtype, STREAM);
}

// A, B, D, offsets, activation, gated, bias, Z, R, transB is "N", scales, alpha
int grouped_act(PyObject* const* a)
{
    const at::Tensor &A = tensor(a[2], "A"), &B = tensor(a[3], "B"), &D = tensor(a[4], "D");
    const at::Tensor *bias = maybe(a[8], "bias"), *Z = maybe(a[9], "Z"), *R = maybe(a[10], "R");
    const at::ScalarType to = D.scalar_type();
    same_type(A, &B, "A and B must have one dtype");
    for (const at::Tensor* t : {bias, Z, R}) same_type(D, t, "D, Z, R and bias must have one dtype");
    const gemm_dtype_t dtype = two_types(A.scalar_type(), to);
    const Matrix ma = matrix(A, "A"), md = matrix(D, "D");
    const bool plain = truth(a[11]), gated = truth(a[7]), grouped = a[5] != Py_None;
    int64_t G = 1, rows, W, ldb, stride_b = 0;
    if (!grouped && B.dim() == 2) {
        const Matrix mb = matrix(B, "B");
        rows = mb.rows, W = mb.cols, ldb = mb.ld;
    } else {
        if (B.dim() != 3 || (B.size(2) > 1 && B.stride(2) != 1))
            wrong_value("B must be a 3-D tensor with unit stride in its last axis");
        G = B.size(0), rows = B.size(1), W = B.size(2);
        ldb = rows > 1 ? B.stride(1) : W > 1 ? W : 1;
        stride_b = B.stride(0);
    }
    if (!plain) std::swap(rows, W);
    if (rows != ma.cols || md.rows != ma.rows || W != (gated ? 2 : 1) * md.cols || (!grouped && G != 1))
        wrong_value("inconsistent grouped GEMM shapes");
    const Device device(D);
    device.holds(A, "A");
    device.holds(B, "B");
    gemm_act_t act{(gemm_activation_t)small(a[6]), gated, nullptr, 0, nullptr, 0, nullptr, 0};
    if (bias) {
        const bool each = bias->dim() == 2;
        if ((each ? bias->size(0) != G || bias->size(1) != W : bias->dim() != 1 || bias->size(0) != W) ||
            (W > 1 && bias->stride(-1) != 1))
            wrong_value("bias must be groups x width, or width, with unit stride");
        device.holds(*bias, "bias");
        act.bias = bias->data_ptr();
        act.stride_bias = each && G > 1 ? bias->stride(0) : 0;
    }
    const Matrix mz = shaped(Z, to, ma.rows, W, device, "Z"), mr = shaped(R, to, ma.rows, md.cols, device, "R");
    act.Z = mz.p, act.ldz = mz.ld, act.R = mr.p, act.ldr = mr.ld;
    const Groups groups(a[5], a[12], G, device);
    return gemm_run_grouped_act(HANDLE, plain ? GEMM_OP_N : GEMM_OP_T, ma.rows, md.cols, ma.cols,
                                number(a[13]), ma.p, ma.ld, B.data_ptr(), ldb, stride_b, md.p, md.ld, dtype,
                                groups.get(), &act, STREAM);
}

// Z, dD, dZ, offsets, activation, gated, H, dbias, workspace
int grouped_act_grad(PyObject* const* a)
{
    const at::Tensor &Z = tensor(a[2], "Z"), &dD = tensor(a[3], "dD"), &dZ = tensor(a[4], "dZ");
    const at::Tensor* H = maybe(a[8], "H");
    const at::ScalarType ti = dZ.scalar_type();
    same_type(Z, &dD, "Z and dD must have one dtype");
    same_type(dZ, H, "dZ and H must have one dtype");
    const gemm_dtype_t dtype = two_types(ti, Z.scalar_type());
    const Matrix mz = matrix(Z, "Z"), md = matrix(dD, "dD");
    const bool gated = truth(a[7]);
    const Workspace ws(a[10]);
    if (md.rows != mz.rows || mz.cols != (gated ? 2 : 1) * md.cols) wrong_value("inconsistent shapes of Z and dD");
    const Device device(Z);
    device.holds(dD, "dD");
    const Matrix mdz = shaped(&dZ, ti, mz.rows, mz.cols, device, "dZ");
    const Matrix mh = shaped(H, ti, mz.rows, md.cols, device, "H");
    int64_t G = 1;
    if (a[5] != Py_None) {
        const at::Tensor& offsets = tensor(a[5], "offsets");
        if (offsets.dim() != 1 || offsets.size(0) < 1) wrong_value("offsets must hold groups + 1 entries");
        G = offsets.size(0) - 1;
    }
    const Groups groups(a[5], Py_None, G, device);
    return gemm_run_grouped_act_grad(HANDLE, mz.rows, md.cols, (gemm_activation_t)small(a[6]), gated, mz.p,
                                     mz.ld, md.p, md.ld, mdz.p, mdz.ld, mh.p, mh.ld,
                                     packed_as<float>(a[9], G, mz.cols, device, "dbias"), dtype, groups.get(),
                                     ws.on(device), ws.bytes(), STREAM);
}

template <int (*F)(PyObject* const*), int ARGS>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n)
{
    if (n != ARGS) {
        PyErr_Format(PyExc_TypeError, "expected %d arguments, got %zd", ARGS, n);
        return nullptr;
    }
    try {
        return PyLong_FromLong(F(args));
    } catch (const Failure& f) {
        PyErr_SetString(f.type, f.what());
    } catch (const Raised&) {
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

template <int (*F)(PyObject* const*), int ARGS>
PyMethodDef method(const char* name)
{
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<F, ARGS>)), METH_FASTCALL,
            nullptr};
}

PyMethodDef methods[] = {method<route, 16>("route"),
                         method<route_grad, 9>("route_grad"),
                         method<gather_rows, 7>("gather_rows"),
                         method<combine_rows, 8>("combine_rows"),
                         method<combine_rows_grad, 8>("combine_rows_grad"),
                         method<grouped_act, 14>("grouped_act"),
                         method<grouped_act_grad, 11>("grouped_act_grad"),
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_bind", "Marshalling of torch tensors.", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__bind() { return PyModule_Create(&module); }
