// Python binding of the expert training operators: tensors in, tensors out.  It only checks and marshals
// arguments and allocates results (PyTorch's allocator, on the current stream); the work is the library's, whose
// entry points are handed over by address.  Native because a call's host time is what a decode-size step waits
// for: a dropout takes 2.3 us through here (3.8 with a new output), 8.4 us through Python and ctypes, 2 to 3 us of
// either the library's.
#include <Python.h>

#include <ATen/core/grad_mode.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include <string>

#include "k3moe.h"

namespace {

struct Refusal {
    int code;
    std::string what;
};

[[noreturn]] void refuse(const std::string &what, int code = K3MOE_ERR_ARG) { throw Refusal{code, what}; }
struct PythonError {};                       // a Python exception is already set

void need(bool ok, const char *what)
{
    if (!ok) refuse(what);
}

// ---------------------------------------------------------------------------- state handed over by setup()
PyObject *g_error = nullptr;                 // the exception class, called with (code, what)
PyObject *g_new_status = nullptr;            // callable: device index -> address of its status word
int32_t *g_status[64] = {};

enum Entry { PLAN_BYTES, PLAN, GATHER, COMBINE, COMBINE_GRAD, MM, MM_GRAD_X, MM_GRAD_W, GLU, GLU_GRAD, DROPOUT, ENTRIES };
const char *const ENTRY_NAMES[ENTRIES] = {
    "k3moe_rows_plan_workspace_bytes", "k3moe_rows_plan", "k3moe_rows_gather", "k3moe_rows_combine",
    "k3moe_rows_combine_grad", "k3moe_group_mm", "k3moe_group_mm_grad_x", "k3moe_group_mm_grad_w",
    "k3moe_glu_dropout", "k3moe_glu_dropout_grad", "k3moe_dropout"};
void *g_entry[ENTRIES] = {};

template <Entry E, class F>
F *entry(F *)
{
    return reinterpret_cast<F *>(g_entry[E]);
}

void check(int rc, const char *what)
{
    if (rc != K3MOE_OK) refuse(what, rc);
}

// ---------------------------------------------------------------------------- arguments
// A tensor.  The calls record nothing for autograd, so one that needs gradients is refused where they would be
// recorded, rather than left out of them.
const at::Tensor &tensor(PyObject *o, const char *what)
{
    if (!THPVariable_Check(o)) refuse(std::string(what) + ": a tensor");
    const at::Tensor &t = THPVariable_Unpack(o);
    if (t.requires_grad() && at::GradMode::is_enabled())
        refuse(std::string(what) + ": requires gradients, which these calls do not record (detach it, or call under torch.no_grad)",
               K3MOE_ERR_UNSUPPORTED);
    return t;
}

const at::Tensor *maybe(PyObject *o, const char *what) { return o == Py_None ? nullptr : &tensor(o, what); }

int type_code(at::ScalarType t, const char *what)
{
    if (t == at::kFloat) return K3MOE_TYPE_F32;
    if (t == at::kBFloat16) return K3MOE_TYPE_BF16;
    if (t == at::kHalf) return K3MOE_TYPE_F16;
    refuse(std::string(what) + ": fp32, bf16 or f16", K3MOE_ERR_UNSUPPORTED);
}

int as_int(PyObject *o, const char *what)
{
    const long v = PyLong_AsLong(o);
    if (v == -1 && PyErr_Occurred()) {
        PyErr_Clear();
        refuse(std::string(what) + ": an integer");
    }
    if (v != (int)v) refuse(std::string(what) + ": a 32-bit integer");
    return (int)v;
}

uint64_t as_u64(PyObject *o, const char *what)
{
    const unsigned long long v = PyLong_AsUnsignedLongLong(o);
    if (PyErr_Occurred()) {
        PyErr_Clear();
        refuse(std::string(what) + ": a 64-bit unsigned integer");
    }
    return v;
}

double as_double(PyObject *o, const char *what)
{
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) {
        PyErr_Clear();
        refuse(std::string(what) + ": a number");
    }
    return v;
}

// The call's device (that of its first tensor), current while it lasts, and its current stream.
struct Place {
    int dev;
    c10::cuda::OptionalCUDAGuard guard;
    cudaStream_t stream;
    explicit Place(const at::Tensor &t)
    {
        need(t.is_cuda(), "CUDA tensors are needed");
        dev = t.get_device();
        if (dev != c10::cuda::current_device()) guard.set_index((c10::DeviceIndex)dev);
        stream = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream();
    }
    bool has(const at::Tensor &t) const { return t.is_cuda() && t.get_device() == dev; }
    int32_t *status() const
    {
        if (dev >= 64) refuse("device index", K3MOE_ERR_UNSUPPORTED);
        if (!g_status[dev]) {
            PyObject *p = PyObject_CallFunction(g_new_status, "i", dev);
            if (!p) throw PythonError();
            g_status[dev] = static_cast<int32_t *>(PyLong_AsVoidPtr(p));
            Py_DECREF(p);
            if (PyErr_Occurred()) throw PythonError();
        }
        return g_status[dev];
    }
};

// A matrix with contiguous rows.
struct Rows {
    int64_t n, width, ld;
    void *p;
    Rows(const at::Tensor &t, const Place &at, const char *what, int64_t want_width = -1, int64_t want_rows = -1)
    {
        if (t.dim() != 2 || !at.has(t)) refuse(std::string(what) + ": a matrix on the call's device");
        n = t.size(0);
        width = t.size(1);
        ld = n > 1 ? t.stride(0) : width;
        if ((width > 1 && t.stride(1) != 1) || ld < width) refuse(std::string(what) + ": contiguous rows that do not overlap");
        if ((want_width >= 0 && width != want_width) || (want_rows >= 0 && n != want_rows))
            refuse(std::string(what) + ": another shape is expected");
        if (n > INT32_MAX || width > INT32_MAX) refuse(std::string(what) + ": too many rows or columns");
        p = t.data_ptr();
    }
};

// [E, n_out, n_in] with contiguous rows.
struct Matrices {
    int64_t E, rows, cols, ld, stride;
    void *p;
    Matrices(const at::Tensor &t, const Place &at, const char *what)
    {
        if (t.dim() != 3 || !at.has(t)) refuse(std::string(what) + ": [E, n_out, n_in] on the call's device");
        E = t.size(0);
        rows = t.size(1);
        cols = t.size(2);
        if (cols > 1 && t.stride(2) != 1) refuse(std::string(what) + ": contiguous rows");
        ld = rows > 1 ? t.stride(1) : cols;
        stride = E > 1 ? t.stride(0) : 0;
        if (E > INT32_MAX || rows > INT32_MAX || cols > INT32_MAX) refuse(std::string(what) + ": too large");
        p = t.data_ptr();
    }
};

// A contiguous table of the given type.
void *table(const at::Tensor &t, const Place &at, const char *what, at::ScalarType type, at::IntArrayRef shape)
{
    if (!at.has(t) || t.scalar_type() != type || !t.is_contiguous() || t.sizes() != shape)
        refuse(std::string(what) + ": a contiguous table of the right type, shape and device");
    return t.data_ptr();
}

// pos or idx: [T, K] int32.
struct Pairs {
    int64_t T, K;
    int32_t *p;
    Pairs(const at::Tensor &t, const Place &at, const char *what, int64_t want_T = -1)
    {
        if (t.dim() != 2 || !at.has(t) || t.scalar_type() != at::kInt || !t.is_contiguous())
            refuse(std::string(what) + ": [T, K], contiguous int32 on the call's device");
        T = t.size(0);
        K = t.size(1);
        if ((want_T >= 0 && T != want_T) || T > INT32_MAX || K > INT32_MAX) refuse(std::string(what) + ": [T, K]");
        p = static_cast<int32_t *>(t.data_ptr());
    }
};

at::Tensor fresh(at::IntArrayRef shape, const at::Tensor &like, at::ScalarType type)
{
    return at::empty(shape, like.options().dtype(type).requires_grad(false));
}

// The given output, or a new [n, width] matrix.
at::Tensor output(PyObject *o, int64_t n, int64_t width, const at::Tensor &like, at::ScalarType type)
{
    const at::Tensor *given = maybe(o, "out");
    if (!given) return fresh({n, width}, like, type);
    if (given->scalar_type() != type) refuse("out: another type is expected");
    return *given;
}

struct Random {
    double p;
    uint64_t seed, offset;
    Random(PyObject *p_, PyObject *s, PyObject *o) : p(as_double(p_, "p")), seed(as_u64(s, "seed")), offset(as_u64(o, "offset"))
    {
        need(p >= 0.0 && p < 1.0, "p: 0 <= p < 1");
    }
};

int act_code(PyObject *o)
{
    if (PyUnicode_Check(o)) {
        if (PyUnicode_CompareWithASCIIString(o, "silu") == 0) return K3MOE_ACT_SILU;
        if (PyUnicode_CompareWithASCIIString(o, "situ") == 0) return K3MOE_ACT_SITU;
    }
    refuse("act: silu or situ");
}

PyObject *wrap(at::Tensor t) { return THPVariable_Wrap(std::move(t)); }

// The output of a call, `given` by the caller or new.  A given one was written in place: autograd is told, as any
// graph that has saved it must notice.
PyObject *written(at::Tensor t, PyObject *given)
{
    if (given != Py_None && !t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
    return wrap(std::move(t));
}

PyObject *pair(PyObject *x, at::Tensor b)
{
    PyObject *y = x ? wrap(std::move(b)) : nullptr;
    PyObject *t = y ? PyTuple_Pack(2, x, y) : nullptr;
    Py_XDECREF(x);
    Py_XDECREF(y);
    return t;
}

// ---------------------------------------------------------------------------- calls (all arguments positional)
typedef PyObject *const *Args;

PyObject *plan_rows(Args a)                  // idx, n_experts, first_expert
{
    const at::Tensor &idx = tensor(a[0], "idx");
    const Place at(idx);
    const Pairs x(idx, at, "idx");
    const int E = as_int(a[1], "n_experts"), first = as_int(a[2], "first_expert");
    const size_t nb = entry<PLAN_BYTES>(&k3moe_rows_plan_workspace_bytes)((int)x.T, (int)x.K, E);
    const at::Tensor ws = fresh({(int64_t)(nb / 4 + 1)}, idx, at::kInt);
    // sizes that the library refuses get no tables (nb is 0 for them)
    at::Tensor offsets = fresh({nb ? E + 1 : 1}, idx, at::kInt), pos = fresh({x.T, x.K}, idx, at::kInt);
    check(entry<PLAN>(&k3moe_rows_plan)(x.p, (int)x.T, (int)x.K, first, E, static_cast<int32_t *>(offsets.data_ptr()),
                                        static_cast<int32_t *>(pos.data_ptr()), ws.data_ptr(), nb, at.stream),
          "plan_rows");
    return pair(wrap(std::move(offsets)), std::move(pos));
}

PyObject *gather_rows(Args a)                // x, pos, n_rows, out
{
    const at::Tensor &xt = tensor(a[0], "x");
    const Place at(xt);
    const Rows x(xt, at, "x");
    const Pairs pos(tensor(a[1], "pos"), at, "pos", x.n);
    const int64_t n = a[2] == Py_None ? -1 : as_int(a[2], "n_rows");
    need(n >= 0 || a[2] == Py_None, "n_rows: not negative");
    at::Tensor out = output(a[3], n < 0 ? pos.T * pos.K : n, x.width, xt, xt.scalar_type());
    const Rows o(out, at, "out", x.width);
    need(n <= o.n, "out: at least n_rows rows");
    check(entry<GATHER>(&k3moe_rows_gather)(x.p, x.ld, pos.p, (int)pos.T, (int)pos.K, (int)x.width,
                                            type_code(xt.scalar_type(), "x"), o.p, o.ld, (int)(n < 0 ? o.n : n), at.status(),
                                            at.stream),
          "gather_rows");
    return written(std::move(out), a[3]);
}

PyObject *combine_rows(Args a)               // y, pos, weights, out
{
    const at::Tensor &yt = tensor(a[0], "y");
    const Place at(yt);
    const Rows y(yt, at, "y");
    const Pairs pos(tensor(a[1], "pos"), at, "pos");
    const at::Tensor *w = maybe(a[2], "weights");
    const float *wp = w ? static_cast<float *>(table(*w, at, "weights", at::kFloat, {pos.T, pos.K})) : nullptr;
    at::Tensor out = output(a[3], pos.T, y.width, yt, yt.scalar_type());
    const Rows z(out, at, "out", y.width, pos.T);
    check(entry<COMBINE>(&k3moe_rows_combine)(y.p, y.ld, (int)y.n, pos.p, wp, (int)pos.T, (int)pos.K, (int)y.width,
                                              type_code(yt.scalar_type(), "y"), z.p, z.ld, at.status(), at.stream),
          "combine_rows");
    return written(std::move(out), a[3]);
}

PyObject *combine_rows_grad(Args a)          // dz, y, pos, weights, out
{
    const at::Tensor &zt = tensor(a[0], "dz"), &yt = tensor(a[1], "y"), &wt = tensor(a[3], "weights");
    const Place at(zt);
    const Rows dz(zt, at, "dz"), y(yt, at, "y", dz.width);
    const Pairs pos(tensor(a[2], "pos"), at, "pos", dz.n);
    const float *w = static_cast<float *>(table(wt, at, "weights", at::kFloat, {pos.T, pos.K}));
    need(zt.scalar_type() == yt.scalar_type(), "dz: y's type");
    at::Tensor out = output(a[4], y.n, y.width, yt, yt.scalar_type());
    const Rows dy(out, at, "out", y.width, y.n);
    at::Tensor dw = fresh({pos.T, pos.K}, wt, at::kFloat);
    check(entry<COMBINE_GRAD>(&k3moe_rows_combine_grad)(dz.p, dz.ld, y.p, y.ld, (int)y.n, pos.p, w, (int)pos.T, (int)pos.K,
                                                        (int)y.width, type_code(yt.scalar_type(), "y"), dy.p, dy.ld,
                                                        static_cast<float *>(dw.data_ptr()), at.status(), at.stream),
          "combine_rows_grad");
    return pair(written(std::move(out), a[4]), std::move(dw));
}

at::ScalarType scalar_type(PyObject *o, at::ScalarType otherwise)
{
    if (o == Py_None) return otherwise;
    if (!THPDtype_Check(o)) refuse("out_dtype: a torch.dtype");
    return reinterpret_cast<THPDtype *>(o)->scalar_type;
}

template <Entry E>
PyObject *product(Args a, bool mm)           // rows, w, offsets, out, out_dtype
{
    const char *what = mm ? "x" : "dy";
    const at::Tensor &t = tensor(a[0], what), &wt = tensor(a[1], "w");
    const Place at(t);
    const Matrices w(wt, at, "w");
    const Rows x(t, at, what, mm ? w.cols : w.rows);
    need(t.scalar_type() == wt.scalar_type(), "the rows and w: one type");
    const int32_t *off = static_cast<int32_t *>(table(tensor(a[2], "offsets"), at, "offsets", at::kInt, {w.E + 1}));
    const at::Tensor *given = maybe(a[3], "out");
    const at::ScalarType type = scalar_type(a[4], given ? given->scalar_type() : t.scalar_type());
    const int64_t width = mm ? w.rows : w.cols;
    at::Tensor out = output(a[3], x.n, width, t, type);
    const Rows o(out, at, "out", width, x.n);
    check(entry<E>(&k3moe_group_mm)(off, (int)w.E, (int)x.n, (int)w.cols, (int)w.rows, x.p, x.ld, w.p, w.ld, w.stride,
                                    type_code(t.scalar_type(), what), o.p, o.ld, type_code(type, "out"), at.status(),
                                    at.stream),
          mm ? "group_mm" : "group_mm_grad_x");
    return written(std::move(out), a[3]);
}

PyObject *group_mm(Args a) { return product<MM>(a, true); }
PyObject *group_mm_grad_x(Args a) { return product<MM_GRAD_X>(a, false); }

PyObject *group_mm_grad_w(Args a)            // dy, x, offsets, out, out_dtype, accumulate
{
    const at::Tensor &dt = tensor(a[0], "dy"), &xt = tensor(a[1], "x"), &ot = tensor(a[2], "offsets");
    const Place at(dt);
    const Rows dy(dt, at, "dy"), x(xt, at, "x", -1, dy.n);
    need(dt.scalar_type() == xt.scalar_type(), "dy, x: one type");
    need(ot.dim() == 1 && ot.size(0) > 1, "offsets: [E + 1]");
    const int32_t *off = static_cast<int32_t *>(table(ot, at, "offsets", at::kInt, {ot.size(0)}));
    const int64_t E = ot.size(0) - 1;
    const at::Tensor *given = maybe(a[3], "out");
    const int accumulate = PyObject_IsTrue(a[5]);
    if (accumulate < 0) throw PythonError();
    need(given || !accumulate, "accumulate needs out");
    const at::ScalarType type = scalar_type(a[4], given ? given->scalar_type() : at::kFloat);
    need(!given || given->scalar_type() == type, "out: the type asked for");
    at::Tensor out = given ? *given : fresh({E, dy.width, x.width}, xt, type);
    const Matrices o(out, at, "out");
    need(o.E == E && o.rows == dy.width && o.cols == x.width, "out: [E, n_out, n_in]");
    check(entry<MM_GRAD_W>(&k3moe_group_mm_grad_w)(off, (int)E, (int)x.n, (int)x.width, (int)dy.width, dy.p, dy.ld, x.p,
                                                   x.ld, type_code(xt.scalar_type(), "x"), o.p, o.ld, o.stride,
                                                   type_code(type, "out"), accumulate, at.status(), at.stream),
          "group_mm_grad_w");
    return written(std::move(out), a[3]);
}

PyObject *glu_dropout(Args a)                // gu, p, seed, offset, act, situ_beta, situ_linear_beta, out
{
    const at::Tensor &gt = tensor(a[0], "gu");
    const Place at(gt);
    const Rows gu(gt, at, "gu");
    need(gu.width > 0 && gu.width % 2 == 0, "gu: [rows, 2 width]");
    const Random r(a[1], a[2], a[3]);
    const int act = act_code(a[4]);
    const float beta = (float)as_double(a[5], "situ_beta"), linear = (float)as_double(a[6], "situ_linear_beta");
    at::Tensor out = output(a[7], gu.n, gu.width / 2, gt, gt.scalar_type());
    const Rows o(out, at, "out", gu.width / 2, gu.n);
    check(entry<GLU>(&k3moe_glu_dropout)(gu.p, gu.ld, (int)gu.n, (int)(gu.width / 2), type_code(gt.scalar_type(), "gu"), act,
                                         beta, linear, r.p, r.seed, r.offset, o.p, o.ld, at.stream),
          "glu_dropout");
    return written(std::move(out), a[7]);
}

PyObject *glu_dropout_grad(Args a)           // da, gu, p, seed, offset, act, situ_beta, situ_linear_beta, out
{
    const at::Tensor &dt = tensor(a[0], "da"), &gt = tensor(a[1], "gu");
    const Place at(dt);
    const Rows gu(gt, at, "gu");
    need(gu.width > 0 && gu.width % 2 == 0, "gu: [rows, 2 width]");
    const Rows da(dt, at, "da", gu.width / 2, gu.n);
    need(dt.scalar_type() == gt.scalar_type(), "da: gu's type");
    const Random r(a[2], a[3], a[4]);
    const int act = act_code(a[5]);
    const float beta = (float)as_double(a[6], "situ_beta"), linear = (float)as_double(a[7], "situ_linear_beta");
    at::Tensor out = output(a[8], gu.n, gu.width, gt, gt.scalar_type());
    const Rows o(out, at, "out", gu.width, gu.n);
    check(entry<GLU_GRAD>(&k3moe_glu_dropout_grad)(da.p, da.ld, gu.p, gu.ld, (int)gu.n, (int)(gu.width / 2),
                                                   type_code(gt.scalar_type(), "gu"), act, beta, linear, r.p, r.seed,
                                                   r.offset, o.p, o.ld, at.stream),
          "glu_dropout_grad");
    return written(std::move(out), a[8]);
}

PyObject *dropout(Args a)                    // x, p, seed, offset, residual, out
{
    const at::Tensor &xt = tensor(a[0], "x");
    const Place at(xt);
    const Random r(a[1], a[2], a[3]);
    need(xt.is_contiguous(), "x: a contiguous tensor");
    const at::Tensor *res = maybe(a[4], "residual"), *given = maybe(a[5], "out");
    const void *rp = res ? table(*res, at, "residual", xt.scalar_type(), xt.sizes()) : nullptr;
    at::Tensor out = given ? *given : fresh(xt.sizes(), xt, xt.scalar_type());
    void *op = table(out, at, "out", xt.scalar_type(), xt.sizes());
    check(entry<DROPOUT>(&k3moe_dropout)(xt.data_ptr(), rp, xt.numel(), type_code(xt.scalar_type(), "x"), r.p, r.seed,
                                         r.offset, op, at.stream),
          "dropout");
    return written(std::move(out), a[5]);
}

// No C++ exception leaves a call: refusals become the error class, others a RuntimeError.
template <PyObject *(*F)(Args), int N>
PyObject *call(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    try {
        if (n != N) refuse("wrong number of arguments");
        if (!g_error) refuse("the binding is not set up", K3MOE_ERR_STATE);
        return F(args);
    } catch (const Refusal &r) {
        PyObject *e = g_error ? PyObject_CallFunction(g_error, "is", r.code, r.what.c_str()) : nullptr;
        if (e) {
            PyErr_SetObject(g_error, e);
            Py_DECREF(e);
        } else if (!PyErr_Occurred()) {
            PyErr_SetString(PyExc_RuntimeError, r.what.c_str());
        }
    } catch (const PythonError &) {
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    } catch (...) {
        PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
    }
    return nullptr;
}

// setup(error_class, new_status, {entry name: address})
PyObject *setup(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    if (n != 3 || !PyDict_Check(args[2])) {
        PyErr_SetString(PyExc_TypeError, "setup(error_class, new_status, addresses)");
        return nullptr;
    }
    for (int i = 0; i < ENTRIES; ++i) {
        PyObject *p = PyDict_GetItemString(args[2], ENTRY_NAMES[i]);
        g_entry[i] = p ? PyLong_AsVoidPtr(p) : nullptr;
        if (!g_entry[i]) {
            if (!PyErr_Occurred()) PyErr_Format(PyExc_RuntimeError, "no address of %s", ENTRY_NAMES[i]);
            return nullptr;
        }
    }
    Py_INCREF(args[1]);
    Py_XSETREF(g_new_status, args[1]);
    Py_INCREF(args[0]);
    Py_XSETREF(g_error, args[0]);
    Py_RETURN_NONE;
}

#define CALL(name, n) {#name, (PyCFunction)(void (*)(void))call<name, n>, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {{"setup", (PyCFunction)(void (*)(void))setup, METH_FASTCALL, nullptr},
                         CALL(plan_rows, 3),
                         CALL(gather_rows, 4),
                         CALL(combine_rows, 4),
                         CALL(combine_rows_grad, 5),
                         CALL(group_mm, 5),
                         CALL(group_mm_grad_x, 5),
                         CALL(group_mm_grad_w, 6),
                         CALL(glu_dropout, 8),
                         CALL(glu_dropout_grad, 9),
                         CALL(dropout, 6),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_experts", "Binding of the expert training operators.", -1, methods};

}  // namespace

extern "C" __attribute__((visibility("default"))) PyObject *PyInit__experts() { return PyModule_Create(&module); }
