// The tensor functions of a transformer block's operators (block.py): checks of
// the operands, their strides, outputs and workspace from torch's allocator, and
// one call of a C entry on the current stream of the operands' device.
//
// In C++ because a call of a few microseconds on the device should not wait for
// ten of them on the host: layer_norm of 300 x 256 with a residual takes the
// host 5 us this way and took 16 by ctypes.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <ATen/ops/empty_like.h>
#include <c10/core/impl/LocalDispatchKeySet.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>
#include <stdexcept>
#include <string>

#include "gbnms.h"

namespace {

// The C entries, set once by bind().
decltype(&nms_linear_workspace_size) linear_workspace_size;
decltype(&nms_linear_run) linear_run;
decltype(&nms_linear_grad_workspace_size) linear_grad_workspace_size;
decltype(&nms_linear_grad_run) linear_grad_run;
decltype(&nms_layer_norm_run) layer_norm_run;
decltype(&nms_layer_norm_workspace_size) layer_norm_workspace_size;
decltype(&nms_layer_norm_grad_run) layer_norm_grad_run;
decltype(&nms_rotary_run) rotary_run;

// Operands that a function refuses: a ValueError.
struct Refused : std::runtime_error {
    using std::runtime_error::runtime_error;
};

[[noreturn]] void refuse(const char* where, const std::string& what) { throw Refused(std::string(where) + ": " + what); }

// A tensor whose memory holds its values (a view can have their negation pending).
const at::Tensor& unpack(PyObject* o, const char* where, const char* name)
{
    const at::Tensor& t = THPVariable_Unpack(o);
    if (t.is_neg()) refuse(where, std::string(name) + " is a negated view: resolve_neg() it");
    return t;
}

// A tensor argument, or an undefined tensor for None.
const at::Tensor& argument(PyObject* o, const char* where, const char* name)
{
    static const at::Tensor none;
    if (o == Py_None) return none;
    if (!THPVariable_Check(o)) refuse(where, std::string(name) + " must be a tensor");
    return unpack(o, where, name);
}

const at::Tensor& operand(PyObject* o, const char* where, const char* name)
{
    if (!THPVariable_Check(o)) refuse(where, std::string(name) + " must be a tensor");
    return unpack(o, where, name);
}

int type_code(at::ScalarType t)
{
    return t == at::kFloat ? NMS_TYPE_F32 : t == at::kHalf ? NMS_TYPE_F16 : t == at::kBFloat16 ? NMS_TYPE_BF16 : -1;
}

int type_of(const at::Tensor& x, const char* where, const char* name)
{
    const int code = type_code(x.scalar_type());
    if (code < 0) refuse(where, std::string(name) + " must be a float32, float16 or bfloat16 CUDA tensor");
    return code;
}

// The last of the checks, so that the others do not need a device.
void on_device(const at::Tensor& x, const char* where, const char* name)
{
    if (!x.is_cuda()) refuse(where, std::string(name) + " must be a float32, float16 or bfloat16 CUDA tensor");
}

void same(const at::Tensor& x, const at::Tensor& like, const char* where, const char* name)
{
    if (x.sizes() != like.sizes() || x.scalar_type() != like.scalar_type() || x.device() != like.device())
        refuse(where, std::string(name) + " must have the shape, type and device of the other operand");
}

// Rows [..., width] at one stride; copied only where they do not lie so.
struct Rows {
    at::Tensor t;
    int64_t row, rows, width;
    const void* at() const { return t.data_ptr(); }
};

Rows rows_of(const at::Tensor& x, const char* where)
{
    const int64_t dims = x.dim();
    if (dims == 0) refuse(where, "rows must be [..., width]");
    const int64_t width = x.size(dims - 1);
    int64_t rows = 1;
    for (int64_t d = 0; d < dims - 1; ++d) rows *= x.size(d);
    if (x.is_contiguous()) return {x, width, rows, width};
    bool fits = width <= 1 || x.stride(dims - 1) == 1, set = false;
    int64_t step = width, span = 0;
    for (int64_t d = dims - 2; d >= 0; --d) {
        if (x.size(d) == 1) continue;
        if (!set) step = x.stride(d);
        else if (x.stride(d) != span) fits = false;
        set = true;
        span = x.stride(d) * x.size(d);
    }
    if (fits) return {x, step, rows, width};
    return {x.contiguous(), width, rows, width};
}

at::Tensor like(const at::Tensor& x) { return at::empty_like(x, {}, at::MemoryFormat::Contiguous); }

at::Tensor scratch(size_t bytes, const at::Tensor& x)
{
    return at::empty({static_cast<int64_t>(bytes)}, x.options().dtype(at::kByte));
}

void* address(const at::Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; }

bool even(const Rows& r, const at::Tensor& x)
{
    return reinterpret_cast<uintptr_t>(r.at()) % 16 == 0 && r.row * x.element_size() % 16 == 0 && r.row >= r.width;
}

// The weight [outer, inner] as rows.
Rows weight_rows(const at::Tensor& x, const at::Tensor& weight, int64_t inner, const char* where)
{
    if (weight.dim() != 2 || weight.size(1) != inner || weight.scalar_type() != x.scalar_type() ||
        weight.device() != x.device())
        refuse(where, "weight must be [outer, inner] of x's type beside x");
    const int64_t outer = weight.size(0);
    if (inner > 1 && weight.stride(1) != 1) return {weight.contiguous(), inner, outer, inner};
    return {weight, outer > 1 ? weight.stride(0) : inner, outer, inner};
}

// Type of parameters [width] beside x: binary32 or x's, all alike.
int params(const at::Tensor& x, int64_t width, std::initializer_list<std::pair<const char*, const at::Tensor*>> of,
           const char* where, const char* shape)
{
    int kind = -1;
    for (const auto& [name, p] : of) {
        if (!p->defined()) continue;
        const auto t = p->scalar_type();
        if (p->dim() != 1 || p->size(0) != width || p->device() != x.device() || !p->is_contiguous() ||
            (t != at::kFloat && t != x.scalar_type()) || (kind >= 0 && kind != type_code(t)))
            refuse(where, std::string(name) + " must be a contiguous " + shape +
                              " tensor beside x, float32 or of x's type, all of them alike");
        kind = type_code(t);
    }
    return kind < 0 ? NMS_TYPE_F32 : kind;
}

// A C entry on the current stream of x's device, that device current.
template <typename Entry, typename... Args>
int launch(const at::Tensor& x, Entry entry, Args... args)
{
    const c10::cuda::OptionalCUDAGuard guard(x.device());
    void* stream = c10::cuda::getCurrentCUDAStream(x.get_device()).stream();
    PyThreadState* state = PyEval_SaveThread();
    const int code = entry(args..., stream);
    PyEval_RestoreThread(state);
    return code;
}

PyObject* result(int code, std::initializer_list<at::Tensor> outs)
{
    if (code != NMS_OK) return PyLong_FromLong(code);
    PyObject* tuple = PyTuple_New(static_cast<Py_ssize_t>(outs.size()));
    if (!tuple) return nullptr;
    Py_ssize_t i = 0;
    for (const at::Tensor& t : outs) {
        PyObject* o = t.defined() ? THPVariable_Wrap(t) : Py_NewRef(Py_None);
        if (!o) {
            Py_DECREF(tuple);
            return nullptr;
        }
        PyTuple_SET_ITEM(tuple, i++, o);
    }
    return tuple;
}

// A function's body: no C++ exception leaves it.
template <typename Body>
PyObject* guarded(Py_ssize_t given, Py_ssize_t wanted, Body body)
{
    HANDLE_TH_ERRORS
    if (given != wanted) {
        PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
        return nullptr;
    }
    try {
        const c10::impl::ExcludeDispatchKeyGuard plain(c10::autograd_dispatch_keyset);
        return body();
    } catch (const Refused& e) {
        PyErr_SetString(PyExc_ValueError, e.what());
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

// The C entries' dev_status: a tensor argument's word, or NULL for None.
int32_t* status_word(const at::Tensor& status, const at::Tensor& x, const char* where)
{
    if (!status.defined()) return nullptr;
    if (status.scalar_type() != at::kInt || status.numel() != 1 || status.device() != x.device())
        refuse(where, "status must be one int32 beside x");
    return static_cast<int32_t*>(status.data_ptr());
}

// Whether the C entries' 32-bit sizes hold these.
bool fits(std::initializer_list<int64_t> sizes)
{
    for (const int64_t v : sizes)
        if (v > INT32_MAX) return false;
    return true;
}

// linear_act(x, weight, bias, act, residual, return_pre, status) -> (y,) or (y, pre)
PyObject* linear_act(PyObject*, PyObject* const* args, Py_ssize_t n)
{
    return guarded(n, 7, [&]() -> PyObject* {
        const char* where = "linear_act";
        const at::Tensor &x = operand(args[0], where, "x"), &weight = operand(args[1], where, "weight"),
                         &bias = argument(args[2], where, "bias"), &residual = argument(args[4], where, "residual"),
                         &status = argument(args[6], where, "status");
        const int act = static_cast<int>(PyLong_AsLong(args[3]));
        const int type = type_of(x, where, "x");
        const Rows xs = rows_of(x, where), ws = weight_rows(x, weight, xs.width, where);
        if (!fits({xs.width, ws.rows})) return result(NMS_ERR_CAPACITY, {});
        const int bias_type = params(x, ws.rows, {{"bias", &bias}}, where, "[outer]");
        c10::DimVector shape(x.sizes().begin(), x.sizes().end());
        shape.back() = ws.rows;
        Rows res{{}, 0, 0, 0};
        if (residual.defined()) {
            if (residual.sizes() != at::IntArrayRef(shape) || residual.scalar_type() != x.scalar_type() ||
                residual.device() != x.device())
                refuse(where, "residual must be [..., outer] of x's type beside x");
            res = rows_of(residual, where);
        }
        int32_t* const word = status_word(status, x, where);
        on_device(x, where, "x");
        const at::Tensor y = at::empty(shape, x.options());
        const at::Tensor pre = args[5] == Py_True ? at::empty(shape, x.options()) : at::Tensor();
        size_t bytes = 0;
        int code = linear_workspace_size(type, xs.rows, xs.width, ws.rows, even(xs, x) && even(ws, x), &bytes);
        if (code != NMS_OK) return result(code, {});
        const at::Tensor work = bytes ? scratch(bytes, x) : at::Tensor();
        code = launch(x, linear_run, xs.at(), xs.row, type, xs.rows, xs.width, ws.at(), ws.row, ws.rows, address(bias),
                      bias_type, act, address(res.t), res.row, address(y), address(pre), word, address(work), bytes);
        return pre.defined() ? result(code, {y, pre}) : result(code, {y});
    });
}

// linear_act_grad(dy, x, weight, pre, act, status, need_dx, need_dweight, need_dbias) -> (dx, dweight, dbias)
PyObject* linear_act_grad(PyObject*, PyObject* const* args, Py_ssize_t n)
{
    return guarded(n, 9, [&]() -> PyObject* {
        const char* where = "linear_act_grad";
        const at::Tensor &dy = operand(args[0], where, "dy"), &x = operand(args[1], where, "x"),
                         &weight = operand(args[2], where, "weight"), &given = argument(args[3], where, "pre"),
                         &status = argument(args[5], where, "status");
        const int act = static_cast<int>(PyLong_AsLong(args[4]));
        const bool need_x = PyObject_IsTrue(args[6]) == 1, need_w = PyObject_IsTrue(args[7]) == 1,
                   need_b = PyObject_IsTrue(args[8]) == 1;
        const int type = type_of(x, where, "x");
        const Rows xs = rows_of(x, where), ws = weight_rows(x, weight, xs.width, where);
        if (!fits({xs.width, ws.rows})) return result(NMS_ERR_CAPACITY, {});
        c10::DimVector shape(x.sizes().begin(), x.sizes().end());
        shape.back() = ws.rows;
        if (dy.sizes() != at::IntArrayRef(shape) || dy.scalar_type() != x.scalar_type() || dy.device() != x.device())
            refuse(where, "dy must be [..., outer] of x's type beside x");
        const Rows dys = rows_of(dy, where);
        at::Tensor pre;
        if ((act & ~NMS_ACT_ROUND_SLOPES) != NMS_ACT_NONE) {
            if (!given.defined()) refuse(where, "an activation's gradient needs the forward's pre");
            same(given, dy, where, "pre");
            pre = given.contiguous();
        }
        int32_t* const word = status_word(status, x, where);
        on_device(x, where, "x");
        if (!need_x && !need_w && !need_b) return result(NMS_OK, {{}, {}, {}});
        const at::Tensor dx = need_x ? like(x) : at::Tensor();
        const at::Tensor dw = need_w ? at::empty({ws.rows, ws.width}, x.options()) : at::Tensor();
        const at::Tensor db = need_b ? at::empty({ws.rows}, x.options().dtype(at::kFloat)) : at::Tensor();
        size_t bytes = 0;
        int code = linear_grad_workspace_size(type, xs.rows, xs.width, ws.rows, even(xs, x) && even(ws, x) && even(dys, x),
                                              &bytes);
        if (code != NMS_OK) return result(code, {});
        const at::Tensor work = scratch(bytes, x);
        code = launch(x, linear_grad_run, dys.at(), dys.row, xs.at(), xs.row, type, xs.rows, xs.width, ws.at(), ws.row,
                      ws.rows, address(pre), act, address(dx), address(dw), static_cast<float*>(address(db)), word,
                      address(work), bytes);
        return result(code, {dx, dw, db});
    });
}

// layer_norm(x, weight, bias, eps, residual, return_stats) -> (y[, sum][, mean, rstd])
PyObject* layer_norm(PyObject*, PyObject* const* args, Py_ssize_t n)
{
    return guarded(n, 6, [&]() -> PyObject* {
        const char* where = "layer_norm";
        const at::Tensor &x = operand(args[0], where, "x"), &weight = argument(args[1], where, "weight"),
                         &bias = argument(args[2], where, "bias"), &residual = argument(args[4], where, "residual");
        const double eps = PyFloat_AsDouble(args[3]);
        if (PyErr_Occurred()) return nullptr;
        const int type = type_of(x, where, "x");
        const Rows xs = rows_of(x, where);
        if (!fits({xs.width})) return result(NMS_ERR_CAPACITY, {});
        const int param_type = params(x, xs.width, {{"weight", &weight}, {"bias", &bias}}, where, "[width]");
        Rows res{{}, 0, 0, 0};
        if (residual.defined()) {
            same(residual, x, where, "residual");
            res = rows_of(residual, where);
        }
        on_device(x, where, "x");
        const at::Tensor y = like(x), sum = residual.defined() ? like(x) : at::Tensor();
        at::Tensor mean, rstd;
        if (args[5] == Py_True) {
            mean = at::empty(x.sizes().slice(0, x.dim() - 1), x.options().dtype(at::kFloat));
            rstd = at::empty_like(mean);
        }
        const int code = launch(x, layer_norm_run, xs.at(), xs.row, address(res.t), res.row, type, xs.rows, xs.width,
                                address(weight), address(bias), param_type, static_cast<float>(eps), address(y), address(sum),
                                static_cast<float*>(address(mean)), static_cast<float*>(address(rstd)));
        if (sum.defined()) return mean.defined() ? result(code, {y, sum, mean, rstd}) : result(code, {y, sum});
        return mean.defined() ? result(code, {y, mean, rstd}) : result(code, {y});
    });
}

// layer_norm_grad(dy, x, mean, rstd, weight, dsum) -> (dx, dweight, dbias)
PyObject* layer_norm_grad(PyObject*, PyObject* const* args, Py_ssize_t n)
{
    return guarded(n, 6, [&]() -> PyObject* {
        const char* where = "layer_norm_grad";
        const at::Tensor &dy = operand(args[0], where, "dy"), &x = operand(args[1], where, "x"),
                         &mean = operand(args[2], where, "mean"), &rstd = operand(args[3], where, "rstd"),
                         &weight = argument(args[4], where, "weight"), &dsum = argument(args[5], where, "dsum");
        const int type = type_of(x, where, "x");
        same(dy, x, where, "dy");
        const Rows xs = rows_of(x, where), dys = rows_of(dy, where);
        if (!fits({xs.width})) return result(NMS_ERR_CAPACITY, {});
        const int param_type = params(x, xs.width, {{"weight", &weight}}, where, "[width]");
        for (const at::Tensor* s : {&mean, &rstd})
            if (s->sizes() != x.sizes().slice(0, x.dim() - 1) || s->scalar_type() != at::kFloat ||
                s->device() != x.device() || !s->is_contiguous())
                refuse(where, "mean and rstd must be contiguous float32 [...] tensors beside x");
        Rows more{{}, 0, 0, 0};
        if (dsum.defined()) {
            same(dsum, x, where, "dsum");
            more = rows_of(dsum, where);
        }
        on_device(x, where, "x");
        const at::Tensor dx = like(x), dw = at::empty({xs.width}, x.options().dtype(at::kFloat)), db = at::empty_like(dw);
        size_t bytes = 0;
        int code = layer_norm_workspace_size(xs.rows, xs.width, &bytes);
        if (code != NMS_OK) return result(code, {});
        const at::Tensor work = scratch(bytes, x);
        code = launch(x, layer_norm_grad_run, dys.at(), dys.row, xs.at(), xs.row, address(more.t), more.row, type, xs.rows,
                      xs.width, static_cast<const float*>(mean.data_ptr()), static_cast<const float*>(rstd.data_ptr()),
                      address(weight), param_type, address(dx), static_cast<float*>(address(dw)),
                      static_cast<float*>(address(db)), address(work), bytes);
        return result(code, {dx, dw, db});
    });
}

// rotary(x, positions, lut, halves, inverse) -> (y,)
PyObject* rotary(PyObject*, PyObject* const* args, Py_ssize_t n)
{
    return guarded(n, 5, [&]() -> PyObject* {
        const bool inverse = PyObject_IsTrue(args[4]) == 1;
        const char* where = inverse ? "rotary_grad" : "rotary";
        const at::Tensor &given = operand(args[0], where, "x"), &positions = operand(args[1], where, "positions"),
                         &lut = operand(args[2], where, "lut");
        const int type = type_of(given, where, "x");
        if (given.dim() != 4) refuse(where, "x must be [batch, tokens, heads, dim]");
        const int64_t B = given.size(0), tokens = given.size(1), H = given.size(2), D = given.size(3);
        const auto kind = positions.scalar_type();
        if ((kind != at::kInt && kind != at::kFloat) || positions.dim() != 3 ||
            (positions.size(0) != 1 && positions.size(0) != B) || positions.size(1) != tokens ||
            positions.device() != given.device())
            refuse(where, "positions must be int32 or float32 [1 or batch, tokens, axes] beside x");
        if (lut.scalar_type() != at::kLong || lut.dim() != 2 || lut.size(0) != 2 || lut.device() != given.device() ||
            2 * lut.size(1) > D)
            refuse(where, "lut must be int64 [2, pairs] beside x, of no more pairs than x's vectors have");
        on_device(given, where, "x");
        if (!fits({H, D, positions.size(2)})) return result(NMS_ERR_CAPACITY, {});
        const at::Tensor p = positions.contiguous(), table = lut.contiguous();
        const at::Tensor x = D > 1 && given.stride(3) != 1 ? given.contiguous() : given;
        at::Tensor y = at::empty_like(x);  // a dense x keeps the order of its axes
        if (D > 1 && y.stride(3) != 1) y = like(x);
        const int code = launch(x, rotary_run, x.data_ptr(), x.stride(0), x.stride(1), x.stride(2), type, B, tokens, H, D,
                                p.data_ptr(), kind == at::kInt ? NMS_POSITION_I32 : NMS_TYPE_F32, p.size(0), p.size(2),
                                static_cast<const int64_t*>(table.data_ptr()), table.size(1),
                                PyObject_IsTrue(args[3]) == 1, inverse, y.data_ptr(), y.stride(0), y.stride(1), y.stride(2));
        return result(code, {y});
    });
}

// bind(address, ...): the C entries, in the order of the declarations above.
PyObject* bind(PyObject*, PyObject* const* args, Py_ssize_t n)
{
    void** const entries[] = {reinterpret_cast<void**>(&linear_workspace_size),
                              reinterpret_cast<void**>(&linear_run),
                              reinterpret_cast<void**>(&linear_grad_workspace_size),
                              reinterpret_cast<void**>(&linear_grad_run),
                              reinterpret_cast<void**>(&layer_norm_run),
                              reinterpret_cast<void**>(&layer_norm_workspace_size),
                              reinterpret_cast<void**>(&layer_norm_grad_run),
                              reinterpret_cast<void**>(&rotary_run)};
    if (n != static_cast<Py_ssize_t>(std::size(entries))) {
        PyErr_SetString(PyExc_TypeError, "wrong number of entries");
        return nullptr;
    }
    for (Py_ssize_t i = 0; i < n; ++i) {
        void* p = PyLong_AsVoidPtr(args[i]);
        if (!p) {
            if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "an entry without address");
            return nullptr;
        }
        *entries[i] = p;
    }
    Py_RETURN_NONE;
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyMethodDef method(const char* name)
{
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(F)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {method<bind>("bind"),
                         method<linear_act>("linear_act"),
                         method<linear_act_grad>("linear_act_grad"),
                         method<layer_norm>("layer_norm"),
                         method<layer_norm_grad>("layer_norm_grad"),
                         method<rotary>("rotary"),
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "gbblock", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_gbblock() { return PyModule_Create(&module); }
