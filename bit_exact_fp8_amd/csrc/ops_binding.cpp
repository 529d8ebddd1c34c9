// ops_binding.cpp -- the Python side of include/emu_operators.h and
// emu_block_operators.h for torch tensors: argument checks, outputs, workspaces
// and the call on torch's current stream.  Compiled, since a decoded token's
// call is shorter on the GPU than its checks are in Python (1 x 5760 x 1920 int8:
// 10.5 us a call with a binding through ctypes, the kernel 5).
//
// The emu_* functions are those of the library that is loaded before this
// module is (operators._binding).  Nothing is thrown across the C API: every
// entry turns what it catches into a Python error.
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/core/DeviceGuard.h>
#include <c10/core/AutogradState.h>
#include <c10/core/GradMode.h>
#include <c10/core/impl/VirtualGuardImpl.h>
#include <c10/hip/HIPStream.h>

#include <optional>
#include <string>

#include "../../include/emu_block_operators.h"

namespace {

using at::ScalarType;
using at::Tensor;

PyObject *g_emu_error = nullptr;  // api.EmuError

// What a call raises: a Python type and its text, or a status of the C ABI.
struct Refusal {
    PyObject *type;
    std::string text;
    int status = 0;
};
[[noreturn]] void value_error(const std::string &text) { throw Refusal{PyExc_ValueError, text}; }
[[noreturn]] void type_error(const std::string &text) { throw Refusal{PyExc_TypeError, text}; }
[[noreturn]] void unsupported(const std::string &text) { throw Refusal{g_emu_error, text, EMU_ERR_UNSUPPORTED}; }

std::string str(ScalarType t)
{
    switch (t) {
    case ScalarType::BFloat16: return "torch.bfloat16";
    case ScalarType::Half: return "torch.float16";
    case ScalarType::Float: return "torch.float32";
    default: return c10::toString(t);
    }
}
std::string str(at::IntArrayRef shape)
{
    std::string s = "(";
    for (size_t i = 0; i < shape.size(); ++i) s += (i ? ", " : "") + std::to_string(shape[i]);
    return s + (shape.size() == 1 ? ",)" : ")");
}

int code_of(ScalarType t)
{
    switch (t) {
    case ScalarType::BFloat16: return EMU_DT_BF16;
    case ScalarType::Half: return EMU_DT_FP16;
    case ScalarType::Float: return EMU_DT_FP32;
    case ScalarType::Float8_e4m3fn: return EMU_DT_E4M3FN;
    case ScalarType::Float8_e5m2: return EMU_DT_E5M2;
    case ScalarType::Char: return EMU_DT_INT8;
    default: return -1;
    }
}
emu_dtype code(const Tensor &t) { return static_cast<emu_dtype>(code_of(t.scalar_type())); }
bool is_float(ScalarType t) { return t == ScalarType::BFloat16 || t == ScalarType::Half || t == ScalarType::Float; }

// ---- arguments ----

const Tensor &tensor(const char *name, PyObject *o)
{
    if (!THPVariable_Check(o)) type_error(std::string(name) + " must be a tensor");
    return THPVariable_Unpack(o);
}
const Tensor *optional(const char *name, PyObject *o) { return o == Py_None ? nullptr : &tensor(name, o); }

const Tensor &gpu(const char *name, PyObject *o)
{
    if (!THPVariable_Check(o) || !THPVariable_Unpack(o).is_cuda()) value_error(std::string(name) + " must be a CUDA tensor");
    return THPVariable_Unpack(o);
}

// Refuses what autograd would lose: a gradient of an input or of an output that
// is given, and (torch.no_grad leaves those on) a forward-mode tangent.
// Arguments that are no tensors are refused later, by name.
void outside_autograd(std::initializer_list<PyObject *> inputs, std::initializer_list<PyObject *> outputs = {})
{
    const bool backward = c10::GradMode::is_enabled(), forward = c10::AutogradState::get_tls_state().get_fw_grad_mode();
    const auto check = [&](std::initializer_list<PyObject *> objects, const char *what, const char *then) {
        for (PyObject *o : objects) {
            if (o == Py_None || !THPVariable_Check(o)) continue;  // (None takes that check the long way: 0.3 us of a 5 us call)
            const Tensor &t = THPVariable_Unpack(o);
            if (backward && t.requires_grad())
                throw Refusal{PyExc_RuntimeError, std::string(what) + " requires a gradient: call under torch.no_grad()" + then};
            if (forward && t._fw_grad(0).defined())
                throw Refusal{PyExc_RuntimeError,
                              std::string(what) + " has a forward-mode tangent, which the call would drop: pass its primal"};
        }
    };
    check(inputs, "an input", " and make the backward call");
    check(outputs, "an output", "");
}

void floating(const char *name, const Tensor &t)
{
    if (!is_float(t.scalar_type()))
        type_error(std::string(name) + " must be bfloat16, float16 or float32, not " + str(t.scalar_type()));
}
void floating(const char *name, const Tensor &t, ScalarType beside)
{
    if (t.scalar_type() != beside && t.scalar_type() != ScalarType::Float)
        type_error(std::string(name) + " must be " + str(beside) + " or float32, not " + str(t.scalar_type()));
}

void on_device(const char *name, const Tensor &t, c10::Device device)
{
    if (t.device() != device)
        value_error(std::string(name) + " must be a CUDA tensor on the operands' device (" + device.str() + "), not " +
                    t.device().str());
}

// A tensor whose leading axes are rows.
struct Rows {
    int64_t T, n, ld;
};
Rows rows(const char *name, const Tensor &t)
{
    const int64_t dim = t.dim();
    if (dim == 0) value_error(std::string(name) + " must have at least one axis");
    Rows r{1, t.size(dim - 1), t.size(dim - 1)};
    for (int64_t d = 0; d < dim - 1; ++d) r.T *= t.size(d);
    if (r.T == 0 || r.n == 0) return r;
    if (r.n > 1 && t.stride(dim - 1) != 1) value_error(std::string(name) + " must have unit stride along its last axis");
    int64_t next = -1;  // the stride that the axis before must have
    for (int64_t d = dim - 2; d >= 0; --d) {
        if (t.size(d) == 1) continue;
        if (next < 0)
            r.ld = t.stride(d);
        else if (t.stride(d) != next)
            value_error(std::string(name) + "'s leading axes must be one axis of rows with one stride");
        next = t.stride(d) * t.size(d);
    }
    return r;
}
// The leading dimension of `t`, which has to have the shape and device of `like`.
int64_t same(const char *name, const Tensor &t, const Tensor &like)
{
    if (t.sizes() != like.sizes())
        value_error(std::string(name) + " must have shape " + str(like.sizes()) + ", not " + str(t.sizes()));
    on_device(name, t, like.device());
    return rows(name, t).ld;
}
void vector(const char *name, const Tensor &t, int64_t n, c10::Device device)
{
    if (t.dim() != 1 || t.size(0) != n || (n > 1 && t.stride(0) != 1))
        value_error(std::string(name) + " must be a dense vector of " + std::to_string(n) + " values");
    on_device(name, t, device);
}

ScalarType dtype_of(PyObject *o, bool (*allowed)(ScalarType))
{
    if (!THPDtype_Check(o) || !allowed(reinterpret_cast<THPDtype *>(o)->scalar_type)) {
        PyObject *s = PyObject_Str(o);
        const char *text = s ? PyUnicode_AsUTF8(s) : nullptr;
        std::string what = "output dtype " + std::string(text ? text : "?") + " is not supported";
        Py_XDECREF(s);
        PyErr_Clear();
        unsupported(what);
    }
    return reinterpret_cast<THPDtype *>(o)->scalar_type;
}

Tensor empty(at::IntArrayRef shape, const Tensor &like, ScalarType t)
{
    return at::empty(shape, at::TensorOptions().dtype(t).device(like.device()));
}
Tensor workspace(size_t bytes, const Tensor &like)
{
    return bytes ? empty({static_cast<int64_t>(bytes)}, like, ScalarType::Byte) : Tensor();
}
void *ptr(const Tensor *t) { return t ? t->data_ptr() : nullptr; }
void *ptr(const Tensor &t) { return t.defined() ? t.data_ptr() : nullptr; }
template <typename T>
T *as(const Tensor *t) { return static_cast<T *>(ptr(t)); }
template <typename T>
T *as(const Tensor &t) { return static_cast<T *>(ptr(t)); }

// f(stream) on torch's current stream of `device`, without the interpreter's lock.
template <typename F>
void launch(c10::Device device, F f)
{
    const c10::impl::VirtualGuardImpl impl(device.type());
    std::optional<c10::DeviceGuard> guard;
    if (impl.getDevice() != device) guard.emplace(device);
    const hipStream_t stream = c10::hip::getCurrentHIPStream(device.index()).stream();
    emu_status s;
    Py_BEGIN_ALLOW_THREADS
    s = f(stream);
    Py_END_ALLOW_THREADS
    if (s != EMU_OK) throw Refusal{g_emu_error, emu_last_error_message(), s};
}

// Autograd is told that a call has written `t`, as for torch's own operators
// (a tensor of inference mode counts no versions, and nothing saves one).
void written(const Tensor &t)
{
    if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

// ---- the calls ----

PyObject *wrap(const Tensor &t)
{
    if (t.defined()) return THPVariable_Wrap(t);
    Py_RETURN_NONE;
}
PyObject *held(PyObject *o)
{
    Py_INCREF(o);
    return o;
}
// A tuple of new references (any of which may be null: an error is set then).
PyObject *tuple(std::initializer_list<PyObject *> items)
{
    PyObject *t = PyTuple_New(static_cast<Py_ssize_t>(items.size()));
    Py_ssize_t i = 0;
    bool bad = !t;
    for (PyObject *o : items) {
        bad |= !o;
        if (t && o)
            PyTuple_SET_ITEM(t, i, o);
        else
            Py_XDECREF(o);
        ++i;
    }
    if (bad) Py_CLEAR(t);
    return t;
}

// x, weight, residual, eps, out_dtype, scale, h_out
PyObject *add_rms_norm_quant(PyObject *const *a)
{
    outside_autograd({a[0], a[1], a[2], a[5]}, {a[6]});
    const Tensor &x = gpu("x", a[0]), &weight = tensor("weight", a[1]);
    const Tensor *residual = optional("residual", a[2]), *scale = optional("scale", a[5]), *given_h = optional("h_out", a[6]);
    const c10::Device dev = x.device();
    floating("x", x);
    floating("weight", weight, x.scalar_type());
    const Rows r = rows("x", x);
    vector("weight", weight, r.n, dev);
    const double eps = PyFloat_AsDouble(a[3]);
    if (eps == -1.0 && PyErr_Occurred()) return nullptr;
    const ScalarType out = dtype_of(a[4], [](ScalarType t) {
        return t == ScalarType::Float8_e4m3fn || t == ScalarType::Float8_e5m2 || t == ScalarType::Char;
    });
    int64_t ldr = 0, ldh = 0;
    Tensor h;
    if (residual) {
        floating("residual", *residual, x.scalar_type());
        ldr = same("residual", *residual, x);
        ldh = r.n;
        if (given_h) {
            if (given_h->scalar_type() != residual->scalar_type()) type_error("h_out must be of the residual's type");
            ldh = same("h_out", *given_h, x);
        } else {
            h = empty(x.sizes(), x, residual->scalar_type());
        }
    } else if (given_h) {
        value_error("h_out needs a residual");
    }
    Tensor own;
    if (!scale) {
        c10::SmallVector<int64_t, 6> shape(x.sizes().begin(), x.sizes().end());
        shape.back() = 1;
        own = empty(shape, x, ScalarType::Float);
    } else {
        if (scale->numel() != 1 || scale->scalar_type() != ScalarType::Float)
            value_error("scale must be a one-element float32 tensor");
        on_device("scale", *scale, dev);
    }
    const Tensor codes = empty(x.sizes(), x, out);
    launch(dev, [&](hipStream_t stream) {
        return emu_add_rms_norm_quant(ptr(x), code(x), r.ld, ptr(weight), code(weight), ptr(residual),
                                      residual ? code(*residual) : EMU_DT_BF16, ldr, r.T, r.n, static_cast<float>(eps),
                                      ptr(codes), code(codes), r.n, as<float>(scale), as<float>(own),
                                      given_h ? ptr(given_h) : ptr(h), ldh, stream);
    });
    if (given_h) written(*given_h);
    return tuple({wrap(codes), scale ? held(a[5]) : wrap(own), given_h ? held(a[6]) : wrap(h)});
}

// g, h, weight, eps, grad_h
PyObject *add_rms_norm_backward(PyObject *const *a)
{
    outside_autograd({a[0], a[1], a[2], a[4]});
    const Tensor &g = gpu("g", a[0]), &h = tensor("h", a[1]), &weight = tensor("weight", a[2]);
    const Tensor *grad_h = optional("grad_h", a[4]);
    const c10::Device dev = g.device();
    floating("g", g);
    floating("h", h, g.scalar_type());
    floating("weight", weight, g.scalar_type());
    const Rows r = rows("g", g);
    const int64_t ldh = same("h", h, g);
    vector("weight", weight, r.n, dev);
    const double eps = PyFloat_AsDouble(a[3]);
    if (eps == -1.0 && PyErr_Occurred()) return nullptr;
    int64_t ldgh = 0;
    if (grad_h) {
        floating("grad_h", *grad_h, g.scalar_type());
        ldgh = same("grad_h", *grad_h, g);
    }
    const Tensor grad_in = empty(g.sizes(), g, g.scalar_type()), grad_weight = empty({r.n}, g, weight.scalar_type());
    const size_t bytes = emu_add_rms_norm_backward_workspace(r.T, r.n);
    const Tensor ws = workspace(bytes, g);
    launch(dev, [&](hipStream_t stream) {
        return emu_add_rms_norm_backward(ptr(g), code(g), r.ld, ptr(h), code(h), ldh, ptr(weight), code(weight), ptr(grad_h),
                                         grad_h ? code(*grad_h) : EMU_DT_BF16, ldgh, r.T, r.n, static_cast<float>(eps),
                                         ptr(grad_in), r.n, ptr(grad_weight), ptr(ws), bytes, stream);
    });
    return tuple({wrap(grad_in), wrap(grad_weight)});
}

// 1 where `s` has a scale for each row (or column), 0 where it has one for all.
int scale_per_row(const char *name, const Tensor &s, int64_t n, bool column, c10::Device device)
{
    if (s.scalar_type() != ScalarType::Float) value_error(std::string(name) + " must be a float32 tensor");
    on_device(name, s, device);
    if (s.numel() == 1) return 0;
    const bool shaped = (s.dim() == 1 && s.size(0) == n) ||
                        (s.dim() == 2 && s.size(column ? 0 : 1) == 1 && s.size(column ? 1 : 0) == n);
    if (!shaped || !s.is_contiguous()) {
        const std::string v = std::to_string(n);
        value_error(std::string(name) + " must be dense with one value, or of shape (" + v + ",) or " +
                    (column ? "(1, " + v + ")" : "(" + v + ", 1)"));
    }
    return 1;
}

// mat1, mat2, scale_a, scale_b, bias, out_dtype, out
PyObject *int8_scaled_mm(PyObject *const *a)
{
    outside_autograd({a[2], a[3], a[4]}, {a[6]});
    const Tensor &x = tensor("mat1", a[0]), &w = tensor("mat2", a[1]);
    if (x.scalar_type() != ScalarType::Char || w.scalar_type() != ScalarType::Char)
        type_error("expected int8 operands, got " + str(x.scalar_type()) + " and " + str(w.scalar_type()));
    if (x.dim() != 2 || w.dim() != 2) value_error("mat1 and mat2 must be 2-D");
    const int64_t M = x.size(0), K = x.size(1), N = w.size(1);
    if (w.size(0) != K)
        value_error("inner dimensions differ: " + std::to_string(K) + " vs " + std::to_string(w.size(0)));
    if (K > 1 && x.stride(1) != 1) value_error("mat1 must be row-major [M, K] (unit stride along K)");
    if (K > 1 && w.stride(0) != 1) value_error("mat2 must be column-major [K, N] (pass w.t() for a row-major w)");
    if (!x.is_cuda()) value_error("the operands must be CUDA tensors, not " + x.device().str());
    const c10::Device dev = x.device();
    on_device("mat2", w, dev);
    const int64_t lda = M > 1 && K > 0 ? x.stride(0) : K, ldw = N > 1 && K > 0 ? w.stride(1) : K;
    const ScalarType out_dtype = dtype_of(a[5], is_float);
    if (!THPVariable_Check(a[2])) value_error("scale_a must be a float32 tensor");
    if (!THPVariable_Check(a[3])) value_error("scale_b must be a float32 tensor");
    const Tensor &sa = tensor("scale_a", a[2]), &sb = tensor("scale_b", a[3]);
    const int per_a = scale_per_row("scale_a", sa, M, false, dev), per_b = scale_per_row("scale_b", sb, N, true, dev);
    const Tensor *bias = optional("bias", a[4]), *given = optional("out", a[6]);
    if (bias) {
        floating("bias", *bias, out_dtype);
        vector("bias", *bias, N, dev);
    }
    int64_t ldo = N;
    Tensor out;
    if (given) {
        on_device("out", *given, dev);
        if (given->dim() != 2 || given->size(0) != M || given->size(1) != N || given->scalar_type() != out_dtype ||
            (N > 1 && given->stride(1) != 1))
            value_error("out must be a row-major [M, N] tensor of out_dtype");
        if (M > 1) ldo = given->stride(0);
    } else {
        out = empty({M, N}, x, out_dtype);
    }
    const int8_t *xp = as<int8_t>(x), *wp = as<int8_t>(w);
    const bool aligned = !((reinterpret_cast<uintptr_t>(xp) | reinterpret_cast<uintptr_t>(wp) | lda | ldw) & 15) &&
                         lda <= EMU_INT8_MAX_ALIGNED_LD && ldw <= EMU_INT8_MAX_ALIGNED_LD;
    const size_t bytes = emu_int8_scaled_mm_workspace(M, N, K, aligned);
    const Tensor ws = workspace(bytes, x);
    launch(dev, [&](hipStream_t stream) {
        return emu_int8_scaled_mm(xp, lda, wp, ldw, M, N, K, as<float>(sa), per_a, as<float>(sb), per_b, ptr(bias),
                                  bias ? code(*bias) : EMU_DT_BF16, given ? ptr(given) : ptr(out),
                                  static_cast<emu_dtype>(code_of(out_dtype)), ldo, ptr(ws), bytes, stream);
    });
    if (given) written(*given);
    return given ? held(a[6]) : wrap(out);
}

// Tokens of the logits' leading axes, with or without one of their own; C to a row.
int64_t tokens_of(const Tensor &tokens, const Tensor &logits)
{
    const at::IntArrayRef lead = logits.sizes().slice(0, logits.dim() - 1), shape = tokens.sizes();
    if (tokens.scalar_type() != ScalarType::Long) type_error("tokens must be int64, not " + str(tokens.scalar_type()));
    const bool one = shape == lead;
    if (!one && (shape.empty() || shape.slice(0, shape.size() - 1) != lead))
        value_error("tokens must have shape " + str(lead) + ", or that and one axis more, not " + str(shape));
    on_device("tokens", tokens, logits.device());
    return one ? 1 : shape.back();
}

// A dense tensor of one value a row (or few): an expanded gradient is laid out.
Tensor small(const char *name, const Tensor &t, at::IntArrayRef shape, c10::Device device, ScalarType dtype = ScalarType::Float)
{
    if (t.sizes() != shape || t.scalar_type() != dtype)
        value_error(std::string(name) + " must be a " + (dtype == ScalarType::Long ? "torch.int64" : "torch.float32") +
                    " tensor of shape " + str(shape));
    on_device(name, t, device);
    return t.contiguous();
}

c10::SmallVector<int64_t, 6> with_axis(at::IntArrayRef lead, int64_t k)
{
    c10::SmallVector<int64_t, 6> s(lead.begin(), lead.end());
    s.push_back(k);
    return s;
}

// logits, tokens, top_k
PyObject *token_logprobs(PyObject *const *a)
{
    outside_autograd({a[0]});
    const Tensor &logits = gpu("logits", a[0]), &given = tensor("tokens", a[1]);
    floating("logits", logits);
    const Rows r = rows("logits", logits);
    const int64_t C = tokens_of(given, logits);
    const int64_t k = PyLong_AsLongLong(a[2]);
    if (k == -1 && PyErr_Occurred()) return nullptr;
    const Tensor tokens = given.contiguous();
    const at::IntArrayRef lead = logits.sizes().slice(0, logits.dim() - 1);
    const Tensor lp = empty(given.sizes(), logits, ScalarType::Float), entropy = empty(lead, logits, ScalarType::Float),
                 lse = empty(lead, logits, ScalarType::Float);
    Tensor top_lp, top;
    if (k > 0) {
        top_lp = empty(with_axis(lead, k), logits, ScalarType::Float);
        top = empty(with_axis(lead, k), logits, ScalarType::Long);
    }
    const size_t bytes = emu_token_logprobs_workspace(r.T, r.n, k);
    const Tensor ws = workspace(bytes, logits);
    launch(logits.device(), [&](hipStream_t stream) {
        return emu_token_logprobs(ptr(logits), code(logits), r.ld, r.T, r.n, as<int64_t>(tokens), C, k, as<float>(lp),
                                  as<float>(entropy), as<float>(lse), as<float>(top_lp), as<int64_t>(top), ptr(ws), bytes,
                                  stream);
    });
    return tuple({wrap(lp), wrap(entropy), wrap(lse), wrap(top_lp), wrap(top)});
}

// logits, tokens, lse, entropy, grad_logprobs, grad_entropy, top_tokens, grad_top, out
PyObject *token_logprobs_backward(PyObject *const *a)
{
    outside_autograd({a[0], a[2], a[3], a[4], a[5], a[7]}, {a[8]});
    const Tensor &logits = gpu("logits", a[0]), &given = tensor("tokens", a[1]), &lse0 = tensor("lse", a[2]);
    const Tensor *entropy0 = optional("entropy", a[3]), *g0 = optional("grad_logprobs", a[4]),
                 *ge0 = optional("grad_entropy", a[5]), *top0 = optional("top_tokens", a[6]), *gt0 = optional("grad_top", a[7]),
                 *given_out = optional("out", a[8]);
    const c10::Device dev = logits.device();
    floating("logits", logits);
    const Rows r = rows("logits", logits);
    const int64_t C = tokens_of(given, logits);
    const Tensor tokens = given.contiguous();
    const at::IntArrayRef lead = logits.sizes().slice(0, logits.dim() - 1);
    const Tensor lse = small("lse", lse0, lead, dev);
    Tensor entropy, g, ge, top, gt, out;
    if (entropy0) entropy = small("entropy", *entropy0, lead, dev);
    if (g0) g = small("grad_logprobs", *g0, given.sizes(), dev);
    if (ge0) {
        if (!entropy0) value_error("grad_entropy needs the entropy");
        ge = small("grad_entropy", *ge0, lead, dev);
    }
    int64_t k = 0;
    if (gt0) {
        if (!top0) value_error("grad_top needs top_tokens");
        k = gt0->dim() ? gt0->size(gt0->dim() - 1) : 0;
        gt = small("grad_top", *gt0, with_axis(lead, k), dev);
        top = small("top_tokens", *top0, with_axis(lead, k), dev, ScalarType::Long);
    }
    int64_t ldo = r.n;
    if (given_out) {
        if (given_out->scalar_type() != logits.scalar_type()) type_error("out must be of the logits' type");
        ldo = same("out", *given_out, logits);
    } else {
        out = empty(logits.sizes(), logits, logits.scalar_type());
    }
    launch(dev, [&](hipStream_t stream) {
        return emu_token_logprobs_backward(ptr(logits), code(logits), r.ld, r.T, r.n, as<int64_t>(tokens), C, as<float>(lse),
                                           as<float>(entropy), as<float>(g), as<float>(ge), as<int64_t>(top), as<float>(gt), k,
                                           given_out ? ptr(given_out) : ptr(out), ldo, stream);
    });
    if (given_out) written(*given_out);
    return given_out ? held(a[8]) : wrap(out);
}

// ---- codes with a scale for each block of 128 ----

int64_t blocks_of(int64_t n) { return (n + EMU_BLOCK - 1) / EMU_BLOCK; }
bool is_code(ScalarType t) { return t == ScalarType::Float8_e4m3fn || t == ScalarType::Float8_e5m2; }
bool is_scale(ScalarType t) { return t == ScalarType::Float || t == ScalarType::Float8_e8m0fnu; }
emu_scale_type scale_code(ScalarType t) { return t == ScalarType::Float ? EMU_SCALE_FP32 : EMU_SCALE_E8M0; }
void codes(const char *name, const Tensor &t)
{
    if (!is_code(t.scalar_type()))
        type_error(std::string(name) + " must be float8_e4m3fn or float8_e5m2, not " + str(t.scalar_type()));
}
void scales(const char *name, const Tensor &t)
{
    if (!is_scale(t.scalar_type()))
        type_error(std::string(name) + " must be float32 or float8_e8m0fnu, not " + str(t.scalar_type()));
}
void shaped(const char *name, const Tensor &t, at::IntArrayRef shape, c10::Device device)
{
    if (t.sizes() != shape) value_error(std::string(name) + " must have shape " + str(shape) + ", not " + str(t.sizes()));
    on_device(name, t, device);
}
void dense(const char *name, const Tensor &t, at::IntArrayRef shape, c10::Device device)
{
    shaped(name, t, shape, device);
    if (!t.is_contiguous()) value_error(std::string(name) + " must be dense");
}
// A gradient, laid out where it is one value (or row) expanded.
Tensor laid_out(const Tensor &t)
{
    for (int64_t d = 0; d < t.dim(); ++d)
        if (t.stride(d) == 0 && t.size(d) > 1) return t.contiguous();
    return t;
}
bool truth(PyObject *o)
{
    const int b = PyObject_IsTrue(o);
    if (b < 0) {
        PyErr_Clear();
        type_error("expected a truth value");
    }
    return b != 0;
}

// Each group's end in rows: their bits.
int ends_bits(const Tensor &ends, int64_t E, c10::Device device)
{
    if (ends.scalar_type() != ScalarType::Int && ends.scalar_type() != ScalarType::Long)
        type_error("ends must be int32 or int64, not " + str(ends.scalar_type()));
    dense("ends", ends, {E}, device);
    return ends.scalar_type() == ScalarType::Int ? 32 : 64;
}

// x, block_rows, out_dtype, scale_dtype
PyObject *block_quant(PyObject *const *a)
{
    outside_autograd({a[0]});
    const Tensor &x = gpu("x", a[0]);
    floating("x", x);
    const int64_t block_rows = PyLong_AsLongLong(a[1]);
    if (block_rows == -1 && PyErr_Occurred()) return nullptr;
    if (block_rows != 1 && block_rows != EMU_BLOCK) value_error("block_rows must be 1 or 128");
    const ScalarType out = dtype_of(a[2], is_code), scale = dtype_of(a[3], is_scale);
    c10::SmallVector<int64_t, 6> shape(x.sizes().begin(), x.sizes().end());
    int64_t E = 1, stride = 0;
    Rows r{};
    if (block_rows == 1) {
        r = rows("x", x);
    } else {
        const int64_t dim = x.dim();
        if (dim != 2 && dim != 3) value_error("x must be a matrix or a batch of them");
        E = dim == 3 ? x.size(0) : 1;
        stride = E > 1 ? x.stride(0) : 0;
        r = {x.size(dim - 2), x.size(dim - 1), x.size(dim - 2) > 1 ? x.stride(dim - 2) : x.size(dim - 1)};
        if (E > 0 && r.T > 0 && r.n > 1 && x.stride(dim - 1) != 1) value_error("x must have unit stride along its last axis");
        shape[dim - 2] = blocks_of(r.T);
    }
    shape.back() = blocks_of(r.n);
    const Tensor q = empty(x.sizes(), x, out), s = empty(shape, x, scale);
    launch(x.device(), [&](hipStream_t stream) {
        return emu_block_quant(ptr(x), code(x), r.ld, stride, E, r.T, r.n, static_cast<int>(block_rows), ptr(q), code(q), ptr(s),
                               scale_code(scale), stream);
    });
    return tuple({wrap(q), wrap(s)});
}

// gate, up, out_dtype, scale_dtype, keep
PyObject *swiglu_block_quant(PyObject *const *a)
{
    outside_autograd({a[0], a[1]});
    const Tensor &gate = gpu("gate", a[0]), &up = tensor("up", a[1]);
    floating("gate", gate);
    if (up.scalar_type() != gate.scalar_type()) type_error("up must be of gate's type");
    const Rows r = rows("gate", gate);
    const int64_t ldup = same("up", up, gate);
    const ScalarType out = dtype_of(a[2], is_code), scale = dtype_of(a[3], is_scale);
    const bool keep = truth(a[4]);
    c10::SmallVector<int64_t, 6> shape(gate.sizes().begin(), gate.sizes().end());
    const Tensor q = empty(shape, gate, out);
    shape.back() = blocks_of(r.n);
    const Tensor s = empty(shape, gate, scale);
    Tensor kept, kept_s;
    if (keep) {
        shape.back() = 2 * blocks_of(r.n);
        kept_s = empty(shape, gate, scale);
        shape.back() = 2 * r.n;
        kept = empty(shape, gate, out);
    }
    launch(gate.device(), [&](hipStream_t stream) {
        return emu_swiglu_block_quant(ptr(gate), r.ld, ptr(up), ldup, code(gate), r.T, r.n, ptr(q), code(q), ptr(s),
                                      scale_code(scale), ptr(kept), ptr(kept_s), stream);
    });
    return tuple({wrap(q), wrap(s), wrap(kept), wrap(kept_s)});
}

// grad_h, kept, kept_scale
PyObject *swiglu_block_backward(PyObject *const *a)
{
    outside_autograd({a[0], a[1], a[2]});
    const Tensor &given = gpu("grad_h", a[0]), &kept = tensor("kept", a[1]), &kept_s = tensor("kept_scale", a[2]);
    floating("grad_h", given);
    const Tensor g = laid_out(given);
    codes("kept", kept);
    scales("kept_scale", kept_s);
    const Rows r = rows("grad_h", g);
    c10::SmallVector<int64_t, 6> shape(g.sizes().begin(), g.sizes().end());
    shape.back() = 2 * blocks_of(r.n);
    dense("kept_scale", kept_s, shape, g.device());
    shape.back() = 2 * r.n;
    dense("kept", kept, shape, g.device());
    const Tensor grad = empty(shape, g, g.scalar_type());
    launch(g.device(), [&](hipStream_t stream) {
        return emu_swiglu_block_backward(ptr(g), code(g), r.ld, ptr(kept), code(kept), ptr(kept_s),
                                         scale_code(kept_s.scalar_type()), r.T, r.n, ptr(grad), 2 * r.n, stream);
    });
    return wrap(grad);
}

// Codes, their scales, and where both lie: rows (of one matrix) by K.
struct Coded {
    int8_t *p;
    int64_t rows, K, ld, stride;
    void *scales;
    int64_t s_row, s_block, s_stride;
    bool aligned() const
    {
        return !((reinterpret_cast<uintptr_t>(p) | ld | stride) & 15) && ld <= EMU_BLOCK_MAX_ALIGNED_LD;
    }
};
// mat1 [M, K] with scale_a [M, blocks of K]
Coded left(const Tensor &x, const Tensor &s)
{
    codes("mat1", x);
    scales("scale_a", s);
    if (x.dim() != 2) value_error("mat1 must be 2-D");
    if (!x.is_cuda()) value_error("the operands must be CUDA tensors, not " + x.device().str());
    const int64_t M = x.size(0), K = x.size(1);
    if (K > 1 && M > 0 && x.stride(1) != 1) value_error("mat1 must be row-major [M, K] (unit stride along K)");
    shaped("scale_a", s, {M, blocks_of(K)}, x.device());
    return {as<int8_t>(x), M, K, M > 1 && K > 0 ? x.stride(0) : K, 0, ptr(s), M > 1 ? s.stride(0) : 0,
            K > EMU_BLOCK ? s.stride(1) : 0, 0};
}
// mat2 [K, N] (or [E, K, N]) column-major, with scale_b [blocks of K, blocks of N] (or [E, ...])
Coded right(const Tensor &w, const Tensor &s, const Tensor &x, int64_t K, bool grouped)
{
    codes("mat2", w);
    scales("scale_b", s);
    const int64_t d = grouped ? 1 : 0;
    if (w.dim() != 2 + d) value_error(grouped ? "mat2 must be 3-D" : "mat2 must be 2-D");
    on_device("mat2", w, x.device());
    const int64_t N = w.size(1 + d), E = grouped ? w.size(0) : 1;
    if (w.size(d) != K) value_error("inner dimensions differ: " + std::to_string(K) + " vs " + std::to_string(w.size(d)));
    if (K > 1 && N > 0 && E > 0 && w.stride(d) != 1) value_error("mat2 must be column-major [K, N] (pass w.t() for a row-major w)");
    if (grouped)
        shaped("scale_b", s, {E, blocks_of(K), blocks_of(N)}, x.device());
    else
        shaped("scale_b", s, {blocks_of(K), blocks_of(N)}, x.device());
    return {as<int8_t>(w), N, K, N > 1 && K > 0 ? w.stride(1 + d) : K, E > 1 ? w.stride(0) : 0, ptr(s),
            N > EMU_BLOCK ? s.stride(1 + d) : 0, K > EMU_BLOCK ? s.stride(d) : 0, E > 1 ? s.stride(0) : 0};
}
// An output given, or a new one, of [M, N].
struct Output {
    Tensor own;
    void *p;
    int64_t ld;
};
Output output(const Tensor *given, int64_t M, int64_t N, ScalarType dtype, const Tensor &x)
{
    Output o{Tensor(), nullptr, N};
    if (!given) {
        o.own = empty({M, N}, x, dtype);
        o.p = ptr(o.own);
        return o;
    }
    on_device("out", *given, x.device());
    if (given->dim() != 2 || given->size(0) != M || given->size(1) != N || given->scalar_type() != dtype ||
        (N > 1 && M > 0 && given->stride(1) != 1))
        value_error("out must be a row-major [M, N] tensor of out_dtype");
    if (M > 1) o.ld = given->stride(0);
    o.p = given->data_ptr();
    return o;
}
void one_type(const Tensor &a, const Tensor &b)
{
    if (a.scalar_type() != b.scalar_type()) type_error("scale_a and scale_b must be of one type");
}

// mat1, mat2, scale_a, scale_b, bias, out_dtype, out
PyObject *block_scaled_mm(PyObject *const *a)
{
    outside_autograd({a[0], a[1], a[2], a[3], a[4]}, {a[6]});
    const Tensor &x = tensor("mat1", a[0]), &w = tensor("mat2", a[1]), &sa = tensor("scale_a", a[2]), &sb = tensor("scale_b", a[3]);
    const Coded l = left(x, sa), r = right(w, sb, x, l.K, false);
    one_type(sa, sb);
    const ScalarType dtype = dtype_of(a[5], is_float);
    const Tensor *bias = optional("bias", a[4]), *given = optional("out", a[6]);
    if (bias) {
        floating("bias", *bias, dtype);
        vector("bias", *bias, r.rows, x.device());
    }
    const Output o = output(given, l.rows, r.rows, dtype, x);
    const emu_dtype out_code = static_cast<emu_dtype>(code_of(dtype));
    const size_t bytes = emu_block_scaled_mm_workspace(l.rows, r.rows, l.K, out_code, l.aligned(), r.aligned());
    const Tensor ws = workspace(bytes, x);
    launch(x.device(), [&](hipStream_t stream) {
        return emu_block_scaled_mm(l.p, code(x), l.ld, r.p, code(w), r.ld, l.rows, r.rows, l.K, l.scales, l.s_row, l.s_block,
                                   r.scales, r.s_row, r.s_block, scale_code(sa.scalar_type()), ptr(bias),
                                   bias ? code(*bias) : EMU_DT_BF16, o.p, out_code, o.ld, ptr(ws), bytes, stream);
    });
    if (given) written(*given);
    return given ? held(a[6]) : wrap(o.own);
}

// mat1, mat2, scale_a, scale_b, ends, out_dtype, out
PyObject *grouped_block_scaled_mm(PyObject *const *a)
{
    outside_autograd({a[0], a[1], a[2], a[3]}, {a[6]});
    const Tensor &x = tensor("mat1", a[0]), &w = tensor("mat2", a[1]), &sa = tensor("scale_a", a[2]), &sb = tensor("scale_b", a[3]),
                 &ends = tensor("ends", a[4]);
    const Coded l = left(x, sa), r = right(w, sb, x, l.K, true);
    one_type(sa, sb);
    const int64_t E = w.size(0);
    const int bits = ends_bits(ends, E, x.device());
    const ScalarType dtype = dtype_of(a[5], is_float);
    const Tensor *given = optional("out", a[6]);
    const Output o = output(given, l.rows, r.rows, dtype, x);
    const emu_dtype out_code = static_cast<emu_dtype>(code_of(dtype));
    const size_t bytes = emu_grouped_block_scaled_mm_workspace(l.rows, E, r.rows, l.K, out_code, l.aligned(), r.aligned());
    const Tensor ws = workspace(bytes, x);
    launch(x.device(), [&](hipStream_t stream) {
        return emu_grouped_block_scaled_mm(l.p, code(x), l.ld, r.p, code(w), r.ld, r.stride, l.rows, E, r.rows, l.K, l.scales, l.s_row,
                                           l.s_block, r.scales, r.s_row, r.s_block, r.s_stride, scale_code(sa.scalar_type()),
                                           ptr(ends), bits, given ? 0 : 1, o.p, out_code, o.ld, ptr(ws), bytes, stream);
    });
    if (given) written(*given);
    return given ? held(a[6]) : wrap(o.own);
}

// grad, codes, scale, ends, out_dtype, out
PyObject *block_weight_grad(PyObject *const *a)
{
    outside_autograd({a[0], a[1], a[2]}, {a[5]});
    const Tensor &grad = gpu("grad", a[0]), &x = tensor("codes", a[1]), &s = tensor("scale", a[2]);
    const Tensor *ends = optional("ends", a[3]), *given = optional("out", a[5]);
    floating("grad", grad);
    const Tensor g = laid_out(grad);
    codes("codes", x);
    if (s.scalar_type() != ScalarType::Float8_e8m0fnu)
        type_error("scale must be float8_e8m0fnu (powers of two), not " + str(s.scalar_type()));
    if (g.dim() < 2 || x.dim() < 2) value_error("grad and codes must be matrices of rows");
    const Rows r = rows("grad", g), c = rows("codes", x);
    on_device("codes", x, g.device());
    if (g.sizes().slice(0, g.dim() - 1) != x.sizes().slice(0, x.dim() - 1))
        value_error("codes must have grad's rows " + str(g.sizes().slice(0, g.dim() - 1)) + ", not " +
                    str(x.sizes().slice(0, x.dim() - 1)));
    c10::SmallVector<int64_t, 6> shape(x.sizes().begin(), x.sizes().end());
    shape.back() = blocks_of(c.n);
    shaped("scale", s, shape, g.device());
    int64_t s_row = 0, s_block = c.n > EMU_BLOCK ? s.stride(s.dim() - 1) : 0;
    if (s.dim() == 2) {
        if (c.T > 1) s_row = s.stride(0);
    } else {
        if (!s.is_contiguous()) value_error("scale of more than two axes must be dense");
        s_row = blocks_of(c.n);
    }
    int64_t E = 0;
    int bits = 32;
    if (ends) {
        if (ends->dim() != 1) value_error("ends must be a dense vector");
        E = ends->size(0);
        bits = ends_bits(*ends, E, g.device());
    }
    const ScalarType dtype = a[4] == Py_None ? g.scalar_type() : dtype_of(a[4], is_float);
    c10::SmallVector<int64_t, 3> out_shape;
    if (ends) out_shape.push_back(E);
    out_shape.push_back(r.n);
    out_shape.push_back(c.n);
    Tensor own;
    int64_t ldo = c.n, stride = r.n * c.n;
    if (given) {
        shaped("out", *given, out_shape, g.device());
        if (given->scalar_type() != dtype) type_error("out must be of out_dtype");
        const int64_t d = given->dim();
        if (given->numel() && c.n > 1 && given->stride(d - 1) != 1) value_error("out must be row-major");
        if (given->numel() && r.n > 1) ldo = given->stride(d - 2);
        if (given->numel() && E > 1) stride = given->stride(0);
    } else {
        own = empty(out_shape, g, dtype);
    }
    const int64_t unit = 16 / g.element_size();
    const auto at = [](const Tensor &t) { return reinterpret_cast<uintptr_t>(t.data_ptr()); };
    const bool ga = !(at(g) & 15) && r.ld % unit == 0 && r.ld <= EMU_BLOCK_MAX_ALIGNED_LD,
               ca = !(at(x) & 15) && c.ld % 16 == 0 && c.ld <= EMU_BLOCK_MAX_ALIGNED_LD;
    if (ends && E == 0) return given ? held(a[5]) : wrap(own);
    const size_t bytes = emu_block_weight_grad_workspace(r.T, E, r.n, c.n, code(g), ga, ca);
    const Tensor ws = workspace(bytes, g);
    launch(g.device(), [&](hipStream_t stream) {
        return emu_block_weight_grad(ptr(g), code(g), r.ld, ptr(x), code(x), c.ld, ptr(s), s_row, s_block, r.T, r.n, c.n,
                                     ptr(ends), bits, E, given ? ptr(given) : ptr(own),
                                     static_cast<emu_dtype>(code_of(dtype)), ldo, stride, ptr(ws), bytes, stream);
    });
    if (given) written(*given);
    return given ? held(a[5]) : wrap(own);
}

template <PyObject *(*call)(PyObject *const *), int N>
PyObject *entry(PyObject *, PyObject *const *args, Py_ssize_t nargs)
{
    HANDLE_TH_ERRORS
    try {
        if (nargs != N) throw Refusal{PyExc_TypeError, "wrong number of arguments"};
        return call(args);
    } catch (const Refusal &r) {
        if (r.type == g_emu_error) {
            PyObject *e = PyObject_CallFunction(g_emu_error, "is", r.status, r.text.c_str());
            if (e) PyErr_SetObject(g_emu_error, e);
            Py_XDECREF(e);
        } else {
            PyErr_SetString(r.type, r.text.c_str());
        }
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

template <PyObject *(*call)(PyObject *const *), int N>
PyCFunction function()
{
    return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<call, N>));
}

PyMethodDef g_methods[] = {
    {"add_rms_norm_quant", function<add_rms_norm_quant, 7>(), METH_FASTCALL, nullptr},
    {"add_rms_norm_backward", function<add_rms_norm_backward, 5>(), METH_FASTCALL, nullptr},
    {"int8_scaled_mm", function<int8_scaled_mm, 7>(), METH_FASTCALL, nullptr},
    {"token_logprobs", function<token_logprobs, 3>(), METH_FASTCALL, nullptr},
    {"token_logprobs_backward", function<token_logprobs_backward, 9>(), METH_FASTCALL, nullptr},
    {"block_quant", function<block_quant, 4>(), METH_FASTCALL, nullptr},
    {"swiglu_block_quant", function<swiglu_block_quant, 5>(), METH_FASTCALL, nullptr},
    {"swiglu_block_backward", function<swiglu_block_backward, 3>(), METH_FASTCALL, nullptr},
    {"block_scaled_mm", function<block_scaled_mm, 7>(), METH_FASTCALL, nullptr},
    {"grouped_block_scaled_mm", function<grouped_block_scaled_mm, 7>(), METH_FASTCALL, nullptr},
    {"block_weight_grad", function<block_weight_grad, 6>(), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_ops", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" __attribute__((visibility("default"))) PyObject *PyInit__ops()
{
    PyObject *api = PyImport_ImportModule("bit_exact_fp8_amd.api");
    if (!api) return nullptr;
    g_emu_error = PyObject_GetAttrString(api, "EmuError");
    Py_DECREF(api);
    return g_emu_error ? PyModule_Create(&g_module) : nullptr;
}
