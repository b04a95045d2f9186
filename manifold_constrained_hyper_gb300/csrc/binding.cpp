// Python binding of the gated residual block, the 8-bit checkpoints and the
// weight gradient (include/mhc.h): argument checks, outputs from torch's
// allocator on the current stream, one call of the C ABI. In C++ because these
// calls are short: at small sizes the same steps in Python take several times
// what the GPU does. Nothing is computed here and nothing is kept between calls.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/core/GradMode.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "mhc.h"

namespace {

// The library's entry points, by address from the loader, and the error to raise.
struct Entries {
    decltype(&mhc_block_norm) norm;
    decltype(&mhc_block_norm_backward) backward;
    decltype(&mhc_block_norm_backward_workspace_bytes) backward_bytes;
    decltype(&mhc_ckpt_pack) pack;
    decltype(&mhc_ckpt_unpack) unpack;
    decltype(&mhc_ckpt_linear_dw) dw;
    decltype(&mhc_ckpt_linear_dw_workspace_bytes) dw_bytes;
    decltype(&mhc_linear) linear;
    decltype(&mhc_linear_workspace_bytes) linear_bytes;
    decltype(&mhc_linear_dx) linear_dx;
    decltype(&mhc_linear_dx_workspace_bytes) linear_dx_bytes;
    decltype(&mhc_linear_dw) linear_dw;
    decltype(&mhc_linear_dw_workspace_bytes) linear_dw_bytes;
    decltype(&mhc_linear_rows_aligned) rows_aligned;
    decltype(&mhc_layer_norm) layer_norm;
    decltype(&mhc_layer_norm_backward) layer_norm_backward;
    decltype(&mhc_layer_norm_backward_workspace_bytes) layer_norm_backward_bytes;
    decltype(&mhc_orthogonalize) orthogonalize;
    decltype(&mhc_orthogonalize_workspace_bytes) orthogonalize_bytes;
} g_lib;
PyObject *g_error = nullptr;
PyObject *g_eps_post, *g_eps_pre, *g_gate_act, *g_weight_offset, *g_post_norm;

// Raised as ValueError.
struct Refused {
    std::string what;
};

std::string str(c10::IntArrayRef s) {
    std::string t = "[";
    for (size_t i = 0; i < s.size(); ++i) t += (i ? ", " : "") + std::to_string(s[i]);
    return t + "]";
}
std::string str(const at::Tensor &t) {
    return str(t.sizes()) + " " + c10::toString(t.scalar_type()) + " on " + t.device().str();
}

// A tensor argument; undefined for None.
at::Tensor tensor(PyObject *o, const char *name, bool optional = false) {
    if (optional && o == Py_None) return at::Tensor();
    if (!THPVariable_Check(o)) throw Refused{std::string(name) + " must be a tensor"};
    return THPVariable_Unpack(o);
}
int dtype_of(at::ScalarType t) {
    return t == at::kFloat ? MHC_F32 : t == at::kBFloat16 ? MHC_BF16 : t == at::kHalf ? MHC_F16 : -1;
}

at::ScalarType scalar_of(long type) { return type == MHC_F32 ? at::kFloat : type == MHC_BF16 ? at::kBFloat16 : at::kHalf; }

struct Shape {
    int64_t T, H;
    c10::Device device{c10::kCPU};
};
Shape shape_2d(const at::Tensor &t, const char *name) {
    if (t.dim() != 2 || !t.is_cuda()) throw Refused{std::string(name) + " must be a 2-D CUDA tensor"};
    return {t.size(0), t.size(1), t.device()};
}
// Rows of `type` whose elements are contiguous: their stride.
int64_t rows(const at::Tensor &t, const char *name, const Shape &s, at::ScalarType type) {
    if (t.dim() != 2 || t.size(0) != s.T || t.size(1) != s.H || t.scalar_type() != type || t.device() != s.device ||
        (s.H > 1 && t.stride(1) != 1))
        throw Refused{std::string(name) + " must be a " + str({s.T, s.H}) + " " + c10::toString(type) + " tensor on " +
                      s.device.str() + " with contiguous rows: got " + str(t)};
    return t.stride(0);
}
// A new tensor, without the dispatcher's part of a torch.empty (a forward call's three: 0.9 us less).
at::Tensor fresh(c10::IntArrayRef size, at::ScalarType type, c10::Device device) {
    return at::Tensor(at::detail::empty_cuda(size, type, device, std::nullopt));
}
// `size` elements of `type` from byte `at` of `t` on, a tensor of its own over the same storage.
at::Tensor part_of(const at::Tensor &t, int64_t at, c10::IntArrayRef size, at::ScalarType type) {
    at::Tensor v = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(t.storage()), t.key_set(),
                                                            c10::scalarTypeToTypeMeta(type));
    v.unsafeGetTensorImpl()->set_storage_offset(at / static_cast<int64_t>(c10::elementSize(type)));
    v.unsafeGetTensorImpl()->set_sizes_contiguous(size);
    return v;
}
// The new tensors of a call, each of an allocation of its own: what is kept of a call holds on to
// nothing else, and what is freed frees nothing else (one for all of a small call's is 1 us of host time
// less forward, 3 backward). Those marked `grouped` are parts of one.
constexpr int64_t kPart = 256;
class NewTensors {
  public:
    explicit NewTensors(c10::Device d) : device_(d) {}
    void add(at::Tensor *to, c10::IntArrayRef size, at::ScalarType type, bool grouped = false) {
        Item &i = items_[count_++];
        i.to = to;
        i.size.assign(size.begin(), size.end());
        i.type = type;
        i.grouped = grouped;
        i.bytes = c10::multiply_integers(size) * static_cast<int64_t>(c10::elementSize(type));
    }
    // `given`, checked, or a new tensor.
    void add_or(at::Tensor *to, const at::Tensor &given, const char *name, c10::IntArrayRef size, at::ScalarType type) {
        if (!given.defined()) return add(to, size, type);
        if (given.sizes() != size || given.scalar_type() != type || given.device() != device_ || !given.is_contiguous())
            throw Refused{std::string(name) + " must be a contiguous " + str(size) + " " + c10::toString(type) +
                          " tensor on " + device_.str() + ": got " + str(given)};
        *to = given;
    }
    void make() {
        int64_t grouped = 0, at = 0;
        for (int i = 0; i < count_; ++i)
            if (items_[i].grouped) grouped += up(items_[i].bytes);
        at::Tensor group;
        if (grouped) group = fresh({grouped}, at::kByte, device_);
        for (int i = 0; i < count_; ++i) {
            Item &n = items_[i];
            // none of a group's bytes: nothing of its own either
            if (!n.grouped || !grouped) {
                *n.to = fresh(n.size, n.type, device_);
                continue;
            }
            *n.to = part_of(group, at, n.size, n.type);
            at += up(n.bytes);
        }
    }

  private:
    static int64_t up(int64_t bytes) { return (bytes + kPart - 1) / kPart * kPart; }
    struct Item {
        at::Tensor *to;
        c10::SmallVector<int64_t, 2> size;
        at::ScalarType type;
        bool grouped;
        int64_t bytes;
    };
    c10::Device device_;
    Item items_[8];
    int count_ = 0;
};

// A checkpoint argument: codes and scales (either None: none).
struct Held {
    at::Tensor codes, scales;
    mhc_ckpt c{nullptr, nullptr};
    const mhc_ckpt *get() const { return codes.defined() ? &c : nullptr; }
};
Held held(PyObject *codes, PyObject *scales, const char *name, const Shape &s) {
    Held h;
    if (codes == Py_None) return h;
    h.codes = tensor(codes, name);
    h.scales = tensor(scales, name);
    const int64_t groups = (s.H + 31) / 32;
    if (h.codes.dim() != 2 || h.codes.size(0) != s.T || h.codes.size(1) != s.H || h.codes.device() != s.device ||
        h.scales.dim() != 2 || h.scales.size(0) != s.T || h.scales.size(1) != groups || h.scales.device() != s.device ||
        h.codes.scalar_type() != at::kByte || h.scales.scalar_type() != at::kByte || !h.codes.is_contiguous() ||
        !h.scales.is_contiguous())
        throw Refused{std::string(name) + " must be a " + str({s.T, s.H}) + " checkpoint on " + s.device.str() + ": got " +
                      str(h.codes)};
    h.c = {h.codes.data_ptr<uint8_t>(), h.scales.data_ptr<uint8_t>()};
    return h;
}

// A workspace argument; undefined for None. Its address goes to the kernels as it is.
at::Tensor scratch(PyObject *o, c10::Device device) {
    at::Tensor t = tensor(o, "workspace", true);
    if (t.defined() && (t.device() != device || !t.is_contiguous()))
        throw Refused{"workspace must be a contiguous tensor on " + device.str() + ": got " + str(t)};
    return t;
}

// Nothing here records a history: outputs of tensors whose gradients are being recorded would end
// them without a word.
void no_history(const at::Tensor &t, const char *name, const char *call) {
    if (t.defined() && t.requires_grad() && c10::GradMode::is_enabled())
        throw Refused{std::string(name) + " requires grad, and " + call + " records no history: call it under "
                      "torch.no_grad(), or both directions in a torch.autograd.Function"};
}

double number(PyObject *o, PyObject *name) {
    PyObject *v = PyObject_GetAttr(o, name);
    const double d = v ? PyFloat_AsDouble(v) : -1.0;
    Py_XDECREF(v);
    if (PyErr_Occurred()) throw std::runtime_error("");
    return d;
}

const void *weight(const at::Tensor &w, const char *name, const Shape &s, mhc_dtype *type) {
    *type = MHC_F32;
    if (!w.defined()) return nullptr;
    const int t = dtype_of(w.scalar_type());
    if (t < 0 || w.dim() != 1 || w.size(0) != s.H || !w.is_contiguous() || w.device() != s.device)
        throw Refused{std::string(name) + " must be a contiguous " + str({s.H}) + " float tensor on " + s.device.str() +
                      ": got " + str(w)};
    *type = static_cast<mhc_dtype>(t);
    return w.data_ptr();
}

// The block's description; what it points into lives in the caller's tensors.
mhc_block block(const Shape &s, at::ScalarType type, at::ScalarType r_type, const at::Tensor &w_post,
                const at::Tensor &w_pre, const at::Tensor &gate, const at::Tensor &res_scale, PyObject *params) {
    mhc_block b = {};
    const int t = dtype_of(type);
    if (t < 0 || (r_type != type && r_type != at::kFloat))
        throw Refused{std::string("y must be float32, bfloat16 or float16 and residual the same or float32: got ") +
                      c10::toString(type) + " and " + c10::toString(r_type)};
    b.tokens = s.T;
    b.hidden = s.H > INT32_MAX ? INT32_MAX : static_cast<int>(s.H);
    b.dtype = static_cast<mhc_dtype>(t);
    b.residual_dtype = static_cast<mhc_dtype>(dtype_of(r_type));
    b.w_post = weight(w_post, "w_post", s, &b.w_post_dtype);
    b.w_pre = weight(w_pre, "w_pre", s, &b.w_pre_dtype);
    PyObject *const act = PyObject_GetAttr(params, g_gate_act);
    const char *const a = act && PyUnicode_Check(act) ? PyUnicode_AsUTF8(act) : "";
    const std::string name = a ? a : "";
    Py_XDECREF(act);
    if (PyErr_Occurred()) throw std::runtime_error("");
    b.gate_act = name == "sigmoid" ? MHC_ACT_SIGMOID : name == "tanh" ? MHC_ACT_TANH : MHC_ACT_NONE;
    if ((b.gate_act == MHC_ACT_NONE && name != "none") || (b.gate_act != MHC_ACT_NONE && !gate.defined()))
        throw Refused{"gate_act must be \"none\", \"sigmoid\" or \"tanh\", and \"none\" without a gate: got \"" + name + "\""};
    if (gate.defined()) {
        const int gt = dtype_of(gate.scalar_type());
        if ((gt != t && gt != MHC_F32) || gate.device() != s.device)
            throw Refused{std::string("gate must be ") + c10::toString(type) + " or float32 on " + s.device.str() + ": got " +
                          str(gate)};
        if (gate.dim() == 1 && gate.size(0) == s.H && (gate.is_contiguous() || s.H == 1)) {
            b.gate_form = MHC_GATE_CHANNEL;
        } else if (gate.dim() == 2 && gate.size(0) == s.T && gate.size(1) == 1) {
            b.gate_form = MHC_GATE_TOKEN;
            b.gate_stride = gate.stride(0);
        } else if (gate.dim() == 2 && gate.size(0) == s.T && gate.size(1) == s.H && gate.stride(1) == 1) {
            b.gate_form = MHC_GATE_FULL;
            b.gate_stride = gate.stride(0);
        } else {
            throw Refused{"gate must be " + str({s.H}) + ", " + str({s.T, 1}) + " or " + str({s.T, s.H}) +
                          " with contiguous rows: got " + str(gate)};
        }
        b.gate = gate.data_ptr();
        b.gate_dtype = static_cast<mhc_dtype>(gt);
    }
    if (res_scale.defined()) {
        const int64_t n = res_scale.numel();
        if (res_scale.scalar_type() != at::kFloat || res_scale.dim() > 1 || (n != 1 && n != s.H) ||
            !res_scale.is_contiguous() || res_scale.device() != s.device)
            throw Refused{"res_scale must be a contiguous [1] or " + str({s.H}) + " float32 tensor on " + s.device.str() +
                          ": got " + str(res_scale)};
        b.scale_form = n == 1 ? MHC_SCALE_ONE : MHC_SCALE_CHANNEL;
        b.res_scale = static_cast<const float *>(res_scale.data_ptr());
    }
    b.eps_post = static_cast<float>(number(params, g_eps_post));
    b.eps_pre = static_cast<float>(number(params, g_eps_pre));
    b.weight_offset = static_cast<float>(number(params, g_weight_offset));
    PyObject *const post = PyObject_GetAttr(params, g_post_norm);
    b.post_norm = post ? PyObject_IsTrue(post) : -1;
    Py_XDECREF(post);
    if (b.post_norm < 0) throw std::runtime_error("");
    return b;
}

void *stream_on(c10::Device d) { return c10::cuda::getCurrentCUDAStream(d.index()).stream(); }
void *ptr(const at::Tensor &t) { return t.defined() ? t.data_ptr() : nullptr; }

void check(mhc_status s, const char *where) {
    if (s == MHC_OK) return;
    PyObject *const e = PyObject_CallFunction(g_error, "is", static_cast<int>(s), where);
    if (e) {
        PyErr_SetObject(g_error, e);
        Py_DECREF(e);
    }
    throw std::runtime_error("");
}

// A checkpoint's two tensors, of one allocation.
void empty_ckpt(const Shape &s, at::Tensor *codes, at::Tensor *scales) {
    const int64_t groups = (s.H + 31) / 32, first = (s.T * s.H + 15) / 16 * 16;
    const at::Tensor all = fresh({first + s.T * groups}, at::kByte, s.device);
    *codes = part_of(all, 0, {s.T, s.H}, at::kByte);
    *scales = part_of(all, first, {s.T, groups}, at::kByte);
}
PyObject *wrap(const at::Tensor &t) {
    if (t.defined()) return THPVariable_Wrap(t);
    Py_RETURN_NONE;
}
PyObject *tuple(std::initializer_list<at::Tensor> ts) {
    PyObject *const r = PyTuple_New(static_cast<Py_ssize_t>(ts.size()));
    Py_ssize_t i = 0;
    for (const at::Tensor &t : ts) {
        PyObject *const o = r ? wrap(t) : nullptr;
        if (!o) {
            Py_XDECREF(r);
            return nullptr;
        }
        PyTuple_SET_ITEM(r, i++, o);
    }
    return r;
}

// Runs an entry point's body; no C++ exception passes into Python. torch's own become what torch raises
// (an allocation that fails: torch.OutOfMemoryError).
template <class F>
PyObject *guarded(Py_ssize_t n, Py_ssize_t want, F body) {
    if (n != want) {
        PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, n);
        return nullptr;
    }
    try {
        return body();
    } catch (const Refused &e) {
        PyErr_SetString(PyExc_ValueError, e.what.c_str());
    } catch (...) {
        if (!PyErr_Occurred()) torch::translate_exception_to_python(std::current_exception());
    }
    return nullptr;
}

// y, residual, w_post, w_pre, gate, res_scale, params, residual_out, h, rstd,
// format, then codes and scales of the checkpoints of y, residual and h
PyObject *block_norm(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 17, [&]() -> PyObject * {
        const at::Tensor y = tensor(a[0], "y"), residual = tensor(a[1], "residual"), w_post = tensor(a[2], "w_post", true),
                         w_pre = tensor(a[3], "w_pre", true), gate = tensor(a[4], "gate", true),
                         res_scale = tensor(a[5], "res_scale", true);
        no_history(y, "y", "mhc_block_norm");
        no_history(residual, "residual", "mhc_block_norm");
        no_history(w_post, "w_post", "mhc_block_norm");
        no_history(w_pre, "w_pre", "mhc_block_norm");
        no_history(gate, "gate", "mhc_block_norm");
        no_history(res_scale, "res_scale", "mhc_block_norm");
        const Shape s = shape_2d(y, "y");
        const at::ScalarType t = y.scalar_type(), rt = residual.scalar_type();
        const int64_t ys = rows(y, "y", s, t), rs = rows(residual, "residual", s, rt);
        const mhc_block b = block(s, t, rt, w_post, w_pre, gate, res_scale, a[6]);
        const long format = PyLong_AsLong(a[10]);
        const Held cy = held(a[11], a[12], "ckpt_y", s), cr = held(a[13], a[14], "ckpt_residual", s),
                   ch = held(a[15], a[16], "ckpt_h", s);
        const c10::cuda::CUDAGuard guard(s.device);
        at::Tensor ro, h, rstd;
        NewTensors fresh_ones(s.device);
        fresh_ones.add_or(&ro, tensor(a[7], "residual_out", true), "residual_out", {s.T, s.H}, rt);
        fresh_ones.add_or(&h, tensor(a[8], "h", true), "h", {s.T, s.H}, t);
        fresh_ones.add_or(&rstd, tensor(a[9], "rstd", true), "rstd", {s.T, 2}, at::kFloat);
        fresh_ones.make();
        check(g_lib.norm(&b, y.data_ptr(), ys, residual.data_ptr(), rs, ro.data_ptr(), h.data_ptr(),
                         static_cast<float *>(rstd.data_ptr()), static_cast<mhc_ckpt_format>(format), cy.get(), cr.get(),
                         ch.get(), stream_on(s.device)),
              "mhc_block_norm");
        return tuple({ro, h, rstd});
    });
}

// d_residual_out, d_h, y, residual (each tensor or None), rstd, w_post, w_pre, gate,
// res_scale, params, the residual's type as a tensor of it or None, d_y, d_residual,
// workspace, format, then codes and scales of y and residual
PyObject *block_norm_backward(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 19, [&]() -> PyObject * {
        const at::Tensor d_ro = tensor(a[0], "d_residual_out", true), d_h = tensor(a[1], "d_h"), y = tensor(a[2], "y", true),
                         residual = tensor(a[3], "residual", true), rstd = tensor(a[4], "rstd"),
                         w_post = tensor(a[5], "w_post", true), w_pre = tensor(a[6], "w_pre", true),
                         gate = tensor(a[7], "gate", true), res_scale = tensor(a[8], "res_scale", true),
                         typed = tensor(a[10], "residual_dtype", true);
        no_history(d_ro, "d_residual_out", "mhc_block_norm_backward");
        no_history(d_h, "d_h", "mhc_block_norm_backward");
        const Shape s = shape_2d(d_h, "d_h");
        const at::ScalarType t = d_h.scalar_type();
        const at::ScalarType rt = typed.defined() ? typed.scalar_type() : d_ro.defined() ? d_ro.scalar_type()
                                  : residual.defined() ? residual.scalar_type() : t;
        const int64_t dhs = rows(d_h, "d_h", s, t);
        const int64_t drs = d_ro.defined() ? rows(d_ro, "d_residual_out", s, rt) : 0;
        const mhc_block b = block(s, t, rt, w_post, w_pre, gate, res_scale, a[9]);
        const int64_t ys = y.defined() ? rows(y, "y", s, t) : 0;
        const int64_t rs = residual.defined() ? rows(residual, "residual", s, rt) : 0;
        const long format = PyLong_AsLong(a[14]);
        const Held cy = held(a[15], a[16], "y", s), cr = held(a[17], a[18], "residual", s);
        const c10::cuda::CUDAGuard guard(s.device);
        at::Tensor d_y, d_residual, d_w_post, d_w_pre, d_gate, d_scale, workspace = scratch(a[13], s.device), same;
        NewTensors fresh_ones(s.device);
        fresh_ones.add_or(&same, rstd, "rstd", {s.T, 2}, at::kFloat);
        fresh_ones.add_or(&d_y, tensor(a[11], "d_y", true), "d_y", {s.T, s.H}, t);
        fresh_ones.add_or(&d_residual, tensor(a[12], "d_residual", true), "d_residual", {s.T, s.H}, rt);
        const bool full = b.gate_form == MHC_GATE_FULL;
        if (w_post.defined()) fresh_ones.add(&d_w_post, {s.H}, at::kFloat, true);
        if (w_pre.defined()) fresh_ones.add(&d_w_pre, {s.H}, at::kFloat, true);
        if (gate.defined()) fresh_ones.add(&d_gate, gate.sizes(), full ? gate.scalar_type() : at::kFloat, !full);
        if (res_scale.defined()) fresh_ones.add(&d_scale, res_scale.sizes(), at::kFloat, true);
        if (!workspace.defined()) {
            const size_t need = g_lib.backward_bytes(s.T, b.hidden);
            fresh_ones.add(&workspace, {static_cast<int64_t>(need < 16 ? 16 : need)}, at::kByte);
        }
        fresh_ones.make();
        check(g_lib.backward(&b, ptr(d_ro), drs, d_h.data_ptr(), dhs, ptr(y), ys, ptr(residual), rs,
                             static_cast<mhc_ckpt_format>(format), cy.get(), cr.get(),
                             static_cast<const float *>(rstd.data_ptr()), d_y.data_ptr(), d_residual.data_ptr(),
                             static_cast<float *>(ptr(d_w_post)), static_cast<float *>(ptr(d_w_pre)), ptr(d_gate),
                             static_cast<float *>(ptr(d_scale)), workspace.data_ptr(), workspace.nbytes(),
                             stream_on(s.device)),
              "mhc_block_norm_backward");
        return tuple({d_y, d_residual, d_w_post, d_w_pre, d_gate, d_scale});
    });
}

// tokens, hidden, the device's number (-1: the current one) -> codes, scales
PyObject *ckpt_empty(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 3, [&]() -> PyObject * {
        const int64_t T = PyLong_AsLongLong(a[0]), H = PyLong_AsLongLong(a[1]);
        const long device = PyLong_AsLong(a[2]);
        if (PyErr_Occurred()) throw std::runtime_error("");
        if (T < 0 || H < 0) throw Refused{"a checkpoint's sizes must not be negative: got " + str({T, H})};
        at::Tensor codes, scales;
        empty_ckpt({T, H, c10::Device(c10::kCUDA, device < 0 ? c10::cuda::current_device() : static_cast<int8_t>(device))},
                   &codes, &scales);
        return tuple({codes, scales});
    });
}

// x, format, codes, scales (None: new) -> codes, scales
PyObject *ckpt_pack(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 4, [&]() -> PyObject * {
        const at::Tensor x = tensor(a[0], "x");
        const Shape s = shape_2d(x, "x");
        const int t = dtype_of(x.scalar_type());
        if (t < 0) throw Refused{std::string("x must be float32, bfloat16 or float16: got ") + c10::toString(x.scalar_type())};
        const int64_t stride = rows(x, "x", s, x.scalar_type());
        const long format = PyLong_AsLong(a[1]);
        const c10::cuda::CUDAGuard guard(s.device);
        Held out = held(a[2], a[3], "out", s);
        if (!out.codes.defined()) {
            empty_ckpt(s, &out.codes, &out.scales);
            out.c = {static_cast<uint8_t *>(out.codes.data_ptr()), static_cast<uint8_t *>(out.scales.data_ptr())};
        }
        check(g_lib.pack(x.data_ptr(), stride, static_cast<mhc_dtype>(t), s.T,
                         s.H > INT32_MAX ? INT32_MAX : static_cast<int>(s.H), static_cast<mhc_ckpt_format>(format), &out.c,
                         stream_on(s.device)),
              "mhc_ckpt_pack");
        return tuple({out.codes, out.scales});
    });
}

// codes, scales, format, the type (a number of mhc_dtype), out -> x
PyObject *ckpt_unpack(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 5, [&]() -> PyObject * {
        const at::Tensor codes = tensor(a[0], "codes");
        const Shape s = shape_2d(codes, "codes");
        const Held c = held(a[0], a[1], "ckpt", s);
        const long format = PyLong_AsLong(a[2]), type = PyLong_AsLong(a[3]);
        const c10::cuda::CUDAGuard guard(s.device);
        at::Tensor out;
        NewTensors fresh_ones(s.device);
        fresh_ones.add_or(&out, tensor(a[4], "out", true), "out", {s.T, s.H}, scalar_of(type));
        fresh_ones.make();
        check(g_lib.unpack(&c.c, static_cast<mhc_ckpt_format>(format), s.T,
                           s.H > INT32_MAX ? INT32_MAX : static_cast<int>(s.H), static_cast<mhc_dtype>(type), out.data_ptr(),
                           stream_on(s.device)),
              "mhc_ckpt_unpack");
        return wrap(out);
    });
}

// d_out, codes, scales, format, d_w, its type (a number of mhc_dtype), accumulate, workspace -> d_w
PyObject *ckpt_linear_dw(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 8, [&]() -> PyObject * {
        const at::Tensor d_out = tensor(a[0], "d_out"), codes = tensor(a[1], "x");
        no_history(d_out, "d_out", "mhc_ckpt_linear_dw");
        const Shape s = shape_2d(d_out, "d_out");
        const at::ScalarType t = d_out.scalar_type();
        if (t != at::kBFloat16 && t != at::kHalf)
            throw Refused{std::string("d_out must be bfloat16 or float16: got ") + c10::toString(t)};
        const int64_t stride = rows(d_out, "d_out", s, t);
        if (codes.dim() != 2) throw Refused{"x must be a checkpoint"};
        const int64_t K = codes.size(1);
        const Held x = held(a[1], a[2], "x", {s.T, K, s.device});
        const long format = PyLong_AsLong(a[3]), type = PyLong_AsLong(a[5]);
        const c10::cuda::CUDAGuard guard(s.device);
        const int N = s.H > INT32_MAX ? INT32_MAX : static_cast<int>(s.H), k = K > INT32_MAX ? INT32_MAX : static_cast<int>(K);
        at::Tensor d_w, workspace = scratch(a[7], s.device);
        NewTensors fresh_ones(s.device);
        fresh_ones.add_or(&d_w, tensor(a[4], "d_w", true), "d_w", {s.H, K}, scalar_of(type));
        if (!workspace.defined()) {
            const bool aligned = reinterpret_cast<uintptr_t>(d_out.data_ptr()) % 16 == 0 &&
                                 (s.T == 1 || (stride % 8 == 0 && stride >= s.H && stride < (int64_t(1) << 38)));
            const size_t need = g_lib.dw_bytes(s.T, N, k, aligned);
            if (need) fresh_ones.add(&workspace, {static_cast<int64_t>(need)}, at::kByte);
        }
        fresh_ones.make();
        check(g_lib.dw(d_out.data_ptr(), stride, static_cast<mhc_dtype>(dtype_of(t)), &x.c,
                       static_cast<mhc_ckpt_format>(format), s.T, N, k, d_w.data_ptr(), static_cast<mhc_dtype>(type),
                       PyObject_IsTrue(a[6]) == 1, ptr(workspace), workspace.defined() ? workspace.nbytes() : 0,
                       stream_on(s.device)),
              "mhc_ckpt_linear_dw");
        return wrap(d_w);
    });
}

// A matrix of 16-bit rows as a product reads it.
struct Rows {
    at::Tensor t;
    int64_t rows, stride;
    int width;
    bool aligned;
};
int width_of(int64_t w) { return w > INT32_MAX ? INT32_MAX : static_cast<int>(w); }
Rows product_rows(const at::Tensor &t, const char *name, const Shape &s, at::ScalarType type) {
    Rows r{t, s.T, rows(t, name, s, type), width_of(s.H), false};
    r.aligned = g_lib.rows_aligned(t.data_ptr(), r.stride, s.T, r.width) != 0;
    return r;
}
at::ScalarType half_type(const at::Tensor &t, const char *name) {
    const at::ScalarType s = t.scalar_type();
    if (s != at::kBFloat16 && s != at::kHalf)
        throw Refused{std::string(name) + " must be bfloat16 or float16: got " + c10::toString(s)};
    return s;
}
// A parameter [H], contiguous, of float32 or one other type (any: of the three).
void parameter(const at::Tensor &t, const char *name, int64_t H, c10::Device device, at::ScalarType other, bool any) {
    if (!t.defined()) return;
    const at::ScalarType s = t.scalar_type();
    if (t.dim() != 1 || t.size(0) != H || t.device() != device || !t.is_contiguous() ||
        !(any ? dtype_of(s) >= 0 : s == at::kFloat || s == other))
        throw Refused{std::string(name) + " must be a contiguous " + str({H}) + " tensor of " +
                      (any ? "float32, bfloat16 or float16" : std::string("float32 or ") + c10::toString(other)) + " on " +
                      device.str() + ": got " + str(t)};
}
void workspace_or(at::Tensor *workspace, size_t need, NewTensors *made) {
    if (!workspace->defined() && need) made->add(workspace, {static_cast<int64_t>(need)}, at::kByte);
}
mhc_dtype mhc_type(at::ScalarType t) { return static_cast<mhc_dtype>(dtype_of(t)); }

// x, w, bias, residual, act, out, z, whether z is wanted, out's type (-1: the residual's, else x's), workspace -> out, z
PyObject *linear(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 10, [&]() -> PyObject * {
        const at::Tensor x = tensor(a[0], "x"), w = tensor(a[1], "w"), bias = tensor(a[2], "bias", true),
                         residual = tensor(a[3], "residual", true);
        for (auto [t, name] : {std::pair{&x, "x"}, {&w, "w"}, {&bias, "bias"}, {&residual, "residual"}})
            no_history(*t, name, "mhc_linear");
        const Shape s = shape_2d(x, "x"), ws = shape_2d(w, "w");
        const at::ScalarType t = half_type(x, "x");
        const Rows xr = product_rows(x, "x", s, t), wr = product_rows(w, "w", {ws.T, s.H, s.device}, t);
        const int64_t N = ws.T;
        parameter(bias, "bias", N, s.device, t, false);
        const long act = PyLong_AsLong(a[4]), type = PyLong_AsLong(a[8]);
        at::Tensor out = tensor(a[5], "out", true), z = tensor(a[6], "z", true);
        const at::ScalarType o = out.defined() ? out.scalar_type() : type >= 0 ? scalar_of(type) : residual.defined() ? residual.scalar_type() : t;
        if (o != t && o != at::kFloat) throw Refused{std::string("out must be float32 or of x's type: got ") + c10::toString(o)};
        const Shape os{s.T, N, s.device};
        const int64_t rstride = residual.defined() ? rows(residual, "residual", os, o) : 0;
        const c10::cuda::CUDAGuard guard(s.device);
        at::Tensor workspace = scratch(a[9], s.device), out_, z_;
        NewTensors made(s.device);
        made.add_or(&out_, out, "out", {s.T, N}, o);
        if (z.defined() || PyObject_IsTrue(a[7]) == 1) made.add_or(&z_, z, "z", {s.T, N}, t);
        workspace_or(&workspace, g_lib.linear_bytes(s.T, width_of(N), xr.width, xr.aligned, wr.aligned), &made);
        made.make();
        check(g_lib.linear(x.data_ptr(), xr.stride, w.data_ptr(), wr.stride, mhc_type(t), s.T, width_of(N), xr.width, ptr(bias),
                           bias.defined() ? mhc_type(bias.scalar_type()) : MHC_F32, ptr(residual), rstride,
                           static_cast<mhc_linear_act>(act), out_.data_ptr(), mhc_type(o), ptr(z_), ptr(workspace),
                           workspace.defined() ? workspace.nbytes() : 0, stream_on(s.device)),
              "mhc_linear");
        return z_.defined() ? tuple({out_, z_}) : wrap(out_);
    });
}

// d_out, w, z, act, d_x, its type (-1: d_out's), workspace -> d_x
PyObject *linear_dx(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 7, [&]() -> PyObject * {
        const at::Tensor d_out = tensor(a[0], "d_out"), w = tensor(a[1], "w"), z = tensor(a[2], "z", true);
        for (auto [t, name] : {std::pair{&d_out, "d_out"}, {&w, "w"}, {&z, "z"}}) no_history(*t, name, "mhc_linear_dx");
        const Shape s = shape_2d(d_out, "d_out"), ws = shape_2d(w, "w");
        const at::ScalarType t = half_type(d_out, "d_out");
        const Rows dr = product_rows(d_out, "d_out", s, t), wr = product_rows(w, "w", {s.H, ws.H, s.device}, t);
        const int64_t K = ws.H;
        const long act = PyLong_AsLong(a[3]), type = PyLong_AsLong(a[5]);
        if (act != MHC_LINEAR_NONE && !z.defined()) throw Refused{"z is needed for the slope of the activation"};
        if (act == MHC_LINEAR_NONE && z.defined()) throw Refused{"z has no use without an activation"};
        const int64_t zstride = z.defined() ? rows(z, "z", {s.T, K, s.device}, t) : 0;
        at::Tensor given = tensor(a[4], "d_x", true), d_x, workspace = scratch(a[6], s.device);
        const at::ScalarType o = given.defined() ? given.scalar_type() : type >= 0 ? scalar_of(type) : t;
        if (o != t && o != at::kFloat) throw Refused{std::string("d_x must be float32 or of d_out's type: got ") + c10::toString(o)};
        const c10::cuda::CUDAGuard guard(s.device);
        NewTensors made(s.device);
        made.add_or(&d_x, given, "d_x", {s.T, K}, o);
        workspace_or(&workspace, g_lib.linear_dx_bytes(s.T, dr.width, width_of(K), dr.aligned, wr.aligned), &made);
        made.make();
        check(g_lib.linear_dx(d_out.data_ptr(), dr.stride, w.data_ptr(), wr.stride, mhc_type(t), s.T, dr.width, width_of(K), ptr(z),
                              zstride, static_cast<mhc_linear_act>(act), d_x.data_ptr(), mhc_type(o), ptr(workspace),
                              workspace.defined() ? workspace.nbytes() : 0, stream_on(s.device)),
              "mhc_linear_dx");
        return wrap(d_x);
    });
}

// d_out, x, d_w, its type, whether the bias's is wanted, d_bias, accumulate, workspace -> d_w, d_bias
PyObject *linear_dw(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 8, [&]() -> PyObject * {
        const at::Tensor d_out = tensor(a[0], "d_out"), x = tensor(a[1], "x");
        for (auto [t, name] : {std::pair{&d_out, "d_out"}, {&x, "x"}}) no_history(*t, name, "mhc_linear_dw");
        const Shape s = shape_2d(d_out, "d_out"), xs = shape_2d(x, "x");
        const at::ScalarType t = half_type(d_out, "d_out");
        const Rows dr = product_rows(d_out, "d_out", s, t), xr = product_rows(x, "x", {s.T, xs.H, s.device}, t);
        const int64_t K = xs.H;
        const long type = PyLong_AsLong(a[3]);
        const at::Tensor bias = tensor(a[5], "d_bias", true);
        at::Tensor d_w, d_bias, workspace = scratch(a[7], s.device);
        const c10::cuda::CUDAGuard guard(s.device);
        NewTensors made(s.device);
        made.add_or(&d_w, tensor(a[2], "d_w", true), "d_w", {s.H, K}, scalar_of(type));
        if (bias.defined() || PyObject_IsTrue(a[4]) == 1) made.add_or(&d_bias, bias, "d_bias", {s.H}, at::kFloat);
        const bool with_bias = bias.defined() || PyObject_IsTrue(a[4]) == 1;
        workspace_or(&workspace, g_lib.linear_dw_bytes(s.T, dr.width, width_of(K), dr.aligned, xr.aligned), &made);
        made.make();
        check(g_lib.linear_dw(d_out.data_ptr(), dr.stride, x.data_ptr(), xr.stride, mhc_type(t), s.T, dr.width, width_of(K),
                              d_w.data_ptr(), static_cast<mhc_dtype>(type), static_cast<float *>(ptr(d_bias)),
                              PyObject_IsTrue(a[6]) == 1, ptr(workspace), workspace.defined() ? workspace.nbytes() : 0,
                              stream_on(s.device)),
              "mhc_linear_dw");
        return with_bias ? tuple({d_w, d_bias}) : wrap(d_w);
    });
}

// out's type beside x's
void norm_type(at::ScalarType x, at::ScalarType out, const char *name) {
    if (dtype_of(x) < 0) throw Refused{std::string("x must be float32, bfloat16 or float16: got ") + c10::toString(x)};
    if (dtype_of(out) < 0 || (out != x && x != at::kFloat))
        throw Refused{std::string(name) + " must be of x's type, or of 16 bits beside a float32 x: got " + c10::toString(out)};
}

// x, w, b, eps, out, stats, out's type (-1: x's) -> out, stats
PyObject *layer_norm(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 7, [&]() -> PyObject * {
        const at::Tensor x = tensor(a[0], "x"), w = tensor(a[1], "w", true), b = tensor(a[2], "b", true);
        for (auto [t, name] : {std::pair{&x, "x"}, {&w, "w"}, {&b, "b"}}) no_history(*t, name, "mhc_layer_norm");
        const Shape s = shape_2d(x, "x");
        const at::ScalarType t = x.scalar_type();
        const long type = PyLong_AsLong(a[6]);
        const double eps = PyFloat_AsDouble(a[3]);
        if (PyErr_Occurred()) throw std::runtime_error("");
        const at::Tensor given = tensor(a[4], "out", true);
        const at::ScalarType o = given.defined() ? given.scalar_type() : type >= 0 ? scalar_of(type) : t;
        norm_type(t, o, "out");
        const int64_t stride = rows(x, "x", s, t);
        parameter(w, "w", s.H, s.device, t, true);
        parameter(b, "b", s.H, s.device, t, true);
        const c10::cuda::CUDAGuard guard(s.device);
        at::Tensor out, stats;
        NewTensors made(s.device);
        made.add_or(&out, given, "out", {s.T, s.H}, o);
        made.add_or(&stats, tensor(a[5], "stats", true), "stats", {s.T, 2}, at::kFloat);
        made.make();
        check(g_lib.layer_norm(x.data_ptr(), stride, mhc_type(t), s.T, width_of(s.H), ptr(w),
                               w.defined() ? mhc_type(w.scalar_type()) : MHC_F32, ptr(b),
                               b.defined() ? mhc_type(b.scalar_type()) : MHC_F32, static_cast<float>(eps), out.data_ptr(),
                               mhc_type(o), static_cast<float *>(stats.data_ptr()), stream_on(s.device)),
              "mhc_layer_norm");
        return tuple({out, stats});
    });
}

// d_out, x, stats, w, whether the bias's is wanted, d_residual, d_x, workspace -> d_x, d_w, d_b
PyObject *layer_norm_backward(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 8, [&]() -> PyObject * {
        const at::Tensor d_out = tensor(a[0], "d_out"), x = tensor(a[1], "x"), stats = tensor(a[2], "stats"),
                         w = tensor(a[3], "w", true), d_residual = tensor(a[5], "d_residual", true);
        for (auto [t, name] : {std::pair{&d_out, "d_out"}, {&x, "x"}, {&stats, "stats"}, {&w, "w"}, {&d_residual, "d_residual"}})
            no_history(*t, name, "mhc_layer_norm_backward");
        const Shape s = shape_2d(x, "x");
        const at::ScalarType t = x.scalar_type(), o = d_out.scalar_type();
        norm_type(t, o, "d_out");
        const int64_t xstride = rows(x, "x", s, t), dstride = rows(d_out, "d_out", s, o),
                      rstride = d_residual.defined() ? rows(d_residual, "d_residual", s, t) : 0;
        if (stats.dim() != 2 || stats.size(0) != s.T || stats.size(1) != 2 || stats.scalar_type() != at::kFloat ||
            stats.device() != s.device || !stats.is_contiguous())
            throw Refused{"stats must be a contiguous " + str({s.T, 2}) + " float32 tensor on " + s.device.str() + ": got " + str(stats)};
        parameter(w, "w", s.H, s.device, t, true);
        const bool bias = PyObject_IsTrue(a[4]) == 1;
        const c10::cuda::CUDAGuard guard(s.device);
        at::Tensor d_x, d_w, d_b, workspace = scratch(a[7], s.device);
        NewTensors made(s.device);
        made.add_or(&d_x, tensor(a[6], "d_x", true), "d_x", {s.T, s.H}, t);
        if (w.defined()) made.add(&d_w, {s.H}, at::kFloat, true);
        if (bias) made.add(&d_b, {s.H}, at::kFloat, true);
        if (w.defined() || bias) workspace_or(&workspace, g_lib.layer_norm_backward_bytes(s.T, width_of(s.H)), &made);
        made.make();
        check(g_lib.layer_norm_backward(d_out.data_ptr(), dstride, mhc_type(o), x.data_ptr(), xstride, mhc_type(t),
                                        static_cast<const float *>(stats.data_ptr()), s.T, width_of(s.H), ptr(w),
                                        w.defined() ? mhc_type(w.scalar_type()) : MHC_F32, ptr(d_residual), rstride,
                                        d_x.data_ptr(), static_cast<float *>(ptr(d_w)), static_cast<float *>(ptr(d_b)),
                                        ptr(workspace), workspace.defined() ? workspace.nbytes() : 0, stream_on(s.device)),
              "mhc_layer_norm_backward");
        return tuple({d_x, d_w, d_b});
    });
}

// g, steps, a, b, c, eps, out, its type, workspace -> out
PyObject *orthogonalize(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 9, [&]() -> PyObject * {
        const at::Tensor g = tensor(a[0], "g");
        no_history(g, "g", "mhc_orthogonalize");
        const int64_t dims = g.dim();
        if ((dims != 2 && dims != 3) || !g.is_cuda()) throw Refused{"g must be a 2-D or 3-D CUDA tensor"};
        const at::ScalarType t = g.scalar_type();
        if (dtype_of(t) < 0) throw Refused{std::string("g must be float32, bfloat16 or float16: got ") + c10::toString(t)};
        const int64_t B = dims == 3 ? g.size(0) : 1, M = g.size(dims - 2), N = g.size(dims - 1);
        if (N > 1 && g.stride(dims - 1) != 1) throw Refused{"g's rows must be contiguous: got strides " + str(g.strides())};
        const long steps = PyLong_AsLong(a[1]), type = PyLong_AsLong(a[7]);
        const double ca = PyFloat_AsDouble(a[2]), cb = PyFloat_AsDouble(a[3]), cc = PyFloat_AsDouble(a[4]), eps = PyFloat_AsDouble(a[5]);
        if (PyErr_Occurred()) throw std::runtime_error("");
        if (type != MHC_BF16 && type != MHC_F16) throw Refused{"out must be bfloat16 or float16"};
        const c10::cuda::CUDAGuard guard(g.device());
        at::Tensor out, workspace = scratch(a[8], g.device());
        NewTensors made(g.device());
        made.add_or(&out, tensor(a[6], "out", true), "out", g.sizes(), scalar_of(type));
        const int batch = width_of(B), m = width_of(M), k = width_of(N);
        workspace_or(&workspace, g_lib.orthogonalize_bytes(batch, m, k), &made);
        made.make();
        check(g_lib.orthogonalize(g.data_ptr(), g.stride(dims - 2), dims == 3 ? g.stride(0) : 0, mhc_type(t), batch, m, k,
                                  steps > INT32_MAX ? INT32_MAX : steps < 0 ? -1 : static_cast<int>(steps), static_cast<float>(ca),
                                  static_cast<float>(cb), static_cast<float>(cc), static_cast<float>(eps), out.data_ptr(),
                                  static_cast<mhc_dtype>(type), ptr(workspace), workspace.defined() ? workspace.nbytes() : 0,
                                  stream_on(g.device())),
              "mhc_orthogonalize");
        return wrap(out);
    });
}

// The entry points' addresses, in the order of Entries, and the error class.
PyObject *init(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 20, [&]() -> PyObject * {
        constexpr int kEntries = 19;
        void *p[kEntries];
        for (int i = 0; i < kEntries; ++i) {
            p[i] = PyLong_AsVoidPtr(a[i]);
            if (!p[i]) throw std::runtime_error("an entry point is missing");
        }
        g_lib = {reinterpret_cast<decltype(g_lib.norm)>(p[0]), reinterpret_cast<decltype(g_lib.backward)>(p[1]),
                 reinterpret_cast<decltype(g_lib.backward_bytes)>(p[2]), reinterpret_cast<decltype(g_lib.pack)>(p[3]),
                 reinterpret_cast<decltype(g_lib.unpack)>(p[4]), reinterpret_cast<decltype(g_lib.dw)>(p[5]),
                 reinterpret_cast<decltype(g_lib.dw_bytes)>(p[6]), reinterpret_cast<decltype(g_lib.linear)>(p[7]),
                 reinterpret_cast<decltype(g_lib.linear_bytes)>(p[8]), reinterpret_cast<decltype(g_lib.linear_dx)>(p[9]),
                 reinterpret_cast<decltype(g_lib.linear_dx_bytes)>(p[10]), reinterpret_cast<decltype(g_lib.linear_dw)>(p[11]),
                 reinterpret_cast<decltype(g_lib.linear_dw_bytes)>(p[12]), reinterpret_cast<decltype(g_lib.rows_aligned)>(p[13]),
                 reinterpret_cast<decltype(g_lib.layer_norm)>(p[14]),
                 reinterpret_cast<decltype(g_lib.layer_norm_backward)>(p[15]),
                 reinterpret_cast<decltype(g_lib.layer_norm_backward_bytes)>(p[16]),
                 reinterpret_cast<decltype(g_lib.orthogonalize)>(p[17]),
                 reinterpret_cast<decltype(g_lib.orthogonalize_bytes)>(p[18])};
        Py_INCREF(a[kEntries]);
        Py_XDECREF(g_error);
        g_error = a[kEntries];
        Py_RETURN_NONE;
    });
}

#define MHC_METHOD(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(f)), METH_FASTCALL, nullptr}
PyMethodDef g_methods[] = {MHC_METHOD(init),          MHC_METHOD(block_norm),  MHC_METHOD(block_norm_backward),
                           MHC_METHOD(ckpt_empty),    MHC_METHOD(ckpt_pack),     MHC_METHOD(ckpt_unpack), MHC_METHOD(ckpt_linear_dw),
                           MHC_METHOD(linear),        MHC_METHOD(linear_dx),     MHC_METHOD(linear_dw),   MHC_METHOD(layer_norm),
                           MHC_METHOD(layer_norm_backward), MHC_METHOD(orthogonalize),
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() {
    g_eps_post = PyUnicode_InternFromString("eps_post");
    g_eps_pre = PyUnicode_InternFromString("eps_pre");
    g_gate_act = PyUnicode_InternFromString("gate_act");
    g_weight_offset = PyUnicode_InternFromString("weight_offset");
    g_post_norm = PyUnicode_InternFromString("post_norm");
    return PyModule_Create(&g_module);
}
