// Python binding of the row-wise operators (dispatch, combine, SwiGLU, norms): a CPython module that checks torch tensors and
// calls the C entry points of include/dg.h.  These calls last a few microseconds on the GPU, about as long as the checks of
// their arguments take in Python; here a tensor is checked in about 50 ns.  It holds no arithmetic and no state but the error
// class it is given.  The entry points themselves run without the interpreter's lock.
#include <torch/csrc/autograd/python_variable.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>

#include <cstdarg>
#include <initializer_list>
#include <string>

#include "dg.h"

namespace {

PyObject *g_error_class = nullptr;  // DGError(status, message)

struct Refused {
    int status;
    std::string message;
};

[[noreturn]] void refuse(const char *fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof(buf), fmt, ap);
    va_end(ap);
    throw Refused{DG_ERR_INVALID_ARG, buf};
}

using Shape = c10::IntArrayRef;
using c10::ScalarType;

enum Kind { BF16, F32, ACT, I32, ID, FP8 };  // what an element type may be

bool is_kind(ScalarType t, Kind k) {
    switch (k) {
        case BF16: return t == ScalarType::BFloat16;
        case F32: return t == ScalarType::Float;
        case ACT: return t == ScalarType::BFloat16 || t == ScalarType::Float;
        case I32: return t == ScalarType::Int;
        case ID: return t == ScalarType::Int || t == ScalarType::Long;
        default: return t == ScalarType::Byte || t == ScalarType::Float8_e4m3fn;
    }
}

const char *kind_name(Kind k) {
    switch (k) {
        case BF16: return "torch.bfloat16";
        case F32: return "torch.float32";
        case ACT: return "torch.bfloat16 or torch.float32";
        case I32: return "torch.int32";
        case ID: return "torch.int32 or torch.int64";
        default: return "torch.float8_e4m3fn or torch.uint8";
    }
}

std::string text(Shape s) {
    std::string r = "[";
    for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
    return r + "]";
}

// One call's arguments: the tensors have to be on the current device, on whose current stream the call runs.
struct Call {
    PyObject *const *args;

    static int device() { return static_cast<int>(c10::cuda::current_device()); }

    const at::Tensor &tensor(int i, const char *name) const {
        if (!THPVariable_Check(args[i])) refuse("%s must be a torch.Tensor", name);
        return THPVariable_Unpack(args[i]);
    }
    const at::Tensor *optional(int i, const char *name) const {
        return args[i] == Py_None ? nullptr : &tensor(i, name);
    }
    const at::Tensor &dims(int i, const char *name, int least, int most) const {
        const at::Tensor &t = tensor(i, name);
        if (t.dim() < least || t.dim() > most)
            refuse(least == most ? "%s must have %d dims, got %s" : "%s must have %d or more dims, got %s", name, least,
                   text(t.sizes()).c_str());
        for (int64_t n : t.sizes())
            if (n > 0x7fffffff) refuse("%s has an extent of %lld, past 2^31", name, static_cast<long long>(n));
        return t;
    }
    void check(const at::Tensor &t, const char *name, Shape shape, Kind kind) const {
        if (!is_kind(t.scalar_type(), kind))
            refuse("%s has dtype %s, expected %s", name, c10::toString(t.scalar_type()), kind_name(kind));
        if (t.sizes() != shape) refuse("%s must be %s, got %s", name, text(shape).c_str(), text(t.sizes()).c_str());
        if (!t.is_contiguous()) refuse("%s must be contiguous", name);
        if (!t.is_cuda()) refuse("%s must be a CUDA tensor", name);
        if (t.get_device() != device())
            refuse("%s is on device %d, the current one is %d", name, static_cast<int>(t.get_device()), device());
    }
    void check(const at::Tensor *t, const char *name, Shape shape, Kind kind) const {
        if (t) check(*t, name, shape, kind);
    }
    dg_stream_t stream() const {
        return reinterpret_cast<dg_stream_t>(c10::cuda::getCurrentCUDAStream().stream());
    }
};

int code(const at::Tensor &t) { return t.scalar_type() == ScalarType::Float ? DG_F32 : DG_BF16; }
Kind same_as(const at::Tensor &t) { return t.scalar_type() == ScalarType::Float ? F32 : BF16; }
int size(const at::Tensor &t, int d) { return static_cast<int>(t.size(d)); }

template <typename T = void> T *ptr(const at::Tensor &t) { return static_cast<T *>(t.data_ptr()); }
template <typename T = void> T *ptr(const at::Tensor *t) { return t ? static_cast<T *>(t->data_ptr()) : nullptr; }

// The C call, its arguments already made, without the interpreter's lock: a launch waits where the queue of launches is full, and
// what drains the queue may be a callback that needs the lock.  (The caller holds its tensors until the call returns.)
template <typename F, typename... Args> int without_lock(F f, Args... args) {
    PyThreadState *state = PyEval_SaveThread();
    const int status = f(args...);
    PyEval_RestoreThread(state);
    return status;
}

// [rows, cols] or [G, M_max, cols]: a tensor of `kind`, or a pair (e4m3 codes, scales) as a GEMM's lhs.
struct RowOperand {
    const at::Tensor *a = nullptr, *sf = nullptr;
    int rows = 0, rows_per_group = 0;
};

RowOperand row_operand(const Call &c, int i, const char *name, int64_t cols, Kind kind) {
    RowOperand r;
    PyObject *o = c.args[i], *codes = o, *scales = nullptr;
    if (PyTuple_Check(o) || PyList_Check(o)) {
        if (PySequence_Fast_GET_SIZE(o) != 2) refuse("%s must be a tensor or a pair (codes, scales)", name);
        codes = PySequence_Fast_GET_ITEM(o, 0);
        scales = PySequence_Fast_GET_ITEM(o, 1);
        if (!THPVariable_Check(scales)) refuse("%s scales must be a torch.Tensor", name);
    }
    const Call one{&codes};
    r.a = &one.dims(0, name, 2, 3);
    const bool grouped = r.a->dim() == 3;
    const int64_t per = r.a->size(-2), G = grouped ? r.a->size(0) : 1;
    const int64_t shape[3] = {G, per, cols}, sf_shape[3] = {G, cols / 128, (per + 3) / 4 * 4};
    const size_t skip = grouped ? 0 : 1;
    c.check(*r.a, name, Shape(shape + skip, 3 - skip), scales ? FP8 : kind);
    if (scales) {
        r.sf = &THPVariable_Unpack(scales);
        c.check(*r.sf, (std::string(name) + " scales").c_str(), Shape(sf_shape + skip, 3 - skip), F32);
    }
    if (G * per > 0x7fffffff) refuse("%s has more than 2^31 rows", name);
    r.rows = static_cast<int>(G * per);
    r.rows_per_group = static_cast<int>(per);
    return r;
}

struct Sorted {
    const at::Tensor &ids, &rows, &counts;
    int T, k, G;
};

// (topk_ids, row_of_slot, counts)
Sorted sort_args(const Call &c, int rows, int counts) {
    const at::Tensor &ids = c.dims(0, "topk_ids", 2, 2), &n = c.dims(counts, "counts", 1, 1);
    const at::Tensor &r = c.tensor(rows, "row_of_slot");
    c.check(ids, "topk_ids", ids.sizes(), ID);
    c.check(r, "row_of_slot", ids.sizes(), I32);
    c.check(n, "counts", n.sizes(), I32);
    return Sorted{ids, r, n, size(ids, 0), size(ids, 1), size(n, 0)};
}

int id_bytes(const Sorted &s) { return s.ids.scalar_type() == ScalarType::Long ? 8 : 4; }

// (topk_ids, row_of_slot, m_indices, counts)
int sort_contiguous(const Call &c) {
    const Sorted s = sort_args(c, 1, 3);
    const at::Tensor &m = c.dims(2, "m_indices", 1, 1);
    c.check(m, "m_indices", m.sizes(), I32);
    return without_lock(dg_moe_sort_contiguous, ptr(s.ids), id_bytes(s), s.T, s.k, s.G, size(m, 0), ptr<int>(s.rows),
                        ptr<int>(m), ptr<int>(s.counts), c.stream());
}

// (topk_ids, row_of_slot, counts)
int sort_nopad(const Call &c) {
    const Sorted s = sort_args(c, 1, 2);
    return without_lock(dg_moe_sort_nopad, ptr(s.ids), id_bytes(s), s.T, s.k, s.G, ptr<int>(s.rows), ptr<int>(s.counts),
                        c.stream());
}

int integer(PyObject *o, const char *name) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) {
        PyErr_Clear();
        refuse("%s must be an integer", name);
    }
    if (v > 0x7fffffff || v < -0x7fffffff) refuse("%s=%lld is out of range", name, v);
    return static_cast<int>(v);
}

float number(PyObject *o, const char *name) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) {
        PyErr_Clear();
        refuse("%s must be a number", name);
    }
    return static_cast<float>(v);
}

// (topk_ids, row_of_slot, masked_m, m_max)
int sort_masked(const Call &c) {
    const Sorted s = sort_args(c, 1, 2);
    return without_lock(dg_moe_sort_masked, ptr(s.ids), id_bytes(s), s.T, s.k, s.G, integer(c.args[3], "m_max"),
                        ptr<int>(s.rows), ptr<int>(s.counts), c.stream());
}

// (x, row_of_slot, out)
int permute(const Call &c) {
    const at::Tensor &x = c.dims(0, "x", 2, 2), &row = c.dims(1, "row_of_slot", 2, 2);
    c.check(x, "x", x.sizes(), ACT);
    c.check(row, "row_of_slot", {x.size(0), row.size(1)}, I32);
    const RowOperand out = row_operand(c, 2, "out", x.size(1), same_as(x));
    return without_lock(dg_moe_permute, ptr(x), code(x), ptr<int>(row), size(x, 0), size(row, 1), size(x, 1), out.rows,
                        out.rows_per_group, ptr(out.a), ptr<float>(out.sf), c.stream());
}

const at::Tensor &rows_in(const Call &c, int i, int &n) {
    const at::Tensor &rows = c.dims(i, "rows", 2, 3);
    c.check(rows, "rows", rows.sizes(), ACT);
    const int64_t all = rows.dim() == 3 ? rows.size(0) * rows.size(1) : rows.size(0);
    if (all > 0x7fffffff) refuse("rows has more than 2^31 rows");
    n = static_cast<int>(all);
    return rows;
}

// (rows, row_of_slot, out, weights)
int unpermute(const Call &c) {
    int n;
    const at::Tensor &rows = rows_in(c, 0, n), &row = c.dims(1, "row_of_slot", 2, 2), &out = c.tensor(2, "out");
    const at::Tensor *w = c.optional(3, "weights");
    c.check(row, "row_of_slot", row.sizes(), I32);
    c.check(out, "out", {row.size(0), rows.size(-1)}, same_as(rows));
    c.check(w, "weights", row.sizes(), F32);
    return without_lock(dg_moe_unpermute, ptr(rows), code(rows), ptr<int>(row), ptr<float>(w), size(row, 0), size(row, 1),
                        size(rows, -1), n, ptr(out), c.stream());
}

// (d_out, rows, row_of_slot, weights, d_rows, d_weights)
int unpermute_backward(const Call &c) {
    int n;
    const at::Tensor &rows = rows_in(c, 1, n), &row = c.dims(2, "row_of_slot", 2, 2), &d_out = c.tensor(0, "d_out"),
                     &w = c.tensor(3, "weights"), &d_w = c.tensor(5, "d_weights");
    c.check(row, "row_of_slot", row.sizes(), I32);
    c.check(d_out, "d_out", {row.size(0), rows.size(-1)}, same_as(rows));
    c.check(w, "weights", row.sizes(), F32);
    c.check(d_w, "d_weights", row.sizes(), F32);
    const RowOperand d = row_operand(c, 4, "d_rows", rows.size(-1), same_as(rows));
    if (d.a->sizes() != rows.sizes())
        refuse("d_rows must be shaped as rows, %s, got %s", text(rows.sizes()).c_str(), text(d.a->sizes()).c_str());
    return without_lock(dg_moe_unpermute_backward, ptr(d_out), ptr(rows), code(rows), ptr<int>(row), ptr<float>(w),
                        size(row, 0), size(row, 1), size(rows, -1), n, d.rows_per_group, ptr(d.a), ptr<float>(d.sf),
                        ptr<float>(d_w), c.stream());
}

// (d_out or None, gate_up, out or d_gate_up, m_indices, counts, masked_m): None for d_out is the forward
int swiglu(const Call &c) {
    const at::Tensor *d_out = c.optional(0, "d_out");
    const at::Tensor &gu = c.dims(1, "gate_up", 2, 3);
    const char *name = d_out ? "d_gate_up" : "out";
    c.check(gu, "gate_up", gu.sizes(), ACT);
    const int64_t cols = gu.size(-1), I = cols / 2;
    if (cols % 2) refuse("gate_up must have an even number of columns");
    const bool grouped = gu.dim() == 3;
    const int64_t d_shape[3] = {grouped ? gu.size(0) : 1, gu.size(-2), I};
    c.check(d_out, "d_out", Shape(d_shape + !grouped, grouped ? 3 : 2), same_as(gu));
    const RowOperand out = row_operand(c, 2, name, d_out ? cols : I, same_as(gu));
    if (out.a->dim() != gu.dim() || out.a->size(0) != gu.size(0) || out.a->size(-2) != gu.size(-2))
        refuse("%s must have the rows of gate_up, %s, got %s", name, text(gu.sizes()).c_str(), text(out.a->sizes()).c_str());
    const at::Tensor *m = c.optional(3, "m_indices"), *counts = c.optional(4, "counts"), *masked = c.optional(5, "masked_m");
    if ((m != nullptr) + (counts != nullptr) + (masked != nullptr) > 1)
        refuse("at most one of m_indices, counts and masked_m may be given");
    int G = 0;
    c.check(m, "m_indices", {out.rows}, I32);
    if (counts) {
        c.check(c.dims(4, "counts", 1, 1), "counts", counts->sizes(), I32);
        G = size(*counts, 0);
    }
    if (masked) {
        c.check(c.dims(5, "masked_m", 1, 1), "masked_m", masked->sizes(), I32);
        G = size(*masked, 0);
    }
    if (grouped != (masked != nullptr) || (masked && G != gu.size(0)))
        refuse("tensors of three dims [G, M_max, ...] go with masked_m [G], and masked_m with them");
    if (d_out)
        return without_lock(dg_swiglu_backward, ptr(d_out), ptr(gu), code(gu), out.rows, static_cast<int>(I), ptr<int>(m),
                            ptr<int>(counts), ptr<int>(masked), G, ptr(out.a), ptr<float>(out.sf), c.stream());
    return without_lock(dg_swiglu, ptr(gu), code(gu), out.rows, static_cast<int>(I), ptr<int>(m), ptr<int>(counts),
                        ptr<int>(masked), G, ptr(out.a), ptr<float>(out.sf), c.stream());
}

// (x, weight, out, eps, rstd)
int rms_norm(const Call &c) {
    const at::Tensor &x = c.dims(0, "x", 2, 2), &w = c.tensor(1, "weight");
    const at::Tensor *rstd = c.optional(4, "rstd");
    c.check(x, "x", x.sizes(), ACT);
    c.check(w, "weight", {x.size(1)}, ACT);
    c.check(rstd, "rstd", {x.size(0)}, F32);
    Kind kind = BF16;
    if (THPVariable_Check(c.args[2])) {
        const at::Tensor &o = THPVariable_Unpack(c.args[2]);
        if (!is_kind(o.scalar_type(), ACT)) refuse("out must be bf16 or fp32, or a pair (e4m3, sfa)");
        kind = same_as(o);
    }
    const RowOperand out = row_operand(c, 2, "out", x.size(1), kind);
    if (out.a->sizes() != x.sizes()) refuse("out must be %s, got %s", text(x.sizes()).c_str(), text(out.a->sizes()).c_str());
    return without_lock(dg_rms_norm, ptr(x), code(x), ptr(w), code(w), number(c.args[3], "eps"), size(x, 0), size(x, 1),
                        ptr(out.a), kind == F32 ? DG_F32 : DG_BF16, ptr<float>(out.sf), ptr<float>(rstd), c.stream());
}

// (d_out, x, weight, rstd, d_x, d_weight, d_skip)
int rms_norm_backward(const Call &c) {
    const at::Tensor &x = c.dims(1, "x", 2, 2), &d_out = c.tensor(0, "d_out"), &w = c.tensor(2, "weight"),
                     &rstd = c.tensor(3, "rstd"), &d_x = c.tensor(4, "d_x"), &d_w = c.tensor(5, "d_weight");
    const at::Tensor *skip = c.optional(6, "d_skip");
    c.check(x, "x", x.sizes(), ACT);
    c.check(d_out, "d_out", x.sizes(), ACT);
    c.check(w, "weight", {x.size(1)}, ACT);
    c.check(rstd, "rstd", {x.size(0)}, F32);
    c.check(d_x, "d_x", x.sizes(), same_as(x));
    c.check(d_w, "d_weight", {x.size(1)}, F32);
    c.check(skip, "d_skip", x.sizes(), same_as(x));
    return without_lock(dg_rms_norm_backward, ptr(d_out), ptr(skip), ptr(x), code(x), code(d_out), ptr(w), code(w),
                        ptr<float>(rstd), size(x, 0), size(x, 1), ptr(d_x), ptr<float>(d_w), c.stream());
}

// weight, weight_post and a gate [H] have one type, bf16 or fp32; a gate [T, H] has y's.
struct NormParamArgs {
    const at::Tensor *w, *w_post, *gate;
    int gate_kind, type;
};

NormParamArgs norm_params(const Call &c, int w, int w_post, int gate, const at::Tensor &y) {
    NormParamArgs p{c.optional(w, "weight"), c.optional(w_post, "weight_post"), c.optional(gate, "gate"), 0, DG_F32};
    if (p.gate) p.gate_kind = c.dims(gate, "gate", 1, 2).dim();
    const at::Tensor *first = p.w ? p.w : p.w_post ? p.w_post : p.gate_kind == 1 ? p.gate : nullptr;
    Kind kind = F32;
    if (first) {
        if (!is_kind(first->scalar_type(), ACT)) refuse("the norms' parameters have dtype %s, expected %s",
                                                        c10::toString(first->scalar_type()), kind_name(ACT));
        kind = same_as(*first);
        p.type = code(*first);
    }
    const int64_t H = y.size(1);
    c.check(p.w, "weight", {H}, kind);
    c.check(p.w_post, "weight_post", {H}, kind);
    if (p.gate_kind == 1) c.check(p.gate, "gate", {H}, kind);
    if (p.gate_kind == 2) c.check(p.gate, "gate", y.sizes(), same_as(y));
    return p;
}

// (x, y, x_out, weight, out, weight_post, gate, alpha, eps, rstd, rstd_post)
int residual_rms_norm(const Call &c) {
    const at::Tensor &x = c.dims(0, "x", 2, 2), &y = c.tensor(1, "y"), &x_out = c.tensor(2, "x_out");
    c.check(x, "x", x.sizes(), ACT);
    c.check(y, "y", x.sizes(), ACT);
    c.check(x_out, "x_out", x.sizes(), same_as(x));
    const NormParamArgs p = norm_params(c, 3, 5, 6, y);
    if ((c.args[3] == Py_None) != (c.args[4] == Py_None)) refuse("weight and out go together");
    const at::Tensor *rstd = c.optional(9, "rstd"), *rstd_post = c.optional(10, "rstd_post");
    c.check(rstd, "rstd", {x.size(0)}, F32);
    c.check(rstd_post, "rstd_post", {x.size(0)}, F32);
    RowOperand out;
    if (p.w) {
        out = row_operand(c, 4, "out", x.size(1), same_as(y));
        if (out.a->sizes() != x.sizes())
            refuse("out must be %s, got %s", text(x.sizes()).c_str(), text(out.a->sizes()).c_str());
    }
    return without_lock(dg_residual_rms_norm, ptr(x), code(x), ptr(y), code(y), ptr(p.w), ptr(p.w_post), ptr(p.gate),
                        p.gate_kind, p.type, number(c.args[7], "alpha"), number(c.args[8], "eps"), size(x, 0), size(x, 1),
                        ptr(x_out), ptr(out.a), ptr<float>(out.sf), ptr<float>(rstd), ptr<float>(rstd_post), c.stream());
}

// (d_x_out, y, d_x, d_y, d_out, x_out, weight, rstd, weight_post, rstd_post, gate, alpha, d_weight, d_weight_post, d_gate)
int residual_rms_norm_backward(const Call &c) {
    const at::Tensor &y = c.dims(1, "y", 2, 2), &d_x = c.tensor(2, "d_x"), &d_y = c.tensor(3, "d_y");
    const at::Tensor *d_x_out = c.optional(0, "d_x_out"), *d_out = c.optional(4, "d_out"), *x_out = c.optional(5, "x_out"),
                     *rstd = c.optional(7, "rstd"), *rstd_post = c.optional(9, "rstd_post"), *d_w = c.optional(12, "d_weight"),
                     *d_w_post = c.optional(13, "d_weight_post"), *d_gate = c.optional(14, "d_gate");
    const int64_t T = y.size(0), H = y.size(1);
    c.check(y, "y", y.sizes(), ACT);
    c.check(d_y, "d_y", y.sizes(), same_as(y));
    c.check(d_x, "d_x", y.sizes(), ACT);
    const NormParamArgs p = norm_params(c, 6, 8, 10, y);
    c.check(d_x_out, "d_x_out", y.sizes(), same_as(d_x));
    c.check(d_out, "d_out", y.sizes(), same_as(y));
    c.check(x_out, "x_out", y.sizes(), same_as(d_x));
    c.check(rstd, "rstd", {T}, F32);
    c.check(rstd_post, "rstd_post", {T}, F32);
    c.check(d_w, "d_weight", {H}, F32);
    c.check(d_w_post, "d_weight_post", {H}, F32);
    if (p.gate_kind == 1) c.check(d_gate, "d_gate", {H}, F32);
    else c.check(d_gate, "d_gate", y.sizes(), same_as(y));
    return without_lock(dg_residual_rms_norm_backward, ptr(d_x_out), ptr(d_out), ptr(x_out), code(d_x), ptr(y), code(y),
                        ptr(p.w), ptr(p.w_post), ptr(p.gate), p.gate_kind, p.type, number(c.args[11], "alpha"),
                        ptr<float>(rstd), ptr<float>(rstd_post), size(y, 0), size(y, 1), ptr(d_x), ptr(d_y), ptr<float>(d_w),
                        ptr<float>(d_w_post), ptr(d_gate), c.stream());
}

PyObject *raise(int status, const char *message) {
    PyObject *args = Py_BuildValue("(is)", status, message);
    if (args) PyErr_SetObject(g_error_class ? g_error_class : PyExc_RuntimeError, args);
    Py_XDECREF(args);
    return nullptr;
}

template <int (*F)(const Call &), int N> PyObject *entry(PyObject *, PyObject *const *args, Py_ssize_t n) {
    if (n != N) {
        PyErr_Format(PyExc_TypeError, "expected %d arguments, got %zd", N, n);
        return nullptr;
    }
    try {
        const int status = F(Call{args});
        if (status != DG_OK) return raise(status, dg_last_error());
        Py_RETURN_NONE;
    } catch (const Refused &r) {
        return raise(r.status, r.message.c_str());
    } catch (const c10::Error &e) {
        return raise(DG_ERR_CUDA, e.what_without_backtrace());
    } catch (const std::exception &e) {
        return raise(DG_ERR_CUDA, e.what());
    }
}

PyObject *set_error(PyObject *, PyObject *cls) {
    Py_INCREF(cls);
    Py_XSETREF(g_error_class, cls);
    Py_RETURN_NONE;
}

#define ENTRY(name, f, n) \
    {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(entry<f, n>)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {
    {"set_error", set_error, METH_O, nullptr},
    ENTRY("moe_sort_contiguous", sort_contiguous, 4),
    ENTRY("moe_sort_nopad", sort_nopad, 3),
    ENTRY("moe_sort_masked", sort_masked, 4),
    ENTRY("moe_permute", permute, 3),
    ENTRY("moe_unpermute", unpermute, 4),
    ENTRY("moe_unpermute_backward", unpermute_backward, 6),
    ENTRY("swiglu", swiglu, 6),
    ENTRY("rms_norm", rms_norm, 5),
    ENTRY("rms_norm_backward", rms_norm_backward, 7),
    ENTRY("residual_rms_norm", residual_rms_norm, 11),
    ENTRY("residual_rms_norm_backward", residual_rms_norm_backward, 15),
    {nullptr, nullptr, 0, nullptr}};
#undef ENTRY

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_rowwise", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__rowwise() { return PyModule_Create(&module); }
