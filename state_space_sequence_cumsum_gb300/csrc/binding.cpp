// Native binding of the layer operators: checks tensors, allocates outputs and
// workspace on the current stream and calls the C ABI.  layer.py holds the
// signatures and their documentation.  A call on a few tokens is shorter than
// the checks of its dozen tensors in Python (about 30 us against 5 us here),
// which is why these are compiled.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/ssd.h"

namespace {

using at::Tensor;

PyObject *g_error = nullptr;  // the package's SsdError

PyObject *raise_status(ssd_status_t s, const char *where)
{
    PyObject *e = PyObject_CallFunction(g_error, "is", (int)s, where);
    if (e) {
        PyErr_SetObject(g_error, e);
        Py_DECREF(e);
    }
    return nullptr;
}

Tensor tensor(PyObject *o, const char *name)
{
    TORCH_CHECK_TYPE(THPVariable_Check(o), name, " must be a tensor");
    return THPVariable_Unpack(o);
}
Tensor optional(PyObject *o, const char *name) { return o == Py_None ? Tensor() : tensor(o, name); }

template <typename T = void> T *ptr(const Tensor &t)
{
    return t.defined() ? static_cast<T *>(t.data_ptr()) : nullptr;
}

PyObject *wrap(const Tensor &t)
{
    if (!t.defined())
        Py_RETURN_NONE;
    return THPVariable_Wrap(t);
}

template <typename... Ts> PyObject *tuple(const Ts &...ts)
{
    PyObject *r = PyTuple_New(sizeof...(ts));
    if (!r)
        return nullptr;
    Py_ssize_t i = 0;
    bool ok = true;
    auto put = [&](const Tensor &t) {
        PyObject *w = wrap(t);
        ok = ok && w;
        PyTuple_SET_ITEM(r, i++, w);
    };
    (put(ts), ...);
    if (!ok) {
        Py_DECREF(r);
        return nullptr;
    }
    return r;
}

// ------------------------------------------------------------------ checks

ssd_dtype_t dtype_code(const Tensor &t, const char *name)
{
    const auto s = t.scalar_type();
    TORCH_CHECK_TYPE(s == at::kBFloat16 || s == at::kFloat, name, " must be bfloat16 or float32, got ", s);
    return s == at::kBFloat16 ? SSD_BF16 : SSD_F32;
}

// Shape, type and device of a (possibly absent) tensor.
void same(const Tensor &t, const char *name, at::IntArrayRef shape, at::ScalarType type, const Tensor &like,
          bool contiguous)
{
    if (!t.defined())
        return;
    TORCH_CHECK_VALUE(t.sizes() == shape, name, " must be ", shape, ", got ", t.sizes());
    TORCH_CHECK_TYPE(t.scalar_type() == type, name, " must be ", type, ", got ", t.scalar_type());
    TORCH_CHECK_VALUE(t.device() == like.device(), name, " must be on ", like.device());
    TORCH_CHECK_VALUE(!contiguous || t.is_contiguous(), name, " must be contiguous");
}
void same_f32(const Tensor &t, const char *name, at::IntArrayRef shape, const Tensor &like)
{
    same(t, name, shape, at::kFloat, like, true);
}

void on_gpu(const Tensor &t, const char *name)
{
    TORCH_CHECK_VALUE(t.is_cuda(), name, ": the layer operators take CUDA tensors");
}

// Elements between consecutive rows, whose last `inner` dimensions are one
// contiguous run and whose others are evenly spaced.
int64_t row_of(const Tensor &t, const char *name, int inner = 1)
{
    const auto sz = t.sizes(), st = t.strides();
    const int n = (int)sz.size(), lead = n - inner;
    int64_t len = 1;
    for (int i = n - 1; i >= lead; --i) {
        TORCH_CHECK_VALUE(sz[i] <= 1 || t.numel() == 0 || st[i] == len, name,
                          ": the last dimension must be contiguous");
        len *= sz[i];
    }
    if (t.numel() == 0)
        return len;
    int64_t row = -1, step = -1;
    for (int i = lead - 1; i >= 0; --i) {
        if (sz[i] == 1)
            continue;
        if (step < 0)
            row = st[i];
        else
            TORCH_CHECK_VALUE(st[i] == step, name, ": rows must be evenly spaced");
        step = st[i] * sz[i];
    }
    if (row < 0 && step < 0)
        return len;
    TORCH_CHECK_VALUE(row >= len, name, ": rows overlap");
    return row;
}

// A new tensor beside `like`, allocated directly: a backward returns nine, and
// the dispatcher would cost as much as the allocation.  The price: dispatch
// modes do not see these allocations, and torch.utils.deterministic's fill of
// uninitialised memory passes them by (the kernels write every element).
Tensor fresh(at::IntArrayRef shape, at::ScalarType type, const Tensor &like)
{
    return Tensor(at::detail::empty_cuda(shape, type, like.device(), std::nullopt));
}

// The caller's output, checked, or a new one.
Tensor output(PyObject *given, const char *name, at::IntArrayRef shape, at::ScalarType type, const Tensor &like,
              bool wanted = true)
{
    Tensor t = optional(given, name);
    if (!t.defined())
        return wanted ? fresh(shape, type, like) : t;
    same(t, name, shape, type, like, true);
    return t;
}

// Tells autograd that a tensor of the caller's was written: a backward that
// saved it before then raises instead of using the new values.  (Inference
// tensors keep no count and cannot be saved.)
void written(const Tensor &t)
{
    if (t.defined() && !t.is_inference())
        t.unsafeGetTensorImpl()->bump_version();
}
template <typename... Ts> void written_if(PyObject *given, const Tensor &t, const Ts &...more)
{
    if (given != Py_None)
        written(t);
    if constexpr (sizeof...(more) > 0)
        written_if(more...);
}

// Workspace of n bytes: the caller's Workspace object grown to it, or a buffer
// that the allocator takes back in stream order.  The caller's may come from
// another stream's pool: the allocator is told of this one, so that a buffer
// that the object grows out of is not given away while the call still uses it.
struct Scratch {
    Tensor t;
    Scratch(PyObject *ws, size_t n, const Tensor &like, PyObject *like_obj)
    {
        if (n == 0)
            return;
        if (ws == Py_None) {
            t = fresh({(int64_t)n}, at::kByte, like);
            return;
        }
        PyObject *dev = PyObject_GetAttrString(like_obj, "device");
        PyObject *got = dev ? PyObject_CallMethod(ws, "get", "nO", (Py_ssize_t)n, dev) : nullptr;
        Py_XDECREF(dev);
        if (!got)
            throw python_error();
        if (THPVariable_Check(got))
            t = THPVariable_Unpack(got);
        Py_DECREF(got);
        TORCH_CHECK_VALUE(t.defined() && t.device() == like.device(), "workspace.get must return a tensor on ",
                          like.device());
        c10::cuda::CUDACachingAllocator::recordStream(t.storage().data_ptr(),
                                                      c10::cuda::getCurrentCUDAStream(t.device().index()));
    }
    void *p() const { return t.defined() ? t.data_ptr() : nullptr; }
    size_t n() const { return t.defined() ? (size_t)t.nbytes() : 0; }
};

struct On {
    c10::cuda::CUDAGuard guard;
    void *stream;
    explicit On(const Tensor &t) : guard(t.device()), stream(c10::cuda::getCurrentCUDAStream(t.device().index())) {}
};

bool truth(PyObject *o)
{
    const int r = PyObject_IsTrue(o);
    if (r < 0)
        throw python_error();
    return r != 0;
}
double number(PyObject *o)
{
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred())
        throw python_error();
    return v;
}

void count(Py_ssize_t got, Py_ssize_t want)
{
    TORCH_CHECK_TYPE(got == want, "expected ", want, " arguments, got ", got);
}

// ------------------------------------------------------------- convolution

struct Conv {
    ssd_dtype_t code;
    ssd_conv_dims_t d;
    int64_t state[3];
    at::IntArrayRef state_shape() const { return {state, 3}; }
    Conv(const Tensor &x, const Tensor &w, const Tensor &bias, int lead)
    {
        code = dtype_code(x, "x");
        TORCH_CHECK_VALUE(x.dim() == lead + 1, "x must be ", lead == 2 ? "[batch, seqlen, dim]" : "[batch, dim]");
        const int64_t dim = x.size(-1);
        TORCH_CHECK_VALUE(w.dim() == 2 && w.size(0) == dim, "weight must be [dim, width]");
        same_f32(w, "weight", w.sizes(), x);
        same_f32(bias, "bias", {dim}, x);
        d = {x.size(0), lead == 2 ? x.size(1) : 1, dim, w.size(1)};
        state[0] = d.batch;
        state[1] = d.width > 0 ? d.width - 1 : 0;
        state[2] = dim;
    }
};

// x, weight, bias, silu, initial_state, want_final, y, final_state
PyObject *causal_conv(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    count(n, 8);
    const Tensor x = tensor(a[0], "x"), w = tensor(a[1], "weight"), bias = optional(a[2], "bias");
    const Tensor init = optional(a[4], "initial_state");
    const Conv c(x, w, bias, 2);
    const int64_t row = row_of(x, "x");
    same(init, "initial_state", c.state_shape(), x.scalar_type(), x, true);
    on_gpu(x, "x");
    const On on(x);
    const Tensor y = output(a[6], "y", x.sizes(), x.scalar_type(), x);
    const Tensor fin = output(a[7], "final_state", c.state_shape(), x.scalar_type(), x, truth(a[5]));
    const ssd_status_t s = ssd_causal_conv(ptr(x), row, ptr<float>(w), ptr<float>(bias), ptr(init), ptr(y), ptr(fin),
                                           c.d, truth(a[3]), c.code, on.stream);
    if (s != SSD_OK)
        return raise_status(s, "ssd_causal_conv");
    written_if(a[6], y, a[7], fin);
    return tuple(y, fin);
    END_HANDLE_TH_ERRORS
}

// x, weight, dy, bias, silu, initial_state, dfinal, want_dinit, workspace
PyObject *causal_conv_bwd(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    count(n, 9);
    const Tensor x = tensor(a[0], "x"), w = tensor(a[1], "weight"), dy = tensor(a[2], "dy");
    const Tensor bias = optional(a[3], "bias"), init = optional(a[5], "initial_state"), df = optional(a[6], "dfinal");
    const Conv c(x, w, bias, 2);
    const auto type = x.scalar_type();
    same(dy, "dy", x.sizes(), type, x, false);
    const int64_t row = row_of(x, "x"), row_dy = row_of(dy, "dy");
    same(init, "initial_state", c.state_shape(), type, x, true);
    same(df, "dfinal", c.state_shape(), type, x, true);
    on_gpu(x, "x");
    const On on(x);
    const Tensor dx = fresh(x.sizes(), type, x), dw = fresh(w.sizes(), at::kFloat, x);
    const Tensor db = bias.defined() ? fresh(bias.sizes(), at::kFloat, x) : Tensor();
    const Tensor di = truth(a[7]) ? fresh(c.state_shape(), type, x) : Tensor();
    const Scratch ws(a[8], ssd_causal_conv_bwd_workspace_size(c.d), x, a[0]);
    const ssd_status_t s =
        ssd_causal_conv_bwd(ptr(x), row, ptr<float>(w), ptr<float>(bias), ptr(init), ptr(dy), row_dy, ptr(df), ptr(dx),
                            ptr<float>(dw), ptr<float>(db), ptr(di), c.d, truth(a[4]), c.code, ws.p(), ws.n(), on.stream);
    return s == SSD_OK ? tuple(dx, dw, db, di) : raise_status(s, "ssd_causal_conv_bwd");
    END_HANDLE_TH_ERRORS
}

// x, weight, state, bias, silu, state_out, y
PyObject *causal_conv_step(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    count(n, 7);
    const Tensor x = tensor(a[0], "x"), w = tensor(a[1], "weight"), state = tensor(a[2], "state");
    const Tensor bias = optional(a[3], "bias");
    const Conv c(x, w, bias, 1);
    const int64_t row = row_of(x, "x");
    same(state, "state", c.state_shape(), x.scalar_type(), x, true);
    on_gpu(x, "x");
    const On on(x);
    Tensor out = optional(a[5], "state_out");
    if (out.defined())
        same(out, "state_out", c.state_shape(), x.scalar_type(), x, true);
    else
        out = state;
    const Tensor y = output(a[6], "y", x.sizes(), x.scalar_type(), x);
    const ssd_status_t s = ssd_causal_conv_step(ptr(x), row, ptr<float>(w), ptr<float>(bias), ptr(state), ptr(out),
                                                ptr(y), c.d, truth(a[4]), c.code, on.stream);
    if (s != SSD_OK)
        return raise_status(s, "ssd_causal_conv_step");
    written(out);
    written_if(a[6], y);
    return tuple(y, out);
    END_HANDLE_TH_ERRORS
}

// ---------------------------------------------------------- selective scan

struct Scan {
    ssd_dtype_t code;
    ssd_scan_dims_t d;
    ssd_scan_rows_t r;
    int64_t state[3], kept[4];
    at::IntArrayRef state_shape() const { return {state, 3}; }
    at::IntArrayRef kept_shape() const { return {kept, 4}; }
    Scan(const Tensor &u, const Tensor &dt, const Tensor &A, const Tensor &B, const Tensor &C, const Tensor &D,
         const Tensor &z, const Tensor &bias, const Tensor &dy, int lead)
    {
        code = dtype_code(u, "u");
        TORCH_CHECK_VALUE(u.dim() == lead + 1, "u must be ", lead == 2 ? "[batch, seqlen, dim]" : "[batch, dim]");
        const auto type = u.scalar_type();
        const int64_t dim = u.size(-1);
        TORCH_CHECK_VALUE(A.dim() == 2 && A.size(0) == dim, "A must be [dim, dstate]");
        const int64_t N = A.size(1);
        const bool grouped = B.dim() == lead + 2;
        TORCH_CHECK_VALUE(grouped || B.dim() == lead + 1,
                          "B and C must be [..., dstate] or [..., ngroups, dstate]");
        const int64_t G = grouped ? B.size(-2) : 1;
        TORCH_CHECK_VALUE(G > 0 && dim % G == 0, "dim must be a multiple of the groups of B and C");
        int64_t bc[4];
        int k = 0;
        for (; k < lead; ++k)
            bc[k] = u.size(k);
        if (grouped)
            bc[k++] = G;
        bc[k++] = N;
        same(B, "B", {bc, (size_t)k}, type, u, false);
        same(C, "C", {bc, (size_t)k}, type, u, false);
        same(dt, "dt", u.sizes(), type, u, false);
        same(z, "z", u.sizes(), type, u, false);
        same(dy, "dy", u.sizes(), type, u, false);
        same_f32(A, "A", A.sizes(), u);
        same_f32(D, "D", {dim}, u);
        same_f32(bias, "dt_bias", {dim}, u);
        d = {u.size(0), lead == 2 ? u.size(1) : 1, dim, N, G};
        r = {row_of(u, "u"),
             row_of(dt, "dt"),
             z.defined() ? row_of(z, "z") : dim,
             row_of(B, "B", grouped ? 2 : 1),
             row_of(C, "C", grouped ? 2 : 1),
             dy.defined() ? row_of(dy, "dy") : dim};
        state[0] = d.batch;
        state[1] = dim;
        state[2] = N;
        const int64_t T = ssd_selective_scan_chunk();
        kept[0] = d.batch;
        kept[1] = (d.seqlen + T - 1) / T;
        kept[2] = dim;
        kept[3] = N;
    }
};

// u, dt, A, B, C, D, z, dt_bias, softplus, initial_state, want_final, want_chunks, y, final_state,
// chunk_states, workspace
PyObject *selective_scan(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    count(n, 16);
    const Tensor u = tensor(a[0], "u"), dt = tensor(a[1], "dt"), A = tensor(a[2], "A"), B = tensor(a[3], "B"),
                 C = tensor(a[4], "C"), D = optional(a[5], "D"), z = optional(a[6], "z"),
                 bias = optional(a[7], "dt_bias"), init = optional(a[9], "initial_state");
    const Scan c(u, dt, A, B, C, D, z, bias, Tensor(), 2);
    same_f32(init, "initial_state", c.state_shape(), u);
    on_gpu(u, "u");
    const On on(u);
    const Tensor y = output(a[12], "y", u.sizes(), u.scalar_type(), u);
    const Tensor fin = output(a[13], "final_state", c.state_shape(), at::kFloat, u, truth(a[10]));
    const Tensor kept = output(a[14], "chunk_states", c.kept_shape(), at::kFloat, u, truth(a[11]));
    const Scratch ws(a[15], ssd_selective_scan_workspace_size(c.d), u, a[0]);
    const ssd_status_t s = ssd_selective_scan(ptr(u), ptr(dt), ptr<float>(A), ptr(B), ptr(C), ptr<float>(D), ptr(z),
                                              ptr<float>(bias), ptr<float>(init), ptr(y), ptr<float>(fin),
                                              ptr<float>(kept), c.d, c.r, truth(a[8]), c.code, ws.p(), ws.n(), on.stream);
    if (s != SSD_OK)
        return raise_status(s, "ssd_selective_scan");
    written_if(a[12], y, a[13], fin, a[14], kept);
    return tuple(y, fin, kept);
    END_HANDLE_TH_ERRORS
}

// u, dt, A, B, C, D, dy, z, dt_bias, softplus, initial_state, dfinal, chunk_states, want_dinit, workspace
PyObject *selective_scan_bwd(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    count(n, 15);
    const Tensor u = tensor(a[0], "u"), dt = tensor(a[1], "dt"), A = tensor(a[2], "A"), B = tensor(a[3], "B"),
                 C = tensor(a[4], "C"), D = optional(a[5], "D"), dy = tensor(a[6], "dy"), z = optional(a[7], "z"),
                 bias = optional(a[8], "dt_bias"), init = optional(a[10], "initial_state"),
                 df = optional(a[11], "dfinal"), kept = optional(a[12], "chunk_states");
    const Scan c(u, dt, A, B, C, D, z, bias, dy, 2);
    same_f32(init, "initial_state", c.state_shape(), u);
    same_f32(df, "dfinal", c.state_shape(), u);
    same_f32(kept, "chunk_states", c.kept_shape(), u);
    on_gpu(u, "u");
    const On on(u);
    const auto type = u.scalar_type();
    const Tensor none;
    const Tensor du = fresh(u.sizes(), type, u), ddt = fresh(u.sizes(), type, u), dA = fresh(A.sizes(), at::kFloat, u),
                 dB = fresh(B.sizes(), type, u), dC = fresh(C.sizes(), type, u),
                 dD = D.defined() ? fresh(D.sizes(), at::kFloat, u) : none,
                 dz = z.defined() ? fresh(u.sizes(), type, u) : none,
                 db = bias.defined() ? fresh(bias.sizes(), at::kFloat, u) : none,
                 di = truth(a[13]) ? fresh(c.state_shape(), at::kFloat, u) : none;
    const Scratch ws(a[14], ssd_selective_scan_bwd_workspace_size(c.d, kept.defined()), u, a[0]);
    const ssd_status_t s = ssd_selective_scan_bwd(
        ptr(u), ptr(dt), ptr<float>(A), ptr(B), ptr(C), ptr<float>(D), ptr(z), ptr<float>(bias), ptr<float>(init), ptr(dy),
        ptr<float>(df), ptr<float>(kept), ptr(du), ptr(ddt), ptr<float>(dA), ptr(dB), ptr(dC), ptr<float>(dD), ptr(dz),
        ptr<float>(db), ptr<float>(di), c.d, c.r, truth(a[9]), c.code, ws.p(), ws.n(), on.stream);
    return s == SSD_OK ? tuple(du, ddt, dA, dB, dC, dD, dz, db, di) : raise_status(s, "ssd_selective_scan_bwd");
    END_HANDLE_TH_ERRORS
}

// u, dt, A, B, C, D, state, z, dt_bias, softplus, state_out, y
PyObject *selective_scan_step(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    count(n, 12);
    const Tensor u = tensor(a[0], "u"), dt = tensor(a[1], "dt"), A = tensor(a[2], "A"), B = tensor(a[3], "B"),
                 C = tensor(a[4], "C"), D = optional(a[5], "D"), state = tensor(a[6], "state"),
                 z = optional(a[7], "z"), bias = optional(a[8], "dt_bias");
    const Scan c(u, dt, A, B, C, D, z, bias, Tensor(), 1);
    same_f32(state, "state", c.state_shape(), u);
    on_gpu(u, "u");
    const On on(u);
    Tensor out = optional(a[10], "state_out");
    if (out.defined())
        same_f32(out, "state_out", c.state_shape(), u);
    else
        out = state;
    const Tensor y = output(a[11], "y", u.sizes(), u.scalar_type(), u);
    const ssd_status_t s = ssd_selective_scan_step(ptr(u), ptr(dt), ptr<float>(A), ptr(B), ptr(C), ptr<float>(D), ptr(z),
                                                   ptr<float>(bias), ptr<float>(state), ptr<float>(out), ptr(y), c.d,
                                                   c.r, truth(a[9]), c.code, on.stream);
    if (s != SSD_OK)
        return raise_status(s, "ssd_selective_scan_step");
    written(out);
    written_if(a[11], y);
    return tuple(y, out);
    END_HANDLE_TH_ERRORS
}

// -------------------------------------------------------------- block norm

struct Norm {
    ssd_dtype_t code;
    int64_t tokens, dim, rows;
    Norm(const Tensor &y, const Tensor &w, const Tensor &pw, const Tensor &gate)
    {
        code = dtype_code(y, "y");
        TORCH_CHECK_VALUE(y.dim() >= 1 && y.size(-1) > 0, "y must be [..., dim]");
        TORCH_CHECK_VALUE(y.is_contiguous(), "y must be contiguous");
        dim = y.size(-1);
        tokens = y.numel() / dim;
        same_f32(w, "weight", {dim}, y);
        same_f32(pw, "post_weight", {dim}, y);
        rows = 0;
        if (gate.defined()) {
            TORCH_CHECK_VALUE(gate.dim() >= 1 && gate.size(-1) == dim, "gate must be [..., dim]");
            same_f32(gate, "gate", gate.sizes(), y);
            rows = gate.numel() / dim;
            TORCH_CHECK_VALUE(rows > 0 && tokens % rows == 0, "the tokens must be a multiple of the gate's rows");
        }
    }
    ssd_dtype_t residual(const Tensor &y, const Tensor &r) const
    {
        TORCH_CHECK_TYPE(r.scalar_type() == y.scalar_type() || r.scalar_type() == at::kFloat, "the residual must be ",
                         y.scalar_type(), " or Float, got ", r.scalar_type());
        return r.scalar_type() == at::kFloat ? SSD_F32 : SSD_BF16;
    }
};

// y, residual, weight, post_weight, gate, scale, eps, out, residual_out, residual_f32
PyObject *block_norm(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    count(n, 10);
    const Tensor y = tensor(a[0], "y"), res = optional(a[1], "residual"), w = tensor(a[2], "weight"),
                 pw = optional(a[3], "post_weight"), gate = optional(a[4], "gate");
    const Norm c(y, w, pw, gate);
    Tensor rout = optional(a[8], "residual_out");
    const at::ScalarType rt = res.defined()    ? res.scalar_type()
                              : rout.defined() ? rout.scalar_type()
                              : truth(a[9])    ? at::kFloat
                                               : y.scalar_type();
    same(res, "residual", y.sizes(), rt, y, true);
    on_gpu(y, "y");
    const On on(y);
    const Tensor out = output(a[7], "out", y.sizes(), y.scalar_type(), y);
    rout = output(a[8], "residual_out", y.sizes(), rt, y);
    const ssd_status_t s = ssd_block_norm(ptr(y), ptr(res), ptr<float>(w), ptr<float>(pw), ptr<float>(gate), ptr(out),
                                          ptr(rout), c.tokens, c.dim, c.rows, (float)number(a[5]), (float)number(a[6]),
                                          c.code, c.residual(y, rout), on.stream);
    if (s != SSD_OK)
        return raise_status(s, "ssd_block_norm");
    written_if(a[7], out, a[8], rout);
    return tuple(out, rout);
    END_HANDLE_TH_ERRORS
}

// y, residual_out, weight, dout, dresidual_out, post_weight, gate, scale, eps, workspace
PyObject *block_norm_bwd(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    count(n, 10);
    const Tensor y = tensor(a[0], "y"), r = tensor(a[1], "residual_out"), w = tensor(a[2], "weight"),
                 dout = tensor(a[3], "dout"), dr = optional(a[4], "dresidual_out"),
                 pw = optional(a[5], "post_weight"), gate = optional(a[6], "gate");
    const Norm c(y, w, pw, gate);
    const ssd_dtype_t rcode = c.residual(y, r);
    same(r, "residual_out", y.sizes(), r.scalar_type(), y, true);
    same(dout, "dout", y.sizes(), y.scalar_type(), y, true);
    same(dr, "dresidual_out", y.sizes(), r.scalar_type(), y, true);
    on_gpu(y, "y");
    const On on(y);
    const Tensor dy = fresh(y.sizes(), y.scalar_type(), y), dres = fresh(y.sizes(), r.scalar_type(), y),
                 dw = fresh(w.sizes(), at::kFloat, y),
                 dpw = pw.defined() ? fresh(pw.sizes(), at::kFloat, y) : Tensor(),
                 dg = gate.defined() ? fresh(gate.sizes(), at::kFloat, y) : Tensor();
    const Scratch ws(a[9], ssd_block_norm_bwd_workspace_size(c.tokens, c.dim, c.rows), y, a[0]);
    const ssd_status_t s =
        ssd_block_norm_bwd(ptr(y), ptr(r), ptr<float>(w), ptr<float>(pw), ptr<float>(gate), ptr(dout), ptr(dr), ptr(dy),
                           ptr(dres), ptr<float>(dw), ptr<float>(dpw), ptr<float>(dg), c.tokens, c.dim, c.rows,
                           (float)number(a[7]), (float)number(a[8]), c.code, rcode, ws.p(), ws.n(), on.stream);
    return s == SSD_OK ? tuple(dy, dres, dw, dpw, dg) : raise_status(s, "ssd_block_norm_bwd");
    END_HANDLE_TH_ERRORS
}

PyObject *set_error(PyObject *, PyObject *cls)
{
    Py_INCREF(cls);
    Py_XDECREF(g_error);
    g_error = cls;
    Py_RETURN_NONE;
}

#define FAST(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FAST(causal_conv),      FAST(causal_conv_bwd),     FAST(causal_conv_step),
                         FAST(selective_scan),   FAST(selective_scan_bwd),  FAST(selective_scan_step),
                         FAST(block_norm),       FAST(block_norm_bwd),
                         {"set_error", set_error, METH_O, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_native", "Native binding of the layer operators.", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__native(void) { return PyModule_Create(&module); }
