// Python binding of the paged-cache operators (module _paged).
//
// A serving step calls these once per layer on a few tokens, where the kernels take
// a few microseconds and a binding written in Python ten times that (measured, at its
// leanest: 21 us of checks and marshalling for the attention of one step, 46 for the
// norms' gradient; here 7 and 9).  So the checks of tensors, the allocation of outputs and workspace and
// the call of the C ABI are here; paged.py holds the signatures and the
// documentation.  Refusals raise HGAError with the package's wording.
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/core/LegacyTypeDispatch.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <numeric>
#include <sstream>
#include <stdexcept>
#include <string>
#include <vector>

#include "../../include/hga.h"

namespace {

PyObject *g_error = nullptr, *g_out_of_memory = nullptr;   // HGAError, torch's

struct Refused : std::runtime_error {
    using std::runtime_error::runtime_error;
};
struct Raised {};              // a Python exception is already set

template <typename... A> [[noreturn]] void refuse(const A &...a) {
    std::ostringstream s;
    (s << ... << a);
    throw Refused(s.str());
}

std::string text(at::IntArrayRef v) {
    std::ostringstream s;
    s << '(';
    for (size_t i = 0; i < v.size(); ++i) s << (i ? ", " : "") << v[i];
    s << (v.size() == 1 ? ",)" : ")");
    return s.str();
}

const at::Tensor &tensor(PyObject *o, const char *name) {
    if (!THPVariable_Check(o)) refuse(name, " must be a torch.Tensor");
    const at::Tensor &t = THPVariable_Unpack(o);
    if (!t.is_cuda()) refuse(name, " must be a CUDA tensor");
    return t;
}
inline bool none(PyObject *o) { return o == Py_None; }

// What a call works on: its device, stream and element type.
struct Call {
    int dev;
    void *stream;
    c10::optional<c10::cuda::CUDAStream> other;   // a given stream
    c10::cuda::OptionalCUDAGuard guard;

    Call(const at::Tensor &t, PyObject *stream_obj) : dev(t.get_device()) {
        if (none(stream_obj)) {
            stream = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream();
        } else {
            const long long id = number(stream_obj, "stream_id"), ix = number(stream_obj, "device_index"),
                            ty = number(stream_obj, "device_type");
            if (ix != dev) refuse("stream is on cuda:", ix, ", the call's tensors are on cuda:", dev);
            other = c10::cuda::CUDAStream::unpack3(id, (c10::DeviceIndex)ix, (c10::DeviceType)ty);
            stream = other->stream();
        }
        guard.set_index((c10::DeviceIndex)dev);
    }
    static long long number(PyObject *o, const char *attr) {
        PyObject *v = PyObject_GetAttrString(o, attr);
        if (!v) throw Raised();
        const long long x = PyLong_AsLongLong(v);
        Py_DECREF(v);
        if (x == -1 && PyErr_Occurred()) throw Raised();
        return x;
    }
    // A new tensor, of the given stream's memory: blocks that the current stream has
    // freed may still be written to by what is queued there.
    at::Tensor empty(at::IntArrayRef shape, at::ScalarType dt) const {
        const auto options = at::TensorOptions().dtype(dt).device(at::Device(at::kCUDA, (c10::DeviceIndex)dev));
        if (!other) return at::empty(shape, options);
        const c10::cuda::CUDAStreamGuard on(*other);
        return at::empty(shape, options);
    }
};

void on_device(const at::Tensor &t, const char *name, int dev) {
    if (t.get_device() != dev)
        refuse(name, " is on ", t.device().str(), ", the call's tensors are on cuda:", dev);
}

// The address of a contiguous tensor of that shape and type on the call's device.
void *dense(PyObject *o, const char *name, at::IntArrayRef shape, at::ScalarType dt, const Call &c) {
    const at::Tensor &t = tensor(o, name);
    on_device(t, name, c.dev);
    if (!t.is_contiguous()) refuse(name, " must be contiguous");
    if (t.sizes() != shape) refuse(name, " has shape ", text(t.sizes()), ", expected ", text(shape));
    if (t.scalar_type() != dt)
        refuse(name, " has dtype ", c10::toString(t.scalar_type()), ", expected ", c10::toString(dt));
    return t.data_ptr();
}
void *dense_or_null(PyObject *o, const char *name, at::IntArrayRef shape, at::ScalarType dt,
                    const Call &c) {
    return none(o) ? nullptr : dense(o, name, shape, dt, c);
}
int32_t *ints(PyObject *o, const char *name, at::IntArrayRef shape, const Call &c) {
    return static_cast<int32_t *>(dense(o, name, shape, at::kInt, c));
}
int32_t *ints_or_null(PyObject *o, const char *name, at::IntArrayRef shape, const Call &c) {
    return none(o) ? nullptr : ints(o, name, shape, c);
}

// A given output, or a new one.
at::Tensor output(PyObject *o, const char *name, at::IntArrayRef shape, at::ScalarType dt, const Call &c) {
    if (none(o)) return c.empty(shape, dt);
    dense(o, name, shape, dt, c);
    return THPVariable_Unpack(o);
}

int dtype_code(const at::Tensor &t) {
    if (t.scalar_type() == at::kFloat) return HGA_F32;
    if (t.scalar_type() == at::kBFloat16) return HGA_BF16;
    refuse("unsupported dtype ", c10::toString(t.scalar_type()), ": float32 or bfloat16");
}

long long whole(PyObject *o, const char *name) {
    const long long x = PyLong_AsLongLong(o);
    if (x == -1 && PyErr_Occurred()) throw Raised();
    if (x < 0 || x > INT32_MAX) refuse(name, " is ", x, ", expected 0 .. 2^31 - 1");
    return x;
}
double real(PyObject *o) {
    const double x = PyFloat_AsDouble(o);
    if (x == -1.0 && PyErr_Occurred()) throw Raised();
    return x;
}
bool truth(PyObject *o) {
    const int x = PyObject_IsTrue(o);
    if (x < 0) throw Raised();
    return x > 0;
}
int32_t size32(int64_t x, const char *name) {
    if (x > INT32_MAX) refuse(name, " of ", x, " is beyond 2^31 - 1");
    return (int32_t)x;
}

// The workspace of a call: the given tensor from its first 256-byte boundary, or a
// new one.  `keep` holds it until the call has been enqueued.
void *workspace(PyObject *o, size_t need, const Call &c, at::Tensor &keep, size_t &bytes) {
    if (none(o)) {
        keep = c.empty({(int64_t)need + 256}, at::kByte);
    } else {
        keep = tensor(o, "workspace");
        on_device(keep, "workspace", c.dev);
        if (!keep.is_contiguous()) refuse("workspace must be contiguous");
    }
    const uintptr_t start = (uintptr_t)keep.data_ptr(), base = (start + 255) & ~(uintptr_t)255;
    const int64_t avail = (int64_t)keep.nbytes() - (int64_t)(base - start);
    if (avail < (int64_t)need)
        refuse("workspace too small: need ", need, " bytes from its first 256-byte boundary, have ",
               avail < 0 ? 0 : avail);
    bytes = (size_t)avail;
    return (void *)base;
}

void check(hga_status s, const char *what) {
    if (s == HGA_OK) return;
    if (s == HGA_ERR_CUDA)
        refuse(what, ": ", hga_status_string(s), " (cuda error ", hga_last_cuda_error(), ")");
    refuse(what, ": ", hga_status_string(s));
}

PyObject *wrap(const at::Tensor &t) { return THPVariable_Wrap(t); }
PyObject *wrap_or_none(const at::Tensor &t) {
    if (t.defined()) return THPVariable_Wrap(t);
    Py_RETURN_NONE;
}

// HGARope(rotary_dim, theta, layout, scaling, factor, original_len, beta_fast,
// beta_slow, magnitude)
hga_rope rope_of(PyObject *o, int64_t D) {
    if (!PyTuple_Check(o) || PyTuple_GET_SIZE(o) != 9) refuse("rope must be an HGARope");
    auto at = [&](int i) { return PyTuple_GET_ITEM(o, i); };
    auto pick = [&](int i, const char *what, std::initializer_list<const char *> names) {
        int k = 0;
        for (const char *n : names) {
            if (PyUnicode_Check(at(i)) && PyUnicode_CompareWithASCIIString(at(i), n) == 0) return k;
            ++k;
        }
        std::string all;
        for (const char *n : names) all += std::string(all.empty() ? "" : ", ") + n;
        refuse(what, " must be one of ", all);
    };
    hga_rope r = {};
    r.rotary_dim = none(at(0)) ? (int32_t)D : (int32_t)whole(at(0), "rotary_dim");
    r.theta = real(at(1));
    r.layout = pick(2, "layout", {"half", "interleaved"});
    r.scaling = pick(3, "scaling", {"none", "linear", "yarn"});
    r.factor = real(at(4));
    r.original_len = (int32_t)whole(at(5), "original_len");
    r.beta_fast = real(at(6));
    r.beta_slow = real(at(7));
    r.magnitude = real(at(8));
    return r;
}

// [tokens, H, D] or [B, T, H, D]: its leading shape and heads.
struct Rows {
    at::IntArrayRef lead;
    int64_t H, D;
    Rows(const at::Tensor &t, const char *name) {
        if (t.dim() != 3 && t.dim() != 4) refuse(name, " must be [tokens, H, D] or [B, T, H, D]");
        lead = t.sizes().slice(0, t.dim() - 2);
        H = t.size(-2);
        D = t.size(-1);
    }
};

at::DimVector with(at::IntArrayRef lead, int64_t H, int64_t D) {
    at::DimVector s(lead.begin(), lead.end());
    s.push_back(H);
    s.push_back(D);
    return s;
}

// Elements between the tokens of a tensor whose heads are adjacent rows of D and
// whose tokens are evenly spaced (a view of a fused buffer).
int64_t token_stride(const at::Tensor &t, const char *name, at::IntArrayRef lead, int64_t H, int64_t D,
                     at::ScalarType dt, const Call &c) {
    on_device(t, name, c.dev);
    if (t.scalar_type() != dt)
        refuse(name, " has dtype ", c10::toString(t.scalar_type()), ", expected ", c10::toString(dt));
    const size_t k = lead.size();
    if (t.dim() != (int64_t)k + 2 || t.sizes().slice(0, k) != lead || t.size(-2) != H || t.size(-1) != D)
        refuse(name, " has shape ", text(t.sizes()), ", expected ", text(with(lead, H, D)));
    const at::IntArrayRef s = t.strides();
    if ((D > 1 && s[k + 1] != 1) || (H > 1 && s[k] != D))
        refuse(name, ": heads must be adjacent rows of ", D, " (strides ", text(s), ")");
    if (k == 1) return lead[0] > 1 ? s[0] : H * D;
    if (lead[0] > 1 && lead[1] > 1 && s[0] != lead[1] * s[1])
        refuse(name, ": tokens must be evenly spaced (strides ", text(s), ")");
    return lead[1] > 1 ? s[1] : lead[0] > 1 ? s[0] : H * D;
}

hga_dims token_dims(at::IntArrayRef lead, int64_t Hq, int64_t Hkv, int64_t D, int code) {
    hga_dims d = {};
    d.B = lead.size() == 2 ? size32(lead[0], "B") : 1;
    d.T = size32(lead.back(), "tokens");
    if (lead.size() == 2 && lead[0] == 0) d.B = 1, d.T = 0;
    d.Hq = size32(Hq, "Hq");
    d.Hkv = size32(Hkv, "Hkv");
    d.D = size32(D, "D");
    d.dtype = code;
    return d;
}

// ---------------------------------------------------------------- calls --

// lens, new_tokens, free_pages, free_count, block_table, page_size, n_slots, release,
// lens_out, free_count_out, cu_tokens, granted, slot, pos, workspace, stream
PyObject *plan(PyObject *const *a) {
    const at::Tensor &table = tensor(a[4], "block_table");
    if (table.dim() != 2) refuse("block_table must be [B, max_pages]");
    const Call c(table, a[15]);
    const int64_t B = table.size(0), M = table.size(1);
    const int64_t P = tensor(a[2], "free_pages").numel();
    const int32_t n = (int32_t)whole(a[6], "n_slots");
    hga_paged_dims d = {};
    d.B = size32(B, "B");
    d.num_pages = size32(P, "free_pages");
    d.page_size = (int32_t)whole(a[5], "page_size");
    d.max_pages = size32(M, "max_pages");
    hga_paged_plan_io io = {};
    io.lens = ints(a[0], "lens", {B}, c);
    io.new_tokens = ints(a[1], "new_tokens", {B}, c);
    io.free_pages = ints(a[2], "free_pages", {P}, c);
    io.free_count = ints(a[3], "free_count", {1}, c);
    io.block_table = ints(a[4], "block_table", {B, M}, c);
    io.release = ints_or_null(a[7], "release", {B}, c);
    const int64_t size[6] = {B, 1, B + 1, B, n, n};
    static const char *const name[6] = {"lens_out", "free_count_out", "cu_tokens", "granted", "slot",
                                        "pos"};
    int32_t **const at_[6] = {&io.lens_out, &io.free_count_out, &io.cu_tokens,
                              &io.granted,  &io.slot,           &io.pos};
    // one allocation for what the caller does not bring
    at::Tensor out[6];
    std::vector<int64_t> missing;
    for (int i = 0; i < 6; ++i)
        if (none(a[8 + i])) missing.push_back(size[i]);
    std::vector<at::Tensor> parts;
    if (!missing.empty())
        parts = c.empty({std::accumulate(missing.begin(), missing.end(), (int64_t)0)}, at::kInt)
                    .split_with_sizes(missing);
    size_t used = 0;
    for (int i = 0; i < 6; ++i) {
        if (none(a[8 + i])) {
            out[i] = std::move(parts[used++]);
            *at_[i] = out[i].data_ptr<int32_t>();
        } else {
            *at_[i] = ints(a[8 + i], name[i], {size[i]}, c);
            out[i] = THPVariable_Unpack(a[8 + i]);
        }
    }
    at::Tensor keep;
    size_t bytes = 0;
    void *ws = workspace(a[14], hga_paged_plan_workspace(d.B, n), c, keep, bytes);
    check(hga_paged_plan(&d, &io, n, ws, bytes, c.stream), "hga_paged_plan");
    return Py_BuildValue("{s:N,s:N,s:N,s:N,s:N,s:N}", "lens", wrap(out[0]), "free_count", wrap(out[1]),
                         "cu_tokens", wrap(out[2]), "granted", wrap(out[3]), "slot", wrap(out[4]), "pos",
                         wrap(out[5]));
}

// q, k, v, pos, rope, q_weight, k_weight, eps, k_pages, v_pages, slot, q_out, k_out,
// v_out, stream
PyObject *qk(PyObject *const *a) {
    const at::Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k");
    const Rows rq(q, "q"), rk(k, "k");
    const int code = dtype_code(q);
    const at::ScalarType dt = q.scalar_type();
    const int64_t D = rq.D, Hkv = rk.H;
    const hga_rope rope = rope_of(a[4], D);
    const Call c(q, a[14]);
    hga_qk_io io = {};
    io.q = q.data_ptr();
    io.k = k.data_ptr();
    io.q_stride = token_stride(q, "q", rq.lead, rq.H, D, dt, c);
    io.k_stride = token_stride(k, "k", rq.lead, Hkv, D, dt, c);
    const bool has_v = !none(a[2]);
    if (has_v) {
        const at::Tensor &v = tensor(a[2], "v");
        io.v_stride = token_stride(v, "v", rq.lead, Hkv, D, dt, c);
        io.v = v.data_ptr();
    }
    io.pos = ints_or_null(a[3], "pos", rq.lead, c);
    if (!io.pos && rope.rotary_dim && none(a[3])) refuse("pos is needed with a rotation");
    io.q_weight = dense_or_null(a[5], "q_weight", {D}, dt, c);
    io.k_weight = dense_or_null(a[6], "k_weight", {D}, dt, c);
    io.eps = real(a[7]);
    const bool paged = !none(a[8]) || !none(a[9]);
    if (paged) {
        if (none(a[8]) || none(a[10]) || none(a[9]) == has_v)
            refuse("k_pages, v_pages (with v) and slot come together");
        const at::Tensor &kp = tensor(a[8], "k_pages");
        if (kp.dim() != 4) refuse("k_pages must be [num_pages, page_size, Hkv, D]");
        const int64_t shape[4] = {kp.size(0), kp.size(1), Hkv, D};
        io.k_pages = dense(a[8], "k_pages", shape, dt, c);
        io.v_pages = dense_or_null(a[9], "v_pages", shape, dt, c);
        io.slot = ints(a[10], "slot", rq.lead, c);
        io.num_slots = shape[0] * shape[1];
    }
    if (!has_v && !none(a[13])) refuse("v_out without v");
    const at::DimVector kv = with(rq.lead, Hkv, D);
    at::Tensor qo = output(a[11], "q_out", q.sizes(), dt, c), ko, vo;
    if (!paged || !none(a[12])) ko = output(a[12], "k_out", kv, dt, c);
    if (has_v && (!paged || !none(a[13]))) vo = output(a[13], "v_out", kv, dt, c);
    io.q_out = qo.data_ptr();
    io.k_out = ko.defined() ? ko.data_ptr() : nullptr;
    io.v_out = vo.defined() ? vo.data_ptr() : nullptr;
    const hga_dims d = token_dims(rq.lead, rq.H, Hkv, D, code);
    check(hga_qk_norm_rope(&d, &rope, &io, c.stream), "hga_qk_norm_rope");
    return Py_BuildValue("(NNN)", wrap(qo), wrap_or_none(ko), wrap_or_none(vo));
}

// q, k, d_q, d_k, pos, rope, q_weight, k_weight, eps, d_v, dq, dk, dv, workspace, stream
PyObject *qk_backward(PyObject *const *a) {
    const at::Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k"), &dqi = tensor(a[2], "d_q");
    const Rows rq(q, "q"), rk(k, "k");
    const int code = dtype_code(q);
    const at::ScalarType dt = q.scalar_type(), gt = dqi.scalar_type();
    const int64_t D = rq.D, Hkv = rk.H;
    const hga_rope rope = rope_of(a[5], D);
    const Call c(q, a[14]);
    if (gt != at::kFloat && gt != dt)
        refuse("d_q has dtype ", c10::toString(gt), ", expected Float or ", c10::toString(dt));
    const at::DimVector kv = with(rq.lead, Hkv, D);
    hga_qk_grad_io io = {};
    io.q = q.data_ptr();
    io.k = k.data_ptr();
    io.q_stride = token_stride(q, "q", rq.lead, rq.H, D, dt, c);
    io.k_stride = token_stride(k, "k", rq.lead, Hkv, D, dt, c);
    io.pos = ints_or_null(a[4], "pos", rq.lead, c);
    if (!io.pos && rope.rotary_dim && none(a[4])) refuse("pos is needed with a rotation");
    io.q_weight = dense_or_null(a[6], "q_weight", {D}, dt, c);
    io.k_weight = dense_or_null(a[7], "k_weight", {D}, dt, c);
    io.eps = real(a[8]);
    io.d_q = dense(a[2], "d_q", q.sizes(), gt, c);
    io.d_k = dense(a[3], "d_k", kv, gt, c);
    io.d_v = dense_or_null(a[9], "d_v", kv, gt, c);
    io.grad_dtype = gt == at::kFloat ? HGA_F32 : code;
    const bool has_v = !none(a[9]);
    if (!has_v && !none(a[12])) refuse("dv without d_v");
    auto grad = [&](PyObject *o, const char *name, at::IntArrayRef shape) {
        return none(o) ? c.empty(shape, dt) : tensor(o, name);
    };
    const at::Tensor dq = grad(a[10], "dq", q.sizes()), dk = grad(a[11], "dk", kv);
    at::Tensor dv, dqw, dkw, keep;
    if (has_v) dv = grad(a[12], "dv", kv);
    io.dq = dq.data_ptr();
    io.dk = dk.data_ptr();
    io.dq_stride = token_stride(dq, "dq", rq.lead, rq.H, D, dt, c);
    io.dk_stride = token_stride(dk, "dk", rq.lead, Hkv, D, dt, c);
    if (has_v) {
        io.dv_stride = token_stride(dv, "dv", rq.lead, Hkv, D, dt, c);
        io.dv = dv.data_ptr();
    }
    if (io.q_weight) dqw = c.empty({D}, at::kFloat), io.d_q_weight = dqw.data_ptr<float>();
    if (io.k_weight) dkw = c.empty({D}, at::kFloat), io.d_k_weight = dkw.data_ptr<float>();
    const hga_dims d = token_dims(rq.lead, rq.H, Hkv, D, code);
    size_t bytes = 0;
    void *ws = nullptr;
    if (io.q_weight || io.k_weight || !none(a[13]))
        ws = workspace(a[13], hga_qk_norm_rope_backward_workspace(&d), c, keep, bytes);
    check(hga_qk_norm_rope_backward(&d, &rope, &io, ws, bytes, c.stream), "hga_qk_norm_rope_backward");
    return Py_BuildValue("(NNNNN)", wrap(dq), wrap(dk), wrap_or_none(dv), wrap_or_none(dqw),
                         wrap_or_none(dkw));
}

// q, k_pages, v_pages, block_table, lens, window, sinks, scale, out, want_lse, lse,
// workspace, stream
PyObject *decode(PyObject *const *a) {
    const at::Tensor &q = tensor(a[0], "q"), &kp = tensor(a[1], "k_pages"),
                     &table = tensor(a[3], "block_table");
    if (q.dim() != 3) refuse("q must be [B, Hq, D]");
    if (kp.dim() != 4) refuse("k_pages must be [num_pages, page_size, Hkv, D]");
    if (table.dim() != 2) refuse("block_table must be [B, max_pages]");
    const int code = dtype_code(q);
    const at::ScalarType dt = q.scalar_type();
    const Call c(q, a[12]);
    const int64_t B = q.size(0), Hq = q.size(1), D = q.size(2);
    const int64_t shape[4] = {kp.size(0), kp.size(1), kp.size(2), D};
    hga_paged_dims d = {};
    d.B = size32(B, "B");
    d.Hq = size32(Hq, "Hq");
    d.Hkv = size32(shape[2], "Hkv");
    d.D = size32(D, "D");
    d.dtype = code;
    d.num_pages = size32(shape[0], "num_pages");
    d.page_size = size32(shape[1], "page_size");
    d.max_pages = size32(table.size(1), "max_pages");
    const void *pq = dense(a[0], "q", {B, Hq, D}, dt, c), *pk = dense(a[1], "k_pages", shape, dt, c),
               *pv = dense(a[2], "v_pages", shape, dt, c);
    const int32_t *pt = ints(a[3], "block_table", {B, table.size(1)}, c), *pl = ints(a[4], "lens", {B}, c);
    const int32_t window = (int32_t)whole(a[5], "window"), sinks = (int32_t)whole(a[6], "sinks");
    const double scale = real(a[7]);
    const at::Tensor out = output(a[8], "out", {B, Hq, D}, dt, c);
    at::Tensor lse, keep;
    if (!none(a[10]) || truth(a[9])) lse = output(a[10], "lse", {B, Hq}, at::kFloat, c);
    size_t bytes = 0;
    void *ws = workspace(a[11], hga_paged_decode_workspace(&d), c, keep, bytes);
    check(hga_paged_decode(&d, pq, pk, pv, pt, pl, window, sinks, scale, out.data_ptr(),
                           lse.defined() ? lse.data_ptr<float>() : nullptr, ws, bytes, c.stream),
          "hga_paged_decode");
    if (!lse.defined()) return wrap(out);
    return Py_BuildValue("(NN)", wrap(out), wrap(lse));
}

// Runs a call with its argument count checked and every C++ exception turned into a
// Python one.
template <PyObject *(*F)(PyObject *const *), Py_ssize_t N>
PyObject *entry(PyObject *, PyObject *const *args, Py_ssize_t n) {
    if (n != N) {
        PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", N, n);
        return nullptr;
    }
    try {
        // new tensors and views of them take no part in automatic differentiation
        const at::AutoDispatchBelowADInplaceOrView below;
        return F(args);
    } catch (const Refused &e) {
        PyErr_SetString(g_error ? g_error : PyExc_RuntimeError, e.what());
    } catch (const Raised &) {
    } catch (python_error &e) {
        e.restore();
    } catch (const c10::OutOfMemoryError &e) {
        PyErr_SetString(g_out_of_memory ? g_out_of_memory : PyExc_MemoryError, e.what_without_backtrace());
    } catch (const c10::Error &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what_without_backtrace());
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    } catch (...) {
        PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
    }
    return nullptr;
}

// set_errors(HGAError, OutOfMemoryError): the classes that refusals raise
PyObject *set_errors(PyObject *, PyObject *args) {
    PyObject *e, *m;
    if (!PyArg_ParseTuple(args, "OO", &e, &m)) return nullptr;
    Py_XSETREF(g_error, Py_NewRef(e));
    Py_XSETREF(g_out_of_memory, Py_NewRef(m));
    Py_RETURN_NONE;
}

#define HGA_FAST(f, n) (PyCFunction)(void (*)(void))entry<f, n>, METH_FASTCALL, nullptr
PyMethodDef kMethods[] = {{"plan", HGA_FAST(plan, 16)},
                          {"qk", HGA_FAST(qk, 15)},
                          {"qk_backward", HGA_FAST(qk_backward, 15)},
                          {"decode", HGA_FAST(decode, 13)},
                          {"set_errors", set_errors, METH_VARARGS, nullptr},
                          {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_paged", nullptr, -1, kMethods,
                       nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__paged(void) { return PyModule_Create(&kModule); }
