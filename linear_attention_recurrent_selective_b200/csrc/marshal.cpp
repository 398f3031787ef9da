// marshal.cpp -- native argument marshalling of the Python binding (module _marshal).
//
// The same work as the ctypes calls in ssu.py -- check that tensors are CUDA tensors of one
// device with the expected types, shapes and layouts, read their sizes and strides, and pass
// raw pointers and the stream to a C entry point of libssu -- for the entry points whose
// kernels run for a few microseconds, where a dozen tensors' checks in Python would take
// longer than the call. No arithmetic happens here. Every function takes the address of its
// entry point (from the loaded library) and the stream (None: the current one of the tensors'
// device) first, raises ValueError for arguments that do not fit and returns the ssu_status.
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>

#include <initializer_list>
#include <stdexcept>
#include <string>

#include "ssu.h"

namespace {

using at::ScalarType;
using at::Tensor;

[[noreturn]] void refuse(const std::string &what) { throw std::invalid_argument(what); }

// The positional arguments of a call, read in order.
struct Reader {
    PyObject *const *args;
    Py_ssize_t left;
    int device = -1;

    PyObject *next()
    {
        if (left-- <= 0)
            refuse("too few arguments");
        return *args++;
    }
    const Tensor *optional(const char *name)
    {
        PyObject *const o = next();
        if (o == Py_None)
            return nullptr;
        if (!THPVariable_Check(o))
            refuse(std::string(name) + " must be a tensor");
        const Tensor &t = THPVariable_Unpack(o);
        if (!t.is_cuda())
            refuse(std::string(name) + " must be a CUDA tensor, got one on " + t.device().str());
        if (device < 0)
            device = t.get_device();
        else if (t.get_device() != device)
            refuse(std::string(name) + " is on " + t.device().str() + ", other tensors on cuda:" +
                   std::to_string(device));
        return &t;
    }
    const Tensor &tensor(const char *name)
    {
        const Tensor *const t = optional(name);
        if (!t)
            refuse(std::string(name) + " is missing");
        return *t;
    }
    int64_t integer(int64_t none)
    {
        PyObject *const o = next();
        if (o == Py_None)
            return none;
        const long long v = PyLong_AsLongLong(o);
        if (v == -1 && PyErr_Occurred()) {
            PyErr_Clear();
            refuse("expected a whole number");
        }
        return v;
    }
    int64_t size()                              // -1: not given
    {
        const int64_t v = integer(-1);
        if (v < 0 && args[-1] != Py_None)
            refuse("a size is negative: " + std::to_string(v));
        return v;
    }
    int32_t int32(int64_t none)
    {
        const int64_t v = integer(none);
        if (v != (int32_t)v)
            refuse("a size does not fit 32 bits: " + std::to_string(v));
        return (int32_t)v;
    }
    int truth()
    {
        const int v = PyObject_IsTrue(next());
        if (v < 0) {
            PyErr_Clear();
            refuse("expected a truth value");
        }
        return v;
    }
};

int32_t fit32(int64_t v, const char *name)
{
    if (v != (int32_t)v)
        refuse(std::string(name) + " does not fit 32 bits: " + std::to_string(v));
    return (int32_t)v;
}

int code(const Tensor &t, const char *name)
{
    switch (t.scalar_type()) {
    case ScalarType::Float: return SSU_F32;
    case ScalarType::Half: return SSU_F16;
    case ScalarType::BFloat16: return SSU_BF16;
    default: refuse(std::string(name) + " is not fp32, fp16 or bf16");
    }
}

bool has_shape(const Tensor &t, std::initializer_list<int64_t> shape)
{
    return t.sizes() == at::IntArrayRef(shape);
}

std::string text(at::IntArrayRef v)
{
    std::string s = "[";
    for (size_t i = 0; i < v.size(); ++i)
        s += (i ? ", " : "") + std::to_string(v[i]);
    return s + "]";
}

// Pointer of a contiguous tensor of a shape and type; a missing one stays NULL.
template <typename P = void>
P *dense(const Tensor *t, const char *name, std::initializer_list<int64_t> shape, ScalarType type)
{
    if (!t)
        return nullptr;
    if (t->scalar_type() != type || !has_shape(*t, shape) || !t->is_contiguous())
        refuse(std::string(name) + " must be contiguous " + text(at::IntArrayRef(shape)) + " of " +
               c10::toString(type) + ", got " + text(t->sizes()) + " of " +
               c10::toString(t->scalar_type()));
    return static_cast<P *>(t->data_ptr());
}

const int32_t *indices(const Tensor *t, const char *name, std::initializer_list<int64_t> shape)
{
    return dense<const int32_t>(t, name, shape, ScalarType::Int);
}

// Lists of accepted nodes [rows, most]: a missing one is NULL, one of no columns is not. It has
// no elements and torch no address for it, so it gets that of another tensor, never read.
int32_t *node_lists(const Tensor *t, const char *name, int64_t rows, int64_t most,
                    const Tensor &other)
{
    int32_t *const p = dense<int32_t>(t, name, {rows, most}, ScalarType::Int);
    return t && !p ? static_cast<int32_t *>(other.data_ptr()) : p;
}

void same_type(const Tensor *t, const Tensor &as, const char *name, const char *other)
{
    if (t && t->scalar_type() != as.scalar_type())
        refuse(std::string(name) + " must have " + other + "'s dtype");
}

// Elements between consecutive tokens of t, whose shape is `lead` (1: rows, 2: rows and
// tokens) leading sizes and then those of a token: each token is dense, and the tokens of all
// rows are equally far apart (slices of wider rows).
int64_t tokens(const Tensor &t, const char *name, std::initializer_list<int64_t> shape, int lead)
{
    if (!has_shape(t, shape))
        refuse(std::string(name) + " must be " + text(at::IntArrayRef(shape)) + ", got " +
               text(t.sizes()));
    const auto size = t.sizes(), step = t.strides();
    int64_t far = 1;
    for (int i = (int)size.size() - 1; i >= lead; --i) {
        if (size[i] != 1 && step[i] != far)
            refuse(std::string(name) + ": a token's elements must be dense");
        far *= size[i];
    }
    if (lead == 2 && size[1] > 1) {
        if (size[0] > 1 && step[0] != size[1] * step[1])
            refuse(std::string(name) + ": rows must follow one another, T tokens apart");
        return step[1];
    }
    return size[0] > 1 ? step[0] : far;
}

// Elements of storage from a tensor's first element to its last one.
int64_t extent(const Tensor &t)
{
    if (t.numel() == 0)
        return 0;
    int64_t n = 1;
    for (int64_t i = 0; i < t.dim(); ++i)
        n += (t.size(i) - 1) * t.stride(i);
    return n;
}

// A conv pool: the tensor must reach over every slot's taps.
struct ConvPool {
    void *p = nullptr;
    int64_t slot = 0, c = 0, k = 0;
    int32_t P = 0;
};

ConvPool conv_pool(const Tensor *pool, const Tensor &xbc, int64_t channels, int32_t width,
                   int64_t slot, int64_t c, int64_t k, int64_t P)
{
    ConvPool r;
    if (width <= 1 || !pool) {
        r.P = P < 0 ? INT32_MAX : fit32(P, "P");
        return r;
    }
    same_type(pool, xbc, "conv_state", "xbc");
    if (P < 0)
        P = pool->dim() == 3 ? pool->size(0) : pool->numel() / (slot > 0 ? slot : 1);
    r.P = fit32(P, "P");
    const __int128 last = (__int128)(P - 1) * slot + (__int128)(channels - 1) * c +
                          (__int128)(width - 2) * k;
    if (P > 0 && last >= extent(*pool))
        refuse("conv_state does not hold " + std::to_string(P) + " slots with these strides");
    r.p = pool->data_ptr();
    r.slot = slot;
    r.c = c;
    r.k = k;
    return r;
}

ssu_stream_t stream_of(PyObject *stream, int device)
{
    if (stream == Py_None)
        return reinterpret_cast<ssu_stream_t>(
            c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)device).stream());
    PyObject *const raw = PyObject_GetAttrString(stream, "cuda_stream");
    PyObject *const index = raw ? PyObject_GetAttrString(stream, "device_index") : nullptr;
    const unsigned long long v = index ? PyLong_AsUnsignedLongLong(raw) : 0;
    const long d = index ? PyLong_AsLong(index) : -1;
    const bool bad = !index || PyErr_Occurred();
    Py_XDECREF(raw);
    Py_XDECREF(index);
    if (bad) {
        PyErr_Clear();
        refuse("stream must be a torch.cuda.Stream");
    }
    if (d != device)
        refuse("stream of cuda:" + std::to_string(d) + " given for tensors on cuda:" +
               std::to_string(device));
    return reinterpret_cast<ssu_stream_t>((uintptr_t)v);
}

// Calls an entry point without the interpreter's lock, as ctypes does: a launch into a full
// queue waits for the device, which may itself wait for a host function of another thread.
struct Unlocked {
    PyThreadState *const thread = PyEval_SaveThread();
    ~Unlocked() { PyEval_RestoreThread(thread); }
};

template <typename Fn, typename... Args> int unlocked(Fn fn, Args... args)
{
    const Unlocked on;
    return fn(args...);
}

// Runs `body` (Reader, entry point, stream argument) and turns what it throws into a
// Python exception.
template <typename Fn, typename Body>
PyObject *guarded(PyObject *const *args, Py_ssize_t n, const Body &body)
{
    try {
        Reader r{args, n};
        const unsigned long long address = PyLong_AsUnsignedLongLong(r.next());
        if (PyErr_Occurred())
            return nullptr;
        PyObject *const stream = r.next();
        return PyLong_FromLong(body(r, reinterpret_cast<Fn>((uintptr_t)address), stream));
    } catch (const std::invalid_argument &e) {
        PyErr_SetString(PyExc_ValueError, e.what());
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

// (pointer, channels) of an output of the convolution; a missing one has no channels.
int32_t conv_out(const Tensor *t, const char *name, const Tensor &xbc, void *&p)
{
    p = nullptr;
    if (!t)
        return 0;
    if (t->scalar_type() != xbc.scalar_type() || t->dim() < 3 || t->size(0) != xbc.size(0) ||
        t->size(1) != xbc.size(1) || !t->is_contiguous())
        refuse(std::string(name) + " must be contiguous [batch, T, ...] in xbc's dtype");
    p = t->data_ptr();
    int64_t n = 1;
    for (int64_t i = 2; i < t->dim(); ++i)
        n *= t->size(i);
    return fit32(n, name);
}

PyObject *conv_prefill(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    return guarded<decltype(&ssu_conv_prefill)>(args, n, [](Reader &r, auto fn, PyObject *stream) {
        const Tensor &xbc = r.tensor("xbc"), &weight = r.tensor("conv_weight");
        const Tensor *const pool = r.optional("conv_state");
        const Tensor *const x = &r.tensor("x");
        const Tensor *const B = r.optional("B"), *const C = r.optional("C");
        const Tensor *const bias = r.optional("conv_bias");
        const Tensor *const idx = r.optional("state_indices");
        const Tensor *const len = r.optional("context_lengths");
        const Tensor *const parents = r.optional("parent_ids");
        const Tensor *const err = r.optional("err_flags");
        const int32_t width = r.int32(0);
        const int64_t cs = r.integer(0), cc = r.integer(0), ck = r.integer(0);
        const int silu = r.truth(), update = r.truth();
        const int64_t P = r.size();
        if (xbc.dim() != 3)
            refuse("xbc must be [batch, T, channels]");
        const int64_t b = xbc.size(0), T = xbc.size(1), ch = xbc.size(2);
        const int32_t active = r.int32(b);
        const int64_t ld = tokens(xbc, "xbc", {b, T, ch}, 2);
        void *px, *pB, *pC;
        const int32_t xd = conv_out(x, "x", xbc, px), bd = conv_out(B, "B", xbc, pB);
        const int32_t cd = conv_out(C, "C", xbc, pC);
        if (bd != cd || xd + 2 * (int64_t)bd != ch)
            refuse("x, B and C hold " + std::to_string(xd) + ", " + std::to_string(bd) + " and " +
                   std::to_string(cd) + " channels, xbc " + std::to_string(ch));
        const ConvPool cp = conv_pool(pool, xbc, ch, width, cs, cc, ck, P);
        const ScalarType type = xbc.scalar_type();
        const c10::cuda::CUDAGuard on((c10::DeviceIndex)r.device);
        return unlocked(
            fn, xbc.data_ptr(), code(xbc, "xbc"), ld,
            dense(&weight, "conv_weight", {ch, width}, type),
            dense(bias, "conv_bias", {ch}, type), cp.p, cp.slot, cp.c, cp.k, width, silu,
            cp.P, px, pB, pC, indices(idx, "state_indices", {b}),
            indices(len, "context_lengths", {b}), indices(parents, "parent_ids", {b, T}),
            update, fit32(b, "batch"), active, fit32(T, "T"), xd, bd,
            dense<int32_t>(err, "err_flags", {1}, ScalarType::Int),
            stream_of(stream, r.device));
    });
}

PyObject *conv_replay(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    return guarded<decltype(&ssu_conv_replay)>(args, n, [](Reader &r, auto fn, PyObject *stream) {
        const Tensor &xbc = r.tensor("xbc");
        const Tensor *const pool = r.optional("conv_state");
        const Tensor &acc = r.tensor("accepted_lengths");
        const Tensor *const idx = r.optional("state_indices");
        const Tensor *const ids = r.optional("accepted_node_ids");
        const Tensor *const err = r.optional("err_flags");
        const int32_t width = r.int32(0);
        const int64_t cs = r.integer(0), cc = r.integer(0), ck = r.integer(0), P = r.size();
        if (xbc.dim() != 3 || (ids && ids->dim() != 2))
            refuse("xbc must be [batch, T, channels], accepted_node_ids [batch, maxAcceptLen]");
        const int64_t b = xbc.size(0), T = xbc.size(1), ch = xbc.size(2);
        const int64_t most = ids ? ids->size(1) : 0;
        const int32_t active = r.int32(b);
        const int64_t ld = tokens(xbc, "xbc", {b, T, ch}, 2);
        const ConvPool cp = conv_pool(pool, xbc, ch, width, cs, cc, ck, P);
        const c10::cuda::CUDAGuard on((c10::DeviceIndex)r.device);
        return unlocked(
            fn, xbc.data_ptr(), code(xbc, "xbc"), ld, cp.p, cp.slot, cp.c, cp.k, width,
            cp.P,
            indices(&acc, "accepted_lengths", {b}), indices(idx, "state_indices", {b}),
            fit32(b, "batch"), active, fit32(T, "T"), fit32(ch, "channels"),
            node_lists(ids, "accepted_node_ids", b, most, acc), fit32(most, "maxAcceptLen"),
            dense<int32_t>(err, "err_flags", {1}, ScalarType::Int),
            stream_of(stream, r.device));
    });
}

// What scan_prefill and scan_decode share.
struct Scan {
    const Tensor *x, *dt, *A, *B, *C, *state, *out, *D, *z, *bias, *idx, *err;
    int64_t b, T, ch, G, N, per, stride;
    int64_t ldx, lddt, ldz, ldb, ldc;
    int32_t P, active;
    int softplus, lead;

    // Tensors in the order x, dt, A, B, C, state, out, D, z, dt_bias, state_indices,
    // err_flags; then dt_softplus, slot_stride, P, active_batch.
    Scan(Reader &r, int lead_) : lead(lead_)
    {
        x = &r.tensor("x");
        dt = &r.tensor("dt");
        A = &r.tensor("A");
        B = &r.tensor("B");
        C = r.optional("C");
        state = &r.tensor("state");
        out = r.optional("out");
        D = r.optional("D");
        z = r.optional("z");
        bias = r.optional("dt_bias");
        idx = r.optional("state_indices");
        err = r.optional("err_flags");
        if (x->dim() != lead + 1 || B->dim() != lead + 2)
            refuse(lead == 2 ? "x must be [batch, T, channels], B [batch, T, groups, dstate]"
                             : "x must be [batch, channels], B [batch, groups, dstate]");
        b = x->size(0);
        T = lead == 2 ? x->size(1) : 1;
        ch = x->size(lead);
        G = B->size(lead);
        N = B->size(lead + 1);
        per = G * N;
        softplus = r.truth();
        stride = r.size();
        int64_t slots = r.size();
        active = r.int32(b);
        same_type(z, *x, "z", "x");
        same_type(C, *B, "C", "B");
        same_type(out, *x, "out", "x");
        ldx = rows(x, "x");
        lddt = rows(dt, "dt");
        ldz = z ? rows(z, "z") : 0;
        ldb = states(B, "B");
        ldc = C ? states(C, "C") : per;
        if (out && (out->sizes() != x->sizes() || !out->is_contiguous()))
            refuse("out must be contiguous, in x's shape");
        if (state->dim() == 3) {
            if (state->size(1) != ch || state->size(2) != N || state->stride(1) != N ||
                state->stride(2) != 1)
                refuse("state must be [P, " + std::to_string(ch) + ", " + std::to_string(N) +
                       "], contiguous inside a slot");
            stride = stride < 0 ? state->stride(0) : stride;
            slots = slots < 0 ? state->size(0) : slots;
        } else {
            if (state->dim() != 1 || !state->is_contiguous())
                refuse("state must be [P, channels, dstate] or flat contiguous storage");
            stride = stride < 0 ? ch * N : stride;
            slots = slots < 0 ? state->numel() / (stride > 0 ? stride : 1) : slots;
        }
        P = fit32(slots, "P");
        if (P > 0 && (__int128)(P - 1) * stride + ch * N > extent(*state))
            refuse("state does not hold " + std::to_string(P) + " slots of stride " +
                   std::to_string(stride));
    }
    int64_t rows(const Tensor *t, const char *name) const
    {
        return lead == 2 ? tokens(*t, name, {b, T, ch}, 2) : tokens(*t, name, {b, ch}, 1);
    }
    int64_t states(const Tensor *t, const char *name) const
    {
        return lead == 2 ? tokens(*t, name, {b, T, G, N}, 2) : tokens(*t, name, {b, G, N}, 1);
    }
    static void *ptr(const Tensor *t) { return t ? t->data_ptr() : nullptr; }
    const float *f32(const Tensor *t, const char *name) const
    {
        return dense<const float>(t, name, {ch}, ScalarType::Float);
    }
};

PyObject *scan_prefill_(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    return guarded<decltype(&scan_prefill)>(args, n, [](Reader &r, auto fn, PyObject *stream) {
        const Scan s(r, 2);
        const Tensor *const len = r.optional("context_lengths");
        const int update = r.truth();
        const c10::cuda::CUDAGuard on((c10::DeviceIndex)r.device);
        return unlocked(
            fn, s.x->data_ptr(), code(*s.x, "x"), s.ldx, s.dt->data_ptr(),
            code(*s.dt, "dt"), s.lddt,
            dense<const float>(s.A, "A", {s.ch, s.N}, ScalarType::Float), s.B->data_ptr(),
            Scan::ptr(s.C), code(*s.B, "B"), s.ldb, s.ldc, s.f32(s.bias, "dt_bias"),
            s.f32(s.D, "D"), Scan::ptr(s.z), s.ldz, s.state->data_ptr(),
            code(*s.state, "state"), s.stride, s.P, Scan::ptr(s.out),
            indices(s.idx, "state_indices", {s.b}), indices(len, "context_lengths", {s.b}),
            update, fit32(s.b, "batch"), s.active, fit32(s.T, "T"), fit32(s.ch, "channels"),
            fit32(s.G, "groups"), fit32(s.N, "dstate"), s.softplus,
            dense<int32_t>(s.err, "err_flags", {1}, ScalarType::Int),
            stream_of(stream, r.device));
    });
}

PyObject *scan_decode_(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    return guarded<decltype(&scan_decode)>(args, n, [](Reader &r, auto fn, PyObject *stream) {
        const Scan s(r, 1);
        const c10::cuda::CUDAGuard on((c10::DeviceIndex)r.device);
        return unlocked(
            fn, s.x->data_ptr(), code(*s.x, "x"), s.ldx, s.dt->data_ptr(),
            code(*s.dt, "dt"), s.lddt,
            dense<const float>(s.A, "A", {s.ch, s.N}, ScalarType::Float), s.B->data_ptr(),
            Scan::ptr(s.C), code(*s.B, "B"), s.ldb, s.ldc, s.f32(s.bias, "dt_bias"),
            s.f32(s.D, "D"), Scan::ptr(s.z), s.ldz, s.state->data_ptr(),
            code(*s.state, "state"), s.stride, s.P, Scan::ptr(s.out),
            indices(s.idx, "state_indices", {s.b}), fit32(s.b, "batch"), s.active,
            fit32(s.ch, "channels"), fit32(s.G, "groups"), fit32(s.N, "dstate"), s.softplus,
            dense<int32_t>(s.err, "err_flags", {1}, ScalarType::Int),
            stream_of(stream, r.device));
    });
}

PyObject *spec_verify_(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    return guarded<decltype(&spec_verify)>(args, n, [](Reader &r, auto fn, PyObject *stream) {
        const Tensor &tok = r.tensor("tokens"), &p = r.tensor("target_probs");
        const Tensor &u = r.tensor("uniforms"), &us = r.tensor("uniform_sample");
        const Tensor &acc = r.tensor("accepted_lengths"), &nxt = r.tensor("next_tokens");
        const Tensor *const q = r.optional("draft_probs");
        const Tensor *const parents = r.optional("parent_ids");
        const Tensor *const nodes = r.optional("accepted_node_ids");
        const Tensor *const len = r.optional("context_lengths");
        const Tensor *const idx = r.optional("state_indices");
        const Tensor *const err = r.optional("err_flags");
        if (p.dim() != 3 || (nodes && nodes->dim() != 2))
            refuse("target_probs must be [batch, T, vocab], accepted_node_ids [batch, "
                   "maxAcceptLen]");
        const int64_t b = p.size(0), T = p.size(1), V = p.size(2);
        if (T == 0)
            refuse("target_probs has no tokens: there is no row to draw from");
        const int32_t active = r.int32(b);
        same_type(q, p, "draft_probs", "target_probs");
        const int64_t most = nodes ? nodes->size(1) : 0;
        const int64_t ldp = tokens(p, "target_probs", {b, T, V}, 2);
        const int64_t ldq = q ? tokens(*q, "draft_probs", {b, T > 0 ? T - 1 : 0, V}, 2) : 0;
        const c10::cuda::CUDAGuard on((c10::DeviceIndex)r.device);
        return unlocked(
            fn, indices(&tok, "tokens", {b, T}), p.data_ptr(),
            q ? q->data_ptr() : nullptr, code(p, "target_probs"), ldp, ldq,
            dense<const float>(&u, "uniforms", {b, T}, ScalarType::Float),
            dense<const float>(&us, "uniform_sample", {b}, ScalarType::Float),
            indices(len, "context_lengths", {b}), indices(parents, "parent_ids", {b, T}),
            indices(idx, "state_indices", {b}),
            dense<int32_t>(&acc, "accepted_lengths", {b}, ScalarType::Int),
            dense<int32_t>(&nxt, "next_tokens", {b}, ScalarType::Int),
            node_lists(nodes, "accepted_node_ids", b, most, acc),
            fit32(most, "maxAcceptLen"), fit32(b, "batch"), active, fit32(T, "T"),
            fit32(V, "vocab"), dense<int32_t>(err, "err_flags", {1}, ScalarType::Int),
            stream_of(stream, r.device));
    });
}

#define SSU_METHOD(name, fn) \
    {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(fn)), METH_FASTCALL, nullptr}

PyMethodDef methods[] = {
    SSU_METHOD("ssu_conv_prefill", conv_prefill), SSU_METHOD("ssu_conv_replay", conv_replay),
    SSU_METHOD("scan_prefill", scan_prefill_),    SSU_METHOD("scan_decode", scan_decode_),
    SSU_METHOD("spec_verify", spec_verify_),      {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() { return PyModule_Create(&module); }
