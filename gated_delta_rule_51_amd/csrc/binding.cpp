// The Python calls of the convolution, scan, verification and commit in native
// code: argument checks, output allocation and the C call in one step, since
// around a one-token kernel of a few microseconds the same work in Python costs
// twice the kernel.  A call whose arguments do not all fit is declined (None),
// and the Python function, which makes the same checks one by one, says why.
//
// Every function takes the raw stream first; the caller has made sure that the
// first tensor's device is the current one.
#include <Python.h>

#include <ATen/ATen.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>

#include "kda.h"

namespace {

using at::ScalarType;
using at::Tensor;

struct Declined {};   // an argument does not fit

void need(bool ok) {
    if (!ok) throw Declined{};
}

int code(ScalarType t) {
    need(t == at::kFloat || t == at::kBFloat16);
    return t == at::kBFloat16 ? KDA_BF16 : KDA_F32;
}

// The tensors of one call: all on the device of the first.
struct Args {
    PyObject *const *v;
    int device = -1;

    const Tensor *maybe(int i) {
        if (v[i] == Py_None) return nullptr;
        need(THPVariable_Check(v[i]));
        const Tensor &t = THPVariable_Unpack(v[i]);
        need(t.is_cuda() && t.layout() == at::kStrided);
        if (device < 0) device = t.get_device();
        need(t.get_device() == device);
        return &t;
    }
    const Tensor &tensor(int i) {
        const Tensor *t = maybe(i);
        need(t != nullptr);
        return *t;
    }
    bool flag(int i) {
        need(PyBool_Check(v[i]));
        return v[i] == Py_True;
    }
    void *stream() { return PyLong_AsVoidPtr(v[0]); }
};

// [>= n, a] (b 0) or [>= n, a, b], contiguous within a row; returns the
// elements between two rows, which must not overlap.
int64_t rows(const Tensor &t, ScalarType type, int64_t n, int64_t a, int64_t b = 0) {
    const auto size = t.sizes(), step = t.strides();
    need(t.scalar_type() == type && (int64_t)size.size() == (b ? 3 : 2) && size[0] >= n && size[1] == a);
    if (b) need(size[2] == b && (step[2] == 1 || b == 1) && (step[1] == b || a == 1));
    else need(step[1] == 1 || a == 1);
    const int64_t width = b ? a * b : a;
    if (size[0] <= 1) return width;
    need(step[0] >= width);
    return step[0];
}

// Contiguous [>= n, tail...].
void whole(const Tensor &t, ScalarType type, int64_t n, at::IntArrayRef tail) {
    need(t.scalar_type() == type && t.dim() == (int64_t)tail.size() + 1 && t.size(0) >= n && t.sizes().slice(1) == tail && t.is_contiguous());
}
void exactly(const Tensor *t, ScalarType type, at::IntArrayRef sizes) {
    if (t) need(t->scalar_type() == type && t->sizes() == sizes && t->is_contiguous());
}

template <typename T = void> T *ptr(const Tensor *t) { return t ? static_cast<T *>(t->data_ptr()) : nullptr; }
template <typename T = void> T *ptr(const Tensor &t) { return static_cast<T *>(t.data_ptr()); }

Tensor fresh(const Tensor &like, at::IntArrayRef sizes, ScalarType type) {
    return at::empty(sizes, at::TensorOptions().dtype(type).device(like.device()));
}

int32_t narrow(int64_t n) {
    need(n >= 0 && n <= INT32_MAX);
    return (int32_t)n;
}

// N of cu_seqlens [N + 1].
int32_t sequences(const Tensor &cu) {
    whole(cu, at::kInt, 1, {});
    return narrow(cu.size(0) - 1);
}

// A step cache [>= n, steps, a, b, c]: its pitch in steps.
int64_t cache_pitch(const Tensor &t, ScalarType type, int64_t n, int64_t a, int64_t b, int64_t c) {
    const auto size = t.sizes(), step = t.strides();
    const int64_t unit = a * b * c;
    need(unit > 0 && t.scalar_type() == type && size.size() == 5 && size[0] >= n && size[2] == a && size[3] == b && size[4] == c);
    need(step[1] == unit && step[2] == b * c && step[3] == c && step[4] == 1 && step[0] % unit == 0 && step[0] / unit >= size[1]);
    return step[0] / unit;
}

PyObject *done(kda_status s) {
    if (s != KDA_OK) return PyLong_FromLong(s);
    Py_RETURN_TRUE;
}
PyObject *done(kda_status s, const Tensor &t) { return s != KDA_OK ? PyLong_FromLong(s) : THPVariable_Wrap(t); }
// (y, final): the pool's own object in pool mode, a new tensor, or None.
PyObject *done(kda_status s, const Tensor &y, PyObject *pool, const Tensor &last) {
    if (s != KDA_OK) return PyLong_FromLong(s);
    PyObject *second = pool ? Py_NewRef(pool) : last.defined() ? THPVariable_Wrap(last) : Py_NewRef(Py_None);
    PyObject *pair = PyTuple_New(2);
    PyTuple_SET_ITEM(pair, 0, THPVariable_Wrap(y));
    PyTuple_SET_ITEM(pair, 1, second);
    return pair;
}

// x, weight, bias at 1, 2, 3: the descriptor of a convolution.
kda_conv_desc conv_desc(Args &a, int64_t n, bool silu) {
    const Tensor &x = a.tensor(1), &w = a.tensor(2);
    need(x.dim() == 2 && w.dim() == 2);
    const int64_t T = x.size(0), D = x.size(1);
    kda_conv_desc d{};
    d.num_seqs = narrow(n);
    d.total_tokens = narrow(T);
    d.channels = narrow(D);
    d.width = narrow(w.size(1));
    d.io_dtype = code(x.scalar_type());
    d.silu = silu;
    d.x_stride = rows(x, x.scalar_type(), T, D);
    exactly(&w, x.scalar_type(), {D, w.size(1)});
    exactly(a.maybe(3), x.scalar_type(), {D});
    need(d.width >= 1);
    return d;
}

// conv_prefill(stream, x, weight, bias, cu, state, indices, silu, output_final, update_pool)
PyObject *conv_prefill(Args &a) {
    const Tensor &x = a.tensor(1), &cu = a.tensor(4);
    const int64_t N = sequences(cu);
    kda_conv_desc d = conv_desc(a, N, a.flag(7));
    const Tensor *state = a.maybe(5), *idx = a.maybe(6);
    const int64_t D = d.channels, W = d.width;
    need(state || !idx);
    if (state) whole(*state, x.scalar_type(), idx ? 1 : N, {W - 1, D});
    if (idx) whole(*idx, at::kInt, N, {});
    d.num_slots = idx ? narrow(state->size(0)) : 0;
    d.update_pool = a.flag(9);
    const Tensor y = fresh(x, {x.size(0), D}, x.scalar_type());
    const Tensor last = !idx && a.flag(8) ? fresh(x, {N, W - 1, D}, x.scalar_type()) : Tensor();
    return done(kda_conv_prefill(&d, ptr(x), ptr(a.tensor(2)), ptr(a.maybe(3)), ptr<int32_t>(cu), ptr(state), ptr<int32_t>(idx),
                                 last.defined() ? ptr(last) : nullptr, ptr(y), a.stream()),
                y, idx ? a.v[5] : nullptr, last);
}

// conv_decode(stream, x, weight, bias, pool, indices, silu)
PyObject *conv_decode(Args &a) {
    const Tensor &x = a.tensor(1), &pool = a.tensor(4), &idx = a.tensor(5);
    need(x.dim() == 2);
    kda_conv_desc d = conv_desc(a, x.size(0), a.flag(6));
    whole(pool, x.scalar_type(), 1, {d.width - 1, d.channels});
    whole(idx, at::kInt, d.num_seqs, {});
    d.num_slots = narrow(pool.size(0));
    const Tensor y = fresh(x, x.sizes(), x.scalar_type());
    return done(kda_conv_decode(&d, ptr(x), ptr(a.tensor(2)), ptr(a.maybe(3)), ptr(pool), ptr<int32_t>(idx), ptr(y), a.stream()), y);
}

// conv_commit(stream, x, cu, steps, pool, indices)
PyObject *conv_commit(Args &a) {
    const Tensor &x = a.tensor(1), &cu = a.tensor(2), &steps = a.tensor(3), &pool = a.tensor(4), &idx = a.tensor(5);
    need(x.dim() == 2 && pool.dim() == 3);
    kda_conv_desc d{};
    d.num_seqs = sequences(cu);
    d.total_tokens = narrow(x.size(0));
    d.channels = narrow(x.size(1));
    d.width = narrow(pool.size(1) + 1);
    d.io_dtype = code(x.scalar_type());
    d.num_slots = narrow(pool.size(0));
    d.x_stride = rows(x, x.scalar_type(), x.size(0), x.size(1));
    whole(pool, x.scalar_type(), 1, {d.width - 1, d.channels});
    whole(idx, at::kInt, d.num_seqs, {});
    whole(steps, at::kInt, d.num_seqs, {});
    return done(kda_conv_commit(&d, ptr(x), ptr<int32_t>(cu), ptr<int32_t>(steps), ptr(pool), ptr<int32_t>(idx), a.stream()));
}

// x, dt, A_log, B, C, D, z, dt_bias from 1 on: the descriptor of a scan.
kda_ssm_desc ssm_desc(Args &a, int64_t n, ScalarType states) {
    const Tensor &x = a.tensor(1), &B = a.tensor(4);
    need(x.dim() == 3 && B.dim() == 3);
    const int64_t T = x.size(0), H = x.size(1), P = x.size(2), G = B.size(1), S = B.size(2);
    const ScalarType io = x.scalar_type();
    need(H > 0 && P > 0 && G > 0 && S > 0 && H % G == 0);
    kda_ssm_desc d{};
    d.num_seqs = narrow(n);
    d.total_tokens = narrow(T);
    d.heads = narrow(H);
    d.groups = narrow(G);
    d.head_dim = narrow(P);
    d.state_dim = narrow(S);
    d.io_dtype = code(io);
    d.state_dtype = code(states);
    d.x_stride = rows(x, io, T, H, P);
    d.dt_stride = rows(a.tensor(2), io, T, H);
    d.b_stride = rows(B, io, T, G, S);
    d.c_stride = rows(a.tensor(5), io, T, G, S);
    if (const Tensor *z = a.maybe(7)) d.z_stride = rows(*z, io, T, H, P);
    exactly(&a.tensor(3), at::kFloat, {H});
    exactly(a.maybe(6), at::kFloat, {H});
    exactly(a.maybe(8), at::kFloat, {H});
    return d;
}

// ssm_prefill(stream, x, dt, A_log, B, C, D, z, dt_bias, cu, state, indices, output_final, state_bf16)
PyObject *ssm_prefill(Args &a) {
    const Tensor &x = a.tensor(1), &cu = a.tensor(9);
    const Tensor *state = a.maybe(10), *idx = a.maybe(11);
    const int64_t N = sequences(cu);
    const ScalarType st = state ? state->scalar_type() : a.flag(13) ? at::kBFloat16 : at::kFloat;
    kda_ssm_desc d = ssm_desc(a, N, st);
    need(state || !idx);
    if (state) whole(*state, st, idx ? 1 : N, {d.heads, d.head_dim, d.state_dim});
    if (idx) whole(*idx, at::kInt, N, {});
    d.num_slots = idx ? narrow(state->size(0)) : 0;
    const Tensor y = fresh(x, x.sizes(), x.scalar_type());
    const Tensor last = !idx && a.flag(12) ? fresh(x, {N, d.heads, d.head_dim, d.state_dim}, st) : Tensor();
    const size_t bytes = kda_ssm_prefill_workspace_size(&d);
    const Tensor ws = bytes ? fresh(x, {(int64_t)bytes}, at::kByte) : Tensor();
    return done(kda_ssm_prefill(&d, ptr(x), ptr(a.tensor(2)), ptr<float>(a.tensor(3)), ptr(a.tensor(4)), ptr(a.tensor(5)),
                                ptr<float>(a.maybe(6)), ptr(a.maybe(7)), ptr<float>(a.maybe(8)), ptr<int32_t>(cu), ptr(state),
                                ptr<int32_t>(idx), last.defined() ? ptr(last) : nullptr, ptr(y), bytes ? ptr(ws) : nullptr, bytes,
                                a.stream()),
                y, idx ? a.v[10] : nullptr, last);
}

// ssm_decode(stream, x, dt, A_log, B, C, D, z, dt_bias, pool, indices)
PyObject *ssm_decode(Args &a) {
    const Tensor &x = a.tensor(1), &pool = a.tensor(9), &idx = a.tensor(10);
    need(x.dim() == 3);
    kda_ssm_desc d = ssm_desc(a, x.size(0), pool.scalar_type());
    whole(pool, pool.scalar_type(), 1, {d.heads, d.head_dim, d.state_dim});
    whole(idx, at::kInt, d.num_seqs, {});
    d.num_slots = narrow(pool.size(0));
    const Tensor y = fresh(x, x.sizes(), x.scalar_type());
    return done(kda_ssm_decode(&d, ptr(x), ptr(a.tensor(2)), ptr<float>(a.tensor(3)), ptr(a.tensor(4)), ptr(a.tensor(5)),
                               ptr<float>(a.maybe(6)), ptr(a.maybe(7)), ptr<float>(a.maybe(8)), ptr(pool), ptr<int32_t>(idx), ptr(y),
                               a.stream()),
                y);
}

// ssm_decode_multi(stream, x, dt, A_log, B, C, D, z, dt_bias, cu, pool, indices, cache, update_pool)
PyObject *ssm_decode_multi(Args &a) {
    const Tensor &x = a.tensor(1), &cu = a.tensor(9), &pool = a.tensor(10), &idx = a.tensor(11);
    const Tensor *cache = a.maybe(12);
    const ScalarType st = pool.scalar_type();
    kda_ssm_desc d = ssm_desc(a, sequences(cu), st);
    whole(pool, st, 1, {d.heads, d.head_dim, d.state_dim});
    whole(idx, at::kInt, d.num_seqs, {});
    d.num_slots = narrow(pool.size(0));
    if (cache) {
        d.cache_pitch = narrow(cache_pitch(*cache, st, d.num_seqs, d.heads, d.head_dim, d.state_dim));
        d.cache_steps = narrow(cache->size(1));
    }
    d.update_pool = a.flag(13);
    const Tensor y = fresh(x, x.sizes(), x.scalar_type());
    return done(kda_ssm_decode_multi(&d, ptr(x), ptr(a.tensor(2)), ptr<float>(a.tensor(3)), ptr(a.tensor(4)), ptr(a.tensor(5)),
                                     ptr<float>(a.maybe(6)), ptr(a.maybe(7)), ptr<float>(a.maybe(8)), ptr<int32_t>(cu), ptr(pool),
                                     ptr<int32_t>(idx), d.cache_steps ? ptr(cache) : nullptr, ptr(y), a.stream()),
                y);
}

// verify_drafts(stream, target, tokens, cu, uniform, uniform_next, draft)
PyObject *verify_drafts(Args &a) {
    const Tensor &p = a.tensor(1), &tokens = a.tensor(2), &cu = a.tensor(3), &u = a.tensor(4), &r = a.tensor(5);
    const Tensor *q = a.maybe(6);
    whole(tokens, at::kInt, 0, {});
    need(p.dim() == 2 && p.size(1) > 0);
    const int64_t T = tokens.size(0), V = p.size(1);
    kda_verify_desc d{};
    d.num_seqs = sequences(cu);
    d.total_tokens = narrow(T);
    d.vocab = narrow(V);
    d.prob_dtype = code(p.scalar_type());
    d.target_stride = rows(p, p.scalar_type(), T, V);
    d.draft_stride = q ? rows(*q, p.scalar_type(), T, V) : 0;
    whole(u, at::kFloat, T, {});
    whole(r, at::kFloat, d.num_seqs, {});
    const Tensor accepted = fresh(p, {d.num_seqs}, at::kInt), next = fresh(p, {d.num_seqs}, at::kInt), out = fresh(p, {T}, at::kInt);
    const size_t bytes = kda_verify_drafts_workspace_size(&d);
    const Tensor ws = fresh(p, {(int64_t)std::max<size_t>(bytes, 16)}, at::kByte);
    const kda_status s = kda_verify_drafts(&d, ptr<int32_t>(tokens), ptr(p), ptr(q), ptr<int32_t>(cu), ptr<float>(u), ptr<float>(r),
                                           ptr<int32_t>(accepted), ptr<int32_t>(next), ptr<int32_t>(out), ptr(ws),
                                           std::max<size_t>(bytes, 16), a.stream());
    if (s != KDA_OK) return PyLong_FromLong(s);
    PyObject *three = PyTuple_New(3);
    PyTuple_SET_ITEM(three, 0, THPVariable_Wrap(accepted));
    PyTuple_SET_ITEM(three, 1, THPVariable_Wrap(next));
    PyTuple_SET_ITEM(three, 2, THPVariable_Wrap(out));
    return three;
}

// commit_states(stream, pool, indices, cache, steps)
PyObject *commit_states(Args &a) {
    const Tensor &pool = a.tensor(1), &idx = a.tensor(2), &cache = a.tensor(3), &steps = a.tensor(4);
    need(pool.dim() == 4 && steps.dim() == 1 && pool.size(0) >= 1 && pool.is_contiguous());
    kda_commit_desc d{};
    d.num_seqs = narrow(steps.size(0));
    d.num_slots = narrow(pool.size(0));
    whole(steps, at::kInt, 0, {});
    whole(idx, at::kInt, d.num_seqs, {});
    d.cache_pitch = narrow(cache_pitch(cache, pool.scalar_type(), d.num_seqs, pool.size(1), pool.size(2), pool.size(3)));
    d.cache_steps = narrow(cache.size(1));
    d.row_bytes = pool.size(1) * pool.size(2) * pool.size(3) * (int64_t)pool.element_size();
    return done(kda_commit_states(&d, ptr(pool), ptr<int32_t>(idx), ptr(cache), ptr<int32_t>(steps), a.stream()));
}

template <PyObject *(*F)(Args &), int N> PyObject *call(PyObject *, PyObject *const *args, Py_ssize_t count) {
    HANDLE_TH_ERRORS
    if (count != N) {
        PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
        return nullptr;
    }
    Args a{args};
    try {
        return F(a);
    } catch (const Declined &) {
        Py_RETURN_NONE;
    }
    END_HANDLE_TH_ERRORS
}

template <PyObject *(*F)(Args &), int N> PyCFunction fast() {
    return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&call<F, N>));
}

PyMethodDef methods[] = {
    {"conv_prefill", fast<conv_prefill, 10>(), METH_FASTCALL, nullptr},
    {"conv_decode", fast<conv_decode, 7>(), METH_FASTCALL, nullptr},
    {"conv_commit", fast<conv_commit, 6>(), METH_FASTCALL, nullptr},
    {"ssm_prefill", fast<ssm_prefill, 14>(), METH_FASTCALL, nullptr},
    {"ssm_decode", fast<ssm_decode, 11>(), METH_FASTCALL, nullptr},
    {"ssm_decode_multi", fast<ssm_decode_multi, 14>(), METH_FASTCALL, nullptr},
    {"verify_drafts", fast<verify_drafts, 7>(), METH_FASTCALL, nullptr},
    {"commit_states", fast<commit_states, 5>(), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
