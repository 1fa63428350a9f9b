// ops_binding.cpp -- Python binding of include/kda_ops.h: checks of the tensors,
// allocation of the results through torch, and the call.  Argument marshalling
// only; ops.py holds the documented functions and calls these with every
// argument in place.  It is native because for a single token the call is the
// host's time: 13 us in Python for a convolution of one token, most of it looking
// at tensors.  Everything runs on the current stream of the device that all of a
// call's tensors are on.
#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <string>

#include "../../include/kda_ops.h"

namespace {

PyObject* g_error = nullptr;   // KdaError

struct Refused {};             // a Python error is set

[[noreturn]] void refuse(PyObject* type, const std::string& what) {
    PyErr_SetString(type, what.c_str());
    throw Refused();
}
std::string text(c10::ScalarType t) { return std::string("torch.") + [&]() -> std::string {
    switch (t) {
        case at::kBFloat16: return "bfloat16";
        case at::kHalf: return "float16";
        case at::kFloat: return "float32";
        case at::kInt: return "int32";
        case at::kLong: return "int64";
        case at::kByte: return "uint8";
        default: return c10::toString(t);
    }
}(); }
std::string text(at::IntArrayRef s) {
    std::string r = "(";
    for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
    return r + (s.size() == 1 ? ",)" : ")");
}

// A tensor argument; nullptr for None.
const at::Tensor* tensor(const char* name, PyObject* o, bool optional = false) {
    if (THPVariable_Check(o)) return &THPVariable_Unpack(o);
    if (o == Py_None && optional) return nullptr;
    refuse(PyExc_TypeError, std::string(name) + " must be a tensor");
}
// What a call's tensors have in common: the device of its first one.
struct Call {
    c10::Device device;
};
void need_device(const Call& c, const char* name, const at::Tensor& t) {
    if (!t.is_cuda()) refuse(PyExc_ValueError, std::string(name) + " must be a CUDA tensor");
    if (t.device() != c.device)
        refuse(PyExc_ValueError, std::string(name) + " is on " + t.device().str() + ", the call's first tensor on " +
                                     c.device.str());
}
void need_cuda(const Call& c, const char* name, const at::Tensor& t, c10::ScalarType dtype) {
    need_device(c, name, t);
    if (t.scalar_type() != dtype)
        refuse(PyExc_TypeError, std::string(name) + " must be " + text(dtype) + ", got " + text(t.scalar_type()));
}
// KDA_DTYPE_* of a bf16 or fp16 CUDA tensor.
int32_t elem(const char* name, const at::Tensor& t) {
    if (!t.is_cuda()) refuse(PyExc_ValueError, std::string(name) + " must be a CUDA tensor");
    if (t.scalar_type() == at::kBFloat16) return KDA_DTYPE_BF16;
    if (t.scalar_type() == at::kHalf) return KDA_DTYPE_F16;
    refuse(PyExc_TypeError, std::string(name) + " must be bf16 or fp16, got " + text(t.scalar_type()));
}
// Address of a contiguous CUDA tensor of one type and shape (None: null).
template <typename T = void>
T* flat(const Call& c, const char* name, PyObject* o, c10::ScalarType dtype, at::IntArrayRef shape) {
    const at::Tensor* t = tensor(name, o, true);
    if (!t) return nullptr;
    need_cuda(c, name, *t, dtype);
    if (t->sizes() != shape || !t->is_contiguous())
        refuse(PyExc_ValueError, std::string(name) + " must be contiguous of shape " + text(shape) + ", got " +
                                     text(t->sizes()));
    return static_cast<T*>(t->data_ptr());
}
int32_t* status_word(const Call& c, PyObject* o) {
    const at::Tensor* t = tensor("device_status", o, true);
    if (!t) return nullptr;
    need_cuda(c, "device_status", *t, at::kInt);
    if (t->numel() < 1) refuse(PyExc_ValueError, "device_status must hold an int32");
    return static_cast<int32_t*>(t->data_ptr());
}
// A strided operand of a given shape with a channel dim of stride 1.
void strided(const Call& c, const char* name, const at::Tensor& t, at::IntArrayRef shape, c10::ScalarType dtype) {
    need_cuda(c, name, t, dtype);
    if (t.sizes() != shape || t.stride(-1) != 1)
        refuse(PyExc_ValueError, std::string(name) + " must have shape " + text(shape) +
                                     " and a channel dim of stride 1, got " + text(t.sizes()));
}
// Stride of a dim.  That of a dim of size 1 says nothing (torch calls a row of a transposed
// column contiguous, with a stride of 1): one that the library would refuse is rounded up.
int64_t step(const at::Tensor& t, int64_t dim) {
    const int64_t s = t.stride(dim);
    return t.size(dim) > 1 ? s : (s + 7) / 8 * 8;
}
// (batch, token, head) strides of a [T, H, D] or [B, T, H, D] tensor.
void heads(const Call& c, const char* name, const at::Tensor& t, at::IntArrayRef shape, c10::ScalarType dtype,
           int64_t (&s)[3]) {
    strided(c, name, t, shape, dtype);
    const bool batched = shape.size() == 4;
    s[0] = batched ? step(t, 0) : 0;
    s[1] = step(t, batched);
    s[2] = step(t, 1 + batched);
}
// (page, row, head) strides of a cache.
void cache(const Call& c, const char* name, const at::Tensor& t, int64_t num_heads, int64_t dim,
           c10::ScalarType dtype, int64_t (&s)[3]) {
    need_cuda(c, name, t, dtype);
    if (t.dim() != 4 || t.size(2) != num_heads || t.size(3) != dim || t.stride(3) != 1)
        refuse(PyExc_ValueError, std::string(name) + " must be [pages, page_size, " + std::to_string(num_heads) + ", " +
                                     std::to_string(dim) + "] with a channel dim of stride 1");
    for (int i = 0; i < 3; ++i) s[i] = step(t, i);
}
int64_t integer(PyObject* o) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw Refused();
    return v;
}
float real(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw Refused();
    return (float)v;
}
bool truth(PyObject* o) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw Refused();
    return v != 0;
}
void* stream_of(const at::Tensor& t) { return c10::cuda::getCurrentCUDAStream(t.get_device()).stream(); }

void done(kda_status st) {
    if (st == KDA_OK) return;
    PyObject* e = PyObject_CallFunction(g_error, "i", (int)st);
    if (e) {
        PyErr_SetObject(g_error, e);
        Py_DECREF(e);
    }
    throw Refused();
}
PyObject* none() { Py_RETURN_NONE; }

// Every entry: exceptions of the checks and of torch become Python errors.
template <PyObject* (*F)(PyObject* const*)>
PyObject* entry(PyObject*, PyObject* const* a, Py_ssize_t) {
    try {
        return F(a);
    } catch (const Refused&) {
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

// x, weight, bias, conv_state, slot, has_state, cu_seqlens, accepted, silu,
// norm_channels, norm_eps, out, state_only, device_status
PyObject* short_conv(PyObject* const* o) {
    const at::Tensor &x = *tensor("x", o[0]), &w = *tensor("weight", o[1]);
    kda_short_conv_args a{};
    a.dtype = elem("x", x);
    const Call c{x.device()};
    const auto dt = x.scalar_type();
    const at::Tensor *pool = tensor("conv_state", o[3], true), *cu = tensor("cu_seqlens", o[6], true);
    if (x.dim() != (cu ? 2 : 3) || x.stride(-1) != 1)
        refuse(PyExc_ValueError, "x must be [T_total, C] with cu_seqlens, [B, T, C] without, its last stride 1");
    const int64_t C = x.size(-1);
    if (cu) {
        if (cu->dim() != 1 || cu->size(0) < 1) refuse(PyExc_ValueError, "cu_seqlens must be int32 [N+1]");
        a.num_seqs = cu->size(0) - 1;
        a.seqlen = x.size(0);
        a.x_stride[1] = step(x, 0);
        a.cu_seqlens = flat<int32_t>(c, "cu_seqlens", o[6], at::kInt, {a.num_seqs + 1});
    } else {
        a.num_seqs = x.size(0);
        a.seqlen = x.size(1);
        a.x_stride[0] = step(x, 0);
        a.x_stride[1] = step(x, 1);
    }
    if (w.dim() != 2) refuse(PyExc_ValueError, "weight must be [C, W]");
    const int64_t W = w.size(1);
    const bool f32 = w.scalar_type() == at::kFloat;
    const bool state_only = truth(o[12]);
    a.x = x.data_ptr();
    a.weight = flat(c, "weight", o[1], f32 ? at::kFloat : dt, {C, W});
    a.bias = flat<float>(c, "bias", o[2], at::kFloat, {C});
    if (pool) {
        if (pool->dim() < 1) refuse(PyExc_ValueError, "conv_state must be [P, W-1, C]");
        a.pool_size = pool->size(0);
        a.conv_state = flat(c, "conv_state", o[3], dt, {a.pool_size, W - 1, C});
        if (o[4] == Py_None && a.pool_size < a.num_seqs)
            refuse(PyExc_ValueError, "conv_state has " + std::to_string(a.pool_size) + " entries for " +
                                         std::to_string(a.num_seqs) + " sequences");
    } else if (state_only) {
        refuse(PyExc_ValueError, "state_only needs conv_state");
    }
    a.slot = flat<int32_t>(c, "slot", o[4], at::kInt, {a.num_seqs});
    a.has_state = flat<int32_t>(c, "has_state", o[5], at::kInt, {a.num_seqs});
    a.accepted = flat<int32_t>(c, "accepted", o[7], at::kInt, {a.num_seqs});
    a.device_status = status_word(c, o[13]);
    a.channels = C;
    a.norm_channels = integer(o[9]);
    a.width = (int32_t)W;
    a.weight_dtype = f32 ? KDA_DTYPE_F32 : a.dtype;
    a.silu = truth(o[8]);
    a.norm_eps = real(o[10]);
    const at::Tensor* given = state_only ? nullptr : tensor("out", o[11], true);
    if (given) strided(c, "out", *given, x.sizes(), dt);
    const c10::cuda::CUDAGuard guard(c.device);   // the library launches on the current device
    at::Tensor out;
    if (!state_only) {
        out = given ? *given : at::empty(x.sizes(), x.options());
        a.out = out.data_ptr();
        a.out_stride[0] = cu ? 0 : step(out, 0);
        a.out_stride[1] = step(out, cu ? 0 : 1);
    }
    done(kda_short_conv(&a, stream_of(x)));
    return state_only ? none() : THPVariable_Wrap(out);
}

// q, k, positions, inv_freq, q_weight, k_weight, norm, norm_eps, interleaved,
// rope_scale, q_out, k_out, v, k_cache, v_cache, slots, device_status
PyObject* qk_norm_rope(PyObject* const* o) {
    const at::Tensor &q = *tensor("q", o[0]), &k = *tensor("k", o[1]);
    const at::Tensor *freq = tensor("inv_freq", o[3], true), *v = tensor("v", o[12], true),
                     *kc = tensor("k_cache", o[13], true), *vc = tensor("v_cache", o[14], true);
    kda_qk_norm_rope_args a{};
    a.dtype = elem("q", q);
    const Call c{q.device()};
    const auto dt = q.scalar_type();
    const int64_t nd = q.dim();
    if (nd != 3 && nd != 4) refuse(PyExc_ValueError, "q must be [T, H, D] or [B, T, H, D]");
    const auto lead = q.sizes().slice(0, nd - 2);
    a.head_dim = q.size(-1);
    if (k.dim() != nd || k.sizes().slice(0, nd - 2) != lead || k.size(-1) != a.head_dim)
        refuse(PyExc_ValueError, "q and k must have the same tokens and head size");
    a.num_q_heads = q.size(-2);
    a.num_k_heads = k.size(-2);
    a.batch = nd == 4 ? lead[0] : 1;
    a.seqlen = lead[nd - 3];
    if (freq) {
        if (freq->dim() != 1) refuse(PyExc_ValueError, "inv_freq must be fp32 [rot_dim / 2]");
        a.rot_dim = 2 * freq->size(0);
        a.inv_freq = flat<float>(c, "inv_freq", o[3], at::kFloat, {freq->size(0)});
        a.positions = flat<int32_t>(c, "positions", o[2], at::kInt, lead);
    }
    const at::Tensor *qw = tensor("q_weight", o[4], true), *kw = tensor("k_weight", o[5], true);
    if (qw && kw && qw->scalar_type() != kw->scalar_type())
        refuse(PyExc_TypeError, "the weights must have the same type");
    const at::Tensor* any = qw ? qw : kw;
    const bool f32 = !any || any->scalar_type() == at::kFloat;
    a.weight_dtype = f32 ? KDA_DTYPE_F32 : a.dtype;
    a.q_weight = flat(c, "q_weight", o[4], f32 ? at::kFloat : dt, {a.head_dim});
    a.k_weight = flat(c, "k_weight", o[5], f32 ? at::kFloat : dt, {a.head_dim});
    heads(c, "q", q, q.sizes(), dt, a.q_stride);
    heads(c, "k", k, k.sizes(), dt, a.k_stride);
    a.q = q.data_ptr();
    a.k = k.data_ptr();
    if (kc) {
        cache(c, "k_cache", *kc, a.num_k_heads, a.head_dim, dt, a.k_cache_stride);
        a.k_cache = kc->data_ptr();
        a.num_pages = kc->size(0);
        a.page_size = kc->size(1);
        a.slots = flat<int64_t>(c, "slots", o[15], at::kLong, lead);
        if (o[15] == Py_None && a.batch * a.seqlen > 0) refuse(PyExc_ValueError, "k_cache needs slots");
        if (vc) {
            cache(c, "v_cache", *vc, a.num_k_heads, a.head_dim, dt, a.v_cache_stride);
            if (!v || vc->sizes() != kc->sizes()) refuse(PyExc_ValueError, "v_cache needs v, and k_cache's shape");
            heads(c, "v", *v, k.sizes(), dt, a.v_stride);
            a.v = v->data_ptr();
            a.v_cache = vc->data_ptr();
        }
    } else if (vc || o[15] != Py_None) {
        refuse(PyExc_ValueError, "slots and v_cache need k_cache");
    }
    const at::Tensor *q_given = tensor("q_out", o[10], true), *k_given = tensor("k_out", o[11], true);
    if (q_given) heads(c, "q_out", *q_given, q.sizes(), dt, a.q_out_stride);
    if (k_given) heads(c, "k_out", *k_given, k.sizes(), dt, a.k_out_stride);
    a.device_status = status_word(c, o[16]);
    const c10::cuda::CUDAGuard guard(c.device);
    at::Tensor q_out, k_out;
    q_out = q_given ? *q_given : at::empty(q.sizes(), q.options());
    if (!q_given) heads(c, "q_out", q_out, q.sizes(), dt, a.q_out_stride);
    a.q_out = q_out.data_ptr();
    if (k_given) k_out = *k_given;
    else if (!kc) k_out = at::empty(k.sizes(), k.options());
    if (k_out.defined()) {
        if (!k_given) heads(c, "k_out", k_out, k.sizes(), dt, a.k_out_stride);
        a.k_out = k_out.data_ptr();
    }
    a.norm = truth(o[6]);
    a.norm_eps = real(o[7]);
    a.interleaved = truth(o[8]);
    a.rope_scale = real(o[9]);
    done(kda_qk_norm_rope(&a, stream_of(q)));
    PyObject* qo = o[10] != Py_None ? Py_NewRef(o[10]) : THPVariable_Wrap(q_out);
    PyObject* ko = o[11] != Py_None ? Py_NewRef(o[11]) : k_out.defined() ? THPVariable_Wrap(k_out) : none();
    PyObject* r = PyTuple_Pack(2, qo, ko);
    Py_DECREF(qo);
    Py_DECREF(ko);
    return r;
}

// q, k_cache, v_cache, page_table, context_lens, tree_mask, num_nodes, scale,
// max_context, out, return_lse, workspace, device_status, address of a kda_overrides
PyObject* tree_attention(PyObject* const* o) {
    const at::Tensor &q = *tensor("q", o[0]), &kc = *tensor("k_cache", o[1]), &vc = *tensor("v_cache", o[2]),
                     &table = *tensor("page_table", o[3]);
    kda_tree_attention_args a{};
    a.dtype = elem("q", q);
    const Call c{q.device()};
    const auto dt = q.scalar_type();
    if (q.dim() != 4 || q.stride(3) != 1)
        refuse(PyExc_ValueError, "q must be [R, N, Hq, D] with a channel dim of stride 1");
    const int64_t R = q.size(0), N = q.size(1), Hq = q.size(2), D = q.size(3);
    need_device(c, "k_cache", kc);
    if (kc.dim() != 4) refuse(PyExc_ValueError, "k_cache must be [pages, page_size, Hk, D]");
    a.num_k_heads = kc.size(2);
    cache(c, "k_cache", kc, a.num_k_heads, D, dt, a.k_cache_stride);
    cache(c, "v_cache", vc, a.num_k_heads, D, dt, a.v_cache_stride);
    if (vc.sizes() != kc.sizes()) refuse(PyExc_ValueError, "k_cache and v_cache must have the same shape");
    need_cuda(c, "page_table", table, at::kInt);
    if (table.dim() != 2 || table.size(0) != R || (table.size(1) > 1 && table.stride(1) != 1))
        refuse(PyExc_ValueError, "page_table must be int32 [R, pages] with contiguous rows");
    if (o[4] == Py_None) refuse(PyExc_TypeError, "context_lens must be a tensor");
    a.context_lens = flat<int32_t>(c, "context_lens", o[4], at::kInt, {R});
    a.tree_mask = flat<uint64_t>(c, "tree_mask", o[5], at::kLong, {R, N, (N + 63) / 64});
    a.num_nodes = flat<int32_t>(c, "num_nodes", o[6], at::kInt, {R});
    a.device_status = status_word(c, o[12]);
    const at::Tensor *given = tensor("out", o[9], true), *given_ws = tensor("workspace", o[11], true);
    if (given) strided(c, "out", *given, q.sizes(), dt);
    if (given_ws) {
        need_cuda(c, "workspace", *given_ws, at::kByte);
        if (!given_ws->is_contiguous()) refuse(PyExc_ValueError, "workspace must be contiguous");
    }
    a.max_context = o[8] == Py_None ? 0 : integer(o[8]);
    a.scale = o[7] == Py_None ? (D > 0 ? 1.f / sqrtf((float)D) : 1.f) : real(o[7]);
    const bool want_lse = truth(o[10]);
    const c10::cuda::CUDAGuard guard(c.device);
    at::Tensor out = given ? *given : at::empty(q.sizes(), q.options()), lse, ws;
    if (want_lse) {
        lse = at::empty({R, N, Hq}, q.options().dtype(at::kFloat));
        a.lse = static_cast<float*>(lse.data_ptr());
    }
    a.q = q.data_ptr();
    a.k_cache = kc.data_ptr();
    a.v_cache = vc.data_ptr();
    a.out = out.data_ptr();
    a.page_table = static_cast<int32_t*>(table.data_ptr());
    for (int i = 0; i < 3; ++i) {
        a.q_stride[i] = step(q, i);
        a.out_stride[i] = step(out, i);
    }
    a.page_table_stride = table.stride(0);
    a.num_requests = R;
    a.max_nodes = N;
    a.num_q_heads = Hq;
    a.head_dim = D;
    a.num_pages = kc.size(0);
    a.page_size = kc.size(1);
    a.pages_per_request = table.size(1);
    if (given_ws) ws = *given_ws;
    else if (const size_t need = kda_tree_attention_workspace_size(&a))
        ws = at::empty({(int64_t)need}, q.options().dtype(at::kByte));
    if (ws.defined()) {
        a.workspace = ws.data_ptr();
        a.workspace_bytes = (size_t)ws.numel();
    }
    const auto* overrides = o[13] == Py_None ? nullptr : static_cast<const kda_overrides*>(PyLong_AsVoidPtr(o[13]));
    if (PyErr_Occurred()) throw Refused();
    done(kda_tree_attention_ex(&a, overrides, stream_of(q)));
    PyObject* ro = o[9] != Py_None ? Py_NewRef(o[9]) : THPVariable_Wrap(out);
    if (!want_lse) return ro;
    PyObject* rl = THPVariable_Wrap(lse);
    PyObject* r = PyTuple_Pack(2, ro, rl);
    Py_DECREF(ro);
    Py_DECREF(rl);
    return r;
}

PyObject* set_error(PyObject* const* o) {
    Py_XDECREF(g_error);
    g_error = Py_NewRef(o[0]);
    return none();
}

// The callers (ops.py) pass every argument; a wrong count would read past the array.
template <PyObject* (*F)(PyObject* const*), int kArgs>
PyObject* counted(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    if (n != kArgs) {
        PyErr_Format(PyExc_TypeError, "%d arguments expected, got %zd", kArgs, n);
        return nullptr;
    }
    return entry<F>(self, a, n);
}

template <PyObject* (*F)(PyObject* const*), int kArgs>
PyMethodDef method(const char* name) {
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(counted<F, kArgs>)), METH_FASTCALL, nullptr};
}
PyMethodDef methods[] = {method<short_conv, 14>("short_conv"), method<qk_norm_rope, 17>("qk_norm_rope"),
                         method<tree_attention, 14>("tree_attention"), method<set_error, 1>("set_error"),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_kda_ops", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__kda_ops(void) { return PyModule_Create(&module); }
