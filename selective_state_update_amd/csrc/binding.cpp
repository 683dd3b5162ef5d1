// binding.cpp -- the Python entry points of the sequence operators
// (linear_attention, gated_delta_rule, their steps, qk_norm_rope, add_rms_norm,
// paged_attention, shared_prefix_attention): tensors checked, turned into the views of include/ssu.h and passed on, with
// outputs and workspaces from torch's allocator on torch's current stream.
// Native because the operators' smallest calls run for 3 to 5 us and checking
// and packing nine to twelve tensors in Python took 6 to 10.

#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/core/GradMode.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <initializer_list>
#include <string>

#include "ssu.h"

namespace {

PyObject *g_error = nullptr;  // SSUError(status, where)

[[noreturn]] void refuse(PyObject *type, const std::string &what)
{
    PyErr_SetString(type, what.c_str());
    throw python_error();
}

const at::Tensor &tensor(PyObject *o, const char *name)
{
    if (!THPVariable_Check(o))
        refuse(PyExc_TypeError, std::string(name) + " must be a tensor");
    return THPVariable_Unpack(o);
}

std::string list(at::IntArrayRef sizes)
{
    std::string s = "[";
    for (size_t i = 0; i < sizes.size(); ++i)
        s += (i ? ", " : "") + std::to_string(sizes[i]);
    return s + "]";
}

int gpu_of(const at::Tensor &t, const char *name)
{
    if (!t.is_cuda())
        refuse(PyExc_ValueError, std::string(name) + " must be on a GPU");
    return t.get_device();
}

int32_t tag_of(at::ScalarType t)
{
    switch (t) {
    case at::kFloat: return SSU_F32;
    case at::kBFloat16: return SSU_BF16;
    case at::kHalf: return SSU_F16;
    case at::kInt: return SSU_I32;
    case at::kLong: return SSU_I64;
    case at::kFloat8_e4m3fn: return SSU_E4M3;
    default: return -1;
    }
}

using Types = std::initializer_list<at::ScalarType>;

// The view of a tensor after checking its shape, dtype and device.
ssu_view view(const at::Tensor &t, const char *name, at::IntArrayRef shape, Types types, int gpu)
{
    if (t.sizes() != shape)
        refuse(PyExc_ValueError, std::string(name) + " must be " + list(shape) + ", got " + list(t.sizes()));
    bool known = false;
    for (const at::ScalarType s : types)
        known |= s == t.scalar_type();
    if (!known)
        refuse(PyExc_TypeError, std::string(name) + ": dtype " + c10::toString(t.scalar_type()) + " not supported here");
    if (!t.is_cuda() || t.get_device() != gpu)
        refuse(PyExc_ValueError, std::string(name) + " is on " + t.device().str() + ", expected cuda:" + std::to_string(gpu));
    if (t.requires_grad() && c10::GradMode::is_enabled())
        refuse(PyExc_ValueError, std::string("inference only: no gradient is recorded for ") + name +
                                     "; call under torch.no_grad() or detach it");
    if (t._fw_grad(0).defined())
        refuse(PyExc_ValueError, std::string("inference only: no tangent is carried for ") + name + "; unpack the dual tensor");
    if (t.is_neg())  // (as the imaginary part of a conjugate is)
        refuse(PyExc_ValueError, std::string(name) + " is a view of negated memory; call resolve_neg() on it");
    ssu_view v{};
    v.ptr = t.data_ptr();
    v.dtype = tag_of(t.scalar_type());
    for (int64_t i = 0; i < t.dim(); ++i)
        v.stride[i] = t.stride(i);
    return v;
}

ssu_view view(PyObject *o, const char *name, at::IntArrayRef shape, Types types, int gpu)
{
    return view(tensor(o, name), name, shape, types, gpu);
}

ssu_view view_or_none(PyObject *o, const char *name, at::IntArrayRef shape, Types types, int gpu)
{
    return o == Py_None ? ssu_view{} : view(o, name, shape, types, gpu);
}

int32_t i32(int64_t n, const char *name)
{
    if (n > INT32_MAX || n < INT32_MIN)
        refuse(PyExc_ValueError, std::string(name) + " is too large: " + std::to_string(n));
    return static_cast<int32_t>(n);
}

float number(PyObject *o)
{
    const double x = PyFloat_AsDouble(o);
    if (x == -1.0 && PyErr_Occurred())
        throw python_error();
    return static_cast<float>(x);
}

int64_t integer(PyObject *o)
{
    const long long n = PyLong_AsLongLong(o);
    if (n == -1 && PyErr_Occurred())
        throw python_error();
    return n;
}

bool truth(PyObject *o)
{
    const int x = PyObject_IsTrue(o);
    if (x < 0)
        throw python_error();
    return x != 0;
}

at::Tensor make(at::IntArrayRef shape, at::ScalarType type, int gpu)
{
    return at::empty(shape, at::TensorOptions().dtype(type).device(at::kCUDA, static_cast<c10::DeviceIndex>(gpu)));
}

// A caller's output or a new one.
at::Tensor given_or(PyObject *o, const char *name, at::IntArrayRef shape, at::ScalarType type, int gpu)
{
    return o == Py_None ? make(shape, type, gpu) : tensor(o, name);
}

PyObject *object(PyObject *given, const at::Tensor &t)
{
    if (given == Py_None)
        return THPVariable_Wrap(t);
    Py_INCREF(given);
    return given;
}

// A call's workspace: the caller's, or a new one (kept alive by `keep` until
// the launch; the allocator hands its memory out again in the stream's order).
template <typename Args>
void workspace(PyObject *given, int64_t need, int gpu, Args &a, at::Tensor &keep)
{
    if (given != Py_None) {
        const at::Tensor &t = tensor(given, "workspace");
        if (!t.is_cuda() || t.get_device() != gpu || !t.is_contiguous())
            refuse(PyExc_ValueError, "workspace must be contiguous, on cuda:" + std::to_string(gpu));
        a.workspace = t.data_ptr();
        a.workspace_bytes = static_cast<int64_t>(t.nbytes());
    } else if (need > 0) {
        keep = make({need}, at::kByte, gpu);
        a.workspace = keep.data_ptr();
        a.workspace_bytes = need;
    }
}

template <typename Args>
void call(ssu_status (*fn)(const Args *, hipStream_t), const Args &a, int gpu, const char *where)
{
    const hipStream_t stream = c10::hip::getCurrentHIPStream(static_cast<c10::DeviceIndex>(gpu)).stream();
    ssu_status s;
    Py_BEGIN_ALLOW_THREADS;
    s = fn(&a, stream);
    Py_END_ALLOW_THREADS;
    if (s == SSU_OK)
        return;
    PyObject *const e = PyObject_CallFunction(g_error, "is", static_cast<int>(s), where);
    if (e) {
        PyErr_SetObject(g_error, e);
        Py_DECREF(e);
    }
    throw python_error();
}

void count(Py_ssize_t n, Py_ssize_t want)
{
    if (n != want)
        refuse(PyExc_TypeError, "expected " + std::to_string(want) + " arguments");
}

// The operators on state slots, over prompts and for single tokens.
template <typename Args>
struct Recurrence {
    ssu_status (*prompts)(const Args *, hipStream_t), (*step)(const Args *, hipStream_t);
    int64_t (*need)(const Args *);
    const char *where, *where_step;
};

constexpr Recurrence<ssu_linear_args> kLinear{&ssu_linear_attention, &ssu_linear_attention_step, &ssu_linear_attention_workspace,
                                              "ssu_linear_attention", "ssu_linear_attention_step"};
constexpr Recurrence<ssu_delta_args> kDelta{&ssu_gated_delta_rule, &ssu_gated_delta_rule_step, &ssu_gated_delta_rule_workspace,
                                            "ssu_gated_delta_rule", "ssu_gated_delta_rule_step"};

// o: state, q, k, v, log_decay, cu_seqlens | None, idx, beta | None, scale, out | None, workspace | None
template <typename Args>
PyObject *recurrence(const Recurrence<Args> &fn, Args a, PyObject *const *o)
{
    const at::Tensor &state = tensor(o[0], "state"), &q = tensor(o[1], "q"), &v = tensor(o[3], "v");
    const at::Tensor &decay = tensor(o[4], "log_decay"), &idx = tensor(o[6], "state_batch_indices");
    const int gpu = gpu_of(state, "state");
    if (state.dim() != 4 || q.dim() != 3 || v.dim() != 3 || idx.dim() != 1)
        refuse(PyExc_ValueError, "state must be [pool, H, P, N], q and k [tokens, G, N], v [tokens, H, P], "
                                 "state_batch_indices [batch]");
    const bool prompts = o[5] != Py_None;
    const int64_t H = state.size(1), P = state.size(2), N = state.size(3), T = q.size(0), G = q.size(1), B = idx.size(0);
    if (!prompts && T != B)
        refuse(PyExc_ValueError, "q has " + std::to_string(T) + " tokens for " + std::to_string(B) + " requests");
    a.batch = i32(B, "batch");
    a.nheads = i32(H, "H");
    a.headdim = i32(P, "P");
    a.dstate = i32(N, "N");
    a.ngroups = i32(G, "G");
    a.device = gpu;
    a.ntokens = T;
    a.pool_slots = state.size(0);
    a.scale = number(o[8]);
    a.state = view(state, "state", {a.pool_slots, H, P, N}, {at::kFloat}, gpu);
    a.idx = view(idx, "state_batch_indices", {B}, {at::kInt, at::kLong}, gpu);
    a.cu_seqlens = view_or_none(o[5], "cu_seqlens", {B + 1}, {at::kInt}, gpu);
    a.q = view(q, "q", {T, G, N}, {at::kBFloat16}, gpu);
    a.k = view(o[2], "k", {T, G, N}, {at::kBFloat16}, gpu);
    a.v = view(v, "v", {T, H, P}, {at::kBFloat16}, gpu);
    if (decay.dim() == 1) {  // one rate for each head
        a.log_decay = view(decay, "log_decay", {H}, {at::kFloat}, gpu);
        a.log_decay.stride[1] = a.log_decay.stride[0];
        a.log_decay.stride[0] = 0;
    } else {
        a.log_decay = view(decay, "log_decay", {T, H}, {at::kFloat}, gpu);
    }
    a.beta = view_or_none(o[7], "beta", {T, H}, {at::kFloat}, gpu);
    const at::Tensor out = given_or(o[9], "out", {T, H, P}, at::kBFloat16, gpu);
    a.out = view(out, "out", {T, H, P}, {at::kBFloat16}, gpu);
    at::Tensor keep;
    if (prompts)
        workspace(o[10], fn.need(&a), gpu, a, keep);
    call(prompts ? fn.prompts : fn.step, a, gpu, prompts ? fn.where : fn.where_step);
    return object(o[9], out);
}

// linear(state, q, k, v, log_decay, cu_seqlens | None, idx, beta | None, scale, out | None, workspace | None)
PyObject *linear(PyObject *, PyObject *const *o, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    count(n, 11);
    return recurrence(kLinear, {}, o);
    END_HANDLE_TH_ERRORS
}

// delta(the same, normalize)
PyObject *delta(PyObject *, PyObject *const *o, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    count(n, 12);
    ssu_delta_args a{};
    a.normalize = truth(o[11]);
    return recurrence(kDelta, a, o);
    END_HANDLE_TH_ERRORS
}

// norm(x, residual | None, weight | None, eps, quantize, group, out | None, scales | None)
PyObject *norm(PyObject *, PyObject *const *o, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    count(n, 8);
    const at::Tensor &x = tensor(o[0], "x");
    const int gpu = gpu_of(x, "x");
    if (x.dim() != 2)
        refuse(PyExc_ValueError, "x must be [tokens, D]");
    const at::ScalarType type = x.scalar_type();
    const Types half = {type}, wide = {type, at::kFloat}, eight = {at::kFloat8_e4m3fn};
    if (type != at::kBFloat16 && type != at::kHalf)
        refuse(PyExc_TypeError, std::string("x: dtype ") + c10::toString(type) + " not supported here");
    const bool quantize = truth(o[4]);
    const int64_t T = x.size(0), D = x.size(1), group = integer(o[5]);
    if (!quantize && (group != 0 || o[7] != Py_None))
        refuse(PyExc_ValueError, "group and scales go with quantize");
    if (group < 0 || (group > 0 && D % group))
        refuse(PyExc_ValueError, "group " + std::to_string(group) + " does not divide D = " + std::to_string(D));
    ssu_norm_args a{};
    a.ntokens = T;
    a.width = i32(D, "D");
    a.group = i32(group, "group");
    a.device = gpu;
    a.eps = number(o[3]);
    a.x = view(x, "x", {T, D}, half, gpu);
    a.residual = view_or_none(o[1], "residual", {T, D}, wide, gpu);
    a.weight = view_or_none(o[2], "weight", {D}, wide, gpu);
    const at::Tensor out = given_or(o[6], "out", {T, D}, quantize ? at::kFloat8_e4m3fn : type, gpu);
    a.out = view(out, "out", {T, D}, quantize ? eight : half, gpu);
    at::Tensor scales;
    if (quantize) {
        const int64_t shape[] = {T, group > 0 ? D / group : 1};
        scales = given_or(o[7], "scales", shape, at::kFloat, gpu);
        a.scales = view(scales, "scales", shape, {at::kFloat}, gpu);
    }
    call(&ssu_add_rms_norm, a, gpu, "ssu_add_rms_norm");
    if (!quantize)
        return object(o[6], out);
    PyObject *const first = object(o[6], out);
    return Py_BuildValue("(NN)", first, object(o[7], scales));
    END_HANDLE_TH_ERRORS
}

// qk(q, k, positions, cos_sin, q_weight | None, k_weight | None, eps, interleaved, q_out | None, k_out | None,
//    v | None, k_cache | None, v_cache | None, slots | None)
PyObject *qk(PyObject *, PyObject *const *o, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    count(n, 14);
    const at::Tensor &q = tensor(o[0], "q"), &k = tensor(o[1], "k"), &cos_sin = tensor(o[3], "cos_sin");
    const int gpu = gpu_of(q, "q");
    if (q.dim() != 3 || k.dim() != 3 || cos_sin.dim() != 2)
        refuse(PyExc_ValueError, "q must be [tokens, Hq, D], k [tokens, Hk, D], cos_sin [max_pos, rot]");
    const bool cached = o[11] != Py_None;
    if ((o[10] != Py_None) != cached || (o[12] != Py_None) != cached || (o[13] != Py_None) != cached)
        refuse(PyExc_ValueError, "v, k_cache, v_cache and slots go together");
    const at::ScalarType type = q.scalar_type();
    const Types half = {type}, weight = {type, at::kFloat}, ints = {at::kInt, at::kLong};
    if (type != at::kBFloat16 && type != at::kHalf)
        refuse(PyExc_TypeError, std::string("q: dtype ") + c10::toString(type) + " not supported here");
    const int64_t T = q.size(0), nq = q.size(1), D = q.size(2), nk = k.size(1);
    ssu_qk_args a{};
    a.ntokens = T;
    a.nq = i32(nq, "Hq");
    a.nk = i32(nk, "Hk");
    a.headdim = i32(D, "D");
    a.rot = i32(cos_sin.size(1), "rot");
    a.interleaved = truth(o[7]);
    a.device = gpu;
    a.eps = number(o[6]);
    a.max_pos = cos_sin.size(0);
    a.q = view(q, "q", {T, nq, D}, half, gpu);
    a.k = view(k, "k", {T, nk, D}, half, gpu);
    a.q_weight = view_or_none(o[4], "q_weight", {D}, weight, gpu);
    a.k_weight = view_or_none(o[5], "k_weight", {D}, weight, gpu);
    a.positions = view(o[2], "positions", {T}, ints, gpu);
    a.cos_sin = view(cos_sin, "cos_sin", {a.max_pos, a.rot}, {at::kFloat}, gpu);
    if (cached) {
        const at::Tensor &cache = tensor(o[11], "k_cache");
        if (cache.dim() != 4)
            refuse(PyExc_ValueError, "k_cache must be [pages, page_size, Hk, D]");
        a.num_pages = cache.size(0);
        a.page_size = i32(cache.size(1), "page_size");
        const int64_t shape[] = {a.num_pages, a.page_size, nk, D};
        a.v = view(o[10], "v", {T, nk, D}, half, gpu);
        a.k_cache = view(cache, "k_cache", shape, half, gpu);
        a.v_cache = view(o[12], "v_cache", shape, half, gpu);
        a.slots = view(o[13], "slots", {T}, ints, gpu);
    }
    const at::Tensor q_out = given_or(o[8], "q_out", {T, nq, D}, type, gpu);
    a.q_out = view(q_out, "q_out", {T, nq, D}, half, gpu);
    const bool to_k = !cached || o[9] != Py_None;
    at::Tensor k_out;
    if (to_k) {
        k_out = given_or(o[9], "k_out", {T, nk, D}, type, gpu);
        a.k_out = view(k_out, "k_out", {T, nk, D}, half, gpu);
    }
    call(&ssu_qk_norm_rope, a, gpu, "ssu_qk_norm_rope");
    PyObject *const first = object(o[8], q_out);
    PyObject *second = Py_None;
    if (to_k)
        second = object(o[9], k_out);
    else
        Py_INCREF(second);
    return Py_BuildValue("(NN)", first, second);
    END_HANDLE_TH_ERRORS
}

// What both attentions share: o: q, k_cache, v_cache, block_table, seq_lens, scale | None, out | None, return_lse,
// workspace | None. `fill` sets what only one of them has.
template <typename Args, typename Fill>
PyObject *attend(PyObject *const *o, Fill fill, int64_t (*need)(const Args *), ssu_status (*fn)(const Args *, hipStream_t),
                 const char *where)
{
    const at::Tensor &q = tensor(o[0], "q"), &cache = tensor(o[1], "k_cache"), &table = tensor(o[3], "block_table");
    const int gpu = gpu_of(q, "q");
    if (q.dim() != 3 || cache.dim() != 4 || table.dim() != 2)
        refuse(PyExc_ValueError,
               "q must be [batch, Hq, D], k_cache [pages, page_size, Hk, D], block_table [batch, max_pages]");
    const at::ScalarType type = q.scalar_type();
    const Types half = {type};
    if (type != at::kBFloat16 && type != at::kHalf)
        refuse(PyExc_TypeError, std::string("q: dtype ") + c10::toString(type) + " not supported here");
    const int64_t B = q.size(0), nq = q.size(1), D = q.size(2);
    Args args{};
    ssu_attn_args &a = fill(args, gpu);
    a.batch = i32(B, "batch");
    a.nq = i32(nq, "Hq");
    a.nk = i32(cache.size(2), "Hk");
    a.headdim = i32(D, "D");
    a.page_size = i32(cache.size(1), "page_size");
    a.device = gpu;
    a.num_pages = cache.size(0);
    a.max_pages = table.size(1);
    a.scale = o[5] == Py_None ? static_cast<float>(1.0 / std::sqrt(static_cast<double>(D))) : number(o[5]);
    const int64_t shape[] = {a.num_pages, a.page_size, a.nk, D};
    a.q = view(q, "q", {B, nq, D}, half, gpu);
    a.k_cache = view(cache, "k_cache", shape, half, gpu);
    a.v_cache = view(o[2], "v_cache", shape, half, gpu);
    a.block_table = view(table, "block_table", {B, a.max_pages}, {at::kInt}, gpu);
    a.seq_lens = view(o[4], "seq_lens", {B}, {at::kInt}, gpu);
    const at::Tensor out = given_or(o[6], "out", {B, nq, D}, type, gpu);
    a.out = view(out, "out", {B, nq, D}, half, gpu);
    const bool with_lse = truth(o[7]);
    at::Tensor lse, keep;
    if (with_lse) {
        lse = make({B, nq}, at::kFloat, gpu);
        a.lse = view(lse, "lse", {B, nq}, {at::kFloat}, gpu);
    }
    workspace(o[8], need(&args), gpu, a, keep);
    call(fn, args, gpu, where);
    if (!with_lse)
        return object(o[6], out);
    PyObject *const first = object(o[6], out);
    return Py_BuildValue("(NN)", first, THPVariable_Wrap(lse));
}

// attention(as in attend)
PyObject *attention(PyObject *, PyObject *const *o, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    count(n, 9);
    const auto fill = [](ssu_attn_args &a, int) -> ssu_attn_args & { return a; };
    return attend<ssu_attn_args>(o, fill, &ssu_paged_attention_workspace, &ssu_paged_attention, "ssu_paged_attention");
    END_HANDLE_TH_ERRORS
}

// shared(as in attend, prefix_table, prefix_len)
PyObject *shared(PyObject *, PyObject *const *o, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    count(n, 11);
    const auto fill = [o](ssu_shared_args &a, int gpu) -> ssu_attn_args & {
        const at::Tensor &prefix = tensor(o[9], "prefix_table");
        if (prefix.dim() != 1)
            refuse(PyExc_ValueError, "prefix_table must be [prefix_pages]");
        a.prefix_pages = prefix.size(0);
        a.prefix_table = view(prefix, "prefix_table", {a.prefix_pages}, {at::kInt}, gpu);
        a.prefix_len = view(o[10], "prefix_len", {1}, {at::kInt}, gpu);
        return a.attn;
    };
    return attend<ssu_shared_args>(o, fill, &ssu_shared_prefix_attention_workspace, &ssu_shared_prefix_attention,
                                   "ssu_shared_prefix_attention");
    END_HANDLE_TH_ERRORS
}

PyObject *bytes_of(int64_t n)
{
    if (n < 0)
        refuse(PyExc_ValueError, ssu_last_error());
    return PyLong_FromLongLong(n);
}

template <typename Args>
PyObject *recurrence_workspace(const Recurrence<Args> &fn, PyObject *const *o)
{
    Args a{};
    a.batch = i32(integer(o[0]), "batch");
    a.ntokens = integer(o[1]);
    a.nheads = i32(integer(o[2]), "H");
    a.headdim = i32(integer(o[3]), "P");
    a.dstate = i32(integer(o[4]), "N");
    a.ngroups = i32(integer(o[5]), "G");
    return bytes_of(fn.need(&a));
}

// linear_workspace(batch, ntokens, H, P, N, G)
PyObject *linear_workspace(PyObject *, PyObject *const *o, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    count(n, 6);
    return recurrence_workspace(kLinear, o);
    END_HANDLE_TH_ERRORS
}

// delta_workspace(the same)
PyObject *delta_workspace(PyObject *, PyObject *const *o, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    count(n, 6);
    return recurrence_workspace(kDelta, o);
    END_HANDLE_TH_ERRORS
}

ssu_attn_args attention_sizes(PyObject *const *o)
{
    ssu_attn_args a{};
    a.batch = i32(integer(o[0]), "batch");
    a.nq = i32(integer(o[1]), "Hq");
    a.nk = i32(integer(o[2]), "Hk");
    a.headdim = i32(integer(o[3]), "D");
    a.page_size = i32(integer(o[4]), "page_size");
    a.max_pages = integer(o[5]);
    return a;
}

// shared_workspace(batch, Hq, Hk, D, page_size, max_pages, prefix_pages)
PyObject *shared_workspace(PyObject *, PyObject *const *o, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    count(n, 7);
    ssu_shared_args a{};
    a.attn = attention_sizes(o);
    a.prefix_pages = integer(o[6]);
    return bytes_of(ssu_shared_prefix_attention_workspace(&a));
    END_HANDLE_TH_ERRORS
}

// attention_workspace(batch, Hq, Hk, D, page_size, max_pages)
PyObject *attention_workspace(PyObject *, PyObject *const *o, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    count(n, 6);
    const ssu_attn_args a = attention_sizes(o);
    return bytes_of(ssu_paged_attention_workspace(&a));
    END_HANDLE_TH_ERRORS
}

PyObject *errors(PyObject *, PyObject *cls)
{
    Py_INCREF(cls);
    Py_XSETREF(g_error, cls);
    Py_RETURN_NONE;
}

template <PyObject *(*F)(PyObject *, PyObject *const *, Py_ssize_t)>
PyCFunction fast()
{
    return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(F));
}

PyMethodDef methods[] = {
    {"linear", fast<linear>(), METH_FASTCALL, nullptr},
    {"delta", fast<delta>(), METH_FASTCALL, nullptr},
    {"norm", fast<norm>(), METH_FASTCALL, nullptr},
    {"qk", fast<qk>(), METH_FASTCALL, nullptr},
    {"attention", fast<attention>(), METH_FASTCALL, nullptr},
    {"shared", fast<shared>(), METH_FASTCALL, nullptr},
    {"linear_workspace", fast<linear_workspace>(), METH_FASTCALL, nullptr},
    {"delta_workspace", fast<delta_workspace>(), METH_FASTCALL, nullptr},
    {"shared_workspace", fast<shared_workspace>(), METH_FASTCALL, nullptr},
    {"attention_workspace", fast<attention_workspace>(), METH_FASTCALL, nullptr},
    {"errors", errors, METH_O, "Set the class that a failed call raises: cls(status, where)."},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_native", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__native() { return PyModule_Create(&module); }
