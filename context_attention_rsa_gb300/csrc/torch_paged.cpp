// The Python binding of the paged-cache calls, compiled: it checks torch tensors,
// makes the outputs that the caller did not pass and calls the C ABI (rsa.h) on
// the tensors' device and stream.
//
// A decode step makes these calls once a layer, on kernels of 7 to 15 us.  The same
// checks and allocations in Python took 20 to 35 us a call, more than the kernels;
// in here they take a few.  The functions of librsa are not linked: bind() gets
// their addresses from the library that the package has loaded (the RSA_DEBUG
// variant has the same).
#include <Python.h>

#include <ATen/Context.h>
#include <ATen/ops/empty.h>
#include <c10/core/impl/TorchDispatchModeTLS.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <ATen/cuda/EmptyTensor.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <initializer_list>
#include <string>
#include <vector>

#include "rsa.h"

namespace {

decltype(&rsa_page_plan) page_plan_fn;
decltype(&rsa_qk_norm_rope_fwd) rope_fn;
decltype(&rsa_qk_norm_rope_bwd) rope_bwd_fn;
decltype(&rsa_qk_norm_rope_bwd_workspace_size) rope_bwd_size_fn;
decltype(&rsa_prefix_attn_fwd) attn_fn;
decltype(&rsa_prefix_attn_workspace_size) attn_size_fn;
decltype(&rsa_tree_plan) tree_plan_fn;
decltype(&rsa_tree_attn_fwd) tree_attn_fn;
decltype(&rsa_tree_attn_workspace_size) tree_attn_size_fn;
decltype(&rsa_cache_compact) compact_fn;
decltype(&rsa_page_fork) fork_fn;
decltype(&rsa_page_free) free_fn;
PyObject *share_fn;  // (stream, device index, tensors): memory of the current stream used on another one

// A Python exception to raise.
struct Refusal {
    PyObject *type;
    std::string text;
};
struct Raised {};  // ... which is set already

[[noreturn]] void type_error(const std::string &s) { throw Refusal{PyExc_TypeError, s}; }
[[noreturn]] void value_error(const std::string &s) { throw Refusal{PyExc_ValueError, s}; }

int64_t integer(PyObject *o)
{
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred())
        throw Raised();
    return v;
}

int small_integer(PyObject *o, const char *name)
{
    const int64_t v = integer(o);
    if (v < INT32_MIN || v > INT32_MAX)
        value_error(std::string(name) + " does not fit 32 bits");
    return (int)v;
}

std::string text(const at::IntArrayRef &shape)
{
    std::string s = "(";
    for (size_t i = 0; i < shape.size(); ++i)
        s += (i ? ", " : "") + std::to_string(shape[i]);
    return s + ")";
}

const at::Tensor &on_device(const char *name, PyObject *o, const c10::Device &dev)
{
    if (!THPVariable_Check(o) || !THPVariable_Unpack(o).is_cuda() || THPVariable_Unpack(o).device() != dev)
        type_error(std::string(name) + " must be a CUDA tensor on " + dev.str());
    return THPVariable_Unpack(o);
}

const at::Tensor &check(const char *name, PyObject *o, int64_t dim, at::ScalarType type, const c10::Device &dev,
                        bool contiguous = true)
{
    const at::Tensor &t = on_device(name, o, dev);
    if (t.scalar_type() != type || t.dim() != dim)
        value_error(std::string(name) + " must be a " + std::to_string(dim) + "-d " + c10::toString(type) + " tensor (got " +
                    std::to_string(t.dim()) + "-d " + c10::toString(t.scalar_type()) + ")");
    if (contiguous && !t.is_contiguous())
        value_error(std::string(name) + " must be contiguous");
    return t;
}

// A [T, H, d] operand (of shape `want`, if given).
rsa_heads rows(const char *name, PyObject *o, at::ScalarType type, const c10::Device &dev, const at::Tensor *want = nullptr)
{
    const at::Tensor &t = check(name, o, 3, type, dev, false);
    if (want && t.sizes() != want->sizes())
        value_error(std::string(name) + " must be " + text(want->sizes()) + " (got " + text(t.sizes()) + ")");
    if (t.stride(2) != 1)
        value_error(std::string("the last dimension of ") + name + " must be contiguous");
    // the stride of a dimension of one says nothing: put the dense one in its place
    const int64_t head = t.size(1) == 1 ? t.size(2) : t.stride(1);
    return rsa_heads{t.data_ptr(), t.size(0) == 1 ? t.size(1) * head : t.stride(0), head};
}

rsa_heads dense_rows(const at::Tensor &t) { return rsa_heads{t.data_ptr(), t.size(1) * t.size(2), t.size(2)}; }

// q [T, Hq, d], which says the call's type and device.
const at::Tensor &queries(PyObject *o, rsa_dtype *dt)
{
    if (!THPVariable_Check(o) || !THPVariable_Unpack(o).is_cuda() || THPVariable_Unpack(o).dim() != 3)
        type_error("q must be a CUDA tensor [T, Hq, d]");
    const at::Tensor &q = THPVariable_Unpack(o);
    if (q.scalar_type() == at::kFloat)
        *dt = RSA_F32;
    else if (q.scalar_type() == at::kBFloat16)
        *dt = RSA_BF16;
    else
        type_error(std::string("unsupported dtype ") + c10::toString(q.scalar_type()) + " (float32 or bfloat16)");
    return q;
}

const at::Tensor &workspace(PyObject *o, const c10::Device &dev)
{
    const at::Tensor &t = on_device("workspace", o, dev);
    if (!t.is_contiguous())
        value_error("workspace must be contiguous");
    return t;
}

// One call: its device, its stream, and the tensors that it made.
class Call {
public:
    // Straight from the allocator, 1 to 2 us a call less than by way of the dispatcher,
    // unless that would do more: a mode sees the tensor, or its memory is filled.
    Call(const c10::Device &dev, PyObject *stream) : dev_(dev), guard_(dev), stream_(stream)
    {
        const at::Context &c = at::globalContext();
        plain_ = !c10::impl::TorchDispatchModeTLS::any_modes_set() &&
                 !(c.deterministicAlgorithms() && c.deterministicFillUninitializedMemory());
    }

    at::Tensor make(at::IntArrayRef shape, at::ScalarType type)
    {
        if (plain_)
            made_.push_back(at::detail::empty_cuda(shape, type, dev_, std::nullopt));
        else
            made_.push_back(at::empty(shape, at::TensorOptions(dev_).dtype(type)));
        return made_.back();
    }

    // The handle of the call's stream: the device's current one, or what the caller
    // passed.  Tensors made on the current stream and used on another one: their memory
    // may still be in use there, and is not to be handed out again before the call is done.
    rsa_stream_t stream()
    {
        const rsa_stream_t current = c10::cuda::getCurrentCUDAStream(dev_.index()).stream();
        if (stream_ == Py_None)
            return current;
        PyObject *h = PyObject_GetAttrString(stream_, "cuda_stream");
        const bool bare = h == nullptr;
        if (bare) {
            PyErr_Clear();
            h = Py_NewRef(stream_);
        }
        const unsigned long long v = PyLong_AsUnsignedLongLong(h);
        Py_DECREF(h);
        if (PyErr_Occurred())
            throw Raised();
        const rsa_stream_t handle = reinterpret_cast<rsa_stream_t>(v);
        if (handle == current || made_.empty())
            return handle;
        if (bare)
            value_error("with a bare stream handle other than the current stream's, pass every output and workspace");
        PyObject *list = PyList_New(0);
        bool ok = list != nullptr;
        for (size_t i = 0; ok && i < made_.size(); ++i) {
            PyObject *t = THPVariable_Wrap(made_[i]);
            ok = t && PyList_Append(list, t) == 0;
            Py_XDECREF(t);
        }
        PyObject *r = ok ? PyObject_CallFunction(share_fn, "OiO", stream_, (int)dev_.index(), list) : nullptr;
        Py_XDECREF(list);
        if (!r)
            throw Raised();
        Py_DECREF(r);
        return handle;
    }

private:
    c10::Device dev_;
    c10::cuda::CUDAGuard guard_;
    PyObject *stream_;
    bool plain_;
    std::vector<at::Tensor> made_;
};

// A call that takes a while if the device's queue is full.
template <class F>
rsa_status launch(F f)
{
    rsa_status st;
    Py_BEGIN_ALLOW_THREADS
    st = f();
    Py_END_ALLOW_THREADS
    return st;
}

// The results, None for those that are not defined; or the status of a refused call.
PyObject *results(rsa_status st, std::initializer_list<at::Tensor> ts)
{
    if (st != RSA_OK)
        return PyLong_FromLong(st);
    PyObject *out = PyTuple_New((Py_ssize_t)ts.size());
    if (!out)
        throw Raised();
    Py_ssize_t i = 0;
    for (const at::Tensor &t : ts) {
        PyObject *o = t.defined() ? THPVariable_Wrap(t) : Py_NewRef(Py_None);
        if (!o) {
            Py_DECREF(out);
            throw Raised();
        }
        PyTuple_SET_ITEM(out, i++, o);
    }
    return out;
}

void caches(PyObject *ko, PyObject *vo, int64_t Hkv, int64_t d, at::ScalarType type, const c10::Device &dev, const at::Tensor **k,
            const at::Tensor **v)
{
    *k = &check("k_cache", ko, 4, type, dev);
    *v = &check("v_cache", vo, 4, type, dev);
    const auto s = (*k)->sizes();
    if ((*v)->sizes() != s || s[1] != Hkv || s[3] != d)
        value_error("k_cache and v_cache must both be [n_pages, Hkv=" + std::to_string(Hkv) + ", page_size, d=" +
                    std::to_string(d) + "]");
}

int64_t table_stride(const at::Tensor &t)
{
    if (t.stride(1) != 1 && t.size(1) > 1)
        value_error("rows of block_table must be contiguous");
    return t.size(0) == 1 ? t.size(1) : t.stride(0);
}

// cached_len, new_len, block_table, free_pages, page_size, n_pages, max_tokens, free_start, pos0, out, stream
PyObject *page_plan(PyObject *const *a)
{
    if (!THPVariable_Check(a[0]) || !THPVariable_Unpack(a[0]).is_cuda())
        type_error("cached_len must be a CUDA tensor");
    const c10::Device dev = THPVariable_Unpack(a[0]).device();
    const at::Tensor &cached = check("cached_len", a[0], 1, at::kInt, dev), &fresh = check("new_len", a[1], 1, at::kInt, dev);
    const at::Tensor &table = check("block_table", a[2], 2, at::kInt, dev, false);
    const at::Tensor &pages = check("free_pages", a[3], 1, at::kInt, dev);
    const int64_t R = cached.size(0), max_pages = table.size(1);
    if (fresh.size(0) != R || table.size(0) != R)
        value_error("new_len and block_table must have cached_len's requests");
    if (R > INT32_MAX || max_pages > INT32_MAX)
        value_error("block_table is too large");
    const int64_t stride = table_stride(table);
    const int page_size = small_integer(a[4], "page_size");
    const int64_t n_pages = integer(a[5]), max_tokens = integer(a[6]), pos0 = integer(a[8]);
    const int64_t *start = nullptr;
    if (a[7] != Py_None) {
        const at::Tensor &t = check("free_start", a[7], 1, at::kLong, dev);
        if (t.size(0) < 1)
            value_error("free_start must hold one entry");
        start = t.data_ptr<int64_t>();
    }
    if (max_tokens < 0)
        value_error("max_tokens must be >= 0");
    Call call(dev, a[10]);
    at::Tensor cu, kv, slots, pos, info;
    if (a[9] == Py_None) {
        cu = call.make({R + 1}, at::kInt);
        kv = call.make({R}, at::kInt);
        slots = call.make({max_tokens}, at::kLong);
        pos = call.make({max_tokens}, at::kLong);
        info = call.make({4}, at::kLong);
    } else {
        if (!PyTuple_Check(a[9]) || PyTuple_GET_SIZE(a[9]) != 5)
            type_error("out must be a PagePlan");
        auto given = [&](int i, const char *name, at::ScalarType type, int64_t n) {
            const at::Tensor &t = check(name, PyTuple_GET_ITEM(a[9], i), 1, type, dev);
            if (t.size(0) != n)
                value_error(std::string(name) + " must hold " + std::to_string(n) + " entries");
            return t;
        };
        cu = given(0, "out.cu_new", at::kInt, R + 1);
        kv = given(1, "out.kv_len", at::kInt, R);
        slots = given(2, "out.slot_map", at::kLong, max_tokens);
        pos = given(3, "out.positions", at::kLong, max_tokens);
        info = given(4, "out.info", at::kLong, 4);
    }
    const rsa_stream_t stream = call.stream();
    const rsa_status st = launch([&] {
        return page_plan_fn(cached.data_ptr<int>(), fresh.data_ptr<int>(), (int)R, page_size, n_pages, table.data_ptr<int>(), stride,
                            (int)max_pages, pages.data_ptr<int>(), pages.size(0), start, pos0, max_tokens, cu.data_ptr<int>(),
                            kv.data_ptr<int>(), slots.data_ptr<int64_t>(), pos.data_ptr<int64_t>(), info.data_ptr<int64_t>(), stream);
    });
    return results(st, {cu, kv, slots, pos, info});
}

// q, k, q_weight, k_weight, positions, cos_sin, eps, interleaved, sections
rsa_qk_norm_rope_args norm_rope_args(PyObject *const *a, const at::Tensor **q_, const at::Tensor **k_)
{
    rsa_qk_norm_rope_args r = {};
    const at::Tensor &q = queries(a[0], &r.dt);
    const c10::Device dev = q.device();
    const at::ScalarType type = q.scalar_type();
    r.q = rows("q", a[0], type, dev);
    r.k = rows("k", a[1], type, dev);
    const at::Tensor &k = THPVariable_Unpack(a[1]);
    if (k.size(0) != q.size(0) || k.size(2) != q.size(2))
        value_error("q [T, Hq, d] and k [T, Hkv, d] must agree");
    if (q.size(1) > INT32_MAX || k.size(1) > INT32_MAX || q.size(2) > INT32_MAX)
        value_error("too many heads");
    r.T = q.size(0);
    r.Hq = (int)q.size(1);
    r.Hkv = (int)k.size(1);
    r.d = (int)q.size(2);
    for (int i = 0; i < 2; ++i) {
        if (a[2 + i] == Py_None)
            continue;
        const at::Tensor &w = check(i ? "k_weight" : "q_weight", a[2 + i], 1, type, dev);
        if (w.size(0) != r.d)
            value_error("q_weight and k_weight must hold d=" + std::to_string(r.d) + " values");
        (i ? r.k_weight : r.q_weight) = w.data_ptr();
    }
    const double eps = PyFloat_AsDouble(a[6]);
    if (eps == -1.0 && PyErr_Occurred())
        throw Raised();
    r.eps = (float)eps;
    r.interleaved = PyObject_IsTrue(a[7]);
    if (r.interleaved < 0)
        throw Raised();
    r.n_axes = 1;
    if (a[5] != Py_None) {
        const at::Tensor &table = check("cos_sin", a[5], 2, at::kFloat, dev);
        if (table.size(1) > INT32_MAX)
            value_error("cos_sin is too wide");
        r.max_pos = table.size(0);
        r.rot = (int)table.size(1);
        r.cos_sin = table.data_ptr<float>();
        if (a[8] != Py_None) {
            PyObject *s = PySequence_Fast(a[8], "sections must be a sequence");
            if (!s)
                throw Raised();
            const Py_ssize_t n = PySequence_Fast_GET_SIZE(s);
            bool ok = n >= 1 && n <= 4;
            for (Py_ssize_t i = 0; ok && i < n; ++i) {
                const long v = PyLong_AsLong(PySequence_Fast_GET_ITEM(s, i));
                if (PyErr_Occurred()) {
                    Py_DECREF(s);
                    throw Raised();
                }
                r.sections[i] = v < -1 || v > r.d ? -1 : (int)v;  // (the call refuses it)
            }
            Py_DECREF(s);
            if (!ok)
                value_error("sections must name one to four axes");
            r.n_axes = (int)n;
            if (n == 1 && r.sections[0] != r.rot / 2)
                value_error("one section must hold all rot/2 frequencies");
        }
        if (!THPVariable_Check(a[4]))
            type_error("positions must be a CUDA tensor");
        const at::Tensor &pos = check("positions", a[4], r.n_axes == 1 ? THPVariable_Unpack(a[4]).dim() : 2, at::kLong, dev);
        if (pos.dim() < 1 || pos.size(-1) != r.T || pos.numel() != r.n_axes * r.T)
            value_error("positions must be int64 [" + (r.n_axes > 1 ? std::to_string(r.n_axes) + ", " : std::string()) +
                        std::to_string(r.T) + "]");
        r.positions = pos.data_ptr<int64_t>();
    }
    *q_ = &q;
    *k_ = &k;
    return r;
}

// A result of `like`'s shape: the caller's, or a new one.
rsa_heads result_rows(Call &call, const char *name, PyObject *given, const at::Tensor &like, at::Tensor *t)
{
    if (given != Py_None) {
        *t = on_device(name, given, like.device());
        return rows(name, given, like.scalar_type(), like.device(), &like);
    }
    *t = call.make(like.sizes(), like.scalar_type());
    return dense_rows(*t);
}

// ..., v, slot_map, k_cache, v_cache, q_out, k_out, stream
PyObject *qk_norm_rope(PyObject *const *a)
{
    const at::Tensor *q, *k, *kc = nullptr, *vc = nullptr;
    const rsa_qk_norm_rope_args args = norm_rope_args(a, &q, &k);
    const c10::Device dev = q->device();
    Call call(dev, a[15]);
    at::Tensor qt, kt;
    const rsa_heads qo = result_rows(call, "q_out", a[13], *q, &qt);
    rsa_heads ko = {}, v = {};
    const bool cache = a[10] != Py_None;
    if (a[14] != Py_None || !cache)
        ko = result_rows(call, "k_out", a[14], *k, &kt);
    const int64_t *slots = nullptr;
    int64_t n_pages = 0, page_size = 0;
    if (cache) {
        const at::Tensor &s = check("slot_map", a[10], 1, at::kLong, dev);
        if (s.size(0) != args.T)
            value_error("slot_map must hold T=" + std::to_string(args.T) + " slots");
        slots = s.data_ptr<int64_t>();
        v = rows("v", a[9], q->scalar_type(), dev, k);
        caches(a[11], a[12], args.Hkv, args.d, q->scalar_type(), dev, &kc, &vc);
        n_pages = kc->size(0);
        page_size = std::min<int64_t>(kc->size(2), INT32_MAX);
    } else if (a[9] != Py_None || a[11] != Py_None || a[12] != Py_None) {
        value_error("v, k_cache and v_cache go with slot_map");
    }
    const rsa_stream_t stream = call.stream();
    const rsa_status st = launch([&] {
        return rope_fn(&args, qo, ko, v, slots, kc ? kc->data_ptr() : nullptr, vc ? vc->data_ptr() : nullptr, (int)page_size, n_pages,
                       stream);
    });
    return results(st, {qt, kt});
}

// ..., dq_out, dk_out, dq, dk, dq_weight, dk_weight, workspace, stream
PyObject *qk_norm_rope_bwd(PyObject *const *a)
{
    const at::Tensor *q, *k;
    const rsa_qk_norm_rope_args args = norm_rope_args(a, &q, &k);
    const c10::Device dev = q->device();
    const rsa_heads gq = rows("dq_out", a[9], q->scalar_type(), dev, q), gk = rows("dk_out", a[10], q->scalar_type(), dev, k);
    Call call(dev, a[16]);
    at::Tensor dq, dk, dw[2], ws;
    const rsa_heads dqo = result_rows(call, "dq", a[11], *q, &dq), dko = result_rows(call, "dk", a[12], *k, &dk);
    for (int i = 0; i < 2; ++i) {
        if (a[13 + i] != Py_None) {
            dw[i] = check(i ? "dk_weight" : "dq_weight", a[13 + i], 1, at::kFloat, dev);
            if (dw[i].size(0) != args.d)
                value_error("dq_weight and dk_weight must hold d=" + std::to_string(args.d) + " values");
        } else if (i ? args.k_weight : args.q_weight) {
            dw[i] = call.make({args.d}, at::kFloat);
        }
    }
    if (a[15] != Py_None) {
        ws = workspace(a[15], dev);
    } else {
        size_t n = 0;
        const rsa_status st = rope_bwd_size_fn(args.d, &n);
        if (st != RSA_OK)
            return PyLong_FromLong(st);
        ws = call.make({(int64_t)n}, at::kByte);
    }
    const rsa_stream_t stream = call.stream();
    const rsa_status st = launch([&] {
        return rope_bwd_fn(&args, gq, gk, dqo, dko, dw[0].defined() ? dw[0].data_ptr<float>() : nullptr,
                           dw[1].defined() ? dw[1].data_ptr<float>() : nullptr, ws.data_ptr(), ws.nbytes(), stream);
    });
    return results(st, {dq, dk, dw[0], dw[1]});
}

// q, k_cache, v_cache, cu_q, block_table, kv_len, then those of `b`: prefix_pages, prefix_len, out, lse, workspace,
// stream; with a mask (mask_arg) for drafted tokens, or none (NULL).
PyObject *attention(PyObject *const *a, PyObject *mask_arg, PyObject *const *b)
{
    rsa_dtype dt;
    const at::Tensor &q = queries(a[0], &dt);
    const c10::Device dev = q.device();
    const at::ScalarType type = q.scalar_type();
    const rsa_heads qh = rows("q", a[0], type, dev);
    const int64_t T = q.size(0), Hq = q.size(1), d = q.size(2);
    const at::Tensor &first = on_device("k_cache", a[1], dev);
    if (first.dim() != 4)
        value_error("k_cache must be [n_pages, Hkv, page_size, d]");
    const at::Tensor *kc, *vc;
    caches(a[1], a[2], first.size(1), d, type, dev, &kc, &vc);
    const int64_t n_pages = kc->size(0), Hkv = kc->size(1), page_size = kc->size(2);
    const at::Tensor &cu = check("cu_q", a[3], 1, at::kInt, dev), &kv = check("kv_len", a[5], 1, at::kInt, dev);
    const at::Tensor &table = check("block_table", a[4], 2, at::kInt, dev, false);
    const int64_t R = table.size(0), max_pages = table.size(1);
    if (cu.size(0) != R + 1 || kv.size(0) != R)
        value_error("cu_q [R + 1], kv_len [R] and block_table [R, max_pages] must agree");
    if (std::max({Hq, Hkv, d, page_size, R, max_pages}) > INT32_MAX)
        value_error("a dimension does not fit 32 bits");
    const int64_t stride = table_stride(table), prefix_len = integer(b[1]);
    const int32_t *prefix = nullptr;
    if (prefix_len != 0) {
        const at::Tensor &t = check("prefix_pages", b[0], 1, at::kInt, dev);
        if (t.size(0) < prefix_len / std::max<int64_t>(page_size, 1) + (prefix_len % std::max<int64_t>(page_size, 1) > 0))
            value_error("prefix_pages hold " + std::to_string(t.size(0) * page_size) + " tokens, prefix_len is " +
                        std::to_string(prefix_len));
        prefix = t.data_ptr<int>();
    }
    const uint32_t *mask = nullptr;
    int64_t mask_stride = 0, words = 0;
    if (mask_arg) {
        const at::Tensor &t = check("tree_mask", mask_arg, 2, at::kInt, dev, false);
        if (t.size(0) != T)
            value_error("tree_mask must hold T=" + std::to_string(T) + " rows");
        if (t.stride(1) != 1 && t.size(1) > 1)
            value_error("rows of tree_mask must be contiguous");
        mask = static_cast<const uint32_t *>(t.data_ptr());
        words = std::min<int64_t>(t.size(1), INT32_MAX);
        mask_stride = T == 1 ? words : t.stride(0);
    }
    Call call(dev, b[5]);
    at::Tensor out, lse, ws;
    if (b[2] == Py_None) {
        out = call.make(q.sizes(), type);
    } else {
        out = check("out", b[2], 3, type, dev);
        if (out.sizes() != q.sizes())
            value_error("out must have q's shape");
    }
    if (b[3] == Py_None) {
        lse = call.make({T, Hq}, at::kFloat);
    } else {
        lse = check("lse", b[3], 2, at::kFloat, dev);
        if (lse.size(0) != T || lse.size(1) != Hq)
            value_error("lse must be [T, Hq]");
    }
    if (b[4] != Py_None) {
        ws = workspace(b[4], dev);
    } else {
        size_t n = 0;
        const rsa_status st = (mask_arg ? tree_attn_size_fn : attn_size_fn)(dt, T, (int)Hq, (int)Hkv, (int)d, (int)R, &n);
        if (st != RSA_OK)
            return PyLong_FromLong(st);
        ws = call.make({(int64_t)n}, at::kByte);
    }
    const rsa_stream_t stream = call.stream();
    const rsa_status st = launch([&] {
        if (mask_arg)
            return tree_attn_fn(qh.data, qh.token_stride, qh.head_stride, kc->data_ptr(), vc->data_ptr(), dt, T, (int)Hq, (int)Hkv,
                                (int)d, (int)page_size, n_pages, cu.data_ptr<int>(), kv.data_ptr<int>(), (int)R,
                                table.data_ptr<int>(), stride, (int)max_pages, prefix, prefix_len, mask, mask_stride, (int)words,
                                out.data_ptr(), lse.data_ptr<float>(), ws.data_ptr(), ws.nbytes(), stream);
        return attn_fn(qh.data, qh.token_stride, qh.head_stride, kc->data_ptr(), vc->data_ptr(), dt, T, (int)Hq, (int)Hkv, (int)d,
                       (int)page_size, n_pages, cu.data_ptr<int>(), kv.data_ptr<int>(), (int)R, table.data_ptr<int>(), stride,
                       (int)max_pages, prefix, prefix_len, out.data_ptr(), lse.data_ptr<float>(), ws.data_ptr(), ws.nbytes(), stream);
    });
    return results(st, {out, lse});
}

PyObject *prefix_attn(PyObject *const *a) { return attention(a, nullptr, a + 6); }

// ..., kv_len, tree_mask, prefix_pages, ...
PyObject *tree_attn(PyObject *const *a) { return attention(a, a[6], a + 7); }

// A result of `n` entries: the caller's, or a new one.
at::Tensor result_list(Call &call, const char *name, PyObject *given, int64_t n, at::ScalarType type, const c10::Device &dev)
{
    if (given == Py_None)
        return call.make({n}, type);
    const at::Tensor &t = check(name, given, 1, type, dev);
    if (t.size(0) != n)
        value_error(std::string(name) + " must hold " + std::to_string(n) + " entries");
    return t;
}

// A list of `n` (any, if negative) 32-bit integers.
const at::Tensor &list(const char *name, PyObject *o, int64_t n, const c10::Device &dev)
{
    const at::Tensor &t = check(name, o, 1, at::kInt, dev);
    if (n >= 0 && t.size(0) != n)
        value_error(std::string(name) + " must hold " + std::to_string(n) + " entries");
    return t;
}

const int64_t *free_start(PyObject *o, const c10::Device &dev)
{
    if (o == Py_None)
        return nullptr;
    const at::Tensor &t = check("free_start", o, 1, at::kLong, dev);
    if (t.size(0) < 1)
        value_error("free_start must hold one entry");
    return t.data_ptr<int64_t>();
}

c10::Device device_of(const char *name, PyObject *o)
{
    if (!THPVariable_Check(o) || !THPVariable_Unpack(o).is_cuda())
        type_error(std::string(name) + " must be a CUDA tensor");
    return THPVariable_Unpack(o).device();
}

// block_table, whose rows and pages fit 32 bits.
const at::Tensor &tables(PyObject *o, const c10::Device &dev)
{
    const at::Tensor &t = check("block_table", o, 2, at::kInt, dev, false);
    if (t.size(0) > INT32_MAX || t.size(1) > INT32_MAX)
        value_error("block_table is too large");
    return t;
}

// Caches of one layer [n_pages, Hkv, page_size, d] or of several [layers, n_pages, ...].
rsa_cache layers(PyObject *ko, PyObject *vo, const c10::Device &dev)
{
    rsa_cache c = {};
    const at::Tensor &k = on_device("k_cache", ko, dev), &v = on_device("v_cache", vo, dev);
    if ((k.dim() != 4 && k.dim() != 5) || v.sizes() != k.sizes() || v.scalar_type() != k.scalar_type())
        value_error("k_cache and v_cache must both be [n_pages, Hkv, page_size, d] or [layers, n_pages, Hkv, page_size, d]");
    if (!k.is_contiguous() || !v.is_contiguous())
        value_error("k_cache and v_cache must be contiguous");
    if (k.scalar_type() == at::kFloat)
        c.dt = RSA_F32;
    else if (k.scalar_type() == at::kBFloat16)
        c.dt = RSA_BF16;
    else
        type_error(std::string("unsupported dtype ") + c10::toString(k.scalar_type()) + " (float32 or bfloat16)");
    for (int64_t n : k.sizes())
        if (n > INT32_MAX)
            value_error("a dimension does not fit 32 bits");
    const int64_t *s = k.sizes().data() + (k.dim() - 4);
    c.k_cache = k.data_ptr();
    c.v_cache = v.data_ptr();
    c.layers = k.dim() == 5 ? (int)k.size(0) : 1;
    c.n_pages = s[0];
    c.Hkv = (int)s[1];
    c.page_size = (int)s[2];
    c.d = (int)s[3];
    return c;
}

// parent, cu_new, kv_len, max_tree, pos0, out, stream
PyObject *tree_plan(PyObject *const *a)
{
    const c10::Device dev = device_of("parent", a[0]);
    const at::Tensor &parent = list("parent", a[0], -1, dev), &kv = list("kv_len", a[2], -1, dev);
    const int64_t T = parent.size(0), R = kv.size(0);
    if (R >= INT32_MAX)
        value_error("kv_len is too large");
    const at::Tensor &cu = list("cu_new", a[1], R + 1, dev);
    const int64_t most = integer(a[3]), pos0 = integer(a[4]);
    if (most < 1 || most > 1024)
        value_error("max_tree=" + std::to_string(most) + " must be in [1, 1024]");
    const int64_t words = (most + 31) / 32;
    Call call(dev, a[6]);
    at::Tensor pos, mask;
    if (a[5] == Py_None) {
        pos = call.make({T}, at::kLong);
        mask = call.make({T, words}, at::kInt);
    } else {
        if (!PyTuple_Check(a[5]) || PyTuple_GET_SIZE(a[5]) != 2)
            type_error("out must be a TreePlan");
        pos = result_list(call, "out.positions", PyTuple_GET_ITEM(a[5], 0), T, at::kLong, dev);
        mask = check("out.mask", PyTuple_GET_ITEM(a[5], 1), 2, at::kInt, dev);
        if (mask.size(0) != T || mask.size(1) != words)
            value_error("out.mask must be [" + std::to_string(T) + ", " + std::to_string(words) + "]");
    }
    const rsa_stream_t stream = call.stream();
    const rsa_status st = launch([&] {
        return tree_plan_fn(parent.data_ptr<int>(), T, cu.data_ptr<int>(), kv.data_ptr<int>(), (int)R, (int)words, pos0,
                            pos.data_ptr<int64_t>(), static_cast<uint32_t *>(mask.data_ptr()), stream);
    });
    return results(st, {pos, mask});
}

// k_cache, v_cache, block_table, cached_len, kv_len, keep, keep_len, out, stream
PyObject *cache_compact(PyObject *const *a)
{
    const c10::Device dev = device_of("k_cache", a[0]);
    const rsa_cache c = layers(a[0], a[1], dev);
    const at::Tensor &table = tables(a[2], dev);
    const int64_t R = table.size(0), stride = table_stride(table);
    const at::Tensor &cached = list("cached_len", a[3], R, dev), &kv = list("kv_len", a[4], R, dev);
    const at::Tensor &keep = check("keep", a[5], 2, at::kInt, dev, false), &n = list("keep_len", a[6], R, dev);
    if (keep.size(0) != R || keep.size(1) > INT32_MAX || (keep.stride(1) != 1 && keep.size(1) > 1))
        value_error("keep must hold a contiguous row for each of block_table's " + std::to_string(R) + " requests");
    const int64_t keep_stride = R == 1 ? keep.size(1) : keep.stride(0);
    Call call(dev, a[8]);
    const at::Tensor out = result_list(call, "out", a[7], R, at::kInt, dev);
    const rsa_stream_t stream = call.stream();
    const rsa_status st = launch([&] {
        return compact_fn(&c, table.data_ptr<int>(), stride, (int)table.size(1), cached.data_ptr<int>(), kv.data_ptr<int>(), (int)R,
                          keep.data_ptr<int>(), keep_stride, (int)keep.size(1), n.data_ptr<int>(), out.data_ptr<int>(), stream);
    });
    return results(st, {out});
}

// k_cache, v_cache, block_table, kv_len, src, dst, free_pages, free_start, shares, out, stream
PyObject *page_fork(PyObject *const *a)
{
    const c10::Device dev = device_of("k_cache", a[0]);
    const rsa_cache c = layers(a[0], a[1], dev);
    const at::Tensor &table = tables(a[2], dev);
    const int64_t R = table.size(0), stride = table_stride(table);
    const at::Tensor &kv = list("kv_len", a[3], R, dev), &src = list("src", a[4], -1, dev);
    const at::Tensor &dst = list("dst", a[5], src.size(0), dev), &pages = list("free_pages", a[6], -1, dev);
    if (src.size(0) > INT32_MAX)
        value_error("src is too large");
    const int64_t *start = free_start(a[7], dev);
    int32_t *shares = a[8] == Py_None ? nullptr : list("shares", a[8], c.n_pages, dev).data_ptr<int>();
    Call call(dev, a[10]);
    const at::Tensor info = result_list(call, "out", a[9], 4, at::kLong, dev);
    const rsa_stream_t stream = call.stream();
    const rsa_status st = launch([&] {
        return fork_fn(&c, table.data_ptr<int>(), stride, (int)table.size(1), kv.data_ptr<int>(), (int)R, src.data_ptr<int>(),
                       dst.data_ptr<int>(), (int)src.size(0), pages.data_ptr<int>(), pages.size(0), start, shares,
                       info.data_ptr<int64_t>(), stream);
    });
    return results(st, {info});
}

// block_table, kv_len, keep_len, free_pages, free_start, page_size, n_pages, shares, out, stream
PyObject *page_free(PyObject *const *a)
{
    const c10::Device dev = device_of("block_table", a[0]);
    const at::Tensor &table = tables(a[0], dev);
    const int64_t R = table.size(0), stride = table_stride(table);
    const at::Tensor &kv = list("kv_len", a[1], R, dev), &keep = list("keep_len", a[2], R, dev), &pages = list("free_pages", a[3], -1, dev);
    if (a[4] == Py_None)
        type_error("free_start must be a CUDA tensor on " + dev.str());
    const int64_t *start = free_start(a[4], dev);
    const int page_size = small_integer(a[5], "page_size");
    const int64_t n_pages = integer(a[6]);
    int32_t *shares = a[7] == Py_None ? nullptr : list("shares", a[7], n_pages, dev).data_ptr<int>();
    Call call(dev, a[9]);
    const at::Tensor info = result_list(call, "out", a[8], 4, at::kLong, dev);
    const rsa_stream_t stream = call.stream();
    const rsa_status st = launch([&] {
        return free_fn(table.data_ptr<int>(), stride, (int)table.size(1), kv.data_ptr<int>(), keep.data_ptr<int>(), (int)R, page_size,
                       n_pages, pages.data_ptr<int>(), pages.size(0), start, shares, info.data_ptr<int64_t>(), stream);
    });
    return results(st, {info});
}

// A function of N arguments; C++ exceptions become Python's.
template <PyObject *(*F)(PyObject *const *), Py_ssize_t N>
PyObject *entry(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    if (n != N) {
        PyErr_Format(PyExc_TypeError, "%zd arguments wanted, got %zd", N, n);
        return nullptr;
    }
    try {
        return F(args);
    } catch (const Refusal &r) {
        PyErr_SetString(r.type, r.text.c_str());
        return nullptr;
    } catch (const Raised &) {
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

// The addresses of the twelve functions, and share_fn.
PyObject *bind(PyObject *const *a)
{
    void *p[12];
    for (int i = 0; i < 12; ++i)
        p[i] = reinterpret_cast<void *>(integer(a[i]));
    page_plan_fn = reinterpret_cast<decltype(page_plan_fn)>(p[0]);
    rope_fn = reinterpret_cast<decltype(rope_fn)>(p[1]);
    rope_bwd_fn = reinterpret_cast<decltype(rope_bwd_fn)>(p[2]);
    rope_bwd_size_fn = reinterpret_cast<decltype(rope_bwd_size_fn)>(p[3]);
    attn_fn = reinterpret_cast<decltype(attn_fn)>(p[4]);
    attn_size_fn = reinterpret_cast<decltype(attn_size_fn)>(p[5]);
    tree_plan_fn = reinterpret_cast<decltype(tree_plan_fn)>(p[6]);
    tree_attn_fn = reinterpret_cast<decltype(tree_attn_fn)>(p[7]);
    compact_fn = reinterpret_cast<decltype(compact_fn)>(p[8]);
    fork_fn = reinterpret_cast<decltype(fork_fn)>(p[9]);
    free_fn = reinterpret_cast<decltype(free_fn)>(p[10]);
    tree_attn_size_fn = reinterpret_cast<decltype(tree_attn_size_fn)>(p[11]);
    Py_XSETREF(share_fn, Py_NewRef(a[12]));
    Py_RETURN_NONE;
}

#define RSA_ENTRY(f, n) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<f, n>)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {RSA_ENTRY(bind, 13),       RSA_ENTRY(page_plan, 11),    RSA_ENTRY(qk_norm_rope, 16), RSA_ENTRY(qk_norm_rope_bwd, 17),
                         RSA_ENTRY(prefix_attn, 12), RSA_ENTRY(tree_plan, 7),     RSA_ENTRY(tree_attn, 13),    RSA_ENTRY(cache_compact, 9),
                         RSA_ENTRY(page_fork, 11),   RSA_ENTRY(page_free, 10),    {nullptr, nullptr, 0, nullptr}};
#undef RSA_ENTRY

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_paged", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__paged() { return PyModule_Create(&module); }
