// Python binding of the generation operators (serve.py): the checks of a
// call's tensors, its outputs and its workspace, and the call into libdf11.
//
// The smallest calls take a few microseconds on the GPU, so what stands in
// front of them is native: the same checks and allocations in Python took 17
// of a call's 17 us against 10 here (two launches are 6 of either).
//
// libdf11's functions come as addresses from the library that the package
// has loaded (bind), so there is no second copy of it.  Every exception ends
// at the entry points: it becomes a Python one.
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ATen.h>
#include <ATen/core/LegacyTypeDispatch.h>
#include <ATen/core/grad_mode.h>
#include <torch/csrc/Exceptions.h>

#include <cmath>
#include <string>

#include "../../include/df11.h"

namespace {

struct Functions {
    decltype(&df11_prefix_attention_workspace_bytes) prefix_bytes;
    decltype(&df11_prefix_attention) prefix;
    decltype(&df11_cache_attention_workspace_bytes) attend_bytes;
    decltype(&df11_cache_attention) attend;
    decltype(&df11_cache_insert) insert;
    decltype(&df11_cache_compact) compact;
    decltype(&df11_verify_drafts_workspace_bytes) verify_bytes;
    decltype(&df11_verify_drafts) verify;
} lib;
PyObject *raise_status;   // raises what a status means

struct Refused {
    PyObject *type;
    std::string text;
};

[[noreturn]] void wrong_type(const std::string &text) { throw Refused{PyExc_TypeError, text}; }
[[noreturn]] void wrong_value(const std::string &text) { throw Refused{PyExc_ValueError, text}; }

struct Status {};   // a Python error is set

void check(int status, const char *who)
{
    if (status == DF11_OK) return;
    PyObject *r = PyObject_CallFunction(raise_status, "is", status, who);
    Py_XDECREF(r);
    throw Status{};
}

const at::Tensor &tensor(PyObject *o, const char *name)
{
    if (!THPVariable_Check(o)) wrong_type(std::string(name) + " must be a tensor");
    return THPVariable_Unpack(o);
}

std::string text(at::IntArrayRef v)
{
    std::string s = "(";
    for (size_t i = 0; i < v.size(); i++) s += (i ? ", " : "") + std::to_string(v[i]);
    return s + ")";
}

void same(const char *name, const at::Tensor &t, at::ScalarType type, at::Device device, at::IntArrayRef shape)
{
    if (t.scalar_type() != type)
        wrong_type(std::string(name) + " must be " + c10::toString(type) + ", got " + c10::toString(t.scalar_type()));
    if (t.device() != device)
        wrong_value(std::string(name) + " is on " + t.device().str() + ", the other operands on " + device.str());
    if (t.requires_grad() && at::GradMode::is_enabled())
        wrong_value(std::string(name) + " requires a gradient, which these operators do not give: call them under torch.no_grad()");
    if (t.sizes() != shape)
        wrong_value(std::string(name) + " has shape " + text(t.sizes()) + ", not " + text(shape));
}

// A contiguous tensor of this type, device and shape.
void *flat(const char *name, const at::Tensor &t, at::ScalarType type, at::Device device, at::IntArrayRef shape)
{
    same(name, t, type, device, shape);
    if (!t.is_contiguous()) wrong_value(std::string(name) + " must be contiguous");
    return t.data_ptr();
}

// A tensor of rows: its last axis is contiguous.  The stride of an axis of
// one is never used and counts as 0.
struct Strides {
    int64_t s[4] = {0, 0, 0, 0};
    bool operator!=(const Strides &o) const
    {
        return s[0] != o.s[0] || s[1] != o.s[1] || s[2] != o.s[2] || s[3] != o.s[3];
    }
};

Strides rows(const char *name, const at::Tensor &t, at::ScalarType type, at::Device device, at::IntArrayRef shape)
{
    same(name, t, type, device, shape);
    Strides r;
    const int n = (int)shape.size();
    for (int i = 0; i < n; i++) r.s[i] = shape[i] == 1 ? 0 : t.stride(i);
    if (shape[n - 1] > 1 && r.s[n - 1] != 1) wrong_value("the last axis of " + std::string(name) + " must be contiguous");
    return r;
}

Strides pair(const char *a_name, const at::Tensor &a, const char *b_name, const at::Tensor &b, at::ScalarType type,
             at::Device device, at::IntArrayRef shape)
{
    const Strides s = rows(a_name, a, type, device, shape);
    if (rows(b_name, b, type, device, shape) != s)
        wrong_value(std::string(a_name) + " and " + b_name + " must have the same strides");
    return s;
}

int64_t dtype_of(const char *name, const at::Tensor &t, bool floats)
{
    if (!t.is_cuda()) wrong_value(std::string(name) + " must be on the GPU");
    switch (t.scalar_type()) {
    case at::kBFloat16: return DF11_BF16;
    case at::kHalf: return DF11_FP16;
    case at::kFloat:
        if (floats) return DF11_FP32;
        break;
    default: break;
    }
    wrong_type(std::string(name) + " must be bfloat16" + (floats ? ", float16 or float32" : " or float16") + ", got " +
               c10::toString(t.scalar_type()));
}

void dims(const char *name, const at::Tensor &t, int64_t n)
{
    if (t.dim() != n) wrong_value(std::string(name) + " must have " + std::to_string(n) + " axes");
}

at::Tensor make(at::IntArrayRef shape, const at::Tensor &like, at::ScalarType type)
{
    return at::empty(shape, like.options().dtype(type));
}

// A tensor that a call has written in place: its version counts that, so that
// what autograd saved of it is known to have changed.
void written(const at::Tensor &t)
{
    if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

struct Workspace {
    at::Tensor t;
    uint64_t bytes;
    Workspace(uint64_t n, const at::Tensor &like) : bytes(n)
    {
        if (n) t = make({(int64_t)n}, like, at::kByte);
    }
    void *data() { return bytes ? t.data_ptr() : nullptr; }
};

double number(PyObject *o)
{
    const double x = PyFloat_AsDouble(o);
    if (x == -1.0 && PyErr_Occurred()) throw Status{};
    return x;
}

int64_t whole(PyObject *o)
{
    const long long x = PyLong_AsLongLong(o);
    if (x == -1 && PyErr_Occurred()) throw Status{};
    return x;
}

bool truth(PyObject *o)
{
    const int x = PyObject_IsTrue(o);
    if (x < 0) throw Status{};
    return x;
}

double scale_of(PyObject *o, int64_t dim) { return o == Py_None ? 1.0 / std::sqrt((double)(dim ? dim : 1)) : number(o); }

PyObject *both(const at::Tensor &a, const at::Tensor &b)
{
    PyObject *x = THPVariable_Wrap(a), *y = THPVariable_Wrap(b);
    PyObject *r = x && y ? PyTuple_Pack(2, x, y) : nullptr;
    Py_XDECREF(x);
    Py_XDECREF(y);
    return r;
}

typedef PyObject *const *Arguments;

// q, prefix_k, prefix_v, k, v, lengths, block_table, scale, out, return_lse, stream
PyObject *prefix_attention(Arguments x)
{
    const at::Tensor &q = tensor(x[0], "q"), &pk = tensor(x[1], "prefix_k"), &pv = tensor(x[2], "prefix_v");
    const at::Tensor &k = tensor(x[3], "k"), &v = tensor(x[4], "v"), &lengths = tensor(x[5], "lengths");
    df11_prefix_attention_args a{};
    a.dtype = dtype_of("q", q, false);
    const auto type = q.scalar_type();
    const auto device = q.device();
    dims("q", q, 4), dims("prefix_k", pk, 3), dims("k", k, 4);
    a.batch = q.size(0), a.tokens = q.size(1), a.heads = q.size(2), a.dim = q.size(3);
    a.prefix = pk.size(0), a.kv_heads = pk.size(1);
    const Strides sq = rows("q", q, type, device, q.sizes());
    const Strides sp = pair("prefix_k", pk, "prefix_v", pv, type, device, {a.prefix, a.kv_heads, a.dim});
    Strides sk;
    if (x[6] == Py_None) {
        a.suffix = k.size(1);
        sk = pair("k", k, "v", v, type, device, {a.batch, a.suffix, a.kv_heads, a.dim});
    } else {
        const at::Tensor &table = tensor(x[6], "block_table");
        dims("block_table", table, 2);
        a.n_pages = k.size(0), a.page = k.size(1);
        sk = pair("k", k, "v", v, type, device, {a.n_pages, a.page, a.kv_heads, a.dim});
        a.block_table = (const int32_t *)flat("block_table", table, at::kInt, device, {a.batch, table.size(1)});
        a.table_batch = table.size(1);
        a.suffix = a.table_batch * a.page;
    }
    a.lengths = (const int32_t *)flat("lengths", lengths, at::kInt, device, {a.batch});
    at::Tensor out;
    if (x[8] == Py_None) out = make(q.sizes(), q, type);
    else out = tensor(x[8], "out");
    a.out = flat("out", out, type, device, q.sizes());
    const bool return_lse = truth(x[9]);
    at::Tensor lse;
    if (return_lse) {
        lse = make({a.batch, a.tokens, a.heads}, q, at::kFloat);
        a.lse = (float *)lse.data_ptr();
    }
    a.q = q.data_ptr(), a.prefix_k = pk.data_ptr(), a.prefix_v = pv.data_ptr(), a.k = k.data_ptr(), a.v = v.data_ptr();
    a.q_batch = sq.s[0], a.q_token = sq.s[1], a.q_head = sq.s[2], a.prefix_token = sp.s[0], a.prefix_head = sp.s[1];
    a.k_batch = sk.s[0], a.k_token = sk.s[1], a.k_head = sk.s[2];
    a.scale = scale_of(x[7], a.dim);
    Workspace ws(lib.prefix_bytes(&a), q);
    check(lib.prefix(&a, ws.data(), ws.bytes, (void *)whole(x[10])), "df11_prefix_attention");
    if (x[8] != Py_None) written(out);
    return return_lse ? both(out, lse) : THPVariable_Wrap(out);
}

df11_cache make_cache(const at::Tensor &k, const at::Tensor &v, const at::Tensor &weights, const at::Tensor &positions,
                      const at::Tensor &lengths)
{
    df11_cache c{};
    c.dtype = dtype_of("k", k, false);
    dims("k", k, 4);
    c.batch = k.size(0), c.kv_heads = k.size(1), c.slots = k.size(2), c.dim = k.size(3);
    const auto device = k.device();
    const Strides s = pair("k", k, "v", v, k.scalar_type(), device, k.sizes());
    c.k = k.data_ptr(), c.v = v.data_ptr();
    c.weights = (float *)flat("weights", weights, at::kFloat, device, k.sizes().slice(0, 3));
    c.positions = (int32_t *)flat("positions", positions, at::kInt, device, k.sizes().slice(0, 3));
    c.lengths = (const int32_t *)flat("lengths", lengths, at::kInt, device, {c.batch});
    c.stride_batch = s.s[0], c.stride_head = s.s[1], c.stride_slot = s.s[2];
    return c;
}

// The cache of a tuple (k, v, weights, positions, lengths), which serve.py's
// BoundedCache keeps: the tensors are looked at in every call, since their
// memory may have moved since the last one.
df11_cache cache_of(PyObject *o)
{
    if (!PyTuple_Check(o) || PyTuple_GET_SIZE(o) != 5) wrong_type("not a BoundedCache");
    const auto at = [&](int i, const char *name) -> const at::Tensor & { return tensor(PyTuple_GET_ITEM(o, i), name); };
    return make_cache(at(0, "k"), at(1, "v"), at(2, "weights"), at(3, "positions"), at(4, "lengths"));
}

// `n` tensors of such a tuple, from `first` on, were written.
void written(PyObject *cache, int first, int n)
{
    for (int i = first; i < first + n; i++) written(THPVariable_Unpack(PyTuple_GET_ITEM(cache, i)));
}

// k, v, weights, positions, lengths: the tuple of them, looked over
PyObject *cache(Arguments x)
{
    PyObject *r = PyTuple_Pack(5, x[0], x[1], x[2], x[3], x[4]);
    if (!r) return nullptr;
    try {
        cache_of(r);
    } catch (...) {
        Py_DECREF(r);
        throw;
    }
    return r;
}

// cache, its k, q, pos, scale, out, stream
PyObject *cache_attention(Arguments x)
{
    const df11_cache c = cache_of(x[0]);
    const at::Tensor &k = tensor(x[1], "k"), &q = tensor(x[2], "q"), &pos = tensor(x[3], "pos");
    const auto type = k.scalar_type();
    const auto device = k.device();
    dims("q", q, 4);
    df11_cache_attention_args a{};
    a.tokens = q.size(1), a.heads = q.size(2);
    const Strides s = rows("q", q, type, device, {c.batch, a.tokens, a.heads, c.dim});
    at::Tensor out;
    if (x[5] == Py_None) out = make(q.sizes(), q, type);
    else out = tensor(x[5], "out");
    a.out = flat("out", out, type, device, q.sizes());
    a.q = q.data_ptr();
    a.pos = (const int32_t *)flat("pos", pos, at::kInt, device, {c.batch});
    a.q_batch = s.s[0], a.q_token = s.s[1], a.q_head = s.s[2];
    a.scale = scale_of(x[4], c.dim);
    Workspace ws(lib.attend_bytes(&c, &a), q);
    check(lib.attend(&c, &a, ws.data(), ws.bytes, (void *)whole(x[6])), "df11_cache_attention");
    if (x[5] != Py_None) written(out);
    written(x[0], 2, 1);   // weights
    return THPVariable_Wrap(out);
}

// cache, its k, k_new, v_new, pos, recent, stream
PyObject *cache_insert(Arguments x)
{
    const df11_cache c = cache_of(x[0]);
    const at::Tensor &k = tensor(x[1], "k"), &k_new = tensor(x[2], "k_new"), &v_new = tensor(x[3], "v_new");
    const at::Tensor &pos = tensor(x[4], "pos");
    const auto device = k.device();
    const Strides s = pair("k_new", k_new, "v_new", v_new, k.scalar_type(), device, {c.batch, c.kv_heads, c.dim});
    const int32_t *p = (const int32_t *)flat("pos", pos, at::kInt, device, {c.batch});
    const at::Tensor slots = make({c.batch, c.kv_heads}, pos, at::kInt), lengths = make({c.batch}, pos, at::kInt);
    check(lib.insert(&c, k_new.data_ptr(), v_new.data_ptr(), s.s[0], s.s[1], p, whole(x[5]), (int32_t *)slots.data_ptr(),
                     (int32_t *)lengths.data_ptr(), (void *)whole(x[6])),
          "df11_cache_insert");
    written(x[0], 0, 4);   // k, v, weights, positions
    return both(slots, lengths);
}

// cache, its k, pos, budget, recent, slots, stream: the new cache's k, v,
// weights, positions and lengths, and kept
PyObject *cache_compact(Arguments x)
{
    const df11_cache c = cache_of(x[0]);
    const at::Tensor &k = tensor(x[1], "k"), &pos = tensor(x[2], "pos");
    const int64_t budget = whole(x[3]), recent = whole(x[4]), slots = whole(x[5]);
    if (slots < 1) wrong_value("the new cache needs a slot");
    const int32_t *p = (const int32_t *)flat("pos", pos, at::kInt, k.device(), {c.batch});
    const at::Tensor k2 = make({c.batch, c.kv_heads, slots, c.dim}, k, k.scalar_type());
    const at::Tensor v2 = make(k2.sizes(), k, k.scalar_type());
    const at::Tensor weights = make({c.batch, c.kv_heads, slots}, pos, at::kFloat);
    const at::Tensor positions = make(weights.sizes(), pos, at::kInt), kept = make(weights.sizes(), pos, at::kInt);
    const at::Tensor lengths = make({c.batch}, pos, at::kInt);
    const df11_cache out = make_cache(k2, v2, weights, positions, lengths);
    check(lib.compact(&c, p, budget, recent, &out, (int32_t *)kept.data_ptr(), (int32_t *)lengths.data_ptr(),
                      (void *)whole(x[6])),
          "df11_cache_compact");
    PyObject *r = PyTuple_New(6);
    if (!r) return nullptr;
    const at::Tensor *parts[6] = {&k2, &v2, &weights, &positions, &lengths, &kept};
    for (int i = 0; i < 6; i++) PyTuple_SET_ITEM(r, i, THPVariable_Wrap(*parts[i]));
    return r;
}

// draft_tokens, target_probs, uniforms, draft_probs, counts, stream
PyObject *verify_drafts(Arguments x)
{
    const at::Tensor &drafts = tensor(x[0], "draft_tokens"), &target = tensor(x[1], "target_probs");
    const at::Tensor &uniforms = tensor(x[2], "uniforms");
    df11_verify_args a{};
    a.dtype = dtype_of("target_probs", target, true);
    dims("draft_tokens", drafts, 2), dims("target_probs", target, 3);
    const auto kind = drafts.scalar_type(), type = target.scalar_type();
    const auto device = target.device();
    if (kind != at::kInt && kind != at::kLong)
        wrong_type(std::string("draft_tokens must be int32 or int64, got ") + c10::toString(kind));
    a.batch = drafts.size(0), a.drafts = drafts.size(1), a.vocab = target.size(2), a.token_bytes = kind == at::kInt ? 4 : 8;
    a.draft_tokens = flat("draft_tokens", drafts, kind, device, drafts.sizes());
    const Strides sp = rows("target_probs", target, type, device, {a.batch, a.drafts + 1, a.vocab});
    a.target_probs = target.data_ptr(), a.target_batch = sp.s[0], a.target_row = sp.s[1];
    if (x[3] != Py_None) {
        const at::Tensor &draft = tensor(x[3], "draft_probs");
        const Strides sq = rows("draft_probs", draft, type, device, {a.batch, a.drafts, a.vocab});
        a.draft_probs = draft.data_ptr(), a.draft_batch = sq.s[0], a.draft_row = sq.s[1];
    }
    a.uniforms = (const float *)flat("uniforms", uniforms, at::kFloat, device, {a.batch, a.drafts + 1});
    if (x[4] != Py_None) a.counts = (const int32_t *)flat("counts", tensor(x[4], "counts"), at::kInt, device, {a.batch});
    const at::Tensor tokens = make({a.batch, a.drafts + 1}, drafts, kind), accepted = make({a.batch}, drafts, at::kInt);
    a.tokens = tokens.data_ptr(), a.accepted = (int32_t *)accepted.data_ptr();
    Workspace ws(lib.verify_bytes(&a), drafts);
    check(lib.verify(&a, ws.data(), ws.bytes, (void *)whole(x[5])), "df11_verify_drafts");
    return both(tokens, accepted);
}

// raise_status, then the addresses of libdf11's functions
PyObject *bind(Arguments x)
{
    Py_INCREF(x[0]);
    Py_XDECREF(raise_status);
    raise_status = x[0];
    void *p[8];
    for (int i = 0; i < 8; i++) p[i] = PyLong_AsVoidPtr(x[1 + i]);
    if (PyErr_Occurred()) throw Status{};
    lib.prefix_bytes = (decltype(lib.prefix_bytes))p[0], lib.prefix = (decltype(lib.prefix))p[1];
    lib.attend_bytes = (decltype(lib.attend_bytes))p[2], lib.attend = (decltype(lib.attend))p[3];
    lib.insert = (decltype(lib.insert))p[4], lib.compact = (decltype(lib.compact))p[5];
    lib.verify_bytes = (decltype(lib.verify_bytes))p[6], lib.verify = (decltype(lib.verify))p[7];
    Py_RETURN_NONE;
}

template <PyObject *(*F)(Arguments), int N>
PyObject *entry(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    if (n != N) {
        PyErr_Format(PyExc_TypeError, "%d arguments, not %zd", N, n);
        return nullptr;
    }
    try {
        at::AutoDispatchBelowADInplaceOrView no_grad;   // nothing here is recorded for a gradient
        return F(args);
    } catch (const Refused &e) {
        PyErr_SetString(e.type, e.text.c_str());
    } catch (const Status &) {
    } catch (python_error &e) {
        e.restore();
    } catch (const c10::OutOfMemoryError &e) {
        PyObject *torch = PyImport_ImportModule("torch");
        PyObject *type = torch ? PyObject_GetAttrString(torch, "OutOfMemoryError") : nullptr;
        PyErr_Clear();
        PyErr_SetString(type ? type : PyExc_MemoryError, e.what_without_backtrace());
        Py_XDECREF(type);
        Py_XDECREF(torch);
    } catch (const c10::Error &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what_without_backtrace());
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

#define DF11_ENTRY(name, count) \
    {#name, (PyCFunction)(void (*)(void))entry<name, count>, METH_FASTCALL, nullptr}

PyMethodDef methods[] = {DF11_ENTRY(bind, 9),
                         DF11_ENTRY(prefix_attention, 11),
                         DF11_ENTRY(cache, 5),
                         DF11_ENTRY(cache_attention, 7),
                         DF11_ENTRY(cache_insert, 7),
                         DF11_ENTRY(cache_compact, 7),
                         DF11_ENTRY(verify_drafts, 6),
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_df11_serve", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__df11_serve(void) { return PyModule_Create(&module); }
