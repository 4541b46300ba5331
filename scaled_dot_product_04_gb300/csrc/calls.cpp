// Python entry of the paged-cache operators: checks what a bare pointer cannot
// say (types, shapes, layouts, devices), allocates outputs that were not given
// and calls the C ABI.  A serving step makes a call a layer for each of these
// operators, a few microseconds of GPU work each at small batches, so the
// checks are done here rather than in Python (22-28 us a call there, 3-4 here, launch included).
//
// The C entry points are handed over as addresses (bind), so they are those of
// the library that the package has loaded.
#include <cstdint>
#include <string>

#include <ATen/ops/empty.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/sdpa.h"

namespace {

struct Refused {
    int status;
    std::string message;
};
[[noreturn]] void refuse(std::string message, int status = SDPA_ERR_INVALID_ARG) { throw Refused{status, std::move(message)}; }
struct PythonError {};  // already set

PyObject *g_error_class = nullptr;
decltype(&sdpa_cache_plan) g_plan = nullptr;
decltype(&sdpa_cache_append) g_append = nullptr;
decltype(&sdpa_cache_accept) g_accept = nullptr;
decltype(&sdpa_tree_fwd) g_tree = nullptr;
decltype(&sdpa_tree_fwd_workspace_size) g_tree_ws = nullptr;
decltype(&sdpa_last_error) g_last_error = nullptr;

const at::Tensor *tensor(PyObject *o, const char *name, bool optional = false) {
    if (o == Py_None && optional) return nullptr;
    if (!THPVariable_Check(o)) {
        PyErr_Format(PyExc_TypeError, "%s must be a tensor", name);
        throw PythonError{};
    }
    return &THPVariable_Unpack(o);
}

int integer(PyObject *o, const char *name) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw PythonError{};
    if (v > INT32_MAX || v < INT32_MIN) refuse(std::string(name) + " does not fit 32 bits");
    return (int)v;
}

std::string shape_text(at::IntArrayRef s) {
    std::string out = "(";
    for (size_t i = 0; i < s.size(); ++i) out += (i ? ", " : "") + (s[i] < 0 ? std::string("*") : std::to_string(s[i]));
    return out + ")";
}

// On the GPU, contiguous, of this shape (negative: any length), and within 32-bit sizes.
void check_shape(const at::Tensor &t, const char *name, at::IntArrayRef shape) {
    if (!t.is_cuda()) refuse(std::string(name) + " is not on the GPU");
    bool ok = t.dim() == (int64_t)shape.size() && t.is_contiguous();
    for (size_t i = 0; ok && i < shape.size(); ++i) ok = (shape[i] < 0 || t.size(i) == shape[i]) && t.size(i) <= INT32_MAX;
    if (!ok)
        refuse(std::string(name) + " must be contiguous of shape " + shape_text(shape) + " (got " + shape_text(t.sizes()) + ")");
}
void check_dtype(const at::Tensor &t, const char *name, at::ScalarType want) {
    if (t.scalar_type() != want)
        refuse(std::string(name) + " has dtype " + c10::toString(t.scalar_type()), SDPA_ERR_UNSUPPORTED);
}
void dense(const at::Tensor &t, const char *name, at::ScalarType type, at::IntArrayRef shape) {
    check_dtype(t, name, type);
    check_shape(t, name, shape);
}

int code16(const at::Tensor &t, const char *name) {
    if (t.scalar_type() == at::kBFloat16) return SDPA_BF16;
    if (t.scalar_type() == at::kHalf) return SDPA_FP16;
    refuse(std::string(name) + " has dtype " + c10::toString(t.scalar_type()), SDPA_ERR_UNSUPPORTED);
}

// A cache pair [num_pages, h_kv, page_size, d]; torch.uint8 stands for E4M3 codes.
int caches(const at::Tensor &k, const at::Tensor &v) {
    const auto t = k.scalar_type();
    const int code = t == at::kFloat8_e4m3fn || t == at::kByte ? SDPA_FP8_E4M3 : code16(k, "k_cache");
    check_shape(k, "k_cache", {-1, -1, -1, -1});
    check_dtype(v, "v_cache", t);
    check_shape(v, "v_cache", k.sizes());
    return code;
}

// [tokens, heads, d] whose tokens may be apart; the elements between two tokens.
int64_t token_stride(const at::Tensor &t, const char *name, int64_t heads, int64_t d) {
    if (!t.is_cuda()) refuse(std::string(name) + " is not on the GPU");
    if (t.dim() != 3 || (heads >= 0 && t.size(1) != heads) || t.size(2) != d || t.size(0) > INT32_MAX)
        refuse(std::string(name) + " must be " + shape_text({-1, heads, d}) + " (got " + shape_text(t.sizes()) + ")");
    if (t.numel() == 0) return t.size(1) * d;
    if (t.stride(2) != 1 || (t.stride(1) != d && t.size(1) != 1))
        refuse(std::string("the heads of one token of ") + name + " must be dense");
    return t.size(0) > 1 ? t.stride(0) : t.size(1) * d;
}

struct SameDevice {
    c10::Device device;
    explicit SameDevice(const at::Tensor &first) : device(first.device()) {
        if (device.index() != c10::cuda::current_device())
            refuse("the tensors live on " + device.str() + ", which is not the current device");
    }
    void also(const at::Tensor *t) const {
        if (t && t->device() != device) refuse("the tensors live on different devices");
    }
    template <class... T>
    void all(const T *...t) const {
        (also(t), ...);
    }
};

sdpa_stream_t stream_of(PyObject *o) {
    if (o == Py_None) return c10::cuda::getCurrentCUDAStream().stream();
    PyObject *n = PyLong_Check(o) ? Py_NewRef(o) : PyObject_GetAttrString(o, "cuda_stream");
    if (!n) throw PythonError{};
    void *p = PyLong_AsVoidPtr(n);
    Py_DECREF(n);
    if (!p && PyErr_Occurred()) throw PythonError{};
    return p;
}

void check(int status) {
    if (status != SDPA_OK) refuse(g_last_error(), status);
}
template <class T>
T *data(const at::Tensor *t) {
    return t ? static_cast<T *>(t->data_ptr()) : nullptr;
}
// Memory that a call allocates for the work that it puts on `stream`.  It is that stream's: memory
// freed on the current stream may have writes to come there.  What is returned is also kept until
// the current stream, where the caller goes on, is through with it.
at::Tensor empty(at::IntArrayRef shape, at::ScalarType type, const at::Tensor &like, sdpa_stream_t stream, bool returned = true) {
    auto s = static_cast<cudaStream_t>(stream);
    if (s == cudaStreamLegacy) s = nullptr;
    const auto current = c10::cuda::getCurrentCUDAStream();
    if (s == current.stream()) return at::empty(shape, like.options().dtype(type));
    const c10::cuda::CUDAStreamGuard guard(c10::cuda::getStreamFromExternal(s, like.get_device()));
    at::Tensor t = at::empty(shape, like.options().dtype(type));
    if (returned) c10::cuda::CUDACachingAllocator::recordStream(t.storage().data_ptr(), current);
    return t;
}

// ------------------------------------------------------------------ the calls
// cache_plan(ctx_lens, new_lens, held, ring_state, free_ring, block_table, page_size, max_new,
//            parents, mask_words, out, stream) -> the seven tensors of a plan
PyObject *cache_plan(PyObject *const *a) {
    const at::Tensor &ctx = *tensor(a[0], "ctx_lens"), &fresh = *tensor(a[1], "new_lens"), &held = *tensor(a[2], "held"),
                     &state = *tensor(a[3], "ring_state"), &ring = *tensor(a[4], "free_ring"),
                     &table = *tensor(a[5], "block_table");
    const int page = integer(a[6], "page_size"), max_new = integer(a[7], "max_new"), words = integer(a[9], "mask_words");
    const at::Tensor *parents = tensor(a[8], "parents", true);
    if (max_new < 0 || words < 0) refuse("max_new and mask_words must not be negative");
    dense(ctx, "ctx_lens", at::kInt, {-1});
    const int64_t b = ctx.size(0);
    dense(fresh, "new_lens", at::kInt, {b});
    dense(held, "held", at::kInt, {b});
    dense(state, "ring_state", at::kInt, {3});
    dense(ring, "free_ring", at::kInt, {-1});
    dense(table, "block_table", at::kInt, {b, -1});
    if (parents) dense(*parents, "parents", at::kInt, {max_new});
    const SameDevice same(ctx);
    same.all(&fresh, &held, &state, &ring, &table, parents);
    const sdpa_stream_t stream = stream_of(a[11]);
    at::Tensor out[7];  // cu_new, kv_lens, slot_map, positions, tree_mask, held, ring_state
    const at::DimVector shapes[7] = {{b + 1}, {b}, {max_new}, {max_new}, {max_new, words}, {b}, {3}};
    static const char *names[7] = {"out.cu_new",    "out.kv_lens", "out.slot_map",  "out.positions",
                                   "out.tree_mask", "out.held",    "out.ring_state"};
    if (a[10] != Py_None) {
        if (!PyTuple_Check(a[10]) || PyTuple_GET_SIZE(a[10]) != 7) refuse("out must be a CachePlan");
        for (int i = 0; i < 7; ++i) {
            PyObject *o = PyTuple_GET_ITEM(a[10], i);
            if (i == 4 && (o != Py_None) != (words > 0)) refuse("out.tree_mask does not go with mask_words");
            if (i == 4 && words == 0) continue;
            out[i] = *tensor(o, names[i]);
            dense(out[i], names[i], at::kInt, shapes[i]);
            same.also(&out[i]);
        }
    } else {
        for (int i = 0; i < 7; ++i)
            if (i != 4 || words > 0) out[i] = empty(shapes[i], at::kInt, ctx, stream);
    }
    using I = int32_t;
    check(g_plan(data<I>(&ctx), data<I>(&fresh), data<I>(parents), data<I>(&held), data<I>(&state), data<I>(&ring),
                 data<I>(&table), data<I>(&out[5]), data<I>(&out[6]), data<I>(&out[0]), data<I>(&out[1]), data<I>(&out[2]),
                 data<I>(&out[3]), words > 0 ? data<uint32_t>(&out[4]) : nullptr, (int)b, (int)table.size(1), page,
                 (int)ring.size(0), max_new, words, stream));
    if (a[10] != Py_None) return Py_NewRef(a[10]);
    PyObject *r = PyTuple_New(7);
    for (int i = 0; r && i < 7; ++i) PyTuple_SET_ITEM(r, i, i == 4 && words == 0 ? Py_NewRef(Py_None) : THPVariable_Wrap(out[i]));
    return r;
}

// cache_append(k, v, k_cache, v_cache, slot_map, scale_k, scale_v, stream)
PyObject *cache_append(PyObject *const *a) {
    const at::Tensor &k = *tensor(a[0], "k"), &v = *tensor(a[1], "v"), &kc = *tensor(a[2], "k_cache"),
                     &vc = *tensor(a[3], "v_cache"), &slots = *tensor(a[4], "slot_map");
    const at::Tensor *sk = tensor(a[5], "scale_k", true), *sv = tensor(a[6], "scale_v", true);
    const int cache = caches(kc, vc), type = code16(k, "k");
    check_dtype(v, "v", k.scalar_type());
    const int64_t h = kc.size(1), d = kc.size(3);
    const int64_t ks = token_stride(k, "k", h, d), vs = token_stride(v, "v", h, d);
    if (v.size(0) != k.size(0)) refuse("k and v have different numbers of tokens");
    dense(slots, "slot_map", at::kInt, {k.size(0)});
    if (sk) dense(*sk, "scale_k", at::kFloat, {1});
    if (sv) dense(*sv, "scale_v", at::kFloat, {1});
    const SameDevice same(k);
    same.all(&v, &kc, &vc, &slots, sk, sv);
    check(g_append(k.data_ptr(), v.data_ptr(), kc.data_ptr(), vc.data_ptr(), data<int32_t>(&slots), data<float>(sk),
                   data<float>(sv), (int)k.size(0), ks, vs, (int)h, (int)d, (int)kc.size(0), (int)kc.size(2), type, cache,
                   stream_of(a[7])));
    Py_RETURN_NONE;
}

// cache_accept(k_cache, v_cache, block_table, ctx_lens, new_lens, path, path_lens, out, stream) -> out
PyObject *cache_accept(PyObject *const *a) {
    const at::Tensor &kc = *tensor(a[0], "k_cache"), &vc = *tensor(a[1], "v_cache"), &table = *tensor(a[2], "block_table"),
                     &ctx = *tensor(a[3], "ctx_lens"), &fresh = *tensor(a[4], "new_lens"), &path = *tensor(a[5], "path"),
                     &lens = *tensor(a[6], "path_lens");
    const at::Tensor *given = tensor(a[7], "out", true);
    const int cache = caches(kc, vc);
    dense(ctx, "ctx_lens", at::kInt, {-1});
    const int64_t b = ctx.size(0);
    dense(fresh, "new_lens", at::kInt, {b});
    dense(lens, "path_lens", at::kInt, {b});
    dense(table, "block_table", at::kInt, {b, -1});
    dense(path, "path", at::kInt, {b, -1});
    if (given) dense(*given, "out", at::kInt, {b});
    const SameDevice same(kc);
    same.all(&vc, &table, &ctx, &fresh, &path, &lens, given);
    const sdpa_stream_t stream = stream_of(a[8]);
    const at::Tensor out = given ? *given : empty({b}, at::kInt, ctx, stream);
    using I = int32_t;
    check(g_accept(kc.data_ptr(), vc.data_ptr(), data<I>(&table), data<I>(&ctx), data<I>(&fresh), data<I>(&path),
                   data<I>(&lens), data<I>(&out), (int)b, (int)table.size(1), (int)path.size(1), (int)kc.size(1),
                   (int)kc.size(3), (int)kc.size(0), (int)kc.size(2), cache, stream));
    return given ? Py_NewRef(a[7]) : THPVariable_Wrap(out);
}

at::Tensor tree_workspace(const at::Tensor &q, const at::Tensor &kc, int b, int max_q, int max_kv, sdpa_stream_t stream) {
    const size_t size = g_tree_ws(b, max_q, max_kv, (int)q.size(1), (int)kc.size(1), (int)kc.size(3));
    if (size == (size_t)-1) refuse("sizes that attention_tree does not take");
    return empty({size > 0 ? (int64_t)size : 1}, at::kByte, q, stream, false);
}

// attention_tree_workspace(q, k_cache, num_seqs, max_seqlen_q, max_seqlen_kv)
PyObject *attention_tree_workspace(PyObject *const *a) {
    const at::Tensor &q = *tensor(a[0], "q"), &kc = *tensor(a[1], "k_cache");
    check_shape(kc, "k_cache", {-1, -1, -1, -1});
    token_stride(q, "q", -1, kc.size(3));
    return THPVariable_Wrap(tree_workspace(q, kc, integer(a[2], "num_seqs"), integer(a[3], "max_seqlen_q"),
                                           integer(a[4], "max_seqlen_kv"), stream_of(Py_None)));
}

// attention_tree(q, k_cache, v_cache, block_table, cu_seqlens_q, kv_lens, max_seqlen_q, max_seqlen_kv,
//                tree_mask, scale, descale_k, descale_v, out, workspace, stream) -> (o, lse)
PyObject *attention_tree(PyObject *const *a) {
    const at::Tensor &q = *tensor(a[0], "q"), &kc = *tensor(a[1], "k_cache"), &vc = *tensor(a[2], "v_cache"),
                     &table = *tensor(a[3], "block_table"), &cu = *tensor(a[4], "cu_seqlens_q"),
                     &lens = *tensor(a[5], "kv_lens");
    const int max_q = integer(a[6], "max_seqlen_q"), max_kv = integer(a[7], "max_seqlen_kv");
    const at::Tensor *mask = tensor(a[8], "tree_mask", true);
    const double scale = PyFloat_AsDouble(a[9]);
    if (scale == -1.0 && PyErr_Occurred()) throw PythonError{};
    const at::Tensor *dk = tensor(a[10], "descale_k", true), *dv = tensor(a[11], "descale_v", true);
    const int cache = caches(kc, vc), type = code16(q, "q");
    const int64_t d = kc.size(3), stride = token_stride(q, "q", -1, d), total = q.size(0), h = q.size(1);
    dense(lens, "kv_lens", at::kInt, {-1});
    const int64_t b = lens.size(0);
    dense(cu, "cu_seqlens_q", at::kInt, {b + 1});
    dense(table, "block_table", at::kInt, {b, -1});
    if (mask) dense(*mask, "tree_mask", at::kInt, {total, -1});
    if (dk) dense(*dk, "descale_k", at::kFloat, {1});
    if (dv) dense(*dv, "descale_v", at::kFloat, {1});
    const SameDevice same(q);
    same.all(&kc, &vc, &table, &cu, &lens, mask, dk, dv);
    const sdpa_stream_t stream = stream_of(a[14]);
    at::Tensor o, lse;
    const bool given = a[12] != Py_None;
    if (given) {
        if (!PyTuple_Check(a[12]) || PyTuple_GET_SIZE(a[12]) != 2) refuse("out must be a pair (o, lse)");
        o = *tensor(PyTuple_GET_ITEM(a[12], 0), "o");
        dense(o, "o", q.scalar_type(), {total, h, d});
        same.also(&o);
        if (const at::Tensor *l = tensor(PyTuple_GET_ITEM(a[12], 1), "lse", true)) {
            dense(*l, "lse", at::kFloat, {total, h});
            same.also(l);
            lse = *l;
        }
    } else {
        o = empty({total, h, d}, q.scalar_type(), q, stream);
        lse = empty({total, h}, at::kFloat, q, stream);
    }
    at::Tensor ws;
    if (a[13] == Py_None) {
        ws = tree_workspace(q, kc, (int)b, max_q, max_kv, stream);
    } else {
        ws = *tensor(a[13], "workspace");
        dense(ws, "workspace", at::kByte, {-1});
        same.also(&ws);
    }
    check(g_tree(q.data_ptr(), kc.data_ptr(), vc.data_ptr(), o.data_ptr(), lse.defined() ? data<float>(&lse) : nullptr,
                 data<int32_t>(&table), data<int32_t>(&cu), data<int32_t>(&lens), data<uint32_t>(mask), data<float>(dk),
                 data<float>(dv), (int)b, (int)total, max_q, max_kv, (int)table.size(1), mask ? (int)mask->size(1) : 0,
                 stride, (int)h, (int)kc.size(1), (int)d, (int)kc.size(0), (int)kc.size(2), (float)scale, type, cache,
                 ws.data_ptr(), (size_t)ws.numel(), stream));
    if (given) return Py_NewRef(a[12]);
    PyObject *r = PyTuple_New(2);
    if (!r) return nullptr;
    PyTuple_SET_ITEM(r, 0, THPVariable_Wrap(o));
    PyTuple_SET_ITEM(r, 1, THPVariable_Wrap(lse));
    return r;
}

// No C++ exception leaves a call: refusals become SdpaError(status, message).
template <PyObject *(*kCall)(PyObject *const *), int kArgs>
PyObject *entry(PyObject *, PyObject *const *args, Py_ssize_t n) {
    try {
        if (n != kArgs || !g_last_error) {
            PyErr_Format(PyExc_TypeError, "expected %d arguments (got %zd) after bind()", kArgs, n);
            return nullptr;
        }
        return kCall(args);
    } catch (const Refused &r) {
        if (PyObject *e = PyObject_CallFunction(g_error_class, "is", r.status, r.message.c_str())) {
            PyErr_SetObject(g_error_class, e);
            Py_DECREF(e);
        }
    } catch (const PythonError &) {
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

// bind(error class, addresses of the six C entry points)
PyObject *bind(PyObject *, PyObject *const *a, Py_ssize_t n) {
    if (n != 7) {
        PyErr_SetString(PyExc_TypeError, "bind takes the error class and six addresses");
        return nullptr;
    }
    void *p[6];
    for (int i = 0; i < 6; ++i) {
        p[i] = PyLong_AsVoidPtr(a[i + 1]);
        if (!p[i]) {
            if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "a NULL entry point");
            return nullptr;
        }
    }
    Py_XSETREF(g_error_class, Py_NewRef(a[0]));
    g_plan = reinterpret_cast<decltype(g_plan)>(p[0]);
    g_append = reinterpret_cast<decltype(g_append)>(p[1]);
    g_accept = reinterpret_cast<decltype(g_accept)>(p[2]);
    g_tree = reinterpret_cast<decltype(g_tree)>(p[3]);
    g_tree_ws = reinterpret_cast<decltype(g_tree_ws)>(p[4]);
    g_last_error = reinterpret_cast<decltype(g_last_error)>(p[5]);
    Py_RETURN_NONE;
}

using Fast = PyObject *(*)(PyObject *, PyObject *const *, Py_ssize_t);
PyCFunction fast(Fast f) { return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)); }

PyMethodDef g_methods[] = {
    {"bind", fast(bind), METH_FASTCALL, nullptr},
    {"cache_plan", fast(entry<cache_plan, 12>), METH_FASTCALL, nullptr},
    {"cache_append", fast(entry<cache_append, 8>), METH_FASTCALL, nullptr},
    {"cache_accept", fast(entry<cache_accept, 9>), METH_FASTCALL, nullptr},
    {"attention_tree_workspace", fast(entry<attention_tree_workspace, 5>), METH_FASTCALL, nullptr},
    {"attention_tree", fast(entry<attention_tree, 15>), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_sdpa_calls", nullptr, -1, g_methods};

}  // namespace

PyMODINIT_FUNC PyInit__sdpa_calls() { return PyModule_Create(&g_module); }
