// Argument marshalling of the paged cache's operators (include/attn.h) for the Python binding:
// tensors are checked against the cache and handed to libgdn's C ABI.  The calls of a decode step
// take a few microseconds on the GPU, less than checking their operands one by one in Python
// took; here that is a fraction of one.  Nothing is computed here.
//
// Each function returns the call's results, or the gdn_status as an int when libgdn refused it.
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/csrc/utils/object_ptr.h>

#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <string>

#include "attn.h"

namespace {

struct Cache {
    gdn_paged_kv c;
    at::Tensor k, v, table;                // keeps the memory
    at::ScalarType dtype;
    c10::Device device;
    int64_t seqs;
};

[[noreturn]] __attribute__((format(printf, 2, 3))) void refuse(PyObject *type, const char *format, ...) {
    char message[512];
    va_list args;
    va_start(args, format);
    std::vsnprintf(message, sizeof message, format, args);
    va_end(args);
    PyErr_SetString(type, message);
    throw python_error();
}

std::string text(at::ScalarType t) {
    switch (t) {
    case at::kFloat: return "torch.float32";
    case at::kDouble: return "torch.float64";
    case at::kBFloat16: return "torch.bfloat16";
    case at::kHalf: return "torch.float16";
    case at::kInt: return "torch.int32";
    case at::kLong: return "torch.int64";
    case at::kByte: return "torch.uint8";
    default: return c10::toString(t);
    }
}
std::string text(at::IntArrayRef s) {
    std::string r = "(";
    for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
    return r + (s.size() == 1 ? ",)" : ")");
}

const at::Tensor &tensor(PyObject *o, const char *name) {
    if (!THPVariable_Check(o)) refuse(PyExc_TypeError, "%s must be a tensor", name);
    return THPVariable_Unpack(o);
}
const at::Tensor *maybe(PyObject *o, const char *name) {
    return o == Py_None ? nullptr : &tensor(o, name);
}

const Cache &cache(PyObject *o) {
    auto *c = static_cast<const Cache *>(PyCapsule_GetPointer(o, "gdn.cache"));
    if (!c) throw python_error();
    return *c;
}

void on_device(const at::Tensor &t, const char *name, const Cache &kv) {
    if (t.device() != kv.device)
        refuse(PyExc_ValueError, "%s is on %s, the cache on %s", name, t.device().str().c_str(), kv.device.str().c_str());
}

// Address of an operand (null stays null) after checking type, shape, layout and device.
void *address(const at::Tensor *t, const char *name, at::ScalarType dtype, at::IntArrayRef shape, const Cache &kv) {
    if (!t) return nullptr;
    if (t->scalar_type() != dtype)
        refuse(PyExc_TypeError, "%s must be %s, got %s", name, text(dtype).c_str(), text(t->scalar_type()).c_str());
    if (t->sizes() != shape)
        refuse(PyExc_ValueError, "%s has shape %s, expected %s", name, text(t->sizes()).c_str(), text(shape).c_str());
    if (!t->is_contiguous()) refuse(PyExc_ValueError, "%s must be contiguous", name);
    on_device(*t, name, kv);
    return t->data_ptr();
}

// Address and token stride of [T_total, heads, d] (or [B, T, heads, d]) whose heads and dims are
// contiguous; tokens may lie further apart.  heads < 0: any number.
const void *token_rows(const at::Tensor &t, const char *name, int64_t tokens, int64_t heads, const Cache &kv,
                       int64_t &apart) {
    const int64_t dims = t.dim();
    if (t.scalar_type() != kv.dtype)
        refuse(PyExc_TypeError, "%s must have the cache's dtype %s, got %s", name, text(kv.dtype).c_str(),
                               text(t.scalar_type()).c_str());
    on_device(t, name, kv);
    if ((dims != 3 && dims != 4) || t.size(-1) != kv.c.d || (heads >= 0 && t.size(-2) != heads))
        refuse(PyExc_ValueError, "%s has shape %s, expected [.., %s, %d]", name, text(t.sizes()).c_str(),
                                heads < 0 ? "heads" : std::to_string(heads).c_str(), kv.c.d);
    if (t.numel() != tokens * t.size(-2) * kv.c.d)
        refuse(PyExc_ValueError, "%s has shape %s, expected %lld tokens", name, text(t.sizes()).c_str(), (long long)tokens);
    apart = t.size(-2) * kv.c.d;
    if (t.is_contiguous()) return t.data_ptr();
    apart = t.stride(-3);
    if (dims == 4 && t.size(0) > 1) {
        if (t.size(1) == 1) apart = t.stride(0);
        else if (t.stride(0) != t.size(1) * apart) refuse(PyExc_ValueError, "%s's tokens must be evenly spaced", name);
    }
    if (t.stride(-1) != 1 || (t.stride(-2) != kv.c.d && t.size(-2) > 1))
        refuse(PyExc_ValueError, "%s's heads and dims must be contiguous", name);
    return t.data_ptr();
}

// Tokens and sequences of packed [T_total, heads, d] with offsets, or dense [B, T, heads, d].
void sequences(const at::Tensor &x, const at::Tensor *cu, const Cache &kv, int64_t &tokens, int64_t &n) {
    if (cu) {
        if (cu->scalar_type() != at::kInt) refuse(PyExc_TypeError, "cu_seqlens must be int32");
        if (cu->dim() != 1 || cu->numel() < 1) refuse(PyExc_ValueError, "cu_seqlens must be 1-D with num_seqs + 1 entries");
        if (x.dim() != 3) refuse(PyExc_ValueError, "packed tokens must be [T_total, heads, d]");
        tokens = x.size(0);
        n = cu->numel() - 1;
    } else if (x.dim() == 4) {
        n = x.size(0);
        tokens = n * x.size(1);
    } else if (x.dim() == 3) {
        n = 1;
        tokens = x.size(0);
    } else {
        refuse(PyExc_ValueError, "tokens must be [T_total, heads, d] or [B, T, heads, d]");
    }
    if (n > kv.seqs)
        refuse(PyExc_ValueError, "page_table has %lld rows for %lld sequences", (long long)kv.seqs, (long long)n);
}

// The cache's device made current for the call, and the stream that is current on it.  Last before
// the library is called: every operand was found on the cache's device before.
struct Place {
    c10::cuda::OptionalCUDAGuard guard;
    explicit Place(const Cache &kv) {
        if (!kv.device.is_cuda()) refuse(PyExc_ValueError, "the cache must be in CUDA tensors (libgdn has no CPU path)");
        guard.set_device(kv.device);
    }
    cudaStream_t stream(const Cache &kv) const { return c10::cuda::getCurrentCUDAStream(kv.device.index()).stream(); }
};

float number(PyObject *o) {
    const double x = PyFloat_AsDouble(o);
    if (x == -1.0 && PyErr_Occurred()) throw python_error();
    return static_cast<float>(x);
}
int32_t whole(PyObject *o) {
    int overflow = 0;
    const long x = PyLong_AsLongAndOverflow(o, &overflow);
    if (x == -1 && PyErr_Occurred()) throw python_error();
    if (overflow || x < INT32_MIN || x > INT32_MAX) refuse(PyExc_ValueError, "a number does not fit in 32 bits");
    return static_cast<int32_t>(x);
}
float scale_of(PyObject *o, const Cache &kv) {
    return o == Py_None ? static_cast<float>(1.0 / std::sqrt(static_cast<double>(kv.c.d))) : number(o);
}
void expect(Py_ssize_t given, Py_ssize_t want) {
    if (given != want) refuse(PyExc_TypeError, "%d arguments, expected %d", (int)given, (int)want);
}
at::Tensor empty(at::IntArrayRef shape, at::ScalarType dtype, const Cache &kv) {
    return at::empty(shape, at::TensorOptions().dtype(dtype).device(kv.device));
}
// A result the caller gave, or a new tensor: Python objects to return.
PyObject *given_or(PyObject *o, const at::Tensor &made) {
    if (o != Py_None) { Py_INCREF(o); return o; }
    return THPVariable_Wrap(made);
}
struct Scratch {
    at::Tensor made;
    void *at = nullptr;
    size_t bytes = 0;
};
void scratch(Scratch &s, const at::Tensor *given, const Cache &kv) {
    if (!given) return;
    if (given->device() != kv.device || !given->is_contiguous())
        refuse(PyExc_ValueError, "workspace must be contiguous and on %s", kv.device.str().c_str());
    s.at = given->data_ptr();
    s.bytes = given->nbytes();
}

// cache(k, v, page_table): the handle that PagedKV keeps (its Python side checks the tensors)
PyObject *make_cache(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    expect(n, 3);
    const at::Tensor &k = tensor(a[0], "k"), &v = tensor(a[1], "v"), &table = tensor(a[2], "page_table");
    for (int64_t x : {k.size(0), k.size(1), k.size(2), k.size(3), table.size(1)})
        if (x > INT32_MAX) refuse(PyExc_ValueError, "a size does not fit in 32 bits");
    auto *kv = new Cache{{}, k, v, table, k.scalar_type(), k.device(), table.size(0)};
    kv->c.k = k.data_ptr();
    kv->c.v = v.data_ptr();
    kv->c.page_table = static_cast<const int32_t *>(table.data_ptr());
    kv->c.num_pages = (int32_t)k.size(0);
    kv->c.max_pages = (int32_t)table.size(1);
    kv->c.page_size = (int32_t)k.size(1);
    kv->c.H_kv = (int32_t)k.size(2);
    kv->c.d = (int32_t)k.size(3);
    kv->c.dtype = k.scalar_type() == at::kFloat ? GDN_F32 : GDN_BF16;
    return PyCapsule_New(kv, "gdn.cache", [](PyObject *o) { delete static_cast<Cache *>(PyCapsule_GetPointer(o, "gdn.cache")); });
    END_HANDLE_TH_ERRORS
}

// append(cache, k, v, cu_seqlens, pos0, q, q_out, inv_freq, rope_pos, rope_sections, interleaved)
PyObject *append(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    expect(n, 11);
    const Cache &kv = cache(a[0]);
    const at::Tensor &k = tensor(a[1], "k"), &v = tensor(a[2], "v");
    const at::Tensor *cu = maybe(a[3], "cu_seqlens"), *pos0 = maybe(a[4], "pos0"), *q = maybe(a[5], "q"),
                     *q_out = maybe(a[6], "q_out"), *freq = maybe(a[7], "inv_freq"), *rope_pos = maybe(a[8], "rope_pos");
    int64_t tokens, seqs, k_apart, v_apart, q_apart = 0;
    sequences(k, cu, kv, tokens, seqs);
    const void *kp = token_rows(k, "k", tokens, kv.c.H_kv, kv, k_apart);
    const void *vp = token_rows(v, "v", tokens, kv.c.H_kv, kv, v_apart), *qp = nullptr;
    at::Tensor made;
    void *qo = nullptr;
    int64_t heads = 0;
    if (q) {
        qp = token_rows(*q, "q", tokens, -1, kv, q_apart);
        heads = q->size(-2);
        if (!q_out) { made = empty(q->sizes(), kv.dtype, kv); q_out = &made; }
        qo = address(q_out, "q_out", kv.dtype, q->sizes(), kv);
    } else if (q_out) {
        refuse(PyExc_ValueError, "q_out needs q");
    }
    int32_t sections[GDN_ROPE_MAX_AXES] = {}, axes = 1, rope_dims = 0;
    const int32_t *sec = nullptr;
    if (freq) {
        if (freq->numel() > 4096) refuse(PyExc_ValueError, "inv_freq has %lld entries", (long long)freq->numel());
        rope_dims = 2 * (int32_t)freq->numel();
        if (a[9] != Py_None) {
            PyObject *seq = PySequence_Fast(a[9], "rope_sections must be a sequence");
            if (!seq) throw python_error();
            const THPObjectPtr hold(seq);
            const Py_ssize_t count = PySequence_Fast_GET_SIZE(seq);
            if (count < 1 || count > GDN_ROPE_MAX_AXES)
                refuse(PyExc_ValueError, "rope_sections must have 1 to %d entries", GDN_ROPE_MAX_AXES);
            axes = (int32_t)count;
            if (axes > 1 && !rope_pos) refuse(PyExc_ValueError, "several axes need rope_pos");
            for (Py_ssize_t i = 0; i < count; ++i) sections[i] = whole(PySequence_Fast_GET_ITEM(seq, i));
            sec = sections;
        }
    } else if (rope_pos || a[9] != Py_None) {
        refuse(PyExc_ValueError, "rope_pos and rope_sections need inv_freq");
    }
    const auto *cup = static_cast<const int32_t *>(address(cu, "cu_seqlens", at::kInt, {seqs + 1}, kv));
    const auto *pp = static_cast<const int32_t *>(address(pos0, "pos0", at::kInt, {seqs}, kv));
    const auto *fp = static_cast<const float *>(address(freq, "inv_freq", at::kFloat, {rope_dims / 2}, kv));
    const auto *rp = static_cast<const int32_t *>(address(rope_pos, "rope_pos", at::kInt, {axes, tokens}, kv));
    const int turn = PyObject_IsTrue(a[10]);
    if (turn < 0) throw python_error();
    const Place place(kv);
    const gdn_status st = gdn_kv_append(&kv.c, kp, vp, qp, qo, k_apart, v_apart, q_apart, cup, pp, (int32_t)seqs, tokens,
                                        (int32_t)heads, fp, rope_dims, rp, sec, axes, turn ? GDN_ROPE_INTERLEAVED : 0u,
                                        place.stream(kv));
    if (st != GDN_OK) return PyLong_FromLong(st);
    if (!q) Py_RETURN_NONE;
    return given_or(a[6], made);
    END_HANDLE_TH_ERRORS
}

// decode(cache, q, q_pos, token_idx, recent, scale, softcap, window, out, lse, want_lse, workspace):
// token_idx None for the whole cache
PyObject *decode(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    expect(n, 12);
    const Cache &kv = cache(a[0]);
    const at::Tensor &q = tensor(a[1], "q"), &q_pos = tensor(a[2], "q_pos");
    const at::Tensor *list = maybe(a[3], "token_idx"), *out = maybe(a[8], "out"), *lse = maybe(a[9], "lse"),
                     *ws = maybe(a[11], "workspace");
    if (q.dim() != 4 || q.size(3) != kv.c.d)
        refuse(PyExc_ValueError, "q must be [N, n_queries, H_q, %d], got %s", kv.c.d, text(q.sizes()).c_str());
    const int64_t seqs = q.size(0), T = q.size(1), heads = q.size(2);
    if (seqs > kv.seqs)
        refuse(PyExc_ValueError, "page_table has %lld rows for %lld sequences", (long long)kv.seqs, (long long)seqs);
    if (T > INT32_MAX || heads > INT32_MAX) refuse(PyExc_ValueError, "a size does not fit in 32 bits");
    const void *qp = address(&q, "q", kv.dtype, q.sizes(), kv);
    const auto *pp = static_cast<const int32_t *>(address(&q_pos, "q_pos", at::kInt, {seqs}, kv));
    const int32_t *lp = nullptr;
    int64_t list_len = 0;
    if (list) {
        if (list->dim() < 2) refuse(PyExc_ValueError, "token_idx must be [N, n_queries, L]");
        list_len = list->size(-1);
        if (list_len > INT32_MAX) refuse(PyExc_ValueError, "a size does not fit in 32 bits");
        if (T == 1 && list->dim() == 2)
            lp = static_cast<const int32_t *>(address(list, "token_idx", at::kInt, {seqs, list_len}, kv));
        else
            lp = static_cast<const int32_t *>(address(list, "token_idx", at::kInt, {seqs, T, list_len}, kv));
    }
    const int32_t recent = whole(a[4]), window = whole(a[7]);
    const float scale = scale_of(a[5], kv), cap = number(a[6]);
    Scratch s;
    scratch(s, ws, kv);
    const int want = PyObject_IsTrue(a[10]);
    if (want < 0) throw python_error();
    if (out) address(out, "out", kv.dtype, q.sizes(), kv);
    if (lse) address(lse, "lse", at::kFloat, {seqs, T, heads}, kv);
    const Place place(kv);
    at::Tensor made_out, made_lse;
    if (!out) { made_out = empty(q.sizes(), kv.dtype, kv); out = &made_out; }
    if (!lse && want) { made_lse = empty({seqs, T, heads}, at::kFloat, kv); lse = &made_lse; }
    if (!ws) {                             // (its error word, which nobody could read, is left as it is)
        const size_t bytes = gdn_attn_decode_workspace_size((int32_t)T, (int32_t)heads, kv.c.H_kv, kv.c.d, kv.c.dtype);
        s.made = empty({(int64_t)bytes}, at::kByte, kv);
        s.at = s.made.data_ptr();
        s.bytes = bytes;
    }
    float *lsep = lse ? static_cast<float *>(lse->data_ptr()) : nullptr;
    const gdn_status st =
        list ? gdn_qsa_attn_decode(qp, pp, &kv.c, lp, (int32_t)list_len, recent, out->data_ptr(), lsep, (int32_t)seqs,
                                   (int32_t)T, (int32_t)heads, scale, cap, s.at, s.bytes, place.stream(kv))
             : gdn_attn_decode(qp, pp, &kv.c, out->data_ptr(), lsep, (int32_t)seqs, (int32_t)T, (int32_t)heads, scale,
                               cap, window, s.at, s.bytes, place.stream(kv));
    if (st != GDN_OK) return PyLong_FromLong(st);
    const THPObjectPtr o(given_or(a[8], made_out));
    if (!lse) return PyTuple_Pack(2, o.get(), Py_None);
    const THPObjectPtr l(given_or(a[9], made_lse));
    return PyTuple_Pack(2, o.get(), l.get());
    END_HANDLE_TH_ERRORS
}

// prefill(cache, q, cu_seqlens, pos0, prefix_len, scale, softcap, window, out, lse, want_lse, workspace)
PyObject *prefill(PyObject *, PyObject *const *a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    expect(n, 12);
    const Cache &kv = cache(a[0]);
    const at::Tensor &q = tensor(a[1], "q");
    const at::Tensor *cu = maybe(a[2], "cu_seqlens"), *pos0 = maybe(a[3], "pos0"), *prefix = maybe(a[4], "prefix_len"),
                     *out = maybe(a[8], "out"), *lse = maybe(a[9], "lse"), *ws = maybe(a[11], "workspace");
    int64_t tokens, seqs;
    sequences(q, cu, kv, tokens, seqs);
    if (q.size(-1) != kv.c.d)
        refuse(PyExc_ValueError, "q has shape %s, expected head dim %d", text(q.sizes()).c_str(), kv.c.d);
    const int64_t heads = q.size(-2);
    if (heads > INT32_MAX) refuse(PyExc_ValueError, "a size does not fit in 32 bits");
    const void *qp = address(&q, "q", kv.dtype, q.sizes(), kv);
    const auto *cup = static_cast<const int32_t *>(address(cu, "cu_seqlens", at::kInt, {seqs + 1}, kv));
    const auto *pp = static_cast<const int32_t *>(address(pos0, "pos0", at::kInt, {seqs}, kv));
    const auto *fp = static_cast<const int32_t *>(address(prefix, "prefix_len", at::kInt, {seqs}, kv));
    const int32_t window = whole(a[7]);
    const float scale = scale_of(a[5], kv), cap = number(a[6]);
    Scratch s;
    scratch(s, ws, kv);
    const int want = PyObject_IsTrue(a[10]);
    if (want < 0) throw python_error();
    const at::IntArrayRef rows = q.sizes().slice(0, q.dim() - 1);
    if (out) address(out, "out", kv.dtype, q.sizes(), kv);
    if (lse) address(lse, "lse", at::kFloat, rows, kv);
    const Place place(kv);
    at::Tensor made_out, made_lse;
    if (!out) { made_out = empty(q.sizes(), kv.dtype, kv); out = &made_out; }
    if (!lse && want) { made_lse = empty(rows, at::kFloat, kv); lse = &made_lse; }
    if (!ws) {
        const size_t bytes = gdn_attn_prefill_workspace_size(&kv.c, cu != nullptr, (int32_t)seqs, tokens, (int32_t)heads);
        if (bytes > 256) {                 // 256: only the error word, which nobody would read
            s.made = empty({(int64_t)bytes}, at::kByte, kv);
            s.at = s.made.data_ptr();
            s.bytes = bytes;
        }
    }
    const gdn_status st = gdn_attn_prefill(qp, &kv.c, cup, pp, fp, out->data_ptr(),
                                           lse ? static_cast<float *>(lse->data_ptr()) : nullptr, (int32_t)seqs, tokens,
                                           (int32_t)heads, scale, cap, window, s.at, s.bytes, place.stream(kv));
    if (st != GDN_OK) return PyLong_FromLong(st);
    const THPObjectPtr o(given_or(a[8], made_out));
    if (!lse) return PyTuple_Pack(2, o.get(), Py_None);
    const THPObjectPtr l(given_or(a[9], made_lse));
    return PyTuple_Pack(2, o.get(), l.get());
    END_HANDLE_TH_ERRORS
}

#define FAST(name, fn) {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(fn)), METH_FASTCALL, nullptr}
PyMethodDef kMethods[] = {FAST("cache", make_cache), FAST("append", append), FAST("decode", decode),
                          FAST("prefill", prefill), {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_marshal", "Operand checks of libgdn's paged attention calls.", -1, kMethods,
                       nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() { return PyModule_Create(&kModule); }
