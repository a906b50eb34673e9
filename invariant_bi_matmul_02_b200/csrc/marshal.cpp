// marshal.cpp -- argument marshalling of the binding's decode-step operators, as a Python extension module.
//
// A decode step calls these operators on a few rows at a time, where checking nine tensors and converting
// thirty arguments in Python costs several times the kernel (17 us for bi_paged_append, whose kernel
// takes 4).  The module does what binding.py's other functions do in Python, and nothing else: it
// checks device, dtype and layout of the torch tensors, allocates outputs with torch when none are
// passed, from the pool of the call's stream, and calls the C entry point with raw device pointers and strides.  The entry
// points' addresses come from the library that binding.py has loaded (bind).
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <cstdint>
#include <string>

#include "bi.h"

namespace {

decltype(&bi_rope) p_rope;
decltype(&bi_paged_append) p_paged_append;
decltype(&bi_paged_decode_attention) p_paged_decode_attention;
decltype(&bi_paged_decode_attention_scratch_bytes) p_scratch_bytes;
decltype(&bi_token_logprobs) p_token_logprobs;
PyObject *g_error;  // binding.BiError(name, status)

using at::Tensor;

[[noreturn]] void refuse(PyObject *type, const std::string &s)
{
    PyErr_SetString(type, s.c_str());
    throw python_error();
}
[[noreturn]] void value_error(const std::string &s) { refuse(PyExc_ValueError, s); }
[[noreturn]] void type_error(const std::string &s) { refuse(PyExc_TypeError, s); }

const char *dtype_name(at::ScalarType t) { return c10::toString(t); }

// A CUDA tensor of one of two dtypes on device `dev` (dev < 0: the current device, which it is set to).
const Tensor &cuda_tensor(PyObject *o, const char *name, at::ScalarType a, at::ScalarType b, int &dev)
{
    if (!THPVariable_Check(o) || !THPVariable_Unpack(o).is_cuda()) value_error(std::string(name) + " must be a CUDA tensor");
    const Tensor &t = THPVariable_Unpack(o);
    if (t.scalar_type() != a && t.scalar_type() != b)
        type_error(std::string(name) + ": dtype " + dtype_name(t.scalar_type()) + " not in (" + dtype_name(a) +
                   (a == b ? "" : std::string(", ") + dtype_name(b)) + ")");
    if (dev < 0) dev = c10::cuda::current_device();
    if (t.device().index() != dev)
        value_error(std::string(name) + " is on cuda:" + std::to_string((int)t.device().index()) +
                    " but the current device is cuda:" + std::to_string(dev) + "; call under `with torch.cuda.device(...)`");
    return t;
}

// [T, H, D] with a head's entries consecutive.
const Tensor &heads(PyObject *o, const char *name, at::ScalarType a, at::ScalarType b, int &dev)
{
    const Tensor &t = cuda_tensor(o, name, a, b, dev);
    if (t.dim() != 3) value_error(std::string(name) + " must be [T, H, D]");
    if (t.size(2) > 1 && t.stride(2) != 1) value_error(std::string(name) + ": a head's entries must be contiguous");
    return t;
}

// A contiguous vector (of n entries unless n < 0).
const Tensor &vec(PyObject *o, const char *name, at::ScalarType a, int64_t n, int &dev)
{
    const Tensor &t = cuda_tensor(o, name, a, a, dev);
    if (t.dim() != 1 || (n >= 0 && t.size(0) != n))
        value_error(std::string(name) + " must be a vector" + (n >= 0 ? " of " + std::to_string(n) : ""));
    if (!t.is_contiguous()) value_error(std::string(name) + " must be contiguous");
    return t;
}

// Leading dimension of a 2-D tensor with unit-stride rows.
int64_t leading(const Tensor &t, const char *name)
{
    if (t.dim() != 2) value_error(std::string(name) + " must be 2-D");
    if (t.size(1) > 1 && t.stride(1) != 1) value_error(std::string(name) + " rows must be contiguous");
    return t.size(0) > 1 ? t.stride(0) : std::max(t.stride(0), t.size(1));
}

bi_rope_layout rope_layout(PyObject *o)
{
    if (PyUnicode_Check(o)) {
        if (PyUnicode_CompareWithASCIIString(o, "half") == 0) return BI_ROPE_HALF;
        if (PyUnicode_CompareWithASCIIString(o, "interleaved") == 0) return BI_ROPE_INTERLEAVED;
    }
    value_error("layout must be 'half' (pairs i, i + R/2) or 'interleaved' (pairs 2i, 2i + 1)");
}

double number(PyObject *o)
{
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw python_error();
    return v;
}

int64_t integer(PyObject *o)
{
    const int64_t v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw python_error();
    return v;
}

int truth(PyObject *o)
{
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw python_error();
    return v;
}

// The call's stream: binding.py passes a raw handle, or None for torch's current stream.  A handle's stream is torch's
// current one while this lives, so that memory made for the call is that stream's: a block whose last work on another
// stream is still to run is not handed out, and one that is freed early is not reused before the call's own work.
struct CallStream {
    void *raw;
    c10::cuda::OptionalCUDAStreamGuard guard;
    CallStream(PyObject *o, int dev)
    {
        if (o == Py_None) {
            raw = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream();
            return;
        }
        raw = PyLong_AsVoidPtr(o);
        if (!raw && PyErr_Occurred()) throw python_error();
        const cudaStream_t s = static_cast<cudaStream_t>(raw);  // cudaStreamLegacy is another handle of the default stream
        guard.reset_stream(c10::cuda::getStreamFromExternal(s == cudaStreamLegacy ? nullptr : s, (c10::DeviceIndex)dev));
    }
};

void *ptr(const Tensor &t) { return t.data_ptr(); }

Tensor empty(at::IntArrayRef sizes, at::ScalarType type, int dev)
{
    return at::empty(sizes, at::TensorOptions().dtype(type).device(c10::kCUDA, (c10::DeviceIndex)dev));
}

void check(const char *name, bi_status st)
{
    if (st == BI_OK) return;
    PyObject *e = PyObject_CallFunction(g_error, "si", name, (int)st);
    if (e) {
        PyErr_SetObject(reinterpret_cast<PyObject *>(Py_TYPE(e)), e);
        Py_DECREF(e);
    }
    throw python_error();
}

void count(Py_ssize_t n, Py_ssize_t want)
{
    if (n != want) type_error("expected " + std::to_string(want) + " arguments, got " + std::to_string(n));
}

// The output an entry point writes: the one passed (returned as the same object) or a new one.
struct Out {
    PyObject *given;
    Tensor made;
    PyObject *result() const
    {
        if (given == Py_None) return THPVariable_Wrap(made);
        Py_INCREF(given);
        return given;
    }
};

#define BI_CALL(name, fn, ...)          \
    {                                   \
        bi_status st_;                  \
        Py_BEGIN_ALLOW_THREADS          \
        st_ = fn(__VA_ARGS__);          \
        Py_END_ALLOW_THREADS            \
        check(name, st_);               \
    }

// rope(x, positions, inv_freq, layout, scale, inverse, out, stream)
PyObject *rope(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    count(n, 8);
    int dev = -1;
    const Tensor &x = heads(a[0], "x", at::kBFloat16, at::kFloat, dev);
    const int64_t T = x.size(0), H = x.size(1), D = x.size(2);
    const Tensor &pos = vec(a[1], "positions", at::kInt, T, dev), &freq = vec(a[2], "inv_freq", at::kDouble, -1, dev);
    const bi_rope_layout layout = rope_layout(a[3]);
    const CallStream stream(a[7], dev);
    Out out{a[6], {}};
    if (out.given == Py_None) out.made = empty({T, H, D}, x.scalar_type(), dev);
    const Tensor &y = out.given == Py_None ? out.made : heads(out.given, "out", x.scalar_type(), x.scalar_type(), dev);
    if (y.sizes() != x.sizes()) value_error("out must be [T, H, D]");
    const float scale = (float)number(a[4]);
    const int inverse = truth(a[5]);
    BI_CALL("bi_rope", p_rope, ptr(x), x.stride(0), x.stride(1), ptr(y), y.stride(0), y.stride(1),
            x.scalar_type() == at::kBFloat16 ? BI_BF16 : BI_F32, static_cast<const int32_t *>(ptr(pos)),
            static_cast<const double *>(ptr(freq)), T, H, D, 2 * freq.size(0), layout, scale, inverse, stream.raw)
    return out.result();
    END_HANDLE_TH_ERRORS
}

bi_paged_cache paged_cache(PyObject *ko, PyObject *vo, int &dev)
{
    const Tensor *t[2];
    const char *names[2] = {"k_cache", "v_cache"};
    PyObject *o[2] = {ko, vo};
    for (int i = 0; i < 2; ++i) {
        t[i] = &cuda_tensor(o[i], names[i], at::kBFloat16, at::kBFloat16, dev);
        if (t[i]->dim() != 4)
            value_error(std::string(names[i]) +
                        " must be [pages, page_size, heads, D] (a transposed view for pages laid out head first)");
        if (t[i]->size(3) > 1 && t[i]->stride(3) != 1)
            value_error(std::string(names[i]) + ": a head's entries must be contiguous");
    }
    if (t[0]->sizes() != t[1]->sizes() || t[0]->strides() != t[1]->strides())
        value_error("k_cache and v_cache must have the same shape and strides");
    const Tensor &k = *t[0];
    return {ptr(k), ptr(*t[1]), k.size(0), k.size(1), k.size(2), k.size(3), k.stride(0), k.stride(1), k.stride(2)};
}

const Tensor &block_table(PyObject *o, int64_t B, int &dev)
{
    const Tensor &t = cuda_tensor(o, "block_table", at::kInt, at::kInt, dev);
    if (t.dim() != 2 || t.size(0) != B) value_error("block_table must be [B, max_pages]");
    return t;
}

// paged_append(k, v, k_cache, v_cache, block_table, seq_lens, cu_new, inv_freq, layout, scale, q, q_out, positions,
//              stream)
PyObject *paged_append(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    count(n, 14);
    constexpr auto bf16 = at::kBFloat16;
    int dev = -1;
    const Tensor &k = heads(a[0], "k", bf16, bf16, dev), &v = heads(a[1], "v", bf16, bf16, dev);
    const bi_paged_cache cache = paged_cache(a[2], a[3], dev);
    const int64_t T = k.size(0);
    if (k.size(1) != cache.heads || k.size(2) != cache.head_dim || v.sizes() != k.sizes())
        value_error("k and v must be [T, heads, D] of the cache's heads and D");
    const Tensor &lens = vec(a[5], "seq_lens", at::kInt, -1, dev);
    const int64_t B = lens.size(0);
    const Tensor &table = block_table(a[4], B, dev);
    const int64_t table_stride = leading(table, "block_table");
    const bool packed = a[6] != Py_None;
    if (!packed && T != B) value_error("without cu_new every sequence has one new token: k must have B tokens");
    const void *cu = packed ? ptr(vec(a[6], "cu_new", at::kInt, B + 1, dev)) : nullptr;
    const Tensor *freq = a[7] == Py_None ? nullptr : &vec(a[7], "inv_freq", at::kDouble, -1, dev);
    const bi_rope_layout layout = rope_layout(a[8]);
    const float scale = (float)number(a[9]);
    const void *pos = a[12] == Py_None ? nullptr : ptr(vec(a[12], "positions", at::kInt, T, dev));
    const CallStream stream(a[13], dev);
    Out out{a[11], {}};
    const Tensor *q = nullptr, *qo = nullptr;
    if (a[10] != Py_None) {
        q = &heads(a[10], "q", bf16, bf16, dev);
        if (q->size(0) != T || q->size(2) != cache.head_dim) value_error("q must be [T, Hq, D]");
        if (out.given == Py_None) out.made = empty(q->sizes(), bf16, dev);
        qo = out.given == Py_None ? &out.made : &heads(out.given, "q_out", bf16, bf16, dev);
        if (qo->sizes() != q->sizes()) value_error("q_out must be [T, Hq, D]");
    } else if (out.given != Py_None) {
        value_error("q_out without q");
    }
    const int64_t Hq = q ? q->size(1) : 0;
    const bool turn = Hq > 0;
    BI_CALL("bi_paged_append", p_paged_append, ptr(k), k.stride(0), k.stride(1), ptr(v), v.stride(0), v.stride(1),
            turn ? ptr(*q) : nullptr, turn ? q->stride(0) : 0, turn ? q->stride(1) : 0, turn ? ptr(*qo) : nullptr,
            turn ? qo->stride(0) : 0, turn ? qo->stride(1) : 0, Hq, &cache, static_cast<const int32_t *>(ptr(table)),
            table_stride, table.size(1), static_cast<const int32_t *>(ptr(lens)), static_cast<const int32_t *>(cu),
            static_cast<const int32_t *>(pos), freq ? static_cast<const double *>(ptr(*freq)) : nullptr,
            freq ? 2 * freq->size(0) : 0, layout, scale, T, B, stream.raw)
    if (!q) Py_RETURN_NONE;
    return out.result();
    END_HANDLE_TH_ERRORS
}

// paged_decode_attention(q, k_cache, v_cache, block_table, seq_lens, max_len, scale, scratch, out, stream)
PyObject *paged_decode_attention(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    count(n, 10);
    constexpr auto bf16 = at::kBFloat16;
    int dev = -1;
    const Tensor &q = heads(a[0], "q", bf16, bf16, dev);
    const bi_paged_cache cache = paged_cache(a[1], a[2], dev);
    const int64_t B = q.size(0), Hq = q.size(1), D = q.size(2);
    if (D != cache.head_dim) value_error("q's head size differs from the cache's");
    if (Hq > 1 && q.stride(1) != D) value_error("q: a token's heads must be contiguous");
    const Tensor &lens = vec(a[4], "seq_lens", at::kInt, B, dev), &table = block_table(a[3], B, dev);
    const int64_t table_stride = leading(table, "block_table"), max_pages = table.size(1);
    const int64_t max_len = a[5] == Py_None ? max_pages * cache.page_size : integer(a[5]);
    const float scale = a[6] == Py_None ? (float)(1.0 / std::sqrt((double)D)) : (float)number(a[6]);
    const CallStream stream(a[9], dev);
    Out out{a[8], {}};
    if (out.given == Py_None) out.made = empty(q.sizes(), bf16, dev);
    const Tensor &o = out.given == Py_None ? out.made : cuda_tensor(out.given, "out", bf16, bf16, dev);
    if (!o.is_contiguous()) value_error("out must be contiguous");
    if (o.sizes() != q.sizes()) value_error("out must be [B, Hq, D]");
    Tensor own;
    const Tensor *scratch = &own;
    if (a[7] == Py_None) {
        own = empty({(int64_t)std::max<size_t>(p_scratch_bytes(B, Hq, D, max_len), 16)}, at::kByte, dev);
    } else {
        if (!THPVariable_Check(a[7]) || !THPVariable_Unpack(a[7]).is_cuda()) value_error("scratch must be device memory");
        scratch = &cuda_tensor(a[7], "scratch", THPVariable_Unpack(a[7]).scalar_type(), THPVariable_Unpack(a[7]).scalar_type(), dev);
        if (!scratch->is_contiguous()) value_error("scratch must be contiguous");
    }
    BI_CALL("bi_paged_decode_attention", p_paged_decode_attention, ptr(q), q.stride(0), &cache,
            static_cast<const int32_t *>(ptr(table)), table_stride, max_pages, static_cast<const int32_t *>(ptr(lens)),
            ptr(o), B, Hq, max_len, scale, ptr(*scratch), scratch->nbytes(), stream.raw)
    return out.result();
    END_HANDLE_TH_ERRORS
}

// token_logprobs(logits, tokens, top_k, scale, stream) -> (logprobs, entropy, logsumexp, top_logprobs, top_tokens)
PyObject *token_logprobs(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    count(n, 5);
    int dev = -1;
    const Tensor &x = cuda_tensor(a[0], "logits", at::kFloat, at::kBFloat16, dev);
    const int64_t ld = leading(x, "logits"), M = x.size(0), V = x.size(1), top = integer(a[2]);
    if (top < 0 || top > V) value_error("top_k must be in 0 .. V");
    const bool scored = a[1] != Py_None;
    const void *tok = scored ? ptr(vec(a[1], "tokens", at::kInt, M, dev)) : nullptr;
    const float scale = (float)number(a[3]);
    const CallStream stream(a[4], dev);
    // Each result has a storage of its own, so that one that is kept or saved takes none of the others along.  The later
    // ones are made beside the dispatcher, as it makes the first (a one-row call 6.6 us on the host, 7.9 with five at::empty).
    const Tensor h = empty({M}, at::kFloat, dev);
    auto make = [&](at::IntArrayRef sizes, at::ScalarType type) {
        const int64_t n = c10::multiply_integers(sizes);
        Tensor t = at::detail::make_tensor<c10::TensorImpl>(
            c10::Storage(c10::Storage::use_byte_size_t(), (size_t)n * 4, h.storage().allocator(), true), h.key_set(),
            c10::scalarTypeToTypeMeta(type));
        t.unsafeGetTensorImpl()->set_sizes_contiguous(sizes);
        return t;
    };
    const Tensor lp = scored ? make({M}, at::kFloat) : Tensor(), lse = make({M}, at::kFloat), tl = make({M, top}, at::kFloat),
                 tt = make({M, top}, at::kInt);
    BI_CALL("bi_token_logprobs", p_token_logprobs, ptr(x), ld, x.scalar_type() == at::kBFloat16 ? BI_BF16 : BI_F32,
            static_cast<const int32_t *>(tok), scale, top, scored ? static_cast<float *>(ptr(lp)) : nullptr,
            static_cast<float *>(ptr(h)), static_cast<float *>(ptr(lse)), static_cast<float *>(ptr(tl)),
            static_cast<int32_t *>(ptr(tt)), M, V, stream.raw)
    PyObject *r = PyTuple_New(5);
    if (!r) return nullptr;
    if (!scored) Py_INCREF(Py_None);
    PyTuple_SET_ITEM(r, 0, scored ? THPVariable_Wrap(lp) : Py_None);
    PyTuple_SET_ITEM(r, 1, THPVariable_Wrap(h));
    PyTuple_SET_ITEM(r, 2, THPVariable_Wrap(lse));
    PyTuple_SET_ITEM(r, 3, THPVariable_Wrap(tl));
    PyTuple_SET_ITEM(r, 4, THPVariable_Wrap(tt));
    return r;
    END_HANDLE_TH_ERRORS
}

// bind(error, rope, paged_append, paged_decode_attention, scratch_bytes, token_logprobs): the exception for a refused
// call and the entry points' addresses.
PyObject *bind(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    count(n, 6);
    void *f[5];
    for (int i = 0; i < 5; ++i) {
        f[i] = PyLong_AsVoidPtr(a[1 + i]);
        if (!f[i]) {
            if (PyErr_Occurred()) throw python_error();
            value_error("an entry point's address is null");
        }
    }
    Py_INCREF(a[0]);
    Py_XSETREF(g_error, a[0]);
    p_rope = reinterpret_cast<decltype(p_rope)>(f[0]);
    p_paged_append = reinterpret_cast<decltype(p_paged_append)>(f[1]);
    p_paged_decode_attention = reinterpret_cast<decltype(p_paged_decode_attention)>(f[2]);
    p_scratch_bytes = reinterpret_cast<decltype(p_scratch_bytes)>(f[3]);
    p_token_logprobs = reinterpret_cast<decltype(p_token_logprobs)>(f[4]);
    Py_RETURN_NONE;
    END_HANDLE_TH_ERRORS
}

#define BI_METHOD(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {BI_METHOD(bind),         BI_METHOD(rope),
                         BI_METHOD(paged_append), BI_METHOD(paged_decode_attention),
                         BI_METHOD(token_logprobs), {nullptr, nullptr, 0, nullptr}};
// The docstring names the torch whose headers this was built with: binding.py loads it with no other.
PyModuleDef module = {PyModuleDef_HEAD_INIT,
                      "_marshal",
                      "Argument marshalling of binding.py's decode-step operators, built for torch " BI_TORCH_VERSION ";",
                      -1,
                      methods,
                      nullptr,
                      nullptr,
                      nullptr,
                      nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal(void) { return PyModule_Create(&module); }
