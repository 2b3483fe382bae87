// Python module _gdn_bind: argument marshalling of the cache operators and of
// draft verification in native code.
//
// These calls take a few microseconds on the GPU; looking at a dozen tensors'
// types, shapes, strides and devices from Python takes several times that.  So
// paged.py hands its tensors to this module, which makes the same checks with
// the same exceptions, allocates outputs that were not given, and calls the C
// ABI of include/gdn.h with raw pointers and the current stream.  It computes
// nothing.
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>

#include <cstdarg>
#include <initializer_list>
#include <optional>
#include <string>

#include "gdn.h"

namespace {

PyObject* g_fail = nullptr;  // raises GDNError for (function name, status)

struct Bad {};  // a Python exception is set

[[noreturn]] void bad(PyObject* type, const char* fmt, ...) {
    char text[512];
    va_list ap;
    va_start(ap, fmt);
    std::vsnprintf(text, sizeof(text), fmt, ap);
    va_end(ap);
    PyErr_SetString(type, text);
    throw Bad{};
}

std::string shape_text(at::IntArrayRef s) {
    std::string t = "(";
    for (size_t i = 0; i < s.size(); ++i) t += (i ? ", " : "") + std::to_string(s[i]);
    return t + (s.size() == 1 ? ",)" : ")");
}

const at::Tensor& tensor(PyObject* o, const char* name) {
    if (!THPVariable_Check(o)) bad(PyExc_TypeError, "%s must be a torch.Tensor", name);
    return THPVariable_Unpack(o);
}

void want_type(const at::Tensor& t, const char* name, at::ScalarType type) {
    if (t.scalar_type() != type)
        bad(PyExc_TypeError, "%s must be %s, got %s", name, c10::toString(type), c10::toString(t.scalar_type()));
}
void want_shape(const at::Tensor& t, const char* name, at::IntArrayRef shape) {
    if (t.sizes() != shape)
        bad(PyExc_ValueError, "%s must have shape %s, got %s", name, shape_text(shape).c_str(),
            shape_text(t.sizes()).c_str());
}
void want_cuda(const at::Tensor& t, const char* name) {
    if (!t.is_cuda()) bad(PyExc_ValueError, "%s must be a CUDA tensor", name);
}
// A contiguous CUDA tensor of this type (and shape).
const at::Tensor& plain(PyObject* o, const char* name, at::ScalarType type) {
    const at::Tensor& t = tensor(o, name);
    want_type(t, name, type);
    if (!t.is_contiguous()) bad(PyExc_ValueError, "%s must be contiguous", name);
    want_cuda(t, name);
    return t;
}
const at::Tensor& plain(PyObject* o, const char* name, at::ScalarType type, at::IntArrayRef shape) {
    const at::Tensor& t = tensor(o, name);
    want_type(t, name, type);
    want_shape(t, name, shape);
    return plain(o, name, type);
}

template <typename T> const T* struct_at(PyObject* o) {
    return static_cast<const T*>(PyLong_AsVoidPtr(o));
}

at::ScalarType type_of(int32_t dtype) { return dtype == GDN_DTYPE_BF16 ? at::kBFloat16 : at::kFloat; }
int32_t dtype_of(at::ScalarType t) { return t == at::kBFloat16 ? GDN_DTYPE_BF16 : GDN_DTYPE_F32; }

// The cache's codes k, v and scales k_scale, v_scale, as they are at this call.
gdn_kv_cache cache_of(const gdn_kv_dims* d, PyObject* const* a) {
    const at::ScalarType code = d->format == GDN_KV_E4M3 ? at::kFloat8_e4m3fn : at::kChar;
    const at::Tensor& k = tensor(a[0], "cache.k");
    const int64_t n = k.dim() > 0 ? k.size(0) : 0;
    const int64_t codes[4] = {n, d->n_kv_heads, d->page_size, d->head_dim}, scales[2] = {n, d->n_kv_heads};
    if (k.scalar_type() != code || k.sizes() != at::IntArrayRef(codes, 4))
        bad(PyExc_ValueError, "the cache was made for other dimensions or codes");
    if (n > 0x7fffffff) bad(PyExc_ValueError, "a cache has at most 2^31 - 1 pages");
    gdn_kv_cache c;
    c.k = plain(a[0], "cache.k", code).data_ptr();
    c.v = plain(a[1], "cache.v", code, codes).data_ptr();
    c.k_scale = plain(a[2], "cache.k_scale", at::kFloat, scales).data_ptr<float>();
    c.v_scale = plain(a[3], "cache.v_scale", at::kFloat, scales).data_ptr<float>();
    c.n_pages = static_cast<int32_t>(n);
    return c;
}

// cu_seqlens as a (device, host) pair of int32 tensors, the lengths and the pages.
gdn_kv_batch batch_of(PyObject* cu_dev, PyObject* cu_host, PyObject* lens, const char* lens_name, PyObject* table,
                      const int32_t** lens_ptr, int64_t* tokens) {
    const at::Tensor& dev = plain(cu_dev, "cu_seqlens (device)", at::kInt);
    const at::Tensor& host = tensor(cu_host, "cu_seqlens (host)");
    want_type(host, "cu_seqlens (host)", at::kInt);
    if (host.is_cuda() || !host.is_contiguous() || host.numel() != dev.numel() || host.numel() < 1)
        bad(PyExc_ValueError, "cu_seqlens pair must be (device tensor, host tensor) of equal size");
    const int64_t n = host.numel() - 1;
    const at::Tensor& l = plain(lens, lens_name, at::kInt, {n});
    const at::Tensor& t = plain(table, "block_table", at::kInt);
    if (t.dim() != 2 || t.size(0) != n)
        bad(PyExc_ValueError, "block_table must have shape (%lld, pages per sequence), got %s", (long long)n,
            shape_text(t.sizes()).c_str());
    *lens_ptr = l.data_ptr<int32_t>();
    gdn_kv_batch b;
    b.n_seq = static_cast<int32_t>(n);
    b.pages_per_seq = static_cast<int32_t>(t.size(1));
    b.cu_seqlens = dev.data_ptr<int32_t>();
    b.cu_seqlens_host = host.data_ptr<int32_t>();
    b.block_table = t.data_ptr<int32_t>();
    *tokens = n > 0 ? b.cu_seqlens_host[n] : 0;
    return b;
}

// Rows [tokens, heads, head_dim] with free token and head strides.
gdn_rows rows_of(PyObject* o, const char* name, const gdn_kv_dims* d, int64_t tokens, int64_t heads) {
    const at::Tensor& t = tensor(o, name);
    want_type(t, name, type_of(d->dtype));
    want_shape(t, name, {tokens, heads, d->head_dim});
    want_cuda(t, name);
    if (t.stride(2) != 1) bad(PyExc_ValueError, "%s: a head's channels must be contiguous", name);
    return gdn_rows{t.data_ptr(), t.stride(0), t.stride(1)};
}

// The output given, checked, or a new one.
at::Tensor output(PyObject* o, const char* name, at::ScalarType type, at::IntArrayRef shape, const at::Tensor& like) {
    if (o != Py_None) return plain(o, name, type, shape);
    return at::empty(shape, like.options().dtype(type));
}

struct Named {
    int at;
    const char* name;
};
// The device of a call: that of its CUDA tensors, which must agree (arguments that are not CUDA
// tensors are refused where they are checked).  Looked at before anything else of them.
std::optional<at::Device> device_of(PyObject* const* a, std::initializer_list<Named> args) {
    std::optional<at::Device> device;
    for (const Named& x : args) {
        if (!THPVariable_Check(a[x.at])) continue;
        const at::Tensor& t = THPVariable_Unpack(a[x.at]);
        if (!t.is_cuda()) continue;
        if (!device) device = t.device();
        if (t.device() != *device)
            bad(PyExc_ValueError, "%s is on device %s, the call's other tensors are on %s", x.name, t.device().str().c_str(),
                device->str().c_str());
    }
    return device;
}

// The current stream of a call's device, which is the current device while this lives: a launch on a
// device's default stream goes to the current device.
struct Launch {
    c10::cuda::CUDAGuard guard;
    explicit Launch(const std::optional<at::Device>& device) : guard(device.value()) {}
    void* stream() const { return c10::cuda::getCurrentCUDAStream(guard.current_device().index()).stream(); }
};

void check(const char* fn, gdn_status st) {
    if (st == GDN_OK) return;
    PyObject* r = g_fail ? PyObject_CallFunction(g_fail, "si", fn, static_cast<int>(st)) : nullptr;
    Py_XDECREF(r);
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, fn);
    throw Bad{};
}

// Runs f, which returns a new reference; C++ exceptions become Python ones.
template <typename F> PyObject* guarded(Py_ssize_t n, Py_ssize_t want, F&& f) {
    if (n != want) {
        PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
        return nullptr;
    }
    try {
        return f();
    } catch (const Bad&) {
        return nullptr;
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}

int32_t as_int(PyObject* o) {
    const long v = PyLong_AsLong(o);
    if (v == -1 && PyErr_Occurred()) throw Bad{};
    if (v > 0x7fffffffL || v < -0x7fffffffL) bad(PyExc_ValueError, "%ld does not fit 32 bits", v);
    return static_cast<int32_t>(v);
}

// dims, the cache's k, v, k_scale, v_scale, cu_dev, cu_host, kv_lens, block_table, k, v, q, rope, positions, q_out
PyObject* kv_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 15, [&]() -> PyObject* {
        const auto device = device_of(a, {{1, "cache.k"}, {2, "cache.v"}, {3, "cache.k_scale"}, {4, "cache.v_scale"}, {5, "cu_seqlens"},
                                          {7, "kv_lens"}, {8, "block_table"}, {9, "k"}, {10, "v"}, {11, "q"}, {12, "rope"},
                                          {13, "positions"}, {14, "q_out"}});
        const auto* d = struct_at<gdn_kv_dims>(a[0]);
        const gdn_kv_cache c = cache_of(d, a + 1);
        const int32_t* lens;
        int64_t tokens;
        const gdn_kv_batch b = batch_of(a[5], a[6], a[7], "kv_lens", a[8], &lens, &tokens);
        const gdn_rows k = rows_of(a[9], "k", d, tokens, d->n_kv_heads);
        const gdn_rows v = rows_of(a[10], "v", d, tokens, d->n_kv_heads);
        const at::Tensor& like = THPVariable_Unpack(a[9]);
        gdn_rows q{};
        at::Tensor out;
        const bool with_q = a[11] != Py_None;
        if (with_q) {
            q = rows_of(a[11], "q", d, tokens, d->n_q_heads);
            out = output(a[14], "q_out", type_of(d->dtype), {tokens, d->n_q_heads, d->head_dim}, like);
        }
        const float* rope = nullptr;
        int64_t rope_rows = 0;
        if (a[12] != Py_None) {
            const at::Tensor& r = plain(a[12], "rope", at::kFloat);
            if (r.dim() != 2 || r.size(1) != d->rope_dim)
                bad(PyExc_ValueError, "rope must have shape (rows, %d), got %s", d->rope_dim,
                    shape_text(r.sizes()).c_str());
            rope = r.data_ptr<float>();
            rope_rows = r.size(0);
        }
        const int32_t* positions =
            a[13] == Py_None ? nullptr : plain(a[13], "positions", at::kInt, {tokens}).data_ptr<int32_t>();
        check("gdn_kv_append",
              gdn_kv_append(d, &c, &b, lens, with_q ? &q : nullptr, &k, &v, rope, static_cast<int32_t>(rope_rows),
                            positions, with_q ? out.data_ptr() : nullptr, Launch(device).stream()));
        if (!with_q) Py_RETURN_NONE;
        return THPVariable_Wrap(out);
    });
}

// dims, the cache's k, v, k_scale, v_scale, cu_dev, cu_host, starts, block_table, dtype, k_out, v_out
PyObject* kv_read(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 12, [&]() -> PyObject* {
        const auto device = device_of(a, {{1, "cache.k"}, {2, "cache.v"}, {3, "cache.k_scale"}, {4, "cache.v_scale"}, {5, "cu_seqlens"},
                                          {7, "starts"}, {8, "block_table"}, {10, "k_out"}, {11, "v_out"}});
        const auto* d = struct_at<gdn_kv_dims>(a[0]);
        const gdn_kv_cache c = cache_of(d, a + 1);
        const int32_t* starts;
        int64_t tokens;
        const gdn_kv_batch b = batch_of(a[5], a[6], a[7], "starts", a[8], &starts, &tokens);
        const int32_t dtype = as_int(a[9]);
        const at::Tensor& like = THPVariable_Unpack(a[8]);
        const int64_t shape[3] = {tokens, d->n_kv_heads, d->head_dim};
        at::Tensor k = output(a[10], "k_out", type_of(dtype), shape, like);
        at::Tensor v = output(a[11], "v_out", type_of(dtype), shape, like);
        check("gdn_kv_read", gdn_kv_read(d, &c, &b, starts, dtype, k.data_ptr(), v.data_ptr(), Launch(device).stream()));
        return Py_BuildValue("NN", THPVariable_Wrap(k), THPVariable_Wrap(v));
    });
}

// dims, the cache's k, v, k_scale, v_scale, cu_dev, cu_host, kv_lens, block_table, q, max_kv_len, out, workspace
PyObject* kv_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 13, [&]() -> PyObject* {
        const auto device = device_of(a, {{1, "cache.k"}, {2, "cache.v"}, {3, "cache.k_scale"}, {4, "cache.v_scale"}, {5, "cu_seqlens"},
                                          {7, "kv_lens"}, {8, "block_table"}, {9, "q"}, {11, "out"}, {12, "workspace"}});
        const auto* d = struct_at<gdn_kv_dims>(a[0]);
        const gdn_kv_cache c = cache_of(d, a + 1);
        const int32_t* lens;
        int64_t tokens;
        const gdn_kv_batch b = batch_of(a[5], a[6], a[7], "kv_lens", a[8], &lens, &tokens);
        const gdn_rows q = rows_of(a[9], "q", d, tokens, d->n_q_heads);
        const at::Tensor& like = THPVariable_Unpack(a[9]);
        int32_t longest;
        if (a[10] == Py_None) {
            const int64_t room = static_cast<int64_t>(b.pages_per_seq) * d->page_size;
            longest = room < 0x7fffffff ? static_cast<int32_t>(room) : 0x7fffffff;
        } else {
            longest = as_int(a[10]);
        }
        at::Tensor out = output(a[11], "out", type_of(d->dtype), {tokens, d->n_q_heads, d->head_dim}, like);
        at::Tensor ws;
        if (a[12] != Py_None) {
            ws = tensor(a[12], "workspace");
            if (!ws.is_contiguous()) bad(PyExc_ValueError, "workspace must be contiguous");
            want_cuda(ws, "workspace");
        } else {
            size_t need = 0;
            check("gdn_kv_attention_workspace_size",
                  gdn_kv_attention_workspace_size(d, b.n_seq, b.cu_seqlens_host, longest, &need));
            if (need) ws = at::empty({static_cast<int64_t>(need)}, like.options().dtype(at::kByte));
        }
        check("gdn_kv_attention",
              gdn_kv_attention(d, &c, &b, lens, longest, &q, out.data_ptr(), ws.defined() ? ws.data_ptr() : nullptr,
                               ws.defined() ? ws.nbytes() : 0, Launch(device).stream()));
        return THPVariable_Wrap(out);
    });
}

// Row stride of distributions [n, rows, vocab]: vocab contiguous, rows evenly spaced throughout.
int64_t dist_stride(const at::Tensor& t, const char* name, at::ScalarType type, int64_t n, int64_t rows, int64_t vocab) {
    want_type(t, name, type);
    want_cuda(t, name);
    const int64_t sn = t.stride(0), sv = t.stride(t.dim() - 1);
    int64_t sr = t.dim() == 3 ? t.stride(1) : sn;
    if (rows == 1) sr = n > 1 ? sn : vocab;
    if ((sv != 1 && vocab > 1) || (n > 1 && sn != rows * sr))
        bad(PyExc_ValueError, "%s: rows must be contiguous and evenly spaced", name);
    return sr;
}

// drafts, target, draft, uniforms, noise, form, temperature, accepted, tokens
PyObject* accept_drafts(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
    return guarded(n_args, 9, [&]() -> PyObject* {
        const auto device = device_of(a, {{0, "drafts"}, {1, "target"}, {2, "draft"}, {3, "uniforms"}, {4, "noise"},
                                          {6, "temperature"}, {7, "accepted"}, {8, "tokens"}});
        const at::Tensor& target = tensor(a[1], "target");
        const at::ScalarType type = target.scalar_type();
        if (type != at::kFloat && type != at::kBFloat16)
            bad(PyExc_TypeError, "target must be torch.float32 or torch.bfloat16");
        const at::Tensor& x = plain(a[0], "drafts", at::kInt);
        if (x.dim() != 2 || target.dim() != 3) bad(PyExc_ValueError, "drafts must be [n, T] and target [n, T + 1, vocab]");
        const int64_t n = x.size(0), T = x.size(1), vocab = target.size(2);
        if (vocab > 0x7fffffff) bad(PyExc_ValueError, "vocab must be below 2^31");
        want_shape(target, "target", {n, T + 1, vocab});
        const int64_t ts = dist_stride(target, "target", type, n, T + 1, vocab);
        const void* draft = nullptr;
        int64_t ds = vocab;
        if (a[2] != Py_None && T > 0) {
            const at::Tensor& q = tensor(a[2], "draft");
            want_type(q, "draft", type);
            want_shape(q, "draft", {n, T, vocab});
            ds = dist_stride(q, "draft", type, n, T, vocab);
            draft = q.data_ptr();
        }
        const at::Tensor& u = plain(a[3], "uniforms", at::kFloat, {n, T});
        const at::Tensor& e = tensor(a[4], "noise");
        want_type(e, "noise", at::kFloat);
        want_shape(e, "noise", {n, vocab});
        const int64_t ns = dist_stride(e, "noise", at::kFloat, n, 1, vocab);
        const float* temp = a[6] == Py_None ? nullptr : plain(a[6], "temperature", at::kFloat, {n}).data_ptr<float>();
        at::Tensor accepted = output(a[7], "accepted", at::kInt, {n}, target);
        at::Tensor tokens = output(a[8], "tokens", at::kInt, {n, T + 1}, target);
        check("gdn_accept_drafts",
              gdn_accept_drafts(static_cast<int32_t>(n), static_cast<int32_t>(T), static_cast<int32_t>(vocab),
                                as_int(a[5]), dtype_of(type), x.data_ptr<int32_t>(), target.data_ptr(), ts, draft, ds,
                                temp, u.data_ptr<float>(), e.data_ptr<float>(), ns, accepted.data_ptr<int32_t>(),
                                tokens.data_ptr<int32_t>(), Launch(device).stream()));
        return Py_BuildValue("NN", THPVariable_Wrap(accepted), THPVariable_Wrap(tokens));
    });
}

PyObject* on_failure(PyObject*, PyObject* f) {
    Py_XDECREF(g_fail);
    Py_INCREF(f);
    g_fail = f;
    Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"kv_append", reinterpret_cast<PyCFunction>(kv_append), METH_FASTCALL, nullptr},
    {"kv_read", reinterpret_cast<PyCFunction>(kv_read), METH_FASTCALL, nullptr},
    {"kv_attention", reinterpret_cast<PyCFunction>(kv_attention), METH_FASTCALL, nullptr},
    {"accept_drafts", reinterpret_cast<PyCFunction>(accept_drafts), METH_FASTCALL, nullptr},
    {"on_failure", on_failure, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_gdn_bind", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__gdn_bind() { return PyModule_Create(&module); }
