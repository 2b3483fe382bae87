// Python module _gdn_bind: argument marshalling of the cache operators (8-bit and
// latent), of expanded attention, page copies and draft verification in native code.
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

#include <algorithm>
#include <cstdarg>
#include <initializer_list>
#include <memory>
#include <optional>
#include <string>
#include <vector>

#include "gdn.h"
#include "gdn_memory.h"

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

// ------------------------------------------------------------ the latent cache
gdn_latent_cache latent_cache_of(const gdn_latent_dims* d, PyObject* rows) {
    const at::Tensor& r = tensor(rows, "cache.rows");
    const int64_t n = r.dim() > 0 ? r.size(0) : 0, shape[3] = {n, d->page_size, d->latent_dim + d->rope_dim};
    if (r.scalar_type() != at::kBFloat16 || r.sizes() != at::IntArrayRef(shape, 3))
        bad(PyExc_ValueError, "the cache was made for other dimensions");
    if (n > 0x7fffffff) bad(PyExc_ValueError, "a cache has at most 2^31 - 1 pages");
    return gdn_latent_cache{plain(rows, "cache.rows", at::kBFloat16).data_ptr(), static_cast<int32_t>(n)};
}

// bf16 rows [tokens, heads, width] (heads 0: [tokens, width]) with free strides.  An axis of one
// element is never stepped along: its stride, which may be anything, is given as the dense one.
gdn_rows bf16_rows(const at::Tensor& t, const char* name, int64_t tokens, int64_t heads, int64_t width) {
    want_type(t, name, at::kBFloat16);
    if (heads > 0) want_shape(t, name, {tokens, heads, width});
    else want_shape(t, name, {tokens, width});
    want_cuda(t, name);
    if (t.numel() > 0 && t.stride(t.dim() - 1) != 1) bad(PyExc_ValueError, "%s: a row's channels must be contiguous", name);
    const int64_t hs = heads > 1 ? t.stride(1) : width;
    return gdn_rows{t.data_ptr(), tokens > 1 ? t.stride(0) : (heads > 1 ? heads : 1) * width, hs};
}
gdn_rows bf16_rows(PyObject* o, const char* name, int64_t tokens, int64_t heads, int64_t width) {
    return bf16_rows(tensor(o, name), name, tokens, heads, width);
}

// What is written (`name`) is no memory that other thread blocks still read.
using gdn::Memory;
Memory memory(const gdn_rows& r, int64_t tokens, int64_t heads, int64_t width) {
    return Memory::rows(r.data, tokens, heads, r.token_stride, r.head_stride, width, 2);
}
Memory memory(const at::Tensor& t) { return Memory::array(t.data_ptr(), static_cast<long long>(t.nbytes())); }
void want_apart(const char* name, const Memory& m, const char* other, const Memory& o) {
    if (gdn::meet(m.joined(), o.joined())) bad(PyExc_ValueError, "%s shares memory with %s", name, other);
}

// dims, cache.rows, cu_dev, cu_host, kv_lens, block_table, c, norm_w, q_rope, q_out, rope, positions, rows_out
PyObject* latent_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 13, [&]() -> PyObject* {
        const auto device = device_of(a, {{1, "cache.rows"}, {2, "cu_seqlens"}, {4, "kv_lens"}, {5, "block_table"}, {6, "c"},
                                          {7, "norm_w"}, {8, "q_rope"}, {9, "q_out"}, {10, "rope"}, {11, "positions"},
                                          {12, "rows_out"}});
        if (a[8] == Py_None && a[9] != Py_None) bad(PyExc_ValueError, "q_out without q_rope");
        const auto* d = struct_at<gdn_latent_dims>(a[0]);
        const gdn_latent_cache c = latent_cache_of(d, a[1]);
        const int32_t* lens;
        int64_t tokens;
        const gdn_kv_batch b = batch_of(a[2], a[3], a[4], "kv_lens", a[5], &lens, &tokens);
        const int64_t width = d->latent_dim + d->rope_dim;
        const gdn_rows rows = bf16_rows(a[6], "c", tokens, 0, width);
        const at::Tensor& like = THPVariable_Unpack(a[6]);
        const float* norm = a[7] == Py_None ? nullptr : plain(a[7], "norm_w", at::kFloat, {d->latent_dim}).data_ptr<float>();
        gdn_rows q{}, q_out{};
        at::Tensor out;
        const bool with_q = a[8] != Py_None;
        if (with_q) {
            q = bf16_rows(a[8], "q_rope", tokens, d->n_heads, d->rope_dim);
            out = a[9] != Py_None ? tensor(a[9], "q_out")
                                  : at::empty({tokens, d->n_heads, d->rope_dim}, like.options().dtype(at::kBFloat16));
            q_out = bf16_rows(out, "q_out", tokens, d->n_heads, d->rope_dim);
            const Memory written = memory(q_out, tokens, d->n_heads, d->rope_dim);
            const Memory read = memory(q, tokens, d->n_heads, d->rope_dim);
            if (!gdn::same(written, read)) want_apart("q_out", written, "q_rope", read);
            want_apart("q_out", written, "c", memory(rows, tokens, 1, width));
            want_apart("q_out", written, "cache.rows", memory(tensor(a[1], "cache.rows")));
        }
        const float* rope = nullptr;
        int64_t rope_rows = 0;
        if (a[10] != Py_None) {
            const at::Tensor& r = plain(a[10], "rope", at::kFloat);
            if (r.dim() != 2 || r.size(1) != d->rope_dim)
                bad(PyExc_ValueError, "rope must have shape (rows, %d), got %s", d->rope_dim, shape_text(r.sizes()).c_str());
            rope = r.data_ptr<float>();
            rope_rows = r.size(0);
            if (rope_rows < 1) bad(PyExc_ValueError, "rope must hold at least one row");
            if (rope_rows > 0x7fffffff) bad(PyExc_ValueError, "rope has at most 2^31 - 1 rows");
        }
        const int32_t* positions =
            a[11] == Py_None ? nullptr : plain(a[11], "positions", at::kInt, {tokens}).data_ptr<int32_t>();
        void* packed = a[12] == Py_None ? nullptr : plain(a[12], "rows_out", at::kBFloat16, {tokens, width}).data_ptr();
        check("gdn_latent_append",
              gdn_latent_append(d, &c, &b, lens, &rows, norm, with_q ? &q : nullptr, with_q ? &q_out : nullptr, rope,
                                static_cast<int32_t>(rope_rows), positions, packed, Launch(device).stream()));
        if (!with_q) Py_RETURN_NONE;
        return THPVariable_Wrap(out);
    });
}

// dims, cache.rows, cu_dev, cu_host, starts, block_table, out
PyObject* latent_read(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 7, [&]() -> PyObject* {
        const auto device = device_of(a, {{1, "cache.rows"}, {2, "cu_seqlens"}, {4, "starts"}, {5, "block_table"}, {6, "out"}});
        const auto* d = struct_at<gdn_latent_dims>(a[0]);
        const gdn_latent_cache c = latent_cache_of(d, a[1]);
        const int32_t* starts;
        int64_t tokens;
        const gdn_kv_batch b = batch_of(a[2], a[3], a[4], "starts", a[5], &starts, &tokens);
        at::Tensor out = output(a[6], "out", at::kBFloat16, {tokens, d->latent_dim + d->rope_dim}, THPVariable_Unpack(a[5]));
        want_apart("out", memory(out), "cache.rows", memory(tensor(a[1], "cache.rows")));
        check("gdn_latent_read", gdn_latent_read(d, &c, &b, starts, out.data_ptr(), Launch(device).stream()));
        return THPVariable_Wrap(out);
    });
}

// dims, cache.rows, cu_dev, cu_host, kv_lens, block_table, q, out, workspace
PyObject* latent_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 9, [&]() -> PyObject* {
        const auto device = device_of(a, {{1, "cache.rows"}, {2, "cu_seqlens"}, {4, "kv_lens"}, {5, "block_table"}, {6, "q"},
                                          {7, "out"}, {8, "workspace"}});
        const auto* d = struct_at<gdn_latent_dims>(a[0]);
        const gdn_latent_cache c = latent_cache_of(d, a[1]);
        const int32_t* lens;
        int64_t tokens;
        const gdn_kv_batch b = batch_of(a[2], a[3], a[4], "kv_lens", a[5], &lens, &tokens);
        const gdn_rows q = bf16_rows(a[6], "q", tokens, d->n_heads, d->latent_dim + d->rope_dim);
        const at::Tensor& like = THPVariable_Unpack(a[6]);
        at::Tensor out = output(a[7], "out", at::kBFloat16, {tokens, d->n_heads, d->latent_dim}, like);
        at::Tensor ws;
        if (a[8] != Py_None) {
            ws = tensor(a[8], "workspace");
            if (!ws.is_contiguous()) bad(PyExc_ValueError, "workspace must be contiguous");
            want_cuda(ws, "workspace");
        } else {
            size_t need = 0;
            check("gdn_latent_attention_workspace_size",
                  gdn_latent_attention_workspace_size(d, b.n_seq, b.cu_seqlens_host, &need));
            if (need) ws = at::empty({static_cast<int64_t>(need)}, like.options().dtype(at::kByte));
        }
        const Memory in_q = memory(q, tokens, d->n_heads, d->latent_dim + d->rope_dim), in_c = memory(tensor(a[1], "cache.rows"));
        want_apart("out", memory(out), "q", in_q);
        want_apart("out", memory(out), "cache.rows", in_c);
        if (a[8] != Py_None) {
            want_apart("workspace", memory(ws), "q", in_q);
            want_apart("workspace", memory(ws), "cache.rows", in_c);
            want_apart("workspace", memory(ws), "out", memory(out));
        }
        check("gdn_latent_attention",
              gdn_latent_attention(d, &c, &b, lens, &q, out.data_ptr(), ws.defined() ? ws.data_ptr() : nullptr,
                                   ws.defined() ? ws.nbytes() : 0, Launch(device).stream()));
        return THPVariable_Wrap(out);
    });
}

// A (device, host) pair of int32 cu_seqlens: entries and pointers.
struct Cu {
    const int32_t *dev, *host;
    int64_t n, total;
};
Cu cu_of(PyObject* cu_dev, PyObject* cu_host, const char* name) {
    const at::Tensor& dev = plain(cu_dev, name, at::kInt);
    const at::Tensor& host = tensor(cu_host, name);
    want_type(host, name, at::kInt);
    if (host.is_cuda() || !host.is_contiguous() || host.numel() != dev.numel() || host.numel() < 1)
        bad(PyExc_ValueError, "%s pair must be (device tensor, host tensor) of equal size", name);
    Cu c{dev.data_ptr<int32_t>(), host.data_ptr<int32_t>(), host.numel() - 1, 0};
    if (c.n > 0) c.total = c.host[c.n];
    return c;
}

// dims, cu_q dev, host, cu_kv dev, host, q, k, k_rope, v, out
PyObject* expanded_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 10, [&]() -> PyObject* {
        const auto device = device_of(a, {{1, "cu_q"}, {3, "cu_kv"}, {5, "q"}, {6, "k"}, {7, "k_rope"}, {8, "v"}, {9, "out"}});
        const auto* d = struct_at<gdn_latent_dims>(a[0]);
        const Cu cq = cu_of(a[1], a[2], "cu_q"), ck = cu_of(a[3], a[4], "cu_kv");
        if (cq.n != ck.n) bad(PyExc_ValueError, "cu_q and cu_kv must name as many sequences");
        const gdn_rows q = bf16_rows(a[5], "q", cq.total, d->n_heads, d->nope_dim + d->rope_dim);
        const gdn_rows k = bf16_rows(a[6], "k", ck.total, d->n_heads, d->nope_dim);
        const gdn_rows r = bf16_rows(a[7], "k_rope", ck.total, 0, d->rope_dim);
        const gdn_rows v = bf16_rows(a[8], "v", ck.total, d->n_heads, d->v_dim);
        at::Tensor out = output(a[9], "out", at::kBFloat16, {cq.total, d->n_heads, d->v_dim}, THPVariable_Unpack(a[5]));
        const Memory written = memory(out);
        want_apart("out", written, "q", memory(q, cq.total, d->n_heads, d->nope_dim + d->rope_dim));
        want_apart("out", written, "k", memory(k, ck.total, d->n_heads, d->nope_dim));
        want_apart("out", written, "k_rope", memory(r, ck.total, 1, d->rope_dim));
        want_apart("out", written, "v", memory(v, ck.total, d->n_heads, d->v_dim));
        check("gdn_expanded_attention",
              gdn_expanded_attention(d, static_cast<int32_t>(cq.n), cq.dev, cq.host, ck.dev, ck.host, &q, &k, &r, &v,
                                     out.data_ptr(), Launch(device).stream()));
        return THPVariable_Wrap(out);
    });
}

// Page numbers: a list or tuple of ints, or a 1-d int32 tensor on the host.
std::vector<int32_t> pages_of(PyObject* o, const char* name) {
    std::vector<int32_t> v;
    if (THPVariable_Check(o)) {
        const at::Tensor& t = THPVariable_Unpack(o);
        want_type(t, name, at::kInt);
        if (t.is_cuda() || t.dim() != 1 || !t.is_contiguous())
            bad(PyExc_ValueError, "%s must be a list of page numbers or a 1-d host tensor", name);
        v.assign(t.data_ptr<int32_t>(), t.data_ptr<int32_t>() + t.numel());
        return v;
    }
    if (!PyList_Check(o) && !PyTuple_Check(o))
        bad(PyExc_TypeError, "%s must be a list of page numbers or a 1-d host tensor", name);
    v.reserve(PySequence_Fast_GET_SIZE(o));
    for (Py_ssize_t i = 0; i < PySequence_Fast_GET_SIZE(o); ++i) {  // an item's __index__ may change the list
        PyObject* item = PySequence_Fast_GET_ITEM(o, i);
        Py_INCREF(item);
        const std::unique_ptr<PyObject, void (*)(PyObject*)> held(item, Py_DecRef);
        v.push_back(as_int(item));
    }
    return v;
}

// the caches' tensors (a tuple, first axis: pages), src, dst
PyObject* copy_pages(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 3, [&]() -> PyObject* {
        if (!PyTuple_Check(a[0])) bad(PyExc_TypeError, "caches must be a tuple of tensors");
        // first: an item's __index__ may do anything, also to the caches' tensors
        const std::vector<int32_t> src = pages_of(a[1], "src"), dst = pages_of(a[2], "dst");
        if (src.size() != dst.size()) bad(PyExc_ValueError, "src and dst must have as many pages (%zu, %zu)", src.size(), dst.size());
        if (src.size() > 0x7fffffff) bad(PyExc_ValueError, "more than 2^31 - 1 pairs");
        const Py_ssize_t n_buffers = PyTuple_GET_SIZE(a[0]);
        std::vector<void*> bases;
        std::vector<size_t> bytes;
        int64_t pages = 0x7fffffff;
        std::optional<at::Device> device;
        for (Py_ssize_t i = 0; i < n_buffers; ++i) {
            const at::Tensor& t = tensor(PyTuple_GET_ITEM(a[0], i), "a cache's tensor");
            want_cuda(t, "a cache's tensor");
            if (!t.is_contiguous() || t.dim() < 2) bad(PyExc_ValueError, "a cache's tensor must be contiguous");
            if (!device) device = t.device();
            if (t.device() != *device)
                bad(PyExc_ValueError, "the caches are on devices %s and %s", device->str().c_str(), t.device().str().c_str());
            pages = std::min(pages, t.size(0));
            if (t.size(0) == 0) continue;
            bases.push_back(t.data_ptr());
            bytes.push_back(t.nbytes() / t.size(0));
        }
        if (bases.empty() && (n_buffers == 0 || src.empty())) Py_RETURN_NONE;
        if (bases.empty()) bad(PyExc_ValueError, "the caches have no pages");
        check("gdn_copy_pages",
              gdn_copy_pages(static_cast<int32_t>(bases.size()), bases.data(), bytes.data(), static_cast<int32_t>(pages),
                             static_cast<int32_t>(src.size()), src.data(), dst.data(), Launch(device).stream()));
        Py_RETURN_NONE;
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
    {"latent_append", reinterpret_cast<PyCFunction>(latent_append), METH_FASTCALL, nullptr},
    {"latent_read", reinterpret_cast<PyCFunction>(latent_read), METH_FASTCALL, nullptr},
    {"latent_attention", reinterpret_cast<PyCFunction>(latent_attention), METH_FASTCALL, nullptr},
    {"expanded_attention", reinterpret_cast<PyCFunction>(expanded_attention), METH_FASTCALL, nullptr},
    {"copy_pages", reinterpret_cast<PyCFunction>(copy_pages), METH_FASTCALL, nullptr},
    {"on_failure", on_failure, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_gdn_bind", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__gdn_bind() { return PyModule_Create(&module); }
