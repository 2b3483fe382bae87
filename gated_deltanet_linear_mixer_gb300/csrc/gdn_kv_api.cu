// C-ABI entry points of the paged 8-bit cache and of draft verification
// (declared in include/gdn.h): host-side validation, error reporting and
// dispatch on the caller's stream.
#include <cmath>

#include "gdn.h"
#include "gdn_internal.h"
#include "gdn_kv.h"

namespace gdn {
// Records the thread's error message (defined with the other entry points).
gdn_status set_error(gdn_status st, const char* fn, const char* fmt, ...);
void clear_error();
// GDN_ERR_INJECTED when the environment variable GDN_FAULT lists `site`.
gdn_status inject_fault(const char* site, const char* fn);
bool fault_site(const char* site);  // whether it does
}  // namespace gdn

using gdn::set_error;
using gdn::timed_launch;

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

gdn_status cuda_status(cudaError_t e, const char* fn, const char* what) {
    if (e == cudaSuccess) return GDN_OK;
    return set_error(GDN_ERR_CUDA, fn, "%s failed: %s (%s)", what, cudaGetErrorName(e), cudaGetErrorString(e));
}

gdn_status check_kv_dims(const gdn_kv_dims* d, const char* fn) {
    if (!d) return set_error(GDN_ERR_INVALID_ARG, fn, "dims is NULL");
    if (d->n_q_heads < 1 || d->n_kv_heads < 1)
        return set_error(GDN_ERR_INVALID_ARG, fn, "head counts must be >= 1 (Hq=%d, Hkv=%d)", d->n_q_heads,
                         d->n_kv_heads);
    if (d->n_q_heads % d->n_kv_heads != 0 || d->n_q_heads / d->n_kv_heads > 64)
        return set_error(GDN_ERR_UNSUPPORTED, fn, "n_q_heads (%d) must be a multiple of n_kv_heads (%d), at most 64 times",
                         d->n_q_heads, d->n_kv_heads);
    if (d->n_q_heads > 4096) return set_error(GDN_ERR_UNSUPPORTED, fn, "n_q_heads %d is above 4096", d->n_q_heads);
    if (d->head_dim != 64 && d->head_dim != 128 && d->head_dim != 256)
        return set_error(GDN_ERR_UNSUPPORTED, fn, "head_dim must be 64, 128 or 256 (got %d)", d->head_dim);
    if (d->page_size != 16 && d->page_size != 32 && d->page_size != 64 && d->page_size != 128)
        return set_error(GDN_ERR_UNSUPPORTED, fn, "page_size must be 16, 32, 64 or 128 (got %d)", d->page_size);
    if (d->dtype != GDN_DTYPE_F32 && d->dtype != GDN_DTYPE_BF16)
        return set_error(GDN_ERR_INVALID_ARG, fn, "dtype %d is not a gdn_dtype", d->dtype);
    if (d->format != GDN_KV_INT8 && d->format != GDN_KV_E4M3)
        return set_error(GDN_ERR_INVALID_ARG, fn, "format %d is not a gdn_kv_format", d->format);
    if (d->rope_dim < 0 || d->rope_dim > d->head_dim || d->rope_dim % 16 != 0)
        return set_error(GDN_ERR_UNSUPPORTED, fn, "rope_dim must be a multiple of 16 in 0..head_dim (got %d)",
                         d->rope_dim);
    if (d->rope_style != GDN_ROPE_HALF && d->rope_style != GDN_ROPE_INTERLEAVED)
        return set_error(GDN_ERR_INVALID_ARG, fn, "rope_style %d is not a gdn_rope_style", d->rope_style);
    if (d->window < 0) return set_error(GDN_ERR_INVALID_ARG, fn, "window must be >= 0 (got %d)", d->window);
    if (!(d->scale > 0.f) || !std::isfinite(d->scale))
        return set_error(GDN_ERR_INVALID_ARG, fn, "scale must be finite and > 0");
    return GDN_OK;
}

gdn_status check_cache(const gdn_kv_cache* c, const char* fn) {
    if (!c) return set_error(GDN_ERR_INVALID_ARG, fn, "cache is NULL");
    if (c->n_pages < 0) return set_error(GDN_ERR_INVALID_ARG, fn, "n_pages must be >= 0 (got %d)", c->n_pages);
    if (c->n_pages > 0 && (!c->k || !c->v || !c->k_scale || !c->v_scale))
        return set_error(GDN_ERR_INVALID_ARG, fn, "a cache pointer is NULL");
    if (!aligned16(c->k) || !aligned16(c->v))
        return set_error(GDN_ERR_INVALID_ARG, fn, "the cache's codes must be 16-byte aligned");
    return GDN_OK;
}

// Validates the host copy of cu_seqlens; fills the batch but for the lengths.
gdn_status check_cu(int32_t n_seq, const int32_t* cu_host, const char* fn) {
    if (n_seq < 0) return set_error(GDN_ERR_INVALID_ARG, fn, "n_seq must be >= 0 (got %d)", n_seq);
    if (n_seq > GDN_MAX_SEQUENCES)
        return set_error(GDN_ERR_UNSUPPORTED, fn, "n_seq %d is above GDN_MAX_SEQUENCES (%d)", n_seq,
                         GDN_MAX_SEQUENCES);
    if (n_seq == 0) return GDN_OK;
    if (!cu_host) return set_error(GDN_ERR_INVALID_ARG, fn, "cu_seqlens pointer is NULL");
    if (cu_host[0] != 0) return set_error(GDN_ERR_INVALID_ARG, fn, "cu_seqlens[0] must be 0");
    for (int i = 0; i < n_seq; ++i)
        if (cu_host[i + 1] < cu_host[i])
            return set_error(GDN_ERR_INVALID_ARG, fn, "cu_seqlens decreases at index %d", i + 1);
    return GDN_OK;
}

gdn_status check_batch(const gdn_kv_batch* b, const int32_t* lens, gdn::KvBatch* out, const char* fn) {
    if (!b) return set_error(GDN_ERR_INVALID_ARG, fn, "batch is NULL");
    gdn_status st = check_cu(b->n_seq, b->cu_seqlens_host, fn);
    if (st != GDN_OK) return st;
    *out = gdn::KvBatch{};
    if (b->n_seq == 0) return GDN_OK;
    const int32_t* cu = b->cu_seqlens_host;
    out->n_seq = b->n_seq;
    out->n_tokens = cu[b->n_seq];
    if (out->n_tokens == 0) return GDN_OK;
    if (b->pages_per_seq < 0) return set_error(GDN_ERR_INVALID_ARG, fn, "pages_per_seq must be >= 0");
    if (!b->cu_seqlens || !lens || (b->pages_per_seq > 0 && !b->block_table))
        return set_error(GDN_ERR_INVALID_ARG, fn, "cu_seqlens, the lengths or block_table is NULL");
    out->pages_per_seq = b->pages_per_seq;
    out->cu = b->cu_seqlens;
    out->kv_lens = lens;
    out->table = b->block_table;
    int lo = cu[1], hi = cu[1];
    for (int i = 1; i < b->n_seq; ++i) {
        const int q = cu[i + 1] - cu[i];
        lo = q < lo ? q : lo;
        hi = q > hi ? q : hi;
    }
    out->max_q = hi;
    out->uniform_q = lo == hi ? hi : 0;
    return GDN_OK;
}

gdn_status check_rows(const gdn_rows* r, const char* name, const gdn_kv_dims* d, gdn::KvRows* out, const char* fn) {
    if (!r || !r->data) return set_error(GDN_ERR_INVALID_ARG, fn, "%s is NULL", name);
    const int64_t per16 = d->dtype == GDN_DTYPE_BF16 ? 8 : 4;
    if (r->token_stride < 0 || r->head_stride < 0)
        return set_error(GDN_ERR_INVALID_ARG, fn, "%s has a negative stride", name);
    if (!aligned16(r->data) || r->token_stride % per16 != 0 || r->head_stride % per16 != 0)
        return set_error(GDN_ERR_INVALID_ARG, fn, "%s: the base and both strides must be multiples of 16 bytes", name);
    *out = gdn::KvRows{r->data, r->token_stride, r->head_stride};
    return GDN_OK;
}

size_t attention_workspace(const gdn_kv_dims* d, int n_seq, int max_q, int max_kv_len) {
    return gdn::kv_attention_workspace(n_seq, max_q, d->n_q_heads, d->n_kv_heads, d->head_dim, d->window,
                                       d->dtype == GDN_DTYPE_BF16, max_kv_len);
}

gdn::KvCache cache_of(const gdn_kv_cache* c) {
    return gdn::KvCache{static_cast<uint8_t*>(c->k), static_cast<uint8_t*>(c->v), c->k_scale, c->v_scale, c->n_pages};
}

}  // namespace

extern "C" {

gdn_status gdn_kv_append(const gdn_kv_dims* dims, const gdn_kv_cache* cache, const gdn_kv_batch* batch,
                         const int32_t* kv_lens, const gdn_rows* q, const gdn_rows* k, const gdn_rows* v,
                         const float* rope, int32_t rope_len, const int32_t* positions, void* q_out, void* stream) {
    const char* fn = "gdn_kv_append";
    gdn_status st;
    gdn::KvAppendArgs a{};
    if ((st = check_kv_dims(dims, fn)) != GDN_OK) return st;
    if ((st = check_cache(cache, fn)) != GDN_OK) return st;
    if ((st = check_batch(batch, kv_lens, &a.b, fn)) != GDN_OK) return st;
    gdn::clear_error();
    if (a.b.n_tokens == 0) return GDN_OK;
    if ((st = check_rows(k, "k", dims, &a.k, fn)) != GDN_OK) return st;
    if ((st = check_rows(v, "v", dims, &a.v, fn)) != GDN_OK) return st;
    if (q) {
        if ((st = check_rows(q, "q", dims, &a.q, fn)) != GDN_OK) return st;
        if (!q_out || !aligned16(q_out))
            return set_error(GDN_ERR_INVALID_ARG, fn, "q_out must be given with q and be 16-byte aligned");
    }
    if (dims->rope_dim > 0 && (!rope || rope_len < 1 || !aligned16(rope)))
        return set_error(GDN_ERR_INVALID_ARG, fn, "rope must hold at least one row and be 16-byte aligned");
    if ((st = gdn::inject_fault("kv_append", fn)) != GDN_OK) return st;
    if ((st = cuda_status(gdn::cache_error_word(&a.error), fn, "finding the error word")) != GDN_OK) return st;
    a.c = cache_of(cache);
    a.n_q_heads = dims->n_q_heads; a.n_kv_heads = dims->n_kv_heads; a.page_size = dims->page_size;
    a.rope_dim = dims->rope_dim; a.rope_style = dims->rope_style; a.rope = rope; a.rope_len = rope_len;
    a.positions = positions; a.q_out = q_out;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return cuda_status(timed_launch("kv_append", s, [&] {
                           return gdn::launch_kv_append(a, dims->head_dim, dims->dtype == GDN_DTYPE_BF16,
                                                        dims->format == GDN_KV_E4M3, s);
                       }), fn, "append launch");
}

gdn_status gdn_kv_read(const gdn_kv_dims* dims, const gdn_kv_cache* cache, const gdn_kv_batch* batch,
                       const int32_t* starts, int32_t out_dtype, void* k_out, void* v_out, void* stream) {
    const char* fn = "gdn_kv_read";
    gdn_status st;
    gdn::KvReadArgs a{};
    if ((st = check_kv_dims(dims, fn)) != GDN_OK) return st;
    if ((st = check_cache(cache, fn)) != GDN_OK) return st;
    if ((st = check_batch(batch, starts, &a.b, fn)) != GDN_OK) return st;
    if (out_dtype != GDN_DTYPE_F32 && out_dtype != GDN_DTYPE_BF16)
        return set_error(GDN_ERR_INVALID_ARG, fn, "out_dtype %d is not a gdn_dtype", out_dtype);
    gdn::clear_error();
    if (a.b.n_tokens == 0) return GDN_OK;
    if (!k_out || !v_out || !aligned16(k_out) || !aligned16(v_out))
        return set_error(GDN_ERR_INVALID_ARG, fn, "k_out and v_out must be given and 16-byte aligned");
    if ((st = gdn::inject_fault("kv_read", fn)) != GDN_OK) return st;
    if ((st = cuda_status(gdn::cache_error_word(&a.error), fn, "finding the error word")) != GDN_OK) return st;
    a.c = cache_of(cache);
    a.n_kv_heads = dims->n_kv_heads; a.page_size = dims->page_size; a.k_out = k_out; a.v_out = v_out;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return cuda_status(timed_launch("kv_read", s, [&] {
                           return gdn::launch_kv_read(a, dims->head_dim, out_dtype == GDN_DTYPE_BF16,
                                                      dims->format == GDN_KV_E4M3, s);
                       }), fn, "read launch");
}

gdn_status gdn_kv_attention_workspace_size(const gdn_kv_dims* dims, int32_t n_seq, const int32_t* cu_seqlens_host,
                                           int32_t max_kv_len, size_t* bytes) {
    const char* fn = "gdn_kv_attention_workspace_size";
    gdn_status st;
    if ((st = check_kv_dims(dims, fn)) != GDN_OK) return st;
    if (!bytes) return set_error(GDN_ERR_INVALID_ARG, fn, "bytes is NULL");
    if ((st = check_cu(n_seq, cu_seqlens_host, fn)) != GDN_OK) return st;
    if (max_kv_len < 0) return set_error(GDN_ERR_INVALID_ARG, fn, "max_kv_len must be >= 0 (got %d)", max_kv_len);
    int max_q = 0;
    for (int i = 0; i < n_seq; ++i) {
        const int q = cu_seqlens_host[i + 1] - cu_seqlens_host[i];
        max_q = q > max_q ? q : max_q;
    }
    *bytes = attention_workspace(dims, n_seq, max_q, max_kv_len);
    gdn::clear_error();
    return GDN_OK;
}

gdn_status gdn_kv_attention(const gdn_kv_dims* dims, const gdn_kv_cache* cache, const gdn_kv_batch* batch,
                            const int32_t* kv_lens, int32_t max_kv_len, const gdn_rows* q, void* out,
                            void* workspace, size_t workspace_bytes, void* stream) {
    const char* fn = "gdn_kv_attention";
    gdn_status st;
    gdn::KvAttnArgs a{};
    if ((st = check_kv_dims(dims, fn)) != GDN_OK) return st;
    if ((st = check_cache(cache, fn)) != GDN_OK) return st;
    if ((st = check_batch(batch, kv_lens, &a.b, fn)) != GDN_OK) return st;
    if (max_kv_len < 0) return set_error(GDN_ERR_INVALID_ARG, fn, "max_kv_len must be >= 0 (got %d)", max_kv_len);
    gdn::clear_error();
    if (a.b.n_tokens == 0) return GDN_OK;
    if ((st = check_rows(q, "q", dims, &a.q, fn)) != GDN_OK) return st;
    if (!out || !aligned16(out)) return set_error(GDN_ERR_INVALID_ARG, fn, "out must be given and 16-byte aligned");
    const size_t need = attention_workspace(dims, a.b.n_seq, a.b.max_q, max_kv_len);
    if (need > 0 && (!workspace || workspace_bytes < need))
        return set_error(GDN_ERR_WORKSPACE, fn, "workspace of %zu bytes needed, %zu given", need,
                         workspace ? workspace_bytes : (size_t)0);
    if (need > 0 && (reinterpret_cast<uintptr_t>(workspace) & 255u))
        return set_error(GDN_ERR_WORKSPACE, fn, "workspace must be 256-byte aligned");
    if ((st = gdn::inject_fault("kv_attention", fn)) != GDN_OK) return st;
    if ((st = cuda_status(gdn::cache_error_word(&a.error), fn, "finding the error word")) != GDN_OK) return st;
    a.c = cache_of(cache);
    a.n_q_heads = dims->n_q_heads; a.n_kv_heads = dims->n_kv_heads; a.page_size = dims->page_size;
    a.window = dims->window; a.scale = dims->scale; a.out = out; a.partial = static_cast<float*>(workspace);
    a.max_kv_len = max_kv_len;
    a.stall = gdn::fault_site("stall_attention") ? 1 : 0;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return cuda_status(gdn::launch_kv_attention(a, dims->head_dim, dims->dtype == GDN_DTYPE_BF16,
                                                dims->format == GDN_KV_E4M3, s), fn, "attention launch");
}

gdn_status gdn_accept_drafts(int32_t n_seq, int32_t T, int32_t vocab, int32_t form, int32_t dtype,
                             const int32_t* drafts, const void* target, int64_t target_stride, const void* draft,
                             int64_t draft_stride, const float* temperature, const float* uniforms,
                             const float* noise, int64_t noise_stride, int32_t* accepted, int32_t* tokens,
                             void* stream) {
    const char* fn = "gdn_accept_drafts";
    gdn_status st;
    if (n_seq < 0 || n_seq > GDN_MAX_SEQUENCES)
        return set_error(GDN_ERR_INVALID_ARG, fn, "n_seq must be 0..GDN_MAX_SEQUENCES (%d) (got %d)",
                         GDN_MAX_SEQUENCES, n_seq);
    if (T < 0 || T > 16) return set_error(GDN_ERR_INVALID_ARG, fn, "T must be 0..16 (got %d)", T);
    if (vocab < 1) return set_error(GDN_ERR_INVALID_ARG, fn, "vocab must be >= 1 (got %d)", vocab);
    if (vocab > gdn::kMostVocab)
        return set_error(GDN_ERR_UNSUPPORTED, fn, "vocab %d is above %d", vocab, gdn::kMostVocab);
    if (form != GDN_DIST_PROBS && form != GDN_DIST_LOGITS)
        return set_error(GDN_ERR_INVALID_ARG, fn, "form %d is not a gdn_dist_form", form);
    if (dtype != GDN_DTYPE_F32 && dtype != GDN_DTYPE_BF16)
        return set_error(GDN_ERR_INVALID_ARG, fn, "dtype %d is not a gdn_dtype", dtype);
    if (form == GDN_DIST_PROBS && dtype != GDN_DTYPE_F32)
        return set_error(GDN_ERR_UNSUPPORTED, fn, "probabilities must be fp32");
    if (form == GDN_DIST_PROBS && temperature)
        return set_error(GDN_ERR_INVALID_ARG, fn, "temperature applies to logits only");
    if (target_stride < vocab || (draft && draft_stride < vocab) || noise_stride < vocab)
        return set_error(GDN_ERR_INVALID_ARG, fn, "a row stride is below vocab (%d)", vocab);
    gdn::clear_error();
    if (n_seq == 0) return GDN_OK;
    if (!target || !noise || !accepted || !tokens || (T > 0 && (!drafts || !uniforms)))
        return set_error(GDN_ERR_INVALID_ARG, fn, "an input or output pointer is NULL");
    const uintptr_t word = dtype == GDN_DTYPE_BF16 ? 1 : 3;
    if ((reinterpret_cast<uintptr_t>(target) & word) || (reinterpret_cast<uintptr_t>(draft) & word) ||
        (reinterpret_cast<uintptr_t>(noise) & 3))
        return set_error(GDN_ERR_INVALID_ARG, fn, "target, draft or noise is not aligned to its element size");
    if ((st = gdn::inject_fault("accept", fn)) != GDN_OK) return st;
    gdn::AcceptArgs a{};
    a.n_seq = n_seq; a.T = T; a.vocab = vocab; a.drafts = drafts; a.target = target; a.draft = T > 0 ? draft : nullptr;
    a.target_stride = target_stride; a.draft_stride = draft_stride; a.noise_stride = noise_stride;
    a.temperature = temperature; a.uniforms = uniforms; a.noise = noise; a.accepted = accepted; a.tokens = tokens;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return cuda_status(timed_launch("accept_drafts", s, [&] {
                           return gdn::launch_accept_drafts(a, form == GDN_DIST_LOGITS, dtype == GDN_DTYPE_BF16, s);
                       }), fn, "accept launch");
}

}  // extern "C"
