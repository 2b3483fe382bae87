// C-ABI entry points of the latent cache, of both forms of its attention and of
// page copies (declared in include/gdn.h): host-side validation, error
// reporting and dispatch on the caller's stream.
#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdlib>
#include <memory>

#include "gdn.h"
#include "gdn_internal.h"
#include "gdn_latent.h"
#include "gdn_memory.h"

namespace gdn {
// Records the thread's error message (defined with the other entry points).
gdn_status set_error(gdn_status st, const char* fn, const char* fmt, ...);
gdn_status cuda_status(cudaError_t e, const char* fn, const char* what);  // GDN_OK, or GDN_ERR_CUDA recorded
void clear_error();
// GDN_ERR_INJECTED when the environment variable GDN_FAULT lists `site`.
gdn_status inject_fault(const char* site, const char* fn);
bool fault_site(const char* site);  // whether it does
}  // namespace gdn

using gdn::aligned16;
using gdn::cuda_status;
using gdn::Memory;
using gdn::set_error;
using gdn::timed_launch;

namespace {

gdn_status check_dims(const gdn_latent_dims* d, const char* fn) {
    if (!d) return set_error(GDN_ERR_INVALID_ARG, fn, "dims is NULL");
    if (d->n_heads < 1) return set_error(GDN_ERR_INVALID_ARG, fn, "n_heads must be >= 1 (got %d)", d->n_heads);
    if (d->n_heads > 1024) return set_error(GDN_ERR_UNSUPPORTED, fn, "n_heads %d is above 1024", d->n_heads);
    if (d->latent_dim != 256 && d->latent_dim != 512)
        return set_error(GDN_ERR_UNSUPPORTED, fn, "latent_dim must be 256 or 512 (got %d)", d->latent_dim);
    if (d->rope_dim != gdn::kRopeDim)
        return set_error(GDN_ERR_UNSUPPORTED, fn, "rope_dim must be %d (got %d)", gdn::kRopeDim, d->rope_dim);
    if (d->page_size != 16 && d->page_size != 32 && d->page_size != 64 && d->page_size != 128)
        return set_error(GDN_ERR_UNSUPPORTED, fn, "page_size must be 16, 32, 64 or 128 (got %d)", d->page_size);
    if (d->rope_style != GDN_ROPE_HALF && d->rope_style != GDN_ROPE_INTERLEAVED)
        return set_error(GDN_ERR_INVALID_ARG, fn, "rope_style %d is not a gdn_rope_style", d->rope_style);
    if ((d->nope_dim != 64 && d->nope_dim != 128) || (d->v_dim != 64 && d->v_dim != 128))
        return set_error(GDN_ERR_UNSUPPORTED, fn, "nope_dim and v_dim must be 64 or 128 (got %d, %d)", d->nope_dim, d->v_dim);
    if (!(d->scale > 0.f) || !std::isfinite(d->scale * 1.4426950408889634f))  // the kernels' scale: they take powers of two
        return set_error(GDN_ERR_INVALID_ARG, fn, "scale must be finite, times log2 e too, and > 0");
    if (!(d->norm_eps >= 0.f) || !std::isfinite(d->norm_eps))
        return set_error(GDN_ERR_INVALID_ARG, fn, "norm_eps must be finite and >= 0");
    return GDN_OK;
}

gdn_status check_cache(const gdn_latent_cache* c, const gdn_latent_dims* d, const char* fn) {
    if (!c) return set_error(GDN_ERR_INVALID_ARG, fn, "cache is NULL");
    if (c->n_pages < 0) return set_error(GDN_ERR_INVALID_ARG, fn, "n_pages must be >= 0 (got %d)", c->n_pages);
    if (c->n_pages > 0 && !c->rows) return set_error(GDN_ERR_INVALID_ARG, fn, "the cache's pointer is NULL");
    if (static_cast<long long>(c->n_pages) * d->page_size > 0x7fffffff)
        return set_error(GDN_ERR_UNSUPPORTED, fn, "%d pages of %d rows are more than 2^31 - 1", c->n_pages, d->page_size);
    if (!aligned16(c->rows)) return set_error(GDN_ERR_INVALID_ARG, fn, "the cache's rows must be 16-byte aligned");
    return GDN_OK;
}

// Validates the host copy of a cu_seqlens.
gdn_status check_cu(int32_t n_seq, const int32_t* cu_host, const char* name, const char* fn) {
    if (n_seq < 0) return set_error(GDN_ERR_INVALID_ARG, fn, "n_seq must be >= 0 (got %d)", n_seq);
    if (n_seq > GDN_MAX_SEQUENCES)
        return set_error(GDN_ERR_UNSUPPORTED, fn, "n_seq %d is above GDN_MAX_SEQUENCES (%d)", n_seq, GDN_MAX_SEQUENCES);
    if (n_seq == 0) return GDN_OK;
    if (!cu_host) return set_error(GDN_ERR_INVALID_ARG, fn, "%s pointer is NULL", name);
    if (cu_host[0] != 0) return set_error(GDN_ERR_INVALID_ARG, fn, "%s[0] must be 0", name);
    for (int i = 0; i < n_seq; ++i)
        if (cu_host[i + 1] < cu_host[i])
            return set_error(GDN_ERR_INVALID_ARG, fn, "%s decreases at index %d", name, i + 1);
    return GDN_OK;
}

// The longest sequence, and every sequence's tokens where they are all alike (else 0).
void spread(const int32_t* cu, int32_t n_seq, int* longest, int* uniform) {
    int lo = cu[1], hi = cu[1];
    for (int i = 1; i < n_seq; ++i) {
        const int q = cu[i + 1] - cu[i];
        lo = q < lo ? q : lo;
        hi = q > hi ? q : hi;
    }
    *longest = hi;
    *uniform = lo == hi ? hi : 0;
}

gdn_status check_batch(const gdn_kv_batch* b, const int32_t* lens, gdn::KvBatch* out, const char* fn) {
    if (!b) return set_error(GDN_ERR_INVALID_ARG, fn, "batch is NULL");
    gdn_status st = check_cu(b->n_seq, b->cu_seqlens_host, "cu_seqlens", fn);
    if (st != GDN_OK) return st;
    *out = gdn::KvBatch{};
    if (b->n_seq == 0) return GDN_OK;
    out->n_seq = b->n_seq;
    out->n_tokens = b->cu_seqlens_host[b->n_seq];
    if (out->n_tokens == 0) return GDN_OK;
    if (b->pages_per_seq < 0) return set_error(GDN_ERR_INVALID_ARG, fn, "pages_per_seq must be >= 0");
    if (!b->cu_seqlens || !lens || (b->pages_per_seq > 0 && !b->block_table))
        return set_error(GDN_ERR_INVALID_ARG, fn, "cu_seqlens, the lengths or block_table is NULL");
    out->pages_per_seq = b->pages_per_seq;
    out->cu = b->cu_seqlens;
    out->kv_lens = lens;
    out->table = b->block_table;
    spread(b->cu_seqlens_host, b->n_seq, &out->max_q, &out->uniform_q);
    return GDN_OK;
}

gdn_status check_rows(const gdn_rows* r, const char* name, gdn::KvRows* out, const char* fn) {
    if (!r || !r->data) return set_error(GDN_ERR_INVALID_ARG, fn, "%s is NULL", name);
    if (r->token_stride < 0 || r->head_stride < 0)
        return set_error(GDN_ERR_INVALID_ARG, fn, "%s has a negative stride", name);
    if (!aligned16(r->data) || r->token_stride % 8 != 0 || r->head_stride % 8 != 0)
        return set_error(GDN_ERR_INVALID_ARG, fn, "%s: the base and both strides must be multiples of 16 bytes", name);
    *out = gdn::KvRows{r->data, r->token_stride, r->head_stride};
    return GDN_OK;
}

int stall(const char* loads, const char* products) { return gdn::fault_site(loads) ? 1 : gdn::fault_site(products) ? 2 : 0; }

// Whether rows that are written may overlap: false where one axis' rows lie apart and
// the other one steps over all of them.
bool rows_overlap(const gdn::KvRows& r, long long tokens, long long heads, long long width) {
    const long long ts = tokens > 1 ? r.token_stride : LLONG_MAX, hs = heads > 1 ? r.head_stride : LLONG_MAX;
    if (ts < width || hs < width) return true;
    if (tokens == 1 || heads == 1) return false;
    return (ts - width) / (heads - 1) < hs && (hs - width) / (tokens - 1) < ts;
}

Memory memory(const gdn::KvRows& r, long long tokens, long long heads, long long channels) {
    return Memory::rows(r.data, tokens, heads, r.token_stride, r.head_stride, channels, 2);
}

}  // namespace

extern "C" {

gdn_status gdn_latent_append(const gdn_latent_dims* dims, const gdn_latent_cache* cache, const gdn_kv_batch* batch,
                             const int32_t* kv_lens, const gdn_rows* c, const float* norm_w, const gdn_rows* q_rope,
                             const gdn_rows* q_out, const float* rope, int32_t rope_len, const int32_t* positions,
                             void* rows_out, void* stream) {
    const char* fn = "gdn_latent_append";
    gdn_status st;
    gdn::LatentAppendArgs a{};
    if ((st = check_dims(dims, fn)) != GDN_OK) return st;
    if ((st = check_cache(cache, dims, fn)) != GDN_OK) return st;
    if ((st = check_batch(batch, kv_lens, &a.b, fn)) != GDN_OK) return st;
    gdn::clear_error();
    if (a.b.n_tokens == 0) return GDN_OK;
    gdn_rows r{};
    if (c) r = gdn_rows{c->data, c->token_stride, 0};
    if ((st = check_rows(&r, "c", &a.rows, fn)) != GDN_OK) return st;
    if (norm_w && !aligned16(norm_w)) return set_error(GDN_ERR_INVALID_ARG, fn, "norm_w must be 16-byte aligned");
    if (q_out && !q_rope) return set_error(GDN_ERR_INVALID_ARG, fn, "q_out is given without q_rope");
    if (q_rope) {
        if (static_cast<long long>(a.b.n_tokens) * dims->n_heads > 0x7fffff00)
            return set_error(GDN_ERR_UNSUPPORTED, fn, "%d tokens of %d heads are more than 2^31 - 256 rows", a.b.n_tokens, dims->n_heads);
        if ((st = check_rows(q_rope, "q_rope", &a.q, fn)) != GDN_OK) return st;
        if ((st = check_rows(q_out, "q_out", &a.q_out, fn)) != GDN_OK) return st;
        if (rows_overlap(a.q_out, a.b.n_tokens, dims->n_heads, dims->rope_dim))
            return set_error(GDN_ERR_INVALID_ARG, fn, "q_out's rows overlap, or its tokens and heads interleave");
    }
    if (rope && (rope_len < 1 || !aligned16(rope)))
        return set_error(GDN_ERR_INVALID_ARG, fn, "rope must hold at least one row and be 16-byte aligned");
    if (rows_out && !aligned16(rows_out)) return set_error(GDN_ERR_INVALID_ARG, fn, "rows_out must be 16-byte aligned");
    // what is written while other warps still read: the same rows, or memory of its own
    const long long tokens = a.b.n_tokens, width = dims->latent_dim + dims->rope_dim;
    const Memory in_q = memory(a.q, tokens, dims->n_heads, dims->rope_dim), to_q = memory(a.q_out, tokens, dims->n_heads, dims->rope_dim);
    if (q_rope && !gdn::same(in_q, to_q) && gdn::meet(in_q, to_q))
        return set_error(GDN_ERR_INVALID_ARG, fn, "q_out shares memory with q_rope and is not the same rows");
    if (rows_out) {
        const Memory packed = Memory::array(rows_out, 2 * tokens * width);
        const bool in_place = rows_out == a.rows.data && (tokens == 1 || a.rows.token_stride == width);
        if (!in_place && gdn::meet(packed, memory(a.rows, tokens, 1, width)))
            return set_error(GDN_ERR_INVALID_ARG, fn, "rows_out shares memory with c and is not the same rows");
        if (gdn::meet(packed, Memory::array(cache->rows, 2ll * cache->n_pages * dims->page_size * width)) ||
            (q_rope && (gdn::meet(packed, in_q) || gdn::meet(packed, to_q))))
            return set_error(GDN_ERR_INVALID_ARG, fn, "rows_out shares memory with the cache, q_rope or q_out");
    }
    if ((st = gdn::inject_fault("latent_append", fn)) != GDN_OK) return st;
    if ((st = cuda_status(gdn::cache_error_word(&a.error), fn, "finding the error word")) != GDN_OK) return st;
    a.c = gdn::LatentCache{cache->rows, cache->n_pages};
    a.n_heads = dims->n_heads; a.page_size = dims->page_size; a.rope_style = dims->rope_style; a.eps = dims->norm_eps;
    a.norm_w = norm_w; a.rope = rope; a.rope_len = rope_len; a.positions = positions; a.rows_out = rows_out;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return cuda_status(timed_launch("latent_append", s, [&] { return gdn::launch_latent_append(a, dims->latent_dim, s); }), fn,
                       "append launch");
}

gdn_status gdn_latent_read(const gdn_latent_dims* dims, const gdn_latent_cache* cache, const gdn_kv_batch* batch,
                           const int32_t* starts, void* out, void* stream) {
    const char* fn = "gdn_latent_read";
    gdn_status st;
    gdn::LatentReadArgs a{};
    if ((st = check_dims(dims, fn)) != GDN_OK) return st;
    if ((st = check_cache(cache, dims, fn)) != GDN_OK) return st;
    if ((st = check_batch(batch, starts, &a.b, fn)) != GDN_OK) return st;
    gdn::clear_error();
    if (a.b.n_tokens == 0) return GDN_OK;
    if (!out || !aligned16(out)) return set_error(GDN_ERR_INVALID_ARG, fn, "out must be given and 16-byte aligned");
    if ((st = gdn::inject_fault("latent_read", fn)) != GDN_OK) return st;
    if ((st = cuda_status(gdn::cache_error_word(&a.error), fn, "finding the error word")) != GDN_OK) return st;
    a.c = gdn::LatentCache{cache->rows, cache->n_pages};
    a.page_size = dims->page_size; a.out = out;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return cuda_status(timed_launch("latent_read", s, [&] { return gdn::launch_latent_read(a, dims->latent_dim, s); }), fn,
                       "read launch");
}

gdn_status gdn_latent_attention_workspace_size(const gdn_latent_dims* dims, int32_t n_seq, const int32_t* cu_seqlens_host,
                                               size_t* bytes) {
    const char* fn = "gdn_latent_attention_workspace_size";
    gdn_status st;
    if ((st = check_dims(dims, fn)) != GDN_OK) return st;
    if (!bytes) return set_error(GDN_ERR_INVALID_ARG, fn, "bytes is NULL");
    if ((st = check_cu(n_seq, cu_seqlens_host, "cu_seqlens", fn)) != GDN_OK) return st;
    int longest = 0, uniform;
    if (n_seq > 0) spread(cu_seqlens_host, n_seq, &longest, &uniform);
    *bytes = gdn::latent_attention_workspace(dims->n_heads, dims->latent_dim, n_seq, longest);
    gdn::clear_error();
    return GDN_OK;
}

gdn_status gdn_latent_attention(const gdn_latent_dims* dims, const gdn_latent_cache* cache, const gdn_kv_batch* batch,
                                const int32_t* kv_lens, const gdn_rows* q, void* out, void* workspace,
                                size_t workspace_bytes, void* stream) {
    const char* fn = "gdn_latent_attention";
    gdn_status st;
    gdn::LatentAttnArgs a{};
    if ((st = check_dims(dims, fn)) != GDN_OK) return st;
    if ((st = check_cache(cache, dims, fn)) != GDN_OK) return st;
    if ((st = check_batch(batch, kv_lens, &a.b, fn)) != GDN_OK) return st;
    gdn::clear_error();
    if (a.b.n_tokens == 0) return GDN_OK;
    if (static_cast<long long>(a.b.n_tokens) * dims->n_heads > 0x7fffff00)
        return set_error(GDN_ERR_UNSUPPORTED, fn, "%d tokens of %d heads are more than 2^31 - 256 rows", a.b.n_tokens, dims->n_heads);
    if ((st = check_rows(q, "q", &a.q, fn)) != GDN_OK) return st;
    if (!out || !aligned16(out)) return set_error(GDN_ERR_INVALID_ARG, fn, "out must be given and 16-byte aligned");
    const size_t need = gdn::latent_attention_workspace(dims->n_heads, dims->latent_dim, a.b.n_seq, a.b.max_q);
    if (need > 0 && (!workspace || workspace_bytes < need))
        return set_error(GDN_ERR_WORKSPACE, fn, "workspace of %zu bytes needed, %zu given", need,
                         workspace ? workspace_bytes : (size_t)0);
    if (need > 0 && (reinterpret_cast<uintptr_t>(workspace) & 255u))
        return set_error(GDN_ERR_WORKSPACE, fn, "workspace must be 256-byte aligned");
    if ((st = gdn::inject_fault("latent_attention", fn)) != GDN_OK) return st;
    if ((st = cuda_status(gdn::cache_error_word(&a.error), fn, "finding the error word")) != GDN_OK) return st;
    a.c = gdn::LatentCache{cache->rows, cache->n_pages};
    a.cu_host = batch->cu_seqlens_host;
    a.n_heads = dims->n_heads; a.scale = dims->scale; a.out = out; a.workspace = workspace;
    while (1 << a.page_shift < dims->page_size) ++a.page_shift;
    a.stall = stall("stall_latent", "stall_latent_products");
    return cuda_status(gdn::launch_latent_attention(a, dims->latent_dim, static_cast<cudaStream_t>(stream)), fn,
                       "attention launch");
}

gdn_status gdn_expanded_attention(const gdn_latent_dims* dims, int32_t n_seq, const int32_t* cu_q, const int32_t* cu_q_host,
                                  const int32_t* cu_kv, const int32_t* cu_kv_host, const gdn_rows* q, const gdn_rows* k,
                                  const gdn_rows* k_rope, const gdn_rows* v, void* out, void* stream) {
    const char* fn = "gdn_expanded_attention";
    gdn_status st;
    gdn::ExpandedArgs a{};
    if ((st = check_dims(dims, fn)) != GDN_OK) return st;
    if ((st = check_cu(n_seq, cu_q_host, "cu_q", fn)) != GDN_OK) return st;
    if ((st = check_cu(n_seq, cu_kv_host, "cu_kv", fn)) != GDN_OK) return st;
    gdn::clear_error();
    if (n_seq == 0 || cu_q_host[n_seq] == 0) return GDN_OK;
    a.n_seq = n_seq; a.n_q = cu_q_host[n_seq]; a.n_kv = cu_kv_host[n_seq];
    int longest, uniform;
    spread(cu_q_host, n_seq, &longest, &uniform);
    if (longest > 1 << 24) return set_error(GDN_ERR_UNSUPPORTED, fn, "a sequence has %d queries, more than 2^24", longest);
    if (a.n_kv > 1 << 30) return set_error(GDN_ERR_UNSUPPORTED, fn, "%d keys are more than 2^30", a.n_kv);
    if (!cu_q || !cu_kv) return set_error(GDN_ERR_INVALID_ARG, fn, "cu_q or cu_kv is NULL");
    if ((st = check_rows(q, "q", &a.q, fn)) != GDN_OK) return st;
    if (a.n_kv > 0) {  // without keys nothing of them is looked at
        gdn_rows r{};
        if (k_rope) r = gdn_rows{k_rope->data, k_rope->token_stride, 0};
        if ((st = check_rows(k, "k", &a.k, fn)) != GDN_OK) return st;
        if ((st = check_rows(&r, "k_rope", &a.k_rope, fn)) != GDN_OK) return st;
        if ((st = check_rows(v, "v", &a.v, fn)) != GDN_OK) return st;
    }
    const gdn::KvRows* rows[4] = {&a.q, &a.k, &a.k_rope, &a.v};
    static const char* const names[4] = {"q", "k", "k_rope", "v"};
    for (int i = 0; i < (a.n_kv > 0 ? 4 : 1); ++i)
        if (rows[i]->token_stride < 1 || rows[i]->token_stride >= 1ll << 36 || rows[i]->head_stride >= 1ll << 36)
            return set_error(GDN_ERR_INVALID_ARG, fn, "%s: strides must be below 2^36, the token stride above 0", names[i]);
    if (!out || !aligned16(out)) return set_error(GDN_ERR_INVALID_ARG, fn, "out must be given and 16-byte aligned");
    if ((st = gdn::inject_fault("expanded_attention", fn)) != GDN_OK) return st;
    if ((st = cuda_status(gdn::cache_error_word(&a.error), fn, "finding the error word")) != GDN_OK) return st;
    a.n_heads = dims->n_heads; a.scale = dims->scale; a.cu_q = cu_q; a.cu_kv = cu_kv; a.out = out;
    a.cu_q_host = cu_q_host; a.cu_kv_host = cu_kv_host;
    a.stall = stall("stall_expanded", "stall_expanded_products");
    return cuda_status(gdn::launch_expanded_attention(a, dims->nope_dim, dims->v_dim, static_cast<cudaStream_t>(stream)), fn,
                       "attention launch");
}

gdn_status gdn_copy_pages(int32_t n_buffers, void* const* bases, const size_t* page_bytes, int32_t n_pages, int32_t n_pairs,
                          const int32_t* src, const int32_t* dst, void* stream) {
    const char* fn = "gdn_copy_pages";
    gdn_status st;
    if (n_buffers < 0 || n_pages < 0 || n_pairs < 0)
        return set_error(GDN_ERR_INVALID_ARG, fn, "n_buffers, n_pages and n_pairs must be >= 0");
    gdn::clear_error();
    if (n_buffers == 0 || n_pairs == 0) return GDN_OK;
    if (!bases || !page_bytes || !src || !dst) return set_error(GDN_ERR_INVALID_ARG, fn, "a list is NULL");
    for (int b = 0; b < n_buffers; ++b) {
        if (!bases[b] || (reinterpret_cast<uintptr_t>(bases[b]) & 3u) || page_bytes[b] == 0 || page_bytes[b] % 4 != 0)
            return set_error(GDN_ERR_INVALID_ARG, fn, "array %d: NULL, or its base or page_bytes is no multiple of 4", b);
        if (page_bytes[b] > 1u << 30) return set_error(GDN_ERR_UNSUPPORTED, fn, "array %d: pages above 2^30 bytes", b);
    }
    struct Free { void operator()(void* p) const { std::free(p); } };
    // arrays side by side: a page of one that is written is no page of another
    struct Range { uintptr_t begin, end; };
    std::unique_ptr<Range, Free> ranges(static_cast<Range*>(std::malloc(n_buffers * sizeof(Range))));
    if (!ranges) return set_error(GDN_ERR_WORKSPACE, fn, "no host memory for %d arrays", n_buffers);
    Range* const r = ranges.get();
    for (int b = 0; b < n_buffers; ++b) {
        const uintptr_t at = reinterpret_cast<uintptr_t>(bases[b]);
        r[b] = Range{at, at + static_cast<size_t>(n_pages) * page_bytes[b]};
    }
    std::sort(r, r + n_buffers, [](const Range& x, const Range& y) { return x.begin < y.begin; });
    for (int b = 1; b < n_buffers; ++b)
        if (r[b].begin < r[b - 1].end) return set_error(GDN_ERR_INVALID_ARG, fn, "two arrays overlap");
    // one bit a page: the pages that are written (zeroed memory is taken as it is touched)
    std::unique_ptr<uint32_t, Free> written(static_cast<uint32_t*>(std::calloc(static_cast<size_t>(n_pages) / 32 + 1, 4)));
    if (!written) return set_error(GDN_ERR_WORKSPACE, fn, "no host memory for %d pages", n_pages);
    for (int i = 0; i < n_pairs; ++i) {
        if (src[i] < 0 || src[i] >= n_pages || dst[i] < 0 || dst[i] >= n_pages)
            return set_error(GDN_ERR_INVALID_ARG, fn, "pair %d: pages %d, %d are not in 0..%d", i, src[i], dst[i], n_pages - 1);
        uint32_t& word = written.get()[dst[i] / 32];
        if (word >> (dst[i] % 32) & 1u) return set_error(GDN_ERR_INVALID_ARG, fn, "page %d is written twice", dst[i]);
        word |= 1u << (dst[i] % 32);
    }
    for (int i = 0; i < n_pairs; ++i)
        if (written.get()[src[i] / 32] >> (src[i] % 32) & 1u)
            return set_error(GDN_ERR_INVALID_ARG, fn, "page %d is both read and written", src[i]);
    if ((st = gdn::inject_fault("copy_pages", fn)) != GDN_OK) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return cuda_status(timed_launch("copy_pages", s, [&] {
                           return gdn::launch_copy_pages(bases, page_bytes, n_buffers, src, dst, n_pairs, s);
                       }), fn, "copy launch");
}

}  // extern "C"
