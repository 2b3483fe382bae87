// Launch interface of the latent cache, of both forms of its attention and of
// page copies (gdn_latent_api.cu validates, these launch).
#pragma once

#include "gdn_kv.h"

namespace gdn {

constexpr int kRopeDim = 64;  // channels of the position key

struct LatentCache {
    void* rows;  // bf16 [n_pages, B, C + kRopeDim]
    int n_pages;
};

struct LatentAppendArgs {
    LatentCache c;
    KvBatch b;
    int n_heads, page_size, rope_style;
    float eps;
    KvRows rows;               // [T, C + kRopeDim]
    const float* norm_w;       // [C] or null
    KvRows q, q_out;           // [T, n_heads, kRopeDim], data null without q
    const float* rope;         // [rope_len, kRopeDim] or null
    int rope_len;
    const int32_t* positions;  // [T] or null
    void* rows_out;            // [T, C + kRopeDim] or null
    int* error;                // cache_error_word
};

struct LatentReadArgs {
    LatentCache c;
    KvBatch b;  // kv_lens: the first positions
    int page_size;
    void* out;
    int* error;
};

struct LatentAttnArgs {
    LatentCache c;
    KvBatch b;
    const int32_t* cu_host;
    int n_heads, page_shift;  // a page has 1 << page_shift tokens
    float scale;
    KvRows q;  // [T, n_heads, C + kRopeDim]
    void* out;
    void* workspace;
    int* error;
    int stall;  // test hooks: 1 no cached row is ever loaded, 2 no scores are computed
};

struct ExpandedArgs {
    int n_seq, n_heads;
    float scale;
    const int32_t *cu_q, *cu_kv, *cu_q_host, *cu_kv_host;
    int n_q, n_kv;  // cu_q[n_seq], cu_kv[n_seq]
    KvRows q, k, k_rope, v;
    void* out;
    int* error;
    int stall;  // test hooks: 1 nothing is ever loaded, 2 no products are issued
};

cudaError_t launch_latent_append(const LatentAppendArgs& a, int latent_dim, cudaStream_t stream);
cudaError_t launch_latent_read(const LatentReadArgs& a, int latent_dim, cudaStream_t stream);
size_t latent_attention_workspace(int n_heads, int latent_dim, int n_seq, int max_q);
cudaError_t launch_latent_attention(const LatentAttnArgs& a, int latent_dim, cudaStream_t stream);
cudaError_t launch_expanded_attention(const ExpandedArgs& a, int nope_dim, int v_dim, cudaStream_t stream);
cudaError_t launch_copy_pages(void* const* bases, const size_t* page_bytes, int n_buffers, const int32_t* src,
                              const int32_t* dst, int n_pairs, cudaStream_t stream);

}  // namespace gdn
