// Launch interface of the paged 8-bit cache operators and of draft
// verification (gdn_kv_api.cu validates, these launch).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace gdn {

// Device error codes of the cache operators (not waits).
constexpr int kKvErrTable = 40;  // block table entry or length out of range
constexpr int kKvErrRope = 41;   // position outside the rotation table
// The word on the current device where the operators' kernels record codes: the
// largest stays, so that a wait that gave up (42..66) outranks data out of range.
cudaError_t cache_error_word(int** word);

struct KvCache {
    uint8_t* k;      // codes [n_pages, Hkv, B, D]
    uint8_t* v;
    float* k_scale;  // [n_pages, Hkv]
    float* v_scale;
    int n_pages;
};

// Rows [T, heads, D]: channels contiguous, strides in elements.
struct KvRows {
    const void* data;
    long long token_stride, head_stride;
};

struct KvBatch {
    int n_seq, pages_per_seq;
    const int32_t* cu;       // [n_seq+1]
    const int32_t* kv_lens;  // [n_seq] (gdn_kv_read: the first positions)
    const int32_t* table;    // [n_seq, pages_per_seq]
    int n_tokens;            // cu[n_seq]
    int max_q;               // longest sequence of the call
    int uniform_q;           // every sequence's tokens where they are all alike, else 0
};

struct KvAppendArgs {
    KvCache c;
    KvBatch b;
    int n_q_heads, n_kv_heads, page_size, rope_dim, rope_style;
    KvRows q, k, v;             // q.data may be null
    const float* rope;          // [rope_len, rope_dim]
    int rope_len;
    const int32_t* positions;   // [T] or null
    void* q_out;
    int* error;                 // cache_error_word
};

struct KvReadArgs {
    KvCache c;
    KvBatch b;
    int n_kv_heads, page_size;
    void *k_out, *v_out;
    int* error;
};

struct KvAttnArgs {
    KvCache c;
    KvBatch b;
    int n_q_heads, n_kv_heads, page_size, window;
    float scale;
    KvRows q;
    void* out;
    float* partial;   // split partials (workspace), see gdn_kv_attn.cu
    int max_kv_len;
    int* error;
    int stall;        // test hook: the kernel for many rows waits for look-ups that never come
};

// The largest vocabulary: the kernel's strides go past a row's end, in 32 bits.
constexpr int kMostVocab = 0x7fffffff - 4096;
struct AcceptArgs {
    int n_seq, T, vocab;
    const int32_t* drafts;
    const void* target;
    const void* draft;  // or null
    long long target_stride, draft_stride, noise_stride;
    const float *temperature, *uniforms, *noise;
    int32_t *accepted, *tokens;
};

cudaError_t launch_kv_append(const KvAppendArgs& a, int head_dim, bool bf16, bool e4m3,
                             cudaStream_t stream);
cudaError_t launch_kv_read(const KvReadArgs& a, int head_dim, bool bf16, bool e4m3,
                           cudaStream_t stream);
size_t kv_attention_workspace(int n_seq, int max_q, int n_q_heads, int n_kv_heads, int head_dim, int window,
                              bool bf16, int max_kv_len);
// Keys split into n ranges of `chunk`; the last takes what is left.
struct KvSplit {
    int n, chunk;
};
// How the kernel for many rows (gdn_kv_prompt.cu) takes a call: thread blocks
// of `rows` rows, tiles of a sequence and head (0: it does not take the call).
struct KvPrompt {
    int tiles, rows;
    KvSplit split;
};
KvPrompt kv_prompt_plan(int n_seq, int max_q, int n_q_heads, int n_kv_heads, int head_dim, int window, bool bf16,
                        long long max_kv_len);
cudaError_t launch_kv_prompt(const KvAttnArgs& a, const KvPrompt& c, int head_dim, bool e4m3, cudaStream_t stream);
// Joins partial results [seq][kv head][tile][split] of rows x D outputs, then
// rows references and rows sums (bf16 activations).
cudaError_t launch_kv_join(const KvAttnArgs& a, const KvSplit& split, int rows, int tiles, int head_dim,
                           cudaStream_t stream);
cudaError_t launch_kv_attention(const KvAttnArgs& a, int head_dim, bool bf16, bool e4m3,
                                cudaStream_t stream);
// form: gdn_dist_form; logits and probabilities in bf16 or f32.
cudaError_t launch_accept_drafts(const AcceptArgs& a, bool logits, bool bf16, cudaStream_t stream);

}  // namespace gdn
