// Attention over the latent cache, absorbed form: one row (token, head) a warp.
#include "gdn_internal.h"
#include "gdn_kv.cuh"
#include "gdn_latent.h"

namespace gdn {

namespace {

using bf16 = __nv_bfloat16;

template <int C>
__global__ void __launch_bounds__(128) latent_attention_kernel(const LatentAttnArgs a) {
    constexpr int W = C + kRopeDim, K = W / 32;
    const int lane = threadIdx.x & 31;
    const long long row = static_cast<long long>(blockIdx.x) * 4 + (threadIdx.x >> 5);
    if (row >= static_cast<long long>(a.b.n_tokens) * a.n_heads) return;
    const int tok = static_cast<int>(row / a.n_heads), h = static_cast<int>(row % a.n_heads);
    const int seq = seq_of_token(a.b.cu, a.b.n_seq, tok);
    const long long cap = static_cast<long long>(a.b.pages_per_seq) * a.page_size;
    long long end = static_cast<long long>(a.b.kv_lens[seq]) - (a.b.cu[seq + 1] - tok) + 1;
    if (a.b.kv_lens[seq] > cap) {
        if (lane == 0) atomicMax(a.error, kKvErrTable);
        end = min(end, cap);
    }
    const bf16* q = static_cast<const bf16*>(a.q.data) + tok * a.q.token_stride + h * a.q.head_stride;
    float x[K], o[C / 32];
#pragma unroll
    for (int i = 0; i < K; ++i) x[i] = to_f32(q[lane + 32 * i]);
#pragma unroll
    for (int i = 0; i < C / 32; ++i) o[i] = 0.0f;
    float m = -INFINITY, l = 0.0f;
    for (long long j = 0; j < end; ++j) {
        const int page = a.b.table[static_cast<size_t>(seq) * a.b.pages_per_seq + j / a.page_size];
        if (page < 0 || page >= a.c.n_pages) {
            if (lane == 0) atomicMax(a.error, kKvErrTable);
            continue;
        }
        const bf16* r = static_cast<const bf16*>(a.c.rows) + (static_cast<size_t>(page) * a.page_size + j % a.page_size) * W;
        float v[K], s = 0.0f;
#pragma unroll
        for (int i = 0; i < K; ++i) {
            v[i] = to_f32(r[lane + 32 * i]);
            s = fmaf(x[i], v[i], s);
        }
        s = group_sum<32>(s) * a.scale;
        const float mn = fmaxf(m, s), f = m == -INFINITY ? 0.0f : expf(m - mn), p = expf(s - mn);
        m = mn;
        l = l * f + p;
#pragma unroll
        for (int i = 0; i < C / 32; ++i) o[i] = o[i] * f + p * v[i];
    }
    const float inv = l > 0.0f ? 1.0f / l : (l == l ? 0.0f : l);
    bf16* out = static_cast<bf16*>(a.out) + row * C;
#pragma unroll
    for (int i = 0; i < C / 32; ++i) out[lane + 32 * i] = from_f32<bf16>(o[i] * inv);
}

}  // namespace

size_t latent_attention_workspace(int, int, int, int) { return 0; }

cudaError_t launch_latent_attention(const LatentAttnArgs& a, int latent_dim, cudaStream_t st) {
    const long long blocks = (static_cast<long long>(a.b.n_tokens) * a.n_heads + 3) / 4;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    if (latent_dim == 512) latent_attention_kernel<512><<<static_cast<unsigned>(blocks), 128, 0, st>>>(a);
    else latent_attention_kernel<256><<<static_cast<unsigned>(blocks), 128, 0, st>>>(a);
    return cudaGetLastError();
}

}  // namespace gdn
