// Causal attention of the expanded form: one row (query, head) a warp.
#include "gdn_internal.h"
#include "gdn_kv.cuh"
#include "gdn_latent.h"

namespace gdn {

namespace {

using bf16 = __nv_bfloat16;

template <int NOPE, int V>
__global__ void __launch_bounds__(128) expanded_kernel(const ExpandedArgs a) {
    constexpr int K = (NOPE + kRopeDim) / 32, KN = NOPE / 32, KV = V / 32;
    const int lane = threadIdx.x & 31;
    const long long row = static_cast<long long>(blockIdx.x) * 4 + (threadIdx.x >> 5);
    if (row >= static_cast<long long>(a.n_q) * a.n_heads) return;
    const int tok = static_cast<int>(row / a.n_heads), h = static_cast<int>(row % a.n_heads);
    const int seq = seq_of_token(a.cu_q, a.n_seq, tok);
    const int k0 = a.cu_kv[seq], end = (a.cu_kv[seq + 1] - k0) - (a.cu_q[seq + 1] - tok) + 1;
    const bf16* q = static_cast<const bf16*>(a.q.data) + tok * a.q.token_stride + h * a.q.head_stride;
    float x[K], o[KV];
#pragma unroll
    for (int i = 0; i < K; ++i) x[i] = to_f32(q[lane + 32 * i]);
#pragma unroll
    for (int i = 0; i < KV; ++i) o[i] = 0.0f;
    float m = -INFINITY, l = 0.0f;
    for (int j = 0; j < end; ++j) {
        const bf16* k = static_cast<const bf16*>(a.k.data) + (k0 + j) * a.k.token_stride + h * a.k.head_stride;
        const bf16* r = static_cast<const bf16*>(a.k_rope.data) + (k0 + j) * a.k_rope.token_stride;
        const bf16* v = static_cast<const bf16*>(a.v.data) + (k0 + j) * a.v.token_stride + h * a.v.head_stride;
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < K; ++i) s = fmaf(x[i], to_f32(i < KN ? k[lane + 32 * i] : r[lane + 32 * (i - KN)]), s);
        s = group_sum<32>(s) * a.scale;
        const float mn = fmaxf(m, s), f = m == -INFINITY ? 0.0f : expf(m - mn), p = expf(s - mn);
        m = mn;
        l = l * f + p;
#pragma unroll
        for (int i = 0; i < KV; ++i) o[i] = o[i] * f + p * to_f32(v[lane + 32 * i]);
    }
    const float inv = l > 0.0f ? 1.0f / l : (l == l ? 0.0f : l);
    bf16* out = static_cast<bf16*>(a.out) + row * V;
#pragma unroll
    for (int i = 0; i < KV; ++i) out[lane + 32 * i] = from_f32<bf16>(o[i] * inv);
}

template <int NOPE, int V>
cudaError_t expanded_t(const ExpandedArgs& a, cudaStream_t st) {
    const long long blocks = (static_cast<long long>(a.n_q) * a.n_heads + 3) / 4;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    return timed_launch("expanded_attention", st, [&] {
        expanded_kernel<NOPE, V><<<static_cast<unsigned>(blocks), 128, 0, st>>>(a);
        return cudaGetLastError();
    });
}

}  // namespace

cudaError_t launch_expanded_attention(const ExpandedArgs& a, int nope_dim, int v_dim, cudaStream_t st) {
    if (nope_dim == 128) return v_dim == 128 ? expanded_t<128, 128>(a, st) : expanded_t<128, 64>(a, st);
    return v_dim == 128 ? expanded_t<64, 128>(a, st) : expanded_t<64, 64>(a, st);
}

}  // namespace gdn
