// Causal attention over the paged 8-bit cache.
//
// kv_attn_rows: one thread block per (token, query head); each of its warps
// walks every fourth key with a running maximum and sum, and the warps'
// results are joined at the end.
#include <algorithm>
#include <climits>

#include "gdn_internal.h"
#include "gdn_kv.cuh"

namespace gdn {

namespace {

__device__ int g_kv_attn_error = 0;

constexpr int kRowWarps = 4;

template <typename T, typename F, int D>
__global__ void __launch_bounds__(32 * kRowWarps) kv_attn_rows_kernel(const KvAttnArgs a) {
    constexpr int E = D / 32;  // channels of a lane: lane + 32 e
    const int tok = blockIdx.x, hq = blockIdx.y, h = hq / (a.n_q_heads / a.n_kv_heads);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int seq = a.b.uniform_q ? tok / a.b.uniform_q : seq_of_token(a.b.cu, a.b.n_seq, tok);
    const long long cap = static_cast<long long>(a.b.pages_per_seq) * a.page_size;
    int len = a.b.kv_lens[seq];
    const int pos = len - (a.b.cu[seq + 1] - tok);
    if (len > cap) {
        if (threadIdx.x == 0) atomicCAS(&g_kv_attn_error, 0, kKvErrTable);
        len = static_cast<int>(cap);
    }
    const int last = min(pos, len - 1), first = a.window ? max(0, pos - a.window + 1) : 0;
    const T* q = static_cast<const T*>(a.q.data) + tok * a.q.token_stride + hq * a.q.head_stride;
    float qr[E], o[E] = {};
#pragma unroll
    for (int e = 0; e < E; ++e) qr[e] = to_f32(q[lane + 32 * e]);
    float m = -INFINITY, l = 0.0f;
    for (int j = first + warp; j <= last; j += kRowWarps) {
        const int page = a.b.table[static_cast<size_t>(seq) * a.b.pages_per_seq + j / a.page_size];
        if (page < 0 || page >= a.c.n_pages) {
            if (lane == 0) atomicCAS(&g_kv_attn_error, 0, kKvErrTable);
            continue;
        }
        const size_t block = static_cast<size_t>(page) * a.n_kv_heads + h;
        const size_t at = (block * a.page_size + j % a.page_size) * D;
        float s = 0.0f;
#pragma unroll
        for (int e = 0; e < E; ++e) s += qr[e] * F::value(a.c.k[at + lane + 32 * e]);
        s = group_sum<32>(s) * (a.c.k_scale[block] * a.scale);
        const float mn = fmaxf(m, s), c = expf(m - mn), p = expf(s - mn);
        const float pv = p * a.c.v_scale[block];
        l = l * c + p;
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = o[e] * c + pv * F::value(a.c.v[at + lane + 32 * e]);
        m = mn;
    }
    __shared__ float sm[kRowWarps], sl[kRowWarps], so[kRowWarps][D];
    if (lane == 0) {
        sm[warp] = m;
        sl[warp] = l;
    }
#pragma unroll
    for (int e = 0; e < E; ++e) so[warp][lane + 32 * e] = o[e];
    __syncthreads();
    float mm = -INFINITY, ll = 0.0f;
    for (int w = 0; w < kRowWarps; ++w) mm = fmaxf(mm, sm[w]);
    for (int w = 0; w < kRowWarps; ++w) ll += sl[w] == 0.0f ? 0.0f : sl[w] * expf(sm[w] - mm);
    T* out = static_cast<T*>(a.out) + (static_cast<size_t>(tok) * a.n_q_heads + hq) * D;
    for (int d = threadIdx.x; d < D; d += 32 * kRowWarps) {
        float x = 0.0f;
        for (int w = 0; w < kRowWarps; ++w) x += sl[w] == 0.0f ? 0.0f : so[w][d] * expf(sm[w] - mm);
        out[d] = from_f32<T>(ll > 0.0f ? x / ll : 0.0f);
    }
}

template <typename T, typename F, int D>
cudaError_t attn_t(const KvAttnArgs& a, cudaStream_t st) {
    kv_attn_rows_kernel<T, F, D>
        <<<dim3(a.b.n_tokens, a.n_q_heads), 32 * kRowWarps, 0, st>>>(a);
    return cudaGetLastError();
}

}  // namespace

size_t kv_attention_workspace(int, const int32_t*, int, int, int, bool, int) { return 0; }

cudaError_t launch_kv_attention(const KvAttnArgs& a, int head_dim, bool bf16, bool e4m3, cudaStream_t stream) {
    return GDN_KV_PICK(attn_t);
}

cudaError_t read_kv_attn_error(int* code, bool reset) {
    cudaError_t e = cudaMemcpyFromSymbol(code, g_kv_attn_error, sizeof(int));
    if (e == cudaSuccess && reset) {
        const int zero = 0;
        e = cudaMemcpyToSymbol(g_kv_attn_error, &zero, sizeof(int));
    }
    return e;
}

}  // namespace gdn
