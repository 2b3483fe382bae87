// Verification of drafted tokens from given random numbers
// (gdn_accept_drafts in include/gdn.h states the rule).
//
// One thread block per sequence walks its rows: logits rows first give their
// maximum (with its lowest index) and sum of exponentials, the draft's two
// probabilities decide whether it stands, and the row where that ends gives
// the token by the largest r / noise.  The race r / noise needs no prefix sums
// over the vocabulary, so the result does not depend on the order in which
// threads add.
#include <cfloat>

#include "gdn_common.cuh"
#include "gdn_internal.h"
#include "gdn_kv.h"

namespace gdn {

namespace {

constexpr int kThreads = 1024;

struct Best {
    float v;
    int i;
};
__device__ __forceinline__ Best better(Best a, Best b) {  // the larger; the lower index on ties
    return (b.v > a.v || (b.v == a.v && b.i < a.i)) ? b : a;
}
__device__ __forceinline__ Best block_best(Best x) {
    __shared__ Best part[32];
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
        const Best y{__shfl_xor_sync(0xffffffffu, x.v, off), __shfl_xor_sync(0xffffffffu, x.i, off)};
        x = better(x, y);
    }
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = x;
    __syncthreads();
    x = part[0];
    for (int w = 1; w < kThreads / 32; ++w) x = better(x, part[w]);
    __syncthreads();
    return x;
}
__device__ __forceinline__ float block_sum(float x) {
    __shared__ float part[32];
    x = group_sum<32>(x);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = x;
    __syncthreads();
    x = 0.0f;
    for (int w = 0; w < kThreads / 32; ++w) x += part[w];
    __syncthreads();
    return x;
}

// A row's distribution: probability of token j is exp((x_j - top) inv_t) / sum.
struct Row {
    float top, inv_sum;
    int at;  // lowest index of the largest logit
};

template <typename T>
__device__ Row row_stats(const T* x, int vocab, float inv_t) {
    Best b{-INFINITY, 0x7fffffff};
    for (int j = threadIdx.x; j < vocab; j += kThreads) b = better(b, Best{to_f32(x[j]), j});
    b = block_best(b);
    float s = 0.0f;
    if (b.v > -INFINITY)
        for (int j = threadIdx.x; j < vocab; j += kThreads) s += expf((to_f32(x[j]) - b.v) * inv_t);
    s = block_sum(s);
    return Row{b.v, s > 0.0f ? 1.0f / s : 0.0f, b.i};
}

template <typename T, bool LOGITS>
__device__ __forceinline__ float prob(const T* x, int j, const Row& r, float inv_t) {
    if (!LOGITS) return to_f32(x[j]);
    return r.inv_sum > 0.0f ? expf((to_f32(x[j]) - r.top) * inv_t) * r.inv_sum : 0.0f;
}

template <typename T, bool LOGITS>
__global__ void __launch_bounds__(kThreads) accept_kernel(const AcceptArgs a) {
    const int seq = blockIdx.x, V = a.vocab;
    const T* target = static_cast<const T*>(a.target) + static_cast<long long>(seq) * (a.T + 1) * a.target_stride;
    const T* draft = static_cast<const T*>(a.draft) + static_cast<long long>(seq) * a.T * a.draft_stride;
    const float temp = LOGITS && a.temperature ? a.temperature[seq] : 1.0f;
    const bool greedy = LOGITS && !(temp > 0.0f);
    const float inv_t = greedy ? 1.0f : 1.0f / temp;
    int32_t* tokens = a.tokens + static_cast<long long>(seq) * (a.T + 1);
    Row p{0, 0, 0}, q{0, 0, 0};
    int t = 0, fallen = -1;
    const T *px = nullptr, *qx = nullptr;
    for (;; ++t) {
        px = target + t * a.target_stride;
        if (LOGITS) p = row_stats(px, V, inv_t);
        fallen = -1;
        if (t == a.T) break;
        const int x = a.drafts[static_cast<long long>(seq) * a.T + t];
        if (x < 0 || x >= V) break;
        fallen = x;
        if (greedy) {
            if (x != p.at) break;
        } else {
            float qv = 1.0f;
            if (a.draft) {
                qx = draft + t * a.draft_stride;
                if (LOGITS) q = row_stats(qx, V, inv_t);
                qv = prob<T, LOGITS>(qx, x, q, inv_t);
            }
            const float u = a.uniforms[static_cast<long long>(seq) * a.T + t];
            if (!(u * qv < prob<T, LOGITS>(px, x, p, inv_t))) break;
        }
        if (threadIdx.x == 0) tokens[t] = x;
    }
    int token;
    if (greedy) {
        token = p.top > -INFINITY ? p.at : -1;
    } else {
        const float* e = a.noise + static_cast<long long>(seq) * a.noise_stride;
        Best b{0.0f, 0x7fffffff};
        for (int pass = fallen >= 0 ? 0 : 1; pass < 2 && !(b.v > 0.0f); ++pass) {
            Best mine{0.0f, 0x7fffffff};
            for (int j = threadIdx.x; j < V; j += kThreads) {
                float r = prob<T, LOGITS>(px, j, p, inv_t);
                if (pass == 0) r -= a.draft ? prob<T, LOGITS>(qx, j, q, inv_t) : (j == fallen ? 1.0f : 0.0f);
                if (r > 0.0f) mine = better(mine, Best{r / e[j], j});
            }
            b = block_best(mine);
        }
        token = b.v > 0.0f ? b.i : -1;
    }
    if (threadIdx.x == 0) {
        a.accepted[seq] = t;
        tokens[t] = token;
        for (int k = t + 1; k <= a.T; ++k) tokens[k] = -1;
    }
}

}  // namespace

cudaError_t launch_accept_drafts(const AcceptArgs& a, bool logits, bool bf16, cudaStream_t stream) {
    if (!logits) accept_kernel<float, false><<<a.n_seq, kThreads, 0, stream>>>(a);
    else if (bf16) accept_kernel<__nv_bfloat16, true><<<a.n_seq, kThreads, 0, stream>>>(a);
    else accept_kernel<float, true><<<a.n_seq, kThreads, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace gdn
