// The latent cache's rows: appending (norm, position rotation, store), reading
// back; and copying pages of any cache.
//
// latent_append: a warp per token and part: its row (latent and position key), or
// the position parts of 32 heads of its q.  A lane's units (8 rotation pairs) of
// different heads turn by the same angles.  The row stays in registers between the
// norm's sum and the store; loads start before the look-ups (sequence, length, page,
// table row) on which only the rotation and the store depend.  Products and sums of
// the rotation are rounded one by one (no fused multiply-add), as the 8-bit cache's
// are.  The chain of look-ups bounds it: 8,688 tokens of 32 heads take 19 us, 5.3
// TB/s of the bytes that have to move, 256 single tokens 2.9 us.  Four tokens a warp with one
// look-up took 19.4 us where one takes 18.3 (8,000 tokens), 50 and 45 us with 128 heads.
// latent_read: a warp takes kReadTokens consecutive rows, whose places its first
// lanes look up side by side; bytes bound it (16,000 rows: 5.9 us, 6.3 TB/s).
// copy_pages: the pairs travel as kernel arguments, so that nothing is copied to
// the device and a captured call keeps its pairs; bytes bound it (2000 pages of 72
// KB: 45 us, 6.6 TB/s, in one launch of up to 2048 pairs; 55 us in five of 400).
#include <algorithm>

#include "gdn_internal.h"
#include "gdn_kv.cuh"
#include "gdn_latent.h"

namespace gdn {

namespace {

using bf16 = __nv_bfloat16;

__device__ __forceinline__ void turn(float& a, float& b, float c, float s) {
    const float ra = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
    const float rb = __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
    a = ra;
    b = rb;
}

// Unit u (0..3) of a position part: 8 rotation pairs as two 8-channel vectors.
__device__ __forceinline__ int unit_first(int u, int style) { return style == 0 ? 8 * u : 16 * u; }
__device__ __forceinline__ int unit_second(int u, int style) { return style == 0 ? 8 * u + kRopeDim / 2 : 16 * u + 8; }

// Cosines and sines of unit u's pairs.
struct Angles {
    float c[8], s[8];
    __device__ __forceinline__ void load(const float* row, int u) {
#pragma unroll
        for (int i = 0; i < 8; i += 4) {
            Vec16<float>::load(row + 8 * u + i, c + i);
            Vec16<float>::load(row + kRopeDim / 2 + 8 * u + i, s + i);
        }
    }
};
// x: the two vectors of a unit.
__device__ __forceinline__ void turn_unit(float* x, const Angles& a, int style) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (style == 0) turn(x[i], x[8 + i], a.c[i], a.s[i]);
        else turn(x[2 * i], x[2 * i + 1], a.c[i], a.s[i]);
    }
}

// Eight values rounded to bf16, finite: NaN becomes 0, infinities the largest number.
__device__ __forceinline__ uint4 finite_bf16(const float* x) {
    constexpr float kTop = 3.3895313892515355e38f;
    float y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = x[i] == x[i] ? fminf(fmaxf(x[i], -kTop), kTop) : 0.0f;
    return make_uint4(pack_bf16_pair(y[0], y[1]), pack_bf16_pair(y[2], y[3]), pack_bf16_pair(y[4], y[5]),
                      pack_bf16_pair(y[6], y[7]));
}

// The norm's range.  Squares of bf16 numbers from 2^64 on are infinite in fp32, those below 2^-75 are 0; a row whose
// mean square (with eps) is out of these bounds is scaled first.  (eps is at most 2^-90 where k is 2^100.)
constexpr float kTopSquare = 1.6615350e35f, kLowSquare = 8.0779357e-28f;  // 2^117, 2^-90
constexpr float kDown = 8.4703295e-22f, kUp = 1.2676506e30f;              // 2^-70, 2^100

constexpr int kAppendThreads = 128;
constexpr int kUnits = 4;   // of a position part
constexpr int kQUnits = 4;  // units of q a lane has in flight: 32 heads a warp

template <int C>
__global__ void __launch_bounds__(kAppendThreads) latent_append_kernel(const LatentAppendArgs a, const uint32_t parts) {
    constexpr int N = C / 256, W = C + kRopeDim;  // 8-channel vectors of the latent a lane holds; channels of a row
    const int lane = threadIdx.x & 31;
    const uint32_t w = blockIdx.x * (kAppendThreads / 32) + (threadIdx.x >> 5);  // below 2^32: the caller checked tokens x heads
    const uint32_t w_tok = w / parts;
    if (w_tok >= static_cast<uint32_t>(a.b.n_tokens)) return;
    const int tok = static_cast<int>(w_tok), part = static_cast<int>(w - w_tok * parts);  // part 0: the row

    // a unit's place does not depend on its head: this lane's are all unit lane % 4, heads apart
    const int u = lane % kUnits, head0 = (part - 1) * 8 * kQUnits + lane / kUnits;
    const int c0 = unit_first(u, a.rope_style), c1 = unit_second(u, a.rope_style);
    uint4 raw[2 * kQUnits];
    if (part == 0) {  // loads first: they depend on nothing
        const bf16* src = static_cast<const bf16*>(a.rows.data) + tok * a.rows.token_stride;
#pragma unroll
        for (int i = 0; i < N; ++i) raw[i] = Vec16<bf16>::load_raw(src + 8 * lane + 256 * i);
        if (lane < kUnits) {
            raw[N] = Vec16<bf16>::load_raw(src + C + c0);
            raw[N + 1] = Vec16<bf16>::load_raw(src + C + c1);
        }
    } else {
        const bf16* src = static_cast<const bf16*>(a.q.data) + tok * a.q.token_stride;
#pragma unroll
        for (int k = 0; k < kQUnits; ++k)
            if (head0 + 8 * k < a.n_heads) {
                const bf16* head = src + (head0 + 8 * k) * a.q.head_stride;
                raw[2 * k] = Vec16<bf16>::load_raw(head + c0);
                raw[2 * k + 1] = Vec16<bf16>::load_raw(head + c1);
            }
    }

    const int seq = a.b.uniform_q ? tok / a.b.uniform_q : warp_seq_of_token(a.b.cu, a.b.n_seq, tok);
    const long long pos = static_cast<long long>(a.b.kv_lens[seq]) - (a.b.cu[seq + 1] - tok);
    Angles angles;
    if (a.rope) {
        long long p = a.positions ? a.positions[tok] : pos;
        if (p < 0 || p >= a.rope_len) {
            if (lane == 0) atomicMax(a.error, kKvErrRope);
            p = p < 0 ? 0 : a.rope_len - 1;
        }
        if (part > 0 || lane < kUnits) angles.load(a.rope + p * kRopeDim, u);
    }
    if (part > 0) {
        bf16* dst = static_cast<bf16*>(const_cast<void*>(a.q_out.data)) + tok * a.q_out.token_stride;
#pragma unroll
        for (int i = 0; i < kQUnits; ++i) {
            if (head0 + 8 * i >= a.n_heads) break;
            float x[16];
            Vec16<bf16>::unpack(raw[2 * i], x);
            Vec16<bf16>::unpack(raw[2 * i + 1], x + 8);
            if (a.rope) turn_unit(x, angles, a.rope_style);
            bf16* head = dst + (head0 + 8 * i) * a.q_out.head_stride;
            Vec16<bf16>::store(head + c0, x);
            Vec16<bf16>::store(head + c1, x + 8);
        }
        return;
    }

    const long long lp = pos < 0 ? -1 : pos / a.page_size;
    const int page = lp >= 0 && lp < a.b.pages_per_seq ? a.b.table[static_cast<size_t>(seq) * a.b.pages_per_seq + lp] : -1;
    const bool mapped = page >= 0 && page < a.c.n_pages;
    if (!mapped && lane == 0) atomicMax(a.error, kKvErrTable);
    float x[8 * N];
#pragma unroll
    for (int i = 0; i < N; ++i) Vec16<bf16>::unpack(raw[i], x + 8 * i);
    if (a.norm_w) {
        float g[8 * N];
#pragma unroll
        for (int i = 0; i < 8 * N; i += 4) Vec16<float>::load(a.norm_w + 8 * lane + 256 * (i / 8) + i % 8, g + i);
        auto mean_square = [&] {
            float sum = 0.0f;
#pragma unroll
            for (int i = 0; i < 8 * N; ++i) sum = fmaf(x[i], x[i], sum);
            return group_sum<32>(sum) * (1.0f / C);
        };
        float eps = a.eps, mean = mean_square();
        if (mean > kTopSquare || mean + eps < kLowSquare) {  // squares that leave fp32: those of k x, with k^2 eps
            const float k = mean > kTopSquare ? kDown : kUp;
#pragma unroll
            for (int i = 0; i < 8 * N; ++i) x[i] *= k;
            eps = eps * k * k;
            mean = mean_square();
        }
        const float r = rsqrtf(mean + eps);
#pragma unroll
        for (int i = 0; i < 8 * N; ++i) x[i] = x[i] * r * g[i];
    }
    uint4 v[N], k0 = make_uint4(0, 0, 0, 0), k1 = k0;
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = finite_bf16(x + 8 * i);
    if (lane < kUnits) {
        float y[16];
        Vec16<bf16>::unpack(raw[N], y);
        Vec16<bf16>::unpack(raw[N + 1], y + 8);
        if (a.rope) turn_unit(y, angles, a.rope_style);
        k0 = finite_bf16(y);
        k1 = finite_bf16(y + 8);
    }
    auto store = [&](bf16* to) {
#pragma unroll
        for (int i = 0; i < N; ++i) *reinterpret_cast<uint4*>(to + 8 * lane + 256 * i) = v[i];
        if (lane < kUnits) {
            *reinterpret_cast<uint4*>(to + C + c0) = k0;
            *reinterpret_cast<uint4*>(to + C + c1) = k1;
        }
    };
    if (mapped)
        store(static_cast<bf16*>(a.c.rows) + (static_cast<size_t>(page) * a.page_size + static_cast<int>(pos % a.page_size)) * W);
    if (a.rows_out) store(static_cast<bf16*>(a.rows_out) + static_cast<size_t>(tok) * W);
}

template <int C>
cudaError_t append_t(const LatentAppendArgs& a, cudaStream_t st) {
    const int parts = 1 + (a.q.data ? (a.n_heads + 8 * kQUnits - 1) / (8 * kQUnits) : 0);
    const unsigned long long blocks = (static_cast<unsigned long long>(a.b.n_tokens) * parts + kAppendThreads / 32 - 1) / (kAppendThreads / 32);
    latent_append_kernel<C><<<static_cast<unsigned>(blocks), kAppendThreads, 0, st>>>(a, parts);
    return cudaGetLastError();
}

constexpr int kReadThreads = 256, kReadTokens = 4;

template <int C>
__global__ void __launch_bounds__(kReadThreads) latent_read_kernel(const LatentReadArgs a) {
    constexpr int V = (C + kRopeDim) / 8, K = (kReadTokens * V + 31) / 32;  // vectors of a row, of a lane
    const int lane = threadIdx.x & 31;
    const long long w = static_cast<long long>(blockIdx.x) * (kReadThreads / 32) + (threadIdx.x >> 5);
    if (w * kReadTokens >= a.b.n_tokens) return;
    const int tok0 = static_cast<int>(w) * kReadTokens, n = min(kReadTokens, a.b.n_tokens - tok0);
    long long at = -1;  // row in the cache of token tok0 + lane
    if (lane < n) {
        const int tok = tok0 + lane, seq = a.b.uniform_q ? tok / a.b.uniform_q : seq_of_token(a.b.cu, a.b.n_seq, tok);
        const long long pos = static_cast<long long>(a.b.kv_lens[seq]) + (tok - a.b.cu[seq]);
        const long long lp = pos < 0 ? -1 : pos / a.page_size;
        const int page = lp >= 0 && lp < a.b.pages_per_seq ? a.b.table[static_cast<size_t>(seq) * a.b.pages_per_seq + lp] : -1;
        if (page >= 0 && page < a.c.n_pages) at = static_cast<long long>(page) * a.page_size + pos % a.page_size;
        else atomicMax(a.error, kKvErrTable);
    }
    const uint4* src = static_cast<const uint4*>(a.c.rows);
    uint4* dst = static_cast<uint4*>(a.out) + static_cast<size_t>(tok0) * V;
    uint4 v[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int i = lane + 32 * k, t = i / V;
        const long long row = __shfl_sync(0xffffffffu, at, t & 31);
        v[k] = t < n && row >= 0 ? src[row * V + i % V] : make_uint4(0, 0, 0, 0);  // zeros of unmapped pages
    }
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int i = lane + 32 * k;
        if (i < n * V) dst[i] = v[k];
    }
}

// ---------------------------------------------------------------- page copies
constexpr int kBuffers = 32, kFewPairs = 256, kManyPairs = 2048;  // of a launch, whose arguments they are
template <int PAIRS> struct CopyArgs {
    uint8_t* base[kBuffers];
    unsigned bytes[kBuffers];
    int n_buffers;
    int2 pair[PAIRS];  // source, destination
};
constexpr int kCopyThreads = 256, kCopyVectors = 4;

// W: what is moved at a time, uint4 or uint32_t.
template <typename W, typename A>
__global__ void __launch_bounds__(kCopyThreads) copy_pages_kernel(const __grid_constant__ A a) {
    const int2 p = a.pair[blockIdx.y];
    const int b = blockIdx.z;
    const unsigned n = a.bytes[b] / sizeof(W);
    const W* src = reinterpret_cast<const W*>(a.base[b] + static_cast<size_t>(p.x) * a.bytes[b]);
    W* dst = reinterpret_cast<W*>(a.base[b] + static_cast<size_t>(p.y) * a.bytes[b]);
    const unsigned i0 = blockIdx.x * (kCopyThreads * kCopyVectors) + threadIdx.x;
    W v[kCopyVectors];
#pragma unroll
    for (int k = 0; k < kCopyVectors; ++k)
        if (i0 + k * kCopyThreads < n) v[k] = src[i0 + k * kCopyThreads];
#pragma unroll
    for (int k = 0; k < kCopyVectors; ++k)
        if (i0 + k * kCopyThreads < n) dst[i0 + k * kCopyThreads] = v[k];
}

// The arrays whose pages all lie on 16 bytes, or (W 32 bits) the others.
template <typename W, int PAIRS>
cudaError_t copy_some(void* const* bases, const size_t* page_bytes, int n_buffers, const int32_t* src, const int32_t* dst,
                      int n_pairs, cudaStream_t st) {
    using A = CopyArgs<PAIRS>;
    A a;
    for (int b = 0; b < n_buffers;) {
        a.n_buffers = 0;
        unsigned most = 0;
        for (; b < n_buffers && a.n_buffers < kBuffers; ++b) {
            const bool wide = page_bytes[b] % 16 == 0 && (reinterpret_cast<uintptr_t>(bases[b]) & 15u) == 0;
            if (wide != (sizeof(W) == 16)) continue;
            a.base[a.n_buffers] = static_cast<uint8_t*>(bases[b]);
            a.bytes[a.n_buffers++] = static_cast<unsigned>(page_bytes[b]);
            most = std::max(most, static_cast<unsigned>(page_bytes[b]));
        }
        if (a.n_buffers == 0) break;
        const unsigned step = kCopyThreads * kCopyVectors * sizeof(W);
        for (int p0 = 0; p0 < n_pairs; p0 += PAIRS) {
            const int n = std::min(PAIRS, n_pairs - p0);
            for (int i = 0; i < n; ++i) a.pair[i] = make_int2(src[p0 + i], dst[p0 + i]);
            copy_pages_kernel<W, A><<<dim3((most + step - 1) / step, n, a.n_buffers), kCopyThreads, 0, st>>>(a);
            const cudaError_t e = cudaGetLastError();
            if (e != cudaSuccess) return e;
        }
    }
    return cudaSuccess;
}

}  // namespace

cudaError_t launch_latent_append(const LatentAppendArgs& a, int latent_dim, cudaStream_t st) {
    return latent_dim == 512 ? append_t<512>(a, st) : append_t<256>(a, st);
}

cudaError_t launch_latent_read(const LatentReadArgs& a, int latent_dim, cudaStream_t st) {
    const long long warps = (static_cast<long long>(a.b.n_tokens) + kReadTokens - 1) / kReadTokens;
    const unsigned blocks = static_cast<unsigned>((warps + kReadThreads / 32 - 1) / (kReadThreads / 32));
    if (latent_dim == 512) latent_read_kernel<512><<<blocks, kReadThreads, 0, st>>>(a);
    else latent_read_kernel<256><<<blocks, kReadThreads, 0, st>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_copy_pages(void* const* bases, const size_t* page_bytes, int n_buffers, const int32_t* src,
                              const int32_t* dst, int n_pairs, cudaStream_t st) {
    auto copy = [&](auto word) {
        using W = decltype(word);
        return n_pairs <= kFewPairs ? copy_some<W, kFewPairs>(bases, page_bytes, n_buffers, src, dst, n_pairs, st)
                                    : copy_some<W, kManyPairs>(bases, page_bytes, n_buffers, src, dst, n_pairs, st);
    };
    const cudaError_t e = copy(uint4{});
    return e != cudaSuccess ? e : copy(uint32_t{});
}

}  // namespace gdn
