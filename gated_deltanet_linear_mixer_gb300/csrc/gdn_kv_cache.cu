// Appending to the paged 8-bit cache (with the position rotation of q and k on
// the way) and reading values back out of it.
//
// kv_append: one thread block per (page the call writes to, kv head, K or V)
// finds the block's largest |new value|, settles the block's scale and writes
// the codes, so the scale needs no atomics and every result is independent of
// order.  A thread holds its (rotated) values in registers between the maximum
// and the rounding, so the new rows are read once.  Products and sums of the
// rotation are rounded one by one (no fused multiply-add) and the division is
// the exact one: the stored codes do not depend on how a compiler contracts an
// expression.  q is rotated by further thread blocks: of the same launch for a
// few tokens, where the chain of look-ups (lengths, page, scale) bounds the time
// and a second launch would add to it; of a kernel beside it for prompts, where
// registers bound how many warps cover that chain (8,688 tokens, 32 + 2 x 8 heads
// of 128: 79 us in one kernel, 52 us in two; the bytes alone take 29 us).
// 256 single tokens with 16 + 2 x 2 heads of 256, appended and read back by
// kv_read, take 12.6 us: the chain, twice.
// kv_read: bytes bound it (16,000 tokens of 8 heads of 128, 98 MB: 16.5 us,
// 5.9 TB/s); for few tokens the launch and its look-ups do (300 tokens: 3.2 us).
#include <algorithm>

#include "gdn_internal.h"
#include "gdn_kv.cuh"

namespace gdn {

namespace {

// 16 channels of a row, as two 8-channel vectors at c0 and c1, such that
// neighbouring units' vectors are neighbours in memory: the two members of 8
// rotation pairs (style half), else vectors that hold whole pairs, or none.
struct Unit {
    int c0, c1;
};
template <int D> __device__ __forceinline__ Unit unit_at(int u, int rope_dim, int style) {
    if (style != 0 || rope_dim == 0) return Unit{8 * u, 8 * u + D / 2};
    if (16 * u < rope_dim) return Unit{8 * u, 8 * u + rope_dim / 2};
    return Unit{rope_dim / 2 + 8 * u, rope_dim / 2 + 8 * u + (D - rope_dim) / 2};
}

template <typename T>
__device__ __forceinline__ void load8(const T* p, float* x) {
    constexpr int N = Vec16<T>::N;
#pragma unroll
    for (int i = 0; i < 8; i += N) Vec16<T>::load(p + i, x + i);
}
template <typename T>
__device__ __forceinline__ void store8(T* p, const float* x) {
    constexpr int N = Vec16<T>::N;
#pragma unroll
    for (int i = 0; i < 8; i += N) Vec16<T>::store(p + i, x + i);
}

__device__ __forceinline__ void rotate_pair(float& a, float& b, float c, float s) {
    const float ra = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
    const float rb = __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
    a = ra;
    b = rb;
}

// x[0..7], x[8..15]: the vectors of unit u; row: the cosines and sines of its token.
__device__ __forceinline__ void rotate_unit(float* x, const float* row, int u, const Unit& w, int rope_dim, int style) {
    float c[8], s[8];
    if (style == 0) {
        if (16 * u >= rope_dim) return;
        load8(row + 8 * u, c);
        load8(row + rope_dim / 2 + 8 * u, s);
#pragma unroll
        for (int i = 0; i < 8; ++i) rotate_pair(x[i], x[8 + i], c[i], s[i]);
    } else {
#pragma unroll
        for (int v = 0; v < 2; ++v) {  // four pairs a vector
            const int ch = v ? w.c1 : w.c0;
            if (ch >= rope_dim) continue;
            Vec16<float>::load(row + ch / 2, c);
            Vec16<float>::load(row + rope_dim / 2 + ch / 2, s);
#pragma unroll
            for (int i = 0; i < 4; ++i) rotate_pair(x[8 * v + 2 * i], x[8 * v + 2 * i + 1], c[i], s[i]);
        }
    }
}

// The rotation table's row of a token; stays inside the table.
__device__ __forceinline__ const float* rope_row(const KvAppendArgs& a, int tok, int pos) {
    int p = a.positions ? a.positions[tok] : pos;
    if (p < 0 || p >= a.rope_len) {
        atomicMax(a.error, kKvErrRope);
        p = p < 0 ? 0 : a.rope_len - 1;
    }
    return a.rope + static_cast<size_t>(p) * a.rope_dim;
}

constexpr int kQUnits = 2;  // units of q a lane has in flight

// q: a warp takes 32 kQUnits units of one token, which has one position and one
// table row.  `block`: thread blocks of q before this one.
template <typename T, int D>
__device__ __forceinline__ void rotate_q(const KvAppendArgs& a, unsigned block) {
    constexpr int U = D / 16;  // units of a row
    const int units = a.n_q_heads * U, parts = (units + 32 * kQUnits - 1) / (32 * kQUnits);
    const long long w = static_cast<long long>(block) * (blockDim.x / 32) + (threadIdx.x >> 5);
    const int tok = static_cast<int>(w / parts);
    if (tok >= a.b.n_tokens) return;
    const int first = static_cast<int>(w % parts) * 32 * kQUnits + (threadIdx.x & 31);
    const T* src = static_cast<const T*>(a.q.data) + tok * a.q.token_stride;
    T* dst = static_cast<T*>(a.q_out) + static_cast<size_t>(tok) * a.n_q_heads * D;
    float x[kQUnits][16];
#pragma unroll
    for (int k = 0; k < kQUnits; ++k) {
        const int i = first + 32 * k;
        if (i < units) {
            const Unit r = unit_at<D>(i % U, a.rope_dim, a.rope_style);
            const T* row = src + i / U * a.q.head_stride;
            load8(row + r.c0, x[k]);
            load8(row + r.c1, x[k] + 8);
        }
    }
    const float* row = nullptr;
    if (a.rope_dim > 0) {
        int pos = 0;
        if (!a.positions) {
            const int s = a.b.uniform_q ? tok / a.b.uniform_q : warp_seq_of_token(a.b.cu, a.b.n_seq, tok);
            pos = a.b.kv_lens[s] - (a.b.cu[s + 1] - tok);
        }
        row = rope_row(a, tok, pos);
    }
#pragma unroll
    for (int k = 0; k < kQUnits; ++k) {
        const int i = first + 32 * k;
        if (i < units) {
            const int u = i % U;
            const Unit r = unit_at<D>(u, a.rope_dim, a.rope_style);
            if (row) rotate_unit(x[k], row, u, r, a.rope_dim, a.rope_style);
            store8(dst + i / U * D + r.c0, x[k]);
            store8(dst + i / U * D + r.c1, x[k] + 8);
        }
    }
}

constexpr int kQThreads = 256;

// Prompts: q by a kernel of its own, which its few registers let fill the SMs,
// beside the storing kernel (a programmatic dependent that depends on nothing of
// it).  Its first thread block waits for that kernel, so that whatever follows
// in the stream follows both.
template <typename T, int D>
__global__ void __launch_bounds__(kQThreads) kv_rotate_q_kernel(const KvAppendArgs a) {
    rotate_q<T, D>(a, blockIdx.x);
    if (blockIdx.x == 0) asm volatile("griddepcontrol.wait;" ::: "memory");
}

// UNITS: units of new rows a thread holds in registers (2: whole pages, q apart;
// 1: a few rows a page, small thread blocks, q by further ones of the launch).
template <typename T, typename F, int D, int UNITS>
__global__ void __launch_bounds__(UNITS == 1 ? 256 : 1024)
kv_append_kernel(const KvAppendArgs a, const int n_store_blocks) {
    constexpr int U = D / 16;  // units of a row
    const int tid = threadIdx.x, nt = blockDim.x;
    const int B = a.page_size;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (UNITS == 1 && static_cast<int>(blockIdx.x) >= n_store_blocks) {
        rotate_q<T, D>(a, blockIdx.x - n_store_blocks);
        return;
    }

    const int is_v = blockIdx.x & 1, item = (blockIdx.x >> 1) / a.n_kv_heads;
    const int h = (blockIdx.x >> 1) - item * a.n_kv_heads;
    int seq, local;
    if (a.b.uniform_q) {
        const int per = (a.b.uniform_q + B - 2) / B + 1;
        seq = item / per;
        local = item - seq * per;
    } else {
        seq = warp_seq_of_slot(a.b.cu, a.b.n_seq, B, item);
        local = item - (a.b.cu[seq] / B + 2 * seq);
    }
    const int q0 = a.b.cu[seq], len = a.b.kv_lens[seq], start = len - (a.b.cu[seq + 1] - q0);
    const long long cap = static_cast<long long>(a.b.pages_per_seq) * B;
    if ((start < 0 || len > cap) && tid == 0) atomicMax(a.error, kKvErrTable);
    const int p0 = max(start, 0), p1 = static_cast<int>(min(static_cast<long long>(len), cap));
    const int lp = p0 / B + local;
    if (p0 >= p1 || lp > (p1 - 1) / B) return;
    const int page = a.b.table[static_cast<size_t>(seq) * a.b.pages_per_seq + lp];
    if (page < 0 || page >= a.c.n_pages) {
        if (tid == 0) atomicMax(a.error, kKvErrTable);
        return;
    }
    const int r0 = max(p0 - lp * B, 0), r1 = min(p1 - lp * B, B);  // new rows of the page
    const int kept = start > lp * B ? r0 : 0;                      // earlier rows of this sequence

    const KvRows& rows = is_v ? a.v : a.k;
    float x[UNITS][16];
    float most = 0.0f;
    const int n_units = (r1 - r0) * U;
#pragma unroll
    for (int it = 0; it < UNITS; ++it) {
        const int i = tid + it * nt;
        if (i < n_units) {
            const int u = i % U, pos = lp * B + r0 + i / U, tok = q0 + (pos - start);
            const Unit w = unit_at<D>(u, is_v ? 0 : a.rope_dim, a.rope_style);
            const T* src = static_cast<const T*>(rows.data) + tok * rows.token_stride + h * rows.head_stride;
            load8(src + w.c0, x[it]);
            load8(src + w.c1, x[it] + 8);
            if (!is_v && a.rope_dim > 0) rotate_unit(x[it], rope_row(a, tok, pos), u, w, a.rope_dim, a.rope_style);
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const float m = fabsf(x[it][e]);
                if (m <= 3.402823466e38f) most = fmaxf(most, m);  // finite values only
            }
        }
    }
    const size_t block = static_cast<size_t>(page) * a.n_kv_heads + h;
    float* scale_at = (is_v ? a.c.v_scale : a.c.k_scale) + block;
    const float old = kept > 0 ? *scale_at : 0.0f;
    __shared__ float part[32];
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, off));
    if ((tid & 31) == 0) part[tid >> 5] = most;
    __syncthreads();
    most = part[0];
    for (int w = 1; w < nt / 32; ++w) most = fmaxf(most, part[w]);
    const float scale = fmaxf(old, __fmul_rn(most, 1.0f / F::top()));
    uint8_t* codes = (is_v ? a.c.v : a.c.k) + block * B * D;
    if (kept > 0 && scale > old) {
        const float ratio = old / scale;
        uint4* p = reinterpret_cast<uint4*>(codes);
        for (int i = tid; i < kept * U; i += nt) {
            const uint4 w = p[i];
            const uint32_t c[4] = {w.x, w.y, w.z, w.w};
            uint32_t n[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float y[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) y[k] = __fmul_rn(F::value(static_cast<uint8_t>(c[e] >> (8 * k))), ratio);
                n[e] = F::code4(y);
            }
            p[i] = make_uint4(n[0], n[1], n[2], n[3]);
        }
    }
#pragma unroll
    for (int it = 0; it < UNITS; ++it) {
        const int i = tid + it * nt;
        if (i < n_units) {
            const int u = i % U, row = r0 + i / U;
            const Unit w = unit_at<D>(u, is_v ? 0 : a.rope_dim, a.rope_style);
            uint32_t c[4] = {0, 0, 0, 0};
            if (scale > 0.0f) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float y[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) y[k] = x[it][4 * e + k] / scale;
                    c[e] = F::code4(y);
                }
            }
            *reinterpret_cast<uint2*>(codes + static_cast<size_t>(row) * D + w.c0) = make_uint2(c[0], c[1]);
            *reinterpret_cast<uint2*>(codes + static_cast<size_t>(row) * D + w.c1) = make_uint2(c[2], c[3]);
        }
    }
    if (tid == 0) *scale_at = scale;
}

constexpr int kReadThreads = 256, kReadVectors = 4;

// A warp takes 32 kReadVectors 16-byte vectors of one token's K and V outputs:
// the token's page is looked up once.
template <typename T, typename F, int D>
__global__ void __launch_bounds__(kReadThreads) kv_read_kernel(const KvReadArgs a) {
    constexpr int N = Vec16<T>::N, P = D / N;  // codes of a vector, vectors of a head
    const int per_row = a.n_kv_heads * P, parts = (per_row + 32 * kReadVectors - 1) / (32 * kReadVectors);
    const long long w = static_cast<long long>(blockIdx.x) * (kReadThreads / 32) + (threadIdx.x >> 5);
    const int tok = static_cast<int>(w / parts);
    if (tok >= a.b.n_tokens) return;
    const int first = static_cast<int>(w % parts) * 32 * kReadVectors + (threadIdx.x & 31);
    const int seq = a.b.uniform_q ? tok / a.b.uniform_q : warp_seq_of_token(a.b.cu, a.b.n_seq, tok);
    const long long pos = static_cast<long long>(a.b.kv_lens[seq]) + (tok - a.b.cu[seq]);
    const long long lp = pos < 0 ? -1 : pos / a.page_size;
    const int page = lp >= 0 && lp < a.b.pages_per_seq
                         ? a.b.table[static_cast<size_t>(seq) * a.b.pages_per_seq + lp] : -1;
    const bool mapped = page >= 0 && page < a.c.n_pages;  // else zeros
    if (!mapped && (threadIdx.x & 31) == 0) atomicMax(a.error, kKvErrTable);
    const size_t block0 = static_cast<size_t>(mapped ? page : 0) * a.n_kv_heads;
    const int slot = mapped ? static_cast<int>(pos % a.page_size) : 0;
    uint2 code[kReadVectors][2];
    float scale[kReadVectors][2];
#pragma unroll
    for (int k = 0; k < kReadVectors; ++k) {
        const int i = first + 32 * k;
        code[k][0] = code[k][1] = make_uint2(0, 0);
        scale[k][0] = scale[k][1] = 0.0f;
        if (i >= per_row || !mapped) continue;
        const size_t block = block0 + i / P;
        const size_t at = (block * a.page_size + slot) * D + i % P * N;
        if (N == 8) {
            code[k][0] = *reinterpret_cast<const uint2*>(a.c.k + at);
            code[k][1] = *reinterpret_cast<const uint2*>(a.c.v + at);
        } else {
            code[k][0].x = *reinterpret_cast<const uint32_t*>(a.c.k + at);
            code[k][1].x = *reinterpret_cast<const uint32_t*>(a.c.v + at);
        }
        scale[k][0] = a.c.k_scale[block];
        scale[k][1] = a.c.v_scale[block];
    }
#pragma unroll
    for (int k = 0; k < kReadVectors; ++k) {
        const int i = first + 32 * k;
        if (i >= per_row) continue;
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
            float x[N];
#pragma unroll
            for (int e = 0; e < N; ++e) {
                const uint32_t word = e < 4 ? code[k][kv].x : code[k][kv].y;
                x[e] = F::value(static_cast<uint8_t>(word >> (8 * (e & 3)))) * scale[k][kv];
            }
            Vec16<T>::store(static_cast<T*>(kv ? a.v_out : a.k_out) + (static_cast<size_t>(tok) * per_row + i) * N, x);
        }
    }
}

template <typename T, typename F, int D, int UNITS>
cudaError_t append_units(const KvAppendArgs& a, int nt, cudaStream_t st) {
    const int B = a.page_size;
    const long long slots = a.b.uniform_q ? static_cast<long long>(a.b.n_seq) * ((a.b.uniform_q + B - 2) / B + 1)
                                          : static_cast<long long>(a.b.n_tokens) / B + 2LL * a.b.n_seq;
    const long long store = slots * a.n_kv_heads * 2;
    const long long parts = (a.n_q_heads * (D / 16) + 32 * kQUnits - 1) / (32 * kQUnits);
    const int q_warps = (UNITS == 1 ? nt : kQThreads) / 32;
    const long long q_blocks = a.q.data ? (a.b.n_tokens * parts + q_warps - 1) / q_warps : 0;
    if (store + q_blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    const long long blocks = store + (UNITS == 1 ? q_blocks : 0);
    kv_append_kernel<T, F, D, UNITS><<<static_cast<unsigned>(blocks), nt, 0, st>>>(a, static_cast<int>(store));
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || UNITS == 1 || q_blocks == 0) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(q_blocks));
    cfg.blockDim = dim3(kQThreads);
    cfg.stream = st;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kv_rotate_q_kernel<T, D>, a);
}

template <typename T, typename F, int D>
cudaError_t append_t(const KvAppendArgs& a, cudaStream_t st) {
    // units of new rows in a page: up to 128 are a small thread block's one each, whole pages two a thread
    // with q apart.  Appended and read back, microseconds one / two a thread: 16 x 8 tokens of 2 heads of
    // 256 6.8 / 7.9, 64 x 4 of 8 heads of 128 8.5 / 8.5, 256 x 1 of 2 heads of 256 13.7 / 13.7.
    const int units = std::min(a.b.max_q, a.page_size) * (D / 16);
    return units <= 128 ? append_units<T, F, D, 1>(a, std::max(64, (units + 31) / 32 * 32), st)
                        : append_units<T, F, D, 2>(a, std::max(64, (units + 63) / 64 * 32), st);
}

template <typename T, typename F, int D>
cudaError_t read_t(const KvReadArgs& a, cudaStream_t st) {
    const int per_row = a.n_kv_heads * (D / Vec16<T>::N);
    const long long warps = static_cast<long long>(a.b.n_tokens) * ((per_row + 32 * kReadVectors - 1) / (32 * kReadVectors));
    const long long blocks = (warps + kReadThreads / 32 - 1) / (kReadThreads / 32);
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    kv_read_kernel<T, F, D><<<static_cast<unsigned>(blocks), kReadThreads, 0, st>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv_append(const KvAppendArgs& a, int head_dim, bool bf16, bool e4m3, cudaStream_t stream) {
    return GDN_KV_PICK(append_t);
}

cudaError_t launch_kv_read(const KvReadArgs& a, int head_dim, bool bf16, bool e4m3, cudaStream_t stream) {
    return GDN_KV_PICK(read_t);
}

}  // namespace gdn
