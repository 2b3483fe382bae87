// Causal attention over the paged 8-bit cache: few query rows per kv head
// (single tokens, drafts), and fp32 activations of any length.
//
// Mathematics.  Row r = (token, head of the group) of one sequence and kv head
// attends to the keys its position and window allow.  Codes are small integers
// (or e4m3 values), exact in f16 and in bf16, so the tensor cores work on the
// codes themselves; a block's scales come in outside of the products:
//   y_rj = (q_r . ck_j) scale s_k[blk(j)] log2 e + log2 s_v[blk(j)]
//   w_rj = 2^(y_rj - m_r),  o_r = sum_j w_rj cv_j / sum_blk (sum_j w_rj) / s_v[blk]
// The value scale enters the exponent; the denominator takes it out again, once
// per 16 keys.  m_r is a reference, not the exact maximum: it moves (and o_r is
// rescaled) only when a score exceeds it by 2^kLazy.
// Queries become f16 after division by a power of two per row (bf16's 8 bits are
// exact from 2^-17 of the row's largest up; below, the error is at most 2^-25 of
// it).  Weights
// become f16, 11 bits, in a group of keys whose weights are all normal f16
// numbers (2^-14 .. 2^15 with kBias, scores within 2^-21 of the reference);
// else two bf16 terms, 16 bits: f16 would drop weights below 2^-24 of the
// largest, all that is left in a channel where the heavy keys are zero, and one
// bf16 term's 2^-8 would be as large as the output's own rounding.  The second
// form in every group costs 207 us against 195 us at 256 sequences of 127..8191
// keys (head_dim 256), 139 us against 110 us at 64 x 4 drafts (head_dim 128).  With fp32 activations
// queries are f16 (hi, lo) pairs, 22 bits, and weights three bf16 terms.
//
// One thread block takes 8, 16 or 32 rows and a range of keys.  Keys (and value
// channels) are the tensor core's M, the rows its N, so that a group of 8 heads
// fills the tile and a code is widened once for all rows:
//   S^T [16 keys x rows] = K Q^T,   O^T [16 channels x rows] += V^T P^T
// The accumulator of S^T holds a key's rows where the second product wants a
// row's keys: one 8 x 8 transpose per 8 keys and term.  V^T's operand comes by
// the transposing 8-bit matrix load, which gives a lane four consecutive keys
// of a channel; S^T's rows take the keys in the order that fits (0, 1, 4, 5, ..,
// then 2, 3, 6, 7, ..).  Each of the four warps takes every fourth group of 16
// keys on its own, with its own running state and its own ring of asynchronous
// copies (no block-wide barrier until the end): 16 keys lie in one page, so a
// group is one contiguous run of codes and two scales.  A long axis is split
// over thread blocks and joined by kv_attn_join.
//
// What bounds it: the codes' bytes for single tokens in groups of 8 heads (256
// sequences: 194 us, 1.16 GB, 6.0 TB/s of the 6.8 that a copy reaches; one of
// 131,000 keys 31 us, 4.3 TB/s, since half a round of thread blocks and the join
// are latency); latency at three thread blocks an SM (168 registers) for drafts,
// whose rows need more of the warps' work per code (64 x 4 drafts of 32 heads:
// 110 us, 4.3 TB/s, issue slots 47% busy, most stalls fixed latencies); the
// two launches for short contexts (1000 keys: 7.5 us).
#include <algorithm>
#include <atomic>

#include "gdn_internal.h"
#include "gdn_kv.cuh"

namespace gdn {

namespace {

constexpr int kWarps = 4, kThreads = 32 * kWarps;
constexpr int kGroup = 16;        // keys of a warp's step
constexpr int kStepKeys = kGroup * kWarps;
constexpr int kSpan = 32;         // steps whose pages and scales are looked up at a time
constexpr float kLazy = 8.0f;     // a reference lags behind the maximum by at most 2^8
constexpr float kBias = 7.0f;     // weights are 2^7 times theirs: at most 2^15
constexpr float kNormal = 21.0f;  // scores down to 2^-21 of the reference are normal f16 weights

__device__ __forceinline__ void mma_f16(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_bf16(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Two 16 x 16 tiles of 8-bit codes, transposed: of tile c, f[2c] and f[2c + 1]
// are four consecutive rows (4 (lane % 4) ..) of columns lane / 4 and that + 8.
__device__ __forceinline__ void load_codes_t(uint32_t addr, uint32_t* f) {
    asm volatile("ldmatrix.sync.aligned.m16n16.x2.trans.shared.b8 {%0,%1,%2,%3}, [%4];"
                 : "=r"(f[0]), "=r"(f[1]), "=r"(f[2]), "=r"(f[3])
                 : "r"(addr)
                 : "memory");
}
// Transposes an 8 x 8 tile of 16-bit values held two a lane.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ float bf16_low(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_high(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// The residual of pack_f16(lo, hi), as f16.
__device__ __forceinline__ uint32_t pack_f16_rest(uint32_t h, float lo, float hi) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
    return pack_f16(lo - f.x, hi - f.y);
}

// Four codes of a word to bf16: codes (0, 1) and (2, 3).
template <typename F> __device__ __forceinline__ void widen_bf16(uint32_t w, uint32_t& a, uint32_t& b);
template <> __device__ __forceinline__ void widen_bf16<KvInt8>(uint32_t w, uint32_t& a, uint32_t& b) {
    // under the exponent of 128 the low seven bits of a code are the bf16 128 + (c & 127); the sign
    // bit alone is 128, or 256 for a negative code; their difference is c
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t x = __byte_perm(w, 0x43434343u, i == 0 ? 0x4140 : 0x4342);
        const uint32_t lo = x & 0xFF7FFF7Fu, hi = x & 0xFF80FF80u;
        const __nv_bfloat162 r =
            __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&lo), *reinterpret_cast<const __nv_bfloat162*>(&hi));
        (i == 0 ? a : b) = *reinterpret_cast<const uint32_t*>(&r);
    }
}
template <> __device__ __forceinline__ void widen_bf16<KvE4m3>(uint32_t w, uint32_t& a, uint32_t& b) {
    // sign, and exponent and fraction moved to their places, are the value times 2^(7 - 127)
    const __nv_bfloat162 up = __bfloat162bfloat162(__ushort_as_bfloat16(0x7B80));  // 2^120
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t h = __byte_perm(w, 0u, i == 0 ? 0x1404 : 0x3424);
        const uint32_t x = ((h >> 4) & 0x07F007F0u) | (h & 0x80008000u);
        const __nv_bfloat162 r = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&x), up);
        (i == 0 ? a : b) = *reinterpret_cast<const uint32_t*>(&r);
    }
}

// Where 16-byte chunk c of row r lies in a group's tile: chunks are permuted so
// that what one shared-memory phase serves (K: two rows of four chunks; V: one
// chunk of eight rows) lies in different banks.
template <int D> __device__ __forceinline__ uint32_t k_at(uint32_t r, uint32_t c) {
    return r * D + ((D >= 128 ? c ^ ((r & 1) << 2) : c) << 4);
}
template <int D> __device__ __forceinline__ uint32_t v_at(uint32_t r, uint32_t c) {
    if (D >= 128) return r * D + ((c ^ (r & 7)) << 4);
    return (r >> 1) * 128 + (((((r & 1) << 2) | c) ^ ((r >> 1) & 3)) << 4);
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool take) {
    const int n = take ? 16 : 0;  // 0: the 16 bytes become zeros
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
    return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
    return v;
}

// Queries before position 0 see nothing.  They are all taken to be at -1, so that
// no position less a window leaves 32 bits.
__device__ __forceinline__ int position(int p) { return max(p, -1); }

// The keys [first, last] that a thread block's rows may see, from their
// positions; first is rounded down to a step.
struct Range {
    int first, end;  // end: one past the last key
};
__device__ __forceinline__ Range key_range(int lo_pos, int hi_pos, int len, int window) {
    Range r;
    r.first = window ? max(0, lo_pos - window + 1) / kStepKeys * kStepKeys : 0;
    r.end = min(hi_pos + 1, len);
    return r;
}

// Rows [rows x tile, ...) of sequence seq: shared by the kernel and the join.
struct Tile {
    int seq, h, row0, n_rows, q0, len, start;
    Range keys;
};
__device__ __forceinline__ bool tile_of(const KvAttnArgs& a, int rows, int tile, int h, int seq, Tile& t) {
    const int G = a.n_q_heads / a.n_kv_heads;
    t.seq = seq;
    t.h = h;
    t.q0 = a.b.cu[seq];
    const int qn = a.b.cu[seq + 1] - t.q0;
    t.row0 = tile * rows;
    t.n_rows = min(rows, qn * G - t.row0);
    if (t.n_rows <= 0) return false;
    t.len = a.b.kv_lens[seq];
    t.start = t.len - qn;
    const long long cap = static_cast<long long>(a.b.pages_per_seq) * a.page_size;
    if (t.len > cap) t.len = static_cast<int>(cap);
    t.keys = key_range(position(t.start + t.row0 / G), position(t.start + (t.row0 + t.n_rows - 1) / G), t.len, a.window);
    return true;
}

using Split = KvSplit;

// Four channels of a row of the output.
template <typename T, int D>
__device__ __forceinline__ void store_row(const KvAttnArgs& a, const Tile& t, int row, int d, float4 x, float f) {
    const int G = a.n_q_heads / a.n_kv_heads;
    T* out = static_cast<T*>(a.out) + (static_cast<size_t>(t.q0 + row / G) * a.n_q_heads + t.h * G + row % G) * D + d;
    if (sizeof(T) == 4)
        *reinterpret_cast<float4*>(out) = make_float4(x.x * f, x.y * f, x.z * f, x.w * f);
    else
        *reinterpret_cast<uint2*>(out) = make_uint2(pack_bf16_pair(x.x * f, x.y * f), pack_bf16_pair(x.z * f, x.w * f));
}

template <typename T, int D, int NQ> struct Cfg {
    static constexpr bool kPair = sizeof(T) == 4;     // fp32 activations: queries as pairs
    static constexpr int kTerms = kPair ? 3 : 2;      // bf16 terms of a weight
    static constexpr int kJoinPitch = D + 4;          // floats of a row of the warps' results
    static constexpr int kRows = 8 * NQ;
    static constexpr int kTile = kGroup * D;          // one group's K (or V) codes
    static constexpr int kStages = D == 256 ? 2 : D == 128 ? 3 : 4;
    static constexpr int kQPitch = D + 16;            // f16 elements
    static constexpr int kRing = kWarps * kStages * 2 * kTile;
    static constexpr int kJoin = kWarps * kRows * kJoinPitch * 4;  // the warps' results, after the ring's use
    static constexpr int kData = kRing > kJoin ? kRing : kJoin;
    static constexpr int kQ = kRows * kQPitch * 2 * (kPair ? 2 : 1);
    static constexpr int kLook = kWarps * kSpan * 16;
    static constexpr int kSmem = kData + kQ + kLook + (kRows + 2 * kWarps * kRows) * 4;
    // thread blocks of an SM that the registers are planned for
    static constexpr int kBlocks = D * NQ <= 128 ? 4 : D * NQ <= 256 ? 3 : 2;
};

template <typename T, typename F, int D, int NQ>
__global__ void __launch_bounds__(kThreads, Cfg<T, D, NQ>::kBlocks)
kv_attn_kernel(const KvAttnArgs a, const Split sp, const int n_tiles) {
    using C = Cfg<T, D, NQ>;
    constexpr int S = C::kStages, R = C::kRows;
    constexpr int MT = D / 16;              // 16-channel tiles of the output
    constexpr int CH = NQ == 1 ? 2 : 1;     // accumulators a score is spread over
    extern __shared__ __align__(128) uint8_t smem[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t4 = lane & 3;
    const int tile = blockIdx.x % n_tiles, split = blockIdx.x / n_tiles;
    const int G = a.n_q_heads / a.n_kv_heads;
    Tile t;
    if (!tile_of(a, R, tile, blockIdx.y, blockIdx.z, t)) return;
    if (tid == 0 && t.len < a.b.kv_lens[t.seq]) atomicMax(a.error, kKvErrTable);
    const int begin = t.keys.first + split * sp.chunk;
    const int end = split == sp.n - 1 ? t.keys.end : min(t.keys.end, begin + sp.chunk);
    if (split > 0 && begin >= end) return;  // the join does not read this one

    __half* q_hi = reinterpret_cast<__half*>(smem + C::kData);
    int* look_page = reinterpret_cast<int*>(smem + C::kData + C::kQ) + warp * kSpan;
    float* look_k = reinterpret_cast<float*>(smem + C::kData + C::kQ) + (kWarps + warp) * kSpan;
    float* look_lv = reinterpret_cast<float*>(smem + C::kData + C::kQ) + (2 * kWarps + warp) * kSpan;
    float* look_inv = reinterpret_cast<float*>(smem + C::kData + C::kQ) + (3 * kWarps + warp) * kSpan;
    float* q_scale = reinterpret_cast<float*>(smem + C::kData + C::kQ + C::kLook);
    float* part_m = q_scale + R;
    float* part_l = part_m + kWarps * R;

    // This warp's groups of a span: pages (one a lane), then the first copies, then the scales, so
    // that the codes of the first groups are on their way before anything else is waited for.
    const uint32_t ring = static_cast<uint32_t>(__cvta_generic_to_shared(smem)) + warp * S * 2 * C::kTile;
    const int n_steps = begin < end ? (end - begin + kStepKeys - 1) / kStepKeys : 0;
    const int min_pos = position(t.start + t.row0 / G);
    int steps = 0, key0 = 0;
    auto fetch = [&](int i) {
        if (i < steps) {
            const int key = key0 + i * kStepKeys, page = look_page[i];
            const size_t at = page < 0 ? 0 : ((static_cast<size_t>(page) * a.n_kv_heads + t.h) * a.page_size +
                                              key % a.page_size) * D;
            const uint32_t slot = ring + (i % S) * 2 * C::kTile;
            const uint8_t *ksrc = a.c.k + at + lane * 16, *vsrc = a.c.v + at + lane * 16;
            if (page >= 0 && key + kGroup <= end) {
#pragma unroll
                for (int c = 0; c < C::kTile / 16; c += 32) {
                    const uint32_t r = (c + lane) / (D / 16), cc = lane % (D / 16);
                    cp_async16(slot + k_at<D>(r, cc), ksrc + c * 16, true);
                    cp_async16(slot + C::kTile + v_at<D>(r, cc), vsrc + c * 16, true);
                }
            } else {  // rows past the end become zeros: what lies there may be no number
#pragma unroll
                for (int c = 0; c < C::kTile / 16; c += 32) {
                    const uint32_t r = (c + lane) / (D / 16), cc = lane % (D / 16);
                    const bool take = page >= 0 && key + static_cast<int>(r) < end;
                    cp_async16(slot + k_at<D>(r, cc), take ? ksrc + c * 16 : a.c.k, take);
                    cp_async16(slot + C::kTile + v_at<D>(r, cc), take ? vsrc + c * 16 : a.c.v, take);
                }
            }
        }
        cp_commit();
    };
    auto open_span = [&](int span) {
        steps = min(kSpan, n_steps - span);
        key0 = begin + span * kStepKeys + warp * kGroup;
        const int key = key0 + lane * kStepKeys;
        int page = -1;
        if (lane < steps && key < end) {
            page = a.b.table[static_cast<size_t>(t.seq) * a.b.pages_per_seq + key / a.page_size];
            if (a.window && key + kGroup - 1 <= min_pos - a.window) {
                // behind every row's window: what the entry points to may be another sequence's by
                // now, or no numbers
                page = -1;
            } else if (page < 0 || page >= a.c.n_pages) {
                atomicMax(a.error, kKvErrTable);
                page = -1;
            }
        }
        __syncwarp();
        look_page[lane] = page;
        __syncwarp();
#pragma unroll
        for (int i = 0; i < S - 1; ++i) fetch(i);
    };
    auto look_scales = [&]() {
        const int page = look_page[lane];
        float ks = 0.0f, vs = 1.0f;
        if (page >= 0) {
            const size_t block = static_cast<size_t>(page) * a.n_kv_heads + t.h;
            ks = a.c.k_scale[block];
            vs = a.c.v_scale[block];
        }
        const bool zero = zero_scale(vs);  // marked by a negative reciprocal
        if (zero) vs = 1.0f;
        look_k[lane] = ks;
        look_lv[lane] = log2f(vs);
        look_inv[lane] = (zero ? -1.0f : 1.0f) / vs;
        __syncwarp();
    };
    if (n_steps > 0) open_span(0);

    // Queries: 8 lanes a row, rounded to f16 under a power of two of the row.
    for (int r = tid >> 3; r < (R + 15) / 16 * 16; r += kThreads / 8) {
        constexpr int N = Vec16<T>::N, V = D / (8 * N);
        const int l8 = tid & 7, row = t.row0 + r;
        float x[V * N];
        float most = 0.0f;
        if (r < t.n_rows) {
            const T* src = static_cast<const T*>(a.q.data) + (t.q0 + row / G) * a.q.token_stride +
                           (t.h * G + row % G) * a.q.head_stride;
#pragma unroll
            for (int v = 0; v < V; ++v) Vec16<T>::load(src + (v * 8 + l8) * N, x + v * N);
        } else {
#pragma unroll
            for (int e = 0; e < V * N; ++e) x[e] = 0.0f;
        }
#pragma unroll
        for (int e = 0; e < V * N; ++e) most = fmaxf(most, fabsf(x[e]));
#pragma unroll
        for (int off = 4; off > 0; off >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, off));
        if (r >= R) continue;
        // the largest's exponent, and its powers of two
        const int ex = most > 0.0f && most <= 3.402823466e38f
                           ? min(max(static_cast<int>(__float_as_uint(most) >> 23) - 127, -100), 126) : 0;
        const float down = __uint_as_float(static_cast<uint32_t>(127 - ex) << 23);
        if (l8 == 0) q_scale[r] = a.scale * kLog2e * __uint_as_float(static_cast<uint32_t>(127 + ex) << 23);
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
            for (int e = 0; e < N; e += 2) {
                const int d = (v * 8 + l8) * N + e;
                const float lo = x[v * N + e] * down, hi = x[v * N + e + 1] * down;
                const uint32_t h = pack_f16(lo, hi);
                *reinterpret_cast<uint32_t*>(q_hi + r * C::kQPitch + d) = h;
                if (C::kPair) *reinterpret_cast<uint32_t*>(q_hi + (R + r) * C::kQPitch + d) = pack_f16_rest(h, lo, hi);
            }
    }
    __syncthreads();

    // B operand of 16 channels: channel order within 64 is (t4, step, 4), the order in which a lane
    // reads 16 codes of a key.
    const uint32_t q_base = static_cast<uint32_t>(__cvta_generic_to_shared(q_hi));
    auto load_q = [&](int step, int part, int nq) {
        const int d = (step >> 2) * 64 + 16 * t4 + 4 * (step & 3);
        return lds64(q_base + ((part * R + nq * 8 + g) * C::kQPitch + d) * 2);
    };
    uint2 qf[C::kPair ? 1 : D / 16][NQ];
    if (!C::kPair)
#pragma unroll
        for (int s = 0; s < D / 16; ++s)
#pragma unroll
            for (int n = 0; n < NQ; ++n) qf[C::kPair ? 0 : s][n] = load_q(s, 0, n);

    const int kr = 4 * (g >> 1) + (g & 1);  // this lane's keys of a group: kr, and kr + 2
    const int max_lo = a.window ? position(t.start + (t.row0 + t.n_rows - 1) / G) - a.window + 1 : 0;
    float o[MT][NQ][4];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int n = 0; n < NQ; ++n) o[i][n][0] = o[i][n][1] = o[i][n][2] = o[i][n][3] = 0.0f;
    float qs[NQ][2], m[NQ][2], l[NQ][2];
    bool fresh = true;  // nothing was added to o and l yet
#pragma unroll
    for (int n = 0; n < NQ; ++n)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            qs[n][c] = q_scale[8 * n + 2 * t4 + c];
            m[n][c] = -INFINITY;
            l[n][c] = 0.0f;
        }

    for (int span = 0; span < n_steps; span += kSpan) {
        if (span > 0) open_span(span);
        look_scales();
        for (int i = 0; i < steps; ++i) {
            if (S > 2) {  // the slot fetched into was read in the step before
                cp_wait<S - 2>();
                __syncwarp();
                fetch(i + S - 1);
            } else {
                __syncwarp();
                fetch(i + 1);
                cp_wait<1>();
                __syncwarp();
            }
            const int key = key0 + i * kStepKeys;
            if (key >= end || look_page[i] < 0) continue;
            const uint32_t kt = ring + (i % S) * 2 * C::kTile, vt = kt + C::kTile;

            float s[CH][NQ][4];
#pragma unroll
            for (int c = 0; c < CH; ++c)
#pragma unroll
                for (int n = 0; n < NQ; ++n) s[c][n][0] = s[c][n][1] = s[c][n][2] = s[c][n][3] = 0.0f;
#pragma unroll
            for (int j = 0; j < D / 64; ++j) {
                const uint4 w0 = lds128(kt + k_at<D>(kr, 4 * j + t4)), w1 = lds128(kt + k_at<D>(kr + 2, 4 * j + t4));
                const uint32_t x0[4] = {w0.x, w0.y, w0.z, w0.w}, x1[4] = {w1.x, w1.y, w1.z, w1.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    uint32_t f[4];
                    widen_f16<F>(x0[e], f[0], f[2]);
                    widen_f16<F>(x1[e], f[1], f[3]);
#pragma unroll
                    for (int n = 0; n < NQ; ++n) {
                        if (C::kPair) {
                            const uint2 lo = load_q(4 * j + e, 1, n), hi = load_q(4 * j + e, 0, n);
                            mma_f16(s[e % CH][n], f, lo.x, lo.y);
                            mma_f16(s[e % CH][n], f, hi.x, hi.y);
                        } else {
                            const uint2 b = qf[C::kPair ? 0 : 4 * j + e][n];
                            mma_f16(s[e % CH][n], f, b.x, b.y);
                        }
                    }
                }
            }
            const float ks = look_k[i], lv = look_lv[i], mark = look_inv[i], inv = fabsf(mark);
            const bool whole = key + kGroup - 1 <= min_pos && key >= max_lo && key + kGroup <= end;
            const float lazy = mark < 0.0f ? kLazy + kZeroLog : kLazy;
            bool lift = false;
            float top[NQ][2];
#pragma unroll
            for (int n = 0; n < NQ; ++n)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const float f = qs[n][c] * ks;
                    float v[2];
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        float x = s[0][n][2 * k + c];
                        if (CH > 1) x += s[CH - 1][n][2 * k + c];
                        v[k] = fmaf(x, f, lv);
                        if (!whole) {
                            const int j = key + kr + 2 * k, pos = position(t.start + (t.row0 + 8 * n + 2 * t4 + c) / G);
                            if (j > pos || j >= end || (a.window && j <= pos - a.window)) v[k] = -INFINITY;
                        }
                        s[0][n][2 * k + c] = v[k];
                    }
                    top[n][c] = fmaxf(v[0], v[1]);
                    lift |= top[n][c] > m[n][c] + lazy;
                }
            if (__any_sync(0xffffffffu, lift)) {
#pragma unroll
                for (int n = 0; n < NQ; ++n)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        float mn = top[n][c];
#pragma unroll
                        for (int off = 4; off < 32; off <<= 1) mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, off));
                        mn = fmaxf(m[n][c], mn - (lazy - kLazy));
                        const float by = m[n][c] == -INFINITY ? 0.0f : m[n][c] - mn;  // l and o are 0 with -inf
                        const float f = exp2_ftz(by);
                        m[n][c] = mn;
                        if (fresh) continue;
                        l[n][c] = times_pow2(l[n][c], by, f);
#pragma unroll
                        for (int i2 = 0; i2 < MT; ++i2) {
                            o[i2][n][c] *= f;
                            o[i2][n][2 + c] *= f;
                        }
                    }
                fresh = false;
            }
            float w[NQ][4];
            bool small = false;
#pragma unroll
            for (int n = 0; n < NQ; ++n)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const float ref = m[n][c] == -INFINITY ? 0.0f : m[n][c] - kBias;
                    small |= fminf(s[0][n][c], s[0][n][2 + c]) < ref + (kBias - kNormal);
                    w[n][c] = exp2_ftz(s[0][n][c] - ref);
                    w[n][2 + c] = exp2_ftz(s[0][n][2 + c] - ref);
                    l[n][c] = fmaf(w[n][c] + w[n][2 + c], inv, l[n][c]);
                }
            if (mark < 0.0f) continue;
            // output: 16-channel tile i holds channel 16 i + g in its first eight rows, + 8 in the others
            const uint32_t vrow = lane & 15, vchunk = lane >> 4;
            if (!C::kPair && !__any_sync(0xffffffffu, small)) {
                uint2 p[NQ];
#pragma unroll
                for (int n = 0; n < NQ; ++n)
                    p[n] = make_uint2(transpose8(pack_f16(w[n][0], w[n][1])), transpose8(pack_f16(w[n][2], w[n][3])));
#pragma unroll
                for (int i2 = 0; i2 < MT; i2 += 2) {
                    uint32_t x[4], f[2][4];
                    load_codes_t(vt + v_at<D>(vrow, i2 + vchunk), x);
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        widen_f16<F>(x[2 * k], f[k][0], f[k][2]);
                        widen_f16<F>(x[2 * k + 1], f[k][1], f[k][3]);
#pragma unroll
                        for (int n = 0; n < NQ; ++n) mma_f16(o[i2 + k][n], f[k], p[n].x, p[n].y);
                    }
                }
            } else {
                uint2 p[C::kTerms][NQ];
#pragma unroll
                for (int n = 0; n < NQ; ++n)
#pragma unroll
                    for (int k = 0; k < C::kTerms; ++k) {
                        const uint32_t u = pack_bf16_pair(w[n][0], w[n][1]), v = pack_bf16_pair(w[n][2], w[n][3]);
                        w[n][0] -= bf16_low(u);
                        w[n][1] -= bf16_high(u);
                        w[n][2] -= bf16_low(v);
                        w[n][3] -= bf16_high(v);
                        p[k][n] = make_uint2(transpose8(u), transpose8(v));
                    }
#pragma unroll
                for (int i2 = 0; i2 < MT; i2 += 2) {
                    uint32_t x[4], f[2][4];
                    load_codes_t(vt + v_at<D>(vrow, i2 + vchunk), x);
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        widen_bf16<F>(x[2 * k], f[k][0], f[k][2]);
                        widen_bf16<F>(x[2 * k + 1], f[k][1], f[k][3]);
#pragma unroll
                        for (int e = C::kTerms - 1; e >= 0; --e)
#pragma unroll
                            for (int n = 0; n < NQ; ++n) mma_bf16(o[i2 + k][n], f[k], p[e][n].x, p[e][n].y);
                    }
                }
            }
        }
        cp_wait<0>();
    }

    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    // Join the four warps: rows' references and sums, then the scaled outputs through shared memory.
#pragma unroll
    for (int n = 0; n < NQ; ++n)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
#pragma unroll
            for (int off = 4; off < 32; off <<= 1) l[n][c] += __shfl_xor_sync(0xffffffffu, l[n][c], off);
            if (g == 0) {
                part_m[warp * R + 8 * n + 2 * t4 + c] = m[n][c];
                part_l[warp * R + 8 * n + 2 * t4 + c] = l[n][c];
            }
        }
    __syncthreads();
    float* row_l = q_scale;  // the rows' sums
    if (tid < R) {
        float top = -INFINITY, sum = 0.0f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) top = fmaxf(top, part_m[w * R + tid]);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float mw = part_m[w * R + tid], by = mw == -INFINITY ? 0.0f : mw - top;
            sum += times_pow2(part_l[w * R + tid], by, exp2_ftz(by));
        }
        row_l[tid] = sum;
    }
    float* all = reinterpret_cast<float*>(smem);  // [warp][row][kJoinPitch]
#pragma unroll
    for (int n = 0; n < NQ; ++n)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            const int row = 8 * n + 2 * t4 + c;
            float top = -INFINITY;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) top = fmaxf(top, part_m[w * R + row]);
            const float f = m[n][c] == -INFINITY ? 0.0f : exp2_ftz(m[n][c] - top);
            float* dst = all + (warp * R + row) * C::kJoinPitch + g;
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                dst[16 * i] = o[i][n][c] * f;
                dst[16 * i + 8] = o[i][n][2 + c] * f;
            }
        }
    __syncthreads();
    const size_t unit = ((static_cast<size_t>(t.seq) * a.n_kv_heads + t.h) * n_tiles + tile) * sp.n + split;
    float* part = a.partial + unit * R * (D + 2);
    for (int i = tid; i < t.n_rows * (D / 4); i += kThreads) {
        const int row = i / (D / 4), d = (i % (D / 4)) * 4;
        float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float4 v = *reinterpret_cast<const float4*>(all + (w * R + row) * C::kJoinPitch + d);
            x.x += v.x; x.y += v.y; x.z += v.z; x.w += v.w;
        }
        const float sum = row_l[row];
        if (sp.n > 1) {
            *reinterpret_cast<float4*>(part + row * D + d) = x;
            if (d == 0) {
                float top = -INFINITY;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) top = fmaxf(top, part_m[w * R + row]);
                part[R * D + row] = top;
                part[R * D + R + row] = sum;
            }
        } else {
            store_row<T, D>(a, t, t.row0 + row, d, x, sum > 0.0f ? 1.0f / sum : 0.0f);
        }
    }
}

// Joins the splits of a row: out = sum_s O_s 2^(m_s - m) / sum_s l_s 2^(m_s - m).
// 16 lanes take 64 channels of a row; GROUPS such groups share one row's splits,
// at most kJoinEach each, all loaded before any is used.  Launched as the main
// kernel's programmatic dependent: it waits for that kernel's results before it
// reads any.
constexpr int kJoinLanes = 16, kJoinCols = 4 * kJoinLanes, kJoinEach = 8;
template <int GROUPS> constexpr int kJoinThreads = GROUPS * kJoinLanes < 256 ? 256 : GROUPS * kJoinLanes;
template <typename T, int D, int GROUPS>
__global__ void __launch_bounds__(kJoinThreads<GROUPS>)
kv_attn_join(const KvAttnArgs a, const Split sp, const int rows, const int n_tiles) {
    constexpr int kUnits = kJoinThreads<GROUPS> / (kJoinLanes * GROUPS);  // (row, 64 channels) of a thread block
    const int lane = threadIdx.x % kJoinLanes, grp = threadIdx.x / kJoinLanes % GROUPS;
    const int here = threadIdx.x / (kJoinLanes * GROUPS), at = blockIdx.x * kUnits + here;
    const int r = at / (D / kJoinCols), tile = r / rows, row = r % rows;
    Tile t;
    const bool mine = tile < n_tiles && tile_of(a, rows, tile, blockIdx.y, blockIdx.z, t) && row < t.n_rows;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int span = mine ? t.keys.end - t.keys.first : 0;
    const int n = mine ? max(1, min(sp.n, (span + sp.chunk - 1) / sp.chunk)) : 0;
    const size_t unit = mine ? ((static_cast<size_t>(t.seq) * a.n_kv_heads + t.h) * n_tiles + tile) * sp.n : 0;
    const size_t next = static_cast<size_t>(rows) * (D + 2);
    const float* part = a.partial + unit * next;
    const int d = at % (D / kJoinCols) * kJoinCols + 4 * lane;
    float ms[kJoinEach], ls[kJoinEach], top = -INFINITY;
    float4 vs[kJoinEach];
#pragma unroll
    for (int k = 0; k < kJoinEach; ++k) {
        const int s = grp + GROUPS * k;
        ms[k] = -INFINITY;
        ls[k] = 0.0f;
        vs[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (s < n) {
            ms[k] = part[s * next + rows * D + row];
            ls[k] = part[s * next + rows * D + rows + row];
            vs[k] = *reinterpret_cast<const float4*>(part + s * next + row * D + d);
        }
    }
#pragma unroll
    for (int k = 0; k < kJoinEach; ++k) top = fmaxf(top, ms[k]);
    float sum = 0.0f, low = 0.0f;
    float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
    for (int k = 0; k < kJoinEach; ++k) {
        const float by = ms[k] == -INFINITY ? 0.0f : ms[k] - top;  // its outputs and sum are 0 with -inf
        const float c = exp2_ftz(by);
        low = fminf(low, by);
        sum += ls[k] * c;
        x.x += vs[k].x * c; x.y += vs[k].y * c; x.z += vs[k].z * c; x.w += vs[k].w * c;
    }
    if (low < -100.0f) {  // factors that are flushed where their products need not be
        sum = 0.0f;
#pragma unroll
        for (int k = 0; k < kJoinEach; ++k) {
            const float by = ms[k] == -INFINITY ? 0.0f : ms[k] - top;
            sum += times_pow2(ls[k], by, exp2_ftz(by));
        }
    }
    if (GROUPS > 1) {
        __shared__ float sm[kUnits][GROUPS], sl[kUnits][GROUPS];
        __shared__ float4 sx[kUnits][GROUPS][kJoinLanes];
        sx[here][grp][lane] = x;
        if (lane == 0) {
            sm[here][grp] = top;
            sl[here][grp] = sum;
        }
        __syncthreads();
        if (grp != 0) return;
#pragma unroll
        for (int w = 0; w < GROUPS; ++w) top = fmaxf(top, sm[here][w]);
        sum = 0.0f;
        x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 8
        for (int w = 0; w < GROUPS; ++w) {
            const float by = sm[here][w] == -INFINITY ? 0.0f : sm[here][w] - top, c = exp2_ftz(by);
            const float4 v = sx[here][w][lane];
            low = fminf(low, by);
            sum += sl[here][w] * c;
            x.x += v.x * c; x.y += v.y * c; x.z += v.z * c; x.w += v.w * c;
        }
        if (low < -100.0f) {
            sum = 0.0f;
            for (int w = 0; w < GROUPS; ++w) {
                const float by = sm[here][w] == -INFINITY ? 0.0f : sm[here][w] - top;
                sum += times_pow2(sl[here][w], by, exp2_ftz(by));
            }
        }
    }
    if (mine) store_row<T, D>(a, t, t.row0 + row, d, x, sum > 0.0f ? 1.0f / sum : 0.0f);
}

template <typename T, int D, int GROUPS>
cudaError_t join_t(const KvAttnArgs& a, const Split sp, int rows, int n_tiles, cudaStream_t st) {
    constexpr int kUnits = kJoinThreads<GROUPS> / (kJoinLanes * GROUPS);
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((n_tiles * rows * (D / kJoinCols) + kUnits - 1) / kUnits, a.n_kv_heads, a.b.n_seq);
    cfg.blockDim = dim3(kJoinThreads<GROUPS>);
    cfg.stream = st;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kv_attn_join<T, D, GROUPS>, a, sp, rows, n_tiles);
}

template <typename T, int D>
cudaError_t join_d(const KvAttnArgs& a, const Split& sp, int rows, int n_tiles, cudaStream_t st) {
    return timed_launch("kv_attn_join", st, [&] {
        return sp.n <= kJoinEach       ? join_t<T, D, 1>(a, sp, rows, n_tiles, st)
               : sp.n <= 4 * kJoinEach ? join_t<T, D, 4>(a, sp, rows, n_tiles, st)
                                       : join_t<T, D, 32>(a, sp, rows, n_tiles, st);
    });
}

// Rows of a thread block: the fewest tiles of 8 that hold a sequence's rows,
// as far as the output's registers (D / 16 x 4 x NQ a lane, at most 128) allow.
int tiles_of_8(int head_dim, long long rows) {
    const int most = head_dim == 256 ? 2 : 4;
    return rows <= 8 ? 1 : rows <= 16 || most == 2 ? 2 : 4;
}

// How many ranges the keys are split into.  Several rounds of thread blocks over
// the SMs' 456 places even out ragged lengths, but a range's fixed cost (its
// queries, its partial result) counts from about 16 thread blocks an SM on: 256
// sequences of 127..8191 keys, head_dim 256, take 224 / 196 / 195 us at 1024 /
// 2048 / 4096 blocks, 64 x 4 drafts of head_dim 128 118 / 107 / 118 us.  One
// sequence is split down to one step a warp (1000 keys: 7.3 us; 9.3 us at 128 keys
// a range), 131,000 keys into half a round (31 us; 36 us at 76 ranges).
constexpr int kMinChunk = kStepKeys;
constexpr long long kTargetBlocks = 152 * 16, kMostSplits = 228;
static_assert(kMostSplits <= 32 * kJoinEach, "the join holds this many splits");
Split split_of(int rows, int n_seq, int max_q, int n_q_heads, int n_kv_heads, int window, long long max_kv_len) {
    const int G = n_q_heads / n_kv_heads;
    const long long tiles = (static_cast<long long>(max_q) * G + rows - 1) / rows;
    const long long units = std::max(1LL, tiles * n_kv_heads * n_seq);
    long long span = std::max(1LL, max_kv_len);
    if (window) span = std::min(span, static_cast<long long>(window) + max_q + kStepKeys);
    long long n = std::min((kTargetBlocks + units - 1) / units, (span + kMinChunk - 1) / kMinChunk);
    n = std::max(1LL, std::min(n, kMostSplits));
    long long chunk = (span + n - 1) / n;
    chunk = (chunk + kStepKeys - 1) / kStepKeys * kStepKeys;
    return Split{static_cast<int>((span + chunk - 1) / chunk), static_cast<int>(chunk)};
}

template <typename T, typename F, int D, int NQ>
cudaError_t attn_nq(const KvAttnArgs& a, cudaStream_t st) {
    using C = Cfg<T, D, NQ>;
    const int G = a.n_q_heads / a.n_kv_heads;
    const Split sp = split_of(C::kRows, a.b.n_seq, a.b.max_q, a.n_q_heads, a.n_kv_heads, a.window, a.max_kv_len);
    const long long tiles = (static_cast<long long>(a.b.max_q) * G + C::kRows - 1) / C::kRows;
    if (tiles * sp.n > 0x7fffffffLL / (C::kRows * (D / kJoinCols))) return cudaErrorInvalidConfiguration;
    static std::atomic<unsigned long long> ready{0};
    cudaError_t e = allow_smem(kv_attn_kernel<T, F, D, NQ>, C::kSmem, ready);
    if (e != cudaSuccess) return e;
    const int nt = static_cast<int>(tiles);
    e = timed_launch("kv_attn", st, [&] {
        kv_attn_kernel<T, F, D, NQ><<<dim3(nt * sp.n, a.n_kv_heads, a.b.n_seq), kThreads, C::kSmem, st>>>(a, sp, nt);
        return cudaGetLastError();
    });
    if (e != cudaSuccess || sp.n == 1) return e;
    return join_d<T, D>(a, sp, C::kRows, nt, st);
}

template <typename T, typename F, int D>
cudaError_t attn_t(const KvAttnArgs& a, cudaStream_t st) {
    switch (tiles_of_8(D, static_cast<long long>(a.b.max_q) * (a.n_q_heads / a.n_kv_heads))) {
        case 1: return attn_nq<T, F, D, 1>(a, st);
        case 2: return attn_nq<T, F, D, 2>(a, st);
        default: return attn_nq<T, F, D, D == 256 ? 2 : 4>(a, st);
    }
}

}  // namespace

size_t kv_attention_workspace(int n_seq, int max_q, int n_q_heads, int n_kv_heads, int head_dim, int window, bool bf16,
                              int max_kv_len) {
    if (max_q == 0) return 0;
    const KvPrompt p = kv_prompt_plan(n_seq, max_q, n_q_heads, n_kv_heads, head_dim, window, bf16, max_kv_len);
    const auto bytes_of = [&](size_t tiles, int n, size_t rows) {
        const size_t bytes = n == 1 ? 0 : tiles * n_kv_heads * n_seq * n * rows * (head_dim + 2) * sizeof(float);
        return (bytes + 255) & ~static_cast<size_t>(255);
    };
    if (p.tiles > 0) return bytes_of(p.tiles, p.split.n, p.rows);
    const long long all = static_cast<long long>(max_q) * (n_q_heads / n_kv_heads);
    const int rows = 8 * tiles_of_8(head_dim, all);
    const Split sp = split_of(rows, n_seq, max_q, n_q_heads, n_kv_heads, window, max_kv_len);
    return bytes_of((all + rows - 1) / rows, sp.n, rows);
}

cudaError_t launch_kv_join(const KvAttnArgs& a, const KvSplit& split, int rows, int tiles, int head_dim,
                           cudaStream_t stream) {
    return head_dim == 64    ? join_d<__nv_bfloat16, 64>(a, split, rows, tiles, stream)
           : head_dim == 128 ? join_d<__nv_bfloat16, 128>(a, split, rows, tiles, stream)
                             : join_d<__nv_bfloat16, 256>(a, split, rows, tiles, stream);
}

cudaError_t launch_kv_attention(const KvAttnArgs& a, int head_dim, bool bf16, bool e4m3, cudaStream_t stream) {
    const KvPrompt p = kv_prompt_plan(a.b.n_seq, a.b.max_q, a.n_q_heads, a.n_kv_heads, head_dim, a.window, bf16, a.max_kv_len);
    if (p.tiles > 0) return launch_kv_prompt(a, p, head_dim, e4m3, stream);
    return GDN_KV_PICK(attn_t);
}

}  // namespace gdn
