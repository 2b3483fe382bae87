// Causal attention over the paged 8-bit cache, many query rows (prompts) of
// bf16 activations, on the 5th-generation tensor cores.
//
// The mathematics is that of gdn_kv_attn.cu: products of the codes, block
// scales outside of them,
//   y_rj = (q_r . ck_j) scale s_k log2 e + log2 s_v,   w_rj = 2^(y_rj - m_r)
//   o_r = sum_j w_rj cv_j / sum_blk (sum_j w_rj) / s_v
// with a reference m_r that lags behind the maximum by at most 2^kLazy.  All
// operands are f16: codes exactly, queries exactly from 2^-17 of a row's largest
// up (below, to 2^-25 of it), weights (times 2^kBias) with 11 bits; weights below
// 2^-31 of the reference are dropped.
//
// One thread block takes one 128-row tile (head_dim 256), or two, of the rows
// (token, head of the group) of a sequence and kv head, and walks its keys in
// tiles of 64.  Roles:
//   8 softmax warps      a thread a row, two groups of four warps: a row tile
//                        each, or (head_dim 256) 32 of the tile's keys each,
//                        agreeing on the reference; scores from tensor memory,
//                        weights back to it as f16, rescaling of the output
//                        when the reference moves, the epilogue
//   4 + 4 converter      codes of K, of V, from global memory (prefetched two
//     warps              tiles ahead in registers) to f16 operand tiles in
//                        shared memory, three buffers each; V needs no
//                        transpose, its operand is MN-major
//   2 look-up warps      pages to where the tiles ahead lie, for the converters,
//                        and pages' scales to block constants, for the softmax
//   2 issuing warps      S = Q K^T, a tile ahead, and O += P V: one of them
//                        waits and fences while the other's products run
// Tensor memory (512 columns): a score tile of 64 columns a row tile, read into
// registers at once so that the next one can follow; two tiles of weights, f16,
// 32 columns each; the output; at head_dim 256 the queries too.  The operands
// that stay (P, and Q of head_dim 256) are there to spare shared memory, which
// at head_dim 256 moves 64 KB of converted codes in and 64 KB out a tile, 1024
// cycles at 128 bytes, as long as the tile's products take; with Q and P in
// shared memory it was 224 KB.
// The converted tiles are written by ordinary stores and read by the tensor
// core: an issuing thread, which has waited for the writers, fences the one
// against the other (a writer's fence would also wait for its loads in flight).
// What bounds it: no unit is saturated, the chain of waits between the roles is.
// A prompt of 4096 tokens (16 heads of 256) takes 133 us, 1.03 PFLOP/s over the
// visible pairs: 1.2 us a tile and SM, of which the products need 1024 cycles
// (tensor pipe 42% busy, issue slots 58%).  16 ragged prompts with a window (32
// heads of 128) take 307 us, 0.68 PFLOP/s (30%, 48%); each thread block there
// also walks fewer keys per start.  Tiles of 128 keys were slower when tried, on
// an earlier form of this kernel: 226 and 609 us, against 222 and 507.
// Every wait is bounded (2 s); a wait that gives up records a code (42..48) in
// the cache operators' device error word and its role stops.
#include <algorithm>

#include "gdn_internal.h"
#include "gdn_kv.cuh"
#include "gdn_tc.cuh"

namespace gdn {

using namespace tc;

namespace {

// The largest code stays.  A call of its own: in line the atomics take registers where nothing fails
// (16 windowed prompts of 32 heads of 128: 317 us in line, 308 us so; a prompt of 4096 tokens 135 us both).

constexpr int kM = 128, kKeys = 64;
constexpr int kGroups = kKeys / 16;  // 16-key groups of a tile: one page each
constexpr int kPass = 32 / kGroups;  // tiles that a look-up warp looks up at a time
constexpr int kStages = 3;           // buffers of K tiles, and of V tiles
constexpr int kSoftWarps = 8, kConvWarps = 4;  // softmax; K's converters, and V's
constexpr int kThreads = 32 * (kSoftWarps + 2 * kConvWarps + 4);
constexpr float kLazy = 8.0f;
constexpr float kBias = 7.0f;        // weights are 2^7 times theirs: at most 2^15

template <int D> struct PCfg {
    static constexpr int kTiles = D == 256 ? 1 : 2;       // row tiles of a thread block
    static constexpr int kHalves = 3 - kTiles;            // softmax threads a row
    static constexpr int kCols = kKeys / kHalves;         // keys of a softmax thread
    static constexpr bool kQInTmem = D == 256;
    static constexpr uint32_t kQ = kM * D * 2, kTile = kKeys * D * 2;  // bytes: a row tile's queries, a K or V tile
    // K tiles, V tiles, then queries; those of tensor memory only pass through K's buffers
    static constexpr uint32_t kData = 2 * kStages * kTile + (kQInTmem ? 0 : kTiles * kQ), kSmem = kData + 4096;
    // tensor memory columns: scores, weights (two tiles a row tile), output, queries
    static constexpr uint32_t kWeights = kTiles * kKeys, kOut = 2 * kWeights, kQCol = kOut + kTiles * D;
};

// Instruction descriptor, kind::f16: f16 A and B, fp32 accumulator.
__host__ __device__ constexpr uint32_t idesc_f16_f32(int M, int N, bool b_mn) {
    return (1u << 4) | ((b_mn ? 1u : 0u) << 16) | (static_cast<uint32_t>(N >> 3) << 17) |
           (static_cast<uint32_t>(M >> 4) << 24);
}

// 32 lanes x N columns of 32-bit, registers to tensor memory.
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* v) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::"r"(v[0]),
        "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]), "r"(v[10]),
        "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t* v) {
    tmem_st16(taddr, v);
    tmem_st16(taddr + 16, v + 16);
}

// D[tmem] (+)= A[tmem] * B[smem]^T, f16, issued by one thread.  A: lane = row,
// a column holds two consecutive K elements.
__device__ __forceinline__ void mma_f16_ta(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                           uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}


// Bulk copy shared -> global of `bytes` (a multiple of 16, both ends aligned),
// tracked by the issuing thread's bulk group.
__device__ __forceinline__ void bulk_store_1d(void* dst, const void* src, uint32_t bytes) {
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(smem_u32(src)), "r"(bytes)
                 : "memory");
}


// Block constants of one 16-key group: factor of the scores, their offset
// (log2 of the value scale), and its reciprocal (negative: values are zero).
struct GroupConst {
    float ks, lv, inv;
};

struct Shared {
    uint64_t q_full, q_staged, k_full[kStages], k_empty[kStages], v_full[kStages], v_empty[kStages];
    uint64_t s_full[2], s_empty[2], p_full[2][2], pv_done[2][2];  // of a row tile (and a buffer of weights)
    uint64_t c_full[2], c_empty[2];  // halves of consts
    uint64_t l_full[2], l_empty[2];  // halves of place
    uint64_t o_full;
    GroupConst consts[2 * kPass][kGroups];
    long long place[2 * kPass][kGroups];  // a group's first code in the cache, or -1
    float swap[2][kM];  // a row's two threads: maxima, sums
    uint32_t tmem_slot;
};
static_assert(sizeof(Shared) <= 4096, "part of kSmem");


// A row tile's queries as they are (bf16; zeros past the last row) by THREADS
// threads into a swizzled tile of kM rows in blocks of 64 channels.
template <int D, int THREADS>
__device__ __forceinline__ void fetch_queries(const KvAttnArgs& a, uint8_t* tile, int row0, int n_rows, int q0, int h, int G,
                                              int tid) {
    constexpr int V = D / 8, STEP = THREADS / V;  // 16-byte vectors of a row; rows at a time
    const int c = tid % V;
    const uint32_t base = smem_u32(tile) + (c / 8) * (kM * 128);
    const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q.data) + 8 * c;
#pragma unroll 4
    for (int r = tid / V; r < kM; r += STEP) {
        const int row = row0 + r;
        const bool take = r < n_rows;
        const __nv_bfloat16* src = q + (q0 + row / G) * a.q.token_stride + (h * G + row % G) * a.q.head_stride;
        cp_async16(base + sw128_offset(r, c % 8), take ? src : q, take);
    }
    asm volatile("cp.async.commit_group;\n\tcp.async.wait_group 0;" ::: "memory");
}
// The exponent under which a row whose largest magnitude is `most` is rounded to f16.
__device__ __forceinline__ int row_exponent(float most) {
    return most > 0.0f && most <= 3.402823466e38f ? min(max(static_cast<int>(__float_as_uint(most) >> 23) - 127, -100), 126) : 0;
}
__device__ __forceinline__ float pow2(int e) { return __uint_as_float(static_cast<uint32_t>(127 + e) << 23); }
__device__ __forceinline__ float most_of(uint4 v, float most) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        most = fmaxf(most, fmaxf(fabsf(__uint_as_float(w[i] << 16)), fabsf(__uint_as_float(w[i] & 0xFFFF0000u))));
    return most;
}
__device__ __forceinline__ uint32_t scaled_f16(uint32_t bf16_pair, float f) {
    return pack_f16(__uint_as_float(bf16_pair << 16) * f, __uint_as_float(bf16_pair & 0xFFFF0000u) * f);
}

// SPLIT: the keys are split, and results are partial ones for the join.  A kernel
// of its own: with both in one the 4096-token prompt took 134 us instead of 131.
template <typename F, int D, bool SPLIT>
__global__ void __launch_bounds__(kThreads, 1) kv_prompt_kernel(const KvAttnArgs a, const KvSplit sp) {
    using C = PCfg<D>;
    constexpr int NT = C::kTiles, NC = C::kCols;
    extern __shared__ __align__(1024) uint8_t smem[];  // the swizzled tiles start on 1024-byte boundaries
    Shared& sh = *reinterpret_cast<Shared*>(smem + C::kData);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int seq = blockIdx.y, h = blockIdx.x, G = a.n_q_heads / a.n_kv_heads;
    const int q0 = a.b.cu[seq], qn = a.b.cu[seq + 1] - q0;
    const int block_tile = (static_cast<int>(gridDim.z) - 1 - static_cast<int>(blockIdx.z)) / (SPLIT ? sp.n : 1);  // most keys first
    const int split = SPLIT ? static_cast<int>(blockIdx.z) % sp.n : 0, row0 = block_tile * (NT * kM);
    const int n_rows = min(NT * kM, qn * G - row0);
    if (n_rows <= 0) return;
    int len = a.b.kv_lens[seq];
    const int start = len - qn;  // position of the call's first query
    const long long cap = static_cast<long long>(a.b.pages_per_seq) * a.page_size;
    if (len > cap) {
        if (tid == 0) record(a.error, kKvErrTable);
        len = static_cast<int>(cap);
    }
    // positions; queries before 0, which see nothing, are all taken to be at -1, so that no position less
    // a window leaves 32 bits
    const int lo_pos = max(start + row0 / G, -1), hi_pos = max(start + (row0 + n_rows - 1) / G, -1);
    // this thread block's range of the keys; the join does not read an empty one past the first
    const int all_first = a.window ? max(0, lo_pos - a.window + 1) / kKeys * kKeys : 0;
    const int span = max(0, min(hi_pos + 1, len) - all_first), from = SPLIT ? split * sp.chunk : 0;
    if (SPLIT && split > 0 && from >= span) return;
    const int first = all_first + from, end = all_first + (!SPLIT || split == sp.n - 1 ? span : min(span, from + sp.chunk));
    const int n_tiles = end > first ? (end - first + kKeys - 1) / kKeys : 0;
    const int active = n_rows > kM ? NT : 1;  // row tiles with rows

    if (smem_u32(smem) & 1023u) {
        if (tid == 0) record(a.error, 48);
        return;
    }
    uint8_t* sk = smem;
    uint8_t* sv = sk + kStages * C::kTile;
    uint8_t* sq = C::kQInTmem ? nullptr : sv + kStages * C::kTile;

    const int soft = C::kHalves == 2 ? kSoftWarps : 4 * active;  // softmax warps at work
    if (tid == 0) {
        mbar_init(&sh.q_full, soft);
        mbar_init(&sh.q_staged, soft);
        mbar_init(&sh.o_full, 1);
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&sh.k_full[i], kConvWarps);
            mbar_init(&sh.v_full[i], kConvWarps);
            mbar_init(&sh.k_empty[i], 1);
            mbar_init(&sh.v_empty[i], 1);
        }
        for (int t = 0; t < 2; ++t) {
            mbar_init(&sh.s_full[t], 1);
            mbar_init(&sh.s_empty[t], C::kHalves == 2 ? kSoftWarps : 4);
            for (int i = 0; i < 2; ++i) {
                mbar_init(&sh.p_full[t][i], C::kHalves == 2 ? kSoftWarps : 4);
                mbar_init(&sh.pv_done[t][i], 1);
            }
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sh.c_full[i], 1);
            mbar_init(&sh.c_empty[i], soft);
            mbar_init(&sh.l_full[i], 1);
            mbar_init(&sh.l_empty[i], 2 * kConvWarps);
        }
        fence_barrier_init();
    }
    constexpr int kPlaceWarp = kSoftWarps + 2 * kConvWarps, kIssueWarp = kPlaceWarp + 2;  // one between: constants
    if (warp == kIssueWarp) tmem_alloc(&sh.tmem_slot, 512);
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = sh.tmem_slot;
    // groups of keys that end here or before are behind every row's window: their entries are not followed
    const int behind = a.window ? lo_pos - a.window : -1;
    auto page_of = [&](int key) {  // negative: past the end, behind, or not mapped
        if (key >= end || key + 15 <= behind) return -1;
        const int page = a.b.table[static_cast<size_t>(seq) * a.b.pages_per_seq + key / a.page_size];
        return page < a.c.n_pages ? page : -1;
    };

    if (warp < kSoftWarps) {
        const int grp = warp >> 2, t = C::kHalves == 2 ? 0 : grp;  // group of four warps; its row tile
        const int r = tid & (kM - 1);                              // row of the tile
        const uint32_t t_lane = (32u * (warp & 3)) << 16;
        const int tile_row0 = row0 + t * kM;
        if (t < active) {
            // ---- queries
            // A thread finds its row's (with a row's two threads: its half's) largest magnitude and rounds
            // the row to f16 under a power of two.
            float qs;
            if (C::kQInTmem) {  // through the first K buffers
                static_assert(!C::kQInTmem || 2 * C::kTile >= C::kQ, "two K buffers hold the queries");
                fetch_queries<D, 32 * kSoftWarps>(a, sk, row0, n_rows, q0, h, G, tid);
                group_sync(1, 32 * kSoftWarps);
                const uint8_t* src = sk + 2 * grp * (kM * 128);
                float most = 0.0f;
#pragma unroll
                for (int c = 0; c < 16; ++c)
                    most = most_of(*reinterpret_cast<const uint4*>(src + (c >> 3) * (kM * 128) + sw128_offset(r, c & 7)), most);
                sh.swap[grp][r] = most;
                group_sync(2, 32 * kSoftWarps);
                const int ex = row_exponent(fmaxf(most, sh.swap[grp ^ 1][r]));
                const float down = pow2(-ex);
                qs = a.scale * kLog2e * pow2(ex);
#pragma unroll 1
                for (int blk = 0; blk < 2; ++blk) {
                    uint32_t w[32];
#pragma unroll
                    for (int c = 0; c < 8; ++c) {
                        const uint4 v = *reinterpret_cast<const uint4*>(src + blk * (kM * 128) + sw128_offset(r, c));
                        w[4 * c] = scaled_f16(v.x, down);
                        w[4 * c + 1] = scaled_f16(v.y, down);
                        w[4 * c + 2] = scaled_f16(v.z, down);
                        w[4 * c + 3] = scaled_f16(v.w, down);
                    }
                    tmem_st32(tmem + t_lane + C::kQCol + 64 * grp + 32 * blk, w);
                }
                tmem_wait_st();
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&sh.q_staged);
                    mbar_arrive(&sh.q_full);
                }
            } else {
                uint8_t* tile = sq + t * C::kQ;
                fetch_queries<D, kM>(a, tile, tile_row0, n_rows - t * kM, q0, h, G, r);
                group_sync(1 + t, kM);
                float most = 0.0f;
#pragma unroll
                for (int c = 0; c < D / 8; ++c)
                    most = most_of(*reinterpret_cast<const uint4*>(tile + (c >> 3) * (kM * 128) + sw128_offset(r, c & 7)), most);
                const int ex = row_exponent(most);
                const float down = pow2(-ex);
                qs = a.scale * kLog2e * pow2(ex);
#pragma unroll 4
                for (int c = 0; c < D / 8; ++c) {
                    uint4* at = reinterpret_cast<uint4*>(tile + (c >> 3) * (kM * 128) + sw128_offset(r, c & 7));
                    const uint4 v = *at;
                    *at = make_uint4(scaled_f16(v.x, down), scaled_f16(v.y, down), scaled_f16(v.z, down), scaled_f16(v.w, down));
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh.q_full);
            }

            // ---- softmax: a thread's row, all keys of a tile or 32 of them
            const int pos = max(start + (tile_row0 + r) / G, -1);
            const int my_lo = start + tile_row0 / G;  // the row tile's first position
            const int max_lo = a.window ? hi_pos - a.window + 1 : 0;
            const uint32_t t_score = tmem + t_lane + t * kKeys + (C::kHalves == 2 ? grp * NC : 0);
            const uint32_t t_weight = tmem + t_lane + C::kWeights + t * kKeys + (C::kHalves == 2 ? grp * NC / 2 : 0);
            const uint32_t t_out = tmem + t_lane + C::kOut + t * D;
            float m = -INFINITY, l = 0.0f;
            bool ok = true;
            for (int i = 0; i < n_tiles; ++i) {
                const int key = first + i * kKeys + (C::kHalves == 2 ? grp * NC : 0), sb = i & 1;
                // A wait that gave up is not waited for again, but the warp goes on through the tiles
                // (with results that are invalid): the barriers between the warps stay complete.
                if (ok && !(ok = __all_sync(0xffffffffu, (i % kPass || mbar_wait_brief(&sh.c_full[i / kPass & 1], (i / (2 * kPass)) & 1)) &&
                                                             mbar_wait_brief(&sh.s_full[t], i & 1))) &&
                    lane == 0)
                    record(a.error, 42);
                tc_fence_after_sync();
                float s[NC];
                if (NC == 64) tmem_ld64(t_score, s);
                else tmem_ld32(t_score, s);
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh.s_empty[t]);  // the next tile's scores may come
                GroupConst gc[NC / 16];
#pragma unroll
                for (int g = 0; g < NC / 16; ++g) gc[g] = sh.consts[i % (2 * kPass)][(C::kHalves == 2 ? grp * (NC / 16) : 0) + g];
#pragma unroll
                for (int g = 0; g < NC / 16; ++g) {
                    const float f = qs * gc[g].ks, o = gc[g].lv;
                    const uint64_t f2 = pair(f, f), o2 = pair(o, o);
#pragma unroll
                    for (int j = 16 * g; j < 16 * g + 16; j += 2) unpair(fma2(pair(s[j], s[j + 1]), f2, o2), s[j], s[j + 1]);
                }
                if (!(key + NC - 1 <= my_lo && key >= max_lo && key + NC <= end)) {
                    const int hi = min(pos, end - 1) - key, lo = a.window ? pos - a.window + 1 - key : 0;
#pragma unroll
                    for (int j = 0; j < NC; ++j) s[j] = j > hi || j < lo ? -INFINITY : s[j];
                }
                float tops[4] = {s[0], s[1], s[2], s[3]};  // four chains
#pragma unroll
                for (int j = 4; j < NC; ++j) tops[j & 3] = fmaxf(tops[j & 3], s[j]);
                float top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
                // whether the reference of any row moves: of the warp, or of both threads of any row
                const bool lift = C::kHalves == 2 ? group_or(1, 32 * kSoftWarps, top > m + kLazy)
                                                  : __any_sync(0xffffffffu, top > m + kLazy);
                float f = 1.0f;
                if (lift) {
                    if (C::kHalves == 2) {
                        sh.swap[grp][r] = top;
                        group_sync(2, 32 * kSoftWarps);
                        top = fmaxf(top, sh.swap[grp ^ 1][r]);
                    }
                    const float mn = fmaxf(m, top);
                    const float by = m == -INFINITY ? 0.0f : m - mn;  // l and the output are 0 with -inf
                    const float half = exp2_ftz(0.5f * by);  // the sum's factor may lie below fp32's normal numbers
                    f = half * half;
                    m = mn;
                    l = l * half * half;
                }
                const float ref = m == -INFINITY ? 0.0f : m - kBias;
                uint32_t p[NC / 2];
#pragma unroll
                for (int g = 0; g < NC / 16; ++g) {
                    const float up = gc[g].inv < 0.0f ? kZeroLog - ref : -ref;
                    const uint64_t ref2 = pair(up, up);
                    uint64_t sums = 0;  // 0.0f twice
#pragma unroll
                    for (int j = 16 * g; j < 16 * g + 16; j += 2) {
                        float w0, w1;
                        unpair(add2(pair(s[j], s[j + 1]), ref2), w0, w1);
                        w0 = exp2_ftz(w0);
                        w1 = exp2_ftz(w1);
                        sums = add2(sums, pair(w0, w1));
                        p[j / 2] = pack_f16(w0, w1);
                    }
                    float s0, s1;
                    unpair(sums, s0, s1);
                    l = fmaf(s0 + s1, fabsf(gc[g].inv), l);
                    if (gc[g].inv < 0.0f) {  // values of a scale of 0: counted, not added
#pragma unroll
                        for (int j = 8 * g; j < 8 * g + 8; ++j) p[j] = 0;
                    }
                }
                // the buffer's last weights were used
                if (ok && i >= 2 &&
                    !(ok = __all_sync(0xffffffffu, mbar_wait_brief(&sh.pv_done[t][sb], ((i >> 1) - 1) & 1))) && lane == 0)
                    record(a.error, 43);
                tc_fence_after_sync();
                if (NC == 64) tmem_st32(t_weight + sb * (kKeys / 2), p);
                else tmem_st16(t_weight + sb * (kKeys / 2), p);
                if (lift && i > 0) {  // the output so far, once the products before this tile's are done
                    if (ok && !(ok = __all_sync(0xffffffffu, mbar_wait_brief(&sh.pv_done[t][sb ^ 1], ((i - 1) >> 1) & 1))) &&
                        lane == 0)
                        record(a.error, 43);
                    tc_fence_after_sync();
                    constexpr int W = D / C::kHalves;  // this thread's share of the row
#pragma unroll 1
                    for (int c = 0; c < W; c += 32) {
                        float v[32];
                        uint32_t u[32];
                        const uint32_t at = t_out + (C::kHalves == 2 ? grp * W : 0) + c;
                        tmem_ld32(at, v);
#pragma unroll
                        for (int e = 0; e < 32; ++e) u[e] = __float_as_uint(v[e] * f);
                        tmem_st32(at, u);
                    }
                }
                tmem_wait_st();
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&sh.p_full[t][sb]);
                    if (i % kPass == kPass - 1) mbar_arrive(&sh.c_empty[i / kPass & 1]);
                }
            }
            // ---- epilogue
            if (ok && n_tiles > 0 && !(ok = __all_sync(0xffffffffu, mbar_wait_brief(&sh.o_full, 0))) && lane == 0)
                record(a.error, 44);
            if (C::kHalves == 2) {  // the row's sum
                group_sync(1, 32 * kSoftWarps);
                sh.swap[grp][r] = l;
                group_sync(2, 32 * kSoftWarps);
                l += sh.swap[grp ^ 1][r];
            }
            if (ok) {
                tc_fence_after_sync();
                constexpr int W = D / C::kHalves;  // this thread's share of the row
                const int c0 = C::kHalves == 2 ? grp * W : 0, row = tile_row0 + r;
                if constexpr (SPLIT) {  // a partial result: unscaled outputs, reference and sum
                    constexpr int R = C::kTiles * kM;
                    float* part = a.partial + (((static_cast<size_t>(seq) * a.n_kv_heads + h) * (gridDim.z / sp.n) + block_tile) *
                                                   sp.n + split) * (static_cast<size_t>(R) * (D + 2));
                    const int rr = t * kM + r;
#pragma unroll 1
                    for (int c = 0; c < W; c += 32) {
                        float v[32];
                        if (n_tiles > 0) tmem_ld32(t_out + c0 + c, v);
                        if (rr < n_rows) {
#pragma unroll
                            for (int e = 0; e < 32; e += 4)
                                *reinterpret_cast<float4*>(part + static_cast<size_t>(rr) * D + c0 + c + e) =
                                    n_tiles > 0 ? make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]) : make_float4(0, 0, 0, 0);
                        }
                    }
                    if (rr < n_rows && c0 == 0) {
                        part[static_cast<size_t>(R) * D + rr] = m;
                        part[static_cast<size_t>(R) * D + R + rr] = l;
                    }
                } else {
                    // through the K and V buffers, whose products are done, so that a row leaves as one piece
                    const float inv = l > 0.0f ? 1.0f / l : 0.0f;
                    constexpr int PITCH = 2 * D + 16;  // 16 bytes more: rows in different banks
                    static_assert(C::kTiles * kM * PITCH <= 2 * kStages * C::kTile, "the buffers hold the output");
                    uint8_t* mine = smem + (t * kM + r) * PITCH + 2 * c0;
#pragma unroll 1
                    for (int c = 0; c < W; c += 32) {
                        float v[32];
                        if (n_tiles > 0) tmem_ld32(t_out + c0 + c, v);
#pragma unroll
                        for (int e = 0; e < 32; e += 8) {
                            float x[8];
#pragma unroll
                            for (int k = 0; k < 8; ++k) x[k] = n_tiles > 0 ? v[e + k] * inv : 0.0f;
                            Vec16<__nv_bfloat16>::store(reinterpret_cast<__nv_bfloat16*>(mine) + c + e, x);
                        }
                    }
                    fence_proxy_async_smem();
                    if (t * kM + r < n_rows) {
                        bulk_store_1d(static_cast<__nv_bfloat16*>(a.out) +
                                          (static_cast<size_t>(q0 + row / G) * a.n_q_heads + h * G + row % G) * D + c0,
                                      mine, 2 * W);
                        bulk_commit();
                        bulk_wait_read();
                    }
                }
            }
        }
    } else if (warp < kPlaceWarp) {
        // ---- converters: a warp takes 16 rows of K's or V's tiles, one 16-key group.  A load covers
        // whole 128-byte lines (4 rows of 128 bytes: a load of 8 half lines took eight times the
        // cycles of the load pipe), 8 neighbouring lanes two rows of one block of 64 channels, whose
        // swizzled chunks lie in different banks.
        constexpr int RS = D == 64 ? 8 : 4, RJ = 16 / RS, P = D == 256 ? 2 : 1;  // rows a load, loads of 16 rows
        const bool is_v = warp >= kSoftWarps + kConvWarps;
        const int cw = warp & (kConvWarps - 1);
        const int r_in = D == 64 ? lane >> 2 : ((lane >> 2) & 1) | (lane >> 4) << 1;
        const int ch = D == 64 ? lane & 3 : (lane & 3) | ((lane >> 3) & 1) << 2;  // 16-byte chunk of a row
        uint64_t* full = is_v ? sh.v_full : sh.k_full;
        uint64_t* empty = is_v ? sh.v_empty : sh.k_empty;
        uint8_t* tiles = is_v ? sv : sk;
        const uint8_t* codes = (is_v ? a.c.v : a.c.k) + r_in * D + 16 * ch;
        // Two tiles of codes are in flight in registers: a tile's registers take the codes two tiles
        // on as soon as they are converted.
        uint4 raw[2][RJ][P];
        bool ok = true;
        auto load = [&](int b, int i) {  // rows past the end, and of unmapped pages, are zeros
            if (i >= n_tiles) return;
            const int hb = i / kPass & 1;
            if (i % kPass == 0 && ok)
                ok = __all_sync(0xffffffffu, mbar_wait_brief(&sh.l_full[hb], (i / (2 * kPass)) & 1));
            // keys from this lane's first row on; none once a wait gave up, after which the places may be anything
            const long long at = sh.place[i % (2 * kPass)][cw];
            const int left = at >= 0 && ok ? end - (first + i * kKeys + 16 * cw + r_in) : 0;
            if (i % kPass == kPass - 1) {
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh.l_empty[hb]);
            }
#pragma unroll
            for (int j = 0; j < RJ; ++j)
#pragma unroll
                for (int q = 0; q < P; ++q)
                    raw[b][j][q] = RS * j < left ? *reinterpret_cast<const uint4*>(codes + at + RS * j * D + 128 * q)
                                                 : make_uint4(0, 0, 0, 0);
        };
#pragma unroll
        for (int b = 0; b < 2; ++b) load(b, b);
        if (C::kQInTmem && !is_v && ok) ok = __all_sync(0xffffffffu, mbar_wait_brief(&sh.q_staged, 0));  // read out of them
        int stage = 0, round = 0;
        for (int i0 = 0; ok && i0 < n_tiles; i0 += 2) {
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                const int i = i0 + b;
                if (i >= n_tiles || !ok) break;
                if (round > 0) ok = __all_sync(0xffffffffu, mbar_wait_brief(&empty[stage], (round - 1) & 1));
                if (!ok) break;
                uint8_t* tile = tiles + stage * C::kTile;
#pragma unroll
                for (int j = 0; j < RJ; ++j)
#pragma unroll
                    for (int q = 0; q < P; ++q) {
                        // 16 codes are two 16-byte chunks of a row of 64 channels, swizzled
                        const uint4 x = raw[b][j][q];
                        uint4 lo, hi;
                        widen_f16<F>(x.x, lo.x, lo.y);
                        widen_f16<F>(x.y, lo.z, lo.w);
                        widen_f16<F>(x.z, hi.x, hi.y);
                        widen_f16<F>(x.w, hi.z, hi.w);
                        const int row = 16 * cw + RS * j + r_in;
                        uint8_t* dst = tile + (2 * q + (ch >> 2)) * (kKeys * 128);
                        *reinterpret_cast<uint4*>(dst + sw128_offset(row, 2 * (ch & 3))) = lo;
                        *reinterpret_cast<uint4*>(dst + sw128_offset(row, 2 * (ch & 3) + 1)) = hi;
                    }
                __syncwarp();
                if (lane == 0) mbar_arrive(&full[stage]);
                load(b, i + 2);
                if (++stage == kStages) {
                    stage = 0;
                    ++round;
                }
            }
        }
        if (!ok && lane == 0) record(a.error, 45);
    } else if (warp < kIssueWarp) {
        // ---- look-ups, kPass tiles of groups at a time, two passes ahead of their readers
        const bool place = warp == kPlaceWarp;
        uint64_t *full = place ? sh.l_full : sh.c_full, *empty = place ? sh.l_empty : sh.c_empty;
        bool ok = !(place && a.stall);  // the test hook: no place is ever published
        for (int i0 = 0, pass = 0; ok && i0 < n_tiles; i0 += kPass, ++pass) {
            const int key = first + i0 * kKeys + 16 * lane, pg = page_of(key), hb = pass & 1;
            const size_t block = static_cast<size_t>(max(pg, 0)) * a.n_kv_heads + h;
            GroupConst g{0.0f, -INFINITY, 1.0f};
            if (!place) {
                if (pg >= 0) {
                    g.ks = a.c.k_scale[block];
                    const float vs = a.c.v_scale[block];
                    g.lv = zero_scale(vs) ? -kZeroLog : log2f(vs);
                    g.inv = zero_scale(vs) ? -1.0f : 1.0f / vs;
                } else if (key < end && key + 15 > behind) {
                    record(a.error, kKvErrTable);
                }
            }
            if (pass >= 2 && !(ok = __all_sync(0xffffffffu, mbar_wait_brief(&empty[hb], ((pass >> 1) - 1) & 1)))) {
                if (lane == 0) record(a.error, 45);
                break;
            }
            const int slot = hb * kPass + lane / kGroups;
            if (place)
                sh.place[slot][lane % kGroups] =
                    pg >= 0 ? static_cast<long long>((block * a.page_size + key % a.page_size) * D) : -1;
            else
                sh.consts[slot][lane % kGroups] = g;
            __syncwarp();
            if (lane == 0) mbar_arrive(&full[hb]);
        }
    } else {
        // ---- issue: scores by one warp, outputs by the next.  The whole warp runs the loop, so that
        // addresses and descriptors stay warp-uniform; one lane issues.
        const bool scores = warp == kIssueWarp, leader = elect_one();
        constexpr uint32_t id_s = idesc_f16_f32(kM, kKeys, false), id_o = idesc_f16_f32(kM, D, true);
        const uint64_t da0 = C::kQInTmem ? 0 : desc_kmajor_sw128(smem_u32(sq));
        const uint64_t db0 = scores ? desc_kmajor_sw128(smem_u32(sk)) : desc_mnmajor_sw128(smem_u32(sv), kKeys * 128);
        auto wait = [&](uint64_t* bar, uint32_t parity) { return __all_sync(0xffffffffu, mbar_wait_brief(bar, parity)) != 0; };
        bool ok = n_tiles == 0 || !scores || wait(&sh.q_full, 0);
        uint64_t* last = nullptr;
        uint32_t last_par = 0;
        int stage = 0, round = 0;  // buffer and round of the tile
        for (int i = 0; ok && i < n_tiles; ++i) {
            const int b = i & 1;
            if (!(ok = wait(scores ? &sh.k_full[stage] : &sh.v_full[stage], round & 1))) break;
            fence_proxy_async_smem();
            const uint64_t db = db0 + static_cast<uint64_t>(stage) * (C::kTile >> 4);
            for (int t = 0; t < active; ++t) {
                // scores: the last ones were read; outputs: the weights are there
                if (scores ? i >= 1 && !(ok = wait(&sh.s_empty[t], (i - 1) & 1))
                           : !(ok = wait(&sh.p_full[t][b], (i >> 1) & 1)))
                    break;
                tc_fence_after_sync();
                if (scores) {
                    const uint64_t da = da0 + static_cast<uint64_t>(t) * (C::kQ >> 4);
                    const uint32_t d = tmem + t * kKeys;
                    if (leader) {
#pragma unroll
                        for (int n = 0; n < D / 64; ++n)
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                const uint64_t dbk = db + (n * (kKeys * 128) >> 4) + 2 * k;
                                if (C::kQInTmem)
                                    mma_f16_ta(d, tmem + C::kQCol + 32 * n + 8 * k, dbk, id_s, (n > 0 || k > 0) ? 1u : 0u);
                                else
                                    mma_bf16(d, da + (n * (kM * 128) >> 4) + 2 * k, dbk, id_s, (n > 0 || k > 0) ? 1u : 0u);
                            }
                        mma_commit(&sh.s_full[t]);
                    }
                    last = &sh.s_full[t];
                    last_par = i & 1;
                } else {
                    const uint32_t d = tmem + C::kOut + t * D, p = tmem + C::kWeights + t * kKeys + b * (kKeys / 2);
                    if (leader) {
#pragma unroll
                        for (int k = 0; k < kKeys / 16; ++k)  // 16 keys of weights are 8 columns
                            mma_f16_ta(d, p + 8 * k, db + k * (2048 >> 4), id_o, (i > 0 || k > 0) ? 1u : 0u);
                        mma_commit(&sh.pv_done[t][b]);
                    }
                    last = &sh.pv_done[t][b];
                    last_par = (i >> 1) & 1;
                }
                __syncwarp();
            }
            if (!ok) break;
            if (leader) mma_commit(scores ? &sh.k_empty[stage] : &sh.v_empty[stage]);
            if (!scores && i == n_tiles - 1) {
                if (leader) mma_commit(&sh.o_full);
                last = &sh.o_full;
                last_par = 0;
            }
            __syncwarp();
            if (++stage == kStages) {
                stage = 0;
                ++round;
            }
        }
        if (!ok && leader) record(a.error, 46);
        // nothing of this warp is in flight when the tensor memory is freed
        if (last && !wait(last, last_par) && leader) record(a.error, 47);
    }
    __syncwarp();
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    if (warp == kIssueWarp) tmem_dealloc(tmem, 512);
}

template <typename F, int D, bool SPLIT>
cudaError_t prompt_s(const KvAttnArgs& a, const KvPrompt& c, cudaStream_t st) {
    using C = PCfg<D>;
    static std::atomic<unsigned long long> ready{0};
    const cudaError_t e = allow_smem(kv_prompt_kernel<F, D, SPLIT>, C::kSmem, ready);
    if (e != cudaSuccess) return e;
    return timed_launch("kv_prompt", st, [&] {
        kv_prompt_kernel<F, D, SPLIT>
            <<<dim3(a.n_kv_heads, a.b.n_seq, c.tiles * c.split.n), kThreads, C::kSmem, st>>>(a, c.split);
        return cudaGetLastError();
    });
}

template <typename F, int D>
cudaError_t prompt_t(const KvAttnArgs& a, const KvPrompt& c, cudaStream_t st) {
    if (c.split.n == 1) return prompt_s<F, D, false>(a, c, st);
    const cudaError_t e = prompt_s<F, D, true>(a, c, st);
    return e != cudaSuccess ? e : launch_kv_join(a, c.split, c.rows, c.tiles, D, st);
}

template <typename F>
cudaError_t prompt_d(const KvAttnArgs& a, const KvPrompt& c, int head_dim, cudaStream_t st) {
    return head_dim == 64    ? prompt_t<F, 64>(a, c, st)
           : head_dim == 128 ? prompt_t<F, 128>(a, c, st)
                             : prompt_t<F, 256>(a, c, st);
}

}  // namespace

// Which calls this kernel takes, and how it splits their keys.
//
// Below 17 rows (33 at head_dim 64) the kernel for few rows reads each code once
// in one tile, and wins where there are many: 64 sequences of 8 kv heads with 32
// rows and 4000 keys take it 150 us at head_dim 64, this one 240 us; at head_dim
// 128 263 and 266 us, at 256, where it has two tiles of 16 rows, 440 and 304 us.
// Above that this one wins once there is enough work for its longer start: 2^19
// row and key pairs (head_dim 128, here against there: 16.4 / 12.3 us at 0.25 M
// pairs, 14.0 / 14.5 at 0.5 M, 14.9 / 22.5 at 1 M, 27 / 70 us at 4 M), or 16 tiles
// of 128 rows (16 sequences of 128 rows and 116 keys, 0.24 M pairs: 10.3 / 13.0).
//
// A call with fewer thread blocks than SMs splits its keys into as many ranges as
// fill them once (38 blocks, 8000 keys, head_dim 256: 130 / 80 / 61 / 52 us in 1 to
// 4 ranges, 72 us in 6), of two steps of 64 keys at least, if that takes 12 steps
// off each block: partial results and the join cost about as much (32 blocks of 18
// steps, head_dim 128: 33 us, 26 us in 4 ranges; 64 blocks: 33 us, 34 us in 2).
// More than 32 ranges need the join's widest form (2 blocks of 8000 keys, head_dim
// 256: 16.5 us in 32, 23 us in 48), which pays for a single block with a long axis
// (30,000 keys, head_dim 64 / 128 / 256: 22 / 24 / 26 us in 32, 13 / 19 / 21 us in 152).
KvPrompt kv_prompt_plan(int n_seq, int max_q, int n_q_heads, int n_kv_heads, int head_dim, int window, bool bf16,
                        long long max_kv_len) {
    KvPrompt p{};
    const long long G = n_q_heads / n_kv_heads, rows = max_q * G, heads = static_cast<long long>(n_kv_heads) * n_seq;
    if (!bf16 || rows <= (head_dim == 64 ? 32 : 16)) return p;
    p.rows = kM * (head_dim == 256 ? PCfg<256>::kTiles : PCfg<128>::kTiles);
    long long keys = std::max(1LL, max_kv_len);  // that a thread block walks
    if (window) keys = std::min(keys, window + p.rows / G + 1LL + kKeys);
    const bool many = rows > 32 && (rows + kM - 1) / kM * heads >= 16;
    if (!many && static_cast<double>(rows) * heads * keys < 1 << 19) return p;
    const long long tiles = (rows + p.rows - 1) / p.rows, blocks = tiles * heads, steps = (keys + kKeys - 1) / kKeys;
    const long long most = blocks == 1 && steps > 8 * 32 ? 152 : 32;
    const long long n = std::max(1LL, std::min({152 / blocks, steps / 2, most}));
    long long each = (steps + n - 1) / n;
    if (steps - each < 12) each = steps;
    p.split = KvSplit{static_cast<int>((steps + each - 1) / each), static_cast<int>(std::min(each * kKeys, 0x7fffffffLL / kKeys * kKeys))};
    if (tiles * p.split.n <= 65535) p.tiles = static_cast<int>(tiles);  // the grid's third dimension
    return p;
}

cudaError_t launch_kv_prompt(const KvAttnArgs& a, const KvPrompt& c, int head_dim, bool e4m3, cudaStream_t stream) {
    return e4m3 ? prompt_d<KvE4m3>(a, c, head_dim, stream) : prompt_d<KvInt8>(a, c, head_dim, stream);
}

}  // namespace gdn
