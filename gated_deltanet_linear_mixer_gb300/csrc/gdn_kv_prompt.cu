// Causal attention over the paged 8-bit cache, many query rows (prompts) of
// bf16 activations, on the 5th-generation tensor cores.
//
// The mathematics is that of gdn_kv_attn.cu: products of the codes, block
// scales outside of them,
//   y_rj = (q_r . ck_j) scale s_k log2 e + log2 s_v,   w_rj = 2^(y_rj - m_r)
//   o_r = sum_j w_rj cv_j / sum_blk (sum_j w_rj) / s_v
// with a reference m_r that lags behind the maximum by at most 2^kLazy.  All
// operands are f16: codes exactly, queries exactly down to 2^-24 of a row's
// largest, weights (times 2^kBias) with 11 bits; weights below 2^-31 of the
// reference are dropped.
//
// One thread block takes 128 rows (token, head of the group) of a sequence and
// kv head and walks its keys in tiles of 64.  Roles:
//   4 softmax warps    a thread a row: score row from tensor memory, weights to
//                      shared memory as f16, rescaling of the output in tensor
//                      memory when the reference moves, and the epilogue
//   converter warps    codes from global memory (prefetched two tiles ahead in
//                      registers) to f16 operand tiles in shared memory, K and
//                      V in turn, two buffers each; V needs no transpose, its
//                      operand is MN-major
//   1 look-up warp     pages' scales to the block constants of the tiles ahead
//   1 issuing thread   S_i+1 = Q K_i+1^T ahead of O += P_i V_i, so that the
//                      softmax of one tile runs under the products of others
// The operand tiles are written by ordinary stores and read by the tensor core:
// the issuing thread, which has waited for the writers, fences the one against
// the other.  (A writer's fence would also wait for the loads that it has in
// flight: 275 us instead of @@ for a prompt of 4096 tokens.)
// Every wait is bounded (2 s); a wait that gives up records a code (42..48) in
// this file's device error word and its role stops.
#include <algorithm>

#include "gdn_internal.h"
#include "gdn_kv.cuh"
#include "gdn_tc.cuh"

namespace gdn {

using namespace tc;

namespace {

__device__ int g_kv_prompt_error = 0;
__device__ __forceinline__ void prompt_fail(int code) { atomicCAS(&g_kv_prompt_error, 0, code); }

constexpr int kM = 128, kKeys = 64;
constexpr int kGroups = kKeys / 16;  // 16-key groups of a tile: one page each
constexpr int kConst = 4;            // tiles whose block constants are kept
constexpr float kLazy = 8.0f;
constexpr float kBias = 7.0f;        // weights are 2^7 times theirs: at most 2^15

template <int D> struct PCfg {
    static constexpr int kConvWarps = D == 256 ? 8 : 4;
    static constexpr int kThreads = 32 * (4 + kConvWarps + 2);
    static constexpr int kPBufs = D == 256 ? 2 : 1;
    static constexpr uint32_t kQ = kM * D * 2, kTile = kKeys * D * 2, kP = kM * kKeys * 2;
    // the operand tiles, then Shared; at head_dim 128 two thread blocks fill an SM's 228 KB to the byte
    static constexpr uint32_t kData = kQ + 4 * kTile + kPBufs * kP, kSmem = kData + 1024;
    static constexpr uint32_t kCols = D == 256 ? 512 : 256;  // tensor memory: two score tiles, then the output
    static constexpr int kBlocks = D == 256 ? 1 : 2;
};

// Instruction descriptor, kind::f16: f16 A and B, fp32 accumulator.
__host__ __device__ constexpr uint32_t idesc_f16_f32(int M, int N, bool b_mn) {
    return (1u << 4) | ((b_mn ? 1u : 0u) << 16) | (static_cast<uint32_t>(N >> 3) << 17) |
           (static_cast<uint32_t>(M >> 4) << 24);
}

// 32 lanes x 32 columns of 32-bit, registers to tensor memory.
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const float* v) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};\n\t"
        "tcgen05.wait::st.sync.aligned;" ::"f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]),
        "f"(v[6]), "f"(v[7]), "f"(v[8]), "f"(v[9]), "f"(v[10]), "f"(v[11]), "f"(v[12]), "f"(v[13]), "f"(v[14]),
        "f"(v[15]), "f"(v[16]), "f"(v[17]), "f"(v[18]), "f"(v[19]), "f"(v[20]), "f"(v[21]), "f"(v[22]), "f"(v[23]),
        "f"(v[24]), "f"(v[25]), "f"(v[26]), "f"(v[27]), "f"(v[28]), "f"(v[29]), "f"(v[30]), "f"(v[31]), "r"(taddr)
        : "memory");
}

// Block constants of one 16-key group: factor of the scores, their offset
// (log2 of the value scale), and its reciprocal (negative: values are zero).
struct GroupConst {
    float ks, lv, inv;
};

struct Shared {
    uint64_t q_full, k_full[2], k_empty[2], v_full[2], v_empty[2], s_full[2], s_empty[2], p_full[2], p_empty[2],
        c_full[kConst], c_empty[kConst], o_full;
    GroupConst consts[kConst][kGroups];
    float q_scale[kM];
    uint32_t tmem_slot;
};
static_assert(sizeof(Shared) <= 1024, "part of kSmem");

template <typename F, int D>
__global__ void __launch_bounds__(PCfg<D>::kThreads, PCfg<D>::kBlocks) kv_prompt_kernel(const KvAttnArgs a) {
    using C = PCfg<D>;
    constexpr int CW = C::kConvWarps, PB = C::kPBufs;
    extern __shared__ __align__(1024) uint8_t smem[];  // the swizzled tiles start on 1024-byte boundaries
    Shared& sh = *reinterpret_cast<Shared*>(smem + C::kData);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int seq = blockIdx.y, h = blockIdx.x, G = a.n_q_heads / a.n_kv_heads;
    const int q0 = a.b.cu[seq], qn = a.b.cu[seq + 1] - q0;
    const int row0 = (static_cast<int>(gridDim.z) - 1 - static_cast<int>(blockIdx.z)) * kM;  // most keys first
    const int n_rows = min(kM, qn * G - row0);
    if (n_rows <= 0) return;
    int len = a.b.kv_lens[seq];
    const int start = len - qn;  // position of the call's first query
    const long long cap = static_cast<long long>(a.b.pages_per_seq) * a.page_size;
    if (len > cap) {
        if (tid == 0) prompt_fail(kKvErrTable);
        len = static_cast<int>(cap);
    }
    const int lo_pos = start + row0 / G, hi_pos = start + (row0 + n_rows - 1) / G;
    const int first = a.window ? max(0, lo_pos - a.window + 1) / kKeys * kKeys : 0;
    const int end = min(hi_pos + 1, len);
    const int n_tiles = end > first ? (end - first + kKeys - 1) / kKeys : 0;

    if (smem_u32(smem) & 1023u) {
        if (tid == 0) prompt_fail(48);
        return;
    }
    uint8_t* sq = smem;
    uint8_t* sk = sq + C::kQ;
    uint8_t* sv = sk + 2 * C::kTile;
    uint8_t* sp = sv + 2 * C::kTile;

    if (tid == 0) {
        mbar_init(&sh.q_full, 4);
        mbar_init(&sh.o_full, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sh.k_full[i], CW);
            mbar_init(&sh.v_full[i], CW);
            mbar_init(&sh.k_empty[i], 1);
            mbar_init(&sh.v_empty[i], 1);
            mbar_init(&sh.s_full[i], 1);
            mbar_init(&sh.s_empty[i], 4);
        }
        for (int i = 0; i < PB; ++i) {
            mbar_init(&sh.p_full[i], 4);
            mbar_init(&sh.p_empty[i], 1);
        }
        for (int i = 0; i < kConst; ++i) {
            mbar_init(&sh.c_full[i], 1);
            mbar_init(&sh.c_empty[i], 4);
        }
        fence_barrier_init();
    }
    if (warp == 5 + CW) tmem_alloc(&sh.tmem_slot, C::kCols);
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = sh.tmem_slot, t_out = tmem + 2 * kKeys;

    auto page_of = [&](int key) {  // negative: past the end, or not mapped
        if (key >= end) return -1;
        const int page = a.b.table[static_cast<size_t>(seq) * a.b.pages_per_seq + key / a.page_size];
        return page < a.c.n_pages ? page : -1;
    };

    if (warp < 4) {
        // ---- queries: 32 rows a warp, rounded to f16 under a power of two of the row
        constexpr int E = D / 32;  // channels of a lane
        for (int r8 = 0; r8 < 32; r8 += 8) {
            uint32_t raw[8][E / 2];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int r = 32 * warp + r8 + i, row = row0 + r;
#pragma unroll
                for (int e = 0; e < E / 2; ++e) raw[i][e] = 0;
                if (r < n_rows) {
                    const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(a.q.data) +
                                               (q0 + row / G) * a.q.token_stride + (h * G + row % G) * a.q.head_stride;
                    memcpy(raw[i], __builtin_assume_aligned(src + E * lane, E * 2), E * 2);
                }
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int r = 32 * warp + r8 + i;
                float most = 0.0f;
#pragma unroll
                for (int e = 0; e < E / 2; ++e)
                    most = fmaxf(most, fmaxf(fabsf(__uint_as_float(raw[i][e] << 16)),
                                             fabsf(__uint_as_float(raw[i][e] & 0xFFFF0000u))));
#pragma unroll
                for (int off = 16; off > 0; off >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, off));
                const int ex = most > 0.0f && most <= 3.402823466e38f
                                   ? min(max(static_cast<int>(__float_as_uint(most) >> 23) - 127, -100), 126) : 0;
                const float down = __uint_as_float(static_cast<uint32_t>(127 - ex) << 23);
                if (lane == 0)
                    sh.q_scale[r] = a.scale * kLog2e * __uint_as_float(static_cast<uint32_t>(127 + ex) << 23);
                uint32_t w[E / 2];
#pragma unroll
                for (int e = 0; e < E / 2; ++e)
                    w[e] = pack_f16(__uint_as_float(raw[i][e] << 16) * down, __uint_as_float(raw[i][e] & 0xFFFF0000u) * down);
                // channel E lane of column block (E lane) / 64
                const uint32_t byte = (E * lane % 64) * 2;
                uint8_t* dst = sq + (E * lane / 64) * (kM * 128) + sw128_offset(r, byte >> 4) + (byte & 15);
                memcpy(__builtin_assume_aligned(dst, E * 2), w, E * 2);
            }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.q_full);

        // ---- softmax: thread = row
        const int r = tid, pos = start + (row0 + r) / G;
        const float qs = sh.q_scale[r];
        const int max_lo = a.window ? hi_pos - a.window + 1 : 0;
        const uint32_t t_lane = (32u * warp) << 16;
        float m = -INFINITY, l = 0.0f;
        bool ok = true;
        for (int i = 0; i < n_tiles; ++i) {
            const int key = first + i * kKeys, sb = i & 1, pb = i % PB;
            if (!(ok = __all_sync(0xffffffffu, mbar_wait_brief(&sh.s_full[sb], (i >> 1) & 1) &&
                                                   mbar_wait_brief(&sh.c_full[i % kConst], (i / kConst) & 1)))) {
                if (lane == 0) prompt_fail(42);
                break;
            }
            tc_fence_after_sync();
            float s[kKeys];
            tmem_ld64(tmem + t_lane + sb * kKeys, s);
            GroupConst gc[kGroups];
#pragma unroll
            for (int g = 0; g < kGroups; ++g) gc[g] = sh.consts[i % kConst][g];
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&sh.s_empty[sb]);
                mbar_arrive(&sh.c_empty[i % kConst]);
            }
            const bool whole = key + kKeys - 1 <= lo_pos && key >= max_lo && key + kKeys <= end;
#pragma unroll
            for (int j = 0; j < kKeys; ++j) s[j] = fmaf(s[j], qs * gc[j / 16].ks, gc[j / 16].lv);
            if (!whole) {
                const int hi = min(pos, end - 1) - key, lo = a.window ? pos - a.window + 1 - key : 0;
#pragma unroll
                for (int j = 0; j < kKeys; ++j) s[j] = j > hi || j < lo ? -INFINITY : s[j];
            }
            float tops[4] = {s[0], s[1], s[2], s[3]};  // four chains
#pragma unroll
            for (int j = 4; j < kKeys; ++j) tops[j & 3] = fmaxf(tops[j & 3], s[j]);
            const float top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
            const bool lift = __any_sync(0xffffffffu, top > m + kLazy);
            float f = 1.0f;
            if (lift) {
                const float mn = fmaxf(m, top);
                f = m == -INFINITY ? 0.0f : exp2_ftz(m - mn);
                m = mn;
                l *= f;
            }
            const float ref = m == -INFINITY ? 0.0f : m - kBias;
            uint32_t p[kKeys / 2];
#pragma unroll
            for (int g = 0; g < kGroups; ++g) {
                float sum = 0.0f;
                const bool dead = gc[g].inv < 0.0f;  // values of a scale of 0: counted, not added
#pragma unroll
                for (int j = 16 * g; j < 16 * g + 16; j += 2) {
                    const float w0 = exp2_ftz(s[j] - ref), w1 = exp2_ftz(s[j + 1] - ref);
                    sum += w0 + w1;
                    p[j / 2] = dead ? 0u : pack_f16(w0, w1);
                }
                l = fmaf(sum, fabsf(gc[g].inv), l);
            }
            // the buffer's earlier weights were used; with one buffer, that is the last tile's product
            if (i >= PB && !(ok = __all_sync(0xffffffffu, mbar_wait_brief(&sh.p_empty[pb], (i / PB - 1) & 1)))) {
                if (lane == 0) prompt_fail(43);
                break;
            }
            uint8_t* prow = sp + pb * C::kP;
#pragma unroll
            for (int c = 0; c < kKeys / 8; ++c)
                *reinterpret_cast<uint4*>(prow + sw128_offset(r, c)) =
                    make_uint4(p[4 * c], p[4 * c + 1], p[4 * c + 2], p[4 * c + 3]);
            if (lift && i > 0) {  // the output so far, once the products before this tile's are done
                const int last = i - 1;
                if (PB > 1 && !(ok = __all_sync(0xffffffffu, mbar_wait_brief(&sh.p_empty[last % PB], (last / PB) & 1)))) {
                    if (lane == 0) prompt_fail(43);
                    break;
                }
                tc_fence_after_sync();
#pragma unroll 1
                for (int c = 0; c < D; c += 32) {
                    float v[32];
                    tmem_ld32(t_out + t_lane + c, v);
#pragma unroll
                    for (int e = 0; e < 32; ++e) v[e] *= f;
                    tmem_st32(t_out + t_lane + c, v);
                }
                tc_fence_before_sync();
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.p_full[pb]);
        }
        // ---- epilogue
        if (ok && n_tiles > 0 && !(ok = __all_sync(0xffffffffu, mbar_wait_brief(&sh.o_full, 0))) && lane == 0) prompt_fail(44);
        if (ok) {
            tc_fence_after_sync();
            const float inv = l > 0.0f ? 1.0f / l : 0.0f;
            const int row = row0 + r;
            __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out) +
                                 (static_cast<size_t>(q0 + row / G) * a.n_q_heads + h * G + row % G) * D;
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
                float v[32];
                if (n_tiles > 0) tmem_ld32(t_out + t_lane + c, v);
                if (r < n_rows) {
#pragma unroll
                    for (int e = 0; e < 32; e += 8) {
                        float x[8];
#pragma unroll
                        for (int k = 0; k < 8; ++k) x[k] = n_tiles > 0 ? v[e + k] * inv : 0.0f;
                        Vec16<__nv_bfloat16>::store(out + c + e, x);
                    }
                }
            }
        }
    } else if (warp < 4 + CW) {
        // ---- converters: a thread takes 16-byte chunks c0, c0 + 4, .. of RT rows of a tile
        constexpr int RT = kKeys / (8 * CW), N = D / 64;
        const int cw = warp - 4, c0 = lane >> 3;
        int row[RT];
#pragma unroll
        for (int i = 0; i < RT; ++i) row[i] = 8 * (cw + CW * i) + (lane & 7);
        const uint8_t* codes[2] = {a.c.k, a.c.v};
        // Two tiles of codes are in flight in registers: a tile's registers take the codes two tiles
        // on as soon as they are converted; pages are looked up one tile before that.
        uint4 raw[2][2][RT][N];
        int page[2][RT];
        auto load = [&](int b, int kv, int i) {  // rows past the end, and of unmapped pages, are zeros
#pragma unroll
            for (int t = 0; t < RT; ++t) {
                const int key = first + i * kKeys + row[t], pg = page[b][t];
                const bool take = pg >= 0;
                const size_t at = take ? ((static_cast<size_t>(pg) * a.n_kv_heads + h) * a.page_size + key % a.page_size) * D
                                       : 0;
#pragma unroll
                for (int n = 0; n < N; ++n)
                    raw[b][kv][t][n] = take ? *reinterpret_cast<const uint4*>(codes[kv] + at + 16 * (c0 + 4 * n))
                                            : make_uint4(0, 0, 0, 0);
            }
        };
        bool ok = true;
#pragma unroll
        for (int b = 0; b < 2; ++b) {
#pragma unroll
            for (int t = 0; t < RT; ++t) page[b][t] = page_of(first + b * kKeys + row[t]);
        }
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            load(b, 0, b);
            load(b, 1, b);
        }
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int t = 0; t < RT; ++t) page[b][t] = page_of(first + (b + 2) * kKeys + row[t]);
        for (int i0 = 0; ok && i0 < n_tiles; i0 += 2) {
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                const int i = i0 + b;
                if (i >= n_tiles || !ok) break;
#pragma unroll
                for (int kv = 0; kv < 2; ++kv) {
                    if (i >= 2 && ok)
                        ok = __all_sync(0xffffffffu, mbar_wait_brief(kv ? &sh.v_empty[b] : &sh.k_empty[b], ((i >> 1) - 1) & 1));
                    if (!ok) break;
                    uint8_t* tile = (kv ? sv : sk) + b * C::kTile;
#pragma unroll
                    for (int t = 0; t < RT; ++t)
#pragma unroll
                        for (int n = 0; n < N; ++n) {
                            // 16 codes are two 16-byte chunks of column block n: row of 64 channels, swizzled
                            const uint4 x = raw[b][kv][t][n];
                            uint4 lo, hi;
                            widen_f16<F>(x.x, lo.x, lo.y);
                            widen_f16<F>(x.y, lo.z, lo.w);
                            widen_f16<F>(x.z, hi.x, hi.y);
                            widen_f16<F>(x.w, hi.z, hi.w);
                            uint8_t* dst = tile + n * (kKeys * 128);
                            *reinterpret_cast<uint4*>(dst + sw128_offset(row[t], 2 * c0)) = lo;
                            *reinterpret_cast<uint4*>(dst + sw128_offset(row[t], 2 * c0 + 1)) = hi;
                        }
                    load(b, kv, i + 2);
                    __syncwarp();
                    if (lane == 0) mbar_arrive(kv ? &sh.v_full[b] : &sh.k_full[b]);
                }
#pragma unroll
                for (int t = 0; t < RT; ++t) page[b][t] = page_of(first + (i + 4) * kKeys + row[t]);
            }
        }
        if (!ok && lane == 0) prompt_fail(45);
    } else if (warp == 4 + CW) {
        // ---- block constants, kConst tiles of groups at a time
        float vs_low = INFINITY;
        bool ok = true;
        for (int i0 = 0; ok && i0 < n_tiles; i0 += kConst) {
            const int key = first + i0 * kKeys + 16 * lane;
            GroupConst g{0.0f, -INFINITY, 1.0f};
            float vs = 1.0f;
            if (lane < kConst * kGroups) {
                const int pg = page_of(key);
                if (pg >= 0) {
                    const size_t block = static_cast<size_t>(pg) * a.n_kv_heads + h;
                    g.ks = a.c.k_scale[block];
                    vs = a.c.v_scale[block];
                    g.lv = 0.0f;
                    if (vs > 0.0f) vs_low = fminf(vs_low, vs);
                } else if (key < end && (!a.window || key + 15 > lo_pos - a.window)) {
                    prompt_fail(kKvErrTable);
                }
            }
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) vs_low = fminf(vs_low, __shfl_xor_sync(0xffffffffu, vs_low, off));
            const bool zero = vs == 0.0f;  // such a group is given the smallest scale in sight, and a mark
            if (zero) vs = vs_low < INFINITY ? vs_low : 1.0f;
            g.lv += log2f(vs);
            g.inv = (zero ? -1.0f : 1.0f) / vs;
            for (int q = 0; q < kConst && i0 + q < n_tiles; ++q) {
                if (i0 > 0 && !(ok = __all_sync(0xffffffffu, mbar_wait_brief(&sh.c_empty[q], (i0 / kConst - 1) & 1)))) {
                    if (lane == 0) prompt_fail(45);
                    break;
                }
                if (lane / kGroups == q) sh.consts[q][lane % kGroups] = g;
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh.c_full[q]);
            }
        }
    } else if (lane == 0) {
        // ---- issue
        constexpr uint32_t id_s = idesc_f16_f32(kM, kKeys, false), id_o = idesc_f16_f32(kM, D, true);
        const uint32_t aq = smem_u32(sq), ak = smem_u32(sk), av = smem_u32(sv), ap = smem_u32(sp);
        bool ok = n_tiles == 0 || mbar_wait_brief(&sh.q_full, 0);
        uint64_t* last = nullptr;
        uint32_t last_par = 0;
        for (int i = 0; ok && i <= n_tiles; ++i) {
            if (i < n_tiles) {
                const int b = i & 1;
                if (!(ok = mbar_wait_brief(&sh.k_full[b], (i >> 1) & 1))) break;
                if (i >= 2 && !(ok = mbar_wait_brief(&sh.s_empty[b], ((i >> 1) - 1) & 1))) break;
                tc_fence_after_sync();
                fence_proxy_async_smem();
#pragma unroll
                for (int n = 0; n < D / 64; ++n) {
                    const uint64_t da = desc_kmajor_sw128(aq + n * (kM * 128));
                    const uint64_t db = desc_kmajor_sw128(ak + b * C::kTile + n * (kKeys * 128));
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        mma_bf16(tmem + b * kKeys, da + 2 * k, db + 2 * k, id_s, (n > 0 || k > 0) ? 1u : 0u);
                }
                mma_commit(&sh.k_empty[b]);
                mma_commit(&sh.s_full[b]);
                last = &sh.s_full[b];
                last_par = (i >> 1) & 1;
            }
            if (i > 0) {
                const int j = i - 1, b = j & 1, pb = j % PB;
                if (!(ok = mbar_wait_brief(&sh.v_full[b], (j >> 1) & 1))) break;
                if (!(ok = mbar_wait_brief(&sh.p_full[pb], (j / PB) & 1))) break;
                tc_fence_after_sync();
                fence_proxy_async_smem();
                const uint64_t da = desc_kmajor_sw128(ap + pb * C::kP);
#pragma unroll
                for (int k = 0; k < kKeys / 16; ++k)
                    mma_bf16(t_out, da + 2 * k, desc_mnmajor_sw128(av + b * C::kTile + k * 2048, kKeys * 128), id_o,
                             (j > 0 || k > 0) ? 1u : 0u);
                mma_commit(&sh.v_empty[b]);
                mma_commit(&sh.p_empty[pb]);
                last = &sh.p_empty[pb];
                last_par = (j / PB) & 1;
                if (i == n_tiles) {
                    mma_commit(&sh.o_full);
                    last = &sh.o_full;
                    last_par = 0;
                }
            }
        }
        if (!ok) prompt_fail(46);
        // nothing of this thread block is in flight when its tensor memory is freed
        if (last && !mbar_wait_brief(last, last_par)) prompt_fail(47);
    }
    __syncwarp();
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    if (warp == 5 + CW) tmem_dealloc(tmem, C::kCols);
}

template <typename F, int D>
cudaError_t prompt_t(const KvAttnArgs& a, cudaStream_t st) {
    using C = PCfg<D>;
    static std::atomic<unsigned long long> ready{0};
    cudaError_t e = allow_smem(kv_prompt_kernel<F, D>, C::kSmem, ready);
    if (e != cudaSuccess) return e;
    const long long tiles = (static_cast<long long>(a.b.max_q) * (a.n_q_heads / a.n_kv_heads) + kM - 1) / kM;
    return timed_launch("kv_prompt", st, [&] {
        kv_prompt_kernel<F, D><<<dim3(a.n_kv_heads, a.b.n_seq, static_cast<unsigned>(tiles)), C::kThreads, C::kSmem, st>>>(a);
        return cudaGetLastError();
    });
}

template <typename F>
cudaError_t prompt_d(const KvAttnArgs& a, int head_dim, cudaStream_t st) {
    return head_dim == 64 ? prompt_t<F, 64>(a, st) : head_dim == 128 ? prompt_t<F, 128>(a, st) : prompt_t<F, 256>(a, st);
}

}  // namespace

// Whole tiles of 128 rows pay once there are enough of them to occupy a fair
// part of the SMs (their keys are not split): below that the kernel for few
// rows spreads the keys.  The grid's third dimension bounds the tiles.
bool kv_prompt_serves(int n_seq, int max_q, int n_q_heads, int n_kv_heads, bool bf16) {
    const long long rows = static_cast<long long>(max_q) * (n_q_heads / n_kv_heads);
    const long long tiles = (rows + kM - 1) / kM;
    return bf16 && rows > 32 && tiles <= 65535 && tiles * n_kv_heads * n_seq >= 40;
}

cudaError_t launch_kv_prompt(const KvAttnArgs& a, int head_dim, bool e4m3, cudaStream_t stream) {
    return e4m3 ? prompt_d<KvE4m3>(a, head_dim, stream) : prompt_d<KvInt8>(a, head_dim, stream);
}

cudaError_t read_kv_prompt_error(int* code, bool reset) {
    cudaError_t e = cudaMemcpyFromSymbol(code, g_kv_prompt_error, sizeof(int));
    if (e == cudaSuccess && reset) {
        const int zero = 0;
        e = cudaMemcpyToSymbol(g_kv_prompt_error, &zero, sizeof(int));
    }
    return e;
}

}  // namespace gdn
