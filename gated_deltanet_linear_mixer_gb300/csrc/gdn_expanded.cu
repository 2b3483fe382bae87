// Causal attention of the expanded form, on the 5th-generation tensor cores.
//
// The mathematics, in powers of two (y = scale log2 e q . k, k = (k_h | k_rope)):
//   w_rj = 2^(y_rj - m_r),   o_r = sum_j w_rj v_j / sum_j w_rj
// with a reference m_r that lags behind the row's maximum by at most 2^kLazy, so
// that the output is rescaled only where the maximum rises by more than that.
// Weights are rounded to bf16 (the values' type, as the tensor core asks), and the
// sum takes the rounded ones.
//
// A thread block takes two tiles of 128 queries of a head and walks the keys in
// tiles of 128 up to the last query's position.  While one tile's softmax runs, the
// tensor core works for the other.  S of a tile takes 128 columns of tensor memory,
// O as many; the weights overwrite their scores' columns and are the second
// product's A operand where they lie.  Keys and values stream through one ring of
// 16 KB blocks (128 keys x 64 channels) in the order in which they are used; the
// position keys come from their own array, which all heads share.
//
// Roles: 8 softmax warps (a thread a row; a rescaling concerns one warp's rows
// alone), a warp for the loads, one issuing the products, in the order
// O0 += P0 V, S0 = Q0 K', O1 += P1 V, S1 = Q1 K'.  Every wait is bounded (2 s); a
// wait that gives up records a code (60..66) in the cache operators' device error
// word.
#include <algorithm>

#include "gdn_internal.h"
#include "gdn_kv.cuh"
#include "gdn_latent.h"
#include "gdn_tc.cuh"
#include "gdn_tma_host.h"

namespace gdn {

using namespace tc;

namespace {

using bf16 = __nv_bfloat16;

constexpr int kM = 128, kKeys = 128, kTiles = 2;
constexpr int kThreads = 384;
constexpr float kLazy = 8.0f;
constexpr uint32_t kBlock = 16384;  // 128 rows x 64 channels
constexpr uint32_t kSmemMax = 232448, kSharedBytes = 3072;
constexpr int kMaxSlots = 12;

template <int NOPE, int V> struct ECfg {
    static constexpr int kQBlocks = NOPE / 64 + 1, kVBlocks = V / 64, kPer = kQBlocks + kVBlocks;  // blocks of a key tile
    static constexpr uint32_t kQ = kQBlocks * kBlock;  // a query tile
    static constexpr int kPitch = 2 * V + 16;          // of a staged output row: neighbours in different banks
    static constexpr uint32_t kStaged = (kM * kPitch + 1023) / 1024 * 1024, kPlace = kQ > kStaged ? kQ : kStaged;
    static constexpr int kFit = (kSmemMax - kSharedBytes - kTiles * kPlace) / kBlock;
    static constexpr int kSlots = kFit < kMaxSlots ? kFit : kMaxSlots;
    static constexpr uint32_t kQAt = kSlots * kBlock, kSharedAt = kQAt + kTiles * kPlace, kSmem = kSharedAt + kSharedBytes;
    static constexpr uint32_t kOut = kTiles * kKeys;   // tensor memory: scores (weights) of both tiles, outputs
    static_assert(kSlots >= kPer + kQBlocks, "a tile and the next tile's keys fit");
};

struct Shared {
    uint64_t full[kMaxSlots], empty[kMaxSlots];
    uint64_t q_full[kTiles], s_full[kTiles], p_full[kTiles], pv_done[kTiles], drained;
    uint32_t tmem_slot;
};
static_assert(sizeof(Shared) <= kSharedBytes, "part of kSmem");

__device__ __noinline__ void record(int* error, int code) { atomicMax(error, code); }

__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(r));
    return r != 0;
}
__device__ __forceinline__ void bulk_store_1d(void* dst, const void* src, uint32_t bytes) {
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(smem_u32(src)), "r"(bytes)
                 : "memory");
}
// 32 lanes x 32 columns of 32-bit, registers to tensor memory.
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t* v) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};" ::"r"(v[0]),
        "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]), "r"(v[10]),
        "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]), "r"(v[19]),
        "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]), "r"(v[28]),
        "r"(v[29]), "r"(v[30]), "r"(v[31]), "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// D[tmem] (+)= A[tmem] * B[smem]^T, bf16.  A: lane = row, a column holds two consecutive K elements.
__device__ __forceinline__ void mma_bf16_ta(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                            uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}
// Two fp32 operations an instruction.
__device__ __forceinline__ uint64_t pair(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void unpair(uint64_t v, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

struct Maps {
    CUtensorMap q, k, r, v;
};

template <int NOPE, int V>
__global__ void __launch_bounds__(kThreads, 1) expanded_kernel(const ExpandedArgs a, const __grid_constant__ Maps maps) {
    using L = ECfg<NOPE, V>;
    constexpr int NS = L::kSlots, QB = L::kQBlocks, VB = L::kVBlocks;
    extern __shared__ __align__(1024) uint8_t smem[];
    Shared& sh = *reinterpret_cast<Shared*>(smem + L::kSharedAt);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int h = blockIdx.x, seq = blockIdx.y;
    const int q0 = a.cu_q[seq], qn = a.cu_q[seq + 1] - q0, k0 = a.cu_kv[seq], kv = a.cu_kv[seq + 1] - k0;
    const int row0 = (static_cast<int>(gridDim.z) - 1 - static_cast<int>(blockIdx.z)) * (kTiles * kM);  // most keys first
    if (row0 >= qn) return;
    const int start = kv - qn;  // position of the sequence's first query
    int n[kTiles];              // key tiles of each query tile
#pragma unroll
    for (int t = 0; t < kTiles; ++t) {
        const int rows = min(kM, qn - row0 - t * kM);
        n[t] = rows > 0 ? max(0, (start + row0 + t * kM + rows - 1) / kKeys + 1) : 0;
        if (start + row0 + t * kM + rows - 1 < 0) n[t] = 0;
    }
    const int n_tiles = max(n[0], n[1]);
    if (smem_u32(smem) & 1023u) {
        if (tid == 0) record(a.error, 66);
        return;
    }
    if (tid == 0) {
        for (int i = 0; i < NS; ++i) {
            mbar_init(&sh.full[i], 1);
            mbar_init(&sh.empty[i], 1);
        }
        for (int t = 0; t < kTiles; ++t) {
            mbar_init(&sh.q_full[t], 1);
            mbar_init(&sh.s_full[t], 1);
            mbar_init(&sh.p_full[t], 4);
            mbar_init(&sh.pv_done[t], 1);
        }
        mbar_init(&sh.drained, 1);
        fence_barrier_init();
    }
    if (warp == 9) tmem_alloc(&sh.tmem_slot, 512);
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = sh.tmem_slot;

    if (warp < 8) {
        // ---- softmax: a thread's row
        const int t = warp >> 2, r = tid & (kM - 1), row = row0 + t * kM + r;
        const bool mine = row < qn;
        const int lim = mine ? max(0, min(start + row + 1, kv)) : 0;  // keys that the row sees
        const int low = __reduce_min_sync(0xffffffffu, lim);
        const uint32_t t_lane = (32u * (warp & 3)) << 16;
        const uint32_t t_score = tmem + t_lane + t * kKeys, t_out = tmem + t_lane + L::kOut + t * V;
        const float scale2 = a.scale * kLog2e;
        float m = -INFINITY, l = 0.0f;
        bool ok = true;
        for (int i = 0; i < n[t]; ++i) {
            const int key0 = i * kKeys;
            if (ok && !(ok = __all_sync(0xffffffffu, mbar_wait_brief(&sh.s_full[t], i & 1))) && lane == 0) record(a.error, 60);
            tc_fence_after_sync();
            float s[kKeys];
            tmem_ld64(t_score, s);
            tmem_ld64(t_score + 64, s + 64);
            if (key0 + kKeys > low) {
                const int hi = lim - key0;
#pragma unroll
                for (int j = 0; j < kKeys; ++j) s[j] = j < hi ? s[j] : -INFINITY;
            }
            float tops[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
            for (int j = 4; j < kKeys; ++j) tops[j & 3] = fmaxf(tops[j & 3], s[j]);
            const float top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3])) * scale2;
            const bool lift = __any_sync(0xffffffffu, top > m + kLazy);
            float f = 1.0f;
            if (lift) {
                const float mn = fmaxf(m, top);
                f = m == -INFINITY ? 0.0f : exp2_ftz(m - mn);
                m = mn;
                l *= f;
            }
            const float ref = m == -INFINITY ? 0.0f : -m;
            const uint64_t scale22 = pair(scale2, scale2), ref2 = pair(ref, ref);
            uint64_t sums[2] = {0, 0};
#pragma unroll
            for (int c = 0; c < kKeys; c += 64) {
                uint32_t p[32];
#pragma unroll
                for (int j = 0; j < 64; j += 2) {
                    float w0, w1;
                    unpair(fma2(pair(s[c + j], s[c + j + 1]), scale22, ref2), w0, w1);
                    const uint32_t w = pack_bf16x2(exp2_ftz(w0), exp2_ftz(w1));
                    p[j / 2] = w;
                    sums[(j / 2) & 1] = add2(sums[(j / 2) & 1], pair(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u)));
                }
                tmem_st32(t_score + c / 2, p);
            }
            float s0, s1;
            unpair(add2(sums[0], sums[1]), s0, s1);
            l += s0 + s1;
            if (lift && i > 0) {  // the output so far
                if (ok && !(ok = __all_sync(0xffffffffu, mbar_wait_brief(&sh.pv_done[t], (i - 1) & 1))) && lane == 0)
                    record(a.error, 61);
                tc_fence_after_sync();
#pragma unroll 1
                for (int c = 0; c < V; c += 32) {
                    float v[32];
                    uint32_t u[32];
                    tmem_ld32(t_out + c, v);
#pragma unroll
                    for (int e = 0; e < 32; ++e) u[e] = __float_as_uint(v[e] * f);
                    tmem_st32(t_out + c, u);
                }
            }
            // rows behind the sequence's last key may be anything: weights of 0 do not undo a NaN.  By the
            // first of the tiles that use them.
            if (key0 + kKeys > kv && (t == 0 || i >= n[0])) {
                for (int b = 0; b < VB; ++b) {
                    const uint32_t fill = i * L::kPer + QB + b, slot = fill % NS;
                    if (ok && !(ok = __all_sync(0xffffffffu, mbar_wait_brief(&sh.full[slot], (fill / NS) & 1))) && lane == 0)
                        record(a.error, 62);
                    uint4* rows = reinterpret_cast<uint4*>(smem + slot * kBlock);
                    for (int x = 8 * (kv - key0) + r; x < 8 * kKeys; x += kM) rows[x] = make_uint4(0, 0, 0, 0);
                }
                fence_proxy_async_smem();
            }
            tmem_wait_st();
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.p_full[t]);
        }
        // ---- epilogue: through the query tile's place, whose products are done, so that a row leaves as one piece
        if (n[t] > 0 && ok && !(ok = __all_sync(0xffffffffu, mbar_wait_brief(&sh.pv_done[t], (n[t] - 1) & 1))) && lane == 0)
            record(a.error, 63);
        tc_fence_after_sync();
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;  // a sum that is no number stays one
        uint8_t* stage = smem + L::kQAt + t * L::kPlace + r * L::kPitch;
#pragma unroll 1
        for (int c = 0; c < V; c += 32) {
            float v[32];
            if (n[t] > 0) tmem_ld32(t_out + c, v);
#pragma unroll
            for (int e = 0; e < 32; e += 8) {
                float x[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) x[k] = n[t] > 0 ? v[e + k] * inv : 0.0f;
                Vec16<bf16>::store(reinterpret_cast<bf16*>(stage) + c + e, x);
            }
        }
        fence_proxy_async_smem();
        if (mine && ok) {
            bulk_store_1d(static_cast<bf16*>(a.out) + (static_cast<size_t>(q0 + row) * a.n_heads + h) * V, stage, 2 * V);
            bulk_commit();
            bulk_wait_read();
        }
    } else if (warp == 8) {
        // ---- loads
        const bool leader = elect_one();
        const int hq = a.q.head_stride ? h : 0, hk = a.k.head_stride ? h : 0, hv = a.v.head_stride ? h : 0;
        bool ok = true;
        uint32_t fills = 0;
        if (leader && n_tiles > 0) {
            for (int t = 0; t < kTiles; ++t) {
                if (n[t] == 0) continue;
                mbar_arrive_expect_tx(&sh.q_full[t], L::kQ);
                for (int b = 0; b < QB; ++b)
                    tma_load_3d(smem + L::kQAt + t * L::kPlace + b * kBlock, &maps.q, &sh.q_full[t], 64 * b, q0 + row0 + t * kM, hq);
            }
        }
        __syncwarp();
        for (int i = 0; ok && i < n_tiles; ++i) {
            const int key = k0 + i * kKeys;
            for (int b = 0; b < L::kPer; ++b, ++fills) {
                const uint32_t slot = fills % NS;
                if (fills >= NS && !(ok = __all_sync(0xffffffffu, mbar_wait_brief(&sh.empty[slot], (fills / NS - 1) & 1)))) break;
                if (leader) {
                    uint8_t* dst = smem + slot * kBlock;
                    mbar_arrive_expect_tx(&sh.full[slot], kBlock);
                    if (b < QB - 1) tma_load_3d(dst, &maps.k, &sh.full[slot], 64 * b, key, hk);
                    else if (b == QB - 1) tma_load_2d(dst, &maps.r, &sh.full[slot], 0, key);
                    else tma_load_3d(dst, &maps.v, &sh.full[slot], 64 * (b - QB), key, hv);
                }
                __syncwarp();
            }
        }
        if (!ok && lane == 0) record(a.error, 64);
        // nothing is in flight when the memory is given back
        for (int t = 0; t < kTiles; ++t)
            if (n[t] > 0) mbar_wait_brief(&sh.q_full[t], 0);
        for (uint32_t s = 0; s < NS; ++s)
            if (fills > s) mbar_wait_brief(&sh.full[s], ((fills - 1 - s) / NS) & 1);
    } else if (warp == 9) {
        // ---- products
        const bool leader = elect_one();
        constexpr uint32_t id_s = idesc_bf16_f32(kM, kKeys), id_o = idesc_bf16_f32(kM, 64, false, true);
        const uint64_t dq = desc_kmajor_sw128(smem_u32(smem + L::kQAt)), dk = desc_kmajor_sw128(smem_u32(smem)),
                       dv = desc_mnmajor_sw128(smem_u32(smem), kBlock);
        auto wait = [&](uint64_t* bar, uint32_t parity) { return __all_sync(0xffffffffu, mbar_wait_brief(bar, parity)) != 0; };
        bool ok = true;
        // scores of tile t and key tile i; the last tile that uses a block gives it back
        auto scores = [&](int t, int i, bool give) {
            for (int b = 0; ok && b < QB; ++b) {
                const uint32_t fill = i * L::kPer + b, slot = fill % NS;
                if (!(ok = wait(&sh.full[slot], (fill / NS) & 1))) return;
                tc_fence_after_sync();
                if (leader) {
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        mma_bf16(tmem + t * kKeys, dq + ((t * L::kPlace + b * kBlock) >> 4) + 2 * k, dk + (slot * kBlock >> 4) + 2 * k,
                                 id_s, (b > 0 || k > 0) ? 1u : 0u);
                    if (give) mma_commit(&sh.empty[slot]);
                }
                __syncwarp();
            }
            if (leader) mma_commit(&sh.s_full[t]);
            __syncwarp();
        };
        for (int t = 0; ok && t < kTiles; ++t)
            if (n[t] > 0) {
                if (!(ok = wait(&sh.q_full[t], 0))) break;
                scores(t, 0, t == kTiles - 1 || n[t + 1 < kTiles ? t + 1 : t] == 0);
            }
        for (int i = 0; ok && i < n_tiles; ++i) {
            for (int t = 0; ok && t < kTiles; ++t) {
                if (i < n[t]) {
                    if (!(ok = wait(&sh.p_full[t], i & 1))) break;
                    const bool give = t == 1 || i >= n[1];
                    for (int b = 0; ok && b < VB; ++b) {
                        const uint32_t fill = i * L::kPer + QB + b, slot = fill % NS;
                        if (!(ok = wait(&sh.full[slot], (fill / NS) & 1))) break;
                        tc_fence_after_sync();
                        if (leader) {
#pragma unroll
                            for (int k = 0; k < kKeys / 16; ++k)  // 16 keys of weights are 8 columns
                                mma_bf16_ta(tmem + L::kOut + t * V + 64 * b, tmem + t * kKeys + 8 * k,
                                            dv + ((slot * kBlock + k * 2048) >> 4), id_o, (i > 0 || k > 0) ? 1u : 0u);
                            if (give) mma_commit(&sh.empty[slot]);
                        }
                        __syncwarp();
                    }
                    if (leader) mma_commit(&sh.pv_done[t]);
                    __syncwarp();
                }
                if (ok && i + 1 < n[t]) scores(t, i + 1, t == 1 || i + 1 >= n[1]);
            }
        }
        if (!ok && lane == 0) record(a.error, 65);
        if (leader) mma_commit(&sh.drained);
        mbar_wait_brief(&sh.drained, 0);
    }
    __syncwarp();
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    if (warp == 9) tmem_dealloc(tmem, 512);
}

// A map of rows [tokens, heads, width] in boxes of 128 tokens x 64 channels of a head.
bool map_rows(CUtensorMap* map, const KvRows& r, int tokens, int heads, int width) {
    return make_tma_map_bf16_3d(map, r.data, width, tokens, r.head_stride ? heads : 1, r.token_stride,
                                r.head_stride ? r.head_stride : r.token_stride, 64, 128, 1);
}

template <int NOPE, int V>
cudaError_t expanded_t(const ExpandedArgs& a, cudaStream_t st) {
    using L = ECfg<NOPE, V>;
    static std::atomic<unsigned long long> ready{0};
    cudaError_t e = allow_smem(expanded_kernel<NOPE, V>, L::kSmem, ready);
    if (e != cudaSuccess) return e;
    Maps maps{};
    if (a.n_kv > 0 &&
        !(map_rows(&maps.q, a.q, a.n_q, a.n_heads, NOPE + kRopeDim) && map_rows(&maps.k, a.k, a.n_kv, a.n_heads, NOPE) &&
          make_tma_map_bf16_2d(&maps.r, a.k_rope.data, a.n_kv, kRopeDim, a.k_rope.token_stride, 128, 64) &&
          map_rows(&maps.v, a.v, a.n_kv, a.n_heads, V)))
        return cudaErrorInvalidValue;
    const int tiles = (a.max_q + kTiles * kM - 1) / (kTiles * kM);
    if (tiles > 65535) return cudaErrorInvalidConfiguration;
    return timed_launch("expanded_attention", st, [&] {
        expanded_kernel<NOPE, V><<<dim3(a.n_heads, a.n_seq, tiles), kThreads, L::kSmem, st>>>(a, maps);
        return cudaGetLastError();
    });
}

}  // namespace

cudaError_t launch_expanded_attention(const ExpandedArgs& a, int nope_dim, int v_dim, cudaStream_t st) {
    if (nope_dim == 128) return v_dim == 128 ? expanded_t<128, 128>(a, st) : expanded_t<128, 64>(a, st);
    return v_dim == 128 ? expanded_t<64, 128>(a, st) : expanded_t<64, 64>(a, st);
}

}  // namespace gdn
