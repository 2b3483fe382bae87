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

// PAIR: a thread block of a pair holds half of a key tile's keys (as keys) and half of its values' channels.
template <int NOPE, int V, bool PAIR> struct ECfg {
    static constexpr int kQBlocks = NOPE / 64 + 1;                     // of 64 channels
    static constexpr uint32_t kQ = kQBlocks * kBlock;                  // a query tile
    static constexpr uint32_t kKBlock = PAIR ? kBlock / 2 : kBlock;    // a key tile's 64 channels
    static constexpr uint32_t kVTile = kKeys * V * 2 / (PAIR ? 2 : 1);
    static constexpr int kPitch = 2 * V + 16;                          // of a staged output row: neighbours in different banks
    static constexpr uint32_t kStaged = (kM * kPitch + 1023) / 1024 * 1024, kPlace = kQ > kStaged ? kQ : kStaged;
    static constexpr uint32_t kRoom = kSmemMax - kSharedBytes - kTiles * kPlace;
    static constexpr int kFit = kRoom / (kQBlocks * kKBlock + kVTile), NV = kFit < 2 ? 2 : kFit;  // slots of value tiles
    static constexpr int kFitK = (kRoom - NV * kVTile) / kKBlock, NK = kFitK < kMaxSlots ? kFitK : kMaxSlots;  // of key blocks
    static constexpr uint32_t kVAt = NK * kKBlock, kQAt = kVAt + NV * kVTile, kSharedAt = kQAt + kTiles * kPlace;
    static constexpr uint32_t kSmem = kSharedAt + kSharedBytes;
    static constexpr uint32_t kOut = kTiles * kKeys;                   // tensor memory: scores (weights) of both tiles, outputs
    static constexpr int kRows = PAIR ? 2 * kM : kM;                   // of a product
    static_assert(NK > kQBlocks, "a tile's keys and the next one's first fit");
    static_assert(NV <= kMaxSlots && (!PAIR || V == 128), "a half of the channels is a 128-byte row");
};

struct Shared {
    uint64_t k_full[kMaxSlots], k_empty[kMaxSlots], v_full[kMaxSlots], v_empty[kMaxSlots];
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

// The same by a pair of thread blocks: 128 rows of A and half of B's N from each.
__device__ __forceinline__ void mma_bf16_ta_pair(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                                 uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}
// mbar_wait_brief that acquires at cluster scope.
__device__ __forceinline__ bool wait_cluster(uint64_t* bar, uint32_t parity) {
    if (mbar_try_wait_cluster(bar, parity)) return true;
    const long long c0 = clock64();
    for (uint32_t n = 1; !mbar_try_wait_cluster(bar, parity); ++n)
        if ((n & 255u) == 0 && clock64() - c0 > (1ll << 32)) return false;
    return true;
}

struct Maps {
    CUtensorMap q, k, r, v;
};

template <int NOPE, int V, bool PAIR>
__global__ void __launch_bounds__(kThreads, 1) expanded_kernel(const ExpandedArgs a, const __grid_constant__ Maps maps) {
    using L = ECfg<NOPE, V, PAIR>;
    constexpr int NK = L::NK, NV = L::NV, QB = L::kQBlocks;
    extern __shared__ __align__(1024) uint8_t smem[];
    Shared& sh = *reinterpret_cast<Shared*>(smem + L::kSharedAt);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = PAIR ? static_cast<int>(blockIdx.x & 1) : 0;
    const int h = PAIR ? blockIdx.x >> 1 : blockIdx.x, seq = blockIdx.y;
    const int q0 = a.cu_q[seq], qn = a.cu_q[seq + 1] - q0, k0 = a.cu_kv[seq], kv = a.cu_kv[seq + 1] - k0;
    // most keys first; tile t of a thread block: rows row0 + t kRows + rank kM onwards
    const int row0 = (static_cast<int>(gridDim.z) - 1 - static_cast<int>(blockIdx.z)) * (kTiles * L::kRows);
    if (row0 >= qn) return;
    const int start = kv - qn;  // position of the sequence's first query
    int n[kTiles];              // key tiles of each query tile (of a pair's both)
#pragma unroll
    for (int t = 0; t < kTiles; ++t) {
        const int last = min(row0 + (t + 1) * L::kRows, qn) - 1;  // the tile's last query
        n[t] = last >= row0 + t * L::kRows && start + last >= 0 ? (start + last) / kKeys + 1 : 0;
    }
    const int n_tiles = max(n[0], n[1]);
    if (smem_u32(smem) & 1023u) {
        if (tid == 0) record(a.error, 66);
        return;
    }
    if (tid == 0) {
        for (int i = 0; i < NK; ++i) {
            mbar_init(&sh.k_full[i], 1);
            mbar_init(&sh.k_empty[i], 1);
        }
        for (int i = 0; i < NV; ++i) {
            mbar_init(&sh.v_full[i], 1);
            mbar_init(&sh.v_empty[i], 1);
        }
        for (int t = 0; t < kTiles; ++t) {
            mbar_init(&sh.q_full[t], 1);
            mbar_init(&sh.s_full[t], 1);
            mbar_init(&sh.p_full[t], PAIR ? 8 : 4);
            mbar_init(&sh.pv_done[t], 1);
        }
        mbar_init(&sh.drained, 1);
        fence_barrier_init();
    }
    if (warp == 9) {
        if (PAIR) tmem_alloc_pair(&sh.tmem_slot, 512);
        else tmem_alloc(&sh.tmem_slot, 512);
    }
    tc_fence_before_sync();
    __syncthreads();
    if (PAIR) {  // the other's barriers are initialised
        cluster_arrive();
        cluster_wait();
    }
    tc_fence_after_sync();
    const uint32_t tmem = sh.tmem_slot;

    if (warp < 8) {
        // ---- softmax: a thread's row
        const int t = warp >> 2, r = tid & (kM - 1), row = row0 + t * L::kRows + rank * kM + r;
        const bool mine = row < qn;
        const int lim = mine ? max(0, min(start + row + 1, kv)) : 0;  // keys that the row sees
        const int low = __reduce_min_sync(0xffffffffu, lim);
        const uint32_t t_lane = (32u * (warp & 3)) << 16;
        const uint32_t t_score = tmem + t_lane + t * kKeys, t_out = tmem + t_lane + L::kOut + t * V;
        const uint32_t p_full = PAIR ? map_to_rank(smem_u32(&sh.p_full[t]), 0) : 0;
        const float scale2 = a.scale * kLog2e;
        float m = -INFINITY, l = 0.0f;
        bool ok = true;
        for (int i = 0; i < n[t]; ++i) {
            const int key0 = i * kKeys;
            // A wait that gave up is not waited for again, but the warp goes on through the tiles (with
            // results that are invalid): the barriers between the warps stay complete.
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
            const bool cleared = key0 + kKeys > kv && (t == 0 || i >= n[0]);
            if (cleared) {
                const int slot = i % NV;
                if (ok && !(ok = __all_sync(0xffffffffu, mbar_wait_brief(&sh.v_full[slot], rank ? 0 : (i / NV) & 1))) && lane == 0)
                    record(a.error, 62);  // (the second block's only ones on its own barrier)
                for (uint32_t b = 0; b < L::kVTile; b += kBlock) {
                    uint4* rows = reinterpret_cast<uint4*>(smem + L::kVAt + slot * L::kVTile + b);
                    for (int x = 8 * (kv - key0) + r; x < 8 * kKeys; x += kM) rows[x] = make_uint4(0, 0, 0, 0);
                }
                fence_proxy_async_smem();
            }
            tmem_wait_st();
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) {
                // Weights are in tensor memory by now; only zeroed rows, in shared memory, are to be released (a
                // releasing arrival on the other thread block's barrier takes some 1500 cycles).
                if (!PAIR) mbar_arrive(&sh.p_full[t]);
                else if (cleared) mbar_arrive_remote(p_full);
                else mbar_arrive_remote_relaxed(p_full, l);
            }
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
        // ---- loads: of a pair the first thread block's keys are the tile's first half, its values the first channels
        const bool leader = elect_one();
        const int hq = a.q.head_stride ? h : 0, hk = a.k.head_stride ? h : 0, hv = a.v.head_stride ? h : 0;
        // The products' issuer, in a pair's first thread block, waits for both blocks' bytes on a barrier of its
        // own.  But the second block's values behind a sequence's end wait for its softmax, which clears them.
        const uint32_t both = PAIR ? 2 : 1;
        auto load = [&](uint8_t* dst, const CUtensorMap* map, uint64_t* bar, int x, int y, int z, bool here) {
            if (!PAIR || here) tma_load_3d(dst, map, bar, x, y, z);
            else tma_load_3d_pair(dst, map, map_to_rank(smem_u32(bar), 0), x, y, z);
        };
        bool ok = true;
        uint32_t fills = 0;  // of key blocks
        int i = 0;
        if (leader && n_tiles > 0) {
            for (int t = 0; t < kTiles; ++t) {
                if (n[t] == 0) continue;
                if (rank == 0) mbar_arrive_expect_tx(&sh.q_full[t], both * L::kQ);
                for (int b = 0; b < QB; ++b)
                    load(smem + L::kQAt + t * L::kPlace + b * kBlock, &maps.q, &sh.q_full[t], 64 * b,
                         q0 + row0 + t * L::kRows + rank * kM, hq, false);
            }
        }
        __syncwarp();
        for (; i < n_tiles; ++i) {
            const int key = k0 + i * kKeys, slot_v = i % NV;
            for (int b = 0; ok && b < QB; ++b) {
                const uint32_t slot = fills % NK;
                if (fills >= NK && !(ok = __all_sync(0xffffffffu, mbar_wait_brief(&sh.k_empty[slot], (fills / NK - 1) & 1)))) break;
                ++fills;
                if (leader) {
                    uint8_t* dst = smem + slot * L::kKBlock;
                    if (rank == 0) mbar_arrive_expect_tx(&sh.k_full[slot], both * L::kKBlock);
                    if (b < QB - 1) load(dst, &maps.k, &sh.k_full[slot], 64 * b, key + rank * (kKeys / 2), hk, false);
                    else load(dst, &maps.r, &sh.k_full[slot], 0, key + rank * (kKeys / 2), 0, false);
                }
                __syncwarp();
            }
            if (ok && i >= NV) ok = __all_sync(0xffffffffu, mbar_wait_brief(&sh.v_empty[slot_v], (i / NV - 1) & 1));
            if (!ok) break;
            if (leader) {
                uint8_t* dst = smem + L::kVAt + slot_v * L::kVTile;
                const bool own = PAIR && (i + 1) * kKeys > kv;  // each block waits for its own
                if (rank == 0 || own) mbar_arrive_expect_tx(&sh.v_full[slot_v], (own ? 1 : both) * L::kVTile);
                for (uint32_t b = 0; b < L::kVTile / kBlock; ++b)
                    load(dst + b * kBlock, &maps.v, &sh.v_full[slot_v], 64 * (b + rank), key, hv, own);
            }
            __syncwarp();
        }
        // nothing is in flight when the memory is given back
        if (!ok) {
            if (lane == 0) record(a.error, 64);
            if (rank == 0) {
                for (uint32_t f = fills > NK ? fills - NK : 0; f < fills; ++f) mbar_wait_brief(&sh.k_full[f % NK], (f / NK) & 1);
                for (int f = max(0, i - NV); f < i; ++f) mbar_wait_brief(&sh.v_full[f % NV], (f / NV) & 1);
            } else {  // its bytes are counted in the other block: a millisecond will do
                const uint64_t t0 = globaltimer_ns();
                const long long c0 = clock64();
                while (globaltimer_ns() - t0 < 1000000 && clock64() - c0 < (1ll << 24)) {}
            }
        }
        if (rank == 0)
            for (int t = 0; t < kTiles; ++t)
                if (n[t] > 0) mbar_wait_brief(&sh.q_full[t], 0);
    } else if (warp == 9 && rank == 0) {
        // ---- products (of a pair by its first thread block)
        const bool leader = elect_one();
        constexpr uint32_t id_s = idesc_bf16_f32(L::kRows, kKeys), id_o = idesc_bf16_f32(L::kRows, V, false, true);
        const uint64_t dq = desc_kmajor_sw128(smem_u32(smem + L::kQAt)), dk = desc_kmajor_sw128(smem_u32(smem)),
                       dv = desc_mnmajor_sw128(smem_u32(smem + L::kVAt), kBlock);
        auto wait = [&](uint64_t* bar, uint32_t parity) {
            return __all_sync(0xffffffffu, PAIR ? wait_cluster(bar, parity) : mbar_wait_brief(bar, parity)) != 0;
        };
        auto commit = [&](uint64_t* bar) {
            if (PAIR) mma_commit_pair(bar, 3);
            else mma_commit(bar);
        };
        bool ok = true;
        // scores of tile t and key tile i; the last tile that uses a block gives it back
        auto scores = [&](int t, int i, bool give) {
            for (int b = 0; b < QB; ++b) {
                const uint32_t fill = i * QB + b, slot = fill % NK;
                if (!(ok = wait(&sh.k_full[slot], (fill / NK) & 1))) return;
                tc_fence_after_sync();
                if (leader) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const uint64_t da = dq + ((t * L::kPlace + b * kBlock) >> 4) + 2 * k, db = dk + (slot * L::kKBlock >> 4) + 2 * k;
                        if (PAIR) mma_bf16_pair(tmem + t * kKeys, da, db, id_s, (b > 0 || k > 0) ? 1u : 0u);
                        else mma_bf16(tmem + t * kKeys, da, db, id_s, (b > 0 || k > 0) ? 1u : 0u);
                    }
                    if (give) commit(&sh.k_empty[slot]);
                }
                __syncwarp();
            }
            if (leader) commit(&sh.s_full[t]);
            __syncwarp();
        };
        for (int t = 0; ok && t < kTiles; ++t)
            if (n[t] > 0) {
                if (!(ok = wait(&sh.q_full[t], 0))) break;
                scores(t, 0, t == 1 || n[1] == 0);
            }
        for (int i = 0; ok && i < n_tiles; ++i) {
            for (int t = 0; ok && t < kTiles; ++t) {
                if (i < n[t]) {
                    const int slot = i % NV;
                    if (!(ok = wait(&sh.p_full[t], i & 1))) break;
                    if (!(ok = wait(&sh.v_full[slot], (i / NV) & 1))) break;
                    tc_fence_after_sync();
                    if (leader) {
#pragma unroll
                        for (int k = 0; k < kKeys / 16; ++k) {  // 16 keys of weights are 8 columns
                            const uint32_t d = tmem + L::kOut + t * V, p = tmem + t * kKeys + 8 * k;
                            const uint64_t db = dv + ((slot * L::kVTile + k * 2048) >> 4);
                            if (PAIR) mma_bf16_ta_pair(d, p, db, id_o, (i > 0 || k > 0) ? 1u : 0u);
                            else mma_bf16_ta(d, p, db, id_o, (i > 0 || k > 0) ? 1u : 0u);
                        }
                        if (t == 1 || i >= n[1]) commit(&sh.v_empty[slot]);
                        commit(&sh.pv_done[t]);
                    }
                    __syncwarp();
                }
                if (ok && i + 1 < n[t]) scores(t, i + 1, t == 1 || i + 1 >= n[1]);
            }
        }
        if (!ok && lane == 0) record(a.error, 65);
        if (leader) {
            if (PAIR) mma_commit_pair(&sh.drained, 1);
            else mma_commit(&sh.drained);
        }
        mbar_wait_brief(&sh.drained, 0);
    }
    __syncwarp();
    tc_fence_before_sync();
    __syncthreads();
    if (PAIR) {  // nothing of the other is on its way here any more, and both are done with tensor memory
        cluster_arrive();
        cluster_wait();
    }
    tc_fence_after_sync();
    if (warp == 9) {
        if (PAIR) tmem_dealloc_pair(tmem, 512);
        else tmem_dealloc(tmem, 512);
    }
}

// A map of rows [tokens, heads, width] in boxes of `box` tokens x 64 channels of a head.
bool map_rows(CUtensorMap* map, const KvRows& r, int tokens, int heads, int width, int box) {
    return make_tma_map_bf16_3d(map, r.data, width, tokens, r.head_stride ? heads : 1, r.token_stride,
                                r.head_stride ? r.head_stride : r.token_stride, 64, box, 1);
}

template <int NOPE, int V, bool PAIR>
cudaError_t expanded_t(const ExpandedArgs& a, cudaStream_t st) {
    using L = ECfg<NOPE, V, PAIR>;
    static std::atomic<unsigned long long> ready{0};
    cudaError_t e = allow_smem(expanded_kernel<NOPE, V, PAIR>, L::kSmem, ready);
    if (e != cudaSuccess) return e;
    Maps maps{};
    const int keys = PAIR ? kKeys / 2 : kKeys;
    if (a.n_kv > 0 &&
        !(map_rows(&maps.q, a.q, a.n_q, a.n_heads, NOPE + kRopeDim, kM) && map_rows(&maps.k, a.k, a.n_kv, a.n_heads, NOPE, keys) &&
          map_rows(&maps.r, KvRows{a.k_rope.data, a.k_rope.token_stride, 0}, a.n_kv, 1, kRopeDim, keys) &&
          map_rows(&maps.v, a.v, a.n_kv, a.n_heads, V, kKeys)))
        return cudaErrorInvalidValue;
    const int tiles = (a.max_q - 1) / (kTiles * L::kRows) + 1;
    if (tiles > 65535) return cudaErrorInvalidConfiguration;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(a.n_heads * (PAIR ? 2 : 1), a.n_seq, tiles);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = L::kSmem;
    cfg.stream = st;
    cudaLaunchAttribute two{};
    two.id = cudaLaunchAttributeClusterDimension;
    two.val.clusterDim.x = 2;
    two.val.clusterDim.y = two.val.clusterDim.z = 1;
    cfg.attrs = &two;
    cfg.numAttrs = PAIR ? 1 : 0;
    return timed_launch("expanded_attention", st, [&] { return cudaLaunchKernelEx(&cfg, expanded_kernel<NOPE, V, PAIR>, a, maps); });
}

template <int NOPE>
cudaError_t expanded_n(const ExpandedArgs& a, int v_dim, cudaStream_t st) {
    if (v_dim == 64) return expanded_t<NOPE, 64, false>(a, st);
    return a.max_q > kTiles * kM ? expanded_t<NOPE, 128, true>(a, st) : expanded_t<NOPE, 128, false>(a, st);
}

}  // namespace

cudaError_t launch_expanded_attention(const ExpandedArgs& a, int nope_dim, int v_dim, cudaStream_t st) {
    return nope_dim == 128 ? expanded_n<128>(a, v_dim, st) : expanded_n<64>(a, v_dim, st);
}

}  // namespace gdn
