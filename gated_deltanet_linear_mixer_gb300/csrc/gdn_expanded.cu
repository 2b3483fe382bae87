// Causal attention of the expanded form, on the 5th-generation tensor cores.
//
// The mathematics, in powers of two (y = scale log2 e q . k, k = (k_h | k_rope)):
//   w_rj = 2^(y_rj - m_r),   o_r = sum_j w_rj v_j / sum_j w_rj
// with a reference m_r that lags behind the row's maximum by at most 2^kLazy, so
// that the output is rescaled only where the maximum rises by more than that.
// Weights are rounded to bf16 (the values' type, as the tensor core asks); the sum
// takes them unrounded, which takes 3% less time than the sum of the rounded ones
// and costs at most 0.0001 of the output's relative error (0.0021 and 0.0023 of the
// two cases below).
//
// A thread block takes two tiles of 128 queries of a head and walks the keys in
// tiles of 128 up to the last query's position.  While one tile's softmax runs, the
// tensor core works for the other.  S of a tile takes 128 columns of tensor memory,
// O as many; the weights overwrite their scores' columns and are the second
// product's A operand where they lie.  Keys stream through a ring of
// 16 KB blocks (128 keys x 64 channels), values through one of whole tiles; the
// position keys come from their own array, which all heads share.  There is a thread
// block an item (sequence, queries, head), the longest sequences' first, and one that is done
// takes on the item of a block that has not started (try_cancel), whose loads begin
// while it finishes its own: 137 and 172 us where every 152nd item was a block's from
// the start, 131 and 163 us so (the two cases below, at that stage).  Where an item
// has one tile of queries, both halves of the thread block take it, for every other
// key tile each, and join their results: a key tile alone takes 1.5 us, 1.0 us so
// (pairs of tiles: 1.9), and 16 ragged prompts take 145 us instead of 159.
//
// Roles: 8 softmax warps (a thread a row; a rescaling concerns one warp's rows
// alone), a warp for the loads, one issuing the products, in the order
// O0 += P0 V, S0 = Q0 K', O1 += P1 V, S1 = Q1 K'.  Every wait is bounded (2 s); a
// wait that gives up records a code (60..66) in the cache operators' device error
// word.
//
// What bounds it (128 channels, 128 wide values): for 128 keys and both tiles the
// tensor core takes 24 instructions of S (128 x 128 x 16, 71 cycles each, measured
// alone) and 16 of O (74, their A operand in tensor memory): 2890 cycles.  The keys
// and values that come in meanwhile, 80 KB, take 640 cycles of the shared memory's
// bandwidth, which those products use in full: 3530.  3680 are reached: 1.92 us at 1.91
// GHz, the SM clock by the kernel's own counters.  The exponentials (32 a cycle and SM:
// 1024 cycles) do not bound it.  4096 tokens, 32 heads: 126 us, 1.36 PFLOP/s, of which 54
// such steps an SM are 104, the last tiles of 3.4 items, which one query tile walks alone, 5,
// the items' ends 6 and the call's start and end 7; 16 ragged prompts of up to 1100 tokens
// behind up to 3000: 142 us, 1.14 PFLOP/s, where tiles that are partly masked or empty weigh more.
//
// Tried and slower (us, the two cases above, with fixed shares and 208 and 88 registers): pairs of thread blocks
// that share keys (134 and 215 where a block of the same form took 141 and 179); two threads a
// row (165 against 140); weights handed over by halves (144); an issuing warp per
// tile (146 and 180); one ring for keys and values (148 and 190); a thread that
// polls both tiles' barriers and issues what is ready (149).  No faster: scores read by
// one load of 128 columns, three-operand maxima, the first item looked up before the
// thread block's barriers are there.
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
// The reference is rounded (m = fl(scale log2 e top)) and a weight 2^fma(scale log2 e, score, -m), so that
// a row's largest weight is 2^e, e the rounding's error: up to half a unit of m's last place, which from 2^31 on
// leaves fp32's exponents (all weights 0, or infinite).  Beyond kFar, where e is 2^-15, differences are taken
// before the scale: two operations a pair of scores instead of one (always so: 134 and 153 us where the two cases above
// take 127 and 143; by this rule as long as before).
constexpr float kFar = 1024.0f;
constexpr uint32_t kBlock = 16384;  // 128 rows x 64 channels
constexpr uint32_t kSmemMax = 232448, kSharedBytes = 2944;
constexpr int kMaxSlots = 12;

template <int NOPE, int V> struct ECfg {
    static constexpr int kQBlocks = NOPE / 64 + 1;     // of a query or key tile
    static constexpr uint32_t kQ = kQBlocks * kBlock, kVTile = kKeys * V * 2;
    static constexpr uint32_t kRoom = kSmemMax - kSharedBytes - kTiles * kQ;
    static constexpr int NV = kRoom / (kQ + kVTile) < 2 ? 2 : kRoom / (kQ + kVTile);  // slots of value tiles
    static constexpr int NK = (kRoom - NV * kVTile) / kBlock;                         // of key blocks
    static constexpr uint32_t kVAt = NK * kBlock, kQAt = kVAt + NV * kVTile, kSharedAt = kQAt + kTiles * kQ;
    static constexpr uint32_t kSmem = kSharedAt + kSharedBytes;
    static constexpr uint32_t kOut = kTiles * kKeys;   // tensor memory: scores (weights) of both tiles, outputs
    static_assert(NK > kQBlocks && NK <= kMaxSlots && NV <= kMaxSlots, "a tile's keys and some of the next one's fit");
};

// One block of queries of a head.
struct Item {
    int h, q0, qn, k0, kv, row0, start;  // h < 0: there is none
    int n0, n1, n_tiles;                 // key tiles of each query tile; that are loaded
    int step;                            // 2: both are the first one, which walk every other key tile each
};
constexpr int kItems = 2;  // that the loading warp tells the others of

struct Shared {
    uint4 next;  // the answer to a request for another thread block's item
    uint64_t next_full, item_full[kItems], item_empty[kItems];
    Item item[kItems];
    uint64_t k_full[kMaxSlots], k_empty[kMaxSlots], v_full[kMaxSlots], v_empty[kMaxSlots];
    uint64_t q_full[kTiles], q_empty[kTiles], s_full[kTiles], p_full[kTiles], pv_done[kTiles], drained;
    uint64_t stat_full[kTiles], merged[kTiles];  // of query tiles that were walked by halves
    float2 stat[kTiles][kM];                     // their references and sums
    uint32_t tmem_slot;
};
static_assert(sizeof(Shared) <= kSharedBytes, "part of kSmem");


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
// 32 bytes of a row: in one instruction where they are aligned to as many.  A warp's
// rows lie apart, so that its stores take the load and store unit by the instruction:
// 4096 tokens take 129 us with, 131.5 without, 16 ragged prompts 159 and 163.
__device__ __forceinline__ void store32(bf16* to, const uint32_t* v, bool wide) {
    if (wide) {
        asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(to), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]),
                     "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                     : "memory");
    } else {
        reinterpret_cast<uint4*>(to)[0] = make_uint4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<uint4*>(to)[1] = make_uint4(v[4], v[5], v[6], v[7]);
    }
}

// What a launch walks: (sequence, block of queries) pairs, of every head.
constexpr int kPairs = 1024;
struct Plan {
    CUtensorMap q, k, r, v;
    uint32_t pair[kPairs];     // sequence << 16 | block
};

// Asks for a thread block of this grid that has not started, which then never does: its
// number comes into the 16 bytes at `to`, and completes as many on `bar`.
__device__ __forceinline__ void ask_for_block(uint4* to, uint64_t* bar) {
    asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
                     smem_u32(to)),
                 "r"(smem_u32(bar))
                 : "memory");
}
// The answer: a block, or -1 where none was left (no more may be asked for then).
__device__ __forceinline__ int block_answered(const uint4* at) {
    uint32_t got, x;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        ".reg .b128 r;\n\t"
        "ld.shared.b128 r, [%2];\n\t"
        "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t"
        "mov.u32 %1, 0;\n\t"
        "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, r;\n\t}"
        : "=r"(got), "=r"(x)
        : "r"(smem_u32(at))
        : "memory");
    return got ? static_cast<int>(x) : -1;
}

template <int NOPE, int V>
__global__ void __launch_bounds__(kThreads, 1) expanded_kernel(const ExpandedArgs a, const __grid_constant__ Plan plan) {
    using L = ECfg<NOPE, V>;
    constexpr int NK = L::NK, NV = L::NV, QB = L::kQBlocks;
    constexpr int kRows = kTiles * kM;  // of an item
    extern __shared__ __align__(1024) uint8_t smem[];
    Shared& sh = *reinterpret_cast<Shared*>(smem + L::kSharedAt);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    auto item_of = [&](int at, Item& x) {  // whether there is one
        const int p = at / a.n_heads, seq = plan.pair[p] >> 16, block = plan.pair[p] & 0xFFFF;
        x.h = at - p * a.n_heads;
        x.q0 = a.cu_q[seq];
        x.qn = a.cu_q[seq + 1] - x.q0;
        x.k0 = a.cu_kv[seq];
        x.kv = a.cu_kv[seq + 1] - x.k0;
        x.row0 = block * kRows;  // tile t: rows row0 + t kM onwards
        if (x.row0 >= x.qn) return false;
        x.start = x.kv - x.qn;  // position of the sequence's first query
        auto tiles = [&](int t) {
            const int last = min(x.row0 + (t + 1) * kM, x.qn) - 1;  // the tile's last query
            return last >= x.row0 + t * kM && x.start + last >= 0 ? (x.start + last) / kKeys + 1 : 0;
        };
        x.n0 = tiles(0);
        x.n1 = tiles(1);
        x.n_tiles = max(x.n0, x.n1);
        x.step = 1;
        if (x.row0 + kM >= x.qn && x.n_tiles > 1) {
            x.step = 2;
            x.n1 = x.n_tiles / 2;
            x.n0 -= x.n1;
        }
        return true;
    };
    // The k-th item as the loading warp tells it; false where the wait for it gave up.
    auto take = [&](uint32_t k, Item& x) {
        const uint32_t s = k % kItems;
        if (!__all_sync(0xffffffffu, mbar_wait_brief(&sh.item_full[s], (k / kItems) & 1))) return false;
        x = sh.item[s];
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.item_empty[s]);
        return true;
    };
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
            mbar_init(&sh.q_empty[t], 1);
            mbar_init(&sh.s_full[t], 1);
            mbar_init(&sh.p_full[t], 4);
            mbar_init(&sh.pv_done[t], 1);
            mbar_init(&sh.stat_full[t], 4);
            mbar_init(&sh.merged[t], 4);
        }
        for (int i = 0; i < kItems; ++i) {
            mbar_init(&sh.item_full[i], 1);
            mbar_init(&sh.item_empty[i], 9);
        }
        mbar_init(&sh.next_full, 1);
        mbar_init(&sh.drained, 1);
        fence_barrier_init();
    }
    if (warp == 8 && a.n_kv > 0) {
        tma_prefetch_desc(&plan.q);
        tma_prefetch_desc(&plan.k);
        tma_prefetch_desc(&plan.r);
        tma_prefetch_desc(&plan.v);
    }
    if (warp == 9) {
        tmem_alloc(&sh.tmem_slot, 512);
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = sh.tmem_slot;

    // the softmax holds a row's scores in registers: 2 x 192 + 120 of the 3 x 168 that a thread block has (with 208 and 88
    // the issuing warp spills: 136 and 159 us where the two cases take 125 and 145)
    if (warp < 8) {
        regs_inc<192>();
        // ---- softmax: a thread's row
        const int t = warp >> 2, r = tid & (kM - 1);
        const uint32_t t_lane = (32u * (warp & 3)) << 16;
        const uint32_t t_score = tmem + t_lane + t * kKeys, t_out = tmem + t_lane + L::kOut + t * V;
        const float scale2 = a.scale * kLog2e;
        const bool wide = (reinterpret_cast<uintptr_t>(a.out) & 31u) == 0;
        bool ok = true;
        uint32_t steps = 0, values = 0, merges = 0;  // key tiles of this query tile so far, of the items before
        for (uint32_t item = 0; ok; ++item) {
            Item x;
            if (!(ok = take(item, x)) && lane == 0) record(a.error, 60);
            if (!ok || x.h < 0) break;
            const int row = x.row0 + (x.step == 2 ? 0 : t * kM) + r, n = t ? x.n1 : x.n0;
            const bool mine = row < x.qn;
            const int lim = mine ? max(0, min(x.start + row + 1, x.kv)) : 0;  // keys that the row sees
            const int low = __reduce_min_sync(0xffffffffu, lim);
            float m = -INFINITY, l = 0.0f;  // the reference (a score before the scale), the sum
            bool far = false;               // whether one of the warp's rows has a reference beyond kFar
            int kt = x.step == 2 ? t : 0;  // the key tile
            for (int i = 0; i < n; ++i, ++steps, kt += x.step) {
                const int key0 = kt * kKeys;
                // A wait that gave up is not waited for again, but the warp goes on through the tiles (with
                // results that are invalid): the barriers between the warps stay complete.
                if (ok && !(ok = __all_sync(0xffffffffu, mbar_wait_brief(&sh.s_full[t], steps & 1))) && lane == 0) record(a.error, 60);
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
                const float top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
                const bool lift = __any_sync(0xffffffffu, (top - m) * scale2 > kLazy);
                float f = 1.0f;
                if (lift) {
                    const float mn = fmaxf(m, top);
                    f = m == -INFINITY ? 0.0f : exp2_ftz((m - mn) * scale2);
                    m = mn;
                    l *= f;
                    far = far || __any_sync(0xffffffffu, m != -INFINITY && fabsf(m * scale2) > kFar);
                }
                float ref = m == -INFINITY ? 0.0f : -m * scale2;
                if (far) {
                    const float less = m == -INFINITY ? 0.0f : m;
#pragma unroll
                    for (int j = 0; j < kKeys; ++j) s[j] -= less;
                    ref = 0.0f;
                }
                const uint64_t scale22 = pair(scale2, scale2), ref2 = pair(ref, ref);
                uint64_t sums[2] = {0, 0};
#pragma unroll
                for (int c = 0; c < kKeys; c += 64) {
                    uint32_t p[32];
#pragma unroll
                    for (int j = 0; j < 64; j += 2) {
                        float w0, w1;
                        unpair(fma2(pair(s[c + j], s[c + j + 1]), scale22, ref2), w0, w1);
                        w0 = exp2_ftz(w0);
                        w1 = exp2_ftz(w1);
                        p[j / 2] = pack_bf16x2(w0, w1);
                        sums[(j / 2) & 1] = add2(sums[(j / 2) & 1], pair(w0, w1));
                    }
                    tmem_st32(t_score + c / 2, p);
                }
                float s0, s1;
                unpair(add2(sums[0], sums[1]), s0, s1);
                l += s0 + s1;
                if (lift && i > 0) {  // the output so far
                    if (ok && !(ok = __all_sync(0xffffffffu, mbar_wait_brief(&sh.pv_done[t], (steps - 1) & 1))) && lane == 0)
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
                if (key0 + kKeys > x.kv && (t == 0 || i >= x.n0 || x.step == 2)) {
                    const uint32_t slot = (values + kt) % NV;
                    if (ok && !(ok = __all_sync(0xffffffffu, mbar_wait_brief(&sh.v_full[slot], ((values + kt) / NV) & 1))) && lane == 0)
                        record(a.error, 62);
                    for (uint32_t b = 0; b < L::kVTile; b += kBlock) {
                        uint4* rows = reinterpret_cast<uint4*>(smem + L::kVAt + slot * L::kVTile + b);
                        for (int y = 8 * (x.kv - key0) + r; y < 8 * kKeys; y += kM) rows[y] = make_uint4(0, 0, 0, 0);
                    }
                    fence_proxy_async_smem();
                }
                tmem_wait_st();
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh.p_full[t]);
            }
            values += x.n_tiles;
            // ---- epilogue
            if (n > 0 && ok && !(ok = __all_sync(0xffffffffu, mbar_wait_brief(&sh.pv_done[t], (steps - 1) & 1))) && lane == 0)
                record(a.error, 63);
            tc_fence_after_sync();
            bf16* out = static_cast<bf16*>(a.out) + (static_cast<size_t>(x.q0 + row) * a.n_heads + x.h) * V;
            if (x.step == 2) {  // both halves' results, half of the channels by the warps of each
                auto meet = [&](uint64_t* bars) {  // the other half's warps
                    tc_fence_before_sync();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bars[t]);
                    if (ok && !(ok = __all_sync(0xffffffffu, mbar_wait_brief(&bars[1 - t], merges & 1))) && lane == 0) record(a.error, 63);
                    tc_fence_after_sync();
                };
                sh.stat[t][r] = make_float2(m, l);
                meet(sh.stat_full);
                const float2 s0 = sh.stat[0][r], s1 = sh.stat[1][r];
                const float top = fmaxf(s0.x, s1.x);
                float f0 = s0.y == 0.0f ? 0.0f : exp2_ftz((s0.x - top) * scale2), f1 = s1.y == 0.0f ? 0.0f : exp2_ftz((s1.x - top) * scale2);
                const float sum = s0.y * f0 + s1.y * f1, inv = sum == 0.0f ? 0.0f : 1.0f / sum;
                f0 *= inv;
                f1 *= inv;
                const uint32_t t_both = tmem + t_lane + L::kOut;
#pragma unroll 1
                for (int c = t * (V / 2); c < (t + 1) * (V / 2); c += 32) {
                    float v0[32], v1[32];
                    tmem_ld32(t_both + c, v0);
                    tmem_ld32(t_both + V + c, v1);
                    if (mine && ok) {
#pragma unroll
                        for (int e = 0; e < 32; e += 16) {
                            uint32_t y[8];
#pragma unroll
                            for (int k = 0; k < 8; ++k)
                                y[k] = pack_bf16x2(v0[e + 2 * k] * f0 + v1[e + 2 * k] * f1, v0[e + 2 * k + 1] * f0 + v1[e + 2 * k + 1] * f1);
                            store32(out + c + e, y, wide);
                        }
                    }
                }
                meet(sh.merged);  // nothing of the other's is read any more
                ++merges;
                continue;
            }
            const float inv = l == 0.0f ? 0.0f : 1.0f / l;  // a sum that is no number stays one
#pragma unroll 1
            for (int c = 0; c < V; c += 32) {
                float v[32];
                if (n > 0) tmem_ld32(t_out + c, v);
                if (mine && ok) {
#pragma unroll
                    for (int e = 0; e < 32; e += 16) {
                        uint32_t y[8];
#pragma unroll
                        for (int k = 0; k < 8; ++k) y[k] = n > 0 ? pack_bf16x2(v[e + 2 * k] * inv, v[e + 2 * k + 1] * inv) : 0u;
                        store32(out + c + e, y, wide);
                    }
                }
            }
            tc_fence_before_sync();
        }
    } else {
        regs_dec<120>();
        if (warp == 8) {
            // ---- loads
            const bool leader = elect_one();
            bool ok = true;
            uint32_t keys = 0, values = 0, queries[kTiles] = {0, 0};  // fills so far
            uint32_t asked = 0;
            auto ask = [&] {
                __syncwarp();
                if (leader) {
                    fence_proxy_async_smem();  // the last answer was read
                    mbar_arrive_expect_tx(&sh.next_full, sizeof(sh.next));
                    ask_for_block(&sh.next, &sh.next_full);
                }
                ++asked;
            };
            auto answer = [&] {  // of the last one asked for
                if (!__all_sync(0xffffffffu, mbar_wait_brief(&sh.next_full, (asked - 1) & 1))) {
                    ok = false;
                    return -1;
                }
                return block_answered(&sh.next);
            };
            int at = blockIdx.x;   // a block an item: this one's, then those of blocks that never start
            bool waiting = false;  // for an answer
            for (uint32_t item = 0; ok; ++item) {
                Item x;
                const bool some = at >= 0 && item_of(at, x);
                if (!some) x.h = -1;
                const uint32_t place = item % kItems;
                if (item >= kItems && !(ok = __all_sync(0xffffffffu, mbar_wait_brief(&sh.item_empty[place], (item / kItems - 1) & 1)))) break;
                if (leader) {
                    sh.item[place] = x;
                    mbar_arrive(&sh.item_full[place]);
                }
                __syncwarp();
                if (!some) break;
                if (a.stall == 1) {  // a test hook: no loads
                    ok = false;
                    break;
                }
                auto load_queries = [&](int t) {  // once the products with the tile's last ones are done
                    if ((t ? x.n1 : x.n0) == 0 || (t == 1 && x.step == 2)) return;
                    uint32_t& before = t ? queries[1] : queries[0];
                    if (before > 0 && !(ok = __all_sync(0xffffffffu, mbar_wait_brief(&sh.q_empty[t], (before - 1) & 1)))) return;
                    ++before;
                    if (leader) {
                        mbar_arrive_expect_tx(&sh.q_full[t], L::kQ);
                        for (int b = 0; b < QB; ++b)
                            tma_load_3d(smem + L::kQAt + t * L::kQ + b * kBlock, &plan.q, &sh.q_full[t], 64 * b, x.q0 + x.row0 + t * kM,
                                        a.q.head_stride ? x.h : 0);
                    }
                    __syncwarp();
                };
                load_queries(0);
                const int early = max(0, x.n_tiles - 2);  // an answer takes less than two tiles
                if (x.n_tiles == 0) ask(), waiting = true;
                for (int i = 0; ok && i < x.n_tiles; ++i) {
                    if (i == early) ask(), waiting = true;
                    if (i == 1) load_queries(1);  // behind the first tile's first keys and values
                    if (!ok) break;
                    const int key = x.k0 + i * kKeys;
                    for (int b = 0; ok && b < QB; ++b) {
                        const uint32_t slot = keys % NK;
                        if (keys >= NK && !(ok = __all_sync(0xffffffffu, mbar_wait_brief(&sh.k_empty[slot], (keys / NK - 1) & 1)))) break;
                        ++keys;
                        if (leader) {
                            uint8_t* dst = smem + slot * kBlock;
                            mbar_arrive_expect_tx(&sh.k_full[slot], kBlock);
                            if (b < QB - 1) tma_load_3d(dst, &plan.k, &sh.k_full[slot], 64 * b, key, a.k.head_stride ? x.h : 0);
                            else tma_load_2d(dst, &plan.r, &sh.k_full[slot], 0, key);
                        }
                        __syncwarp();
                    }
                    const uint32_t slot = values % NV;
                    if (ok && values >= NV) ok = __all_sync(0xffffffffu, mbar_wait_brief(&sh.v_empty[slot], (values / NV - 1) & 1));
                    if (!ok) break;
                    ++values;
                    if (leader) {
                        uint8_t* dst = smem + L::kVAt + slot * L::kVTile;
                        mbar_arrive_expect_tx(&sh.v_full[slot], L::kVTile);
                        for (uint32_t b = 0; b < L::kVTile / kBlock; ++b)
                            tma_load_3d(dst + b * kBlock, &plan.v, &sh.v_full[slot], 64 * b, key, a.v.head_stride ? x.h : 0);
                    }
                    __syncwarp();
                }
                if (ok && x.n_tiles == 1) load_queries(1);
                if (ok) {
                    at = answer();
                    waiting = !ok;
                }
            }
            if (!ok) {  // nothing is in flight when the memory is given back, and no block starts to wait like this one
                if (lane == 0) record(a.error, 64);
                if (at >= 0) {
                    ok = true;
                    if (!waiting) ask();
                    while (ok && answer() >= 0) ask();
                }
                Drain drain;
                for (uint32_t f = keys > NK ? keys - NK : 0; f < keys; ++f) drain.wait(&sh.k_full[f % NK], (f / NK) & 1);
                for (uint32_t f = values > NV ? values - NV : 0; f < values; ++f) drain.wait(&sh.v_full[f % NV], (f / NV) & 1);
                for (int t = 0; t < kTiles; ++t)
                    if (queries[t] > 0) drain.wait(&sh.q_full[t], (queries[t] - 1) & 1);
            }
        } else if (warp == 9) {
            // ---- products
            const bool leader = elect_one();
            constexpr uint32_t id_s = idesc_bf16_f32(kM, kKeys), id_o = idesc_bf16_f32(kM, V, false, true);
            const uint64_t dq = desc_kmajor_sw128(smem_u32(smem + L::kQAt)), dk = desc_kmajor_sw128(smem_u32(smem)),
                           dv = desc_mnmajor_sw128(smem_u32(smem + L::kVAt), kBlock);
            auto wait = [&](uint64_t* bar, uint32_t parity) { return __all_sync(0xffffffffu, mbar_wait_brief(bar, parity)) != 0; };
            bool ok = a.stall != 2;  // a test hook: no products
            uint32_t keys = 0, values = 0, queries[kTiles] = {0, 0}, steps[kTiles] = {0, 0};  // of the items before this one
            for (uint32_t item = 0; ok; ++item) {
                Item x;
                if (!(ok = take(item, x)) || x.h < 0) break;
                auto walk = [&](auto by_halves) {
                    constexpr bool kHalves = decltype(by_halves)::value;
                    auto tile = [](int t, int i) { return kHalves ? 2 * i + t : i; };
                    // scores of tile t and its i-th key tile; the last tile that uses a block gives it back
                    auto scores = [&](int t, int i) {
                        const bool give = kHalves || t == 1 || i >= x.n1;
                        const int kt = tile(t, i), tq = kHalves ? 0 : t;
                        for (int b = 0; b < QB; ++b) {
                            const uint32_t fill = keys + kt * QB + b, slot = fill % NK;
                            if (!(ok = wait(&sh.k_full[slot], (fill / NK) & 1))) return;
                            tc_fence_after_sync();
                            if (leader) {
#pragma unroll
                                for (int k = 0; k < 4; ++k)
                                    mma_bf16(tmem + t * kKeys, dq + ((tq * L::kQ + b * kBlock) >> 4) + 2 * k, dk + (slot * kBlock >> 4) + 2 * k,
                                             id_s, (b > 0 || k > 0) ? 1u : 0u);
                                if (give) mma_commit(&sh.k_empty[slot]);
                            }
                            __syncwarp();
                        }
                        if (leader) {
                            mma_commit(&sh.s_full[t]);
                            if (kHalves ? kt == x.n_tiles - 1 : i == (t ? x.n1 : x.n0) - 1) mma_commit(&sh.q_empty[tq]);
                        }
                        __syncwarp();
                    };
#pragma unroll
                    for (int t = 0; t < kTiles; ++t)
                        if (ok && (t ? x.n1 : x.n0) > 0) {
                            if (!(ok = wait(&sh.q_full[kHalves ? 0 : t], queries[kHalves ? 0 : t] & 1))) break;
                            scores(t, 0);
                        }
                    for (int i = 0; ok && i < x.n_tiles; ++i) {
#pragma unroll
                        for (int t = 0; t < kTiles; ++t) {
                            if (!ok || i >= (t ? x.n1 : x.n0)) continue;
                            const uint32_t fill = values + tile(t, i), slot = fill % NV;
                            if (!(ok = wait(&sh.v_full[slot], (fill / NV) & 1) && wait(&sh.p_full[t], (steps[t] + i) & 1))) break;
                            tc_fence_after_sync();
                            if (leader) {
#pragma unroll
                                for (int k = 0; k < kKeys / 16; ++k)  // 16 keys of weights are 8 columns
                                    mma_bf16_ta(tmem + L::kOut + t * V, tmem + t * kKeys + 8 * k, dv + ((slot * L::kVTile + k * 2048) >> 4), id_o,
                                                (i > 0 || k > 0) ? 1u : 0u);
                                if (kHalves || t == 1 || i >= x.n1) mma_commit(&sh.v_empty[slot]);
                                mma_commit(&sh.pv_done[t]);
                            }
                            __syncwarp();
                            if (i + 1 < (t ? x.n1 : x.n0)) scores(t, i + 1);
                        }
                    }
                };
                if (x.step == 2) walk(std::true_type{});
                else walk(std::false_type{});
                keys += x.n_tiles * QB;
                values += x.n_tiles;
#pragma unroll
                for (int t = 0; t < kTiles; ++t) {
                    steps[t] += (t ? x.n1 : x.n0);
                    queries[t] += (t ? x.n1 : x.n0) > 0 && (t == 0 || x.step == 1);
                }
            }
            if (!ok && lane == 0) record(a.error, 65);
            if (leader) mma_commit(&sh.drained);
            mbar_wait_brief(&sh.drained, 0);
        }
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

// Key tiles that the tile of queries from row0 on walks (0 where it has no queries).
int key_tiles(int q, int kv, int row0, int rows) {
    if (row0 >= q) return 0;
    return std::max(0, kv - q + std::min(row0 + rows, q) - 1 + kKeys) / kKeys;
}

template <int NOPE, int V>
cudaError_t expanded_t(const ExpandedArgs& a, cudaStream_t st) {
    using L = ECfg<NOPE, V>;
    static std::atomic<unsigned long long> ready{0};
    cudaError_t e = allow_smem(expanded_kernel<NOPE, V>, L::kSmem, ready);
    if (e != cudaSuccess) return e;
    Plan plan{};
    if (a.n_kv > 0 &&
        !(map_rows(&plan.q, a.q, a.n_q, a.n_heads, NOPE + kRopeDim) && map_rows(&plan.k, a.k, a.n_kv, a.n_heads, NOPE) &&
          make_tma_map_bf16_2d(&plan.r, a.k_rope.data, a.n_kv, kRopeDim, a.k_rope.token_stride, kKeys, 64) &&
          map_rows(&plan.v, a.v, a.n_kv, a.n_heads, V)))
        return cudaErrorInvalidValue;
    constexpr int rows = kTiles * kM;
    int cost[kPairs], order[kPairs], most[kPairs];  // most: of the sequence's
    uint32_t pair[kPairs];
    int n = 0;
    auto launch = [&] {  // the pairs so far
        for (int i = 0; i < n; ++i) order[i] = i;
        for (int i = 0, j; i < n; i = j) {
            int top = 0;
            for (j = i; j < n && pair[j] >> 16 == pair[i] >> 16; ++j) top = std::max(top, cost[j]);
            for (int k = i; k < j; ++k) most[k] = top;
        }
        // The sequence with the longest item first, so that short items end the launch; a sequence's side by side, so
        // that they read its keys from L2 (16 ragged prompts: 142 us, by items alone 145).
        std::sort(order, order + n, [&](int x, int y) {
            if (most[x] != most[y]) return most[x] > most[y];
            if (pair[x] >> 16 != pair[y] >> 16 || cost[x] == cost[y]) return x < y;
            return cost[x] > cost[y];
        });
        for (int i = 0; i < n; ++i) plan.pair[i] = pair[order[i]];
        const unsigned grid = static_cast<unsigned>(n) * a.n_heads;
        n = 0;
        return timed_launch("expanded_attention", st, [&] {
            expanded_kernel<NOPE, V><<<grid, kThreads, L::kSmem, st>>>(a, plan);
            return cudaGetLastError();
        });
    };
    for (int i = 0; i < a.n_seq; ++i) {
        const int q = a.cu_q_host[i + 1] - a.cu_q_host[i], kv = a.cu_kv_host[i + 1] - a.cu_kv_host[i];
        for (int b = 0; b * rows < q; ++b) {  // (below 2^24 queries: checked by the caller)
            const int n0 = key_tiles(q, kv, b * rows, kM), n1 = key_tiles(q, kv, b * rows + kM, kM);
            // two steps side by side: 10; one alone: 7; those of one query tile, by halves: 5
            cost[n] = n1 == 0 ? 5 * n0 : 3 * std::min(n0, n1) + 7 * std::max(n0, n1);
            pair[n++] = static_cast<uint32_t>(i) << 16 | b;
            if (n == kPairs && (e = launch()) != cudaSuccess) return e;
        }
    }
    return n > 0 ? launch() : cudaSuccess;
}

}  // namespace

cudaError_t launch_expanded_attention(const ExpandedArgs& a, int nope_dim, int v_dim, cudaStream_t st) {
    if (nope_dim == 128) return v_dim == 128 ? expanded_t<128, 128>(a, st) : expanded_t<128, 64>(a, st);
    return v_dim == 128 ? expanded_t<64, 128>(a, st) : expanded_t<64, 64>(a, st);
}

}  // namespace gdn
