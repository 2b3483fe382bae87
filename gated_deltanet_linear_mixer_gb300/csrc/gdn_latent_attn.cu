// Attention over the latent cache, absorbed form, on the 5th-generation tensor
// cores.
//
// The mathematics, in powers of two (y = scale log2 e q . row):
//   w_rj = 2^(y_rj - m_r),   o_r = sum_j w_rj row_j[:C] / sum_j w_rj
// over the rows r = (token, head) of a sequence, which all read the same keys: one
// pass over the cached rows serves up to 64 of them.  The reference m_r lags
// behind the row's maximum by at most 2^kLazy, so that the output is rescaled
// only where the maximum rises by more than that.  Weights are rounded to bf16
// (the values' type, as the tensor core asks), and the sum takes the rounded ones.
//
// A thread block walks tiles of 64 keys.  S = Q K^T has the rows as its M = 64 and
// the keys as its N, so that a row's scores lie in four lanes of one warp.
// O^T = V^T P^T has the latent channels as its M (C / 128 products of 128) and the
// rows as its N: a tile of cached rows is the K-major operand of the first product
// and the MN-major one of the second as it lies in shared memory, and the output
// of 64 rows takes half of the tensor memory, where rows as M would take all of it.
//
// Work.  (sequence, group of row tiles, key tile) in that order is one axis, cut
// into equal spans, one a thread block.  So ragged lengths fill every SM alike,
// whatever they are; lengths are only known on the device, where every thread
// block finds its span by a scan over the sequences.  What a span holds of a
// sequence that it does not hold whole is a partial result (at most two a span);
// a second launch joins them.  Where most sequences have an even number of row tiles a
// group is two of them, of two neighbouring thread blocks that walk the same span, each
// with loads of its own: the later one's rows come from L2 (64 x 4 drafts as below: 106
// us; 110 where a cluster shared its loads).  Else it is one (two_tiles).
//
// Roles: 4 softmax warps (also: rescaling, epilogue), two for the rows' TMA loads
// (with the page look-ups), one loading queries and issuing S, one issuing O^T.
// Cached rows are in a ring of 16 KB slots (64 keys x 128 channels) and one of 8 KB
// slots (position keys).  Every wait is bounded (2 s); a wait that gives up records
// a code (50..57) in the cache operators' device error word, and its role waits for
// nothing more but, once for all of them, what it has in flight: a thread block ends
// within a few such waits.
//
// What bounds it (cycles at 1.95 GHz, the SM clock by the kernel's own counters).  Up to 32
// rows a sequence the rows' bytes: a tile's 72 KB are 3200 cycles of an SM's share of
// DRAM (1.65 us; 1.67 are reached), its products 2160 (16 rows) or 2290 (32).
// 256 single tokens of 32 heads after 127..8191 keys take 222 to 227 us, 87% of the
// measured copy rate, 16 heads 205 to 210 us (90%).  With 64 rows the products: 36 of S at 37
// cycles (64 x 64 x 16) and 16 of O^T at 76 (128 x 64 x 16 with the first operand
// MN-major; 53 were it K-major) make 2540 cycles a tile, of which the ring's two tiles
// let it reach 2870 (1.47 us): 64 x 4 drafts of 32 heads after 500..6000 keys take 106 us,
// of which 48 tiles are 71, the partial results of 152 thread blocks and their join 20,
// the call's start, its queries and the outputs of whole sequences 13.  Tiles of
// 32 keys, four in the ring, were slower (145 us, then 119), and so was fetching
// tiles into L2 ahead of their loads (256 x 1: 229 us without, 246 three tiles
// ahead).  One token after 1000 keys takes 13 us, all of it latency: the plan 2 us,
// the look-up 1.5, a load 1, products and softmax 2.5, the partial result 1, the join 4.
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

constexpr int kSms = 152;
constexpr int kKeys = 64;        // of a tile
constexpr int kRopes = 2;        // slots of position keys
constexpr int kThreads = 256;
constexpr float kLazy = 8.0f;
constexpr int kPieces = 16;      // pieces of a span that are laid out at a time
constexpr int kMasks = 8;
constexpr int kMaxSlots = 12;
constexpr uint32_t kSmemMax = 232448, kSharedBytes = 2944;

template <int C, int NR> struct LCfg {
    static constexpr int W = C + kRopeDim, kBlocks = W / 64, kPairs = C / 128;
    static constexpr uint32_t kRope = kKeys * 128, kSlot = 2 * kRope;            // 64 channels of a tile, and 128
    static constexpr uint32_t kQBlock = NR * 128;                                // 64 channels of the row tile
    static constexpr uint32_t kQ = kBlocks * kQBlock + (64 - NR) * 128;          // M = 64 reads past the last block
    static constexpr uint32_t kP = NR * 128;
    static constexpr int kFit = (kSmemMax - kSharedBytes - kQ - kP - kRopes * kRope) / kSlot;
    static constexpr int kSlots = kFit < kMaxSlots ? kFit : kMaxSlots;
    static constexpr uint32_t kRopeAt = kSlots * kSlot, kQAt = kRopeAt + kRopes * kRope, kPAt = kQAt + kQ, kSharedAt = kPAt + kP;
    static constexpr uint32_t kSmem = kSharedAt + kSharedBytes;
    static constexpr int kActive = NR / 16;                                      // softmax warps with rows
    static constexpr uint32_t kOut = 128;                                        // tensor memory: S twice, then O^T
    static_assert(kSlots >= 2 * kPairs, "two tiles fit");
    static_assert(kOut + kPairs * NR <= 512, "the output fits");
    static constexpr size_t kPart = static_cast<size_t>(NR) * (C + 2);           // floats of a partial result
};

struct Piece {
    int q0;             // the sequence's first token
    int seq;
    int row0, n_rows;   // rows (token, head) of the sequence
    int start, n_keys;  // position of the sequence's first query; keys that some row of the group sees
    int a, b;           // key tiles
    int slot;           // partial result, or -1: the sequence's keys are all here
};

struct Join {  // a sequence's row tile whose pieces start in this span and end in another
    int n_pieces;  // 0: none
    int out_row, n_rows, slot;
};

struct Shared {
    uint64_t pair_full[kMaxSlots], pair_empty[kMaxSlots], rope_full[kRopes], rope_empty[kRopes];
    uint64_t q_full, q_empty, s_full[2], s_empty[2], p_full, pv_done, m_full[kMasks], drained[2];
    long long scan[kThreads / 32];
    int n_round, more;
    int mask[kMasks];
    float factor[64], stat[64];
    Piece piece[kPieces];
    int dead;      // a loading or issuing warp gave up
    int dead_was;  // whether one had when the round began: written between the thread block's barriers, so that all warps read the same
    uint32_t tmem_slot;
};
static_assert(sizeof(Shared) <= kSharedBytes, "part of kSmem");



// How long rows stay in L2: those of sequences that a single group of row tiles
// reads leave before the partial results, which are read again (256 single tokens of
// 32 heads: 224 us, 222 us so; 131,000 keys: 39.3, 37.9), those that other groups
// read after this one do not (256 tokens of 32 heads after 1744: 119 us if they did, 108 us).
__device__ __forceinline__ uint64_t l2_policy(bool once) {
    uint64_t p;
    if (once) asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
    else asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(p));
    return p;
}
__device__ __forceinline__ void load_rows(void* dst, const CUtensorMap* map, uint64_t* bar, int x, int y, uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%2, %3}], [%4], %5;" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(smem_u32(bar)), "l"(policy)
        : "memory");
}
__device__ __forceinline__ void load_halves(void* dst, const CUtensorMap* map, uint64_t* bar, int y, int z, uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%2, %3, %4}], [%5], %6;" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(y), "r"(z), "r"(smem_u32(bar)), "l"(policy)
        : "memory");
}

// 16 lanes x 64 columns of 32-bit: v[4 i + 2 h + e] is row lane / 4 + 8 h, column
// 8 i + 2 (lane % 4) + e.
__device__ __forceinline__ void tmem_ld_rows16(uint32_t taddr, float* v) {
    uint32_t r[32];
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x8.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr)
        : "memory");
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}
// 32 lanes x 16 columns.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float* v) {
    uint32_t r[16];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const float* v) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::"f"(v[0]),
        "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]), "f"(v[8]), "f"(v[9]), "f"(v[10]),
        "f"(v[11]), "f"(v[12]), "f"(v[13]), "f"(v[14]), "f"(v[15]), "r"(taddr)
        : "memory");
}

// What a sequence needs: groups of G row tiles, and key tiles of each (at least one,
// so that rows without keys are somebody's).
struct Need {
    int q0, qn, len, groups, tiles;
};
// x / y, in 32 bits where they fit: a 64-bit division takes several hundred cycles.
__device__ __forceinline__ long long quotient(long long x, long long y) {
    if (((x | y) >> 32) == 0) return static_cast<uint32_t>(x) / static_cast<uint32_t>(y);
    return x / y;
}
// Key tiles of n keys, up to 2^31 - 1.
__device__ __forceinline__ int tiles_of(int n) { return static_cast<int>((static_cast<uint32_t>(n) + kKeys - 1) / kKeys); }
template <int ROWS>
__device__ __forceinline__ Need need_of(const LatentAttnArgs& a, int seq) {
    Need n;
    n.q0 = a.b.cu[seq];
    n.qn = a.b.cu[seq + 1] - n.q0;
    n.len = a.b.kv_lens[seq];
    const long long cap = a.c.n_pages > 0 ? static_cast<long long>(a.b.pages_per_seq) << a.page_shift : 0;
    const int len = static_cast<int>(min(static_cast<long long>(max(n.len, 0)), cap));
    n.groups = (n.qn * a.n_heads + ROWS - 1) / ROWS;
    n.tiles = max(1, tiles_of(len));
    return n;
}

struct Maps {
    CUtensorMap rows;   // boxes of a page's (at most a tile's) rows x 64 channels
    CUtensorMap pairs;  // of a tile's rows x 128 channels, in two halves
    CUtensorMap q;      // of a row tile x 64 channels
};

// G: row tiles of a group, of as many thread blocks.
template <int C, int NR, int G>
__global__ void __launch_bounds__(kThreads, 1)
latent_attention_kernel(const LatentAttnArgs a, const __grid_constant__ Maps maps, const int dense_q, float* parts, Join* joins) {
    using L = LCfg<C, NR>;
    constexpr int NP = L::kPairs, NS = L::kSlots;
    constexpr int kScores = kKeys / 2;  // of a lane: two rows of a quarter of the keys
    extern __shared__ __align__(1024) uint8_t smem[];
    Shared& sh = *reinterpret_cast<Shared*>(smem + L::kSharedAt);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g_own = static_cast<int>(blockIdx.x) % G, span = static_cast<int>(blockIdx.x) / G;
    const int n_spans = static_cast<int>(gridDim.x) / G;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (warp == 7) {
        if (a.c.n_pages > 0) {
            tma_prefetch_desc(&maps.rows);
            tma_prefetch_desc(&maps.pairs);
        }
        if (dense_q) tma_prefetch_desc(&maps.q);
    }

    // ---- this thread block's span of the (sequence, group, key tile) axis
    const int each = (a.b.n_seq + kThreads - 1) / kThreads;
    const int s0 = min(tid * each, a.b.n_seq), s1 = min(s0 + each, a.b.n_seq);
    long long units = 0;
    Need first{};  // of s0: all that this thread has where there are no more sequences than threads
    for (int s = s0; s < s1; ++s) {
        const Need n = need_of<NR * G>(a, s);
        if (s == s0) first = n;
        units += static_cast<long long>(n.groups) * n.tiles;
    }
    long long u_in = units;  // inclusive
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const long long u = __shfl_up_sync(0xffffffffu, u_in, off);
        if (lane >= off) u_in += u;
    }
    if (lane == 31) sh.scan[warp] = u_in;
    if (tid == 32 * 6) {  // beside the warp that most of the sequences are in
        for (int i = 0; i < NS; ++i) {
            mbar_init(&sh.pair_full[i], 1);
            mbar_init(&sh.pair_empty[i], 1);
        }
        for (int i = 0; i < kRopes; ++i) {
            mbar_init(&sh.rope_full[i], 1);
            mbar_init(&sh.rope_empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sh.s_full[i], 1);
            mbar_init(&sh.s_empty[i], L::kActive);
        }
        mbar_init(&sh.q_full, 1);
        mbar_init(&sh.q_empty, 1);
        mbar_init(&sh.p_full, 4);
        mbar_init(&sh.pv_done, 1);
        for (int i = 0; i < kMasks; ++i) mbar_init(&sh.m_full[i], 1);
        for (int i = 0; i < 2; ++i) mbar_init(&sh.drained[i], 1);
        sh.dead = sh.dead_was = 0;
        fence_barrier_init();
    }
    __syncthreads();
    long long u_base = u_in - units, total = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
        if (w < warp) u_base += sh.scan[w];
        total += sh.scan[w];
    }
    const long long per = quotient(total + n_spans - 1, n_spans);  // (0 without any)
    const long long u0 = span * per, u1 = min(u0 + per, total);
    if (u0 >= u1 || (smem_u32(smem) & 1023u)) {
        if (tid == 0) {
            joins[blockIdx.x].n_pieces = 0;
            if (u0 < u1) record(a.error, 58);
        }
        return;
    }
    if (warp == 5) tmem_alloc(&sh.tmem_slot, 512);
    // The thread whose sequences hold the span's first tile lays out the pieces, kPieces at a time.
    long long u_at = u_base;  // where sequence s_at begins
    int s_at = s0, k_at = 0;
    Need n_at = first;
    const bool walker = u_base <= u0 && u0 < u_base + units;
    if (walker) {
        for (long long all = static_cast<long long>(n_at.groups) * n_at.tiles; u_at + all <= u0;
             all = static_cast<long long>(n_at.groups) * n_at.tiles) {
            u_at += all;
            n_at = need_of<NR * G>(a, ++s_at);
        }
        k_at = static_cast<int>(quotient(u0 - u_at, n_at.tiles));
    }
    auto lay_out = [&] {
        const long long cap = a.c.n_pages > 0 ? static_cast<long long>(a.b.pages_per_seq) << a.page_shift : 0;
        int i = 0;
        bool more = true;
        while (i < kPieces) {
            const long long all = static_cast<long long>(n_at.groups) * n_at.tiles;
            const long long head = u_at + static_cast<long long>(k_at) * n_at.tiles;  // the item's first tile
            if (k_at == n_at.groups) {  // on to the next sequence
                u_at += all;
                k_at = 0;
                if (u_at >= u1) {
                    more = false;
                    break;
                }
                n_at = need_of<NR * G>(a, ++s_at);
                continue;
            }
            if (head >= u1) {
                more = false;
                break;
            }
            if (n_at.len > cap) record(a.error, kKvErrTable);
            const int len = static_cast<int>(min(static_cast<long long>(max(n_at.len, 0)), cap));
            const int all_rows = n_at.qn * a.n_heads, row0 = (k_at * G + g_own) * NR, rows = min(NR, all_rows - row0);
            const int last_row = min((k_at + 1) * G * NR, all_rows) - 1;  // of the group
            Piece p;
            p.q0 = n_at.q0;
            p.seq = s_at;
            p.row0 = row0;
            p.n_rows = max(rows, 0);
            p.start = max(n_at.len, 0) - n_at.qn;  // queries before 0 see nothing
            p.n_keys = max(0, min(p.start + last_row / a.n_heads + 1, len));
            p.a = static_cast<int>(max(u0 - head, 0ll));
            const int b = static_cast<int>(min(u1 - head, static_cast<long long>(n_at.tiles)));
            p.b = max(p.a, min(b, tiles_of(p.n_keys)));
            p.slot = p.a == 0 && b == n_at.tiles ? -1 : 2 * span + (head + p.a > u0 ? 1 : 0);
            sh.piece[i++] = p;
            if (head + n_at.tiles >= u1) {  // the span's last one
                Join j{0, 0, 0, 0};
                const long long rest = head + n_at.tiles - u1;  // tiles in the spans that follow
                if (head >= u0 && rest > 0 && rows > 0) {
                    j.n_pieces = 1 + static_cast<int>(quotient(rest + per - 1, per));
                    j.out_row = n_at.q0 * a.n_heads + row0;
                    j.n_rows = rows;
                    j.slot = p.slot;
                }
                joins[blockIdx.x] = j;
                more = false;
                break;
            }
            ++k_at;
        }
        sh.n_round = i;
        sh.more = more;
    };
    if (walker) {
        // the loading warps' first look-up, on its way meanwhile
        const long long key = (u0 - u_at - static_cast<long long>(k_at) * n_at.tiles) * kKeys;
        if (key >> a.page_shift < a.b.pages_per_seq)
            asm volatile("prefetch.global.L2 [%0];" ::"l"(a.b.table + static_cast<size_t>(s_at) * a.b.pages_per_seq + (key >> a.page_shift)));
        lay_out();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = sh.tmem_slot;

    // counts that the roles carry from round to round
    uint32_t g = 0;   // key tiles
    uint32_t qc = 0;  // pieces with tiles whose queries came
    uint32_t asked = 0;  // whose queries were asked for
    bool ok = true;
    uint32_t ropes = 0, pairs = 0;  // loads started

    for (;;) {
        const int n_round = sh.n_round;
        const bool dead = sh.dead_was != 0;
        const bool more = sh.more;
        if (dead) {
            // a wait gave up in an earlier round: nothing more is started.  (The softmax warps meet at a barrier of
            // theirs, which has no time limit: either all of them run a round or none does.)
        } else if (warp < 4) {
            // ---- softmax
            const bool active = warp < L::kActive;
            const float scale2 = a.scale * kLog2e;
            const uint32_t t_lane = (32u * warp) << 16;
            for (int i = 0; i < n_round; ++i) {
                const Piece p = sh.piece[i];
                const int rA = 16 * warp + (lane >> 2), rB = rA + 8;
                int limA = 0, limB = 0;  // keys that this lane's rows see
                if (rA < p.n_rows) limA = min(p.start + (p.row0 + rA) / a.n_heads + 1, p.n_keys);
                if (rB < p.n_rows) limB = min(p.start + (p.row0 + rB) / a.n_heads + 1, p.n_keys);
                const int lim = min(limA, limB);
                float mA = -INFINITY, mB = -INFINITY, lA = 0.0f, lB = 0.0f;
                for (int t = p.a; t < p.b; ++t, ++g) {
                    const int key0 = t * kKeys, valid = p.n_keys - key0;  // keys of the tile that exist
                    const uint32_t sb = g & 1;
                    float s[kScores];
                    bool lift = false;
                    float topA = -INFINITY, topB = -INFINITY;
                    // (Warps without rows do not: they count in no barrier that S waits for, so that they might look
                    // two tiles late.  What they write, rows behind the last key, they write after the lift's barrier.)
                    if (active && ok &&
                        !(ok = __all_sync(0xffffffffu, mbar_wait_brief(&sh.s_full[sb], (g >> 1) & 1) &&
                                                           mbar_wait_brief(&sh.m_full[g % kMasks], (g / kMasks) & 1))) &&
                        lane == 0)
                        record(a.error, 50);
                    if (active) {
                        tc_fence_after_sync();
                        tmem_ld_rows16(tmem + t_lane + kKeys * sb, s);
                        const int mask = sh.mask[g % kMasks];
                        tc_fence_before_sync();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&sh.s_empty[sb]);
#pragma unroll
                        for (int j = 0; j < kScores; ++j) s[j] *= scale2;
                        if (lim - key0 < kKeys || mask != (1 << (kKeys / 16)) - 1) {
                            const int c = key0 + 2 * (lane & 3);
#pragma unroll
                            for (int j = 0; j < kScores; ++j) {
                                const int key = c + 8 * (j >> 2) + (j & 1);
                                if (key >= (j & 2 ? limB : limA) || !(mask >> (j >> 3) & 1)) s[j] = -INFINITY;
                            }
                        }
#pragma unroll
                        for (int j = 0; j < kScores; j += 4) {
                            topA = fmaxf(topA, fmaxf(s[j], s[j + 1]));
                            topB = fmaxf(topB, fmaxf(s[j + 2], s[j + 3]));
                        }
#pragma unroll
                        for (int off = 1; off < 4; off <<= 1) {
                            topA = fmaxf(topA, __shfl_xor_sync(0xffffffffu, topA, off));
                            topB = fmaxf(topB, __shfl_xor_sync(0xffffffffu, topB, off));
                        }
                        lift = topA > mA + kLazy || topB > mB + kLazy;
                    }
                    lift = group_or(1, 128, lift);
                    if (lift) {
                        if (active) {
                            const float nA = fmaxf(mA, topA), nB = fmaxf(mB, topB);
                            const float fA = mA == -INFINITY ? 0.0f : exp2_ftz(mA - nA), fB = mB == -INFINITY ? 0.0f : exp2_ftz(mB - nB);
                            lA *= fA;
                            lB *= fB;
                            mA = nA;
                            mB = nB;
                            if ((lane & 3) == 0) {
                                sh.factor[rA] = fA;
                                sh.factor[rB] = fB;
                            }
                        }
                        if (t > p.a) {  // the output so far
                            group_sync(1, 128);
                            if (ok && !(ok = __all_sync(0xffffffffu, mbar_wait_brief(&sh.pv_done, (g - 1) & 1))) && lane == 0)
                                record(a.error, 51);
                            tc_fence_after_sync();
#pragma unroll 1
                            for (int c = 0; c < NP * NR; c += 16) {
                                float v[16];
                                tmem_ld16(tmem + t_lane + L::kOut + c, v);
#pragma unroll
                                for (int e = 0; e < 16; ++e) v[e] *= sh.factor[c % NR + e];
                                tmem_st16(tmem + t_lane + L::kOut + c, v);
                            }
                            tmem_wait_st();
                            tc_fence_before_sync();
                        }
                    }
                    if (active) {
                        const float refA = mA == -INFINITY ? 0.0f : mA, refB = mB == -INFINITY ? 0.0f : mB;
                        uint32_t w[kScores / 2];
#pragma unroll
                        for (int j = 0; j < kScores; j += 2) {
                            const float ref = j & 2 ? refB : refA;
                            w[j / 2] = pack_bf16x2(exp2_ftz(s[j] - ref), exp2_ftz(s[j + 1] - ref));
                            const float sum = __uint_as_float(w[j / 2] << 16) + __uint_as_float(w[j / 2] & 0xFFFF0000u);
                            if (j & 2) lB += sum;
                            else lA += sum;
                        }
                        // the weights before these were used
                        if (g > 0 && ok && !(ok = __all_sync(0xffffffffu, mbar_wait_brief(&sh.pv_done, (g - 1) & 1))) && lane == 0)
                            record(a.error, 52);
                        uint8_t* tile = smem + L::kPAt;
#pragma unroll
                        for (int c = 0; c < kKeys / 8; ++c) {
                            *reinterpret_cast<uint32_t*>(tile + sw128_offset(rA, c) + 4 * (lane & 3)) = w[2 * c];
                            *reinterpret_cast<uint32_t*>(tile + sw128_offset(rB, c) + 4 * (lane & 3)) = w[2 * c + 1];
                        }
                    }
                    if (valid < kKeys) {  // rows behind the last key may be anything: weights of 0 do not undo a NaN
                        for (int q = 0; q < NP; ++q) {
                            const uint32_t n = g * NP + q, slot = n % NS;
                            if (ok && !(ok = __all_sync(0xffffffffu, mbar_wait_brief(&sh.pair_full[slot], (n / NS) & 1))) && lane == 0)
                                record(a.error, 53);
                            uint4* row = reinterpret_cast<uint4*>(smem + slot * L::kSlot);
                            for (int x = tid; x < 2 * (kKeys - valid) * 8; x += 128) {
                                const int half = x & 1, r = valid + x / 16, c = x / 2 % 8;
                                row[half * (L::kRope / 16) + r * 8 + c] = make_uint4(0, 0, 0, 0);
                            }
                        }
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sh.p_full);
                }
                // ---- epilogue
                const bool any = p.b > p.a;
                if (any && ok && !(ok = __all_sync(0xffffffffu, mbar_wait_brief(&sh.pv_done, (g - 1) & 1))) && lane == 0)
                    record(a.error, 54);
                if (active) {
#pragma unroll
                    for (int off = 1; off < 4; off <<= 1) {
                        lA += __shfl_xor_sync(0xffffffffu, lA, off);
                        lB += __shfl_xor_sync(0xffffffffu, lB, off);
                    }
                    if ((lane & 3) == 0) {
                        if (p.slot < 0) {  // a sum that is no number stays one
                            sh.stat[rA] = lA == 0.0f ? 0.0f : 1.0f / lA;
                            sh.stat[rB] = lB == 0.0f ? 0.0f : 1.0f / lB;
                        } else {
                            float* st = parts + (static_cast<size_t>(p.slot) * G + g_own) * L::kPart + NR * C;
                            st[rA] = mA;
                            st[rB] = mB;
                            st[NR + rA] = lA;
                            st[NR + rB] = lB;
                        }
                    }
                }
                group_sync(1, 128);
                tc_fence_after_sync();
                constexpr int kStep = NR < 32 ? 16 : 32;
                auto load_out = [&](int c, float* v) {
                    if (kStep == 32) tmem_ld32(tmem + t_lane + L::kOut + c, v);
                    else tmem_ld16(tmem + t_lane + L::kOut + c, v);
                };
                if (p.slot < 0) {
                    bf16* out = static_cast<bf16*>(a.out) + (static_cast<size_t>(p.q0) * a.n_heads + p.row0) * C + 32 * warp + lane;
#pragma unroll 1
                    for (int c = 0; c < NP * NR; c += kStep) {
                        float v[kStep];
                        if (any) load_out(c, v);
                        bf16* at = out + static_cast<size_t>(c % NR) * C + c / NR * 128;
#pragma unroll
                        for (int e = 0; e < kStep; ++e)
                            if (c % NR + e < p.n_rows) at[e * C] = __float2bfloat16_rn(any ? v[e] * sh.stat[c % NR + e] : 0.0f);
                    }
                } else if (any) {
                    float* out = parts + (static_cast<size_t>(p.slot) * G + g_own) * L::kPart + 32 * warp + lane;
#pragma unroll 1
                    for (int c = 0; c < NP * NR; c += kStep) {
                        float v[kStep];
                        load_out(c, v);
                        float* at = out + static_cast<size_t>(c % NR) * C + c / NR * 128;
#pragma unroll
                        for (int e = 0; e < kStep; ++e)
                            if (c % NR + e < p.n_rows) at[e * C] = v[e];
                    }
                }
                tc_fence_before_sync();
                group_sync(1, 128);  // stat, and the output in tensor memory, may be written again
            }
        } else if (warp == 4 || warp == 7) {
            // ---- cached rows: page look-ups by the warp, loads by one lane.  A load takes about 55 cycles to
            // issue, and pages of 16 rows need 36 a tile: two warps share them, the first the position keys
            // and two slots, the second the others.
            const int page_size = 1 << a.page_shift, R = min(page_size, kKeys), per_tile = kKeys >> min(a.page_shift, 6);
            const bool leader = elect_one(), lead_warp = warp == 4;
            if (a.stall == 1) ok = false;  // a test hook: no loads
            const int nowhere = a.c.n_pages << a.page_shift;  // past the last row: the load gives zeros
            const uint64_t policy = l2_policy(static_cast<long long>(a.b.max_q) * a.n_heads <= NR * G);
            auto load = [&](uint8_t* dst, uint64_t* bar, int col, int row) { load_rows(dst, &maps.rows, bar, col, row, policy); };
            for (int i = 0; ok && i < n_round; ++i) {
                const Piece p = sh.piece[i];
                int row = 0;
                const int first_chunk = p.a * per_tile, n = (p.b - p.a) * per_tile;
                auto look_up = [&](int x) {  // where chunk x of the piece lies; negative: not mapped
                    if (x >= n) return nowhere;
                    const int key = (first_chunk + x) * R;
                    if (key >= p.n_keys) return nowhere;
                    const int page = a.b.table[static_cast<size_t>(p.seq) * a.b.pages_per_seq + (key >> a.page_shift)];
                    return page >= 0 && page < a.c.n_pages ? (page << a.page_shift) + (key & (page_size - 1)) : -1;
                };
                int ahead = n > 0 ? look_up(lane) : 0;
                for (int t = p.a; ok && t < p.b; ++t, ++g) {
                    const int x = (t - p.a) * per_tile;
                    if (x % 32 == 0) {
                        row = ahead;
                        ahead = look_up(x + 32 + lane);
                    }
                    int at[4];
                    int mask = (1 << (kKeys / 16)) - 1;
#pragma unroll
                    for (int c = 0; c < kKeys / 16; ++c) {
                        at[c] = __shfl_sync(0xffffffffu, row, (x + c) & 31);
                        if (c < per_tile && at[c] < 0) {
                            if (leader && lead_warp) record(a.error, kKvErrTable);
                            mask &= ~(((1 << (R / 16)) - 1) << (c * (R / 16)));
                            at[c] = nowhere;
                        }
                    }
                    if (lead_warp) {
                        if (leader) {
                            sh.mask[g % kMasks] = mask;
                            mbar_arrive(&sh.m_full[g % kMasks]);
                        }
                        const uint32_t rb = g % kRopes;
                        if (g >= kRopes) ok = __all_sync(0xffffffffu, mbar_wait_brief(&sh.rope_empty[rb], (g / kRopes - 1) & 1));
                        if (!ok) break;
                        ++ropes;
                        if (leader) {
                            mbar_arrive_expect_tx(&sh.rope_full[rb], L::kRope);
#pragma unroll
                            for (int c = 0; c < kKeys / 16; ++c)
                                if (c < per_tile) load(smem + L::kRopeAt + rb * L::kRope + c * R * 128, &sh.rope_full[rb], C, at[c]);
                        }
                        __syncwarp();
                    }
                    const int q0 = lead_warp ? 0 : 2;
#pragma unroll
                    for (int qq = 0; qq < 2; ++qq) {
                        const int q = q0 + qq;
                        if (q >= NP) break;
                        const uint32_t fill = g * NP + q, slot = fill % NS;
                        if (fill >= NS) ok = __all_sync(0xffffffffu, mbar_wait_brief(&sh.pair_empty[slot], (fill / NS - 1) & 1));
                        if (!ok) break;
                        pairs = fill + 1;
                        if (leader) {
                            uint8_t* dst = smem + slot * L::kSlot;
                            mbar_arrive_expect_tx(&sh.pair_full[slot], L::kSlot);
                            if (per_tile == 1) {
                                load_halves(dst, &maps.pairs, &sh.pair_full[slot], at[0], 2 * q, policy);
                            } else {
#pragma unroll
                                for (int c = 0; c < kKeys / 16; ++c)
                                    if (c < per_tile) {
                                        load(dst + c * R * 128, &sh.pair_full[slot], 128 * q, at[c]);
                                        load(dst + L::kRope + c * R * 128, &sh.pair_full[slot], 128 * q + 64, at[c]);
                                    }
                            }
                        }
                        __syncwarp();
                    }
                }
            }
            if (!ok && lane == 0) record(a.error, 55);
            __syncwarp();
            if (!ok) sh.dead = 1;
        } else if (warp == 5) {
            // ---- S = Q K^T
            const bool leader = elect_one();
            if (a.stall == 2) ok = false;  // a test hook: no scores
            constexpr uint32_t id = idesc_bf16_f32(64, kKeys);
            const uint64_t dq = desc_kmajor_sw128(smem_u32(smem + L::kQAt)), dr = desc_kmajor_sw128(smem_u32(smem + L::kRopeAt)),
                           dk = desc_kmajor_sw128(smem_u32(smem));
            auto load_queries = [&](const Piece& p) {
                uint8_t* tile = smem + L::kQAt;
                if (dense_q) {  // evenly spaced rows: those behind the sequence's last are another's, or zeros, and not used
                    if (leader) {
                        mbar_arrive_expect_tx(&sh.q_full, L::kBlocks * L::kQBlock);
                        for (int b = 0; b < L::kBlocks; ++b)
                            tma_load_2d(tile + b * L::kQBlock, &maps.q, &sh.q_full, 64 * b, p.q0 * a.n_heads + p.row0);
                    }
                    __syncwarp();
                    return;
                }
                constexpr int V = L::W / 8;
                const bf16* q = static_cast<const bf16*>(a.q.data);
                for (int r0 = 0; r0 < NR; r0 += 32) {
                    const int row = p.row0 + r0 + lane;  // whose place this lane works out
                    const bf16* at = q + (p.q0 + row / a.n_heads) * a.q.token_stride + row % a.n_heads * a.q.head_stride;
                    for (int r = r0; r < min(r0 + 32, NR); ++r) {
                        const bool take = r < p.n_rows;
                        const bf16* src = reinterpret_cast<const bf16*>(__shfl_sync(0xffffffffu, reinterpret_cast<uint64_t>(at), r - r0));
                        for (int c = lane; c < V; c += 32)
                            cp_async16(smem_u32(tile) + (c / 8) * L::kQBlock + sw128_offset(r, c % 8), take ? src + 8 * c : q, take);
                    }
                }
                asm volatile("cp.async.commit_group;\n\tcp.async.wait_group 0;" ::: "memory");
                fence_proxy_async_smem();
                __syncwarp();
                if (leader) mbar_arrive(&sh.q_full);
            };
            for (int i = 0; ok && i < n_round; ++i) {
                const int a0 = sh.piece[i].a, b0 = sh.piece[i].b;
                if (a0 >= b0) continue;
                // queries, once the products with the last ones are done
                if (qc > 0 && !(ok = __all_sync(0xffffffffu, mbar_wait_brief(&sh.q_empty, (qc - 1) & 1)))) break;
                load_queries(sh.piece[i]);
                ++asked;
                if (!(ok = __all_sync(0xffffffffu, mbar_wait_brief(&sh.q_full, qc & 1)))) break;
                ++qc;
                for (int t = a0; ok && t < b0; ++t, ++g) {
                    const uint32_t sb = g & 1;
                    if (g >= 2) ok = __all_sync(0xffffffffu, mbar_wait_brief(&sh.s_empty[sb], ((g >> 1) - 1) & 1));
                    const uint32_t rb = g % kRopes;
                    ok = ok && __all_sync(0xffffffffu, mbar_wait_brief(&sh.rope_full[rb], (g / kRopes) & 1));
                    if (!ok) break;
                    tc_fence_after_sync();
                    if (leader) {
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            mma_bf16(tmem + kKeys * sb, dq + ((C / 64) * L::kQBlock >> 4) + 2 * k, dr + (rb * L::kRope >> 4) + 2 * k, id,
                                     k > 0 ? 1u : 0u);
                        mma_commit(&sh.rope_empty[rb]);
                    }
                    for (int q = 0; q < NP; ++q) {
                        const uint32_t fill = g * NP + q, slot = fill % NS;
                        if (!(ok = __all_sync(0xffffffffu, mbar_wait_brief(&sh.pair_full[slot], (fill / NS) & 1)))) break;
                        tc_fence_after_sync();
                        if (leader) {
#pragma unroll
                            for (int h = 0; h < 2; ++h)
#pragma unroll
                                for (int k = 0; k < 4; ++k)
                                    mma_bf16(tmem + kKeys * sb, dq + ((2 * q + h) * L::kQBlock >> 4) + 2 * k,
                                             dk + ((slot * L::kSlot + h * L::kRope) >> 4) + 2 * k, id, 1u);
                        }
                        __syncwarp();
                    }
                    if (leader) mma_commit(&sh.s_full[sb]);
                    __syncwarp();
                }
                if (leader) mma_commit(&sh.q_empty);
                __syncwarp();
            }
            if (!ok && lane == 0) record(a.error, 56);
            if (!ok) sh.dead = 1;
        } else if (warp == 6) {
            // ---- O^T += V^T P^T
            const bool leader = elect_one();
            constexpr uint32_t id = idesc_bf16_f32(128, NR, true, false);
            const uint64_t dv = desc_mnmajor_sw128(smem_u32(smem), L::kRope), dp = desc_kmajor_sw128(smem_u32(smem + L::kPAt));
            for (int i = 0; ok && i < n_round; ++i) {
                const int a0 = sh.piece[i].a, b0 = sh.piece[i].b;
                for (int t = a0; ok && t < b0; ++t, ++g) {
                    if (!(ok = __all_sync(0xffffffffu, mbar_wait_brief(&sh.p_full, g & 1)))) break;
                    for (int q = 0; q < NP; ++q) {
                        const uint32_t fill = g * NP + q, slot = fill % NS;
                        if (!(ok = __all_sync(0xffffffffu, mbar_wait_brief(&sh.pair_full[slot], (fill / NS) & 1)))) break;
                        tc_fence_after_sync();
                        if (leader) {
#pragma unroll
                            for (int k = 0; k < kKeys / 16; ++k)
                                mma_bf16(tmem + L::kOut + q * NR, dv + ((slot * L::kSlot + k * 2048) >> 4), dp + 2 * k, id,
                                         (t > a0 || k > 0) ? 1u : 0u);
                            mma_commit(&sh.pair_empty[slot]);
                        }
                        __syncwarp();
                    }
                    if (!ok) break;
                    if (leader) mma_commit(&sh.pv_done);
                    __syncwarp();
                }
            }
            if (!ok && lane == 0) record(a.error, 56);
            if (!ok) sh.dead = 1;
        }
        __syncwarp();
        __syncthreads();
        if (!more) break;
        if (walker) lay_out();
        if (tid == 0) sh.dead_was = sh.dead;
        __syncthreads();
    }
    // nothing of this thread block is in flight when its memory is given back
    if ((warp == 4 || warp == 7) && sh.dead) {  // else all of it was used
        Drain drain;
        for (uint32_t s = 0; s < kRopes; ++s)
            if (ropes > s) drain.wait(&sh.rope_full[s], ((ropes - 1 - s) / kRopes) & 1);
        // this warp's last fill of each slot
        for (uint32_t fill = pairs > NS ? pairs - NS : 0; fill < pairs; ++fill)
            if ((fill % NP >= 2) == (warp == 7)) drain.wait(&sh.pair_full[fill % NS], (fill / NS) & 1);
    } else if (warp == 5 || warp == 6) {
        if (warp == 5 && asked > qc) mbar_wait_brief(&sh.q_full, qc & 1);  // queries on their way
        if (elect_one()) mma_commit(&sh.drained[warp - 5]);
        if (!mbar_wait_brief(&sh.drained[warp - 5], 0) && lane == 0) record(a.error, 57);
    }
    __syncwarp();
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    if (warp == 5) tmem_dealloc(tmem, 512);
}

// Joins the pieces of row tiles that were split.  Where every row has at most
// kFew pieces, a warp joins a row; else a thread block joins 128 channels of a
// row, each of its warps every eighth piece.
constexpr int kJoinThreads = 256, kJoinBlocks = 6 * kSms, kFew = 8;
template <int C, int NR>
__global__ void __launch_bounds__(kJoinThreads)
latent_join_kernel(const LatentAttnArgs a, const float* parts, const Join* joins, const int n_joins, const int G) {
    using L = LCfg<C, NR>;
    constexpr int kWarps = kJoinThreads / 32, kCols = C / 128;
    static_assert(kSms <= kJoinThreads, "a thread a join");
    __shared__ Join list[kSms];
    __shared__ int begin[kJoinThreads + 1], warps[kWarps];
    __shared__ float4 sum[kWarps][32];
    __shared__ float2 stat[kWarps];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    int n = 0;
    bool many = false;
    if (tid < n_joins) {  // rows of each, and of those before it
        const Join j = joins[tid];
        list[tid] = j;
        n = j.n_pieces > 0 ? j.n_rows : 0;
        many = j.n_pieces > kFew;
    }
    int in = n;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, in, off);
        if (lane >= off) in += x;
    }
    if (lane == 31) warps[warp] = in;
    const bool few = !__syncthreads_or(many);
    for (int w = 0; w < warp; ++w) in += warps[w];
    begin[tid + 1] = in;
    if (tid == 0) begin[0] = 0;
    __syncthreads();
    const int rows = begin[kJoinThreads];

    Join j{0, 0, 0, 0};
    const float* base = nullptr;  // the first piece's results
    size_t gap = 0;               // from the first following piece's to the next one's
    const float* next = nullptr;  // the first following piece's: the next span's first slot
    auto find = [&](int r) {      // row r of all joins; its number within its own
        int lo = 0, hi = n_joins - 1;
        while (lo < hi) {         // the last join that begins at or before it
            const int mid = (lo + hi + 1) >> 1;
            if (begin[mid] <= r) lo = mid;
            else hi = mid - 1;
        }
        j = list[lo];
        const int g = lo % G;
        base = parts + (static_cast<size_t>(j.slot) * G + g) * L::kPart;
        next = parts + (static_cast<size_t>(2 * (j.slot / 2 + 1)) * G + g) * L::kPart;
        gap = 2 * static_cast<size_t>(G) * L::kPart;
        return r - begin[lo];
    };
    auto part = [&](int p) { return p == 0 ? base : next + (p - 1) * gap; };
    auto store = [&](int row, int col, float4 x, float inv) {
        *reinterpret_cast<uint2*>(static_cast<bf16*>(a.out) + (static_cast<size_t>(j.out_row) + row) * C + col) =
            make_uint2(pack_bf16_pair(x.x * inv, x.y * inv), pack_bf16_pair(x.z * inv, x.w * inv));
    };
    auto add = [](float4& x, float4 v, float w) {
        x.x = fmaf(v.x, w, x.x);
        x.y = fmaf(v.y, w, x.y);
        x.z = fmaf(v.z, w, x.z);
        x.w = fmaf(v.w, w, x.w);
    };

    if (few) {
        for (int r = warp * gridDim.x + blockIdx.x; r < rows; r += gridDim.x * kWarps) {
            const int row = find(r);
            float m = -INFINITY, l = 0.0f;
            if (lane < j.n_pieces) {
                m = part(lane)[NR * C + row];
                l = part(lane)[NR * C + NR + row];
            }
            float4 first[kCols], x[kCols];
#pragma unroll
            for (int c = 0; c < kCols; ++c) first[c] = reinterpret_cast<const float4*>(base + static_cast<size_t>(row) * C)[32 * c + lane];
            float top = m;
#pragma unroll
            for (int off = kFew / 2; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
            // a piece that saw no key has a sum of 0, and its outputs were not written
            const float w = l == 0.0f ? 0.0f : exp2_ftz(m - (top == -INFINITY ? 0.0f : top));
            float total = l == 0.0f ? 0.0f : l * w;
#pragma unroll
            for (int off = kFew / 2; off > 0; off >>= 1) total += __shfl_xor_sync(0xffffffffu, total, off);
            total = __shfl_sync(0xffffffffu, total, 0);
            const unsigned seen = __ballot_sync(0xffffffffu, l != 0.0f);
            const float w0 = __shfl_sync(0xffffffffu, w, 0);
#pragma unroll
            for (int c = 0; c < kCols; ++c) {
                x[c] = make_float4(0, 0, 0, 0);
                if (seen & 1u) add(x[c], first[c], w0);
            }
#pragma unroll 2
            for (int p = 1; p < j.n_pieces; ++p) {
                const float wp = __shfl_sync(0xffffffffu, w, p);
                if (!(seen >> p & 1u)) continue;
                const float4* v = reinterpret_cast<const float4*>(part(p) + static_cast<size_t>(row) * C);
#pragma unroll
                for (int c = 0; c < kCols; ++c) add(x[c], v[32 * c + lane], wp);
            }
            const float inv = total == 0.0f ? 0.0f : 1.0f / total;
#pragma unroll
            for (int c = 0; c < kCols; ++c) store(row, 128 * c + 4 * lane, x[c], inv);
        }
        return;
    }
    for (int task = blockIdx.x; task < rows * kCols; task += gridDim.x) {
        const int row = find(task / kCols), col = task % kCols * 128 + 4 * lane;
        float m = -INFINITY, l = 0.0f;
        float4 x = make_float4(0, 0, 0, 0);
        for (int p0 = warp; p0 < j.n_pieces; p0 += kFew * kWarps) {
            float4 v[kFew];  // all loads of a chunk at once
            const int mine = p0 + lane * kWarps;
            float pm = -INFINITY, pl = 0.0f;
            if (lane < kFew && mine < j.n_pieces) {
                pm = part(mine)[NR * C + row];
                pl = part(mine)[NR * C + NR + row];
            }
#pragma unroll
            for (int k = 0; k < kFew; ++k)
                if (p0 + k * kWarps < j.n_pieces) v[k] = *reinterpret_cast<const float4*>(part(p0 + k * kWarps) + static_cast<size_t>(row) * C + col);
            float top = fmaxf(m, pm);
#pragma unroll
            for (int off = kFew / 2; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
            top = __shfl_sync(0xffffffffu, top, 0);
            const float ref = top == -INFINITY ? 0.0f : top, f = m == -INFINITY ? 0.0f : exp2_ftz(m - ref);
            const float w = exp2_ftz(pm - ref);
            l *= f;
            x.x *= f; x.y *= f; x.z *= f; x.w *= f;
            m = top;
#pragma unroll
            for (int k = 0; k < kFew; ++k) {
                const float lk = __shfl_sync(0xffffffffu, pl, k), wk = __shfl_sync(0xffffffffu, w, k);
                if (lk != 0.0f) {
                    l = fmaf(lk, wk, l);
                    add(x, v[k], wk);
                }
            }
        }
        sum[warp][lane] = x;
        if (lane == 0) stat[warp] = make_float2(m, l);
        __syncthreads();
        if (warp == 0) {
            float top = -INFINITY;
            for (int w = 0; w < kWarps; ++w) top = fmaxf(top, stat[w].x);
            const float ref = top == -INFINITY ? 0.0f : top;
            l = 0.0f;
            x = make_float4(0, 0, 0, 0);
            for (int w = 0; w < kWarps; ++w) {
                if (stat[w].y == 0.0f) continue;
                const float f = exp2_ftz(stat[w].x - ref);
                l = fmaf(stat[w].y, f, l);
                add(x, sum[w][lane], f);
            }
            store(row, col, x, l == 0.0f ? 0.0f : 1.0f / l);
        }
        __syncthreads();
    }
}

int rows_of_tile(long long rows) { return rows <= 16 ? 16 : rows <= 32 ? 32 : 64; }

template <int C, int NR, int G>
cudaError_t launch_t(const LatentAttnArgs& a, cudaStream_t st) {
    using L = LCfg<C, NR>;
    static std::atomic<unsigned long long> ready{0};
    cudaError_t e = allow_smem(latent_attention_kernel<C, NR, G>, L::kSmem, ready);
    if (e != cudaSuccess) return e;
    Maps maps{};
    const uint64_t rows = static_cast<uint64_t>(a.c.n_pages) << a.page_shift;
    if (rows > 0 && !(make_tma_map_bf16_2d(&maps.rows, a.c.rows, rows, L::W, L::W, std::min(1 << a.page_shift, kKeys), 64) &&
                      make_tma_map_bf16_3d(&maps.pairs, a.c.rows, 64, rows, L::W / 64, L::W, 64, 64, kKeys, 2)))
        return cudaErrorInvalidValue;
    // queries whose rows (token, head) are evenly spaced are loaded as one matrix
    const long long pitch = a.n_heads == 1 ? a.q.token_stride : a.q.head_stride;
    const bool dense_q = pitch >= L::W && pitch < 1ll << 36 &&
                         (a.n_heads == 1 || a.b.n_tokens == 1 || a.q.token_stride == a.n_heads * a.q.head_stride);
    if (dense_q && !make_tma_map_bf16_2d(&maps.q, a.q.data, static_cast<uint64_t>(a.b.n_tokens) * a.n_heads, L::W, pitch, NR, 64))
        return cudaErrorInvalidValue;
    const int n = kSms / G * G;
    Join* joins = static_cast<Join*>(a.workspace);
    float* parts = reinterpret_cast<float*>(joins + kSms);
    e = timed_launch("latent_attention", st, [&] {
        latent_attention_kernel<C, NR, G><<<n, kThreads, L::kSmem, st>>>(a, maps, static_cast<int>(dense_q), parts, joins);
        return cudaGetLastError();
    });
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(kJoinBlocks);
    cfg.blockDim = dim3(kJoinThreads);
    cfg.stream = st;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return timed_launch("latent_join", st, [&] {
        return cudaLaunchKernelEx(&cfg, latent_join_kernel<C, NR>, a, static_cast<const float*>(parts), static_cast<const Join*>(joins), n, G);
    });
}

// Whether groups of two row tiles are worth it: they take a tenth less time where they are full, but a
// sequence's odd tile leaves one of its two thread blocks without rows.  By two, by one: 64 x 4 tokens of 32
// heads 106 and 118 us, 64 x 5 216 and 191, 64 x 1..8 169 and 154, 255 single tokens beside 3 of one sequence
// 387 and 238.
bool two_tiles(const LatentAttnArgs& a) {
    long long tiles = 0, odd = 0;
    for (int i = 0; i < a.b.n_seq; ++i) {
        const long long n = (static_cast<long long>(a.cu_host[i + 1] - a.cu_host[i]) * a.n_heads + 63) / 64;
        tiles += n;
        odd += n & 1;
    }
    return 10 * odd <= tiles;
}

template <int C>
cudaError_t launch_c(const LatentAttnArgs& a, cudaStream_t st) {
    const long long rows = static_cast<long long>(a.b.max_q) * a.n_heads;
    switch (rows_of_tile(rows)) {
        case 16: return launch_t<C, 16, 1>(a, st);
        case 32: return launch_t<C, 32, 1>(a, st);
        default: return rows > 64 && two_tiles(a) ? launch_t<C, 64, 2>(a, st) : launch_t<C, 64, 1>(a, st);
    }
}

}  // namespace

size_t latent_attention_workspace(int n_heads, int latent_dim, int n_seq, int max_q) {
    if (n_seq == 0 || max_q == 0) return 0;
    const size_t nr = rows_of_tile(static_cast<long long>(max_q) * n_heads);
    return kSms * sizeof(Join) + 2 * kSms * nr * (latent_dim + 2) * sizeof(float);
}

cudaError_t launch_latent_attention(const LatentAttnArgs& a, int latent_dim, cudaStream_t st) {
    return latent_dim == 512 ? launch_c<512>(a, st) : launch_c<256>(a, st);
}

}  // namespace gdn
