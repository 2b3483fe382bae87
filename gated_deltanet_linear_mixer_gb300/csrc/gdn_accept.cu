// Verification of drafted tokens from given random numbers
// (gdn_accept_drafts in include/gdn.h states the rule).
//
// Mathematics.  p_t(x) = e^((l_x - m_t) / tau) / Z_t needs a row's maximum and
// sum (given probabilities need neither); drafts are then decided one after the
// other; and the row where that ends gives argmax_j r_j / e_j.  The race r / e
// needs no prefix sums over the vocabulary, so a result does not depend on the
// order in which threads add, and a row is read once for its sums and once more
// (from L2) for its race.
//
// A cluster of thread blocks takes a sequence, each block a slice of the
// vocabulary; sums and winners are exchanged through distributed shared memory,
// so a sequence needs one launch and no workspace.  What bounds it: HBM for
// large vocabularies and many sequences (64 x 4 drafts of 131,072 probabilities:
// 20 us, 5.0 TB/s), else the chain of memory round trips: lengths, rows,
// exchange, row again, exchange (48 x 3 drafts of 32,003 bf16 logits: 14.5 us).  Of logits, the rows of `step`
// drafts are summed at a time, different warps on different rows: all of them
// where a block's slice is short, one draft after the other where bytes count
// and a fallen draft spares the rows behind it.
#include <algorithm>
#include <cooperative_groups.h>

#include "gdn_internal.h"
#include "gdn_kv.cuh"
#include "gdn_tc.cuh"

namespace cg = cooperative_groups;

namespace gdn {

namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32, kMaxDrafts = 16, kMaxCluster = 8;
constexpr int kRowsMost = 2 * kMaxDrafts + 1;
constexpr int kUnroll = 8;
static_assert(2 * kUnroll * kThreads <= 0x7fffffff - kMostVocab, "indexes past a row's end fit 32 bits");

// A row's logits over one lane's share: running maximum and sum of exponentials
// (of base 2, arguments times c = log2 e / tau), or maximum and its lowest index.
struct Stat {
    float m, s;
    int at;
};
__device__ __forceinline__ Stat join(const Stat& a, const Stat& b, float c) {
    Stat r;
    r.m = fmaxf(a.m, b.m);
    r.s = (a.m == -INFINITY ? 0.0f : a.s * exp2_ftz((a.m - r.m) * c)) +
          (b.m == -INFINITY ? 0.0f : b.s * exp2_ftz((b.m - r.m) * c));
    r.at = a.m > b.m || (a.m == b.m && a.at < b.at) ? a.at : b.at;
    return r;
}

template <bool GREEDY, int N>
__device__ __forceinline__ void take(Stat& r, const float* v, int at, float c) {
    float top = v[0];
#pragma unroll
    for (int k = 1; k < N; ++k) top = fmaxf(top, v[k]);
    if (!(top > r.m || (!GREEDY && r.m > -INFINITY))) return;
    if (GREEDY) {
#pragma unroll
        for (int k = N - 1; k >= 0; --k)
            if (v[k] == top) r.at = at + k;
        r.m = top;
        return;
    }
    if (top > r.m) {
        r.s = r.m == -INFINITY ? 0.0f : r.s * exp2_ftz((r.m - top) * c);
        r.m = top;
    }
#pragma unroll
    for (int k = 0; k < N; ++k) r.s += exp2_ftz((v[k] - r.m) * c);
}

// Lane `idx` of `lanes`' share of elements lo .. hi - 1 of a row, which may start
// anywhere: single elements up to a 16-byte boundary, then 16-byte vectors, 64
// bytes (bf16; fp32 128) of them in flight, then single elements.
// GREEDY: only where the maximum is.
template <typename T, bool GREEDY>
__device__ __forceinline__ Stat row_stat(const T* x, int lo, int hi, int idx, int lanes, float c) {
    constexpr int N = Vec16<T>::N, U = 32 / N;
    Stat r{-INFINITY, 0.0f, 0x7fffffff};
    const int lead = static_cast<int>((16u - (reinterpret_cast<uintptr_t>(x + lo) & 15u)) & 15u) / static_cast<int>(sizeof(T));
    const int body = min(hi, lo + lead), nv = (hi - body) / N, tail = body + nv * N;
    if (lo + idx < body) {
        const float v = to_f32(x[lo + idx]);
        take<GREEDY, 1>(r, &v, lo + idx, c);
    }
    for (int v = idx; v < nv; v += U * lanes) {
        uint4 raw[U];
#pragma unroll
        for (int k = 0; k < U; ++k)
            if (v + k * lanes < nv) raw[k] = Vec16<T>::load_raw(x + body + (v + k * lanes) * N);
#pragma unroll
        for (int k = 0; k < U; ++k)
            if (v + k * lanes < nv) {
                float f[N];
                Vec16<T>::unpack(raw[k], f);
                take<GREEDY, N>(r, f, body + (v + k * lanes) * N, c);
            }
    }
    if (tail + idx < hi) {
        const float v = to_f32(x[tail + idx]);
        take<GREEDY, 1>(r, &v, tail + idx, c);
    }
    return r;
}

// A row's distribution: p_j = 2^((x_j - top) c) scale.
struct Row {
    float top, scale;
};
template <typename T, bool LOGITS>
__device__ __forceinline__ float prob(float x, float c, const Row& r) {
    return LOGITS ? exp2_ftz((x - r.top) * c) * r.scale : x;
}

// Positive scores order as their bits do; the lower index wins a tie.
__device__ __forceinline__ unsigned long long race_key(float score, int j) {
    return static_cast<unsigned long long>(__float_as_uint(score)) << 32 | (0xFFFFFFFFu - static_cast<uint32_t>(j));
}

struct Shared {
    Stat part[kRowsMost][kWarps];          // of this block's warps
    Stat all[kRowsMost][kMaxCluster];      // of the cluster's blocks
    Row rows[kRowsMost];                   // target rows, then draft rows, of the step
    int top_at[kRowsMost];
    unsigned long long best[kWarps];
    unsigned long long winners[2][kMaxCluster];
};

template <typename T, bool LOGITS>
__global__ void __launch_bounds__(kThreads) accept_kernel(const AcceptArgs a, const int step) {
    __shared__ Shared sh;
    tc::cluster_arrive();  // a block writes to another only once that has started: waited for below
    cg::cluster_group cluster = cg::this_cluster();
    const int C = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
    const int seq = blockIdx.x / C, V = a.vocab, T_ = a.T;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int share = (V + C - 1) / C, lo = min(V, rank * share), hi = min(V, lo + share);
    const T* target = static_cast<const T*>(a.target) + static_cast<long long>(seq) * (T_ + 1) * a.target_stride;
    const T* draft = a.draft ? static_cast<const T*>(a.draft) + static_cast<long long>(seq) * T_ * a.draft_stride : nullptr;
    const float temp = LOGITS && a.temperature ? a.temperature[seq] : 1.0f;
    const bool greedy = LOGITS && !(temp > 0.0f);
    const float c = greedy ? kLog2e : kLog2e / temp;
    // lane t: draft t, whether there is one, and its random number
    int x = -1;
    float u = 0.0f;
    if (lane < T_) {
        x = a.drafts[static_cast<long long>(seq) * T_ + lane];
        u = a.uniforms[static_cast<long long>(seq) * T_ + lane];
    }
    if (x < 0 || x >= V) x = -1;
    const unsigned there = __ballot_sync(0xffffffffu, x >= 0);
    const int drafts = __ffs(~there) - 1;  // drafts before the first gap: rows 0 .. drafts may be drawn from
    // given probabilities, and the logits of the drafts: two numbers a draft
    float px = 0.0f, qx = 1.0f;
    if (lane < drafts && !greedy) {
        px = to_f32(target[lane * a.target_stride + x]);
        if (draft) qx = to_f32(draft[lane * a.draft_stride + x]);
    }

    tc::cluster_wait();
    int t = 0, first = 0;  // drafts that stand; first row of the step in shared memory
    bool fell = false;
    Row p{0.0f, 1.0f}, q{0.0f, 1.0f};
    int top_at = -1;
    if (!LOGITS) {
        const unsigned ok = __ballot_sync(0xffffffffu, lane < drafts && u * qx < px);
        t = __ffs(~ok) - 1;
        fell = t < drafts;
    } else {
        for (;;) {
            // rows of drafts first .. first + n - 1, and the row after them where that is the last
            const int n = min(step, drafts - first), nt = first + n == drafts ? n + 1 : n;
            const int nd = draft && !greedy ? n : 0, rows = nt + nd;
            const int per = max(1, kWarps / rows), lanes = 32 * per;
            for (int r = warp / per; r < rows; r += max(1, kWarps / per)) {
                const T* row = r < nt ? target + (first + r) * a.target_stride : draft + (first + r - nt) * a.draft_stride;
                const int idx = (warp % per) * 32 + lane;
                Stat s = greedy ? row_stat<T, true>(row, lo, hi, idx, lanes, c) : row_stat<T, false>(row, lo, hi, idx, lanes, c);
#pragma unroll
                for (int off = 16; off > 0; off >>= 1) {
                    const Stat o{__shfl_xor_sync(0xffffffffu, s.m, off), __shfl_xor_sync(0xffffffffu, s.s, off),
                                 __shfl_xor_sync(0xffffffffu, s.at, off)};
                    s = join(s, o, c);
                }
                if (lane == 0) sh.part[r][warp % per] = s;
            }
            __syncthreads();
            for (int r = tid; r < rows * C; r += kThreads) {  // this block's result of a row to every block
                const int row = r / C, to = r % C;
                Stat s = sh.part[row][0];
                for (int w = 1; w < per; ++w) s = join(s, sh.part[row][w], c);
                *cluster.map_shared_rank(&sh.all[row][rank], to) = s;
            }
            cluster.sync();
            if (tid < rows) {
                Stat s = sh.all[tid][0];
                for (int b = 1; b < C; ++b) s = join(s, sh.all[tid][b], c);
                // a row without a finite logit leaves nothing
                sh.rows[tid] = s.m > -INFINITY && s.s > 0.0f ? Row{s.m, 1.0f / s.s} : Row{0.0f, 0.0f};
                sh.top_at[tid] = s.m > -INFINITY ? s.at : -1;
            }
            __syncthreads();
            // the step's drafts, a lane each
            bool stands = false;
            if (lane >= first && lane < first + n) {
                const int r = lane - first;
                if (greedy) {
                    stands = sh.top_at[r] == x;
                } else {
                    const float pv = prob<T, true>(px, c, sh.rows[r]);
                    const float qv = draft ? prob<T, true>(qx, c, sh.rows[nt + r]) : 1.0f;
                    stands = u * qv < pv;
                }
            }
            const unsigned ok = __ballot_sync(0xffffffffu, stands) | ((1u << first) - 1);
            t = __ffs(~ok) - 1;
            fell = t < first + n;
            if (fell || first + n == drafts) {
                p = sh.rows[t - first];
                top_at = sh.top_at[t - first];
                if (fell && nd) q = sh.rows[nt + t - first];
                break;
            }
            first += n;
            cluster.sync();  // every block has read its results before the next ones arrive
        }
    }

    int token = -1;
    if (greedy) {
        token = top_at;
    } else {
        const T* pr = target + t * a.target_stride;
        const T* qr = fell && draft ? draft + t * a.draft_stride : nullptr;
        const int certain = fell && !draft ? __shfl_sync(0xffffffffu, x, t) : -1;  // a draft with q = 1
        const float* e = a.noise + static_cast<long long>(seq) * a.noise_stride;
        unsigned long long won = 0;
        for (int pass = fell ? 0 : 1; pass < 2 && won == 0; ++pass) {
            unsigned long long best = 0;
            for (int j = lo + tid; j < hi; j += kUnroll * kThreads) {
                float pv[kUnroll], qv[kUnroll], ev[kUnroll];
#pragma unroll
                for (int k = 0; k < kUnroll; ++k) {
                    const int i = j + k * kThreads;
                    pv[k] = i < hi ? to_f32(pr[i]) : 0.0f;
                    qv[k] = i < hi && pass == 0 && qr ? to_f32(qr[i]) : 0.0f;
                    ev[k] = i < hi ? e[i] : 1.0f;
                }
#pragma unroll
                for (int k = 0; k < kUnroll; ++k) {
                    const int i = j + k * kThreads;
                    float r = prob<T, LOGITS>(pv[k], c, p);
                    if (pass == 0) r -= qr ? prob<T, LOGITS>(qv[k], c, q) : (i == certain ? 1.0f : 0.0f);
                    const float score = r / ev[k];
                    if (i < hi && r > 0.0f && score > 0.0f) {
                        const unsigned long long key = race_key(score, i);
                        best = key > best ? key : best;
                    }
                }
            }
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) {
                const unsigned long long o = __shfl_xor_sync(0xffffffffu, best, off);
                best = o > best ? o : best;
            }
            if (lane == 0) sh.best[warp] = best;
            __syncthreads();
            if (tid < C) {
                for (int w = 0; w < kWarps; ++w) best = sh.best[w] > best ? sh.best[w] : best;
                *cluster.map_shared_rank(&sh.winners[pass][rank], tid) = best;
            }
            cluster.sync();
            for (int b = 0; b < C; ++b) won = sh.winners[pass][b] > won ? sh.winners[pass][b] : won;
        }
        if (won) token = static_cast<int>(0xFFFFFFFFu - static_cast<uint32_t>(won));
    }
    if (rank == 0 && warp == 0) {
        if (lane == 0) a.accepted[seq] = t;
        if (lane <= T_) a.tokens[static_cast<long long>(seq) * (T_ + 1) + lane] = lane < t ? x : lane == t ? token : -1;
    }
    cluster.sync();  // no block leaves while another may still write to it
}

template <typename T, bool LOGITS>
cudaError_t accept_t(const AcceptArgs& a, cudaStream_t st) {
    // Blocks of a sequence: enough to occupy the SMs (four blocks fit on one), no slice below 1024.
    // Microseconds with 1 / 2 / 4 / 8 blocks: 1 sequence of 131,072 probabilities 41 / 22 / 13 / 8.4 (8 taken),
    // of 4000 4.7 / 4.1 / 4.6 / 4.6 (2), 256 of 32,000 25 / 20 / 22 / 28 (2); 48 of 32,003 logits
    // 51 / 32 / 20 / 15 (8), 256 of them 89 / 81 / 95 / 114 (2).
    int C = kMaxCluster;
    while (C > 1 && (static_cast<long long>(a.n_seq) * C > 152 * 4 || a.vocab / C < 1024)) C /= 2;
    // Drafts summed at a time: one where bytes count, all where the round trips do.  Microseconds at
    // 1 / 4 / 16: 64 x 8 drafts of 8000 logits 26 / 14.2 / 13.0 (16 taken), 48 x 3 of 32,003 20 at 1 and 14.8
    // otherwise (16, which with three drafts is what 4 is), 256 x 4 of them, whose slices are longer,
    // 80 / 108 / 108 (1), 64 x 4 of 131,072 84 / 107 / 107 (1).
    const int share = a.vocab / C / kThreads;
    const int step = share * (a.T + 1) <= 128 ? kMaxDrafts : share <= 32 ? 4 : 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(a.n_seq) * C);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = st;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = C;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, accept_kernel<T, LOGITS>, a, step);
}

}  // namespace

cudaError_t launch_accept_drafts(const AcceptArgs& a, bool logits, bool bf16, cudaStream_t stream) {
    if (!logits) return accept_t<float, false>(a, stream);
    return bf16 ? accept_t<__nv_bfloat16, true>(a, stream) : accept_t<float, true>(a, stream);
}

}  // namespace gdn
