// moe_dispatch.hip -- a Mixture-of-Experts layer's tokens sorted by expert and
// back, with the gate weights applied, and the gradients of both.
//
//   dispatch:  entry i = t k + s belongs to expert ids[t][s] (in [0, E), else it is
//              dropped); its position is the number of kept entries of smaller experts
//              plus the earlier entries of its own;  Xs[pos] = X[t]
//   combine:   Y[t] = res[t] + sum_s w[t][s] Ys[pos[t][s]]   (ascending s, dropped
//              entries add nothing); dispatch's gradient is this sum without w
//   backward:  dYs[pos] = w[t][s] dY[t],  dw[t][s] = <Ys[pos], dY[t]>
//   routing:   w = softmax over the k chosen logits, so
//              dlogits[t][ids[t][s]] = w_s (dw_s - sum_j w_j dw_j)
//
// Bound: HBM bytes for many tokens (each row is read once and written where it goes,
// whole 16-byte pieces), launches for few.  Positions come from counts, not from
// atomics on lists, so they never depend on the order of arrival.  Measured: combine's
// gradient of 16384 x 4096 bf16, top 2, 125 us (671 MB, 5.4 TB/s); dispatch of 16384 rows of
// 2048 e4m3 codes to 86000 places 54 us, of which 44 move rows (216 MB, most of them written:
// 4.9 TB/s) and 10 are the two launches of the sort.  (Non-temporal stores of the rows: 44 us
// in all, but what reads the rows next then takes longer than that saves: 98 -> 105 us for
// norm, dispatch, a pass over the rows and combine of 4096 x 2048, top 6.)
#include <type_traits>

#include "ffn_device.h"
#include "rows.h"
#include "sublayer.h"

namespace ffn {

namespace {

constexpr int kThreads = 256;
constexpr int kMaxK = 8, kMaxExperts = 256;
constexpr int kSmallEntries = 2048, kSmallTokens = 1024;   // most of one launch that sorts nothing
constexpr int kSortThreads = 1024;      // most entries of one turn of a workgroup that sorts
constexpr int kSortBlocks = 256;        // most workgroups that sort

struct DispatchArgs {
    const char* X;
    const int32_t* ids;
    const float* scale;
    char* Xs;
    float* scale_sorted;
    int32_t *offsets, *entries, *positions;
    int32_t* counts;       // [sort block][E]
    int64_t M, n, row_bytes, scale_cols;
    int64_t per;           // tokens per sort block
    int E, k, blocks;
    int chunks;            // pieces of a row
};

// Few entries: one launch.  A workgroup takes 256 pieces of one token's row and counts
// the entries before each of the token's k by itself, over all ids (from the L2): nothing
// is sorted, and the row's load is under way meanwhile (1000 tokens of 256, top 2: 4.6 us, by
// the next kernel 5.9; 2000 of 4096, top 1: 11.4, 10.4, since each token counts all).
template <typename Vec, int kEach>
__global__ __launch_bounds__(kThreads) void dispatch_small_kernel(DispatchArgs a) {
    constexpr int kBits = 11;      // of an entry: (expert, entry) is one number to compare
    static_assert(kEach * kThreads <= 1 << kBits && kMaxExperts < 1 << (31 - kBits), "keys of 32 bits");
    __shared__ int s_cnt[kThreads / 64][kMaxK];
    __shared__ int s_hist[kMaxExperts];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int k = a.k, E = a.E, n = (int)a.n;
    const int64_t t = blockIdx.x;
    const int chunk = blockIdx.y * kThreads + tid;
    Vec row{};
    if (chunk < a.chunks)
        row = *reinterpret_cast<const Vec*>(a.X + t * a.row_bytes + (int64_t)chunk * sizeof(Vec));
    const bool scales = a.scale && blockIdx.y == 0;
    float sc = 0.f;
    if (scales && tid < a.scale_cols) sc = a.scale[t * a.scale_cols + tid];
    int key[kEach];
#pragma unroll
    for (int u = 0; u < kEach; ++u) {
        const int i = u * kThreads + tid;
        const int id = i < n ? a.ids[i] : E;
        key[u] = ((unsigned)id < (unsigned)E ? id : E) << kBits | i;   // dropped: after all experts
    }
    int mine[kMaxK];
#pragma unroll
    for (int s = 0; s < kMaxK; ++s) {
        mine[s] = s < k ? a.ids[t * k + s] : -1;
        int before = 0;
        if (s < k) {
            const int me = (int)((unsigned)mine[s] << kBits) | ((int)t * k + s);   // (a dropped one's is not used)
#pragma unroll
            for (int u = 0; u < kEach; ++u) before += __popcll(__ballot(key[u] < me));
        }
        if (lane == 0) s_cnt[wave][s] = before;
    }
    const bool first = blockIdx.x == 0 && blockIdx.y == 0;
    if (first && tid < E) s_hist[tid] = 0;
    __syncthreads();
    if (first) {     // the same for the whole workgroup
#pragma unroll
        for (int u = 0; u < kEach; ++u)
            if (key[u] >> kBits < E) atomicAdd(&s_hist[key[u] >> kBits], 1);   // a count: the order does not matter
        __syncthreads();
        // exclusive prefix over the experts, one a thread: within the waves, then between them
        const int mine_e = tid < E ? s_hist[tid] : 0;
        int run = mine_e;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int v = __shfl_up(run, d);
            if (lane >= d) run += v;
        }
        __syncthreads();            // (read before it is written again)
        if (lane == 63) s_hist[wave] = run;
        __syncthreads();
        for (int q = 0; q < wave; ++q) run += s_hist[q];
        if (tid < E) a.offsets[tid] = run - mine_e;
        if (tid == E - 1) a.offsets[E] = run;
    }
#pragma unroll
    for (int s = 0; s < kMaxK; ++s) {
        if (s >= k) break;
        int pos = 0;
#pragma unroll
        for (int q = 0; q < kThreads / 64; ++q) pos += s_cnt[q][s];
        const bool kept = (unsigned)mine[s] < (unsigned)E;
        if (blockIdx.y == 0 && tid == 0) {
            a.positions[t * k + s] = kept ? pos : -1;
            if (kept) a.entries[pos] = (int32_t)(t * k + s);
        }
        if (!kept) continue;
        if (chunk < a.chunks)
            *reinterpret_cast<Vec*>(a.Xs + (int64_t)pos * a.row_bytes + (int64_t)chunk * sizeof(Vec)) = row;
        if (!scales) continue;
        if (tid < a.scale_cols) a.scale_sorted[pos * a.scale_cols + tid] = sc;
        for (int64_t c = tid + kThreads; c < a.scale_cols; c += kThreads)
            a.scale_sorted[pos * a.scale_cols + c] = a.scale[t * a.scale_cols + c];
    }
}

// Rows r, r + step, ... of `tokens` tokens from `base` on, pieces c0, c0 + tpr, ... of each:
// a piece is read once and written to the row's kept positions (pos: k per token).
template <typename Vec>
__device__ __forceinline__ void move_rows(const DispatchArgs& a, int64_t base, int tokens, const int* pos, int r,
                                          int step, int c0, int tpr) {
    for (; r < tokens; r += step) {
        int at[kMaxK];
#pragma unroll
        for (int s = 0; s < kMaxK; ++s) at[s] = s < a.k ? pos[r * a.k + s] : -1;
        const char* src = a.X + (base + r) * a.row_bytes;
        for (int c = c0; c < a.chunks; c += tpr) {
            const Vec v = *reinterpret_cast<const Vec*>(src + (int64_t)c * sizeof(Vec));
#pragma unroll
            for (int s = 0; s < kMaxK; ++s)
                if (at[s] >= 0)
                    *reinterpret_cast<Vec*>(a.Xs + at[s] * a.row_bytes + (int64_t)c * sizeof(Vec)) = v;
        }
        if (!a.scale) continue;
        for (int64_t c = c0; c < a.scale_cols; c += tpr) {
            const float v = a.scale[(base + r) * a.scale_cols + c];
#pragma unroll
            for (int s = 0; s < kMaxK; ++s)
                if (at[s] >= 0) a.scale_sorted[at[s] * a.scale_cols + c] = v;
        }
    }
}

// More entries than that (kCountAll) in three steps.  1: each block's entries per expert.
__global__ __launch_bounds__(kSortThreads) void dispatch_count_kernel(DispatchArgs a) {
    __shared__ int s_hist[kMaxExperts];
    const int tid = threadIdx.x, E = a.E;
    if (tid < E) s_hist[tid] = 0;
    __syncthreads();
    const int64_t lo = blockIdx.x * a.per * a.k, end = lo + a.per * a.k, hi = end < a.n ? end : a.n;
    for (int64_t i = lo + tid; i < hi; i += kSortThreads) {
        const int e = a.ids[i];
        if ((unsigned)e < (unsigned)E) atomicAdd(&s_hist[e], 1);   // a count: the order does not matter
    }
    __syncthreads();
    if (tid < E) a.counts[(int64_t)blockIdx.x * E + tid] = s_hist[tid];
}

// Step 2: a block adds the counts of the blocks before it and all blocks' totals and ranks
// its tokens' entries in order, up to 1024 at a time: within a wave by ballots over the bits
// of the expert (lanes that agree in every bit are peers), between waves by their counts.
//
// kAll, for up to kCountAll entries, is the only step: every block counts all ids itself and
// moves its rows too (12288 entries, 2048 columns: 15.3 us instead of 17.3 in three launches;
// 16384 of 7168 bytes: 42.1, 40.6: the counting grows with them, and 256 workgroups move rows at
// 3/4 of the rate of many).
template <typename Vec, bool kAll>
__global__ __launch_bounds__(kSortThreads) void dispatch_sort_kernel(DispatchArgs a, int tpr_log) {
    constexpr int kWaves = kSortThreads / 64;
    __shared__ int s_one[kSortThreads], s_two[kSortThreads];   // then: the positions of a turn
    __shared__ int s_base[kMaxExperts], s_scan[kWaves];
    __shared__ int s_w[kWaves][kMaxExperts];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, E = a.E, k = a.k;
    const int64_t t0 = blockIdx.x * a.per, t1 = t0 + a.per < a.M ? t0 + a.per : a.M;
    const int turn = kSortThreads / k;     // tokens of one turn
    auto expert = [&](int64_t base) {      // of this thread's entry in the turn from token `base` on
        return tid < (t1 - base < turn ? (int)(t1 - base) : turn) * k ? a.ids[base * k + tid] : -1;
    };
    int next = expert(t0);                 // (under way while the counts are added)
    int epow = 1, bits = 0;
    while (epow < E) {
        epow <<= 1;
        ++bits;
    }
    {
        int before = 0, total = 0;
        if constexpr (!kAll) {
            const int parts = kSortThreads / epow, e = tid & (epow - 1), p = tid / epow;
            if (e < E)
#pragma unroll 4
                for (int b = p; b < a.blocks; b += parts) {
                    const int c = a.counts[(int64_t)b * E + e];
                    total += c;
                    if (b < (int)blockIdx.x) before += c;
                }
            s_one[tid] = before;
            s_two[tid] = total;
            __syncthreads();
            before = total = 0;
            if (tid < epow)
                for (int q = 0; q < parts; ++q) {
                    before += s_one[q * epow + tid];
                    total += s_two[q * epow + tid];
                }
        } else {
            if (tid < kMaxExperts) s_one[tid] = s_two[tid] = 0;
            __syncthreads();
            constexpr int kBatch = 8;      // loads under way at once
            for (int i0 = tid; i0 < (int)a.n; i0 += kBatch * kSortThreads) {
                int id[kBatch];
#pragma unroll
                for (int u = 0; u < kBatch; ++u) {
                    const int i = i0 + u * kSortThreads;
                    id[u] = i < (int)a.n ? a.ids[i] : -1;
                }
#pragma unroll
                for (int u = 0; u < kBatch; ++u)     // counts: the order does not matter
                    if ((unsigned)id[u] < (unsigned)E)
                        atomicAdd(i0 + u * kSortThreads < (int)t0 * k ? &s_one[id[u]] : &s_two[id[u]], 1);
            }
            __syncthreads();
            if (tid < epow) {
                before = s_one[tid];
                total = before + s_two[tid];
            }
        }
        // prefix of the totals over the experts, one a thread: within the waves, then between them
        int run = tid < epow ? total : 0;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int v = __shfl_up(run, d);
            if (lane >= d) run += v;
        }
        if (lane == 63) s_scan[wave] = run;
        __syncthreads();
        if (tid < E) {
            int off = run - total;
            for (int q = 0; q < wave; ++q) off += s_scan[q];
            s_base[tid] = off + before;
            if (blockIdx.x == 0) {
                a.offsets[tid] = off;
                if (tid == E - 1) a.offsets[E] = off + total;
            }
        }
    }
    const uint64_t lt = lane == 0 ? 0ull : ~0ull >> (64 - lane);
    const int tpr = 1 << tpr_log, c0 = tid & (tpr - 1), r0 = tid >> tpr_log, step = kSortThreads >> tpr_log;
    for (int64_t base = t0; base < t1; base += turn) {
        const int tokens = t1 - base < turn ? (int)(t1 - base) : turn;
        const int64_t i = base * k + tid;
        const bool have = tid < tokens * k;
        const int e = next;
        if (base + turn < t1) next = expert(base + turn);
        const bool kept = (unsigned)e < (unsigned)E;
        // (a wave clears its own counts: slower waves still read theirs of the last turn)
        for (int q = lane; q < kMaxExperts; q += 64) s_w[wave][q] = 0;
        uint64_t peers = __ballot(kept);
        for (int b = 0; b < bits; ++b) {
            const bool one = (e >> b) & 1;
            const uint64_t m = __ballot(one);
            peers &= one ? m : ~m;
        }
        const int rank = __popcll(peers & lt);
        __syncthreads();   // s_w cleared, s_base written; the last turn's positions read
        if (kept && rank == 0) s_w[wave][e] = __popcll(peers);
        __syncthreads();
        if (tid < E) {
            int run = s_base[tid];
#pragma unroll
            for (int q = 0; q < kWaves; ++q) {
                const int c = s_w[q][tid];
                s_w[q][tid] = run;
                run += c;
            }
            s_base[tid] = run;
        }
        __syncthreads();
        int pos = -1;
        if (kept) pos = s_w[wave][e] + rank;
        if (pos >= a.n) pos = -1;   // (only if the ids were changed meanwhile)
        if (have) {
            a.positions[i] = pos;
            if (pos >= 0) a.entries[pos] = (int32_t)i;
        }
        if constexpr (kAll) {
            s_one[tid] = pos;
            __syncthreads();
            move_rows<Vec>(a, base, tokens, s_one, r0, step, c0, tpr);
        }
    }
}

// Step 3: the rows.  A workgroup holds 256 / tpr tokens, tpr threads each.
template <typename Vec>
__global__ __launch_bounds__(kThreads) void dispatch_rows_kernel(DispatchArgs a, int tpr_log) {
    const int tpr = 1 << tpr_log, per = kThreads >> tpr_log;
    const int64_t t = (int64_t)blockIdx.x * per;
    const int tokens = a.M - t < per ? (int)(a.M - t) : per;
    move_rows<Vec>(a, t, tokens, a.positions + t * a.k, threadIdx.x >> tpr_log, per, threadIdx.x & (tpr - 1), tpr);
}

// Threads per row (a power of two up to `most`, 2^l) for `pieces` of a row: log2.
int threads_per_row_log(int64_t pieces, int most) {
    int l = 0;
    while (l < most && ((int64_t)1 << l) < pieces) ++l;
    return l;
}

// Tokens per workgroup of the sort, and its workgroups.  With all ids counted by each the rows
// are spread as far as they go; otherwise whole turns, for fewer counts to add.
constexpr int64_t kCountAll = 12288;   // most entries that every workgroup counts by itself
int64_t sort_tokens(int64_t M, int k) {
    const int64_t even = (M + kSortBlocks - 1) / kSortBlocks, turn = kSortThreads / k;
    if (M * k <= kCountAll) return even > 0 ? even : 1;
    return even > turn ? even : turn;
}
int64_t sort_blocks(int64_t M, int k) { return (M + sort_tokens(M, k) - 1) / sort_tokens(M, k); }

// ---------------------------------------------------------------- combine

struct CombineArgs {
    const void* rows;
    const int32_t* pos;
    const float* w;
    const void* res;
    void* Y;
    int64_t M;
    unsigned R;      // below 2^31
    int N;
};

// All of a piece's k loads are issued before the first is used; the sum is fp32, in
// ascending s, rounded once.
template <bool kF32, int K>
__global__ __launch_bounds__(kThreads) void combine_rows_kernel(CombineArgs a, int tpr_log) {
    const int tpr = 1 << tpr_log;
    const int c0 = (threadIdx.x & (tpr - 1)) * 8;
    const int64_t t = (int64_t)blockIdx.x * (kThreads >> tpr_log) + (threadIdx.x >> tpr_log);
    if (t >= a.M) return;
    int64_t at[K];
    float w[K];
#pragma unroll
    for (int s = 0; s < K; ++s) {
        const int p = a.pos[t * K + s];
        at[s] = (unsigned)p < a.R ? (int64_t)p * a.N : -1;   // (a negative one is past 2^31)
        w[s] = a.w ? a.w[t * K + s] : 1.f;
    }
    for (int c = c0; c < a.N; c += 8 * tpr) {
        Ln8<kF32> in[K], r;
        r.zero();
        if (a.res) r.load(a.res, t * a.N + c);
#pragma unroll
        for (int s = 0; s < K; ++s) {
            in[s].zero();
            if (at[s] >= 0) in[s].load(a.rows, at[s] + c);
        }
        float y[8];
        r.get(y);
#pragma unroll
        for (int s = 0; s < K; ++s) {
            if (at[s] < 0) continue;   // (a dropped entry's weight may be anything)
            float v[8];
            in[s].get(v);
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = fmaf(w[s], v[e], y[e]);
        }
        ln_store<kF32>(a.Y, t * a.N + c, y);
    }
}

struct CombineBackwardArgs {
    const void *dY, *rows;
    const int32_t* pos;
    const float* w;
    void* drows;
    float* dw;
    int64_t M;
    unsigned R;      // below 2^31
    int N, W, G;     // W waves per token, G tokens per workgroup; short rows: W lanes per token
};

// Sum over each W neighbouring lanes (a power of two up to 32), in the last of them: within
// fours, eights and rows of 16 lanes by exchange, into the second of two rows by a copy.
__device__ __forceinline__ float part_sum(float v, int W) {
    if (W > 1) v = dpp_add<0xb1, 0xf>(v);     // quad_perm 1 0 3 2
    if (W > 2) v = dpp_add<0x4e, 0xf>(v);     // quad_perm 2 3 0 1
    if (W > 4) v = dpp_add<0x141, 0xf>(v);    // row_half_mirror
    if (W > 8) v = dpp_add<0x140, 0xf>(v);    // row_mirror
    if (W > 16) v = dpp_add<0x142, 0xa>(v);   // row_bcast:15 into rows 1 and 3
    return v;
}

// dY is read once: every piece is multiplied into the k dot products and written,
// weighted, to the k rows.  The dots are fp32 lane sums over a lane's pieces, then over
// the wave, then over the W waves, in a fixed order.  Rows of up to 256 columns (kShort)
// take as many lanes as they have pieces, several tokens to a wave (28133 x 104 fp32, top
// 7, three quarters dropped: 16 us, a wave each 26).  That is 56 MB, 35 read and 21 written, at
// 3.5 TB/s: a lane has one piece, so its loads of positions, of rows and its stores are one chain
// with no other piece behind it (none dropped: 175 MB in 53 us, 3.3 TB/s; rows of whole lines,
// 128 columns, 3.8 and 4.0).  A token without entries is not read (8000 x 5456 fp32, top 4, three
// quarters dropped: 110 -> 100 us).
template <bool kF32, int K, bool kShort>
__global__ __launch_bounds__(kThreads) void combine_backward_kernel(CombineBackwardArgs a) {
    __shared__ float s_part[kThreads / 64][K];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int g = kShort ? threadIdx.x / a.W : wave / a.W, w = kShort ? 0 : wave % a.W;
    const int piece = kShort ? threadIdx.x % a.W : w * 64 + lane;
    const int64_t t = (int64_t)blockIdx.x * a.G + g;
    const bool on = t < a.M;
    int64_t at[K];
    float wt[K], dot[K];
    bool any = false;
#pragma unroll
    for (int s = 0; s < K; ++s) {
        const int p = on ? a.pos[t * K + s] : -1;
        at[s] = (unsigned)p < a.R ? (int64_t)p * a.N : -1;   // (a negative one is past 2^31)
        wt[s] = on && a.w ? a.w[t * K + s] : 1.f;
        dot[s] = 0.f;
        any |= at[s] >= 0;
    }
    if (any)
        for (int c = piece * 8; c < a.N; c += a.W * kLnCols) {
            Ln8<kF32> d, in[K];
            d.load(a.dY, t * a.N + c);
            if (a.dw) {
#pragma unroll
                for (int s = 0; s < K; ++s) {
                    in[s].zero();
                    if (at[s] >= 0) in[s].load(a.rows, at[s] + c);
                }
            }
            float y[8];
            d.get(y);
#pragma unroll
            for (int s = 0; s < K; ++s) {
                if (at[s] < 0) continue;
                float v[8];
                if (a.dw) {
                    in[s].get(v);
#pragma unroll
                    for (int e = 0; e < 8; ++e) dot[s] = fmaf(y[e], v[e], dot[s]);
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = wt[s] * y[e];
                ln_store<kF32>(a.drows, at[s] + c, v);
            }
        }
    if (!a.dw) return;
    if constexpr (kShort) {
#pragma unroll
        for (int s = 0; s < K; ++s) dot[s] = part_sum(dot[s], a.W);
        if (!on || piece != a.W - 1) return;
#pragma unroll
        for (int s = 0; s < K; ++s) a.dw[t * K + s] = dot[s];
        return;
    }
#pragma unroll
    for (int s = 0; s < K; ++s) {
        const float v = wave_sum(dot[s]);
        if (lane == 0) s_part[wave][s] = v;
    }
    __syncthreads();
    if (on && w == 0 && lane < K) {
        float v = 0.f;
        for (int q = 0; q < a.W; ++q) v += s_part[g * a.W + q][lane];
        a.dw[t * K + lane] = v;
    }
}

// 2^tpr_log threads per token take pieces of V logits each and compare their experts with the
// token's k choices, whose loads are all under way at once (100000 x 256, top 8: 26 us; a thread
// per logit, which loads them for each, 74).
template <int K, int V>
__global__ __launch_bounds__(kThreads) void route_backward_kernel(const int32_t* __restrict__ ids,
                                                                  const float* __restrict__ w,
                                                                  const float* __restrict__ dw,
                                                                  float* __restrict__ dlogits, int64_t M, int E,
                                                                  int tpr_log) {
    const int64_t t = (int64_t)blockIdx.x * (kThreads >> tpr_log) + (threadIdx.x >> tpr_log);
    if (t >= M) return;
    int id[K];
    float wt[K], d[K];
#pragma unroll
    for (int s = 0; s < K; ++s) {
        id[s] = ids[t * K + s];
        wt[s] = w[t * K + s];
        d[s] = dw[t * K + s];
    }
    float mean = 0.f;
#pragma unroll
    for (int s = 0; s < K; ++s) mean = fmaf(wt[s], d[s], mean);
#pragma unroll
    for (int s = 0; s < K; ++s) d[s] = wt[s] * (d[s] - mean);
    for (int e = (threadIdx.x & ((1 << tpr_log) - 1)) * V; e < E; e += V << tpr_log) {
        float sum[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            sum[v] = 0.f;
#pragma unroll
            for (int s = 0; s < K; ++s) sum[v] += id[s] == e + v ? d[s] : 0.f;
        }
        float* out = dlogits + t * E + e;
        if constexpr (V == 4) *reinterpret_cast<float4*>(out) = make_float4(sum[0], sum[1], sum[2], sum[3]);
        else out[0] = sum[0];
    }
}

// A launch holds fewer than 2^32 threads: M tokens, `per` to a workgroup, in slices of at most
// 2^22 workgroups.  go(t0, tokens, grid) launches one.
template <typename F>
hipError_t in_slices(int64_t M, int64_t per, F&& go) {
    const int64_t most = per << 22;
    for (int64_t t0 = 0; t0 < M; t0 += most) {
        const int64_t n = M - t0 < most ? M - t0 : most;
        go(t0, n, dim3((unsigned)((n + per - 1) / per)));
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

template <typename F>
hipError_t with_k(int k, F&& f) {
    switch (k) {
        case 1: return f(std::integral_constant<int, 1>());
        case 2: return f(std::integral_constant<int, 2>());
        case 3: return f(std::integral_constant<int, 3>());
        case 4: return f(std::integral_constant<int, 4>());
        case 5: return f(std::integral_constant<int, 5>());
        case 6: return f(std::integral_constant<int, 6>());
        case 7: return f(std::integral_constant<int, 7>());
        case 8: return f(std::integral_constant<int, 8>());
        default: return hipErrorInvalidValue;
    }
}

}  // namespace

size_t dispatch_count_ints(int64_t M, int64_t E, int k) {
    return M * k <= kCountAll ? 0 : (size_t)(sort_blocks(M, k) * E);
}

hipError_t launch_moe_dispatch(const DispatchIO& io, hipStream_t stream) {
    DispatchArgs a;
    a.X = static_cast<const char*>(io.X);
    a.ids = io.ids;
    a.scale = io.scale;
    a.Xs = static_cast<char*>(io.Xs);
    a.scale_sorted = io.scale_sorted;
    a.offsets = io.offsets;
    a.entries = io.entries;
    a.positions = io.positions;
    a.counts = io.counts;
    a.M = io.M;
    a.n = io.M * io.k;
    a.row_bytes = io.row_bytes;
    a.scale_cols = io.scale_cols;
    a.E = io.E;
    a.k = io.k;
    a.per = sort_tokens(io.M, io.k);
    a.blocks = (int)sort_blocks(io.M, io.k);
    const bool wide = io.row_bytes % 16 == 0;   // e4m3 rows of odd multiples of 8: 8-byte pieces
    a.chunks = (int)(io.row_bytes / (wide ? 16 : 8));
    if (a.n <= kSmallEntries && io.M <= kSmallTokens) {
        const dim3 grid((unsigned)io.M, (unsigned)((a.chunks + kThreads - 1) / kThreads));
        auto go = [&](auto each) {
            if (wide) hipLaunchKernelGGL((dispatch_small_kernel<uint4, each.value>), grid, dim3(kThreads), 0, stream, a);
            else hipLaunchKernelGGL((dispatch_small_kernel<uint2, each.value>), grid, dim3(kThreads), 0, stream, a);
        };
        if (a.n <= 4 * kThreads) go(std::integral_constant<int, 4>());
        else go(std::integral_constant<int, kSmallEntries / kThreads>());
        return hipGetLastError();
    }
    const dim3 blocks((unsigned)a.blocks), threads(kSortThreads);
    if (a.n <= kCountAll) {
        const int l = threads_per_row_log(a.chunks, 10);
        if (wide) hipLaunchKernelGGL((dispatch_sort_kernel<uint4, true>), blocks, threads, 0, stream, a, l);
        else hipLaunchKernelGGL((dispatch_sort_kernel<uint2, true>), blocks, threads, 0, stream, a, l);
        return hipGetLastError();
    }
    hipLaunchKernelGGL(dispatch_count_kernel, blocks, threads, 0, stream, a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((dispatch_sort_kernel<uint4, false>), blocks, threads, 0, stream, a, 0);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    const int l = threads_per_row_log(a.chunks, 8);
    return in_slices(io.M, kThreads >> l, [&](int64_t t0, int64_t n, dim3 grid) {
        DispatchArgs s = a;
        s.X += t0 * a.row_bytes;
        s.positions += t0 * a.k;
        if (a.scale) s.scale += t0 * a.scale_cols;
        s.M = n;
        if (wide) hipLaunchKernelGGL(dispatch_rows_kernel<uint4>, grid, dim3(kThreads), 0, stream, s, l);
        else hipLaunchKernelGGL(dispatch_rows_kernel<uint2>, grid, dim3(kThreads), 0, stream, s, l);
    });
}

hipError_t launch_moe_combine_rows(const void* rows, int64_t R, const int32_t* pos, const float* w,
                                   const void* res, void* Y, int64_t M, int64_t N, int k, bool f32,
                                   hipStream_t stream) {
    const int l = threads_per_row_log(N / 8, 8);
    const int64_t row = N * (f32 ? 4 : 2);
    return with_k(k, [&](auto K) {
        return in_slices(M, kThreads >> l, [&](int64_t t0, int64_t n, dim3 grid) {
            CombineArgs a;
            a.rows = rows;
            a.pos = pos + t0 * k;
            a.w = w ? w + t0 * k : nullptr;
            a.res = res ? static_cast<const char*>(res) + t0 * row : nullptr;
            a.Y = static_cast<char*>(Y) + t0 * row;
            a.M = n;
            a.R = (unsigned)R;
            a.N = (int)N;
            if (f32)
                hipLaunchKernelGGL((combine_rows_kernel<true, K.value>), grid, dim3(kThreads), 0, stream, a, l);
            else
                hipLaunchKernelGGL((combine_rows_kernel<false, K.value>), grid, dim3(kThreads), 0, stream, a, l);
        });
    });
}

hipError_t launch_moe_combine_backward(const void* dY, const void* rows, int64_t R, const int32_t* pos,
                                       const float* w, void* drows, float* dw, int64_t M, int64_t N,
                                       int k, bool f32, hipStream_t stream) {
    const bool part = N <= kLnCols / 2;     // lanes of a wave
    const int W = part ? 1 << threads_per_row_log(N / 8, 5) : N > 2 * kLnCols ? 4 : N > kLnCols ? 2 : 1;
    const int G = (part ? kThreads : kThreads / 64) / W;
    return with_k(k, [&](auto K) {
        return in_slices(M, G, [&](int64_t t0, int64_t n, dim3 grid) {
            CombineBackwardArgs a;
            a.dY = static_cast<const char*>(dY) + t0 * N * (f32 ? 4 : 2);
            a.rows = rows;
            a.pos = pos + t0 * k;
            a.w = w ? w + t0 * k : nullptr;
            a.drows = drows;
            a.dw = dw ? dw + t0 * k : nullptr;
            a.M = n;
            a.R = (unsigned)R;
            a.N = (int)N;
            a.W = W;
            a.G = G;
            const dim3 block(kThreads);
            if (f32 && part) hipLaunchKernelGGL((combine_backward_kernel<true, K.value, true>), grid, block, 0, stream, a);
            else if (f32) hipLaunchKernelGGL((combine_backward_kernel<true, K.value, false>), grid, block, 0, stream, a);
            else if (part) hipLaunchKernelGGL((combine_backward_kernel<false, K.value, true>), grid, block, 0, stream, a);
            else hipLaunchKernelGGL((combine_backward_kernel<false, K.value, false>), grid, block, 0, stream, a);
        });
    });
}

hipError_t launch_moe_route_backward(const int32_t* ids, const float* w, const float* dw, float* dlogits,
                                     int64_t M, int E, int k, hipStream_t stream) {
    // four pieces a thread, where a token has as many
    const bool fours = E % 4 == 0;
    const int l = threads_per_row_log(((fours ? E / 4 : E) + 3) / 4, 6);
    return with_k(k, [&](auto K) {
        return in_slices(M, kThreads >> l, [&](int64_t t0, int64_t n, dim3 grid) {
            const int32_t* i = ids + t0 * k;
            float* out = dlogits + t0 * E;
            if (fours)
                hipLaunchKernelGGL((route_backward_kernel<K.value, 4>), grid, dim3(kThreads), 0, stream, i, w + t0 * k,
                                   dw + t0 * k, out, n, E, l);
            else
                hipLaunchKernelGGL((route_backward_kernel<K.value, 1>), grid, dim3(kThreads), 0, stream, i, w + t0 * k,
                                   dw + t0 * k, out, n, E, l);
        });
    });
}

}  // namespace ffn
