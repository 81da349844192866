// layernorm.hip -- layer normalisation over the last dimension and its
// gradients, bf16 or fp32 data, fp32 statistics and sums.
//
//   forward:   mean = sum_j x_j / N,  rstd = 1 / sqrt(sum_j (x_j - mean)^2 / N + eps)
//              y_j = (x_j - mean) rstd gamma_j + beta_j
//   backward:  z_j = (x_j - mean) rstd,  t_j = dy_j gamma_j
//              dx_j = rstd (t_j - sum t / N - z_j sum (t z) / N)
//              dgamma_j = sum_rows dy_j z_j,   dbeta_j = sum_rows dy_j
//
// Bound: HBM bytes -- the forward reads x and writes y, the backward reads x and
// dy and writes dx; everything between stays in registers.  A row is held by W
// waves, eight consecutive columns per lane and step (one 16-byte load of bf16, two
// of fp32), so it is read once: the variance is the centred sum over the held
// values, with no cancellation.  Workgroups walk many rows, with the next rows' loads
// in flight behind the current row's sums: what a CU has in flight sets the rate (one
// row per workgroup and no prefetch: 72 us forward, 111 us backward at 8192 x 8192
// bf16).
#include <type_traits>

#include "ffn_device.h"
#include "ffn_internal.h"
#include "rows.h"

namespace ffn {

namespace {

constexpr int kLnThreads = 1024;   // largest workgroup

// Sum over the W waves of a row, in ascending wave order.  `part` holds one
// float per wave of the workgroup and is used once between two barriers.
__device__ __forceinline__ float row_sum(float v, float* part, int wave, int first, int W) {
    v = wave_sum(v);
    if (W == 1) return v;
    if ((threadIdx.x & 63) == 0) part[wave] = v;
    __syncthreads();
    float s = 0.f;
    for (int w = 0; w < W; ++w) s += part[first + w];
    return s;
}

// Row group g of a workgroup = W waves; a workgroup takes G rows at once and
// walks on by the grid.
template <bool kF32, int V, int kThreads>
__global__ __launch_bounds__(kThreads) void ln_forward_kernel(
    const void* X, const void* __restrict__ gamma, const void* __restrict__ beta, void* Y,
    float* __restrict__ mean_out, float* __restrict__ rstd_out, int64_t M, int N, int W, int G,
    float eps) {
    __shared__ float s_part[2][kThreads / 64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int g = wave / W, w = wave % W;
    const int64_t step = (int64_t)gridDim.x * G;
    auto column = [&](int v) { return ((v * W + w) * 64 + lane) * 8; };
    Ln8<kF32> ga[V], be[V], next[V];
    auto fetch = [&](int64_t row) {
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (row < M && column(v) < N) next[v].load(X, row * N + column(v));
            else next[v].zero();
    };
    int64_t base = (int64_t)blockIdx.x * G;
    fetch(base + g);
#pragma unroll
    for (int v = 0; v < V; ++v) {
        ga[v].zero();
        be[v].zero();
        if (column(v) < N) {
            ga[v].load(gamma, column(v));
            be[v].load(beta, column(v));
        }
    }
    for (; base < M; base += step) {
        const int64_t row = base + g;
        float x[V][8];
        float s = 0.f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            next[v].get(x[v]);
#pragma unroll
            for (int e = 0; e < 8; ++e) s += x[v][e];
        }
        if (base + step < M) fetch(row + step);
        const float mean = row_sum(s, s_part[0], wave, g * W, W) / (float)N;
        float q = 0.f;
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (column(v) < N) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    x[v][e] -= mean;
                    q += x[v][e] * x[v][e];
                }
            }
        // (a row's first sums are read between this barrier and the one before: the
        // next row's waves write them again only after passing this one)
        const float var = row_sum(q, s_part[1], wave, g * W, W) / (float)N;
        const float rstd = 1.0f / sqrtf(var + eps);
        if (row >= M) continue;
        if (w == 0 && lane == 0) {
            if (mean_out) mean_out[row] = mean;
            if (rstd_out) rstd_out[row] = rstd;
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
            if (column(v) >= N) continue;
            float a[8], b[8], y[8];
            ga[v].get(a);
            be[v].get(b);
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = x[v][e] * rstd * a[e] + b[e];
            ln_store<kF32>(Y, row * N + column(v), y);
        }
    }
}

// A workgroup walks rows blockIdx.x * G + g, + gridDim.x * G, ...; a lane keeps
// its columns' dgamma and dbeta sums in registers over all of them, so the
// column sums cost one partial row per workgroup instead of a second pass over x
// and dy.  part: [workgroup][2][N], dgamma first.  The loads run kAhead rows ahead;
// two steps a lane of fp32 (N > 8192) leave no registers for that, and x and dy are
// read again (from the L2) for dx.
template <bool kF32, int V>
__global__ __launch_bounds__(kLnThreads) void ln_backward_kernel(
    const void* X, const void* dY, const void* __restrict__ gamma,
    const float* __restrict__ mean_in, const float* __restrict__ rstd_in, void* dX,
    float* __restrict__ part, int64_t M, int N, int W, int G) {
    constexpr int kAhead = V == 1 ? (kF32 ? 2 : 3) : kF32 ? 0 : 1;
    __shared__ float s_part[2][2][kLnThreads / 64];
    extern __shared__ float s_col[];   // [G][2][columns held], used once at the end (G > 1)
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int g = wave / W, w = wave % W;
    auto column = [&](int v) { return ((v * W + w) * 64 + lane) * 8; };
    Ln8<kF32> ga[V];
    float sg[V][8], sb[V][8];
#pragma unroll
    for (int v = 0; v < V; ++v) {
#pragma unroll
        for (int e = 0; e < 8; ++e) sg[v][e] = sb[v][e] = 0.f;
        ga[v].zero();
        if (column(v) < N) ga[v].load(gamma, column(v));
    }
    const int64_t step = (int64_t)gridDim.x * G;
    constexpr int kSets = kAhead ? kAhead : 1;
    Ln8<kF32> xr[kSets][V], dr[kSets][V];
    float mr[kSets], rr[kSets];
    auto fetch = [&](int64_t row, int set) {
        const bool on = row < M;
        mr[set] = on ? mean_in[row] : 0.f;
        rr[set] = on ? rstd_in[row] : 0.f;
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (on && column(v) < N) {
                xr[set][v].load(X, row * N + column(v));
                dr[set][v].load(dY, row * N + column(v));
            } else {
                xr[set][v].zero();
                dr[set][v].zero();
            }
    };
    int turn = 0;
    // one row's work: its loads lie in set `set`; `ahead` is the row to load next into it
    auto work = [&](int64_t row, int set, int64_t ahead) {
        const bool on = row < M;
        const float mean = mr[set], rstd = rr[set];
        constexpr int kHeld = kAhead ? V : 1;
        float z[kHeld][8], t[kHeld][8];
        float s1 = 0.f, s2 = 0.f;
        auto split = [&](int v, float (&zz)[8], float (&tt)[8]) {
            xr[set][v].get(zz);
            dr[set][v].get(tt);
            // Columns past N hold x = 0, and mean * rstd may leave fp32 where no column's z does (a
            // constant row); with 0 for rstd their z is 0 and adds nothing to the sums.
            const float by = column(v) < N ? rstd : 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) zz[e] = (zz[e] - mean) * by;
        };
#pragma unroll
        for (int v = 0; v < V; ++v) {
            float(&zz)[8] = z[kAhead ? v : 0];
            float(&tt)[8] = t[kAhead ? v : 0];
            if constexpr (!kAhead) {
                if (on && column(v) < N) {
                    xr[0][v].load(X, row * N + column(v));
                    dr[0][v].load(dY, row * N + column(v));
                } else {
                    xr[0][v].zero();
                    dr[0][v].zero();
                }
            }
            split(v, zz, tt);
            float a[8];
            ga[v].get(a);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                // (columns past N and rows past M have dy = 0)
                sg[v][e] += tt[e] * zz[e];
                sb[v][e] += tt[e];
                tt[e] *= a[e];
                s1 += tt[e];
                s2 += tt[e] * zz[e];
            }
        }
        if constexpr (kAhead > 0) fetch(ahead, set);
        s1 = wave_sum(s1);
        s2 = wave_sum(s2);
        if (W > 1) {   // two slots in turn: one barrier per row
            if (lane == 0) {
                s_part[turn][0][wave] = s1;
                s_part[turn][1][wave] = s2;
            }
            __syncthreads();
            s1 = s2 = 0.f;
            for (int k = 0; k < W; ++k) {
                s1 += s_part[turn][0][g * W + k];
                s2 += s_part[turn][1][g * W + k];
            }
            turn ^= 1;
        }
        s1 /= (float)N;
        s2 /= (float)N;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            if (!on || column(v) >= N) continue;
            float(&zz)[8] = z[kAhead ? v : 0];
            float(&tt)[8] = t[kAhead ? v : 0];
            if constexpr (!kAhead) {
                xr[0][v].load(X, row * N + column(v));
                dr[0][v].load(dY, row * N + column(v));
                split(v, zz, tt);
                float a[8];
                ga[v].get(a);
#pragma unroll
                for (int e = 0; e < 8; ++e) tt[e] *= a[e];
            }
            float d[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) d[e] = rstd * (tt[e] - s1 - zz[e] * s2);
            ln_store<kF32>(dX, row * N + column(v), d);
        }
    };
    int64_t base = (int64_t)blockIdx.x * G;
    if constexpr (kAhead > 0) {
#pragma unroll
        for (int k = 0; k < kAhead; ++k) fetch(base + g + k * step, k);
        for (; base < M; base += kAhead * step) {
#pragma unroll
            for (int k = 0; k < kAhead; ++k)
                if (base + k * step < M)   // the same for the whole workgroup
                    work(base + g + k * step, k, base + g + (k + kAhead) * step);
        }
    } else {
        for (; base < M; base += step) {
            mr[0] = base + g < M ? mean_in[base + g] : 0.f;
            rr[0] = base + g < M ? rstd_in[base + g] : 0.f;
            work(base + g, 0, 0);
        }
    }
    float* out = part + (int64_t)blockIdx.x * 2 * N;
    if (G == 1) {
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (column(v) < N) {
                ln_store<true>(out, column(v), sg[v]);
                ln_store<true>(out, N + column(v), sb[v]);
            }
        return;
    }
    const int held = V * W * kLnCols;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        ln_store<true>(s_col, (g * 2) * held + column(v), sg[v]);
        ln_store<true>(s_col, (g * 2 + 1) * held + column(v), sb[v]);
    }
    __syncthreads();
    for (int k = threadIdx.x; k < 2 * N; k += blockDim.x) {
        const int h = k >= N, c = k - h * N;
        float s = 0.f;
        for (int q = 0; q < G; ++q) s += s_col[(q * 2 + h) * held + c];
        out[k] = s;
    }
}

// dgamma and dbeta from the workgroups' partial rows, in a fixed order: 16
// threads per column add every 16th partial, then one adds the 16 sums.
__global__ __launch_bounds__(1024) void ln_finish_kernel(const float* __restrict__ part, int rows,
                                                         int N, float* __restrict__ dgamma,
                                                         float* __restrict__ dbeta) {
    __shared__ float s[16][64 + 1];
    const int c = threadIdx.x & 63, k = threadIdx.x >> 6;
    const int64_t col = (int64_t)blockIdx.x * 64 + c;   // of 2 N
    float v = 0.f;
    if (col < 2 * N) {
#pragma unroll 8
        for (int r = k; r < rows; r += 16) v += part[(int64_t)r * 2 * N + col];
    }
    s[k][c] = v;
    __syncthreads();
    if (k || col >= 2 * N) return;
    float t = 0.f;
#pragma unroll
    for (int q = 0; q < 16; ++q) t += s[q][c];
    if (col < N) dgamma[col] = t;
    else dbeta[col - N] = t;
}

int64_t ln_backward_blocks(int64_t M, int64_t N) {
    const LnShape s = ln_shape(N, kLnThreads);
    const int64_t need = (M + s.G - 1) / s.G;
    // Two turns: as many workgroups as take two each, for fewer partial rows and no
    // workgroup that is done after one.  Whole calls, unbalanced -> balanced, bf16: 300 x 16384
    // 21.4 -> 18.6 us, 600 x 4096 13.0 -> 12.3, 1013 x 2056 11.8 -> 11.6, 384 x 8192 14.1 -> 14.6,
    // 8000 x 512 11.8 -> 12.6; fp32: 31.7 -> 23.8, 14.6 -> 14.0, 13.0 -> 13.1, 16.5 -> 16.9, 13.2 ->
    // 14.8.  With more turns the loads of all CUs count (5000 x 2048 fp32 26.5, balanced 28.3).
    if (need > kLnBackwardBlocks && need <= 2 * kLnBackwardBlocks) return (need + 1) / 2;
    return need < kLnBackwardBlocks ? need : kLnBackwardBlocks;
}

}  // namespace

size_t layernorm_partial_floats(int64_t M, int64_t N) {
    return (size_t)ln_backward_blocks(M, N) * 2 * N;
}

namespace {
template <bool kF32, int kThreads>
void start_forward(const LnShape& s, dim3 grid, hipStream_t stream, const void* X, const void* gamma,
                   const void* beta, void* Y, float* mean, float* rstd, int64_t M, int N, float eps) {
    const dim3 block(64 * s.W * s.G);
    if (s.V == 1)
        hipLaunchKernelGGL((ln_forward_kernel<kF32, 1, kThreads>), grid, block, 0, stream, X, gamma,
                           beta, Y, mean, rstd, M, N, s.W, s.G, eps);
    else if (s.V == 2)
        hipLaunchKernelGGL((ln_forward_kernel<kF32, 2, kThreads>), grid, block, 0, stream, X, gamma,
                           beta, Y, mean, rstd, M, N, s.W, s.G, eps);
    else if constexpr (kThreads < kLnThreads)
        hipLaunchKernelGGL((ln_forward_kernel<kF32, 4, kThreads>), grid, block, 0, stream, X, gamma,
                           beta, Y, mean, rstd, M, N, s.W, s.G, eps);
}
}  // namespace

hipError_t launch_layernorm_forward(const void* X, const void* gamma, const void* beta, void* Y,
                                    float* mean, float* rstd, int64_t M, int64_t N, bool f32,
                                    float eps, hipStream_t stream) {
    // Many rows: workgroups of four waves (eight past N = 8192), several per CU, each with
    // gamma and beta kept for all its rows (8192 x 8192 bf16: 72 us with sixteen waves a
    // row, 52 with four).  Few rows: up to sixteen waves, one step a lane as far as they
    // reach (16 x 4096: one round trip to memory).
    const bool many = M >= 1024;
    const int threads = !many ? kLnThreads : N <= 16 * kLnCols ? 256 : 512;
    const LnShape s = ln_shape(N, threads);
    const int64_t need = (M + s.G - 1) / s.G, most = many ? kLnForwardBlocks : 1 << 20;
    const dim3 grid((unsigned)(need < most ? need : most));
    auto go = [&](auto f, auto t) {
        start_forward<f.value, t.value>(s, grid, stream, X, gamma, beta, Y, mean, rstd, M, (int)N, eps);
    };
    auto with = [&](auto f) {
        if (threads == 256) go(f, std::integral_constant<int, 256>());
        else if (threads == 512) go(f, std::integral_constant<int, 512>());
        else go(f, std::integral_constant<int, kLnThreads>());
    };
    if (f32) with(std::true_type());
    else with(std::false_type());
    return hipGetLastError();
}

hipError_t launch_layernorm_backward(const void* X, const void* dY, const void* gamma,
                                     const float* mean, const float* rstd, void* dX, float* dgamma,
                                     float* dbeta, float* part, int64_t M, int64_t N, bool f32,
                                     hipStream_t stream) {
    const LnShape s = ln_shape(N, kLnThreads);
    const int64_t blocks = ln_backward_blocks(M, N);
    const dim3 grid((unsigned)blocks), block(64 * s.W * s.G);
    const size_t lds = s.G > 1 ? sizeof(float) * s.G * 2 * s.V * s.W * kLnCols : 0;
#define LN_BWD(F, V)                                                                             \
    do {                                                                                         \
        static std::atomic<bool> lds_set[kMaxDevices] = {};                                      \
        hipError_t e = set_dynamic_lds(reinterpret_cast<const void*>(ln_backward_kernel<F, V>),  \
                                       kLnThreads * 8 * 2 * (int)sizeof(float), lds_set);        \
        if (e != hipSuccess) return e;                                                           \
        hipLaunchKernelGGL((ln_backward_kernel<F, V>), grid, block, lds, stream, X, dY, gamma,   \
                           mean, rstd, dX, part, M, (int)N, s.W, s.G);                           \
    } while (0)
    if (f32) {
        if (s.V == 1) LN_BWD(true, 1);
        else LN_BWD(true, 2);
    } else {
        if (s.V == 1) LN_BWD(false, 1);
        else LN_BWD(false, 2);
    }
#undef LN_BWD
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(ln_finish_kernel, dim3((unsigned)((2 * N + 63) / 64)), dim3(1024), 0, stream,
                       part, (int)blocks, (int)N, dgamma, dbeta);
    return hipGetLastError();
}

}  // namespace ffn
