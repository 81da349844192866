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
// waves of a workgroup, eight consecutive columns per lane and step (one
// 16-byte load of bf16, two of fp32), so it is read once: the variance is the
// centred sum over the held values, with no cancellation.
#include "ffn_device.h"
#include "ffn_internal.h"

namespace ffn {

namespace {

constexpr int kLnThreads = 1024;   // largest workgroup
constexpr int kLnCols = 512;       // columns a wave holds per step: 64 lanes x 8

// Eight consecutive values as floats, and back.
template <bool kF32>
__device__ __forceinline__ void ln_load(const void* p, int64_t at, float (&v)[8]) {
    if constexpr (kF32) {
        const float4 a = *reinterpret_cast<const float4*>(static_cast<const float*>(p) + at);
        const float4 b = *reinterpret_cast<const float4*>(static_cast<const float*>(p) + at + 4);
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    } else {
        const uint4 a = ld16(static_cast<const uint16_t*>(p) + at);
        v[0] = bf16_lo(a.x); v[1] = bf16_hi(a.x); v[2] = bf16_lo(a.y); v[3] = bf16_hi(a.y);
        v[4] = bf16_lo(a.z); v[5] = bf16_hi(a.z); v[6] = bf16_lo(a.w); v[7] = bf16_hi(a.w);
    }
}
template <bool kF32>
__device__ __forceinline__ void ln_store(void* p, int64_t at, const float (&v)[8]) {
    if constexpr (kF32) {
        float* q = static_cast<float*>(p) + at;
        *reinterpret_cast<float4*>(q) = make_float4(v[0], v[1], v[2], v[3]);
        *reinterpret_cast<float4*>(q + 4) = make_float4(v[4], v[5], v[6], v[7]);
    } else {
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + at) =
            make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                       pack_bf16x2(v[6], v[7]));
    }
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int d = 32; d; d >>= 1) v += __shfl_xor(v, d);
    return v;
}

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
// walks on by the grid (more rows than a launch has workgroups).
template <bool kF32, int V>
__global__ __launch_bounds__(kLnThreads) void ln_forward_kernel(
    const void* X, const void* __restrict__ gamma, const void* __restrict__ beta, void* Y,
    float* __restrict__ mean_out, float* __restrict__ rstd_out, int64_t M, int N, int W, int G,
    float eps) {
    __shared__ float s_part[2][kLnThreads / 64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int g = wave / W, w = wave % W;
    for (int64_t base = (int64_t)blockIdx.x * G; base < M; base += (int64_t)gridDim.x * G) {
        const int64_t row = base + g;
        const bool on = row < M;
        float x[V][8];
        float s = 0.f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = ((v * W + w) * 64 + lane) * 8;
            if (on && c < N) {
                ln_load<kF32>(X, row * N + c, x[v]);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) x[v][e] = 0.f;
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) s += x[v][e];
        }
        const float mean = row_sum(s, s_part[0], wave, g * W, W) / (float)N;
        float q = 0.f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = ((v * W + w) * 64 + lane) * 8;
            if (c < N) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    x[v][e] -= mean;
                    q += x[v][e] * x[v][e];
                }
            }
        }
        // (a row's first sum is read between this barrier and the one before: the
        // next row's waves write it again only after passing this one)
        const float var = row_sum(q, s_part[1], wave, g * W, W) / (float)N;
        const float rstd = 1.0f / sqrtf(var + eps);
        if (!on) continue;
        if (w == 0 && lane == 0) {
            if (mean_out) mean_out[row] = mean;
            if (rstd_out) rstd_out[row] = rstd;
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = ((v * W + w) * 64 + lane) * 8;
            if (c >= N) continue;
            float ga[8], be[8], y[8];
            ln_load<kF32>(gamma, c, ga);
            ln_load<kF32>(beta, c, be);
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = x[v][e] * rstd * ga[e] + be[e];
            ln_store<kF32>(Y, row * N + c, y);
        }
    }
}

// A workgroup walks rows blockIdx.x * G + g, + gridDim.x * G, ...; a lane keeps
// its columns' dgamma and dbeta sums in registers over all of them, so the
// column sums cost one partial row per workgroup instead of a second pass over x
// and dy.  part: [workgroup][2][N], dgamma first.
template <bool kF32, int V>
__global__ __launch_bounds__(kLnThreads) void ln_backward_kernel(
    const void* X, const void* dY, const void* __restrict__ gamma,
    const float* __restrict__ mean_in, const float* __restrict__ rstd_in, void* dX,
    float* __restrict__ part, int64_t M, int N, int W, int G) {
    __shared__ float s_part[2][2][kLnThreads / 64];
    extern __shared__ float s_col[];   // [G][2][columns held], used once at the end (G > 1)
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int g = wave / W, w = wave % W;
    float ga[V][8], sg[V][8], sb[V][8];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int c = ((v * W + w) * 64 + lane) * 8;
#pragma unroll
        for (int e = 0; e < 8; ++e) ga[v][e] = sg[v][e] = sb[v][e] = 0.f;
        if (c < N) ln_load<kF32>(gamma, c, ga[v]);
    }
    const int64_t step = (int64_t)gridDim.x * G;
    int turn = 0;
    for (int64_t base = (int64_t)blockIdx.x * G; base < M; base += step, turn ^= 1) {
        const int64_t row = base + g;
        const bool on = row < M;
        const float mean = on ? mean_in[row] : 0.f, rstd = on ? rstd_in[row] : 0.f;
        float z[V][8], t[V][8];
        float s1 = 0.f, s2 = 0.f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = ((v * W + w) * 64 + lane) * 8;
            if (on && c < N) {
                ln_load<kF32>(X, row * N + c, z[v]);
                ln_load<kF32>(dY, row * N + c, t[v]);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    z[v][e] = (z[v][e] - mean) * rstd;
                    sg[v][e] += t[v][e] * z[v][e];
                    sb[v][e] += t[v][e];
                    t[v][e] *= ga[v][e];
                    s1 += t[v][e];
                    s2 += t[v][e] * z[v][e];
                }
            }
        }
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
        }
        s1 /= (float)N;
        s2 /= (float)N;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = ((v * W + w) * 64 + lane) * 8;
            if (on && c < N) {
                float d[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) d[e] = rstd * (t[v][e] - s1 - z[v][e] * s2);
                ln_store<kF32>(dX, row * N + c, d);
            }
        }
    }
    float* out = part + (int64_t)blockIdx.x * 2 * N;
    if (G == 1) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = ((v * W + w) * 64 + lane) * 8;
            if (c < N) {
                ln_store<true>(out, c, sg[v]);
                ln_store<true>(out, N + c, sb[v]);
            }
        }
        return;
    }
    const int held = V * W * kLnCols;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int c = ((v * W + w) * 64 + lane) * 8;
        ln_store<true>(s_col, (g * 2) * held + c, sg[v]);
        ln_store<true>(s_col, (g * 2 + 1) * held + c, sb[v]);
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

struct LnShape {
    int V, W, G;   // steps per lane, waves per row, rows per workgroup at once
};
LnShape ln_shape(int64_t N, int max_threads) {
    const int waves = (int)((N + kLnCols - 1) / kLnCols), most = max_threads / 64;
    LnShape s;
    s.V = waves <= most ? 1 : waves <= 2 * most ? 2 : 4;
    s.W = (waves + s.V - 1) / s.V;
    s.G = most / s.W;
    return s;
}

int64_t ln_backward_blocks(int64_t M, int64_t N) {
    const LnShape s = ln_shape(N, kLnThreads);
    const int64_t need = (M + s.G - 1) / s.G;
    return need < kLnBackwardBlocks ? need : kLnBackwardBlocks;
}

}  // namespace

size_t layernorm_partial_floats(int64_t M, int64_t N) {
    return (size_t)ln_backward_blocks(M, N) * 2 * N;
}

hipError_t launch_layernorm_forward(const void* X, const void* gamma, const void* beta, void* Y,
                                    float* mean, float* rstd, int64_t M, int64_t N, bool f32,
                                    float eps, hipStream_t stream) {
    // four waves per workgroup where they hold the row: more workgroups for few rows
    const LnShape s = ln_shape(N, N <= 4 * kLnCols ? 256 : kLnThreads);
    const int64_t need = (M + s.G - 1) / s.G, most = 1 << 20;
    const dim3 grid((unsigned)(need < most ? need : most)), block(64 * s.W * s.G);
#define LN_FWD(F, V)                                                                             \
    hipLaunchKernelGGL((ln_forward_kernel<F, V>), grid, block, 0, stream, X, gamma, beta, Y,     \
                       mean, rstd, M, (int)N, s.W, s.G, eps)
    if (f32) {
        if (s.V == 1) LN_FWD(true, 1);
        else if (s.V == 2) LN_FWD(true, 2);
        else LN_FWD(true, 4);
    } else {
        if (s.V == 1) LN_FWD(false, 1);
        else if (s.V == 2) LN_FWD(false, 2);
        else LN_FWD(false, 4);
    }
#undef LN_FWD
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
        else if (s.V == 2) LN_BWD(true, 2);
        else LN_BWD(true, 4);
    } else {
        if (s.V == 1) LN_BWD(false, 1);
        else if (s.V == 2) LN_BWD(false, 2);
        else LN_BWD(false, 4);
    }
#undef LN_BWD
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(ln_finish_kernel, dim3((unsigned)((2 * N + 63) / 64)), dim3(1024), 0, stream,
                       part, (int)blocks, (int)N, dgamma, dbeta);
    return hipGetLastError();
}

}  // namespace ffn
