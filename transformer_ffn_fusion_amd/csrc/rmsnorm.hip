// rmsnorm.hip -- root-mean-square norm over the last dimension with the
// residual's addition in front, its gradients, and its output in 8 bits with
// scales; bf16 or fp32 data, fp32 statistics and sums.
//
//   forward:   s = x + r (in fp32, rounded to the data's type; x alone without r)
//              rstd = 1 / sqrt(sum_j s_j^2 / N + eps),  y_j = s_j rstd gamma_j
//   8 bits:    per row and group of 128 columns (or the whole row), from the
//              unrounded y: scale = max(max |y|, 2^-100) / 448, q_j = e4m3(y_j / scale)
//              (of bf16 data exactly that code)
//   backward:  z_j = s_j rstd,  t_j = dy_j gamma_j
//              dx_j = rstd (t_j - z_j sum (t z) / N) + ds_j
//              dgamma_j = sum_rows dy_j z_j
//
// Bound: HBM bytes.  A row stays in the registers of W waves between its one read
// and its one write, eight consecutive columns per lane and step; workgroups walk
// many rows with the next rows' loads in flight.  A group of 128 columns is one
// 16-lane row of a wave, so its largest magnitude needs neither LDS nor a barrier.
// Measured, bf16 with a residual: 8192 x 8192 forward 98 us, backward 105 us (537 MB each,
// 5.1 to 5.5 TB/s, the rate of a large copy); 4096 x 4096 into 8 bits 25.4 us (117 MB).
// Stores that pass the caches by (non-temporal) make a single call faster (8 bits 20 us,
// forward of 4096 x 4096 27 -> 22 us) and the call that reads the rows slower by more: a
// chain of norm, dispatch and combine of 16384 x 4096 takes 374 us with them, 362 without.
#include <type_traits>

#include "ffn_device.h"
#include "ffn_internal.h"
#include "rows.h"
#include "sublayer.h"

namespace ffn {

namespace {

constexpr int kRmsThreads = 1024;          // largest workgroup
constexpr float kE4m3Max = 448.0f;
constexpr float kScaleFloor = 0x1p-100f;   // of a group's largest magnitude: y / scale stays finite
// Codes of bf16 data are those of the exact quotient 448 w / max |w|, ties to the even one.  With
// products of 8-bit factors the quotient is often the halfway point between two codes (6664 of
// 4096 x 4096 values in groups of 128), and the last bit of fp32 would pick one (the odd one 1592
// times).  Let w = a 2^i, max |w| = b 2^j with integers a, b <= 255^2, and t = c 2^k a halfway
// point, c odd below 32, 2^n <= t < 2^(n+1).  A quotient that is not t is off by at least
// 2^n / (16 b), which is 8.06 steps of fp32 at t.  So 448 becomes 448 + 2^-14: that moves a quotient
// up by 1.14 to 2.22 steps, while division and product move it by 1.47 at most.  One that is t
// comes out 0 to 3 steps above it and loses those with its last two bits; one above t stays at
// least 4 above, one below stays below.
constexpr float kTieUp = kE4m3Max + 0x1p-14f;

// Largest value over each row of 16 lanes, in every lane (rotations within the row).
template <int kCtrl>
__device__ __forceinline__ float dpp_max(float v) {
    return fmaxf(v, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), kCtrl, 0xf, 0xf, false)));
}
__device__ __forceinline__ float row16_max(float v) {
    v = dpp_max<0x121>(v);   // row_ror:1
    v = dpp_max<0x122>(v);   // row_ror:2
    v = dpp_max<0x124>(v);   // row_ror:4
    return dpp_max<0x128>(v);   // row_ror:8
}

// Eight floats as e4m3 codes (round to nearest even in the conversion).
__device__ __forceinline__ uint2 pack_e4m3x8(const float (&v)[8]) {
    uint2 o;
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(v[0], v[1], 0, false);
    o.x = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(v[2], v[3], w, true);
    w = __builtin_amdgcn_cvt_pk_fp8_f32(v[4], v[5], 0, false);
    o.y = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(v[6], v[7], w, true);
    return o;
}

struct RmsArgs {
    const void *X, *R, *gamma;
    void *S, *Y;          // Y: the data's type, or e4m3 codes
    float *scale, *rstd;
    int64_t M;
    int N, W, G;
    int groups;           // scales per row (8-bit output)
    bool whole_row;       // one scale per row
    float eps;
};

// Row group g of a workgroup = W waves; a workgroup takes G rows at once and walks on
// by the grid.  Waves past the last whole row group (W does not divide the workgroup)
// do not exist: the workgroup has W G waves.
template <bool kF32, bool kQ8, int V, int kThreads>
__global__ __launch_bounds__(kThreads, V == 4 && kThreads == 512 ? 4 : 1) void rms_forward_kernel(RmsArgs a) {
    __shared__ float s_part[2][2][kThreads / 64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int W = a.W, N = a.N;
    const int g = wave / W, w = wave % W;
    const int64_t step = (int64_t)gridDim.x * a.G;
    const bool add = a.R != nullptr;
    auto column = [&](int v) { return ((v * W + w) * 64 + lane) * 8; };
    Ln8<kF32> ga[V], nx[V], nr[V];
    auto fetch = [&](int64_t row) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            nx[v].zero();
            nr[v].zero();
            if (row < a.M && column(v) < N) {
                nx[v].load(a.X, row * N + column(v));
                if (add) nr[v].load(a.R, row * N + column(v));
            }
        }
    };
    int64_t base = (int64_t)blockIdx.x * a.G;
    fetch(base + g);
#pragma unroll
    for (int v = 0; v < V; ++v) {
        ga[v].zero();
        if (column(v) < N) ga[v].load(a.gamma, column(v));
    }
    int turn = 0;
    for (; base < a.M; base += step) {
        const int64_t row = base + g;
        const bool on = row < a.M;
        float x[V][8];
        float q = 0.f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            nx[v].get(x[v]);
            if (add) {
                float r[8];
                nr[v].get(r);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    x[v][e] += r[e];
                    // the sum as it is kept is what is normed (and what the backward reads)
                    if constexpr (!kF32) x[v][e] = (float)(__bf16)x[v][e];
                }
                if (on && column(v) < N) ln_store<kF32>(a.S, row * N + column(v), x[v]);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) q += x[v][e] * x[v][e];
        }
        if (base + step < a.M) fetch(row + step);
        // two slots in turn: a row's sums are read after its barrier, and written again
        // two rows on, after the next row's
        auto over_row = [&](float v, int slot, auto join) {
            if (W == 1) return v;
            if (lane == 0) s_part[turn][slot][wave] = v;
            __syncthreads();
            float s = s_part[turn][slot][g * W];
            for (int k = 1; k < W; ++k) s = join(s, s_part[turn][slot][g * W + k]);
            return s;
        };
        q = over_row(wave_sum(q), 0, [](float b, float c) { return b + c; });
        const float rstd = 1.0f / sqrtf(q / (float)N + a.eps);
        if (on && a.rstd && w == 0 && lane == 0) a.rstd[row] = rstd;
        if constexpr (!kQ8) {
#pragma unroll
            for (int v = 0; v < V; ++v) {
                if (!on || column(v) >= N) continue;
                float b[8], y[8];
                ga[v].get(b);
#pragma unroll
                for (int e = 0; e < 8; ++e) y[e] = x[v][e] * rstd * b[e];
                ln_store<kF32>(a.Y, row * N + column(v), y);
            }
        } else {
            // rstd = p m, p a power of two: s p is exact, and y = w m with w = (s p) gamma, which of
            // bf16 data is exact too.  y / scale = 448 w / max |w| needs no m, so codes do not hang
            // on rstd's rounding.  (A NaN stays one.)
            const uint32_t bits = __float_as_uint(rstd);
            const float p = rstd != rstd ? rstd : __uint_as_float(bits & 0x7f800000u);
            const float m = __uint_as_float((bits & 0x007fffffu) | 0x3f800000u);
            float top[V];
#pragma unroll
            for (int v = 0; v < V; ++v) {
                float b[8];
                ga[v].get(b);
                top[v] = 0.f;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    // (columns past N hold zeros; 0 * p is 0, since p is finite but in rows of NaN)
                    x[v][e] = x[v][e] * p * b[e];
                    top[v] = fmaxf(top[v], fabsf(x[v][e]));
                }
                top[v] = row16_max(top[v]);
            }
            if (a.whole_row) {
                float all = 0.f;
#pragma unroll
                for (int v = 0; v < V; ++v) all = fmaxf(all, top[v]);
                all = fmaxf(all, __shfl_xor(all, 16));
                all = fmaxf(all, __shfl_xor(all, 32));
                all = over_row(all, 1, [](float b, float c) { return fmaxf(b, c); });
#pragma unroll
                for (int v = 0; v < V; ++v) top[v] = all;
            }
#pragma unroll
            for (int v = 0; v < V; ++v) {
                if (!on || column(v) >= N) continue;
                const float y = top[v] * m;
                const float scale = fmaxf(y, kScaleFloor) / kE4m3Max;
                const float inv = y >= kScaleFloor ? (kF32 ? kE4m3Max : kTieUp) / top[v] : m * (kE4m3Max / kScaleFloor);
                // |w| inv is at most 448 (1 + 2^-22), which rounds to 448
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    x[v][e] *= inv;
                    if constexpr (!kF32) x[v][e] = __uint_as_float(__float_as_uint(x[v][e]) & ~3u);
                }
                *reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.Y) + row * N + column(v)) = pack_e4m3x8(x[v]);
                if (a.whole_row) {
                    if (column(v) == 0) a.scale[row] = scale;
                } else if ((lane & 15) == 0) {
                    a.scale[row * a.groups + column(v) / 128] = scale;
                }
            }
        }
        turn ^= 1;
    }
}

// A workgroup walks rows blockIdx.x * G + g, + gridDim.x * G, ...; a lane keeps its
// columns' dgamma sums in registers over all of them: one partial row per workgroup
// instead of a second pass over s and dy.  part: [workgroup][N].  The loads run kAhead
// rows ahead; two steps a lane of fp32 (N > 8192) leave no registers for that, and of bf16 four
// registers too few (20 bytes a lane are spilled; 4096 x 12288 with dS 82 us, 4096 x 16384 110: 4.9 TB/s).
template <bool kF32, int V>
__global__ __launch_bounds__(kRmsThreads) void rms_backward_kernel(
    const void* S, const void* dY, const void* dS, const void* __restrict__ gamma,
    const float* __restrict__ rstd_in, void* dX, float* __restrict__ part, int64_t M, int N, int W, int G) {
    constexpr int kAhead = V == 1 ? (kF32 ? 2 : 3) : kF32 ? 0 : 1;
    constexpr int kSets = kAhead ? kAhead : 1;
    __shared__ float s_part[2][kRmsThreads / 64];
    extern __shared__ float s_col[];   // [G][columns held], used once at the end (G > 1)
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int g = wave / W, w = wave % W;
    const bool add = dS != nullptr;
    auto column = [&](int v) { return ((v * W + w) * 64 + lane) * 8; };
    Ln8<kF32> ga[V];
    float sg[V][8];
#pragma unroll
    for (int v = 0; v < V; ++v) {
#pragma unroll
        for (int e = 0; e < 8; ++e) sg[v][e] = 0.f;
        ga[v].zero();
        if (column(v) < N) ga[v].load(gamma, column(v));
    }
    const int64_t step = (int64_t)gridDim.x * G;
    Ln8<kF32> xr[kSets][V], dr[kSets][V], er[kSets][V];
    float rr[kSets];
    auto fetch = [&](int64_t row, int set) {
        const bool on = row < M;
        rr[set] = on ? rstd_in[row] : 0.f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            xr[set][v].zero();
            dr[set][v].zero();
            er[set][v].zero();
            if (on && column(v) < N) {
                xr[set][v].load(S, row * N + column(v));
                dr[set][v].load(dY, row * N + column(v));
                if (add) er[set][v].load(dS, row * N + column(v));
            }
        }
    };
    int turn = 0;
    // one row's work: its loads lie in set `set`; `ahead` is the row to load next into it
    auto work = [&](int64_t row, int set, int64_t ahead) {
        const float rstd = rr[set];
        float z[V][8], t[V][8];
        Ln8<kF32> er_now[V];
        float s2 = 0.f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            xr[set][v].get(z[v]);
            dr[set][v].get(t[v]);
            er_now[v] = er[set][v];
            float b[8];
            ga[v].get(b);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                // (columns past N and rows past M have s = dy = 0)
                z[v][e] *= rstd;
                sg[v][e] += t[v][e] * z[v][e];
                t[v][e] *= b[e];
                s2 += t[v][e] * z[v][e];
            }
        }
        if constexpr (kAhead > 0) fetch(ahead, set);
        s2 = wave_sum(s2);
        if (W > 1) {   // two slots in turn: one barrier per row
            if (lane == 0) s_part[turn][wave] = s2;
            __syncthreads();
            s2 = 0.f;
            for (int k = 0; k < W; ++k) s2 += s_part[turn][g * W + k];
            turn ^= 1;
        }
        s2 /= (float)N;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            if (row >= M || column(v) >= N) continue;
            float d[8], b[8];
            er_now[v].get(b);
#pragma unroll
            for (int e = 0; e < 8; ++e) d[e] = rstd * (t[v][e] - z[v][e] * s2) + b[e];
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
            fetch(base + g, 0);
            work(base + g, 0, 0);
        }
    }
    float* out = part + (int64_t)blockIdx.x * N;
    if (G == 1) {
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (column(v) < N) ln_store<true>(out, column(v), sg[v]);
        return;
    }
    const int held = V * W * kLnCols;
#pragma unroll
    for (int v = 0; v < V; ++v) ln_store<true>(s_col, g * held + column(v), sg[v]);
    __syncthreads();
    for (int c = threadIdx.x; c < N; c += blockDim.x) {
        float s = 0.f;
        for (int q = 0; q < G; ++q) s += s_col[q * held + c];
        out[c] = s;
    }
}

// dgamma from the workgroups' partial rows, in a fixed order: 32 threads per column add
// every 32nd partial, whose eight loads are under way at once however many there are, then one
// adds the 32 sums (call of 1000 x 256 bf16 5.7 us; with 16 threads per column 6.05, with 64
// and half the line of a load 5.95).
__global__ __launch_bounds__(1024) void rms_finish_kernel(const float* __restrict__ part, int rows,
                                                          int N, float* __restrict__ dgamma) {
    constexpr int kSlices = 32, kEach = kLnBackwardBlocks / kSlices;
    __shared__ float s[kSlices][32 + 1];
    const int c = threadIdx.x & 31, k = threadIdx.x >> 5;
    const int col = blockIdx.x * 32 + c;
    float v = 0.f;
    if (col < N) {
        float x[kEach];
#pragma unroll
        for (int u = 0; u < kEach; ++u) {
            const int r = k + u * kSlices;
            x[u] = part[(int64_t)(r < rows ? r : rows - 1) * N + col];
        }
#pragma unroll
        for (int u = 0; u < kEach; ++u) v += k + u * kSlices < rows ? x[u] : 0.f;
    }
    s[k][c] = v;
    __syncthreads();
    if (k || col >= N) return;
    float t = 0.f;
#pragma unroll
    for (int q = 0; q < kSlices; ++q) t += s[q][c];
    dgamma[col] = t;
}

// Rows at once.  Two turns and more, so that loads run behind sums: half of a workgroup's
// rows at most (1000 x 256 bf16 7.3 us with four at once, one turn, 6.0 with two).  Eight waves:
// a barrier holds up fewer of them and the columns' sums are joined from fewer rows (2000 x 4096
// bf16: one row 16.3 us, two 18.9; 8000 x 1024: four 16.7, eight 18.2); sixteen rows where a wave
// holds one (8000 x 256: 8.7 us, four 10.5).
LnShape rms_backward_shape(int64_t M, int64_t N) {
    LnShape s = ln_shape(N, kRmsThreads);
    if (s.W > 1) s.G = s.W < 8 ? 8 / s.W : 1;
    const int64_t half = (M + kLnBackwardBlocks - 1) / kLnBackwardBlocks / 2;
    if (half < s.G) s.G = half > 0 ? (int)half : 1;
    return s;
}

int64_t rms_backward_blocks(int64_t M, int64_t N) {
    const LnShape s = rms_backward_shape(M, N);
    const int64_t need = (M + s.G - 1) / s.G;
    return need < kLnBackwardBlocks ? need : kLnBackwardBlocks;
}

// Largest workgroup of the forward.  Few rows: one to a workgroup, of up to sixteen waves, one step
// a lane as far as they reach: one round trip (16 x 4096 bf16: 2.9 us; two to a workgroup 3.35;
// 520 x 4096: 5.6, by the shapes of many rows 5.0).  Many rows of fp32: as few steps a lane
// (3906 x 8192 with a residual: 96 us, with four waves of four steps 100; 5494 x 5824: 97.5, 105).
// Of bf16: four waves, several workgroups per CU (7812 x 8192 into 8 bits: 42 us, with sixteen waves
// 50).  Past 8192 columns two steps a lane, while two workgroups of them fit a CU (5208 x 12288 into
// 8 bits: 45 us, with eight waves of four steps 69); past 12288 one would be alone, and bf16 takes
// four steps in eight waves, held to 128 registers (3906 x 16384: 49 us, with sixteen waves 54;
// into 8 bits 54, 56: there 8 registers are spilled, 36 bytes a lane).
constexpr int64_t kManyRows = 256;
int forward_threads(int64_t M, int64_t N, bool f32) {
    if (M < kManyRows) return kRmsThreads;
    if (f32) return N <= 4 * kLnCols ? 256 : N <= 8 * kLnCols ? 512 : kRmsThreads;
    return N <= 16 * kLnCols ? 256 : N <= 24 * kLnCols ? kRmsThreads : 512;
}

// The steps a lane that forward_threads and ln_shape give: one or two of sixteen waves; of bf16 also
// up to four of four waves and four of eight; of fp32 one of four or eight.
template <bool kF32, bool kQ8, int kThreads>
hipError_t start_forward(const LnShape& s, dim3 grid, hipStream_t stream, const RmsArgs& a) {
    constexpr bool kOne = kF32 || kThreads != 512;
    constexpr bool kTwo = kThreads == kRmsThreads || (!kF32 && kThreads == 256);
    constexpr bool kFour = !kF32 && kThreads < kRmsThreads;
    auto go = [&](auto v) {
        hipLaunchKernelGGL((rms_forward_kernel<kF32, kQ8, v.value, kThreads>), grid, dim3(64 * s.W * s.G), 0, stream, a);
        return hipGetLastError();
    };
    if constexpr (kOne)
        if (s.V == 1) return go(std::integral_constant<int, 1>());
    if constexpr (kTwo)
        if (s.V == 2) return go(std::integral_constant<int, 2>());
    if constexpr (kFour)
        if (s.V == 4) return go(std::integral_constant<int, 4>());
    return hipErrorInvalidValue;    // no rule gives this shape
}

}  // namespace

size_t rmsnorm_partial_floats(int64_t M, int64_t N) { return (size_t)rms_backward_blocks(M, N) * N; }

hipError_t launch_rmsnorm_forward(const RmsForwardIO& io, hipStream_t stream) {
    const int64_t M = io.M, N = io.N;
    const int threads = forward_threads(M, N, io.f32);
    LnShape s = ln_shape(N, threads);
    if (M < kManyRows) s.G = 1;
    const int64_t need = (M + s.G - 1) / s.G, most = M >= kManyRows ? kLnForwardBlocks : 1 << 20;
    const dim3 grid((unsigned)(need < most ? need : most));
    RmsArgs a;
    a.X = io.X;
    a.R = io.R;
    a.gamma = io.gamma;
    a.S = io.S;
    a.Y = io.Y;
    a.scale = io.scale;
    a.rstd = io.rstd;
    a.M = M;
    a.N = (int)N;
    a.W = s.W;
    a.G = s.G;
    a.whole_row = io.group == 0;
    a.groups = io.group ? (int)((N + 127) / 128) : 1;
    a.eps = io.eps;
    auto go = [&](auto f, auto q, auto t) { return start_forward<f.value, q.value, t.value>(s, grid, stream, a); };
    auto with = [&](auto f, auto q) {
        if (threads == 256) return go(f, q, std::integral_constant<int, 256>());
        if (threads == 512) return go(f, q, std::integral_constant<int, 512>());
        return go(f, q, std::integral_constant<int, kRmsThreads>());
    };
    if (io.q8) return io.f32 ? with(std::true_type(), std::true_type()) : with(std::false_type(), std::true_type());
    return io.f32 ? with(std::true_type(), std::false_type()) : with(std::false_type(), std::false_type());
}

hipError_t launch_rmsnorm_backward(const void* S, const void* dY, const void* dS, const void* gamma,
                                   const float* rstd, void* dX, float* dgamma, float* part, int64_t M,
                                   int64_t N, bool f32, hipStream_t stream) {
    const LnShape s = rms_backward_shape(M, N);
    const int64_t blocks = rms_backward_blocks(M, N);
    const dim3 grid((unsigned)blocks), block(64 * s.W * s.G);
    // at most 16 waves x 512 columns of sums: 32 KiB
    const size_t lds = s.G > 1 ? sizeof(float) * s.G * s.V * s.W * kLnCols : 0;
    auto go = [&](auto f, auto v) {
        hipLaunchKernelGGL((rms_backward_kernel<f.value, v.value>), grid, block, lds, stream, S, dY, dS,
                           gamma, rstd, dX, part, M, (int)N, s.W, s.G);
    };
    using One = std::integral_constant<int, 1>;
    using Two = std::integral_constant<int, 2>;
    if (f32) {
        if (s.V == 1) go(std::true_type(), One());
        else go(std::true_type(), Two());
    } else {
        if (s.V == 1) go(std::false_type(), One());
        else go(std::false_type(), Two());
    }
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(rms_finish_kernel, dim3((unsigned)((N + 31) / 32)), dim3(1024), 0, stream, part,
                       (int)blocks, (int)N, dgamma);
    return hipGetLastError();
}

}  // namespace ffn
