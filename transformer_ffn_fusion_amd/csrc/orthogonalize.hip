// orthogonalize.hip -- the orthogonalised update of a weight matrix: five (or
// `steps`) Newton-Schulz steps on its gradient or momentum G (R x C),
//
//   X = G / (||G||_F + 1e-7)
//   X <- a X + (b A + c A^2) X,  A = X X^T      (R <= C; else A = X^T X and
//   a = 3.4445, b = -4.7750, c = 2.0315          X <- a X + X (b A + c A^2))
//
// which drives every singular value of G towards 1 and keeps its singular
// vectors.  A is square in the smaller dimension m, so no transpose is ever
// formed: both forms read X as it lies.
//
// Numbers.  The products run on fp16 matrix instructions with fp32 sums.  Two
// things keep single rounded operands accurate:
//  * X is carried as a pair hi + lo of fp16 (22 bits) and the linear part of a
//    step is formed from the pair.  Rounding X itself would put noise into the
//    directions G does not have, which every step multiplies by a = 3.4; a
//    rounded operand inside (b A + c A^2) X only turns singular vectors that are
//    there already.  (Emulated, a rank-16 448 x 1024 G: 4.3e-2 off without lo,
//    1.7e-3 with, all of it the bf16 output's own rounding.)
//  * the diagonals of A and of b A + c A^2, which dominate once the singular
//    values are near 1, never pass through fp16: with A = D + E (D diagonal),
//    A^2 = E^2 + D E + E D + D^2, the products take E's entries and the epilogues
//    add the terms with D in fp32 (an orthogonal 448 x 1024 G: 3.6e-3 -> 2.3e-3).
//    They multiply hi alone, as the products do: with hi + lo there, D X and E X
//    would see two different X, and the difference is again noise in directions
//    that G does not have (a rank-1 G: 3.3e-3 instead of 1.7e-3).
// Scales keep fp16 clear of its subnormals: X is held times 64, E and the
// polynomial's off-diagonal times 1024 (singular values stay below 1.21, so
// entries stay below 80 and 1.2e4).
//
// Bound: the three products of a step, gemm16.h.
#include "ffn_device.h"
#include "ffn_internal.h"
#include "gemm16.h"

namespace ffn {

namespace {

using Large = TileCfg<256, 256, 2, 4>;
using Small = TileCfg<128, 128, 2, 2>;

constexpr float kNsA = 3.4445f, kNsB = -4.7750f, kNsC = 2.0315f;
constexpr double kNsEps = 1e-7;
constexpr float kScaleX = 64.0f, kScaleSym = 1024.0f;
constexpr int kNormBlocks = 128;   // partial sums of squares per matrix

struct OrthoArgs {
    const void* G;
    uint16_t* U;
    const uint16_t* hi;     // X's high halves that this step reads ...
    uint16_t* hi_next;      // ... and writes
    uint16_t* lo;           // X's low halves, read and written in place
    uint16_t *sym, *poly;   // off-diagonals of A and b A + c A^2, fp16, m x m
    float *diag, *scale;    // diagonals of A and of b A + c A^2
    double* norm;           // kNormBlocks partial sums per matrix
    int64_t R, C, m, n;     // m = min(R, C), n = max(R, C)
    int last;               // the last step writes U
};

__device__ __forceinline__ float f16_bits(uint32_t v) {
    return (float)__builtin_bit_cast(_Float16, (uint16_t)v);
}
__device__ __forceinline__ uint32_t bits_f16(float v) {
    return __builtin_bit_cast(uint16_t, (_Float16)v);
}
__device__ __forceinline__ void load4_f16(const uint16_t* p, float (&v)[4]) {
    const uint2 w = *reinterpret_cast<const uint2*>(p);
    v[0] = f16_bits(w.x & 0xffffu); v[1] = f16_bits(w.x >> 16);
    v[2] = f16_bits(w.y & 0xffffu); v[3] = f16_bits(w.y >> 16);
}
__device__ __forceinline__ void store4_f16(uint16_t* p, const float (&v)[4]) {
    *reinterpret_cast<uint2*>(p) = make_uint2(bits_f16(v[0]) | bits_f16(v[1]) << 16,
                                              bits_f16(v[2]) | bits_f16(v[3]) << 16);
}
// v as hi + lo
__device__ __forceinline__ void store4_pair(uint16_t* hi, uint16_t* lo, const float (&v)[4]) {
    float l[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) l[r] = v[r] - (float)(_Float16)v[r];
    store4_f16(hi, v);
    store4_f16(lo, l);
}

template <bool kF32>
__device__ __forceinline__ void load4_in(const void* p, int64_t at, float (&v)[4]) {
    if constexpr (kF32) {
        const float4 a = *reinterpret_cast<const float4*>(static_cast<const float*>(p) + at);
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    } else {
        const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p) + at);
        v[0] = bf16_lo(w.x); v[1] = bf16_hi(w.x); v[2] = bf16_lo(w.y); v[3] = bf16_hi(w.y);
    }
}

// Sums of squares in fp64: an fp32 gradient's squares leave fp32's range.
template <bool kF32>
__global__ __launch_bounds__(256) void ortho_norm_kernel(OrthoArgs g) {
    __shared__ double s[4];
    const int64_t size = g.R * g.C, base = (int64_t)blockIdx.y * size;
    double q = 0.0;
    for (int64_t k = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4; k < size; k += kNormBlocks * 1024) {
        float v[4];
        load4_in<kF32>(g.G, base + k, v);
#pragma unroll
        for (int r = 0; r < 4; ++r) q += (double)v[r] * v[r];
    }
#pragma unroll
    for (int d = 32; d; d >>= 1) q += __shfl_xor(q, d);
    if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = q;
    __syncthreads();
    if (threadIdx.x == 0) g.norm[blockIdx.y * kNormBlocks + blockIdx.x] = s[0] + s[1] + s[2] + s[3];
}

// X = 64 G / (||G|| + eps) as hi + lo.
template <bool kF32>
__global__ __launch_bounds__(256) void ortho_start_kernel(OrthoArgs g) {
    __shared__ double s[kNormBlocks];
    if (threadIdx.x < kNormBlocks) s[threadIdx.x] = g.norm[blockIdx.y * kNormBlocks + threadIdx.x];
    __syncthreads();
    double q = 0.0;
    for (int k = 0; k < kNormBlocks; ++k) q += s[k];
    const double by = (double)kScaleX / (sqrt(q) + kNsEps);
    const int64_t size = g.R * g.C, base = (int64_t)blockIdx.y * size;
    for (int64_t k = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4; k < size;
         k += (int64_t)gridDim.x * 1024) {
        float v[4];
        load4_in<kF32>(g.G, base + k, v);
#pragma unroll
        for (int r = 0; r < 4; ++r) v[r] = (float)((double)v[r] * by);
        store4_pair(g.hi_next + base + k, g.lo + base + k, v);
    }
}

// PROD_SYM: E = offdiag(A), D.  PROD_POLY: b A + c A^2.  PROD_X: the step.
enum { PROD_SYM = 0, PROD_POLY = 1, PROD_X = 2 };

template <class Cfg, int kProd, bool kTall>
__global__ __launch_bounds__(Cfg::kThreads) void ortho_kernel(OrthoArgs g) {
    constexpr bool kAS = kProd == PROD_SYM && kTall;
    constexpr bool kBS = kProd == PROD_SYM ? kTall : kProd == PROD_X && !kTall;
    extern __shared__ __attribute__((aligned(16))) char smem[];
    const int64_t m = g.m, I = kProd == PROD_X ? g.R : m, J = kProd == PROD_X ? g.C : m;
    int64_t ti, tj;
    if (!tile_place(blockIdx.x, (I + Cfg::TI - 1) / Cfg::TI, (J + Cfg::TJ - 1) / Cfg::TJ, &ti, &tj))
        return;
    const int64_t i0 = ti * Cfg::TI, j0 = tj * Cfg::TJ;
    const int64_t at_x = (int64_t)blockIdx.y * g.R * g.C, at_m = (int64_t)blockIdx.y * m * m;
    const uint16_t* hi = g.hi + at_x;
    const uint16_t* poly = g.poly + at_m;
    const uint16_t* sym = g.sym + at_m;
    float* diag = g.diag + blockIdx.y * m;
    float* scale = g.scale + blockIdx.y * m;

    TileOps op;
    op.pairs = 1;
    const uint16_t *A, *B;
    if constexpr (kProd == PROD_SYM) {
        A = B = hi; op.lda = op.ldb = g.C; op.K = g.n;
    } else if constexpr (kProd == PROD_POLY) {
        A = B = sym; op.lda = op.ldb = m; op.K = m;
    } else if constexpr (kTall) {
        A = hi; op.lda = g.C; B = poly; op.ldb = m; op.K = m;   // X (poly), poly symmetric
    } else {
        A = poly; op.lda = m; B = hi; op.ldb = g.C; op.K = m;   // (poly) X
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        op.a[0][h] = op.a[1][h] = half_walk<kAS>(A, op.lda, I, op.K, i0 + h * Cfg::HI);
        op.b[0][h] = op.b[1][h] = half_walk<kBS>(B, op.ldb, J, op.K, j0 + h * Cfg::HJ);
    }
    TileAcc<Cfg> acc;
    tile_clear<Cfg>(acc);
    tile_product<Cfg, kAS, kBS, true>(smem, op, acc);

    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
    for (int p = 0; p < 2; ++p)
#pragma unroll
        for (int x = 0; x < Cfg::FI; ++x) {
            const int64_t i = i0 + tile_row<Cfg>(wave, p, x) + (lane & 15);
            if (i >= I) continue;
#pragma unroll
            for (int q = 0; q < 2; ++q)
#pragma unroll
                for (int y = 0; y < Cfg::FJ; ++y) {
                    const int64_t j = j0 + tile_col<Cfg>(wave, q, y) + 4 * (lane >> 4);
                    if (j >= J) continue;
                    float v[4] = {acc[p][q][x][y][0], acc[p][q][x][y][1], acc[p][q][x][y][2],
                                  acc[p][q][x][y][3]};
                    if constexpr (kProd == PROD_SYM) {
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            if (i == j + r) {
                                diag[i] = v[r] * (1.0f / (kScaleX * kScaleX));
                                v[r] = 0.f;
                            } else {
                                v[r] *= kScaleSym / (kScaleX * kScaleX);
                            }
                        }
                        store4_f16(g.sym + at_m + i * m + j, v);
                    } else if constexpr (kProd == PROD_POLY) {
                        float e[4];
                        load4_f16(sym + i * m + j, e);
                        const float di = diag[i];
                        const float4 dj = *reinterpret_cast<const float4*>(diag + j);
                        const float d[4] = {dj.x, dj.y, dj.z, dj.w};
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            const float sq = v[r] * (1.0f / (kScaleSym * kScaleSym));
                            if (i == j + r) {
                                scale[i] = kNsB * di + kNsC * (sq + di * di);
                                v[r] = 0.f;
                            } else {
                                const float off = e[r] * (1.0f / kScaleSym);
                                v[r] = kScaleSym * (kNsB * off + kNsC * (sq + (di + d[r]) * off));
                            }
                        }
                        store4_f16(g.poly + at_m + i * m + j, v);
                    } else {
                        const int64_t at = at_x + i * g.C + j;
                        float h[4], l[4], s[4];
                        load4_f16(g.hi + at, h);
                        load4_f16(g.lo + at, l);
                        if constexpr (kTall) {
                            const float4 t = *reinterpret_cast<const float4*>(scale + j);
                            s[0] = t.x; s[1] = t.y; s[2] = t.z; s[3] = t.w;
                        } else {
                            s[0] = s[1] = s[2] = s[3] = scale[i];
                        }
#pragma unroll
                        for (int r = 0; r < 4; ++r)
                            v[r] = kNsA * (h[r] + l[r]) + s[r] * h[r] + v[r] * (1.0f / kScaleSym);
                        if (g.last) {
                            *reinterpret_cast<uint2*>(g.U + at) =
                                make_uint2(pack_bf16x2(v[0] * (1.0f / kScaleX), v[1] * (1.0f / kScaleX)),
                                           pack_bf16x2(v[2] * (1.0f / kScaleX), v[3] * (1.0f / kScaleX)));
                        } else {
                            store4_pair(g.hi_next + at, g.lo + at, v);
                        }
                    }
                }
        }
}

template <class Cfg, int kProd, bool kTall>
hipError_t launch_product_cfg(const OrthoArgs& g, int64_t batch, hipStream_t stream) {
    auto kern = ortho_kernel<Cfg, kProd, kTall>;
    static std::atomic<bool> lds_set[kMaxDevices] = {};
    hipError_t e = set_dynamic_lds(reinterpret_cast<const void*>(kern), Cfg::kLds, lds_set);
    if (e != hipSuccess) return e;
    const int64_t I = kProd == PROD_X ? g.R : g.m, J = kProd == PROD_X ? g.C : g.m;
    const int64_t grid = tile_grid((I + Cfg::TI - 1) / Cfg::TI, (J + Cfg::TJ - 1) / Cfg::TJ);
    hipLaunchKernelGGL(kern, dim3((unsigned)grid, (unsigned)batch), dim3(Cfg::kThreads), Cfg::kLds,
                       stream, g);
    return hipGetLastError();
}

template <int kProd, bool kTall>
hipError_t launch_product(const OrthoArgs& g, int64_t batch, hipStream_t stream) {
    const int64_t I = kProd == PROD_X ? g.R : g.m, J = kProd == PROD_X ? g.C : g.m;
    const int64_t cus = device_cus();
    const int64_t large = batch * ((I + Large::TI - 1) / Large::TI) * ((J + Large::TJ - 1) / Large::TJ);
    const int64_t small = batch * ((I + Small::TI - 1) / Small::TI) * ((J + Small::TJ - 1) / Small::TJ);
    const double t_large = (double)((large + cus - 1) / cus);
    const double t_small = 0.65 * (double)((small + 2 * cus - 1) / (2 * cus));
    if (t_large <= t_small) return launch_product_cfg<Large, kProd, kTall>(g, batch, stream);
    return launch_product_cfg<Small, kProd, kTall>(g, batch, stream);
}

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

}  // namespace

OrthogonalizeLayout orthogonalize_layout(int64_t B, int64_t R, int64_t C) {
    OrthogonalizeLayout L;
    const int64_t m = R < C ? R : C;
    size_t off = 0;
    auto take = [&](size_t bytes) {
        const size_t at = off;
        off += up256(bytes);
        return at;
    };
    L.hi[0] = take(sizeof(uint16_t) * B * R * C);
    L.hi[1] = take(sizeof(uint16_t) * B * R * C);
    L.lo = take(sizeof(uint16_t) * B * R * C);
    L.sym = take(sizeof(uint16_t) * B * m * m);
    L.poly = take(sizeof(uint16_t) * B * m * m);
    L.diag = take(sizeof(float) * B * m);
    L.scale = take(sizeof(float) * B * m);
    L.norm = take(sizeof(double) * B * kNormBlocks);
    L.total = off;
    return L;
}

hipError_t launch_orthogonalize(const void* G, bool f32, uint16_t* U, int64_t B, int64_t R,
                                int64_t C, int steps, char* ws, hipStream_t stream) {
    const OrthogonalizeLayout L = orthogonalize_layout(B, R, C);
    OrthoArgs g;
    g.G = G;
    g.U = U;
    g.lo = reinterpret_cast<uint16_t*>(ws + L.lo);
    g.sym = reinterpret_cast<uint16_t*>(ws + L.sym);
    g.poly = reinterpret_cast<uint16_t*>(ws + L.poly);
    g.diag = reinterpret_cast<float*>(ws + L.diag);
    g.scale = reinterpret_cast<float*>(ws + L.scale);
    g.norm = reinterpret_cast<double*>(ws + L.norm);
    g.R = R;
    g.C = C;
    g.m = R < C ? R : C;
    g.n = R < C ? C : R;
    g.last = 0;
    uint16_t* hi[2] = {reinterpret_cast<uint16_t*>(ws + L.hi[0]),
                       reinterpret_cast<uint16_t*>(ws + L.hi[1])};
    g.hi = hi[1];
    g.hi_next = hi[0];
    hipError_t e;
    int64_t blocks = (R * C + 1023) / 1024;
    if (blocks > 2048) blocks = 2048;
    if (f32) {
        hipLaunchKernelGGL(ortho_norm_kernel<true>, dim3(kNormBlocks, (unsigned)B), dim3(256), 0, stream, g);
        hipLaunchKernelGGL(ortho_start_kernel<true>, dim3((unsigned)blocks, (unsigned)B), dim3(256), 0, stream, g);
    } else {
        hipLaunchKernelGGL(ortho_norm_kernel<false>, dim3(kNormBlocks, (unsigned)B), dim3(256), 0, stream, g);
        hipLaunchKernelGGL(ortho_start_kernel<false>, dim3((unsigned)blocks, (unsigned)B), dim3(256), 0, stream, g);
    }
    if ((e = hipGetLastError()) != hipSuccess) return e;
    const bool tall = R > C;
    for (int s = 0; s < steps; ++s) {
        g.hi = hi[s & 1];
        g.hi_next = hi[(s & 1) ^ 1];
        g.last = s == steps - 1;
        e = tall ? launch_product<PROD_SYM, true>(g, B, stream) : launch_product<PROD_SYM, false>(g, B, stream);
        if (e != hipSuccess) return e;
        if ((e = launch_product<PROD_POLY, false>(g, B, stream)) != hipSuccess) return e;
        e = tall ? launch_product<PROD_X, true>(g, B, stream) : launch_product<PROD_X, false>(g, B, stream);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace ffn
