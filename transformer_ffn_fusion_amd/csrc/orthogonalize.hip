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
// Scales keep fp16 clear of its subnormals.  X's singular values stay below 1.21 and
// it is held times 2^15 (entries below 4e4): the pair has its 22 bits down to entries of
// 2^-18, which the largest matrices' are in the mean.  Where ||G|| is small against
// 1e-7, X is, and it grows by a in each step: it is held times a larger power of two then,
// one that its growth cannot overflow (x_scale).  (Times 64 for all, emulated, 1024 x 1536:
// 4e-3 off at ||G|| = 1e-11, 0.3 at 1e-13.)  E and the polynomial's off-diagonal are held
// times 1024 (entries below 1.2e4).
//
// Bound: the three products of a step, gemm16.h; up to 128 x 512 one workgroup does all
// (ortho_small_kernel).
#include <cmath>

#include "ffn_device.h"
#include "ffn_internal.h"
#include "gemm16.h"

namespace ffn {

namespace {

constexpr float kNsA = 3.4445f, kNsB = -4.7750f, kNsC = 2.0315f;
constexpr double kNsEps = 1e-7;
constexpr int kScaleX = 15;         // X is held times 2^15 at least,
constexpr int kScaleSymBits = 10;   // the square matrices' off-diagonals times 2^10
constexpr float kScaleSym = 1 << kScaleSymBits;
// Partial sums of squares per matrix (3584 x 8192 fp32: 128 of them 60 us, 1024 26 us).
inline int norm_blocks(int64_t size) {
    const int64_t k = size / 8192;
    return k < 32 ? 32 : k > 1024 ? 1024 : (int)k;
}

struct OrthoArgs {
    const void* G;
    uint16_t* U;
    const uint16_t* hi;     // X's high halves that this step reads ...
    uint16_t* hi_next;      // ... and writes
    uint16_t* lo;           // X's low halves, read and written in place
    uint16_t *sym, *poly;   // off-diagonals of A and b A + c A^2, fp16, m x m
    float *diag, *scale;    // diagonals of A and of b A + c A^2
    double* norm;           // norm_blocks partial sums per matrix
    int sums;
    double growth;          // a^steps: what a small X grows by
    int* scale_x;           // X's scale, per matrix: the power of two
    float* part;            // sums of split products, and a counter per tile (tile_join)
    uint32_t* count;
    int64_t counters;
    int64_t full;           // a matrix's tiles of this product that are not split ...
    int splits;             // ... and into how many the others are
    int64_t R, C, m, n;     // m = min(R, C), n = max(R, C)
    int last;               // the last step writes U
};

__device__ __forceinline__ float f16_bits(uint32_t v) {
    return (float)__builtin_bit_cast(_Float16, (uint16_t)v);
}
__device__ __forceinline__ uint32_t bits_f16(float v) {
    return __builtin_bit_cast(uint16_t, (_Float16)v);
}
__device__ __forceinline__ void unpack8_f16(const uint4& w, float (&v)[8]) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        v[2 * r] = f16_bits(u[r] & 0xffffu);
        v[2 * r + 1] = f16_bits(u[r] >> 16);
    }
}
typedef _Float16 f16x4_t __attribute__((ext_vector_type(4)));
__device__ __forceinline__ uint2 f16x4(const float (&v)[4]) {
    return make_uint2(bits_f16(v[0]) | bits_f16(v[1]) << 16, bits_f16(v[2]) | bits_f16(v[3]) << 16);
}
__device__ __forceinline__ void f32x4(const uint2& w, float (&v)[4]) {
    v[0] = f16_bits(w.x & 0xffffu);
    v[1] = f16_bits(w.x >> 16);
    v[2] = f16_bits(w.y & 0xffffu);
    v[3] = f16_bits(w.y >> 16);
}
__device__ __forceinline__ void store8_f16(uint16_t* p, const float (&v)[8]) {
    *reinterpret_cast<uint4*>(p) =
        make_uint4(bits_f16(v[0]) | bits_f16(v[1]) << 16, bits_f16(v[2]) | bits_f16(v[3]) << 16,
                   bits_f16(v[4]) | bits_f16(v[5]) << 16, bits_f16(v[6]) | bits_f16(v[7]) << 16);
}
// v as hi + lo
__device__ __forceinline__ void store8_pair(uint16_t* hi, uint16_t* lo, const float (&v)[8]) {
    float l[8];
#pragma unroll
    for (int r = 0; r < 8; ++r) l[r] = v[r] - (float)(_Float16)v[r];
    store8_f16(hi, v);
    store8_f16(lo, l);
}
__device__ __forceinline__ void load8_f32(const float* p, float (&v)[8]) {
    const float4 a = *reinterpret_cast<const float4*>(p);
    const float4 b = *reinterpret_cast<const float4*>(p + 4);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}

template <bool kF32>
__device__ __forceinline__ void load8_in(const void* p, int64_t at, float (&v)[8]) {
    if constexpr (kF32) {
        load8_f32(static_cast<const float*>(p) + at, v);
    } else {
        const uint4 w = ld16(static_cast<const uint16_t*>(p) + at);
        v[0] = bf16_lo(w.x); v[1] = bf16_hi(w.x); v[2] = bf16_lo(w.y); v[3] = bf16_hi(w.y);
        v[4] = bf16_lo(w.z); v[5] = bf16_hi(w.z); v[6] = bf16_lo(w.w); v[7] = bf16_hi(w.w);
    }
}

// Sum over the 256 threads, the same in all of them.
__device__ __forceinline__ double workgroup_sum(double q, double (&s)[4]) {
#pragma unroll
    for (int d = 32; d; d >>= 1) q += __shfl_xor(q, d);
    if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = q;
    __syncthreads();
    return s[0] + s[1] + s[2] + s[3];
}

// Sums of squares in fp64: an fp32 gradient's squares leave fp32's range.
template <bool kF32>
__global__ __launch_bounds__(256) void ortho_norm_kernel(OrthoArgs g) {
    __shared__ double s[4];
    const int64_t size = g.R * g.C, base = (int64_t)blockIdx.y * size;
    if (blockIdx.x == 0 && blockIdx.y == 0)   // before any product of this call
        for (int64_t k = threadIdx.x; k < g.counters; k += 256) g.count[k] = 0;
    double q = 0.0;
#pragma unroll 4
    for (int64_t k = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8; k < size; k += (int64_t)g.sums * 2048) {
        float v[8];
        load8_in<kF32>(g.G, base + k, v);
#pragma unroll
        for (int r = 0; r < 8; ++r) q += (double)v[r] * v[r];
    }
    q = workgroup_sum(q, s);
    if (threadIdx.x == 0) g.norm[(int64_t)blockIdx.y * g.sums + blockIdx.x] = q;
}

// v by in fp64, as fp32.  What comes of it is rounded to fp16 next; without the barrier
// the compiler rounds the double itself, in some forty instructions (a 128 x 512 matrix
// in one workgroup: 14 us more).
__device__ __forceinline__ float scaled(float v, double by) {
    float x = (float)((double)v * by);
    asm volatile("" : "+v"(x));
    return x;
}

// 2^k, 0 below fp32's normal numbers.
__device__ __forceinline__ float pow2(int k) {
    return __uint_as_float(k < -126 ? 0u : (uint32_t)(127 + k) << 23);
}
// What G is multiplied by to be X = G / (||G|| + eps) times its scale 2^*e; q: G's sum of
// squares, the same in all lanes.  No singular value grows by more than a in a step, so X stays
// below a^steps times its norm here.  (Zeros, NaN and infinities take the plain scale.)
__device__ __forceinline__ double x_scale(double q, double growth, int* e) {
    const double norm = sqrt(q), grown = norm / (norm + kNsEps) * growth;
    int up = 0;
    if (grown > 0.0 && grown < 1.0) up = -ilogb(grown) - 1;   // grown 2^up is in [0.5, 1)
    *e = kScaleX + __builtin_amdgcn_readfirstlane(up < 110 ? up : 110);   // (2^-e stays normal)
    return ldexp(1.0, *e) / (norm + kNsEps);
}

// X as hi + lo.
template <bool kF32>
__global__ __launch_bounds__(256) void ortho_start_kernel(OrthoArgs g) {
    __shared__ double s[4];
    double q = 0.0;
    for (int k = threadIdx.x; k < g.sums; k += 256) q += g.norm[(int64_t)blockIdx.y * g.sums + k];
    q = workgroup_sum(q, s);
    int e;
    const double by = x_scale(q, g.growth, &e);
    if (blockIdx.x == 0 && threadIdx.x == 0) g.scale_x[blockIdx.y] = e;
    const int64_t size = g.R * g.C, base = (int64_t)blockIdx.y * size;
    for (int64_t k = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8; k < size;
         k += (int64_t)gridDim.x * 2048) {
        float v[8];
        load8_in<kF32>(g.G, base + k, v);
#pragma unroll
        for (int r = 0; r < 8; ++r) v[r] = scaled(v[r], by);
        store8_pair(g.hi_next + base + k, g.lo + base + k, v);
    }
}

// PROD_SYM: E = offdiag(A), D.  PROD_POLY: b A + c A^2.  PROD_X: the step.
// The first two are symmetric: only tiles on and below the diagonal are computed,
// and each tile below it is also written transposed.
enum { PROD_SYM = 0, PROD_POLY = 1, PROD_X = 2 };

template <class Cfg, int kProd, bool kTall>
__global__ __launch_bounds__(Cfg::kThreads) void ortho_kernel(OrthoArgs g) {
    constexpr bool kAS = kProd == PROD_SYM && kTall;
    constexpr bool kBS = kProd == PROD_SYM ? kTall : kProd == PROD_X && !kTall;
    constexpr bool kTri = kProd != PROD_X;
    extern __shared__ __attribute__((aligned(16))) char smem[];
    const int64_t m = g.m, I = kProd == PROD_X ? g.R : m, J = kProd == PROD_X ? g.C : m;
    const uint32_t nI = (uint32_t)((I + Cfg::TI - 1) / Cfg::TI), nJ = (uint32_t)((J + Cfg::TJ - 1) / Cfg::TJ);
    TilePlace at;
    if (!tile_place<kTri>(blockIdx.x, nI, nJ, (uint32_t)g.full, (uint32_t)g.splits, &at)) return;
    const int64_t i0 = (int64_t)at.ti * Cfg::TI, j0 = (int64_t)at.tj * Cfg::TJ;
    const int64_t at_x = (int64_t)blockIdx.y * g.R * g.C, at_m = (int64_t)blockIdx.y * m * m;
    const uint16_t* hi = g.hi + at_x;
    const uint16_t* poly = g.poly + at_m;
    const uint16_t* sym = g.sym + at_m;
    float* diag = g.diag + blockIdx.y * m;
    float* scale = g.scale + blockIdx.y * m;
    const int ex = kProd == PROD_POLY ? 0 : g.scale_x[blockIdx.y];

    TileOperand A, B;
    int64_t K;
    if constexpr (kProd == PROD_SYM) {
        A.p = B.p = hi; A.ld = B.ld = g.C; K = g.n;
    } else if constexpr (kProd == PROD_POLY) {
        A.p = B.p = sym; A.ld = B.ld = m; K = m;
    } else if constexpr (kTall) {
        A.p = hi; A.ld = g.C; B.p = poly; B.ld = m; K = m;   // X (poly), poly symmetric
    } else {
        A.p = poly; A.ld = m; B.p = hi; B.ld = g.C; K = m;   // (poly) X
    }
    A.n = I;
    B.n = J;
    A.at[0] = i0;
    A.at[1] = i0 + Cfg::HI;
    B.at[0] = j0;
    B.at[1] = j0 + Cfg::HJ;
    const int nt = (int)((K + kTileK - 1) / kTileK), depth = (nt + at.splits - 1) / at.splits;
    const int t0 = at.split * depth, t1 = t0 + depth < nt ? t0 + depth : nt;
    const bool mirror = kTri && at.ti != at.tj;

    // the epilogue's share of this thread, and what it reads
    const PartThread<Cfg, Cfg::TJ> t;
    const int64_t j = j0 + 8 * t.c;
    const int rows = j >= J ? 0 : (int)(I - i0 < Cfg::TI ? I - i0 : Cfg::TI);
    struct None {};
    struct OfPoly { uint4 e; float d; };       // E, D_i
    struct OfX { uint4 hi, lo; float s; };     // X, scale_i
    using State = std::conditional_t<kProd == PROD_SYM, None,
                                     std::conditional_t<kProd == PROD_POLY, OfPoly, OfX>>;
    PartStates<Cfg, Cfg::TJ, State> states;
    const int64_t ld = kProd == PROD_X ? g.C : m;
    const int64_t first = (kProd == PROD_X ? at_x : 0) + (i0 + t.row0) * ld + j;
    const float* row_vector = (kProd == PROD_POLY ? diag : scale) + i0 + t.row0;
    auto before = [&](int off, State& e) {
        if constexpr (kProd == PROD_POLY) {
            e.e = ld16(sym + first + (int64_t)off * ld);
            e.d = row_vector[off];
        }
        if constexpr (kProd == PROD_X) {
            e.hi = ld16(g.hi + first + (int64_t)off * ld);
            e.lo = ld16(g.lo + first + (int64_t)off * ld);
            if constexpr (!kTall) e.s = row_vector[off];
        }
    };
    if (at.splits == 1) states.load(t, rows, before);   // (the join needs the registers)
    // the column's factors: POLY b + c D_j, X from the right a + scale_j
    float fj[8];
    if constexpr (kProd == PROD_POLY || (kProd == PROD_X && kTall)) {
        if (rows) load8_f32((kProd == PROD_POLY ? diag : scale) + j, fj);
#pragma unroll
        for (int r = 0; r < 8; ++r) fj[r] = kProd == PROD_POLY ? kNsB + kNsC * fj[r] : kNsA + fj[r];
    }

    TileAcc<Cfg> acc;
    tile_clear<Cfg>(acc);
    tile_product<Cfg, kAS, kBS, true, 1>(smem, A, B, K, nullptr, nullptr, nullptr, t0, t1, acc);
    if (at.splits > 1) {
        const int64_t joint = (int64_t)blockIdx.y * (tile_count(nI, nJ, kTri) - g.full) + at.joint;
        if (!tile_join<Cfg>(smem, g.part + joint * at.splits * (Cfg::TI * Cfg::TJ), g.count + joint,
                            at.split, at.splits, (int)(I - i0 < Cfg::TI ? I - i0 : Cfg::TI), acc))
            return;
        states.load(t, rows, before);
    }

    uint16_t* out = (kProd == PROD_SYM ? g.sym : g.poly) + at_m;
    const uint32_t places[1] = {t.place(2 * t.c)};
    // this thread's column of the diagonal in its row off: off + this, 0 to 7 if any
    const int to_diagonal = kTri && !mirror ? (int)(i0 - j0) + t.row0 - 8 * t.c : -(1 << 30);
#pragma unroll
    for (int p = 0; p < PartOf<Cfg>::kParts; ++p) {
        part_put<Cfg>(smem, acc, p);
        __syncthreads();
        states.each(smem, t, places, p, rows, before, [&](int off, int k, const float (&w)[1][8], const State& e) {
            float v[8];
#pragma unroll
            for (int r = 0; r < 8; ++r) v[r] = w[0][r];
            if constexpr (kProd == PROD_X) {
                float h[8], l[8];
                unpack8_f16(e.hi, h);
                unpack8_f16(e.lo, l);
                const float si = kTall ? 0.f : kNsA + e.s;
#pragma unroll
                for (int r = 0; r < 8; ++r)   // a (hi + lo) + scale hi + product
                    v[r] = v[r] * (1.0f / kScaleSym) + (kTall ? fj[r] : si) * h[r] + kNsA * l[r];
                const int64_t at_e = first + (int64_t)off * ld;
                if (g.last) {
#pragma unroll
                    for (int r = 0; r < 8; ++r) v[r] *= pow2(-ex);
                    *reinterpret_cast<uint4*>(g.U + at_e) =
                        make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                   pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
                } else {
                    store8_pair(g.hi_next + at_e, g.lo + at_e, v);
                }
            } else {
                if constexpr (kProd == PROD_SYM) {
#pragma unroll
                    for (int r = 0; r < 8; ++r) v[r] *= pow2(kScaleSymBits - 2 * ex);
                } else {
                    // b E + c (E^2 + (D_i + D_j) E), E and the result times kScaleSym
                    float o[8];
                    unpack8_f16(e.e, o);
                    const float ci = kNsC * e.d;
#pragma unroll
                    for (int r = 0; r < 8; ++r) v[r] = v[r] * (kNsC / kScaleSym) + o[r] * (fj[r] + ci);
                }
                const int on = off + to_diagonal;
                if ((unsigned)on < 8u) {
                    float own = 0.f;   // the diagonal element's sum
#pragma unroll
                    for (int r = 0; r < 8; ++r) {
                        own = r == on ? w[0][r] : own;
                        v[r] = r == on ? 0.f : v[r];
                    }
                    const int64_t i = i0 + t.row0 + off;
                    if constexpr (kProd == PROD_SYM)
                        diag[i] = own * pow2(-2 * ex);
                    else   // b D + c (E^2 + D^2)
                        scale[i] = kNsB * e.d + kNsC * (own * (1.0f / (kScaleSym * kScaleSym)) + e.d * e.d);
                }
                store8_f16(out + first + (int64_t)off * ld, v);
                if (mirror) t.set(smem, places[0], k, v);
            }
        });
        if (kTri && mirror) {   // the same for the whole workgroup
            __syncthreads();
            // rows of the transpose: column jm of the tile, eight of its rows at a time
            const int64_t ip = i0 + p * PartOf<Cfg>::kRows;
#pragma unroll 2
            for (int u = threadIdx.x; u < PartOf<Cfg>::kRows / 8 * Cfg::TJ; u += Cfg::kThreads) {
                const int r = u % (PartOf<Cfg>::kRows / 8), col = u / (PartOf<Cfg>::kRows / 8);
                const int64_t i = ip + 8 * r, jm = j0 + col;
                if (i >= I || jm >= J) continue;
                float v[8];
                part_get_column<Cfg>(smem, r, col, v);
                store8_f16(out + jm * m + i, v);
            }
        }
        if (p + 1 < PartOf<Cfg>::kParts) __syncthreads();
    }
}

template <class Cfg, int kProd, bool kTall>
hipError_t launch_product_cfg(const OrthoArgs& g, int64_t batch, hipStream_t stream) {
    auto kern = ortho_kernel<Cfg, kProd, kTall>;
    static std::atomic<bool> lds_set[kMaxDevices] = {};
    hipError_t e = set_dynamic_lds(reinterpret_cast<const void*>(kern), Cfg::kLds, lds_set);
    if (e != hipSuccess) return e;
    const int64_t I = kProd == PROD_X ? g.R : g.m, J = kProd == PROD_X ? g.C : g.m;
    const int64_t tiles = tile_count((I + Cfg::TI - 1) / Cfg::TI, (J + Cfg::TJ - 1) / Cfg::TJ,
                                     kProd != PROD_X);
    hipLaunchKernelGGL(kern, dim3((unsigned)tile_grid(tiles, g.full, g.splits), (unsigned)batch),
                       dim3(Cfg::kThreads), Cfg::kLds, stream, g);
    return hipGetLastError();
}

template <int kProd>
TilePlan product_plan(int64_t B, int64_t R, int64_t C) {
    const int64_t m = R < C ? R : C, K = kProd == PROD_SYM ? (R < C ? C : R) : m;
    const int strided = kProd == PROD_SYM ? (R > C ? 2 : 0) : kProd == PROD_X && R <= C ? 1 : 0;
    return tile_plan(kProd == PROD_X ? R : m, kProd == PROD_X ? C : m, 1, (K + kTileK - 1) / kTileK,
                     B, kProd != PROD_X, strided);
}

template <int kProd, bool kTall>
hipError_t launch_product(OrthoArgs g, int64_t batch, hipStream_t stream) {
    const TilePlan plan = product_plan<kProd>(batch, g.R, g.C);
    g.splits = plan.splits;
    g.full = plan.full;
    if (plan.tile == TILE_LARGE) return launch_product_cfg<TileLarge, kProd, kTall>(g, batch, stream);
    if constexpr (kProd == PROD_X)
        if (plan.tile == TILE_MID) return launch_product_cfg<TileMid, kProd, kTall>(g, batch, stream);
    return launch_product_cfg<TileSmall, kProd, kTall>(g, batch, stream);
}

// A matrix of at most 128 x 512 (either way round), all steps in one workgroup.  Eight
// waves own 64 columns of X each (n, the larger dimension, runs over the columns: for a
// tall G they are its rows) and hold them, hi and lo, in registers as operands of the X
// product: a lane has column l % 16 of each 16 and, for its group g = l / 16 and each
// 32 rows, rows 4 g to 4 g + 3 and 16 more -- what the product leaves it with, and as
// good an order of the contraction as any if P is stored in it as well.  The sum over the
// columns needs hi the other way round: through LDS, transposed, read by the transposing
// reads; A and the polynomial then lie where it was.
//
// Against the tiled products of this file (17 launches), fp32: one 128 x 512 113 -> 68 us, 256 of
// them 777 -> 86 us, 4096 of 32 x 32 5734 -> 633 us.  What bounds it is that little of its work
// overlaps: a step of 128 x 512 takes 11 us, about 27000 clocks, for LDS reads of 768 KB for A
// (6144 clocks at 128 B) and 512 KB for X (4096), 9200 clocks of matrix instructions and as many
// of vector instructions per SIMD, one after the other between six barriers.  A and A^2 are
// computed in full, although they are symmetric.
constexpr int kSmallM = 128, kSmallN = 512, kSmallThreads = 512;
constexpr int kSquareLd = 2 * kSmallM + 16;   // bytes of a row of A or the polynomial: no conflicts
constexpr int kSquare = kSmallM * kSquareLd;
constexpr int kSmallX = 2 * kSmallM * kSmallN;
constexpr int kSmallLds = kSmallX + 2 * 4 * kSmallM + 64;

inline bool ortho_small(int64_t R, int64_t C) {
    return (R < C ? R : C) <= kSmallM && (R < C ? C : R) <= kSmallN;
}

// Where LDS holds X's rows 16 t + 4 c to + 3 of column n.  The 16 rows of t go to one of
// eight places by n, so that the four columns that each half-wave of a transposing read
// takes from two groups of eight lie on all banks; the last term does it for the writes.
__device__ __forceinline__ int small_x_at(int n, int t, int c) {
    return n * (2 * kSmallM) + ((t ^ ((n & 3) | (n >> 1 & 4))) << 5) + ((c ^ (n >> 1 & 2)) << 3);
}
// ... and rows 16 t + 4 g to + 3 of column j of a square matrix.
__device__ __forceinline__ int small_square_at(int j, int t, int g) {
    return j * kSquareLd + 64 * (t >> 1) + 16 * g + 8 * (t & 1);
}

template <bool kF32, bool kTall>
__global__ __launch_bounds__(kSmallThreads) void ortho_small_kernel(const void* G, uint16_t* U, int R,
                                                                    int C, int steps, double growth) {
    extern __shared__ __attribute__((aligned(16))) char smem[];
    char* const square = smem;             // A's off-diagonal, after X was read
    char* const poly = smem + kSquare;
    float* const diag = reinterpret_cast<float*>(smem + kSmallX);
    float* const scale = diag + kSmallM;
    double* const sums = reinterpret_cast<double*>(scale + kSmallM);
    const int m = kTall ? C : R, n = kTall ? R : C;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    int li = lane & 15, g = lane >> 4;
    const int64_t base = (int64_t)blockIdx.x * R * C;
    const int col0 = 64 * wave;            // this wave's columns

    // X(i, j) is element i * row + j * col of the matrix; four rows from i at a time
    auto load4 = [&](int i, int j, float (&v)[4]) {
        const int64_t at = base + (kTall ? (int64_t)j * C + i : (int64_t)i * C + j);
#pragma unroll
        for (int r = 0; r < 4; ++r) v[r] = 0.f;
        if (i >= m || j >= n) return;      // (m and n are multiples of 8)
        if constexpr (kF32) {
            const float* p = static_cast<const float*>(G) + at;
            if constexpr (kTall) {
                const float4 w = *reinterpret_cast<const float4*>(p);
                v[0] = w.x; v[1] = w.y; v[2] = w.z; v[3] = w.w;
            } else {
#pragma unroll
                for (int r = 0; r < 4; ++r) v[r] = p[(int64_t)r * C];
            }
        } else {
            const uint16_t* p = static_cast<const uint16_t*>(G) + at;
            if constexpr (kTall) {
                const uint2 w = *reinterpret_cast<const uint2*>(p);
                v[0] = bf16_lo(w.x); v[1] = bf16_hi(w.x); v[2] = bf16_lo(w.y); v[3] = bf16_hi(w.y);
            } else {
#pragma unroll
                for (int r = 0; r < 4; ++r) v[r] = bf16_lo(p[(int64_t)r * C]);
            }
        }
    };
    auto store4 = [&](int i, int j, const float (&v)[4]) {
        if (i >= m || j >= n) return;
        uint16_t* p = U + base + (kTall ? (int64_t)j * C + i : (int64_t)i * C + j);
        const uint32_t a = pack_bf16x2(v[0], v[1]), b = pack_bf16x2(v[2], v[3]);
        if constexpr (kTall) {
            *reinterpret_cast<uint2*>(p) = make_uint2(a, b);
        } else {
            p[0] = (uint16_t)a;
            p[C] = (uint16_t)(a >> 16);
            p[2 * (int64_t)C] = (uint16_t)b;
            p[3 * (int64_t)C] = (uint16_t)(b >> 16);
        }
    };

    // [16 columns][16 rows]: rows 4 g to 4 g + 3 of them
    f16x4_t hi[4][8], lo[4][8];
    // ... from w = by^-1 times them: with fp16 results of fp32 multiply-adds, no separate
    // conversions (they bound the kernel otherwise: 9 instead of 4 instructions an element)
    auto split4 = [&](int c, int t, const float (&w)[4], float by) {
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            hi[c][t][r] = (_Float16)__builtin_fmaf(w[r], by, -0.f);
            lo[c][t][r] = (_Float16)__builtin_fmaf(w[r], by, -(float)hi[c][t][r]);
        }
    };
    auto put_x = [&]() {
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int t = 0; t < 8; ++t)
                *reinterpret_cast<uint2*>(smem + (col0 + 16 * c) * (2 * kSmallM) + small_x_at(li, t, g)) =
                    __builtin_bit_cast(uint2, hi[c][t]);
    };

    int ex;
    {   // X = G / (||G|| + eps), scaled
        float v[4][8][4];
        double q = 0.0;
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int t = 0; t < 8; ++t) load4(16 * t + 4 * g, col0 + 16 * c + li, v[c][t]);
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int t = 0; t < 8; ++t)
#pragma unroll
                for (int r = 0; r < 4; ++r) q += (double)v[c][t][r] * v[c][t][r];
#pragma unroll
        for (int d = 32; d; d >>= 1) q += __shfl_xor(q, d);
        if (lane == 0) sums[wave] = q;
        __syncthreads();
        q = 0.0;
#pragma unroll
        for (int w = 0; w < 8; ++w) q += sums[w];
        const double by = x_scale(q, growth, &ex);
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int t = 0; t < 8; ++t) {
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    asm volatile("" : "+v"(v[c][t][r]));   // (not 128 doubles from above)
                    v[c][t][r] = scaled(v[c][t][r], by);
                }
                split4(c, t, v[c][t], 1.f);
            }
    }

    // the square products: rows 64 (wave / 4) and columns 32 (wave % 4) of the output
    const int ti = 4 * (wave >> 2), tj = 2 * (wave & 3);
    const bool square_part = 16 * ti < m && 16 * tj < m;   // else zeros
    for (int step = 0; step < steps; ++step) {
        asm volatile("" : "+v"(li), "+v"(g));   // (addresses anew in each step: no room to keep them)
        if (step) __syncthreads();   // the polynomial is read
        put_x();
        __syncthreads();   // X is written
        floatx4_t acc[4][2];
        auto clear = [&]() {
#pragma unroll
            for (int x = 0; x < 4; ++x)
#pragma unroll
                for (int y = 0; y < 2; ++y) acc[x][y] = floatx4_t{0.f, 0.f, 0.f, 0.f};
        };
        auto multiply = [&](const uint4 (&a)[4], const uint4 (&b)[2]) {
#pragma unroll
            for (int x = 0; x < 4; ++x)
#pragma unroll
                for (int y = 0; y < 2; ++y) acc[x][y] = mfma16<true>(a[x], b[y], acc[x][y]);
        };
        clear();
        if (square_part) {   // A = X X^T, 32 columns of X at a time
            const int row = 8 * g + (li >> 2), q = li & 3;
            auto frag = [&](int k, int t) {
                const uint2 a = lds_read_tr16(smem + 64 * kSmallM * k + small_x_at(row, t, q));
                const uint2 b = lds_read_tr16(smem + 64 * kSmallM * k + small_x_at(row + 4, t, q));
                return make_uint4(a.x, a.y, b.x, b.y);
            };
            for (int k = 0; 32 * k < n; ++k) {
                uint4 a[4], b[2];
#pragma unroll
                for (int x = 0; x < 4; ++x) a[x] = frag(k, ti + x);
#pragma unroll
                for (int y = 0; y < 2; ++y) b[y] = frag(k, tj + y);
                multiply(a, b);
            }
        }
        __syncthreads();   // X is read
        // each lane has rows 16 (ti + x) + 4 g to + 3 of column 16 (tj + y) + li
#pragma unroll
        for (int y = 0; y < 2; ++y)
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const int j = 16 * (tj + y) + li;
                const bool on = ti + x == tj + y && g == li >> 2;   // row 4 g + li % 4 is j
                float v[4], own = 0.f;
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const bool here = on && r == (li & 3);
                    own = here ? acc[x][y][r] : own;
                    v[r] = here ? 0.f : acc[x][y][r] * pow2(kScaleSymBits - 2 * ex);
                }
                if (on) diag[j] = own * pow2(-2 * ex);
                *reinterpret_cast<uint2*>(square + small_square_at(j, ti + x, g)) = f16x4(v);
            }
        __syncthreads();   // A is written
        clear();
        for (int k = 0; k < (square_part ? 4 : 0); ++k) {
            uint4 a[4], b[2];
#pragma unroll
            for (int x = 0; x < 4; ++x)
                a[x] = ld16(square + (16 * (ti + x) + li) * kSquareLd + 64 * k + 16 * g);
#pragma unroll
            for (int y = 0; y < 2; ++y)
                b[y] = ld16(square + (16 * (tj + y) + li) * kSquareLd + 64 * k + 16 * g);
            multiply(a, b);
        }
#pragma unroll
        for (int y = 0; y < 2; ++y) {
            const int j = 16 * (tj + y) + li;
            const float fj = kNsB + kNsC * diag[j];
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const int at = small_square_at(j, ti + x, g);
                const bool on = ti + x == tj + y && g == li >> 2;
                const uint2 e = *reinterpret_cast<const uint2*>(square + at);
                float o[4];
                f32x4(e, o);
                const float4 d4 = *reinterpret_cast<const float4*>(diag + 16 * (ti + x) + 4 * g);
                const float d[4] = {d4.x, d4.y, d4.z, d4.w};
                float v[4], own = 0.f, dj = 0.f;
#pragma unroll
                for (int r = 0; r < 4; ++r) {   // as PROD_POLY
                    const bool here = on && r == (li & 3);
                    own = here ? acc[x][y][r] : own;
                    dj = here ? d[r] : dj;
                    v[r] = here ? 0.f : acc[x][y][r] * (kNsC / kScaleSym) + o[r] * (fj + kNsC * d[r]);
                }
                if (on)   // with the linear term and the scale of the products that it joins
                    scale[j] = kScaleSym * (kNsA + kNsB * dj +
                                            kNsC * (own * (1.0f / (kScaleSym * kScaleSym)) + dj * dj));
                *reinterpret_cast<uint2*>(poly + at) = f16x4(v);
            }
        }
        __syncthreads();   // the polynomial is written
        if (col0 >= n) continue;
#pragma unroll
        for (int h = 0; h < 2; ++h) {   // 32 columns at a time
            floatx4_t out[8][2];
#pragma unroll
            for (int t = 0; t < 8; ++t)
#pragma unroll
                for (int c = 0; c < 2; ++c) out[t][c] = floatx4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
#pragma unroll
                for (int t = 0; t < 8; ++t) {
                    const uint4 p = ld16(poly + (16 * t + li) * kSquareLd + 64 * k + 16 * g);
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const uint2 w0 = __builtin_bit_cast(uint2, hi[2 * h + c][2 * k]);
                        const uint2 w1 = __builtin_bit_cast(uint2, hi[2 * h + c][2 * k + 1]);
                        out[t][c] = mfma16<true>(p, make_uint4(w0.x, w0.y, w1.x, w1.y), out[t][c]);
                    }
                    if (t == 3) tile_fence();   // (few operands in flight: the registers are full)
                }
            }
            tile_fence();   // (one half's sums at a time)
#pragma unroll
            for (int t = 0; t < 8; ++t) {
                const float4 s4 = *reinterpret_cast<const float4*>(scale + 16 * t + 4 * g);
                const float s[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    float v[4];
                    const f16x4_t x = hi[2 * h + c][t], l = lo[2 * h + c][t];
#pragma unroll
                    for (int r = 0; r < 4; ++r)   // as PROD_X, times kScaleSym
                        v[r] = __builtin_fmaf((float)l[r], kScaleSym * kNsA,
                                              __builtin_fmaf((float)x[r], s[r], out[t][c][r]));
                    split4(2 * h + c, t, v, 1.0f / kScaleSym);
                }
                tile_fence();
            }
        }
    }
    // the pair as bf16 (its 22 bits are a rounding of 2^-14 of bf16's)
    asm volatile("" : "+v"(li), "+v"(g));
#pragma unroll
    for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int t = 0; t < 8; ++t) {
            float v[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) v[r] = ((float)hi[c][t][r] + (float)lo[c][t][r]) * pow2(-ex);
            store4(16 * t + 4 * g, col0 + 16 * c + li, v);
        }
}

template <bool kF32, bool kTall>
hipError_t launch_small(const void* G, uint16_t* U, int64_t B, int64_t R, int64_t C, int steps,
                        hipStream_t stream) {
    auto kern = ortho_small_kernel<kF32, kTall>;
    static std::atomic<bool> lds_set[kMaxDevices] = {};
    const hipError_t e = set_dynamic_lds(reinterpret_cast<const void*>(kern), kSmallLds, lds_set);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(kern, dim3((unsigned)B), dim3(kSmallThreads), kSmallLds, stream, G, U, (int)R,
                       (int)C, steps, std::pow((double)kNsA, steps));
    return hipGetLastError();
}

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

}  // namespace

OrthogonalizeLayout orthogonalize_layout(int64_t B, int64_t R, int64_t C) {
    OrthogonalizeLayout L{};
    const int64_t m = R < C ? R : C;
    if (ortho_small(R, C)) return L;
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
    L.norm = take(sizeof(double) * B * norm_blocks(R * C));
    L.scale_x = take(sizeof(int) * B);
    const TilePlan plans[] = {product_plan<PROD_SYM>(B, R, C), product_plan<PROD_POLY>(B, R, C),
                              product_plan<PROD_X>(B, R, C)};
    int64_t part = 0;
    L.counters = 0;
    for (const TilePlan& p : plans) {
        if (p.part_floats > part) part = p.part_floats;
        if (p.counters > L.counters) L.counters = p.counters;
    }
    L.part = take(sizeof(float) * part);
    L.count = take(sizeof(uint32_t) * L.counters);
    L.total = off;
    return L;
}

hipError_t launch_orthogonalize(const void* G, bool f32, uint16_t* U, int64_t B, int64_t R,
                                int64_t C, int steps, char* ws, hipStream_t stream) {
    if (ortho_small(R, C))
        return f32 ? R > C ? launch_small<true, true>(G, U, B, R, C, steps, stream)
                           : launch_small<true, false>(G, U, B, R, C, steps, stream)
               : R > C ? launch_small<false, true>(G, U, B, R, C, steps, stream)
                       : launch_small<false, false>(G, U, B, R, C, steps, stream);
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
    g.scale_x = reinterpret_cast<int*>(ws + L.scale_x);
    g.growth = std::pow((double)kNsA, steps);
    g.part = reinterpret_cast<float*>(ws + L.part);
    g.count = reinterpret_cast<uint32_t*>(ws + L.count);
    g.counters = L.counters;
    g.splits = 1;
    g.full = 0;
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
    g.sums = norm_blocks(R * C);
    int64_t blocks = (R * C + 2047) / 2048, most = 2048 / B;   // a round of workgroups
    if (blocks > most) blocks = most < 1 ? 1 : most;
    if (f32) {
        hipLaunchKernelGGL(ortho_norm_kernel<true>, dim3((unsigned)g.sums, (unsigned)B), dim3(256), 0, stream, g);
        hipLaunchKernelGGL(ortho_start_kernel<true>, dim3((unsigned)blocks, (unsigned)B), dim3(256), 0, stream, g);
    } else {
        hipLaunchKernelGGL(ortho_norm_kernel<false>, dim3((unsigned)g.sums, (unsigned)B), dim3(256), 0, stream, g);
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
