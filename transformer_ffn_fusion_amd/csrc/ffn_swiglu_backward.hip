// ffn_swiglu_backward.hip -- gradients of the gated (SwiGLU) FFN on MFMA.
//
// With a = X Wg, b = X Wu, h = silu(a) * b, Y = h Wd, s = sigmoid(a) and the
// output gradient dY:
//
//   1. dh = dY Wd^T                                            (M x O, fp32)
//   2. a, b, recomputed together; epilogue: h = a s b,
//      da = dh b s (1 + a (1 - s)), db = dh a s                (M x O each, bf16)
//   3. dX = da Wg^T + db Wu^T, one sum over both products      (M x N, bf16)
//   4. dWg = X^T da, dWu = X^T db, as one product X^T [da|db]  (N x O each)
//   5. dWd = h^T dY                                            (O x P)
//
// The forward keeps no H, so the backward recomputes a and b.  dh stays fp32 and
// a, b never leave the accumulators: every gradient sees one bf16 rounding of
// h, da or db (they are matrix-instruction operands) and its own.  Rounding dh or
// the activation's factors to bf16 as well would add a second and a third
// rounding of the same size to dX and the weight gradients.
//
// Bound: the eight products, 12 M N O + 4 M O P operations (gemm16.h).  Every
// output element is one workgroup's sum over the whole depth in a fixed order: no
// atomics, bitwise reproducible.
#include "ffn_device.h"
#include "ffn_internal.h"
#include "gemm16.h"

namespace ffn {

namespace {

using Large = TileCfg<256, 256, 2, 4>;   // eight waves, one workgroup per CU
using Small = TileCfg<128, 128, 2, 2>;   // four waves, two workgroups per CU

struct SwigluBackwardArgs {
    const uint16_t *X, *Wg, *Wu, *Wd, *dY;
    uint16_t* dX;
    void *dWg, *dWu, *dWd;
    float* dH;
    uint16_t *H, *dAB;
    int64_t M, N, O, P;
};

// The steps above.  GATED's tile holds the gate's columns in its first half and
// the up projection's same columns in its second.
enum { STEP_DH = 0, STEP_GATED = 1, STEP_DX = 2, STEP_DGU = 3, STEP_DD = 4 };

template <int kStep>
struct StepShape {
    static constexpr bool kAS = kStep == STEP_DGU || kStep == STEP_DD;
    static constexpr bool kBS = kAS || kStep == STEP_GATED;
    static __host__ __device__ int64_t rows(int64_t M, int64_t N, int64_t O) {
        return kStep == STEP_DGU ? N : kStep == STEP_DD ? O : M;
    }
    // output columns, in the tile's terms (the gated step: hidden columns, TJ / 2 a tile)
    static __host__ __device__ int64_t cols(int64_t N, int64_t O, int64_t P) {
        return kStep == STEP_DX ? N : kStep == STEP_DGU ? 2 * O : kStep == STEP_DD ? P : O;
    }
    template <class Cfg>
    static __host__ __device__ constexpr int width() {
        return kStep == STEP_GATED ? Cfg::HJ : Cfg::TJ;
    }
};

__device__ __forceinline__ void store4_bf16(uint16_t* p, const float (&v)[4]) {
    *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
}
template <bool kGradF32>
__device__ __forceinline__ void store4_grad(void* p, int64_t at, const float (&v)[4]) {
    if constexpr (kGradF32)
        *reinterpret_cast<float4*>(static_cast<float*>(p) + at) = make_float4(v[0], v[1], v[2], v[3]);
    else
        store4_bf16(static_cast<uint16_t*>(p) + at, v);
}

template <class Cfg, int kStep, bool kGradF32>
__global__ __launch_bounds__(Cfg::kThreads) void swiglu_backward_kernel(SwigluBackwardArgs g) {
    using S = StepShape<kStep>;
    extern __shared__ __attribute__((aligned(16))) char smem[];
    const int64_t M = g.M, N = g.N, O = g.O, P = g.P;
    const int64_t I = S::rows(M, N, O), J = S::cols(N, O, P);
    constexpr int kWidth = S::template width<Cfg>();
    int64_t ti, tj;
    if (!tile_place(blockIdx.x, (I + Cfg::TI - 1) / Cfg::TI, (J + kWidth - 1) / kWidth, &ti, &tj))
        return;
    const int64_t i0 = ti * Cfg::TI, j0 = tj * kWidth;

    TileOps op;
    op.pairs = kStep == STEP_DX ? 2 : 1;
    const uint16_t *A, *B, *A2 = nullptr, *B2 = nullptr;
    if constexpr (kStep == STEP_DH) {
        A = g.dY; op.lda = P; B = g.Wd; op.ldb = P; op.K = P;
    } else if constexpr (kStep == STEP_GATED) {
        A = g.X; op.lda = N; B = g.Wg; op.ldb = O; op.K = N;
    } else if constexpr (kStep == STEP_DX) {
        A = g.dAB; op.lda = 2 * O; B = g.Wg; op.ldb = O; op.K = O;
        A2 = g.dAB + O; B2 = g.Wu;
    } else if constexpr (kStep == STEP_DGU) {
        A = g.X; op.lda = N; B = g.dAB; op.ldb = 2 * O; op.K = M;
    } else {
        A = g.H; op.lda = O; B = g.dY; op.ldb = P; op.K = M;
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        op.a[0][h] = half_walk<S::kAS>(A, op.lda, I, op.K, i0 + h * Cfg::HI);
        if constexpr (kStep == STEP_GATED)
            op.b[0][h] = half_walk<S::kBS>(h ? g.Wu : g.Wg, op.ldb, J, op.K, j0);
        else
            op.b[0][h] = half_walk<S::kBS>(B, op.ldb, J, op.K, j0 + h * Cfg::HJ);
        if constexpr (kStep == STEP_DX) {
            op.a[1][h] = half_walk<S::kAS>(A2, op.lda, I, op.K, i0 + h * Cfg::HI);
            op.b[1][h] = half_walk<S::kBS>(B2, op.ldb, J, op.K, j0 + h * Cfg::HJ);
        } else {
            op.a[1][h] = op.a[0][h];
            op.b[1][h] = op.b[0][h];
        }
    }
    TileAcc<Cfg> acc;
    tile_clear<Cfg>(acc);
    tile_product<Cfg, S::kAS, S::kBS, false>(smem, op, acc);

    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
    for (int p = 0; p < 2; ++p)
#pragma unroll
        for (int x = 0; x < Cfg::FI; ++x) {
            const int64_t i = i0 + tile_row<Cfg>(wave, p, x) + (lane & 15);
            if (i >= I) continue;
            // every column count is a multiple of 8: a lane's four are all in or all out
            if constexpr (kStep == STEP_GATED) {
#pragma unroll
                for (int y = 0; y < Cfg::FJ; ++y) {
                    const int64_t j = j0 + tile_col<Cfg>(wave, 0, y) + 4 * (lane >> 4);
                    if (j >= J) continue;
                    const float4 d = *reinterpret_cast<const float4*>(g.dH + i * O + j);
                    const float dh[4] = {d.x, d.y, d.z, d.w};
                    float h[4], da[4], db[4];
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const float a = acc[p][0][x][y][r], b = acc[p][1][x][y][r];
                        const float s = __builtin_amdgcn_rcpf(1.0f + __expf(-a));
                        const float t = a * s;
                        h[r] = t * b;
                        da[r] = dh[r] * b * (s + t * (1.0f - s));
                        db[r] = dh[r] * t;
                    }
                    store4_bf16(g.H + i * O + j, h);
                    store4_bf16(g.dAB + i * 2 * O + j, da);
                    store4_bf16(g.dAB + i * 2 * O + O + j, db);
                }
            } else {
#pragma unroll
                for (int q = 0; q < 2; ++q)
#pragma unroll
                    for (int y = 0; y < Cfg::FJ; ++y) {
                        const int64_t j = j0 + tile_col<Cfg>(wave, q, y) + 4 * (lane >> 4);
                        if (j >= J) continue;
                        const float v[4] = {acc[p][q][x][y][0], acc[p][q][x][y][1],
                                            acc[p][q][x][y][2], acc[p][q][x][y][3]};
                        if constexpr (kStep == STEP_DH)
                            *reinterpret_cast<float4*>(g.dH + i * O + j) =
                                make_float4(v[0], v[1], v[2], v[3]);
                        else if constexpr (kStep == STEP_DX)
                            store4_bf16(g.dX + i * N + j, v);
                        else if constexpr (kStep == STEP_DGU)
                            store4_grad<kGradF32>(j < O ? g.dWg : g.dWu, i * O + (j < O ? j : j - O), v);
                        else
                            store4_grad<kGradF32>(g.dWd, i * P + j, v);
                    }
            }
        }
}

template <class Cfg, int kStep, bool kGradF32>
hipError_t launch_step_cfg(const SwigluBackwardArgs& g, hipStream_t stream) {
    using S = StepShape<kStep>;
    auto kern = swiglu_backward_kernel<Cfg, kStep, kGradF32>;
    static std::atomic<bool> lds_set[kMaxDevices] = {};
    hipError_t e = set_dynamic_lds(reinterpret_cast<const void*>(kern), Cfg::kLds, lds_set);
    if (e != hipSuccess) return e;
    const int64_t I = S::rows(g.M, g.N, g.O), J = S::cols(g.N, g.O, g.P);
    constexpr int kWidth = S::template width<Cfg>();
    const int64_t grid = tile_grid((I + Cfg::TI - 1) / Cfg::TI, (J + kWidth - 1) / kWidth);
    hipLaunchKernelGGL(kern, dim3((unsigned)grid), dim3(Cfg::kThreads), Cfg::kLds, stream, g);
    return hipGetLastError();
}

// Tile choice: the fewer rounds of the chip's CUs, weighted by what a round
// takes.  A round of large tiles (one per CU) does four times the work of a
// round of small ones at two per CU in 1 / 0.65 of the time.
template <int kStep, bool kGradF32>
hipError_t launch_step(const SwigluBackwardArgs& g, hipStream_t stream) {
    using S = StepShape<kStep>;
    const int64_t I = S::rows(g.M, g.N, g.O), J = S::cols(g.N, g.O, g.P), cus = device_cus();
    const int64_t large = ((I + Large::TI - 1) / Large::TI) *
                          ((J + S::template width<Large>() - 1) / S::template width<Large>());
    const int64_t small = ((I + Small::TI - 1) / Small::TI) *
                          ((J + S::template width<Small>() - 1) / S::template width<Small>());
    const double t_large = (double)((large + cus - 1) / cus);
    const double t_small = 0.65 * (double)((small + 2 * cus - 1) / (2 * cus));
    if (t_large <= t_small) return launch_step_cfg<Large, kStep, kGradF32>(g, stream);
    return launch_step_cfg<Small, kStep, kGradF32>(g, stream);
}

template <bool kGradF32>
hipError_t launch_all(const SwigluBackwardArgs& g, hipStream_t stream) {
    hipError_t e;
    if ((e = launch_step<STEP_DH, false>(g, stream)) != hipSuccess) return e;
    if ((e = launch_step<STEP_GATED, false>(g, stream)) != hipSuccess) return e;
    if ((e = launch_step<STEP_DX, false>(g, stream)) != hipSuccess) return e;
    if ((e = launch_step<STEP_DGU, kGradF32>(g, stream)) != hipSuccess) return e;
    return launch_step<STEP_DD, kGradF32>(g, stream);
}

}  // namespace

hipError_t launch_swiglu_backward(const SwigluBackwardIO& io, hipStream_t stream) {
    const SwigluBackwardArgs g{io.X,  io.Wg,  io.Wu, io.Wd, io.dY,  io.dX, io.dWg, io.dWu,
                               io.dWd, io.dH, io.H,  io.dAB, io.M, io.N,  io.O,   io.P};
    return io.grad_f32 ? launch_all<true>(g, stream) : launch_all<false>(g, stream);
}

}  // namespace ffn
