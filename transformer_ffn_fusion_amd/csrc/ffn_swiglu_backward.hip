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

struct SwigluBackwardArgs {
    const uint16_t *X, *Wg, *Wu, *Wd, *dY;
    uint16_t* dX;
    void *dWg, *dWu, *dWd;
    float* dH;
    uint16_t *H, *dAB;
    float* part;        // sums of split products (tile_join)
    uint32_t* count;
    int64_t M, N, O, P;
    int splits;         // of this step
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
    // k-tiles, over both products of the dX step
    static __host__ __device__ int depth(int64_t M, int64_t N, int64_t O, int64_t P) {
        const int64_t K = kStep == STEP_DH ? P : kStep == STEP_GATED ? N : kStep == STEP_DX ? O : M;
        return (int)((K + kTileK - 1) / kTileK) * (kStep == STEP_DX ? 2 : 1);
    }
    static TilePlan plan(int64_t M, int64_t N, int64_t O, int64_t P) {
        return tile_plan(rows(M, N, O), cols(N, O, P), kStep == STEP_GATED ? 2 : 1,
                         depth(M, N, O, P), 1, false);
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
    TilePlace at;
    if (!tile_place<false>(blockIdx.x, (I + Cfg::TI - 1) / Cfg::TI, (J + kWidth - 1) / kWidth,
                           g.splits, &at))
        return;
    const int64_t i0 = at.ti * Cfg::TI, j0 = at.tj * kWidth;

    TileOperand A, B;
    int64_t K;
    const uint16_t *a2 = nullptr, *b2 = nullptr, *b_half2 = nullptr;
    if constexpr (kStep == STEP_DH) {
        A.p = g.dY; A.ld = P; B.p = g.Wd; B.ld = P; K = P;
    } else if constexpr (kStep == STEP_GATED) {
        A.p = g.X; A.ld = N; B.p = g.Wg; B.ld = O; K = N;
        b_half2 = g.Wu;
    } else if constexpr (kStep == STEP_DX) {
        A.p = g.dAB; A.ld = 2 * O; B.p = g.Wg; B.ld = O; K = O;
        a2 = g.dAB + O; b2 = g.Wu;
    } else if constexpr (kStep == STEP_DGU) {
        A.p = g.X; A.ld = N; B.p = g.dAB; B.ld = 2 * O; K = M;
    } else {
        A.p = g.H; A.ld = O; B.p = g.dY; B.ld = P; K = M;
    }
    A.n = I;
    B.n = J;
    A.at[0] = i0;
    A.at[1] = i0 + Cfg::HI;
    B.at[0] = j0;
    B.at[1] = kStep == STEP_GATED ? j0 : j0 + Cfg::HJ;
    constexpr int kPairs = kStep == STEP_DX ? 2 : 1;
    const int nt = S::depth(M, N, O, P), depth = (nt + g.splits - 1) / g.splits;
    const int t0 = at.split * depth, t1 = t0 + depth < nt ? t0 + depth : nt;
    TileAcc<Cfg> acc;
    tile_clear<Cfg>(acc);
    tile_product<Cfg, S::kAS, S::kBS, false, kPairs>(smem, A, B, K, a2, b2, b_half2, t0, t1, acc);
    if (g.splits > 1 &&
        !tile_join<Cfg>(smem, g.part + at.tile * g.splits * (Cfg::TI * Cfg::TJ), g.count + at.tile,
                        at.split, g.splits, acc))
        return;

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
    const int64_t tiles = tile_count((I + Cfg::TI - 1) / Cfg::TI, (J + kWidth - 1) / kWidth, false);
    hipLaunchKernelGGL(kern, dim3((unsigned)tile_grid(tiles, g.splits)), dim3(Cfg::kThreads),
                       Cfg::kLds, stream, g);
    return hipGetLastError();
}

template <int kStep, bool kGradF32>
hipError_t launch_step(SwigluBackwardArgs g, hipStream_t stream) {
    const TilePlan plan = StepShape<kStep>::plan(g.M, g.N, g.O, g.P);
    g.splits = plan.splits;
    if (plan.tile == TILE_LARGE) return launch_step_cfg<TileLarge, kStep, kGradF32>(g, stream);
    if (plan.tile == TILE_MID) return launch_step_cfg<TileMid, kStep, kGradF32>(g, stream);
    return launch_step_cfg<TileSmall, kStep, kGradF32>(g, stream);
}

template <bool kGradF32>
hipError_t launch_all(const SwigluBackwardArgs& g, int64_t counters, hipStream_t stream) {
    hipError_t e = launch_zero_f32(reinterpret_cast<float*>(g.count), counters, stream);
    if (e != hipSuccess) return e;
    if ((e = launch_step<STEP_DH, false>(g, stream)) != hipSuccess) return e;
    if ((e = launch_step<STEP_GATED, false>(g, stream)) != hipSuccess) return e;
    if ((e = launch_step<STEP_DX, false>(g, stream)) != hipSuccess) return e;
    if ((e = launch_step<STEP_DGU, kGradF32>(g, stream)) != hipSuccess) return e;
    return launch_step<STEP_DD, kGradF32>(g, stream);
}

// What the five steps' joins need at most: they run one after the other.
TilePlan join_need(int64_t M, int64_t N, int64_t O, int64_t P) {
    TilePlan most{0, 1, 0, 0};
    const TilePlan plans[] = {StepShape<STEP_DH>::plan(M, N, O, P), StepShape<STEP_GATED>::plan(M, N, O, P),
                              StepShape<STEP_DX>::plan(M, N, O, P), StepShape<STEP_DGU>::plan(M, N, O, P),
                              StepShape<STEP_DD>::plan(M, N, O, P)};
    for (const TilePlan& p : plans) {
        if (p.part_floats > most.part_floats) most.part_floats = p.part_floats;
        if (p.counters > most.counters) most.counters = p.counters;
    }
    return most;
}

}  // namespace

SwigluBackwardLayout swiglu_backward_layout(int64_t M, int64_t N, int64_t O, int64_t P) {
    SwigluBackwardLayout L;
    size_t off = 0;
    auto take = [&](size_t bytes) {
        const size_t at = off;
        off += (bytes + 255) / 256 * 256;
        return at;
    };
    const TilePlan join = M > 0 ? join_need(M, N, O, P) : TilePlan{0, 1, 0, 0};
    L.dH = take(sizeof(float) * M * O);
    L.H = take(sizeof(uint16_t) * M * O);
    L.dAB = take(sizeof(uint16_t) * M * 2 * O);
    L.part = take(sizeof(float) * join.part_floats);
    L.count = take(sizeof(uint32_t) * join.counters);
    L.counters = join.counters;
    L.total = off ? off : 256;
    return L;
}

hipError_t launch_swiglu_backward(const SwigluBackwardIO& io, hipStream_t stream) {
    const SwigluBackwardLayout L = swiglu_backward_layout(io.M, io.N, io.O, io.P);
    SwigluBackwardArgs g;
    g.X = io.X;
    g.Wg = io.Wg;
    g.Wu = io.Wu;
    g.Wd = io.Wd;
    g.dY = io.dY;
    g.dX = io.dX;
    g.dWg = io.dWg;
    g.dWu = io.dWu;
    g.dWd = io.dWd;
    g.dH = reinterpret_cast<float*>(io.ws + L.dH);
    g.H = reinterpret_cast<uint16_t*>(io.ws + L.H);
    g.dAB = reinterpret_cast<uint16_t*>(io.ws + L.dAB);
    g.part = reinterpret_cast<float*>(io.ws + L.part);
    g.count = reinterpret_cast<uint32_t*>(io.ws + L.count);
    g.M = io.M;
    g.N = io.N;
    g.O = io.O;
    g.P = io.P;
    g.splits = 1;
    return io.grad_f32 ? launch_all<true>(g, L.counters, stream) : launch_all<false>(g, L.counters, stream);
}

}  // namespace ffn
