// ffn_swiglu_backward.hip -- gradients of the gated (SwiGLU) FFN on MFMA.
//
// With a = X Wg, b = X Wu, h = silu(a) * b, Y = h Wd, s = sigmoid(a) and the
// output gradient dY:
//
//   1. dh = dY Wd^T                           (M x O, fp32; small calls: inside 2.)
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
// output element is a sum in a fixed order: one workgroup's over the whole depth, or,
// where a tile's depth is split, of up to 16 workgroups' parts, which the last to
// arrive adds in ascending order (tile_join; an integer counter per tile tells who is
// last).  No floating-point atomics, bitwise reproducible.
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
    int64_t full;       // tiles of this step that are not split ...
    int splits;         // ... and into how many the others are
    int64_t clear;      // counters that the first step sets to 0
    uint32_t from_gu, from_dd;   // dX, dWg | dWu and dWd in one launch: first workgroups of the latter
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
                         depth(M, N, O, P), 1, false, kAS ? 2 : kBS ? 1 : 0);
    }
    template <class Cfg>
    static __host__ __device__ constexpr int width() {
        return kStep == STEP_GATED ? Cfg::HJ : Cfg::TJ;
    }
};

__device__ __forceinline__ void load8_f32(const float* p, float (&v)[8]) {
    const float4 a = *reinterpret_cast<const float4*>(p);
    const float4 b = *reinterpret_cast<const float4*>(p + 4);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
template <bool kF32>
__device__ __forceinline__ void store8(void* p, int64_t at, const float (&v)[8]) {
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

// Workgroup w of one step; kOwnDh: the gated step computes its tile of dh itself.
template <class Cfg, int kStep, bool kGradF32, bool kOwnDh = false>
__device__ __forceinline__ void run_step(char* smem, const SwigluBackwardArgs& g, uint32_t w,
                                         uint32_t full, uint32_t splits) {
    using S = StepShape<kStep>;
    const int64_t M = g.M, N = g.N, O = g.O, P = g.P;
    const int64_t I = S::rows(M, N, O), J = S::cols(N, O, P);
    constexpr int kWidth = S::template width<Cfg>();
    if constexpr (kStep == STEP_DH || kOwnDh)   // a later step's counters (this one has no splits then)
        if (w == 0)
            for (int64_t k = threadIdx.x; k < g.clear; k += Cfg::kThreads) g.count[k] = 0;
    TilePlace at;
    if (!tile_place<false>(w, (uint32_t)((I + Cfg::TI - 1) / Cfg::TI),
                           (uint32_t)((J + kWidth - 1) / kWidth), full, splits, &at))
        return;
    const int64_t i0 = (int64_t)at.ti * Cfg::TI, j0 = (int64_t)at.tj * kWidth;

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
    const int nt = S::depth(M, N, O, P), depth = (nt + at.splits - 1) / at.splits;
    const int t0 = at.split * depth, t1 = t0 + depth < nt ? t0 + depth : nt;
    // the epilogue's share of this thread; every column count is a multiple of 8: its
    // eight columns are all in or all out
    constexpr int kCols = kStep == STEP_GATED ? Cfg::HJ : Cfg::TJ;
    const PartThread<Cfg, kCols> t;
    const int64_t j = j0 + 8 * t.c;
    const int rows = j >= J ? 0 : (int)(I - i0 < Cfg::TI ? I - i0 : Cfg::TI);
    struct None {};
    struct Dh { float v[8]; };
    PartStates<Cfg, kCols, std::conditional_t<kStep == STEP_GATED, Dh, None>> states;
    const int64_t first = (i0 + t.row0) * O + j;   // this thread's place in an M x O matrix
    auto before = [&](int off, auto& d) {
        if constexpr (kStep == STEP_GATED) load8_f32(g.dH + first + (int64_t)off * O, d.v);
    };
    if constexpr (kOwnDh) {
        // dY Wd^T of the tile's rows and hidden columns, through LDS to the threads that use it
        using Own = TileCfg<Cfg::TI, Cfg::HJ, Cfg::WI, Cfg::WJ>;
        static_assert(states.kEarly && PartOf<Own>::kParts == PartOf<Cfg>::kParts, "one part, kept");
        TileOperand C = A, D = B;
        C.p = g.dY;
        D.p = g.Wd;
        C.ld = D.ld = P;
        D.at[1] = j0 + Own::HJ;
        TileAcc<Own> dh;
        tile_clear<Own>(dh);
        tile_product<Own, false, false, false, 1>(smem, C, D, P, nullptr, nullptr, nullptr, 0,
                                                  (int)((P + kTileK - 1) / kTileK), dh);
        part_put<Own>(smem, dh, 0);
        __syncthreads();
        const PartThread<Own, kCols> own;
#pragma unroll
        for (int k = 0; k < own.kUnits; ++k) own.get(smem, own.place(2 * own.c), k, states.early[0][k].v);
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        __syncthreads();   // the next product's loads take the place
    } else if (at.splits == 1) {
        states.load(t, rows, before);   // (the join needs the registers)
    }

    TileAcc<Cfg> acc;
    tile_clear<Cfg>(acc);
    tile_product<Cfg, S::kAS, S::kBS, false, kPairs>(smem, A, B, K, a2, b2, b_half2, t0, t1, acc);
    if (at.splits > 1) {
        if (!tile_join<Cfg>(smem, g.part + (int64_t)at.joint * at.splits * (Cfg::TI * Cfg::TJ),
                            g.count + at.joint, at.split, at.splits,
                            (int)(I - i0 < Cfg::TI ? I - i0 : Cfg::TI), acc))
            return;
        states.load(t, rows, before);
    }

    // the output of the other steps, its leading dimension, this thread's place there
    constexpr bool kF32 = kStep == STEP_DH || ((kStep == STEP_DGU || kStep == STEP_DD) && kGradF32);
    void* out = kStep == STEP_DH ? (void*)g.dH : kStep == STEP_DX ? (void*)g.dX
                : kStep == STEP_DD ? g.dWd : j < O ? g.dWg : g.dWu;
    const int64_t ld = kStep == STEP_DX ? N : kStep == STEP_DD ? P : O;
    const int64_t at_out = (i0 + t.row0) * ld + (kStep == STEP_DGU && j >= O ? j - O : j);
    const int64_t first2 = (i0 + t.row0) * 2 * O + j;   // in da | db
#pragma unroll
    for (int p = 0; p < PartOf<Cfg>::kParts; ++p) {
        part_put<Cfg>(smem, acc, p);
        __syncthreads();
        if constexpr (kStep == STEP_GATED) {
            const uint32_t places[2] = {t.place(2 * t.c), t.place(Cfg::HJ / 4 + 2 * t.c)};
            states.each(smem, t, places, p, rows, before, [&](int off, int, const float (&v)[2][8], const Dh& d) {
                float h[8], da[8], db[8];
#pragma unroll
                for (int r = 0; r < 8; ++r) {
                    const float a = v[0][r], b = v[1][r];
                    const float s = __builtin_amdgcn_rcpf(1.0f + __expf(-a));
                    const float u = a * s;
                    h[r] = u * b;
                    da[r] = d.v[r] * b * (s + u * (1.0f - s));
                    db[r] = d.v[r] * u;
                }
                store8<false>(g.H, first + (int64_t)off * O, h);
                store8<false>(g.dAB, first2 + (int64_t)off * 2 * O, da);
                store8<false>(g.dAB, first2 + (int64_t)off * 2 * O + O, db);
            });
        } else {
            const uint32_t places[1] = {t.place(2 * t.c)};
            states.each(smem, t, places, p, rows, before, [&](int off, int, const float (&v)[1][8], const None&) {
                store8<kF32>(out, at_out + (int64_t)off * ld, v[0]);
            });
        }
        if (p + 1 < PartOf<Cfg>::kParts) __syncthreads();
    }
}

template <class Cfg, int kStep, bool kGradF32>
__global__ __launch_bounds__(Cfg::kThreads) void swiglu_backward_kernel(SwigluBackwardArgs g) {
    extern __shared__ __attribute__((aligned(16))) char smem[];
    run_step<Cfg, kStep, kGradF32>(smem, g, blockIdx.x, (uint32_t)g.full, (uint32_t)g.splits);
}

// dh and the gated step in one launch, where that is faster (hidden_together).  The same sums in
// the same order as apart in 128 x 128 tiles: dh stays fp32 and goes through LDS only.
template <class Cfg>
__global__ __launch_bounds__(Cfg::kThreads) void swiglu_backward_hidden_kernel(SwigluBackwardArgs g) {
    extern __shared__ __attribute__((aligned(16))) char smem[];
    run_step<Cfg, STEP_GATED, false, true>(smem, g, blockIdx.x, 0x7fffffffu, 1);
}

// dX, dWg and dWu, and dWd in one launch: they do not depend on each other, and where
// each alone leaves CUs idle, or is over before a launch is, together they fill them
// (whole calls: 8 x 128 x 512 x 128 28 -> 18 us, 16 x 4096 x 1792 x 4096 67 -> 57,
// 1013 x 2056 x 1400 x 1992 110 -> 95; dh still apart).  Only dX may be split (few
// tokens: few tiles of it, each as deep as 2 O).
template <class Cfg, bool kGradF32>
__global__ __launch_bounds__(Cfg::kThreads) void swiglu_backward_outputs_kernel(SwigluBackwardArgs g) {
    extern __shared__ __attribute__((aligned(16))) char smem[];
    const uint32_t w = blockIdx.x;
    // dX first: its tiles are the deep ones where there are few tokens, and a join is
    // best behind other tiles' work
    if (w < g.from_gu)
        run_step<Cfg, STEP_DX, false>(smem, g, w, (uint32_t)g.full, (uint32_t)g.splits);
    else if (w < g.from_dd)
        run_step<Cfg, STEP_DGU, kGradF32>(smem, g, w - g.from_gu, 0x7fffffffu, 1);
    else
        run_step<Cfg, STEP_DD, kGradF32>(smem, g, w - g.from_dd, 0x7fffffffu, 1);
}

template <class Cfg, class Kernel>
hipError_t launch_kernel(Kernel kern, std::atomic<bool> (&lds_set)[kMaxDevices],
                         const SwigluBackwardArgs& g, int64_t grid, hipStream_t stream) {
    hipError_t e = set_dynamic_lds(reinterpret_cast<const void*>(kern), Cfg::kLds, lds_set);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(kern, dim3((unsigned)grid), dim3(Cfg::kThreads), Cfg::kLds, stream, g);
    return hipGetLastError();
}

template <int kStep>
int64_t step_tiles(int kind, int64_t M, int64_t N, int64_t O, int64_t P) {
    using S = StepShape<kStep>;
    return tile_tiles(kind, S::rows(M, N, O), S::cols(N, O, P), kStep == STEP_GATED ? 2 : 1, false);
}

template <class Cfg, int kStep, bool kGradF32>
hipError_t launch_step_cfg(const SwigluBackwardArgs& g, const TilePlan& plan, hipStream_t stream) {
    static std::atomic<bool> lds_set[kMaxDevices] = {};
    const int64_t tiles = step_tiles<kStep>(plan.tile, g.M, g.N, g.O, g.P);
    return launch_kernel<Cfg>(swiglu_backward_kernel<Cfg, kStep, kGradF32>, lds_set, g,
                              tile_grid(tiles, g.full, g.splits), stream);
}

template <int kStep, bool kGradF32>
hipError_t launch_step(SwigluBackwardArgs g, hipStream_t stream) {
    const TilePlan plan = StepShape<kStep>::plan(g.M, g.N, g.O, g.P);
    g.splits = plan.splits;
    g.full = plan.full;
    if (plan.tile == TILE_LARGE) return launch_step_cfg<TileLarge, kStep, kGradF32>(g, plan, stream);
    if (plan.tile == TILE_MID) return launch_step_cfg<TileMid, kStep, kGradF32>(g, plan, stream);
    return launch_step_cfg<TileSmall, kStep, kGradF32>(g, plan, stream);
}

// The last three steps together, in small tiles: bound by all the k-tiles there are at
// the full chip's rate, or by the deepest tile.
TilePlan outputs_plan(int64_t M, int64_t N, int64_t O, int64_t P) {
    TilePlan best{TILE_SMALL, 1, 0, 0, 0, 1e30};
    constexpr int k = TILE_SMALL;
    const int64_t nt_x = StepShape<STEP_DX>::depth(M, N, O, P), nt_w = StepShape<STEP_DD>::depth(M, N, O, P);
    const int64_t slots = kTileKinds[k].slots, tx = step_tiles<STEP_DX>(k, M, N, O, P);
    const int64_t tw = step_tiles<STEP_DGU>(k, M, N, O, P) + step_tiles<STEP_DD>(k, M, N, O, P);
    for (int64_t s = 1; s <= 16 && s <= nt_x; ++s) {
        const int64_t depth = (nt_x + s - 1) / s;
        if ((nt_x + depth - 1) / depth != s || (s > 1 && tx * s > slots)) continue;
        const double all = (double)(tx * s * depth + tw * nt_w) / (double)slots * tile_us(k, slots, 2);
        const double deep = (double)depth * tile_us(k, tx * s + tw, 0) + (s > 1 ? join_us(k, M, tx, s) : 0.0);
        // further rounds pay their way in and out too (tiles of one k-tile hardly)
        const double more = (double)(tx * s + tw) / (double)slots - 1.0;
        const double way = nt_w < 12 ? 2.0 + 0.2 * (double)nt_w : kLaunchUs;
        const double t = kLaunchUs + (more > 0.0 ? way * more : 0.0) + (all > deep ? all : deep);
        if (t < best.us) {
            best.us = t;
            best.splits = (int)s;
            best.full = s == 1 ? tx : 0;
            best.part_floats = s > 1 ? tx * s * (int64_t)kTileKinds[k].ti * kTileKinds[k].tj : 0;
            best.counters = s > 1 ? tx : 0;
        }
    }
    return best;
}
bool outputs_together(const TilePlan& together, int64_t M, int64_t N, int64_t O, int64_t P) {
    return together.us < StepShape<STEP_DX>::plan(M, N, O, P).us + StepShape<STEP_DGU>::plan(M, N, O, P).us +
                             StepShape<STEP_DD>::plan(M, N, O, P).us;
}

template <bool kGradF32>
hipError_t launch_outputs(SwigluBackwardArgs g, const TilePlan& plan, hipStream_t stream) {
    const int64_t M = g.M, N = g.N, O = g.O, P = g.P;
    g.splits = plan.splits;
    g.full = plan.full;
    const int64_t grid_x = tile_grid(step_tiles<STEP_DX>(plan.tile, M, N, O, P), plan.full, plan.splits);
    const int64_t gu = step_tiles<STEP_DGU>(plan.tile, M, N, O, P), dd = step_tiles<STEP_DD>(plan.tile, M, N, O, P);
    const int64_t grid_gu = tile_grid(gu, gu, 1), grid_dd = tile_grid(dd, dd, 1);
    g.from_gu = (uint32_t)grid_x;
    g.from_dd = (uint32_t)(grid_x + grid_gu);
    const int64_t at = grid_x + grid_gu + grid_dd;
    static std::atomic<bool> lds_set[kMaxDevices] = {};
    return launch_kernel<TileSmall>(swiglu_backward_outputs_kernel<TileSmall, kGradF32>, lds_set, g, at, stream);
}

// Whether dh and the gated step go together: few k-tiles on few tiles, where a launch and
// dh's way to memory and back count, against each in the tile and splits that suit it.  The
// way there and back is at 5 TB/s; a k-tile of 128 x 64 is taken as 0.6 of one of 128 x 128.
// Whole calls, apart -> together (* as chosen): 8 x 128 x 512 x 128 18.1 -> 15.3 us *,
// 1013 x 2056 x 1400 x 1992 95.7 -> 87.7 *, 4096 x 256 x 4096 x 256 128 -> 106 *,
// 2048 x 4096 x 1792 x 4096 233 -> 230 *; 1500 x 1000 x 3000 x 1000 120 * -> 123,
// 512 x 4096 x 1792 x 4096 97 * -> 103, 16 x 4096 x 1792 x 4096 55.6 * -> 78.
bool hidden_together(int64_t M, int64_t N, int64_t O, int64_t P) {
    constexpr int k = TILE_SMALL;
    const int64_t tiles = step_tiles<STEP_GATED>(k, M, N, O, P), slots = kTileKinds[k].slots;
    const double each = 0.6 * StepShape<STEP_DH>::depth(M, N, O, P) * tile_us(k, tiles, 0) +
                        StepShape<STEP_GATED>::depth(M, N, O, P) * tile_us(k, tiles, 1);
    return kLaunchUs + 1.0 + (double)((tiles + slots - 1) / slots) * each <
           StepShape<STEP_DH>::plan(M, N, O, P).us + StepShape<STEP_GATED>::plan(M, N, O, P).us +
               (double)M * (double)O * 8e-6 / 5.0;
}

template <bool kGradF32>
hipError_t launch_all(const SwigluBackwardArgs& g, int64_t counters, hipStream_t stream) {
    hipError_t e;
    SwigluBackwardArgs first = g;
    const bool hidden = hidden_together(g.M, g.N, g.O, g.P);
    if (hidden || StepShape<STEP_DH>::plan(g.M, g.N, g.O, g.P).splits == 1) {
        first.clear = counters;
    } else if ((e = launch_zero_f32(reinterpret_cast<float*>(g.count), counters, stream)) != hipSuccess) {
        return e;
    }
    if (hidden) {
        static std::atomic<bool> lds_set[kMaxDevices] = {};
        const int64_t tiles = step_tiles<STEP_GATED>(TILE_SMALL, g.M, g.N, g.O, g.P);
        e = launch_kernel<TileSmall>(swiglu_backward_hidden_kernel<TileSmall>, lds_set, first,
                                     tile_grid(tiles, tiles, 1), stream);
    } else {
        if ((e = launch_step<STEP_DH, false>(first, stream)) != hipSuccess) return e;
        e = launch_step<STEP_GATED, false>(g, stream);
    }
    if (e != hipSuccess) return e;
    const TilePlan together = outputs_plan(g.M, g.N, g.O, g.P);
    if (outputs_together(together, g.M, g.N, g.O, g.P)) return launch_outputs<kGradF32>(g, together, stream);
    if ((e = launch_step<STEP_DX, false>(g, stream)) != hipSuccess) return e;
    if ((e = launch_step<STEP_DGU, kGradF32>(g, stream)) != hipSuccess) return e;
    return launch_step<STEP_DD, kGradF32>(g, stream);
}

// What the steps' joins need at most: they run one after the other.
TilePlan join_need(int64_t M, int64_t N, int64_t O, int64_t P) {
    TilePlan most{0, 1, 0, 0, 0, 0.0};
    const TilePlan plans[] = {StepShape<STEP_DH>::plan(M, N, O, P), StepShape<STEP_GATED>::plan(M, N, O, P),
                              StepShape<STEP_DX>::plan(M, N, O, P), StepShape<STEP_DGU>::plan(M, N, O, P),
                              StepShape<STEP_DD>::plan(M, N, O, P), outputs_plan(M, N, O, P)};
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
    const TilePlan join = M > 0 ? join_need(M, N, O, P) : TilePlan{0, 1, 0, 0, 0, 0.0};
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
    g.full = 0;
    g.clear = 0;
    g.from_gu = g.from_dd = 0;
    return io.grad_f32 ? launch_all<true>(g, L.counters, stream) : launch_all<false>(g, L.counters, stream);
}

}  // namespace ffn
