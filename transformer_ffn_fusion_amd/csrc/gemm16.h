// gemm16.h -- the matrix-product core of the training operators: one output
// tile C[i][j] = sum_k A(i, k) B(j, k) of 16-bit operands (bf16 or fp16) with
// fp32 accumulators, written for the gfx950 matrix instruction
// v_mfma_f32_16x16x32.
//
// Each operand is either k-contiguous (element (i, k) at i * ld + k) or
// k-strided (element (i, k) at k * ld + i), chosen at compile time.  Both are
// staged by direct global->LDS loads in 1 KiB units, in the layouts of
// ffn_device.h: a k-contiguous unit is one 16-index x 32-deep fragment, a
// k-strided one a block of 8 k-rows x 64 indices that the transposing LDS read
// turns into fragments.
//
// Schedule.  A k-tile is 64 deep and cut into four half-tiles: the first and
// second half of A's indices (A0, A1) and of B's (B0, B1).  One k-tile takes
// four phases, each the product of one half-tile pair:
//     phase 0: A0 B0    1: A0 B1    2: A1 B1    3: A1 B0
// A phase reads at most one half-tile from LDS into registers (0: A0, 1: B1,
// 2: A1, 3: the next k-tile's B0) and issues the loads of one half-tile (0:
// A1 of the next k-tile, 1: B0, 2: A0, 3: B1 of the one after that), into the
// place of a half-tile that every wave has read two phases before.  LDS holds
// two k-tiles, so a load has six phases to land: one wait per phase, for all
// but the newest five half-tiles.
//
// Ping-pong.  With eight waves (two per SIMD) the second half of the waves
// runs one barrier behind the first: while one wave of a SIMD multiplies, the
// other reads LDS and issues loads.  Each phase is
//     [LDS reads, loads, wait]  barrier  [products]  barrier
// and the second group passes one more barrier before its first phase, the
// first group one more after its last.
//
// Hazards, by phase number p (a wave's products of p are over before its
// barrier that ends p):
//  * read after load: the wait of phase p - 1 comes before a barrier that every
//    wave passes before any wave's phase-p reads.
//  * load after read: a half-tile read in phase p is loaded over in phase
//    p + 2.  A wave issues in p + 2 after the barrier that ends its p + 1; by
//    then the other group has passed the one that ends its p, and every wave
//    waits for its LDS reads (lgkmcnt 0) before that one.
// K past its end reads zeros in both operands (a k-strided operand through the
// resource's exact size, a k-contiguous one through an offset out of range), so
// values behind the end of a row never meet a product; indices past I or J read
// zeros or other rows and only reach outputs that are not stored.
#pragma once

#include "ffn_device.h"

namespace ffn {

typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));

template <bool kF16>
__device__ __forceinline__ floatx4_t mfma16(const uint4& a, const uint4& b, floatx4_t c) {
    if constexpr (kF16)
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_t, a),
                                                      __builtin_bit_cast(f16x8_t, b), c, 0, 0, 0);
    else
        return mfma16x16x32(a, b, c);
}

constexpr int kTileK = 64;   // depth of a k-tile: two matrix-instruction steps

template <int TI_, int TJ_, int WI_, int WJ_>
struct TileCfg {
    static constexpr int TI = TI_, TJ = TJ_, WI = WI_, WJ = WJ_;
    static constexpr int kWaves = WI * WJ;
    static constexpr int kThreads = 64 * kWaves;
    static constexpr bool kPingPong = kWaves == 8;      // two waves per SIMD
    static constexpr int HI = TI / 2, HJ = TJ / 2;      // indices of a half-tile
    static constexpr int FI = HI / WI / 16, FJ = HJ / WJ / 16;   // a wave's fragments of one
    static constexpr int kHalfA = HI * kTileK * 2, kHalfB = HJ * kTileK * 2;   // bytes
    static constexpr int kBuf = 2 * (kHalfA + kHalfB);
    static constexpr int kLds = 2 * kBuf;
    static constexpr int UA = kHalfA / 1024 / kWaves, UB = kHalfB / 1024 / kWaves;  // loads a wave
    static_assert(HI % 64 == 0 && HJ % 64 == 0, "k-strided operands stage 64-index blocks");
    static_assert(FI * 16 * WI == HI && FJ * 16 * WJ == HJ, "whole fragments per wave");
    static_assert(UA * 1024 * kWaves == kHalfA && UB * 1024 * kWaves == kHalfB,
                  "every wave issues the same loads");
    static_assert(kLds <= 160 * 1024, "LDS budget");
};

// Accumulators of one wave: [A half][B half][fragment of A][fragment of B].
template <class Cfg>
using TileAcc = floatx4_t[2][2][Cfg::FI][Cfg::FJ];

__device__ __forceinline__ void tile_barrier() { asm volatile("s_barrier" ::: "memory"); }
__device__ __forceinline__ void tile_fence() { __builtin_amdgcn_sched_barrier(0); }

// One operand half on its way through k: where the next k-tile starts and how
// many bytes lie between there and the operand's end.
struct HalfWalk {
    uint64_t at;
    int64_t left;
};

// A half starting at index i0 of an operand of n indices and depth K.
template <bool kStrided>
__device__ __forceinline__ HalfWalk half_walk(const uint16_t* p, int64_t ld, int64_t n, int64_t K,
                                              int64_t i0) {
    HalfWalk h;
    const int64_t off = (kStrided ? i0 : i0 * ld) * 2;
    h.at = reinterpret_cast<uint64_t>(p) + (uint64_t)off;
    h.left = (kStrided ? K * ld : n * ld) * 2 - off;
    return h;
}

// What a wave loads of a half-tile of H indices: unit u = wave + W x covers, of
// a k-contiguous operand, fragment u % (H / 16) of k-half u / (H / 16); of a
// k-strided one block (r, c) of k-half u / (H / 16), with u % (H / 16) =
// r (H / 64) + c.
template <bool kStrided, int H, int W, int U>
struct HalfLoads {
    uint32_t off[U];    // byte offsets of this lane's 16 bytes, from the half's place
    uint32_t tail[U];   // the same in the last k-tile: out of range past K

    __device__ __forceinline__ void init(int wave, int lane, int64_t ld, int64_t K) {
        const int rem = (int)(K - (K - 1) / kTileK * kTileK);   // 1 .. 64
#pragma unroll
        for (int x = 0; x < U; ++x) {
            const int u = wave + W * x, kh = u / (H / 16), q = u % (H / 16);
            if constexpr (kStrided) {
                const int r = q / (H / 64), c = q % (H / 64);
                off[x] = (uint32_t)((32 * kh + 8 * r) * ld * 2) + 128u * c +
                         wtile_dma_off(lane, (uint32_t)(ld * 2));
                tail[x] = off[x];
            } else {
                const int k = 32 * kh + 8 * ((lane & 3) ^ ((lane >> 3) & 3));
                off[x] = (uint32_t)((16 * q + (lane >> 2)) * ld * 2) + 2u * k;
                tail[x] = k < rem ? off[x] : kOOB;
            }
        }
    }
    // Loads the k-tile at `h` to `dst` (the half-tile's place in LDS) and moves on.
    __device__ __forceinline__ void issue(HalfWalk& h, int64_t step, bool any, bool last, int wave,
                                          char* dst) const {
        const int32x4_t srd = make_srd(reinterpret_cast<const void*>(h.at), any ? h.left : 0);
#pragma unroll
        for (int x = 0; x < U; ++x)
            dma16(srd, !kStrided && last ? tail[x] : off[x], dst + (wave + W * x) * 1024);
        h.at += (uint64_t)step;
        h.left -= step;
    }
};

// Fragment f (of the half-tile's H / 16) of k-half kh, for this lane.
template <bool kStrided, int H>
__device__ __forceinline__ uint4 half_frag(const char* half, int f, int kh, int lane) {
    const char* st = half + kh * (H / 16) * 1024;
    if constexpr (!kStrided) {
        return ld16(st + f * kFrag + 16 * xfrag_slot(lane & 15, lane >> 4));
    } else {
        const char* p = st + wtile_tr_base(lane, H / 64, f & 3) + 1024 * (f >> 2);
        const uint2 lo = lds_read_tr16(p);
        const uint2 hi = lds_read_tr16(p + 512);
        return make_uint4(lo.x, lo.y, hi.x, hi.y);
    }
}

// The operands of one tile.  A sum over two products with the same depth and
// leading dimensions (C = A B^T + A' B'^T) walks the second pair after the
// first: set `pairs` to 2.
struct TileOps {
    HalfWalk a[2][2], b[2][2];   // [pair][half]
    int64_t lda, ldb;
    int64_t K;                   // depth of each pair, at least 1
    int pairs;
};

// acc += the tile's product.  smem: Cfg::kLds bytes.  Every wave of the
// workgroup calls it; on return the LDS is free and every wave has passed a
// common barrier.
template <class Cfg, bool kAS, bool kBS, bool kF16>
__device__ __forceinline__ void tile_product(char* smem, const TileOps& op, TileAcc<Cfg>& acc) {
    constexpr int FI = Cfg::FI, FJ = Cfg::FJ, UA = Cfg::UA, UB = Cfg::UB;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wi = wave / Cfg::WJ, wj = wave % Cfg::WJ;
    const int per = (int)((op.K + kTileK - 1) / kTileK);   // k-tiles of a pair
    const int nt = per * op.pairs;
    const int64_t step_a = kAS ? op.lda * kTileK * 2 : kTileK * 2;
    const int64_t step_b = kBS ? op.ldb * kTileK * 2 : kTileK * 2;

    HalfLoads<kAS, Cfg::HI, Cfg::kWaves, UA> la;
    HalfLoads<kBS, Cfg::HJ, Cfg::kWaves, UB> lb;
    la.init(wave, lane, op.lda, op.K);
    lb.init(wave, lane, op.ldb, op.K);
    HalfWalk a[2] = {op.a[0][0], op.a[0][1]}, b[2] = {op.b[0][0], op.b[0][1]};

    auto place_a = [&](int t, int h) { return smem + (t & 1) * Cfg::kBuf + h * Cfg::kHalfA; };
    auto place_b = [&](int t, int h) {
        return smem + (t & 1) * Cfg::kBuf + 2 * Cfg::kHalfA + h * Cfg::kHalfB;
    };
    auto load_a = [&](int t, int h) {
        if (t == per) a[h] = op.a[1][h];   // the second pair (or past the end)
        la.issue(a[h], step_a, t < nt, t == per - 1 || t == nt - 1, wave, place_a(t, h));
    };
    auto load_b = [&](int t, int h) {
        if (t == per) b[h] = op.b[1][h];
        lb.issue(b[h], step_b, t < nt, t == per - 1 || t == nt - 1, wave, place_b(t, h));
    };

    uint4 fa[FI][2], fb0[FJ][2], fb1[FJ][2], fbn[FJ][2];
    auto read_a = [&](int t, int h) {
        const char* p = place_a(t, h);
#pragma unroll
        for (int kh = 0; kh < 2; ++kh)
#pragma unroll
            for (int x = 0; x < FI; ++x) fa[x][kh] = half_frag<kAS, Cfg::HI>(p, FI * wi + x, kh, lane);
    };
    auto read_b = [&](int t, int h, uint4 (&f)[FJ][2]) {
        const char* p = place_b(t, h);
#pragma unroll
        for (int kh = 0; kh < 2; ++kh)
#pragma unroll
            for (int y = 0; y < FJ; ++y) f[y][kh] = half_frag<kBS, Cfg::HJ>(p, FJ * wj + y, kh, lane);
    };
    // the middle and the end of a phase: products of the held A half with f
    auto multiply = [&](floatx4_t (&c)[FI][FJ], const uint4 (&f)[FJ][2]) {
        tile_fence();
        tile_barrier();
        tile_fence();
        if constexpr (Cfg::kPingPong) __builtin_amdgcn_s_setprio(1);
#pragma unroll
        for (int kh = 0; kh < 2; ++kh)
#pragma unroll
            for (int x = 0; x < FI; ++x)
#pragma unroll
                for (int y = 0; y < FJ; ++y)
                    // B first: a lane ends with four consecutive output columns of one row
                    c[x][y] = mfma16<kF16>(f[y][kh], fa[x][kh], c[x][y]);
        if constexpr (Cfg::kPingPong) __builtin_amdgcn_s_setprio(0);
        tile_fence();
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        if constexpr (Cfg::kPingPong) tile_barrier();
        tile_fence();
    };

    load_b(0, 0);
    load_a(0, 0);
    load_b(0, 1);
    load_a(0, 1);
    load_b(1, 0);
    load_a(1, 0);
    load_b(1, 1);
    wait_vmcnt<2 * UA + 3 * UB>();
    tile_barrier();
    if (Cfg::kPingPong && wave >= Cfg::kWaves / 2) tile_barrier();
    read_b(0, 0, fb0);
    for (int t = 0; t < nt; ++t) {
        read_a(t, 0);
        load_a(t + 1, 1);
        wait_vmcnt<3 * UA + 2 * UB>();
        multiply(acc[0][0], fb0);
        read_b(t, 1, fb1);
        load_b(t + 2, 0);
        wait_vmcnt<2 * UA + 3 * UB>();
        multiply(acc[0][1], fb1);
        read_a(t, 1);
        load_a(t + 2, 0);
        wait_vmcnt<3 * UA + 2 * UB>();
        multiply(acc[1][1], fb1);
        read_b(t + 1, 0, fbn);   // past the last k-tile: zeros, not used
        load_b(t + 2, 1);
        wait_vmcnt<2 * UA + 3 * UB>();
        multiply(acc[1][0], fb0);
#pragma unroll
        for (int y = 0; y < FJ; ++y) {
            fb0[y][0] = fbn[y][0];
            fb0[y][1] = fbn[y][1];
        }
    }
    wait_vmcnt<0>();
    if (Cfg::kPingPong && wave < Cfg::kWaves / 2) tile_barrier();
    tile_barrier();
}

// First output row (of 16) of A half p's fragment x, and first column of B half
// q's fragment y, within the tile; lane l holds row + l % 16 and the four
// columns from column + 4 (l / 16).
template <class Cfg>
__device__ __forceinline__ int tile_row(int wave, int p, int x) {
    return p * Cfg::HI + 16 * (Cfg::FI * (wave / Cfg::WJ) + x);
}
template <class Cfg>
__device__ __forceinline__ int tile_col(int wave, int q, int y) {
    return q * Cfg::HJ + 16 * (Cfg::FJ * (wave % Cfg::WJ) + y);
}

template <class Cfg>
__device__ __forceinline__ void tile_clear(TileAcc<Cfg>& acc) {
#pragma unroll
    for (int p = 0; p < 2; ++p)
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
            for (int x = 0; x < Cfg::FI; ++x)
#pragma unroll
                for (int y = 0; y < Cfg::FJ; ++y) acc[p][q][x][y] = floatx4_t{0.f, 0.f, 0.f, 0.f};
}

// Workgroup -> output tile.  Workgroups reach the 8 XCDs round-robin and each
// XCD has an L2 of its own: XCD x takes a contiguous run of a grouped order
// (groups of 8 tile rows, rows fastest), a compact rectangle whose panels its
// L2 shares.  Returns false for the padding workgroups.
__host__ __device__ __forceinline__ int64_t tile_grid(int64_t nI, int64_t nJ) {
    return 8 * ((nI * nJ + 7) / 8);
}
__device__ __forceinline__ bool tile_place(int64_t w, int64_t nI, int64_t nJ, int64_t* ti,
                                           int64_t* tj) {
    constexpr int64_t G = 8;
    const int64_t n = nI * nJ, per = (n + 7) / 8;
    const int64_t t = (w & 7) * per + (w >> 3);
    if (t >= n || (w >> 3) >= per) return false;
    const int64_t r = t / (G * nJ);
    const int64_t rows = nI - r * G < G ? nI - r * G : G;
    const int64_t rem = t - r * G * nJ;
    *tj = rem / rows;
    *ti = r * G + rem % rows;
    return true;
}

}  // namespace ffn
