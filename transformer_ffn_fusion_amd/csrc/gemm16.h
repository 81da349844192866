// gemm16.h -- the matrix-product core of the training operators: one output
// tile C[i][j] = sum_k A(i, k) B(j, k) of 16-bit operands (bf16 or fp16) with
// fp32 accumulators, written for the gfx950 matrix instruction
// v_mfma_f32_16x16x32.
//
// Each operand is either k-contiguous (element (i, k) at i * ld + k) or
// k-strided (element (i, k) at k * ld + i), chosen at compile time.  Both are
// staged by direct global->LDS loads; a k-strided one becomes fragments through
// the transposing LDS read.
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
//
// Bound: of a 256 x 256 tile's k-tile the matrix instructions take 2048 clocks
// and so do the LDS reads (1536) and the loads' writes (512) at 128 B per clock;
// 2235 measured.  8192 x 8192 x 8192 bf16: 729 us, 1500 TFLOP/s at the 1.9 GHz
// that the card holds under this load.
//
// K past its end reads zeros in both operands, of either kind: in the last k-tile the
// lanes whose k lies past K (HalfLoads::past) load from an offset out of range, so
// values behind the end of a row or a matrix never meet a product.  Indices past I or
// J read zeros in the same way (HalfLoads::off) and only reach outputs that are not
// stored.
#pragma once

#include <type_traits>

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

// One operand of a tile: its first element, leading dimension and index count,
// and the first index of each half-tile.
struct TileOperand {
    const uint16_t* p;
    int64_t ld, n;
    int64_t at[2];
};

// Direct load of 16 bytes per lane from `base` + the lane's offset to LDS address
// `lds` (+ 16 per lane); past the end (`any` false) or out of range it brings
// zeros and reads no memory.  Every lane's offset is in bounds or kOOB, so the
// resource's size only has to refuse kOOB.
__device__ __forceinline__ void tile_dma(uint64_t base, bool any, uint32_t off, uint32_t lds) {
    int32x4_t srd;
    srd.x = (int)(uint32_t)base;
    srd.y = (int)(uint32_t)(base >> 32);
    srd.z = any ? 0x7fffffff : 0;
    srd.w = kRsrcWord3;
    asm volatile(
        "s_mov_b32 m0, %0\n\t"
        "s_nop 0\n\t"   // a wait state between writing M0 and a load to LDS
        "buffer_load_dwordx4 %1, %2, 0 offen lds"
        :
        : "s"(lds), "v"(off), "s"(srd)
        : "m0");
}

// LDS layouts of a half-tile (H indices x 64 k), in 1 KiB units whose slot l (16
// bytes) is written by lane l of the loading wave.  LDS serves 256 bytes a cycle.
//
//  k-contiguous: unit q holds indices 8q .. 8q + 7, a whole 128-byte line of each;
//  the 8-deep k-group c of index r lies in slot 8r + (c ^ r).  A fragment read
//  takes k-group 4 kh + lane / 16 of index lane % 16 = 8q + r: 8 lanes with the
//  same k-group fill the 8 slots' columns, no bank conflicts.  (Units of 16
//  indices x 32 k, which read half lines, measured the same.)
//
//  k-strided: unit (kh, g, c) holds k-rows 32 kh + 8 g .. + 7 and indices 64 c ..
//  64 c + 63, 128 contiguous bytes a row; the 8-index group u of row r lies in
//  slot 8r + (u ^ 2 (r + g) mod 8).  One transposing read takes, per 16 lanes, 4
//  rows x 2 neighbouring groups; with the row in the swizzle the 16 lanes cover
//  half of the 256 bytes, with the parity of g the next 16 lanes the other half.
__device__ __forceinline__ int strided_swizzle(int r, int g) { return 2 * (r ^ (g & 1)) & 7; }

// What a wave loads of a half-tile: units wave, wave + W, ...
template <bool kStrided, int H, int W, int U>
struct HalfLoads {
    static_assert(!kStrided || H % 64 == 0, "k-strided operands stage 64-index blocks");
    uint32_t off[2][U];   // this lane's byte offset from the k-tile, per half; kOOB past the indices
    bool past[U];         // in the last k-tile: past K
    uint64_t base[2];     // where each half's next k-tile starts

    __device__ __forceinline__ void init(const TileOperand& o, int64_t K, int wave, int lane) {
        const int rem = (int)(K - (K - 1) / kTileK * kTileK);   // 1 .. 64
#pragma unroll
        for (int x = 0; x < U; ++x) {
            const int u = wave + W * x, r = lane >> 3;
            int i, k;   // this lane's first index and k, in the half-tile
            uint32_t at;
            if constexpr (kStrided) {
                const int kh = u / (H / 16), g = u % (H / 16) / (H / 64), c = u % (H / 64);
                i = 64 * c + 8 * ((lane & 7) ^ strided_swizzle(r, g));
                k = 32 * kh + 8 * g + r;
                at = (uint32_t)k * (uint32_t)(o.ld * 2) + 2u * i;
            } else {
                i = 8 * u + r;
                k = 8 * ((lane & 7) ^ r);
                at = (uint32_t)i * (uint32_t)(o.ld * 2) + 2u * k;
            }
            past[x] = k >= rem;
#pragma unroll
            for (int h = 0; h < 2; ++h) off[h][x] = o.at[h] + i < o.n ? at : kOOB;
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) start(o.p, o.ld, o.at[h], h);
    }
    __device__ __forceinline__ void start(const uint16_t* p, int64_t ld, int64_t at, int h) {
        const uint64_t b = reinterpret_cast<uint64_t>(p + (kStrided ? at : at * ld));
        base[h] = (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)b) |
                  (uint64_t)((uint32_t)__builtin_amdgcn_readfirstlane((int)(b >> 32)) & 0xffffu) << 32;
    }
    // Loads half h's next k-tile to `lds` and moves on by `step` bytes.
    __device__ __forceinline__ void issue(int h, bool any, bool last, uint64_t step, int wave,
                                          uint32_t lds) {
#pragma unroll
        for (int x = 0; x < U; ++x)
            tile_dma(base[h], any, last && past[x] ? kOOB : off[h][x], lds + (wave + W * x) * 1024);
        base[h] += step;
    }
};

// Fragment f (of the half-tile's H / 16) of k-half kh, for this lane.
template <bool kStrided, int H>
__device__ __forceinline__ uint4 half_frag(const char* half, int f, int kh, int lane) {
    const int g = lane >> 4;
    if constexpr (!kStrided) {
        const int i = lane & 15, r = i & 7;
        return ld16(half + f * 2048 + (i >> 3) * 1024 + r * 128 + 16 * ((4 * kh + g) ^ r));
    } else {
        // the 8-byte chunk this lane supplies: row j of the read's four, 8-index group
        // 2f + q / 2, half q % 2 of it; the second read takes rows j + 4
        const int j = (lane & 15) >> 2, q = lane & 3;
        const char* p = half + (kh * (H / 16) + g * (H / 64) + (f >> 2)) * 1024 + 128 * j +
                        16 * ((2 * (f & 3) + (q >> 1)) ^ strided_swizzle(j, g)) + 8 * (q & 1);
        const uint2 lo = lds_read_tr16(p);
        const uint2 hi = lds_read_tr16(p + 512);   // (j + 4 swizzles as j does)
        return make_uint4(lo.x, lo.y, hi.x, hi.y);
    }
}

// acc += A B^T over depth K (at least 1), and with kPairs = 2 + A' B'^T of the same
// depth, leading dimensions and indices, A' and B' starting at a2 and b2 (for halves
// of one operand that lie in two matrices, b_half2 is where the second half's
// operand starts; else null).  smem: Cfg::kLds bytes.  Every wave of the workgroup
// calls it; on return the LDS is free and every wave has passed a common barrier.
// The k-tiles t0 <= t < t1 of the ceil(K / 64) kPairs there are (t0 < t1).
template <class Cfg, bool kAS, bool kBS, bool kF16, int kPairs>
__device__ __forceinline__ void tile_product(char* smem, const TileOperand& A, const TileOperand& B,
                                             int64_t K, const uint16_t* a2, const uint16_t* b2,
                                             const uint16_t* b_half2, int t0, int t1,
                                             TileAcc<Cfg>& acc) {
    constexpr int FI = Cfg::FI, FJ = Cfg::FJ, UA = Cfg::UA, UB = Cfg::UB;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wi = wave / Cfg::WJ, wj = wave % Cfg::WJ;
    const int per = (int)((K + kTileK - 1) / kTileK);   // k-tiles of a pair
    const int nt = per * kPairs;
    const uint64_t step_a = (uint64_t)(kAS ? A.ld * kTileK * 2 : kTileK * 2);
    const uint64_t step_b = (uint64_t)(kBS ? B.ld * kTileK * 2 : kTileK * 2);
    const uint32_t lds0 = (uint32_t)(uintptr_t)((lds_void_t*)smem);

    HalfLoads<kAS, Cfg::HI, Cfg::kWaves, UA> la;
    HalfLoads<kBS, Cfg::HJ, Cfg::kWaves, UB> lb;
    la.init(A, K, wave, lane);
    lb.init(B, K, wave, lane);
    if (b_half2) lb.start(b_half2, B.ld, B.at[1], 1);
    if (kPairs == 2 && t0 >= per) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            la.start(a2, A.ld, A.at[h], h);
            lb.start(b2, B.ld, B.at[h], h);
        }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        la.base[h] += step_a * (uint64_t)(t0 >= per ? t0 - per : t0);
        lb.base[h] += step_b * (uint64_t)(t0 >= per ? t0 - per : t0);
    }

    // k-tile t lies in LDS buffer (t - t0) % 2, `buf` below
    auto load_a = [&](int t, int buf, int h) {
        if (kPairs == 2 && t == per && t > t0) la.start(a2, A.ld, A.at[h], h);
        la.issue(h, t < t1, t == nt - 1 || (kPairs == 2 && t == per - 1), step_a, wave,
                 lds0 + buf * Cfg::kBuf + h * Cfg::kHalfA);
    };
    auto load_b = [&](int t, int buf, int h) {
        if (kPairs == 2 && t == per && t > t0) lb.start(b2, B.ld, B.at[h], h);
        lb.issue(h, t < t1, t == nt - 1 || (kPairs == 2 && t == per - 1), step_b, wave,
                 lds0 + buf * Cfg::kBuf + 2 * Cfg::kHalfA + h * Cfg::kHalfB);
    };

    uint4 fa[FI][2], fb[FJ][2], fb0[2][FJ][2];   // fb0: B0 of the even and of the odd k-tiles
    auto read_a = [&](int buf, int h) {
        const char* p = smem + buf * Cfg::kBuf + h * Cfg::kHalfA;
#pragma unroll
        for (int kh = 0; kh < 2; ++kh)
#pragma unroll
            for (int x = 0; x < FI; ++x) fa[x][kh] = half_frag<kAS, Cfg::HI>(p, FI * wi + x, kh, lane);
    };
    auto read_b = [&](int buf, int h, uint4 (&f)[FJ][2]) {
        const char* p = smem + buf * Cfg::kBuf + 2 * Cfg::kHalfA + h * Cfg::kHalfB;
#pragma unroll
        for (int kh = 0; kh < 2; ++kh)
#pragma unroll
            for (int y = 0; y < FJ; ++y) f[y][kh] = half_frag<kBS, Cfg::HJ>(p, FJ * wj + y, kh, lane);
    };
    // the middle and the end of a phase: products of the held A half with f
    auto multiply = [&](floatx4_t (&c)[FI][FJ], const uint4 (&f)[FJ][2]) {
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
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
        if constexpr (Cfg::kPingPong) tile_barrier();
        tile_fence();
    };
    // the four phases of k-tile t, which lies in buffer `buf`
    auto k_tile = [&](int t, int buf) __attribute__((always_inline)) {
        read_a(buf, 0);
        tile_fence();
        load_a(t + 1, buf ^ 1, 1);
        wait_vmcnt<3 * UA + 2 * UB>();
        multiply(acc[0][0], fb0[buf]);
        read_b(buf, 1, fb);
        tile_fence();
        load_b(t + 2, buf, 0);
        wait_vmcnt<2 * UA + 3 * UB>();
        multiply(acc[0][1], fb);
        read_a(buf, 1);
        tile_fence();
        load_a(t + 2, buf, 0);
        wait_vmcnt<3 * UA + 2 * UB>();
        multiply(acc[1][1], fb);
        read_b(buf ^ 1, 0, fb0[buf ^ 1]);   // past the last k-tile: zeros, not used
        tile_fence();
        load_b(t + 2, buf, 1);
        wait_vmcnt<2 * UA + 3 * UB>();
        multiply(acc[1][0], fb0[buf]);
    };

    load_b(t0, 0, 0);
    load_a(t0, 0, 0);
    load_b(t0, 0, 1);
    load_a(t0, 0, 1);
    load_b(t0 + 1, 1, 0);
    load_a(t0 + 1, 1, 0);
    load_b(t0 + 1, 1, 1);
    wait_vmcnt<2 * UA + 3 * UB>();
    tile_barrier();
    if (Cfg::kPingPong && wave >= Cfg::kWaves / 2) tile_barrier();
    read_b(0, 0, fb0[0]);
    // two k-tiles a turn, so that every LDS place is a constant; an odd count is
    // made even with a k-tile of zeros
    for (int t = t0; t < t1; t += 2) {
        k_tile(t, 0);
        k_tile(t + 1, 1);
    }
    wait_vmcnt<0>();
    if (Cfg::kPingPong && wave < Cfg::kWaves / 2) tile_barrier();
    tile_barrier();
}

// The way out: the sums go through LDS, the whole tile where it fits and else its
// two halves of Cfg::HI rows after each other, so that a thread gets eight
// consecutive columns of a row (16 bytes of bf16 or fp16, whole lines per wave) and
// the epilogue is a short loop.  (Straight from the accumulators every fragment's
// epilogue is code of its own, and the stores are half lines: the outer product of
// a 4096 x 1792 update 40 -> 32 us.)  The 16-byte chunk c of row r lies at chunk
// c ^ ((r ^ r / 8) mod 16): writes (16 rows, one column), reads along a row and
// reads along a column meet 16 different chunks.
template <class Cfg>
struct PartOf {
    static constexpr int kParts = Cfg::TI * Cfg::TJ * 4 <= Cfg::kLds ? 1 : 2;
    static constexpr int kRows = Cfg::TI / kParts;
    static_assert(kRows * Cfg::TJ * 4 <= Cfg::kLds, "a part fits the LDS");
};
template <class Cfg>
__device__ __forceinline__ uint32_t part_off(int row, int chunk) {
    return (uint32_t)row * (Cfg::TJ * 4) + 16u * (uint32_t)(chunk ^ ((row ^ (row >> 3)) & 15));
}
template <class Cfg>
__device__ __forceinline__ void part_put(char* smem, const TileAcc<Cfg>& acc, int part) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int wi = wave / Cfg::WJ, wj = wave % Cfg::WJ;
#pragma unroll
    for (int p = 0; p < 2; ++p) {
        if (PartOf<Cfg>::kParts == 2 && p != part) continue;
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
            for (int x = 0; x < Cfg::FI; ++x)
#pragma unroll
                for (int y = 0; y < Cfg::FJ; ++y)
                    *reinterpret_cast<floatx4_t*>(
                        smem + part_off<Cfg>((PartOf<Cfg>::kParts == 2 ? 0 : p * Cfg::HI) +
                                                 16 * (Cfg::FI * wi + x) + (lane & 15),
                                             (q * Cfg::HJ + 16 * (Cfg::FJ * wj + y)) / 4 + (lane >> 4))) =
                        acc[p][q][x][y];
    }
}
// A thread's share of a part with kCols columns: the 8-column group `c` of every
// kStep-th row from `row0`, kUnits rows.  kStep is 16, 32 or 64 and row0 below it, so in
// a row k steps on, the swizzle differs from row0's by an exclusive-or with a
// constant: one instruction per LDS access.
template <class Cfg, int kCols>
struct PartThread {
    static constexpr int kStep = Cfg::kThreads / (kCols / 8);
    static constexpr int kUnits = PartOf<Cfg>::kRows / kStep;
    static_assert(kStep >= 16 && (kStep & (kStep - 1)) == 0 && kUnits * kStep == PartOf<Cfg>::kRows, "whole rows");
    int c, row0;
    __device__ __forceinline__ PartThread() {
        c = threadIdx.x % (kCols / 8);
        row0 = threadIdx.x / (kCols / 8);
    }
    // place of chunk `chunk` of row row0, to be stepped by `at`
    __device__ __forceinline__ uint32_t place(int chunk) const {
        return 16u * (uint32_t)(chunk ^ ((row0 ^ (row0 >> 3)) & 15));
    }
    __device__ __forceinline__ uint32_t at(uint32_t place, int k) const {
        return (uint32_t)(row0 + k * kStep) * (Cfg::TJ * 4) + (place ^ (16u * ((kStep / 8 * k) & 15)));
    }
    // eight columns of row row0 + k kStep, from the group whose first chunk is at `place`
    __device__ __forceinline__ void get(const char* smem, uint32_t place, int k, float (&v)[8]) const {
        const floatx4_t a = *reinterpret_cast<const floatx4_t*>(smem + at(place, k));
        const floatx4_t b = *reinterpret_cast<const floatx4_t*>(smem + at(place ^ 16u, k));
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            v[r] = a[r];
            v[4 + r] = b[r];
        }
    }
    __device__ __forceinline__ void set(char* smem, uint32_t place, int k, const float (&v)[8]) const {
        *reinterpret_cast<floatx4_t*>(smem + at(place, k)) = floatx4_t{v[0], v[1], v[2], v[3]};
        *reinterpret_cast<floatx4_t*>(smem + at(place ^ 16u, k)) = floatx4_t{v[4], v[5], v[6], v[7]};
    }
};
// Eight rows from row 8 r of a column.
template <class Cfg>
__device__ __forceinline__ void part_get_column(const char* smem, int r, int col, float (&v)[8]) {
    const uint32_t base = (uint32_t)r * (8 * Cfg::TJ * 4) + 4u * (col & 3);
    const uint32_t x = 16u * (uint32_t)((col >> 2) ^ ((8 * (r & 1) ^ r) & 15));
#pragma unroll
    for (int k = 0; k < 8; ++k)
        v[k] = *reinterpret_cast<const float*>(smem + base + k * (Cfg::TJ * 4) + (x ^ (16u * k)));
}

// What the epilogue reads per row of a thread, for every row of the tile.  The small
// and mid tiles have registers left to load it before the products (kEarly: its
// latency, 1 to 2 us, is hidden); the large tile loads four rows at a time after them.
//
// The callbacks get a row as its distance `off` from the thread's first row, the same
// for all threads: with a pointer to the first row, off * leading dimension is scalar
// arithmetic.
template <class Cfg, int kCols, class State>
struct PartStates {
    static constexpr bool kEarly = Cfg::FI * Cfg::FJ <= 4 && !std::is_empty<State>::value;
    static constexpr int kUnits = PartThread<Cfg, kCols>::kUnits, kStep = PartThread<Cfg, kCols>::kStep;
    static constexpr int kGroup = kUnits < 4 ? kUnits : 4;
    static_assert(kUnits % kGroup == 0, "whole groups");
    State early[kEarly ? PartOf<Cfg>::kParts : 1][kEarly ? kUnits : 1];

    // before(off, state) for rows below `rows`
    template <class Before>
    __device__ __forceinline__ void load(const PartThread<Cfg, kCols>& t, int rows, Before&& before) {
        if constexpr (kEarly) {
#pragma unroll
            for (int p = 0; p < PartOf<Cfg>::kParts; ++p)
#pragma unroll
                for (int k = 0; k < kUnits; ++k) {
                    const int off = p * PartOf<Cfg>::kRows + k * kStep;
                    if (t.row0 + off < rows) before(off, early[p][k]);
                }
        }
    }
    // after(off, k, values, state) for the rows of part p below `rows`; values[g]: the
    // eight sums at places[g]
    template <int kGets, class Before, class After>
    __device__ __forceinline__ void each(const char* smem, const PartThread<Cfg, kCols>& t,
                                         const uint32_t (&places)[kGets], int p, int rows,
                                         Before&& before, After&& after) {
        auto group = [&](int u, State* st) __attribute__((always_inline)) {
            float v[kGroup][kGets][8];
#pragma unroll
            for (int k = 0; k < kGroup; ++k)
#pragma unroll
                for (int g = 0; g < kGets; ++g) t.get(smem, places[g], u + k, v[k][g]);
#pragma unroll
            for (int k = 0; k < kGroup; ++k) {
                const int off = p * PartOf<Cfg>::kRows + (u + k) * kStep;
                if (t.row0 + off < rows) after(off, u + k, v[k], st[k]);
            }
        };
        if constexpr (kEarly) {
#pragma unroll
            for (int u = 0; u < kUnits; u += kGroup) group(u, &early[p][u]);
        } else {
#pragma unroll 1
            for (int u = 0; u < kUnits; u += kGroup) {
                State st[kGroup];
#pragma unroll
                for (int k = 0; k < kGroup; ++k) {
                    const int off = p * PartOf<Cfg>::kRows + (u + k) * kStep;
                    if (t.row0 + off < rows) before(off, st[k]);
                }
                group(u, st);
            }
        }
    }
};

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

// Work of one launch: nI x nJ output tiles (kTri: the lower triangle of a square
// of nI x nI).  The first `full` tiles are a workgroup's each; each of the others is
// cut into `splits` ranges of k-tiles: all of them where there are few, or those that
// would leave a last round of the CUs half empty.  Workgroups reach the 8 XCDs
// round-robin and each XCD has an L2 of its own: XCD x takes a contiguous run of a
// grouped order (groups of 8 tile rows, rows fastest; a tile's splits side by side), a
// compact rectangle whose panels its L2 shares.
struct TilePlace {
    int ti, tj;
    int split, splits;   // which part of the tile's depth, of how many
    int joint;           // the tile's number among the split ones
};
__host__ __device__ __forceinline__ int64_t tile_count(int64_t nI, int64_t nJ, bool tri) {
    return tri ? nI * (nI + 1) / 2 : nI * nJ;
}
__host__ __device__ __forceinline__ int64_t tile_grid(int64_t tiles, int64_t full, int splits) {
    return 8 * ((full + 7) / 8 + ((tiles - full) * splits + 7) / 8);
}
// Returns false for the padding workgroups.  (32-bit arithmetic: six 64-bit
// divisions took 0.5 us of every launch.)
template <bool kTri>
__device__ __forceinline__ bool tile_place(uint32_t w, uint32_t nI, uint32_t nJ, uint32_t full,
                                           uint32_t splits, TilePlace* at) {
    constexpr uint32_t G = 8;
    const uint32_t tiles = kTri ? nI * (nI + 1) / 2 : nI * nJ;
    if (full > tiles) full = tiles;
    const uint32_t grid = (full + 7) / 8 * 8;
    const bool part = w >= grid;
    if (part) w -= grid;
    const uint32_t n = part ? (tiles - full) * splits : full, per = (n + 7) / 8;
    const uint32_t u = (w & 7) * per + (w >> 3);
    if (u >= n || (w >> 3) >= per) return false;
    uint32_t t = u;
    at->split = 0;
    at->splits = 1;
    at->joint = 0;
    if (part && splits > 1) {
        const uint32_t q = u / splits;
        at->split = (int)(u - q * splits);
        at->splits = (int)splits;
        at->joint = (int)q;
        t = full + q;
    }
    if constexpr (kTri) {
        uint32_t r = (uint32_t)((sqrtf(8.0f * (float)t + 1.0f) - 1.0f) * 0.5f);
        if (r * (r + 1) / 2 > t) --r;   // the root is off by one at most
        if ((r + 1) * (r + 2) / 2 <= t) ++r;
        at->ti = (int)r;
        at->tj = (int)(t - r * (r + 1) / 2);
    } else {
        const uint32_t r = t / (G * nJ);
        const uint32_t rows = nI - r * G < G ? nI - r * G : G;
        const uint32_t rem = t - r * G * nJ;
        const uint32_t tj = rem / rows;
        at->tj = (int)tj;
        at->ti = (int)(r * G + rem - tj * rows);
    }
    return true;
}

// The join of a tile's splits.  Each split's workgroup writes its sums, raises the
// tile's counter, and the one that finds itself last adds all of them in ascending
// split order (so the result does not depend on who is last) and goes on to the
// epilogue; the others are done.  No workgroup waits for another.
//
// The sums cross XCDs, whose L2s are not coherent with each other: they are
// written through to memory (sc0 sc1) and have arrived there (vmcnt 0 in every
// wave, then the barrier) before the counter is raised, and the last workgroup
// reads them with loads that do not stop at its L2 either.  A device-scope release
// fence would write back the XCD's whole L2 instead.
//
// part: splits x (TI * TJ) floats of this tile; count: the tile's counter, 0 before
// the first and again after the last split; rows: the tile's rows that are wanted
// (fragments past them are left out).  Returns whether to go on, with acc the sum.
// smem is used for one word.
constexpr int kCpolThrough = 17;   // buffer cache-policy bits sc0, sc1: system scope

template <class Cfg>
__device__ __forceinline__ bool tile_join(char* smem, float* part, uint32_t* count, int split,
                                          int splits, int rows, TileAcc<Cfg>& acc) {
    constexpr uint32_t kBytes = (uint32_t)Cfg::TI * Cfg::TJ * 4;
    const __amdgpu_buffer_rsrc_t rs = make_rsrc(part, (int64_t)kBytes * splits);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), wi = wave / Cfg::WJ;
    auto wanted = [&](int p, int x) { return p * Cfg::HI + 16 * (Cfg::FI * wi + x) < rows; };
    auto off = [&](int p, int x, int k) {   // k: fragment (q, y) of the block row
        return (uint32_t)(((p * Cfg::FI + x) * 2 * Cfg::FJ + k) * (Cfg::kThreads * 16)) + threadIdx.x * 16u;
    };
    // The split's place is added to the lane's offset, not given as the instruction's scalar
    // offset: with that, the compiler lets the next instruction overwrite the first of a
    // 16-byte store's registers, and now and then the overwritten word is what arrives.
    const uint32_t mine = kBytes * (uint32_t)split;
#pragma unroll
    for (int p = 0; p < 2; ++p)
#pragma unroll
        for (int x = 0; x < Cfg::FI; ++x) {
            if (!wanted(p, x)) continue;
#pragma unroll
            for (int k = 0; k < 2 * Cfg::FJ; ++k)
                __builtin_amdgcn_raw_buffer_store_b128(
                    __builtin_bit_cast(__attribute__((ext_vector_type(4))) unsigned int,
                                       acc[p][k / Cfg::FJ][x][k % Cfg::FJ]),
                    rs, mine + off(p, x, k), 0, kCpolThrough);
        }
    wait_vmcnt<0>();
    __syncthreads();
    uint32_t* last = reinterpret_cast<uint32_t*>(smem);
    if (threadIdx.x == 0) {
        const uint32_t before = __hip_atomic_fetch_add(count, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        *last = before == (uint32_t)splits - 1;
        if (*last) __hip_atomic_store(count, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    __syncthreads();
    const bool go = *last != 0;
    __syncthreads();   // the word is free again
    if (!go) return false;
    tile_clear<Cfg>(acc);
    // ascending split order; each turn's loads are in flight together
    constexpr int kHalves = Cfg::FI * Cfg::FJ <= 4 ? 2 : 1;   // of the tile at once: registers
    constexpr int kRow = 2 * Cfg::FJ;
#pragma unroll
    for (int p0 = 0; p0 < 2; p0 += kHalves)
#pragma unroll 1
        for (int s = 0; s < splits; ++s) {
            floatx4_t v[kHalves][Cfg::FI][kRow];
#pragma unroll
            for (int p = 0; p < kHalves; ++p)
#pragma unroll
                for (int x = 0; x < Cfg::FI; ++x)
                    if (wanted(p0 + p, x))
#pragma unroll
                        for (int k = 0; k < kRow; ++k)
                            v[p][x][k] = __builtin_bit_cast(
                                floatx4_t, __builtin_amdgcn_raw_buffer_load_b128(
                                               rs, off(p0 + p, x, k), (int)(kBytes * (uint32_t)s), kCpolThrough));
#pragma unroll
            for (int p = 0; p < kHalves; ++p)
#pragma unroll
                for (int x = 0; x < Cfg::FI; ++x)
                    if (wanted(p0 + p, x))
#pragma unroll
                        for (int k = 0; k < kRow; ++k)
                            acc[p0 + p][k / Cfg::FJ][x][k % Cfg::FJ] += v[p][x][k];
        }
    return true;
}

// ---- host side: which tile, how many splits

using TileLarge = TileCfg<256, 256, 2, 4>;   // eight waves, one workgroup per CU
using TileMid = TileCfg<256, 128, 4, 2>;     // eight waves, one workgroup per CU
using TileSmall = TileCfg<128, 128, 2, 2>;   // four waves, two workgroups per CU

enum { TILE_LARGE = 0, TILE_MID = 1, TILE_SMALL = 2 };
struct TilePlan {
    int tile, splits;
    int64_t full;                    // of one matrix's tiles: those that are not split
    int64_t part_floats, counters;   // workspace of the join (0 without splits)
    double us;                       // estimated time
};

// Measured on 256 CUs, k-contiguous bf16, in microseconds: per k-tile with few and
// with all CUs at work (large 0.95 to 1.4, mid 0.54 to 0.87, small 0.43 to 0.55
// alone on a CU and 0.6 to 0.95 two on one); beside them a launch takes about 4.5.  A
// join costs (large) 5.5 + 2.7 a split, (mid) 3 + 1.35, (small) 2 + 1 -- the last
// workgroup reads every split's sums alone, at about 0.1 MB/us -- and 0.2 per MB that
// all tiles' splits write, less where few of a tile's rows are wanted.
struct TileKind {
    int ti, tj, slots;
    double join, join_split;
};
constexpr TileKind kTileKinds[3] = {{256, 256, 256, 5.5, 2.7}, {256, 128, 256, 3.0, 1.35}, {128, 128, 512, 2.0, 1.0}};
constexpr double kLaunchUs = 4.5;
// per k-tile, with `units` workgroups at work and `strided` k-strided operands (whose
// reads are twice as many instructions: the mid tile's short phases do not hide them)
inline double tile_us(int kind, int64_t units, int strided) {
    const double slots = kTileKinds[kind].slots, busy = (double)units < slots ? (double)units / slots : 1.0;
    return kind == TILE_LARGE ? 0.95 + 0.45 * busy
           : kind == TILE_MID ? (0.54 + 0.33 * busy) * (1.0 + 0.13 * strided)
           : busy <= 0.5      ? 0.43 + 0.24 * busy
                              : 0.6 + 0.35 * busy;
}
inline int64_t tile_tiles(int kind, int64_t I, int64_t J, int share, bool tri) {
    const int64_t wi = kTileKinds[kind].ti, wj = kTileKinds[kind].tj / share;
    return tile_count((I + wi - 1) / wi, (J + wj - 1) / wj, tri);
}
inline double join_us(int kind, int64_t I, int64_t tiles, int64_t s) {
    const TileKind& k = kTileKinds[kind];
    const double rows = I < k.ti ? (double)((I + 15) / 16 * 16) / k.ti : 1.0;
    return k.join + rows * ((double)s * k.join_split + 0.2 * (double)(tiles * s) * k.ti * k.tj * 4e-6);
}

// The plan with the least estimated time for an I x J output (J in the tile's terms:
// `share` operand columns of a tile belong to one output column) of `nt` k-tiles,
// `batch` times.
inline TilePlan tile_plan(int64_t I, int64_t J, int share, int64_t nt, int64_t batch, bool tri,
                          int strided) {
    TilePlan best{TILE_LARGE, 1, 0, 0, 0, 1e30};
    for (int k = 0; k < 3; ++k) {
        if (tri && kTileKinds[k].ti != kTileKinds[k].tj) continue;
        const int64_t slots = kTileKinds[k].slots, each = tile_tiles(k, I, J, share, tri), tiles = batch * each;
        for (int64_t s = 1; s <= 16 && s <= nt; ++s) {
            const int64_t depth = (nt + s - 1) / s;
            if ((nt + depth - 1) / depth != s) continue;   // an empty last split
            // whole rounds of the CUs stay unsplit; what is split is one round at most
            const int64_t full = s == 1 ? tiles : tiles / slots * slots, rest = tiles - full;
            if (s > 1 && (rest == 0 || rest * s > slots || (full && batch > 1))) continue;
            double t = kLaunchUs + (double)((full + slots - 1) / slots * nt) * tile_us(k, full, strided);
            if (s > 1) t += (double)depth * tile_us(k, rest * s, strided) + join_us(k, I, rest, s);
            if (t < best.us) {
                best.us = t;
                best.tile = k;
                best.splits = (int)s;
                best.full = s == 1 ? each : full;
                best.part_floats = s > 1 ? rest * s * (int64_t)kTileKinds[k].ti * kTileKinds[k].tj : 0;
                best.counters = s > 1 ? rest : 0;
            }
        }
    }
    return best;
}

}  // namespace ffn
