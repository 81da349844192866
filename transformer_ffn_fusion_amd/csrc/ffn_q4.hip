// ffn_q4.hip -- products of few rows with 4-bit weights and group scales: one
// matrix, the gated pair of SwiGLU, and both over the experts' row lists.
//
//   W[k][c] = (q - z) s  (4-bit integers; z = 8 without zero points)  or  e2m1(q) s,
//   one s (and z) per column and group of 32, 64 or 128 k
//   Y = act(X W + b)   or   H = silu(X Wg) * (X Wu);   X, Y bf16, sums fp32
//
// Bound: the HBM time of the codes -- every weight is used for up to 16 rows only, or 32.
//  * The packed layout is the matrix instruction's operand: a tile of 16 columns x 128 k
//    is 64 lanes x 16 bytes in lane order, so a wave loads 1 KiB at once and no value
//    changes lanes.  Lane l's word j holds the 8 codes of column l % 16, k = 32 j +
//    8 (l / 16) + 0..7.
//  * A code becomes bf16 by one shift and one and-or for two integers (the code in the
//    upper mantissa bits of 16: 16 + q) or one conversion for two e2m1 floats; both are
//    exact.  The group's sum x (16 + q) is corrected by (16 + z) sum x, which one more
//    matrix instruction against ones gives in the same registers, and scaled in fp32.
//    (An x far above its group's others leaves a rounding there, 2^-16 |x| s, that the direct
//    form does not.  That form, q - z by fp16 mantissas and one mixed fma a code, takes 17
//    instructions per 8 codes instead of 8 and 23 to 50 % longer: the pair of 8192 x 3584
//    12.8 us instead of 9.3, 8192 x 28672 40.6 instead of 29.6.)
//  * The waves of a workgroup share its columns and split K; their sums are joined in
//    LDS in ascending order, so results do not depend on timing, and one launch is all.
// Measured (replayed in a graph; 16 tokens unless said; cards differ by up to 5 %): pair of
// 8192 x 3584 9.1 to 9.6 us (30.3 MB; without its loads of X 1 us less), experts' pairs of
// 8 x 4096 x 2048 13.6 us (8.65 MB an expert; inputs of which six, eight and six have rows),
// 8192 x 28672 29 to 30 us (121 MB; one token 25.4), 4096 x 4096 with zero points, one token, 4.2 us,
// of which about 3 are a kernel's way in and out.
// Three stages in flight instead of two: slower (16 x 4096 x 4096: 5.0 us, 6.3; 16 x 14336 x
// 4096: 11.0, 12.0), and so are sixteen waves.
#include <type_traits>

#include "ffn_device.h"
#include "sublayer.h"

namespace ffn {

namespace {

constexpr int kMaxWaves = 8;
constexpr int kBlockLds = kQ4Rows * kQ4TileK * 2;  // a wave's 16 rows of one tile, then its sums
enum { kQ4Int = 0, kQ4E2m1 = 1 };

struct Q4Args {
    const uint16_t* X;
    const char* W[2];
    const char* S[2];
    const char* Z[2];      // null: 8 (integers) or none (e2m1)
    const uint16_t* bias;
    uint16_t* Y;
    const int32_t* offsets;
    int64_t K, C;
    int64_t w_stride, s_stride, b_stride;   // per expert: bytes, bytes, elements
    int rows;
    int kt;                                 // tiles along K
    int act;
};

// The mask of decode8, in a vector register: beside the base in a scalar one it lets the
// and and the or be one instruction.
__device__ __forceinline__ uint32_t code_mask() {
    uint32_t m = 0x00780078u;
    asm("" : "+v"(m));
    return m;
}
__device__ __forceinline__ uint4 decode8(uint32_t w, uint32_t mask, std::integral_constant<int, kQ4Int>) {
    // nibbles i and i + 4 are neighbours: bits 3..6 and 19..22 of the shifted word
    constexpr uint32_t kBase = 0x41804180u;   // bf16 16.0 twice
    return make_uint4(((w << 3) & mask) | kBase, ((w >> 1) & mask) | kBase, ((w >> 5) & mask) | kBase,
                      ((w >> 9) & mask) | kBase);
}
__device__ __forceinline__ uint4 decode8(uint32_t w, uint32_t, std::integral_constant<int, kQ4E2m1>) {
    typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
    auto two = [&](auto b) {
        return __builtin_bit_cast(uint32_t, (bf16x2_t)__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, 1.0f, b.value));
    };
    return make_uint4(two(std::integral_constant<int, 0>()), two(std::integral_constant<int, 1>()),
                      two(std::integral_constant<int, 2>()), two(std::integral_constant<int, 3>()));
}

// Orders LDS accesses of one wave's lanes among each other (nothing is executed).
__device__ __forceinline__ void lanes_meet() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// kZero: integers with zero points; kPer groups per tile; kTiles column tiles per wave
// (of each matrix); up to kBlocks times 16 rows at once.
template <int kCode, bool kZero, int kPer, bool kGated, int kTiles, int kBlocks>
__global__ __launch_bounds__(64 * kMaxWaves) void q4_kernel(Q4Args a) {
    constexpr int kMats = kGated ? 2 : 1, kNT = kTiles * kMats;
    constexpr int kSteps = 4 / kPer;              // matrix instructions per group
    constexpr int kWaveLds = kBlocks * kBlockLds;
    static_assert(1024 * kNT <= kBlockLds, "a wave's sums take the place of its rows");
    extern __shared__ __attribute__((aligned(16))) char s_all[];   // kWaveLds per wave
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int c = lane & 15, g = lane >> 4;
    char* s_wave = s_all + wave * kWaveLds;
    const int64_t ct0 = (int64_t)blockIdx.x * kTiles;
    const int64_t tiles = (a.C + kQ4TileCols - 1) / kQ4TileCols;
    const int e = blockIdx.y;
    int lo = 0, hi = a.rows;
    if (a.offsets) {      // kept inside the rows whatever the offsets hold
        const int p = __builtin_amdgcn_readfirstlane(a.offsets[e]);
        const int q = __builtin_amdgcn_readfirstlane(a.offsets[e + 1]);
        lo = p < 0 ? 0 : p > a.rows ? a.rows : p;
        hi = q < lo ? lo : q > a.rows ? a.rows : q;
    }
    if (lo >= hi) return;
    // Loads go through one buffer resource per column tile, with per-lane offsets that never
    // change and the k tile in the scalar offset.  For a tile past the last the per-lane offset
    // is past the resource: the load reads zeros and moves nothing, so the loop's loads need no
    // branch (behind one, the wait for a stage would be a wait for every load).
    __amdgpu_buffer_rsrc_t rw[kNT], rs[kNT], rz[kNT];   // codes, scales, zero points
#pragma unroll
    for (int m = 0; m < kMats; ++m)
#pragma unroll
        for (int t = 0; t < kTiles; ++t) {
            // (a tile past the last column repeats it and is not stored)
            const int64_t ct = ct0 + t < tiles ? ct0 + t : tiles - 1;
            const int i = m * kTiles + t;
            const int64_t groups = e * a.s_stride + ct * a.kt * (32 * kPer);
            rw[i] = make_rsrc(a.W[m] + e * a.w_stride + ct * a.kt * 1024, (int64_t)a.kt * 1024);
            rs[i] = make_rsrc(a.S[m] + groups, (int64_t)a.kt * (32 * kPer));
            if constexpr (kZero) rz[i] = make_rsrc(a.Z[m] + groups, (int64_t)a.kt * (32 * kPer));
        }
    auto load16 = [&](__amdgpu_buffer_rsrc_t r, uint32_t off, int at) {
        return __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(r, off, at, 0));
    };
    auto groups = [&](__amdgpu_buffer_rsrc_t r, uint32_t off, int at, uint32_t (&v)[(kPer + 1) / 2]) {
        if constexpr (kPer == 1) v[0] = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(r, off, at, 0);
        else if constexpr (kPer == 2) v[0] = __builtin_amdgcn_raw_buffer_load_b32(r, off, at, 0);
        else {
            const uint2 u = __builtin_bit_cast(uint2, __builtin_amdgcn_raw_buffer_load_b64(r, off, at, 0));
            v[0] = u.x;
            v[1] = u.y;
        }
    };
    auto value = [&](const uint32_t (&v)[(kPer + 1) / 2], int p) {
        return (p & 1) ? bf16_hi(v[p / 2]) : bf16_lo(v[p / 2]);
    };
    const uint32_t mask = code_mask();
    const uint4 ones = make_uint4(0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u);
    const int waves = blockDim.x >> 6;

    // Rows r0 .. r0 + have, loaded with kXLoads loads per tile: of 4, 8, 16 or 32 rows.
    auto rows = [&](int r0, int have, auto loads) {
        constexpr int kXLoads = loads.value, kB = (kXLoads + 3) / 4;   // blocks of 16 rows
        struct Stage {
            uint4 w[kNT], x[kXLoads];
            uint32_t s[kNT][(kPer + 1) / 2], z[kNT][(kPer + 1) / 2];
        };
        // A load takes 256 B of each of four rows, 16 lanes in order: the operand's own order (64 B
        // of 16 rows, neighbours in lanes 16 apart) is 64 accesses instead of eight lines.  Rows
        // past the last one and, in the last tile, k past K read zeros.
        const uint32_t xin = (uint32_t)((lane >> 4) * a.K * 2 + 16 * c);
        const uint32_t xtail = (a.kt - 1) * kQ4TileK + 8 * c < a.K ? 0u : kOOB;
        const __amdgpu_buffer_rsrc_t rx = make_rsrc(a.X + (int64_t)r0 * a.K, have * a.K * 2);
        auto load = [&](Stage& st, int tile) {
            // Past the resource by one bit of the offset, not by a choice of offsets: the compiler
            // makes a branch of that.  The scalar offset stays inside in any case.
            const uint32_t out = tile < a.kt ? 0u : kOOB;
            const int kt = tile < a.kt ? tile : a.kt - 1;
#pragma unroll
            for (int i = 0; i < kNT; ++i) st.w[i] = load16(rw[i], (uint32_t)(lane * 16) | out, kt * 1024);
            const uint32_t xout = (xtail & (kt == a.kt - 1 ? ~0u : 0u)) | out;
#pragma unroll
            for (int j = 0; j < kXLoads; ++j)
                st.x[j] = load16(rx, (xin + (uint32_t)(4 * j * a.K * 2)) | xout, kt * (kQ4TileK * 2));
            const uint32_t off = (uint32_t)(c * 2 * kPer) | out;
#pragma unroll
            for (int i = 0; i < kNT; ++i) {
                groups(rs[i], off, kt * (32 * kPer), st.s[i]);
                if constexpr (kZero) groups(rz[i], off, kt * (32 * kPer), st.z[i]);
            }
        };
        // The operands of a tile's four steps, through the wave's own LDS (a wave's LDS accesses
        // keep their order): row r's 16-byte piece p lies at 256 r + 16 (p ^ r % 16), so that neither
        // the writes (16 pieces of a row) nor the reads (one piece of 16 rows) meet in a bank.
        // Rows that no load brings hold what was there; their results are not stored.
        auto operands = [&](const Stage& st, uint4 (&x)[kB][4]) {
            lanes_meet();   // (the last tile's reads)
#pragma unroll
            for (int j = 0; j < kXLoads; ++j) {
                const int r = 4 * j + (lane >> 4);
                *reinterpret_cast<uint4*>(s_wave + 256 * r + 16 * (c ^ (r & 15))) = st.x[j];
            }
            lanes_meet();
#pragma unroll
            for (int b = 0; b < kB; ++b)
#pragma unroll
                for (int s = 0; s < 4; ++s)
                    x[b][s] = *reinterpret_cast<const uint4*>(s_wave + kBlockLds * b + 256 * c + 16 * ((4 * s + g) ^ c));
        };
        floatx4_t acc[kB][kNT];
#pragma unroll
        for (int b = 0; b < kB; ++b)
#pragma unroll
            for (int i = 0; i < kNT; ++i) acc[b][i] = floatx4_t{0.f, 0.f, 0.f, 0.f};
        auto multiply = [&](const Stage& st, int kt) {
            uint4 x[kB][4];
            operands(st, x);
#pragma unroll
            for (int p = 0; p < kPer; ++p) {
                // a group past K: its scale may be anything
                const bool real = (int64_t)kt * kQ4TileK + p * (kQ4TileK / kPer) < a.K;
                floatx4_t xs[kB];
#pragma unroll
                for (int b = 0; b < kB; ++b) {
                    xs[b] = floatx4_t{0.f, 0.f, 0.f, 0.f};
                    if constexpr (kCode == kQ4Int)
#pragma unroll
                        for (int j = 0; j < kSteps; ++j) xs[b] = mfma16x16x32(x[b][p * kSteps + j], ones, xs[b]);
                }
#pragma unroll
                for (int i = 0; i < kNT; ++i) {
                    const uint32_t words[4] = {st.w[i].x, st.w[i].y, st.w[i].z, st.w[i].w};
                    floatx4_t sum[kB];
#pragma unroll
                    for (int b = 0; b < kB; ++b) sum[b] = floatx4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int j = 0; j < kSteps; ++j) {
                        const uint4 w = decode8(words[p * kSteps + j], mask, std::integral_constant<int, kCode>());
#pragma unroll
                        for (int b = 0; b < kB; ++b) sum[b] = mfma16x16x32(x[b][p * kSteps + j], w, sum[b]);
                    }
                    const float s = real ? value(st.s[i], p) : 0.f;
                    float z = 24.f;
                    if constexpr (kZero) z = 16.f + (real ? value(st.z[i], p) : 0.f);
#pragma unroll
                    for (int b = 0; b < kB; ++b)
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            const float v = kCode == kQ4Int ? fmaf(-z, xs[b][r], sum[b][r]) : sum[b][r];
                            acc[b][i][r] = fmaf(s, v, acc[b][i][r]);
                        }
                }
            }
        };
        constexpr int kDepth = 2;
        Stage st[kDepth];
#pragma unroll
        for (int d = 0; d < kDepth; ++d) {
            load(st[d], wave + d * waves);
            __builtin_amdgcn_sched_barrier(0);
        }
        for (int kt = wave; kt < a.kt; kt += kDepth * waves) {
#pragma unroll
            for (int d = 0; d < kDepth; ++d) {
                // (left alone, the scheduler joins the stages and waits for all loads at once)
                multiply(st[d], kt + d * waves);
                __builtin_amdgcn_sched_barrier(0);
                load(st[d], kt + (d + kDepth) * waves);
                __builtin_amdgcn_sched_barrier(0);
            }
        }
#pragma unroll
        for (int b = 0; b < kB; ++b)
#pragma unroll
            for (int i = 0; i < kNT; ++i)
                *reinterpret_cast<floatx4_t*>(s_wave + 1024 * (b * kNT + i) + 16 * lane) = acc[b][i];
    };

    constexpr int kRows = kBlocks * kQ4Rows;
    for (int r0 = lo; r0 < hi; r0 += kRows) {
        const int have = hi - r0 < kRows ? hi - r0 : kRows;
        if (have <= 4) rows(r0, have, std::integral_constant<int, 1>());
        else if (have <= 8) rows(r0, have, std::integral_constant<int, 2>());
        else if (have <= 16) rows(r0, have, std::integral_constant<int, 4>());
        else if constexpr (kBlocks > 1) rows(r0, have, std::integral_constant<int, 8>());
        __syncthreads();
        for (int q0 = threadIdx.x; q0 < kTiles * 256 * (have > kQ4Rows ? 2 : 1); q0 += blockDim.x) {
            // a lane's four sums are rows 4 (lane / 16) .. + 3 of column lane % 16
            const int b = q0 / (kTiles * 256), o = q0 % (kTiles * 256);
            const int t = o >> 8, m = kQ4Rows * b + 4 * ((o >> 6) & 3) + (o & 3);
            const int64_t col = (ct0 + t) * kQ4TileCols + ((o >> 2) & 15);
            float v[kMats];
#pragma unroll
            for (int q = 0; q < kMats; ++q) v[q] = 0.f;
            for (int w = 0; w < waves; w += 4)      // (waves is a multiple of four)
#pragma unroll
                for (int u = 0; u < 4; ++u)
#pragma unroll
                    for (int q = 0; q < kMats; ++q)
                        v[q] += *reinterpret_cast<const float*>(s_all + (w + u) * kWaveLds + 1024 * (b * kNT + q * kTiles) + 4 * o);
            if (m >= have || col >= a.C) continue;
            float y;
            if constexpr (kGated) {
                y = silu(v[0]) * v[1];
            } else {
                if (a.bias) v[0] += bf16_to_f32(a.bias[e * a.b_stride + col]);
                // (a NaN stays one: a bad row must not come out as zeros)
                y = a.act == ACT_RELU ? (v[0] <= 0.f ? 0.f : v[0]) : apply_act(a.act, v[0]);
            }
            a.Y[(int64_t)(r0 + m) * a.C + col] = __builtin_bit_cast(uint16_t, (__bf16)y);
        }
        if (r0 + kRows < hi) __syncthreads();   // read before the next rows' sums
    }
}

// ---------------------------------------------------------------- packing

// Nibble of a word that holds its code e (k = .. + e).
__device__ __forceinline__ int nibble_of(int code, int e) {
    return code == kQ4E2m1 ? e : (e >> 1) + 4 * (e & 1);
}

// The e2m1 code nearest to v (|v| beyond 6: 6), ties to the even code.
__device__ __forceinline__ uint32_t to_e2m1(float v) {
    const float m = fabsf(v);
    // halfway points between 0, .5, 1, 1.5, 2, 3, 4, 6; a tie goes to the even code
    const uint32_t q = (m > 0.25f) + (m >= 0.75f) + (m > 1.25f) + (m >= 1.75f) + (m > 2.5f) + (m >= 3.5f) + (m > 5.0f);
    return q | (v < 0.f && q ? 8u : 0u);
}

// 128 k x 64 columns per workgroup: through LDS, so that W is read in whole lines.  A weight passes
// here once in its life, so it was left at this: 4096 x 14336 bf16 145 us, fp32 147 (floors 27, 49).
template <bool kF32>
__global__ __launch_bounds__(256) void q4_quantize_kernel(const void* W, uint8_t* Wq, uint16_t* scale,
                                                          uint16_t* zero, int64_t K, int64_t C, int kt_all,
                                                          int code, int per) {
    __shared__ float s_w[kQ4TileK][64 + 1];
    __shared__ float s_s[4][64], s_z[4][64];
    const int tid = threadIdx.x;
    const int64_t kt = blockIdx.y, c0 = (int64_t)blockIdx.x * 64;
    const int64_t tiles = (C + kQ4TileCols - 1) / kQ4TileCols;
    for (int i = tid; i < kQ4TileK * 64; i += 256) {
        const int64_t k = kt * kQ4TileK + (i >> 6), col = c0 + (i & 63);
        float v = 0.f;
        if (k < K && col < C)
            v = kF32 ? static_cast<const float*>(W)[k * C + col] : bf16_to_f32(static_cast<const uint16_t*>(W)[k * C + col]);
        s_w[i >> 6][i & 63] = v;
    }
    __syncthreads();
    const int len = kQ4TileK / per;
    if (tid < per * 64) {
        const int p = tid >> 6, col = tid & 63;
        float lo = 0.f, hi = 0.f;
        for (int k = 0; k < len; ++k) {
            lo = fminf(lo, s_w[p * len + k][col]);
            hi = fmaxf(hi, s_w[p * len + k][col]);
        }
        const float top = fmaxf(-lo, hi);
        // (half the range: hi - lo may leave fp32 where hi and lo do not)
        float s = code == kQ4E2m1 ? top / 6.f : zero ? (0.5f * hi - 0.5f * lo) / 7.5f : top / 7.f;
        if (top < 0x1p-100f) s = 0.f;         // nothing to keep
        s = (float)(__bf16)s;                 // codes are taken under the scale as it is kept
        float z = 8.f;
        if (zero) z = s > 0.f ? fminf(fmaxf(rintf(-lo / s), 0.f), 15.f) : 8.f;
        s_s[p][col] = s;
        s_z[p][col] = z;
        const int64_t ct = (c0 + col) / kQ4TileCols;
        if (ct < tiles) {
            const int64_t at = ((ct * kt_all + kt) * 16 + col % 16) * per + p;
            scale[at] = __builtin_bit_cast(uint16_t, (__bf16)s);
            if (zero) zero[at] = __builtin_bit_cast(uint16_t, (__bf16)z);
        }
    }
    __syncthreads();
    for (int i = tid; i < 1024; i += 256) {   // one word each: tile, lane, step
        const int t = i >> 8, l = (i >> 2) & 63, j = i & 3;
        const int64_t ct = c0 / kQ4TileCols + t;
        if (ct >= tiles) continue;
        const int col = 16 * t + l % 16, k0 = 32 * j + 8 * (l / 16);
        const float s = s_s[k0 / len][col], z = s_z[k0 / len][col];
        uint32_t word = 0;
        for (int e = 0; e < 8; ++e) {
            const float v = s_w[k0 + e][col];
            uint32_t q;
            if (code == kQ4E2m1) q = s > 0.f ? to_e2m1(v / s) : 0u;
            else q = s > 0.f ? (uint32_t)fminf(fmaxf(rintf(v / s) + z, 0.f), 15.f) : (uint32_t)z;
            word |= q << (4 * nibble_of(code, e));
        }
        reinterpret_cast<uint32_t*>(Wq)[((ct * kt_all + kt) * 64 + l) * 4 + j] = word;
    }
}

// One word per thread; the first threads of a tile also place its scales and zeros.  Eight loads of
// a byte each, a row of codes apart (4096 x 14336: 68 us, floor 17).
__global__ __launch_bounds__(256) void q4_pack_kernel(const uint8_t* codes, const uint16_t* scale_in,
                                                      const uint16_t* zero_in, uint8_t* Wq, uint16_t* scale,
                                                      uint16_t* zero, int64_t K, int64_t C, int kt_all, int code,
                                                      int per) {
    const int64_t tile = blockIdx.x;          // ct * kt_all + kt
    const int64_t ct = tile / kt_all, kt = tile - ct * kt_all;
    const int tid = threadIdx.x, l = tid >> 2, j = tid & 3;
    const int64_t col = ct * kQ4TileCols + l % 16, k0 = kt * kQ4TileK + 32 * j + 8 * (l / 16);
    uint32_t word = 0;
    for (int e = 0; e < 8; ++e) {
        // past the matrix: the code of zero
        uint32_t q = code == kQ4E2m1 ? 0u : 8u;
        if (col < C && k0 + e < K) q = codes[(k0 + e) * C + col] & 15u;
        word |= q << (4 * nibble_of(code, e));
    }
    reinterpret_cast<uint32_t*>(Wq)[tile * 256 + tid] = word;
    if (tid < 16 * per) {
        const int p = tid % per;
        const int64_t cc = ct * kQ4TileCols + tid / per, grp = kt * per + p;
        const bool real = cc < C && grp * (kQ4TileK / per) < K;
        scale[tile * 16 * per + tid] = real ? scale_in[grp * C + cc] : (uint16_t)0;
        if (zero) zero[tile * 16 * per + tid] = real ? zero_in[grp * C + cc] : (uint16_t)0;
    }
}

// Column tiles per wave, waves per workgroup, rows at once.  (Both sides of each rule on one card, in
// turn, replayed in graphs; groups of 128 without zero points unless said.)
//
// Two tiles share a wave's rows of X, which for 16 rows are more bytes than a tile's codes, and
// halve the workgroups: taken where at least one workgroup per CU is left (16 x 8192 x 8192:
// 10.4 us, with one tile 11.8; 16 x 4096 x 14336: 9.9, 11.9; but 16 x 4096 x 4096, 128 workgroups
// with two: 6.0, with one 5.0; the gated pair shares them already).  Four of integers, where their
// fewer workgroups leave no CU with more tiles than two would (16 x 8192 x 28672, eight a CU
// either way: 30.4 us, with two 33.8; 16 x 4096 x 22016, eight instead of six: 14.8, 13.5; e2m1,
// whose rows need no sums, was no faster).
//
// Up to one workgroup per CU takes eight waves (16 rows, pair of 8192 x 3584, 224 workgroups:
// 9.6 us, with four 10.9; 16 x 14336 x 4096: 10.7, 13.0).  More of them take four: of eight, whose
// registers fill half a CU or more, the second waits for the first (16 x 4096 x 14336, 448
// workgroups: 9.9 us, with eight 11.7; pair of 4096 x 8192 with zero points, 512: 10.3, 10.8).
// Experts without rows have workgroups that end at once: those are not counted.
//
// Rows at once: 32 where lists are longer than ten rows on average, so that many pass 16 (pair of
// 8 x 4096 x 2048: 512 rows 57 us, with 16 at once 69; 192 rows 27.2, 32.1; 96 rows 18.4, 19.7; product of
// 8 x 14336 x 4096, 512 rows: 183, 237; but 60 x 2048 x 1408, 512 rows, 8.5 a list: 44.6 with 32,
// 43.7 with 16, for half again as many registers).
struct Q4Shape {
    int tiles, waves, blocks;
};
Q4Shape q4_shape(const Q4IO& io, int64_t tiles, int kt) {
    constexpr int64_t kCUs = 256;
    const int64_t lists = io.rows < io.E ? io.rows : io.E;
    auto groups = [&](int n) { return (tiles + n - 1) / n * lists; };
    auto fullest = [&](int n) { return (groups(n) + kCUs - 1) / kCUs * n; };   // tiles of a CU
    Q4Shape s;
    s.tiles = io.gated || tiles * lists < 2 * kCUs ? 1 : 2;
    // (one matrix, so at most 16 rows)
    if (s.tiles == 2 && io.code == kQ4Int && !io.offsets && groups(4) > kCUs && fullest(4) <= fullest(2)) s.tiles = 4;
    s.waves = groups(s.tiles) > kCUs || kt <= 4 ? 4 : kMaxWaves;
    s.blocks = io.rows > kQ4Rows && io.rows > 10 * lists ? 2 : 1;
    return s;
}

template <int kCode, bool kZero, int kPer, int kBlocks>
hipError_t start(const Q4Args& a, const Q4Shape& s, const Q4IO& io, int64_t tiles, hipStream_t stream) {
    const dim3 grid((unsigned)((tiles + s.tiles - 1) / s.tiles), (unsigned)io.E), block(64 * s.waves);
    const size_t lds = (size_t)s.waves * kBlocks * kBlockLds;
    if (io.gated)
        hipLaunchKernelGGL((q4_kernel<kCode, kZero, kPer, true, 1, kBlocks>), grid, block, lds, stream, a);
    else if (s.tiles == 1)
        hipLaunchKernelGGL((q4_kernel<kCode, kZero, kPer, false, 1, kBlocks>), grid, block, lds, stream, a);
    else if (s.tiles == 2)
        hipLaunchKernelGGL((q4_kernel<kCode, kZero, kPer, false, 2, kBlocks>), grid, block, lds, stream, a);
    else if constexpr (kCode == kQ4Int && kBlocks == 1)
        hipLaunchKernelGGL((q4_kernel<kCode, kZero, kPer, false, 4, 1>), grid, block, lds, stream, a);
    else
        return hipErrorInvalidValue;    // no rule gives this shape
    return hipGetLastError();
}

}  // namespace

hipError_t launch_q4(const Q4IO& io, hipStream_t stream) {
    Q4Args a;
    const int per = kQ4TileK / io.group;
    const int64_t tiles = (io.C + kQ4TileCols - 1) / kQ4TileCols;
    a.kt = (int)((io.K + kQ4TileK - 1) / kQ4TileK);
    for (int m = 0; m < 2; ++m) {
        a.W[m] = reinterpret_cast<const char*>(io.W[m]);
        a.S[m] = reinterpret_cast<const char*>(io.scale[m]);
        a.Z[m] = reinterpret_cast<const char*>(io.zero[m]);
    }
    a.X = io.X;
    a.bias = io.bias;
    a.Y = io.Y;
    a.offsets = io.offsets;
    a.rows = (int)io.rows;
    a.K = io.K;
    a.C = io.C;
    a.w_stride = tiles * a.kt * 1024;
    a.s_stride = tiles * a.kt * 32 * per;
    a.b_stride = io.C;
    a.act = io.act;
    const Q4Shape s = q4_shape(io, tiles, a.kt);
    auto go = [&](auto code, auto z, auto p) {
        return s.blocks == 2 ? start<code.value, z.value, p.value, 2>(a, s, io, tiles, stream)
                             : start<code.value, z.value, p.value, 1>(a, s, io, tiles, stream);
    };
    auto with = [&](auto code, auto z) {
        if (per == 1) return go(code, z, std::integral_constant<int, 1>());
        if (per == 2) return go(code, z, std::integral_constant<int, 2>());
        return go(code, z, std::integral_constant<int, 4>());
    };
    using Int = std::integral_constant<int, kQ4Int>;
    if (io.code == kQ4E2m1) return with(std::integral_constant<int, kQ4E2m1>(), std::false_type());
    if (io.zero[0]) return with(Int(), std::true_type());
    return with(Int(), std::false_type());
}

hipError_t launch_q4_quantize(const void* W, bool f32, uint8_t* Wq, uint16_t* scale, uint16_t* zero,
                              int64_t K, int64_t C, int code, int group, hipStream_t stream) {
    const int kt = (int)((K + kQ4TileK - 1) / kQ4TileK);
    const dim3 grid((unsigned)((C + 63) / 64), (unsigned)kt);
    if (f32)
        hipLaunchKernelGGL(q4_quantize_kernel<true>, grid, dim3(256), 0, stream, W, Wq, scale, zero, K, C, kt,
                           code, kQ4TileK / group);
    else
        hipLaunchKernelGGL(q4_quantize_kernel<false>, grid, dim3(256), 0, stream, W, Wq, scale, zero, K, C, kt,
                           code, kQ4TileK / group);
    return hipGetLastError();
}

hipError_t launch_q4_pack(const uint8_t* codes, const uint16_t* scale_in, const uint16_t* zero_in,
                          uint8_t* Wq, uint16_t* scale, uint16_t* zero, int64_t K, int64_t C, int code,
                          int group, hipStream_t stream) {
    const int kt = (int)((K + kQ4TileK - 1) / kQ4TileK);
    const int64_t tiles = (C + kQ4TileCols - 1) / kQ4TileCols * kt;
    hipLaunchKernelGGL(q4_pack_kernel, dim3((unsigned)tiles), dim3(256), 0, stream, codes, scale_in, zero_in, Wq,
                       scale, zero, K, C, kt, code, kQ4TileK / group);
    return hipGetLastError();
}

}  // namespace ffn
