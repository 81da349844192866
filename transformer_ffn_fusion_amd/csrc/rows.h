// rows.h -- rows of bf16 or fp32 values held by the lanes of one or more waves,
// eight consecutive columns per lane and step: what the norms share.
#pragma once

#include "ffn_device.h"

namespace ffn {

constexpr int kLnCols = 512;       // columns a wave holds per step: 64 lanes x 8

// Eight consecutive values as they lie in memory, as floats, and back.
template <bool kF32>
struct Ln8 {
    uint4 w[kF32 ? 2 : 1];
    __device__ __forceinline__ void load(const void* p, int64_t at) {
        const char* q = static_cast<const char*>(p) + at * (kF32 ? 4 : 2);
        w[0] = ld16(q);
        if constexpr (kF32) w[1] = ld16(q + 16);
    }
    __device__ __forceinline__ void zero() {
        w[0] = zero16();
        if constexpr (kF32) w[1] = zero16();
    }
    __device__ __forceinline__ void get(float (&v)[8]) const {
        if constexpr (kF32) {
            const uint32_t u[8] = {w[0].x, w[0].y, w[0].z, w[0].w, w[1].x, w[1].y, w[1].z, w[1].w};
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = __uint_as_float(u[e]);
        } else {
            const uint32_t u[4] = {w[0].x, w[0].y, w[0].z, w[0].w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                v[2 * e] = bf16_lo(u[e]);
                v[2 * e + 1] = bf16_hi(u[e]);
            }
        }
    }
};
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

// Sum over the wave, in every lane: within rows of 16 lanes, then across them, with
// data-parallel moves (no LDS).  Lanes that a move does not reach add zero.
template <int kCtrl, int kRows>
__device__ __forceinline__ float dpp_add(float v) {
    return v + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), kCtrl, kRows, 0xf, false));
}
__device__ __forceinline__ float wave_sum(float v) {
    v = dpp_add<0x111, 0xf>(v);   // row_shr:1
    v = dpp_add<0x112, 0xf>(v);   // row_shr:2
    v = dpp_add<0x114, 0xf>(v);   // row_shr:4
    v = dpp_add<0x118, 0xf>(v);   // row_shr:8: lane 15 of each row holds the row's sum
    v = dpp_add<0x142, 0xa>(v);   // row_bcast:15 into rows 1 and 3
    v = dpp_add<0x143, 0xc>(v);   // row_bcast:31 into rows 2 and 3
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
}

// How a workgroup's waves share rows.
struct LnShape {
    int V, W, G;   // steps per lane, waves per row, rows per workgroup at once
};
inline LnShape ln_shape(int64_t N, int max_threads) {
    const int waves = (int)((N + kLnCols - 1) / kLnCols), most = max_threads / 64;
    LnShape s;
    s.V = waves <= most ? 1 : waves <= 2 * most ? 2 : 4;
    s.W = (waves + s.V - 1) / s.V;
    s.G = most / s.W;
    return s;   // N up to 4 x 512 columns a wave (past that G is 0), and up to the V that the caller's kernel has
}

}  // namespace ffn
