// sublayer.h -- host-side launch interfaces, between the C-ABI layer and the kernels,
// of the operators around an expert sub-layer: RMS norm, dispatch and combine, products
// with 4-bit weights.  Not installed; the public interface is include/ffn.h.
#pragma once

#include <hip/hip_runtime.h>

#include <stddef.h>
#include <stdint.h>

namespace ffn {

// ---- RMS norm (rmsnorm.hip)

struct RmsForwardIO {
    const void *X = nullptr, *R = nullptr, *gamma = nullptr;   // R may be null
    void *S = nullptr, *Y = nullptr;                            // S with R alone; Y: data or codes
    float *scale = nullptr, *rstd = nullptr;                    // scale: 8-bit output; rstd may be null
    int64_t M = 0, N = 0;
    bool f32 = false, q8 = false;
    int group = 0;                                              // 8-bit output: 128, or 0 for a row
    float eps = 0.f;
};
hipError_t launch_rmsnorm_forward(const RmsForwardIO& io, hipStream_t stream);
size_t rmsnorm_partial_floats(int64_t M, int64_t N);   // the workgroups' column sums
hipError_t launch_rmsnorm_backward(const void* S, const void* dY, const void* dS, const void* gamma,
                                   const float* rstd, void* dX, float* dgamma, float* part, int64_t M,
                                   int64_t N, bool f32, hipStream_t stream);

// ---- tokens by expert and back (moe_dispatch.hip)

struct DispatchIO {
    const void* X = nullptr;            // M rows of row_bytes (a multiple of 8)
    const int32_t* ids = nullptr;       // M x k
    const float* scale = nullptr;       // M x scale_cols, or null
    void* Xs = nullptr;                 // M k rows
    float* scale_sorted = nullptr;      // M k x scale_cols
    int32_t *offsets = nullptr, *entries = nullptr, *positions = nullptr;
    int64_t M = 0, row_bytes = 0, scale_cols = 0;
    int E = 0, k = 0;
    int32_t* counts = nullptr;          // workspace: dispatch_count_ints(M, E, k)
};
size_t dispatch_count_ints(int64_t M, int64_t E, int k);
hipError_t launch_moe_dispatch(const DispatchIO& io, hipStream_t stream);

// Y[t] = res[t] + sum_s w[t,s] rows[pos[t,s]]; w and res may be null.
hipError_t launch_moe_combine_rows(const void* rows, int64_t R, const int32_t* pos, const float* w,
                                   const void* res, void* Y, int64_t M, int64_t N, int k, bool f32,
                                   hipStream_t stream);
hipError_t launch_moe_combine_backward(const void* dY, const void* rows, int64_t R, const int32_t* pos,
                                       const float* w, void* drows, float* dw, int64_t M, int64_t N,
                                       int k, bool f32, hipStream_t stream);
hipError_t launch_moe_route_backward(const int32_t* ids, const float* w, const float* dw, float* dlogits,
                                     int64_t M, int E, int k, hipStream_t stream);

// ---- products with 4-bit weights (ffn_q4.hip)

constexpr int kQ4Rows = 16;      // rows of one matrix instruction
constexpr int kQ4TileCols = 16;  // a packed tile: 16 columns x 128 k, 1 KiB
constexpr int kQ4TileK = 128;
struct Q4IO {
    const uint16_t* X = nullptr;                          // rows x K bf16
    const uint8_t* W[2] = {nullptr, nullptr};             // [1]: the up matrix of the gated form
    const uint16_t* scale[2] = {nullptr, nullptr};
    const uint16_t* zero[2] = {nullptr, nullptr};         // may be null
    const uint16_t* bias = nullptr;                       // C (per expert: E x C) or null
    uint16_t* Y = nullptr;                                // rows x C bf16
    const int32_t* offsets = nullptr;                     // E + 1 row offsets, or null (one matrix)
    int64_t rows = 0, K = 0, C = 0;
    int E = 1, code = 0, group = 128, act = 0;
    bool gated = false;
};
hipError_t launch_q4(const Q4IO& io, hipStream_t stream);
// W (K x C, bf16 or fp32) to codes, scales and (zero != nullptr) zero points.
hipError_t launch_q4_quantize(const void* W, bool f32, uint8_t* Wq, uint16_t* scale, uint16_t* zero,
                              int64_t K, int64_t C, int code, int group, hipStream_t stream);
// Codes (K x C bytes), scales and zeros (groups x C bf16) to the packed layout.
hipError_t launch_q4_pack(const uint8_t* codes, const uint16_t* scale_in, const uint16_t* zero_in,
                          uint8_t* Wq, uint16_t* scale, uint16_t* zero, int64_t K, int64_t C, int code,
                          int group, hipStream_t stream);

}  // namespace ffn
