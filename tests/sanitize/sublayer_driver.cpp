// Exercises the host side of the entry points around an expert sub-layer (RMS
// norm, dispatch and combine, 4-bit products; include/ffn.h) without a GPU, for the
// sanitizer build run by tests/test_sublayer_sanitizers.py: the size queries over
// many shapes, and each call with arguments that the host checks reject before any
// HIP call.  Exits non-zero on an unexpected return code.
#include <cstdint>
#include <cstdio>
#include <cstring>

#include "ffn.h"

namespace {
int failures = 0;
void expect(int got, int want, const char* what) {
    if (got != want) {
        std::fprintf(stderr, "%s: got %d, want %d (%s)\n", what, got, want, ffn_last_error());
        ++failures;
    }
    if (want != FFN_OK && std::strlen(ffn_last_error()) == 0) {
        std::fprintf(stderr, "%s: no error text\n", what);
        ++failures;
    }
}
void require(bool ok, const char* what) {
    if (ok) return;
    std::fprintf(stderr, "%s\n", what);
    ++failures;
}
}  // namespace

int main() {
    const int64_t top = INT64_MAX;
    for (int64_t M : {int64_t(0), int64_t(1), int64_t(255), int64_t(257), int64_t(1) << 30, (int64_t(1) << 31) - 1}) {
        for (int64_t N : {8, 520, 8192, 8200, 16384})
            for (int dt : {FFN_F32, FFN_BF16})
                require(ffn_rmsnorm_backward_workspace_size(M, N, dt) >= (size_t)(M ? 4 * N : 256), "RMS norm size");
        for (int64_t E : {1, 8, 100, 256})
            for (int k : {1, 2, 3, 7, 8}) {
                const size_t n = moe_dispatch_workspace_size(M, E, k);
                if (M * k >= (int64_t(1) << 31)) require(n == 0, "dispatch size past its limit");
                else require(n >= 256 && n <= (size_t)(256 + 4 * 256 * E), "dispatch size");
            }
    }
    for (int64_t K : {8, 128, 136, 8192, 1 << 21})
        for (int64_t C : {8, 16, 24, 520}) {
            const size_t n = ffn_q4_bytes(K, C);
            require(n >= (size_t)(K * C / 2) && n % 1024 == 0, "4-bit size");
        }
    for (int64_t bad : {int64_t(-1), int64_t(0), int64_t(12), top, top - 7, INT64_MIN}) {
        require(ffn_rmsnorm_backward_workspace_size(64, bad, FFN_BF16) == 0, "bad row");
        require(ffn_q4_bytes(bad, 64) == 0 && ffn_q4_bytes(64, bad) == 0, "bad matrix");
        if (bad != 12) require(moe_dispatch_workspace_size(64, bad, 2) == 0, "bad E");
    }
    for (int64_t bad : {int64_t(-1), top, INT64_MIN}) {
        require(ffn_rmsnorm_backward_workspace_size(bad, 64, FFN_BF16) == 0, "bad rows");
        require(moe_dispatch_workspace_size(bad, 8, 2) == 0, "bad tokens");
    }

    // rejected calls: fake, never dereferenced device pointers, 4 MiB apart
    char* at[20];
    for (int i = 0; i < 20; ++i) at[i] = reinterpret_cast<char*>(uintptr_t(0x1000000) + uintptr_t(i) * 0x400000);
    float* f[20];
    int32_t* n[20];
    for (int i = 0; i < 20; ++i) {
        f[i] = reinterpret_cast<float*>(at[i]);
        n[i] = reinterpret_cast<int32_t*>(at[i]);
    }
    const size_t big = 1 << 20;

    auto rms = [&](const void* X, const void* R, void* S, void* Y, float* rstd, int64_t M, int64_t N, int dt, float eps) {
        return ffn_rmsnorm_forward(X, R, at[2], S, Y, rstd, M, N, dt, eps, nullptr);
    };
    expect(rms(nullptr, at[1], at[3], at[4], f[5], 64, 64, FFN_F32, 1e-5f), FFN_EINVAL, "null X");
    expect(rms(at[0], at[1], nullptr, at[4], f[5], 64, 64, FFN_F32, 1e-5f), FFN_EINVAL, "R without S");
    expect(rms(at[0], nullptr, at[3], at[4], f[5], 64, 64, FFN_F32, 1e-5f), FFN_EINVAL, "S without R");
    expect(rms(at[0], at[1], at[3], at[4], f[5], 64, 64, FFN_F32, 0.0f), FFN_EINVAL, "eps");
    expect(rms(at[0], at[1], at[3], at[4], f[5], top, 64, FFN_F32, 1e-5f), FFN_EUNSUPPORTED, "M bound");
    expect(rms(at[0], at[1], at[3], at[4], f[5], 64, top - 7, FFN_F32, 1e-5f), FFN_EUNSUPPORTED, "N bound");
    expect(rms(at[0], at[1], at[3], at[4], f[5], 64, 64, FFN_E4M3, 1e-5f), FFN_EINVAL, "type");
    expect(rms(at[0], at[1], at[3], at[4] + 8, f[5], 64, 64, FFN_BF16, 1e-5f), FFN_EALIGN, "alignment");
    expect(rms(at[0], at[1], at[0] + 16, at[4], f[5], 64, 64, FFN_BF16, 1e-5f), FFN_EINVAL, "S beside X");
    expect(rms(nullptr, nullptr, nullptr, nullptr, nullptr, 0, 64, FFN_BF16, 1e-5f), FFN_OK, "no rows");
    expect(ffn_rmsnorm_q8_forward(at[0], at[1], at[2], at[3], at[4], f[5], f[6], 64, 64, FFN_BF16, 64, 1e-5f, nullptr),
           FFN_EUNSUPPORTED, "group");
    expect(ffn_rmsnorm_q8_forward(at[0], at[1], at[2], at[3], at[4], nullptr, f[6], 64, 64, FFN_BF16, 0, 1e-5f, nullptr),
           FFN_EINVAL, "no scales");
    expect(ffn_rmsnorm_backward(at[0], at[1], at[2], at[3], f[4], at[5], f[6], 64, 64, FFN_BF16, at[7], 255, nullptr),
           FFN_EWORKSPACE, "workspace");
    expect(ffn_rmsnorm_backward(at[0], at[1], nullptr, at[3], f[4], at[5], nullptr, 64, 64, FFN_BF16, at[7], big, nullptr),
           FFN_EINVAL, "no dgamma");
    expect(ffn_rmsnorm_backward(at[0], at[1], at[2], at[3], f[4], at[1] + 16, f[6], 64, 64, FFN_BF16, at[7], big, nullptr),
           FFN_EINVAL, "dX beside dY");

    auto dispatch = [&](const void* X, int64_t M, int64_t N, int64_t E, int k, int dt, const float* scale, int64_t cols,
                        void* ws, size_t wsb) {
        return moe_dispatch(X, n[1], scale, M, N, E, k, dt, cols, at[4], scale ? f[5] : nullptr, n[6], n[7], n[8], ws, wsb,
                            nullptr);
    };
    expect(dispatch(nullptr, 64, 64, 8, 2, FFN_BF16, nullptr, 0, at[9], big), FFN_EINVAL, "null X");
    expect(dispatch(at[0], top, 64, 8, 2, FFN_BF16, nullptr, 0, at[9], big), FFN_EUNSUPPORTED, "M bound");
    expect(dispatch(at[0], 64, top - 7, 8, 2, FFN_BF16, nullptr, 0, at[9], big), FFN_EUNSUPPORTED, "N bound");
    expect(dispatch(at[0], 64, 64, top, 2, FFN_BF16, nullptr, 0, at[9], big), FFN_EUNSUPPORTED, "E bound");
    expect(dispatch(at[0], 64, 64, 8, INT32_MIN, FFN_BF16, nullptr, 0, at[9], big), FFN_EUNSUPPORTED, "k bound");
    expect(dispatch(at[0], 64, 64, 8, 2, FFN_E4M3, f[2], top, at[9], big), FFN_EINVAL, "columns of scales");
    expect(dispatch(at[0], 64, 64, 8, 2, FFN_E4M3, nullptr, 1, at[9], big), FFN_EINVAL, "columns without scales");
    expect(dispatch(at[0], 64, 64, 8, 2, FFN_BF16, nullptr, 0, at[9], 255), FFN_EWORKSPACE, "workspace");
    expect(dispatch(at[0], 64, 64, 8, 2, FFN_BF16, nullptr, 0, nullptr, big), FFN_EINVAL, "no workspace");
    expect(dispatch(at[4], 64, 64, 8, 2, FFN_BF16, nullptr, 0, at[9], big), FFN_EINVAL, "Xs over X");
    expect(moe_combine(at[0], n[1], f[2], at[3], at[4], 64, 64, 2, top, FFN_BF16, nullptr), FFN_EUNSUPPORTED, "rows bound");
    expect(moe_combine(at[0], n[1], f[2], at[3], at[0], 64, 64, 2, 128, FFN_BF16, nullptr), FFN_EINVAL, "Y over Ys");
    expect(moe_combine(at[0], n[1], f[2], at[3], at[4], 64, 64, 2, 128, FFN_E4M3, nullptr), FFN_EUNSUPPORTED, "e4m3");
    expect(moe_dispatch_backward(at[0], nullptr, at[4], 64, 64, 2, 128, FFN_BF16, nullptr), FFN_EINVAL, "no positions");
    expect(moe_combine_backward(at[0], nullptr, n[2], f[3], at[4], f[5], 64, 64, 2, 128, FFN_F32, nullptr), FFN_EINVAL,
           "dw without Ys");
    expect(moe_combine_backward(at[0], at[1], n[2], f[3], at[0], f[5], 64, 64, 2, 128, FFN_F32, nullptr), FFN_EINVAL,
           "dYs over dY");
    expect(moe_route_backward(n[0], f[1], f[2], f[2], 64, 8, 2, nullptr), FFN_EINVAL, "dlogits over dw");
    expect(moe_route_backward(nullptr, nullptr, nullptr, nullptr, 0, 8, 2, nullptr), FFN_OK, "no tokens");

    auto matvec = [&](const void* X, void* Y, int64_t M, int64_t K, int64_t C, int code, int group, int act) {
        return ffn_q4_matvec(X, at[1], at[2], nullptr, at[3], Y, M, K, C, code, group, act, nullptr);
    };
    expect(matvec(nullptr, at[4], 4, 64, 64, FFN_Q4_INT, 128, 0), FFN_EINVAL, "null X");
    expect(matvec(at[0], at[4], 17, 64, 64, FFN_Q4_INT, 128, 0), FFN_EUNSUPPORTED, "rows");
    expect(matvec(at[0], at[4], INT64_MIN, 64, 64, FFN_Q4_INT, 128, 0), FFN_EINVAL, "negative rows");
    expect(matvec(at[0], at[4], 4, top - 7, 8, FFN_Q4_INT, 128, 0), FFN_EUNSUPPORTED, "K bound");
    expect(matvec(at[0], at[4], 4, 8, top - 7, FFN_Q4_INT, 128, 0), FFN_EUNSUPPORTED, "C bound");
    expect(matvec(at[0], at[4], 4, 64, 64, 7, 128, 0), FFN_EINVAL, "code");
    expect(matvec(at[0], at[4], 4, 64, 64, FFN_Q4_E2M1, 48, 0), FFN_EUNSUPPORTED, "group");
    expect(matvec(at[0], at[4], 4, 64, 64, FFN_Q4_E2M1, 32, 9), FFN_EINVAL, "activation");
    expect(matvec(at[0], at[1], 4, 64, 64, FFN_Q4_INT, 128, 0), FFN_EINVAL, "Y over Wq");
    expect(matvec(nullptr, nullptr, 0, 64, 64, FFN_Q4_INT, 128, 0), FFN_OK, "no rows");
    expect(ffn_q4_swiglu(at[0], at[1], at[2], at[3], at[4], at[5], nullptr, at[6], 4, 64, 64, FFN_Q4_INT, 128, nullptr),
           FFN_EINVAL, "one zero point");
    expect(moe_q4_matvec(at[0], nullptr, at[1], at[2], nullptr, nullptr, at[3], 40, 8, 64, 64, FFN_Q4_INT, 128, 0, nullptr),
           FFN_EINVAL, "no offsets");
    expect(moe_q4_swiglu(at[0], n[1], at[2], at[3], nullptr, at[4], at[5], nullptr, at[6], 40, top, 64, 64, FFN_Q4_INT, 128,
                         nullptr), FFN_EUNSUPPORTED, "E bound");
    expect(ffn_q4_quantize(at[0], at[1], at[2], at[3], 64, 64, FFN_F32, FFN_Q4_E2M1, 32, nullptr), FFN_EINVAL,
           "zero points of e2m1");
    expect(ffn_q4_quantize(at[0], at[0], at[2], nullptr, 64, 64, FFN_F32, FFN_Q4_INT, 32, nullptr), FFN_EINVAL, "Wq over W");
    expect(ffn_q4_pack(at[0], at[1], nullptr, at[2], at[3], at[4], 64, 64, FFN_Q4_INT, 32, nullptr), FFN_EINVAL, "zero_in");
    if (failures) return 2;
    std::printf("sub-layer sanitizer driver: ok\n");
    return 0;
}
