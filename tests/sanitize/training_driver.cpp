// Exercises the host side of the training operators' entry points (SwiGLU
// backward, layer norm, orthogonalised update; include/ffn.h) without a GPU, for
// the sanitizer build run by tests/test_training_sanitizers.py: the size queries
// over many shapes (and with them the tile plans and workspace layouts), and each
// call with arguments that the host checks reject before any HIP call.  Exits
// non-zero on an unexpected return code.
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
    // size queries: what the calls keep there at least, 0 for what they refuse
    for (int64_t M : {0, 1, 8, 63, 1013, 4096, 1 << 20, 1 << 30})
        for (int64_t N : {8, 136, 2056, 4096, 1 << 22})
            for (int64_t O : {8, 264, 1400, 8192, 1 << 21})
                for (int64_t P : {8, 520, 4096}) {
                    const size_t n = ffn_swiglu_backward_workspace_size(M, N, O, P, FFN_BF16);
                    const bool taken = N * O < (int64_t(1) << 30) && O * P < (int64_t(1) << 30);
                    require(taken ? n >= 256 && n >= (size_t)(10 * M * O) : n == 0, "SwiGLU backward size");
                    require(ffn_swiglu_backward_workspace_size(M, N, O, P, FFN_F32) == 0, "SwiGLU backward fp32 size");
                }
    for (int64_t M : {int64_t(0), int64_t(1), int64_t(255), int64_t(257), int64_t(1) << 30, (int64_t(1) << 31) - 1})
        for (int64_t N : {8, 520, 8192, 8200, 16384})
            for (int dt : {FFN_F32, FFN_BF16})
                require(ffn_layernorm_backward_workspace_size(M, N, dt) >= (size_t)(M ? 8 * N : 256), "layer norm size");
    for (int64_t B : {0, 1, 3, 8, 65535})
        for (int64_t R : {8, 128, 136, 1024, 4096, 46336})
            for (int64_t C : {8, 512, 520, 8192, 46336}) {
                const size_t n = ffn_orthogonalize_workspace_size(B, R, C, FFN_F32);
                const int64_t m = R < C ? R : C, k = R < C ? C : R;
                if (R * C >= (int64_t(1) << 31)) require(n == 0, "orthogonalise size past its limit");
                else if (m <= 128 && k <= 512) require(n == 256, "orthogonalise size of one workgroup");
                else require(n >= 256 && n >= (size_t)(B * (6 * R * C + 4 * m * m)), "orthogonalise size");
            }
    for (int64_t bad : {int64_t(-1), int64_t(0), int64_t(12), top, top - 7, INT64_MIN}) {
        require(ffn_swiglu_backward_workspace_size(64, bad, 64, 64, FFN_BF16) == 0, "bad N");
        require(ffn_swiglu_backward_workspace_size(64, 64, bad, 64, FFN_BF16) == 0, "bad O");
        require(ffn_swiglu_backward_workspace_size(64, 64, 64, bad, FFN_BF16) == 0, "bad P");
        require(ffn_layernorm_backward_workspace_size(64, bad, FFN_BF16) == 0, "bad row");
        require(ffn_orthogonalize_workspace_size(1, bad, 64, FFN_BF16) == 0, "bad R");
        require(ffn_orthogonalize_workspace_size(1, 64, bad, FFN_BF16) == 0, "bad C");
    }
    for (int64_t bad : {int64_t(-1), top, INT64_MIN}) {
        require(ffn_swiglu_backward_workspace_size(bad, 64, 64, 64, FFN_BF16) == 0, "bad M");
        require(ffn_layernorm_backward_workspace_size(bad, 64, FFN_BF16) == 0, "bad rows");
        require(ffn_orthogonalize_workspace_size(bad, 136, 520, FFN_BF16) == 0, "bad B");
    }

    // rejected calls: fake, never dereferenced device pointers, 1 MiB apart
    char* at[12];
    for (int i = 0; i < 12; ++i) at[i] = reinterpret_cast<char*>(uintptr_t(0x1000000) + uintptr_t(i) * 0x100000);
    float* f[12];
    for (int i = 0; i < 12; ++i) f[i] = reinterpret_cast<float*>(at[i]);
    const size_t big = 1 << 20;
    auto swiglu = [&](const void* X, void* dX, void* dWd, int64_t M, int64_t N, int64_t O, int dt, int gd, void* ws, size_t n) {
        return ffn_swiglu_backward(X, at[1], at[2], at[3], at[4], dX, at[6], at[7], dWd, M, N, O, 64, dt, gd, ws, n, nullptr);
    };
    expect(swiglu(nullptr, at[5], at[8], 64, 64, 64, FFN_BF16, FFN_BF16, at[9], big), FFN_EINVAL, "null X");
    expect(swiglu(at[0], at[5], at[8], 64, 64, 64, FFN_F32, FFN_BF16, at[9], big), FFN_EUNSUPPORTED, "fp32 inputs");
    expect(swiglu(at[0], at[5], at[8], 64, 64, 64, FFN_BF16, 7, at[9], big), FFN_EINVAL, "gradient type");
    expect(swiglu(at[0], at[5], at[8], 64, 1 << 23, 8, FFN_BF16, FFN_BF16, at[9], big), FFN_EUNSUPPORTED, "N bound");
    expect(swiglu(at[0], at[5], at[8], top, 64, 64, FFN_BF16, FFN_BF16, at[9], big), FFN_EUNSUPPORTED, "M bound");
    expect(swiglu(at[0], at[5], at[8] + 8, 64, 64, 64, FFN_BF16, FFN_F32, at[9], big), FFN_EALIGN, "dWd alignment");
    expect(swiglu(at[0], at[5], at[8], 64, 64, 64, FFN_BF16, FFN_F32, at[9] + 16, big), FFN_EALIGN, "workspace alignment");
    expect(swiglu(at[0], at[5], at[8], 64, 64, 64, FFN_BF16, FFN_F32, at[9], 255), FFN_EWORKSPACE, "workspace");
    expect(swiglu(at[0], at[0] + 16, at[8], 64, 64, 64, FFN_BF16, FFN_F32, at[9], big), FFN_EINVAL, "dX over X");
    expect(swiglu(at[0], at[5], at[8], 64, 64, 64, FFN_BF16, FFN_F32, at[8], big), FFN_EINVAL, "workspace over dWd");

    auto forward = [&](const void* X, void* Y, float* mean, float* rstd, int64_t M, int64_t N, int dt, float eps) {
        return ffn_layernorm_forward(X, at[1], at[2], Y, mean, rstd, M, N, dt, eps, nullptr);
    };
    expect(forward(nullptr, at[3], f[4], f[5], 64, 64, FFN_F32, 1e-5f), FFN_EINVAL, "null X");
    expect(forward(at[0], at[3], f[4], f[5], 64, 64, FFN_F32, -1.0f), FFN_EINVAL, "eps");
    expect(forward(at[0], at[3], f[4], f[5], 64, 16392, FFN_F32, 1e-5f), FFN_EUNSUPPORTED, "N bound");
    expect(forward(at[0], at[3], f[4], f[5], top, 64, FFN_F32, 1e-5f), FFN_EUNSUPPORTED, "M bound");
    expect(forward(at[0], at[3], f[4], f[5], 64, 64, 5, 1e-5f), FFN_EINVAL, "type");
    expect(forward(at[0], at[3] + 2, f[4], f[5], 64, 64, FFN_BF16, 1e-5f), FFN_EALIGN, "alignment");
    expect(forward(at[0], at[0] + 16, f[4], f[5], 64, 64, FFN_BF16, 1e-5f), FFN_EINVAL, "Y over X");
    expect(forward(at[0], at[3], f[4], f[4], 64, 64, FFN_BF16, 1e-5f), FFN_EINVAL, "mean over rstd");
    expect(forward(nullptr, nullptr, nullptr, nullptr, 0, 64, FFN_BF16, 1e-5f), FFN_OK, "no rows");

    auto backward = [&](const void* dY, void* dX, float* dbeta, int64_t N, int dt, void* ws, size_t n) {
        return ffn_layernorm_backward(at[0], dY, at[2], f[3], f[4], dX, f[6], dbeta, 64, N, dt, ws, n, nullptr);
    };
    expect(backward(nullptr, at[5], f[7], 64, FFN_F32, at[8], big), FFN_EINVAL, "null dY");
    expect(backward(at[1], at[5], f[7], 20, FFN_F32, at[8], big), FFN_EUNSUPPORTED, "N % 8");
    expect(backward(at[1], at[5], f[7], 64, FFN_F32, at[8], 255), FFN_EWORKSPACE, "workspace");
    expect(backward(at[1], at[5], f[7], 64, FFN_F32, nullptr, big), FFN_EINVAL, "no workspace");
    expect(backward(at[1] + 4, at[5], f[7], 64, FFN_F32, at[8], big), FFN_EALIGN, "alignment");
    expect(backward(at[1], at[1] + 16, f[7], 64, FFN_F32, at[8], big), FFN_EINVAL, "dX over dY");
    expect(backward(at[1], at[5], f[6], 64, FFN_F32, at[8], big), FFN_EINVAL, "dbeta over dgamma");

    auto update = [&](const void* G, void* U, int64_t B, int64_t R, int64_t C, int dt, int steps, void* ws, size_t n) {
        return ffn_orthogonalize(G, U, B, R, C, dt, steps, ws, n, nullptr);
    };
    for (int64_t R : {64, 136}) {
        expect(update(nullptr, at[1], 1, R, 264, FFN_F32, 5, at[4], big), FFN_EINVAL, "null G");
        expect(update(at[0], at[2], 1, R, 264, FFN_F32, 0, at[4], big), FFN_EINVAL, "no steps");
        expect(update(at[0], at[2], 1, R, 264, FFN_F32, 9, at[4], big), FFN_EUNSUPPORTED, "steps");
        expect(update(at[0], at[2], 1, R, 264, FFN_F32, INT32_MAX, at[4], big), FFN_EINVAL, "most steps");
        expect(update(at[0], at[2], 1, R, 264, FFN_F32, 5, at[4], 255), FFN_EWORKSPACE, "workspace");
        expect(update(at[0], at[2], 65536, R, 264, FFN_F32, 5, at[4], big), FFN_EUNSUPPORTED, "B bound");
        expect(update(at[0], at[0] + 16, 1, R, 264, FFN_F32, 5, at[4], big), FFN_EINVAL, "U over G");
        expect(update(at[0], at[2] + 2, 1, R, 264, FFN_BF16, 5, at[4], big), FFN_EALIGN, "alignment");
        expect(update(nullptr, nullptr, 0, R, 264, FFN_BF16, 5, at[4], big), FFN_OK, "no matrices");
    }
    expect(update(at[0], at[2], 1, top - 7, 8, FFN_F32, 5, at[4], big), FFN_EUNSUPPORTED, "R bound");
    if (failures) return 2;
    std::printf("training sanitizer driver: ok\n");
    return 0;
}
