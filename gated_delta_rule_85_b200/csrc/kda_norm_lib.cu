// libkda: the entry points of group norm with an activation (include/kda.h).
#include "kda_host.h"
#include "kda_norm.cuh"

using namespace kda::host;

namespace {

// 65535 blocks of 256 channels; samples and groups that a grid and 32-bit counts hold.
constexpr int kMaxC = 65535 * 256, kMaxL = 1 << 30;
constexpr long long kMaxN = 1LL << 24, kMaxGroups = 1LL << 30;

int check_norm(const void *x, const void *y, const float *mean, const float *rstd, const float *weight,
               const float *bias, const void *gate, long long N, int L, int C, int G, int act, int dtype) {
    if (N < 0 || L < 1 || C < 1 || G < 1) return fail(KDA_ERR_INVALID_ARG, "bad sizes N=%lld L=%d C=%d G=%d", N, L, C, G);
    if (C % G) return fail(KDA_ERR_INVALID_ARG, "C=%d is not a multiple of G=%d", C, G);
    if (act != KDA_ACT_NONE && act != KDA_ACT_SILU && act != KDA_ACT_SIGMOID)
        return fail(KDA_ERR_INVALID_ARG, "act=%d is not a KDA_ACT_* value", act);
    if (dtype != KDA_BF16 && dtype != KDA_F32) return fail(KDA_ERR_UNSUPPORTED, "dtype=%d", dtype);
    if (C > kMaxC || L > kMaxL) return fail(KDA_ERR_UNSUPPORTED, "C=%d above 16776960 or L=%d above 2^30", C, L);
    if (N > kMaxN || N > kMaxGroups / G)
        return fail(KDA_ERR_UNSUPPORTED, "N=%lld with G=%d: at most 2^24 samples and 2^30 groups", N, G);
    if (N == 0) return KDA_OK;
    if (!x || !y || !mean || !rstd) return fail(KDA_ERR_INVALID_ARG, "x, mean, rstd and the outputs are required");
    const void *p16[] = {x, y, gate};
    const char *n16[] = {"x", "y (dx)", "gate"};
    for (int i = 0; i < 3; ++i)
        if (p16[i] && !aligned(p16[i], 16)) return fail(KDA_ERR_MISALIGNED, "%s is not 16-byte aligned", n16[i]);
    const void *p4[] = {mean, rstd, weight, bias};
    for (int i = 0; i < 4; ++i)
        if (p4[i] && !aligned(p4[i], 4)) return fail(KDA_ERR_MISALIGNED, "an fp32 array is not 4-byte aligned");
    return KDA_OK;
}

}  // namespace

extern "C" {

size_t kda_group_norm_workspace_size(long long N, int L, int C, int G, int dtype, int backward) {
    if (N < 1 || L < 1 || C < 1 || G < 1 || C % G || (dtype != KDA_BF16 && dtype != KDA_F32)) return 0;
    if (C > kMaxC || L > kMaxL || N > kMaxN || N > kMaxGroups / G) return 0;   // the calls refuse these
    // (with and without a gate: the forms may differ)
    const int es = dtype == KDA_BF16 ? 2 : 4;
    return std::max(kda::norm::plan_of(N, L, C, G, es, false, backward != 0).ws,
                    kda::norm::plan_of(N, L, C, G, es, true, backward != 0).ws);
}

int kda_group_norm_forward(const void *x, const float *weight, const float *bias, const void *gate, void *y,
                           float *mean, float *rstd, long long N, int L, int C, int G, float eps, int act, int dtype,
                           void *workspace, size_t ws_bytes, void *stream) {
    int rc = check_norm(x, y, mean, rstd, weight, bias, gate, N, L, C, G, act, dtype);
    if (rc) return rc;
    if (!(eps > 0.f)) return fail(KDA_ERR_INVALID_ARG, "eps=%g must be above 0", (double)eps);
    if (N == 0) return KDA_OK;
    const int es = dtype == KDA_BF16 ? 2 : 4;
    const kda::norm::Plan s = kda::norm::plan_of(N, L, C, G, es, gate != nullptr, false);
    if ((rc = check_workspace(workspace, ws_bytes, s.ws))) return rc;
    kda::norm::Args a{};
    a.x = x; a.gate = gate; a.weight = weight; a.bias = bias; a.y = y; a.mean = mean; a.rstd = rstd; a.eps = eps;
    a.ws = workspace; a.N = N;
    const cudaError_t e = es == 2 ? kda::norm::launch<__nv_bfloat16>(s, a, act, false, (cudaStream_t)stream)
                                  : kda::norm::launch<float>(s, a, act, false, (cudaStream_t)stream);
    return e == cudaSuccess ? KDA_OK : cuda_fail(e, "group norm launch");
}

int kda_group_norm_backward(const void *dy, const void *x, const float *mean, const float *rstd, const float *weight,
                            const float *bias, const void *gate, void *dx, void *dgate, float *dweight, float *dbias,
                            long long N, int L, int C, int G, int act, int dtype, void *workspace, size_t ws_bytes,
                            void *stream) {
    int rc = check_norm(x, dx, mean, rstd, weight, bias, gate, N, L, C, G, act, dtype);
    if (rc) return rc;
    if (N == 0) {   // no samples: the sums are empty
        const size_t bytes = (size_t)C * sizeof(float);
        cudaError_t e = cudaSuccess;
        if (dweight) e = cudaMemsetAsync(dweight, 0, bytes, (cudaStream_t)stream);
        if (dbias && e == cudaSuccess) e = cudaMemsetAsync(dbias, 0, bytes, (cudaStream_t)stream);
        return e == cudaSuccess ? KDA_OK : cuda_fail(e, "clearing dweight and dbias");
    }
    if (!dy) return fail(KDA_ERR_INVALID_ARG, "dy is required");
    if (gate && !dgate) return fail(KDA_ERR_INVALID_ARG, "dgate is required with a gate");
    if (!aligned(dy, 16) || (dgate && !aligned(dgate, 16)))
        return fail(KDA_ERR_MISALIGNED, "dy or dgate is not 16-byte aligned");
    if ((dweight && !aligned(dweight, 4)) || (dbias && !aligned(dbias, 4)))
        return fail(KDA_ERR_MISALIGNED, "dweight or dbias is not 4-byte aligned");
    const int es = dtype == KDA_BF16 ? 2 : 4;
    const kda::norm::Plan s = kda::norm::plan_of(N, L, C, G, es, gate != nullptr, true);
    if ((rc = check_workspace(workspace, ws_bytes, s.ws))) return rc;
    kda::norm::Args a{};
    a.dy = dy; a.x = x; a.gate = gate; a.weight = weight; a.bias = bias; a.y = dx; a.dgate = dgate;
    a.mean = const_cast<float *>(mean); a.rstd = const_cast<float *>(rstd); a.dweight = dweight; a.dbias = dbias;
    a.ws = workspace; a.N = N;
    const cudaError_t e = es == 2 ? kda::norm::launch<__nv_bfloat16>(s, a, act, true, (cudaStream_t)stream)
                                  : kda::norm::launch<float>(s, a, act, true, (cudaStream_t)stream);
    return e == cudaSuccess ? KDA_OK : cuda_fail(e, "group norm backward launch");
}

}  // extern "C"
