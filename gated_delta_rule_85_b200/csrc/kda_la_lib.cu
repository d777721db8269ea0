// libkda: the entry points of linear attention with a decay for each head (include/kda.h).
#include "kda_common.cuh"
#include "kda_host.h"
#include "kda_la.cuh"
#include "kda_la_simt.cuh"
#include "kda_la_step.cuh"
#include "kda_la_tc.cuh"

KDA_STATUS_WORD;

using namespace kda::host;

namespace {

constexpr ArgNames kForwardNames{"q, k, v, log_decay and o", "log_decay", "init_state", "o", "final_state"};
constexpr ArgNames kPoolNames{"q, k, v, log_decay and o", "log_decay", "state_pool", "o", "state_pool"};
constexpr ArgNames kBackwardNames{"q, k, v, log_decay and d_o", "log_decay", "init_state", "d_o", "dfinal_state"};
constexpr ArgNames kStepNames{"q, k, v, log_decay, state and o", "log_decay", "state", "o", nullptr};
constexpr ArgNames kPoolStepNames{"q, k, v, log_decay, state_pool and o", "log_decay", "state_pool", "o", nullptr};

// Shared checks of the prefill and its backward pass: s0 and last are two optional fp32 state tensors.
int check_la(const void *q, const void *k, const void *v, const float *log_decay, const float *s0, const void *o,
             const float *last, const int32_t *cu_seqlens, int B, int T, int H, int dk, int dv, int num_seqs, int dtype,
             const ArgNames &names) {
    // beta is not part of this operator: log_decay stands in (both are 4-byte aligned device arrays)
    int rc = check_prefill(q, k, v, log_decay, log_decay, s0, o, last, cu_seqlens, B, T, H, dk, dv, num_seqs, dtype, 64,
                           true, names);
    if (rc) return rc;
    if ((long long)B * T > 0x7fffffffLL)
        return fail(KDA_ERR_UNSUPPORTED, "B*T=%lld exceeds 2^31 - 1 tokens", (long long)B * T);
    return KDA_OK;
}

bool la_sizes_ok(int B, int T, int H, int dk, int dv, int num_seqs, int dtype) {
    return B >= 1 && T >= 0 && H >= 1 && H <= 65535 && num_seqs >= 0 && num_seqs <= 65535 &&
           (long long)B * T <= 0x7fffffffLL && (dk == 64 || dk == 128) && (dv == 64 || dv == 128) &&
           (dtype == KDA_BF16 || dtype == KDA_F32);
}

// A sequence of one chunk at most is never cut between CTAs and needs no carried state.
size_t la_forward_ws(int T, int H, int dk, int dv, int num_seqs, int dtype, bool with_slots) {
    if (T <= (dtype == KDA_BF16 ? kda::la::kC : kda::la::kSimtC)) return 0;
    return kda::la::carry_bytes(kda::la::kSMs, dk, dv) +
           (with_slots ? (size_t)num_seqs * H * dk * dv * sizeof(float) : 0);
}

int la_forward(const kda::la::Call &c, const void *q, const void *k, const void *v, const float *s0, void *o,
               float *last, int dk, int dv, int dtype, void *ws) {
    cudaError_t e = cudaErrorInvalidValue;
#define KDA_LA(DK, DV)                                                                                          \
    if (dk == DK && dv == DV)                                                                                   \
        e = dtype == KDA_BF16                                                                                   \
                ? kda::la::tc_forward<DK, DV>(c, q, k, v, s0, o, last, (float *)ws)                              \
                : kda::la::simt_forward<DK, DV, float>(c, q, k, v, s0, o, last, (float *)ws)
    KDA_LA(64, 64);
    KDA_LA(64, 128);
    KDA_LA(128, 64);
    KDA_LA(128, 128);
#undef KDA_LA
    return e == cudaSuccess ? KDA_OK : cuda_fail(e, "linear attention launch");
}

int la_step(const void *q, const void *k, const void *v, const float *log_decay, float *state, void *o, int N, int H,
            int dk, int dv, int dtype, const int32_t *slots, int num_slots, cudaStream_t st) {
    const unsigned pairs = (unsigned)((long long)N * H);
#define KDA_LA(DK, DV, TT)                                                                                       \
    kda::la::la_step_kernel<DK, DV, TT><<<pairs, 256, 0, st>>>((const TT *)q, (const TT *)k, (const TT *)v, log_decay, \
                                                               state, (TT *)o, slots, num_slots, H)
#define KDA_LA2(DK, DV)                                                 \
    if (dk == DK && dv == DV) {                                         \
        if (dtype == KDA_BF16) KDA_LA(DK, DV, __nv_bfloat16);           \
        else KDA_LA(DK, DV, float);                                     \
    }
    KDA_LA2(64, 64)
    KDA_LA2(64, 128)
    KDA_LA2(128, 64)
    KDA_LA2(128, 128)
#undef KDA_LA2
#undef KDA_LA
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? KDA_OK : cuda_fail(e, "la_step launch");
}

}  // namespace

extern "C" {

size_t kda_la_chunk_forward_workspace_size(int B, int T, int H, int dk, int dv, int num_seqs, int dtype,
                                           int with_slots) {
    if (!la_sizes_ok(B, T, H, dk, dv, num_seqs, dtype) || T == 0 || num_seqs == 0) return 0;
    return la_forward_ws(T, H, dk, dv, num_seqs, dtype, with_slots != 0);
}

int kda_la_chunk_forward(const void *q, const void *k, const void *v, const float *log_decay,
                         const float *init_state, void *o, float *final_state, const int32_t *cu_seqlens, int B,
                         int T, int H, int dk, int dv, int num_seqs, int dtype, void *workspace, size_t ws_bytes,
                         void *stream) {
    int rc = check_la(q, k, v, log_decay, init_state, o, final_state, cu_seqlens, B, T, H, dk, dv, num_seqs, dtype,
                      kForwardNames);
    if (rc) return rc;
    rc = check_workspace(workspace, ws_bytes,
                         kda_la_chunk_forward_workspace_size(B, T, H, dk, dv, num_seqs, dtype, 0));
    if (rc || num_seqs == 0) return rc;
    cudaStream_t st = (cudaStream_t)stream;
    if (T == 0) return state_passthrough(init_state, final_state, num_seqs, H, dk, dv, st);
    const kda::la::Call c{cu_seqlens, nullptr, B, T, H, num_seqs, 0, log_decay, st};
    return la_forward(c, q, k, v, init_state, o, final_state, dk, dv, dtype, workspace);
}

int kda_la_chunk_forward_slots(const void *q, const void *k, const void *v, const float *log_decay,
                               float *state_pool, const int32_t *slots, void *o, const int32_t *cu_seqlens, int B,
                               int T, int H, int dk, int dv, int num_seqs, int num_slots, int dtype,
                               void *workspace, size_t ws_bytes, void *stream) {
    int rc = check_la(q, k, v, log_decay, state_pool, o, state_pool, cu_seqlens, B, T, H, dk, dv, num_seqs, dtype,
                      kPoolNames);
    if (rc) return rc;
    if (num_seqs > 0 && (!state_pool || !slots))
        return fail(KDA_ERR_INVALID_ARG, "state_pool and slots are required");
    if (num_slots < 1) return fail(KDA_ERR_INVALID_ARG, "num_slots=%d must be at least 1", num_slots);
    if (slots && !aligned(slots, 4)) return fail(KDA_ERR_MISALIGNED, "slots is not 4-byte aligned");
    rc = check_workspace(workspace, ws_bytes,
                         kda_la_chunk_forward_workspace_size(B, T, H, dk, dv, num_seqs, dtype, 1));
    if (rc || num_seqs == 0 || T == 0) return rc;   // without tokens the states stay in their slots
    const kda::la::Call c{cu_seqlens, slots, B, T, H, num_seqs, num_slots, log_decay, (cudaStream_t)stream};
    return la_forward(c, q, k, v, state_pool, o, state_pool, dk, dv, dtype, workspace);
}

int kda_la_recurrent_step(const void *q, const void *k, const void *v, const float *log_decay, float *state, void *o,
                          int N, int H, int dk, int dv, int dtype, void *stream) {
    int rc = check_decode(q, k, v, log_decay, log_decay, state, o, N, H, dk, dv, dtype, true, kStepNames);
    if (rc || N == 0) return rc;
    return la_step(q, k, v, log_decay, state, o, N, H, dk, dv, dtype, nullptr, 0, (cudaStream_t)stream);
}

int kda_la_recurrent_step_slots(const void *q, const void *k, const void *v, const float *log_decay,
                                float *state_pool, const int32_t *slots, void *o, int N, int H, int dk, int dv,
                                int num_slots, int dtype, void *stream) {
    int rc = check_decode(q, k, v, log_decay, log_decay, state_pool, o, N, H, dk, dv, dtype, true, kPoolStepNames);
    if (rc || N == 0) return rc;
    if (!slots) return fail(KDA_ERR_INVALID_ARG, "slots is required");
    if (!aligned(slots, 4)) return fail(KDA_ERR_MISALIGNED, "slots is not 4-byte aligned");
    if (num_slots < 1) return fail(KDA_ERR_INVALID_ARG, "num_slots=%d must be at least 1", num_slots);
    return la_step(q, k, v, log_decay, state_pool, o, N, H, dk, dv, dtype, slots, num_slots, (cudaStream_t)stream);
}

size_t kda_la_chunk_backward_workspace_size(int B, int T, int H, int dk, int dv, int num_seqs, int dtype) {
    if (!la_sizes_ok(B, T, H, dk, dv, num_seqs, dtype) || T == 0 || num_seqs == 0) return 0;
    return 2 * la_forward_ws(T, H, dk, dv, num_seqs, dtype, false);
}

int kda_la_chunk_backward(const void *q, const void *k, const void *v, const float *log_decay,
                          const float *init_state, const void *d_o, const float *dfinal_state, void *dq,
                          void *dk_out, void *dv_out, float *dinit_state, const int32_t *cu_seqlens, int B, int T,
                          int H, int dk, int dv, int num_seqs, int dtype, void *workspace, size_t ws_bytes,
                          void *stream) {
    int rc = check_la(q, k, v, log_decay, init_state, d_o, dfinal_state, cu_seqlens, B, T, H, dk, dv, num_seqs, dtype,
                      kBackwardNames);
    if (rc) return rc;
    if (T > 0 && (!dq || !dk_out || !dv_out)) return fail(KDA_ERR_INVALID_ARG, "dq, dk and dv are required");
    const void *p16[] = {dq, dk_out, dv_out, dinit_state};
    const char *n16[] = {"dq", "dk", "dv", "dinit_state"};
    for (int i = 0; i < 4; ++i)
        if (p16[i] && !aligned(p16[i], 16)) return fail(KDA_ERR_MISALIGNED, "%s is not 16-byte aligned", n16[i]);
    rc = check_workspace(workspace, ws_bytes,
                         kda_la_chunk_backward_workspace_size(B, T, H, dk, dv, num_seqs, dtype));
    if (rc || num_seqs == 0) return rc;
    cudaStream_t st = (cudaStream_t)stream;
    if (T == 0) return state_passthrough(dfinal_state, dinit_state, num_seqs, H, dk, dv, st);
    const kda::la::Call c{cu_seqlens, nullptr, B, T, H, num_seqs, 0, log_decay, st};
    cudaError_t e = cudaErrorInvalidValue;
#define KDA_LA(DK, DV)                                                                                             \
    if (dk == DK && dv == DV)                                                                                      \
        e = dtype == KDA_BF16                                                                                      \
                ? kda::la::tc_backward<DK, DV>(c, q, k, v, d_o, init_state, dfinal_state, dq, dk_out, dv_out,      \
                                               dinit_state, (float *)workspace)                                   \
                : kda::la::simt_backward<DK, DV, float>(c, q, k, v, d_o, init_state, dfinal_state, dq, dk_out, dv_out, \
                                                        dinit_state, (float *)workspace)
    KDA_LA(64, 64);
    KDA_LA(64, 128);
    KDA_LA(128, 64);
    KDA_LA(128, 128);
#undef KDA_LA
    return e == cudaSuccess ? KDA_OK : cuda_fail(e, "linear attention backward launch");
}

}  // extern "C"
