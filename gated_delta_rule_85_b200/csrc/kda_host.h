// Host helpers that the translation units of libkda share; defined in kda_lib.cu.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/kda.h"

namespace kda {
namespace host {

// Keeps the message for kda_last_error (per thread) and returns `code`.
int fail(int code, const char *fmt, ...);
int cuda_fail(cudaError_t e, const char *what);
inline bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// What an entry point calls the arguments that its checks share with others, for their messages.
struct ArgNames {
    const char *required;   // all that must be given
    const char *gate, *init_state, *o, *final_state;
};
constexpr ArgNames kDeltaNames{"q, k, v, log_alpha, beta and o", "log_alpha", "init_state", "o", "final_state"};
constexpr ArgNames kDeltaStepNames{"q, k, v, log_alpha, beta, state and o", "log_alpha", "state", "o", nullptr};

// Checks shared by the prefill entry points, and by the decode ones.
int check_prefill(const void *q, const void *k, const void *v, const float *log_alpha, const float *beta,
                  const float *init_state, const void *o, const float *final_state, const int32_t *cu_seqlens, int B,
                  int T, int H, int dk, int dv, int num_seqs, int dtype, int chunk, bool gate_scalar = false,
                  const ArgNames &names = kDeltaNames);
int check_decode(const void *q, const void *k, const void *v, const float *log_alpha, const float *beta,
                 const float *state, const void *o, int N, int H, int dk, int dv, int dtype, bool gate_scalar = false,
                 const ArgNames &names = kDeltaStepNames);
int check_workspace(const void *workspace, size_t ws_bytes, size_t need);

// A unit's device status word, for kda_get_device_status; at most kStatusUnits units have one.
constexpr int kStatusUnits = 4;
struct StatusWord {
    const void *symbol;
    StatusWord *next;
    explicit StatusWord(const void *s);
};
#define KDA_STATUS_WORD static kda::host::StatusWord kda_status_word(&kda::g_status)

// A call without tokens: the final state is the initial state (or zeros).
int state_passthrough(const float *init_state, float *final_state, int num_seqs, int H, int dk, int dv,
                      cudaStream_t st);

}  // namespace host
}  // namespace kda
