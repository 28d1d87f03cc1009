// ssd_delta.h -- host-side launch interface of the gated delta rule kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace ssd {

// Token by token (ssd_delta_step.hip): L tokens on a state that stays in registers.
struct DeltaStepArgs {
    const float *state_in;      // null: zeros
    const void *q, *k, *v;
    const float *a, *beta;
    const int32_t *accept_len;  // null: all L tokens
    void *y;
    float *state_out;           // null: not wanted
    int32_t *err_flag;
    int b, L, H, P, N, G;
    float scale;
    bool bf16;
};

bool delta_step_supported_n(int N);
hipError_t launch_delta_step(const DeltaStepArgs &a, hipStream_t stream);

}  // namespace ssd
