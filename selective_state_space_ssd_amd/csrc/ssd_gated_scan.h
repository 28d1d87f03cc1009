// ssd_gated_scan.h -- host-side launch interface of the gated scan (ssd_gated_scan.hip,
// ssd_gated_scan_step.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace ssd {

// h_t = alpha_t h_{t-1} + u_t per channel.  x, y [b, L, D] io; a [b, L, D] io or fp32; states
// [b, D] fp32; kept [b, ceil(L / kGatedScanKeep), D] fp32, the state before every
// kGatedScanKeep-th token.
constexpr int kGatedScanKeep = 32;

struct GatedScanArgs {
    const void *x, *a;
    const float *init_state;    // null: zeros
    void *y;                    // null: not wanted
    float *kept, *final_state;  // null: not wanted
    const void *dy;             // backward only, as the four below
    const float *d_final;       // null: zeros
    void *dx, *da;
    float *d_init;              // null: not wanted
    void *workspace;
    int b, L, D;
    int looks;                  // at another block's word, before a wait gives up
    bool sigmoid, bf16, a_bf16;
    bool keep_error;            // the workspace's error word stays, of the pass before
};

struct GatedStepArgs {
    const float *state_in;
    const void *x, *a;
    const int32_t *accept_len;  // null: all
    void *y;
    float *state_out;
    int32_t *err_flag;
    int b, K, D;
    bool sigmoid, bf16, a_bf16;
};

// Whether the launches of this shape stay inside a grid's limits.
bool gated_scan_supported(int b, int L, int D);
size_t gated_scan_workspace(int b, int L, int D, bool bf16, bool backward);    // without kept states
// Whether sequences of L > 0 tokens are cut into blocks that wait for each other, whatever their type
// and pass; the others use no workspace.
bool gated_scan_waits(int L);

hipError_t launch_gated_scan_fwd(const GatedScanArgs &a, hipStream_t stream);
hipError_t launch_gated_scan_bwd(const GatedScanArgs &a, hipStream_t stream);   // kept is an input
// err_out = the error word of the last pass in the workspace; null: 0.
hipError_t launch_gated_scan_error(const void *workspace, int32_t *err_out, hipStream_t stream);
hipError_t launch_gated_scan_step(const GatedStepArgs &a, hipStream_t stream);

}  // namespace ssd
