// ssd_norm.h -- host-side launch interface of the norm kernels (ssd_norm.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace ssd {

// The norm after a mixer with its gate.  A segment is one group of `group` channels of
// one row; x, z, y [rows, D], w [D].
struct NormGateArgs {
    const void *x, *z;      // z null: no gate
    const float *w;
    void *y;
    const void *dy;         // backward only, as the four below
    void *dx, *dz;
    float *dw;
    void *workspace;
    int64_t rows;
    int D, group;
    float eps;
    bool gate_first, bf16;
};

// The residual sum and the norm of the next block.  x, y [rows, D] io; residual, sum
// [rows, D] of the residual's type; scale [D] or null; w [D].
struct NormAddArgs {
    const void *x, *residual;
    const float *scale, *w;
    void *sum, *y;
    const void *dy, *dsum;      // backward: sum is an input, dsum may be null
    void *dx, *dres;
    float *dscale, *dw;
    void *workspace;
    int64_t rows;
    int D;
    float eps;
    bool bf16, res_bf16;
};

// Dropout on x: seed and offset of the generator (device), the probability of a zero.
struct NormDropArgs {
    const uint64_t *rng;
    float p;
};

// The norm's output in e4m3 [rows, D] and one scale [rows, D / group] per group of channels.
struct NormQ8Args {
    uint8_t *q;
    float *scale;
    int group;
};

// Backward: row slices, each of which leaves one partial sum per channel and parameter.
struct NormBwdPlan {
    int slices = 0;
    size_t total = 0;           // workspace bytes: fp32 [params][slices][D]
};
NormBwdPlan plan_norm_bwd(int64_t rows, int D, int group, int params, bool bf16);

hipError_t launch_norm_gate_fwd(const NormGateArgs &a, hipStream_t stream);
hipError_t launch_norm_gate_bwd(const NormGateArgs &a, const NormBwdPlan &plan, hipStream_t stream);
hipError_t launch_norm_add_fwd(const NormAddArgs &a, hipStream_t stream);
hipError_t launch_norm_add_bwd(const NormAddArgs &a, const NormBwdPlan &plan, hipStream_t stream);
hipError_t launch_norm_add_drop_fwd(const NormAddArgs &a, const NormDropArgs &d, hipStream_t stream);
hipError_t launch_norm_add_drop_bwd(const NormAddArgs &a, const NormDropArgs &d, const NormBwdPlan &plan, hipStream_t stream);
hipError_t launch_norm_add_q8(const NormAddArgs &a, const NormQ8Args &o, hipStream_t stream);

// out0 (and out1) [D] = the sums of a backward pass's partials over its slices.
hipError_t launch_norm_reduce(const float *part, float *out0, float *out1, int slices, int D, hipStream_t stream);

}  // namespace ssd
