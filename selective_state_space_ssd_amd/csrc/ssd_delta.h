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
int delta_step_most_rows(int N);        // the largest P
hipError_t launch_delta_step(const DeltaStepArgs &a, hipStream_t stream);

// In chunks of 64 tokens on the matrix cores (ssd_delta_chunk.hip): P a multiple of 16, N
// in {32, 64, 128} and, for bf16, 256.
struct DeltaChunkArgs {
    const void *q, *k, *v;
    const float *a, *beta;
    const float *init_state;    // null: zeros
    void *y;
    float *final_state;         // null: not wanted
    int b, L, H, P, N, G;
    float scale;
    bool bf16;
    void *workspace;
};

// A sequence of nc chunks run in segments of `per`, all at once (ssd_delta_chain.h).
struct DeltaCut {
    int segments = 1, per = 0;
};
DeltaCut cut_sequence(int64_t bh, int nc, int P, int N, bool bf16, bool back);   // back: for the backward pass

// fp32 [b, H, segments - 1, P + N, N]: what the segments but the last do to a state, and
// [b, H, segments, P, N]: the states that enter them; none for one segment.
inline size_t map_bytes(size_t bh, int P, int N, const DeltaCut &c) { return bh * (c.segments - 1) * (P + N) * N * 4; }
inline size_t entering_bytes(size_t bh, int P, int N, const DeltaCut &c) { return c.segments > 1 ? bh * c.segments * P * N * 4 : 0; }

struct DeltaChunkPlan {
    bool supported = false;
    DeltaCut cut;
    size_t off_map = 0, off_init = 0;   // behind the images: map and entering states of the segments
    size_t total = 0;                   // workspace bytes
};
bool delta_chunk_supported(int b, int L, int H, int P, int N, int G, bool bf16);
DeltaChunkPlan plan_delta_chunk(int b, int L, int H, int P, int N, int G, bool bf16);
hipError_t launch_delta_chunk(const DeltaChunkArgs &a, const DeltaChunkPlan &plan, hipStream_t stream);

// Gradients (ssd_delta_bwd.hip); the shapes of the chunked path.
struct DeltaBwdArgs {
    const void *q, *k, *v;
    const float *a, *beta;
    const float *init_state;    // null: zeros
    const void *dy;
    const float *d_final;       // null: zero
    void *dq, *dk, *dv;
    float *da, *dbeta;
    float *d_init;              // null: not wanted
    int b, L, H, P, N, G;
    float scale;
    bool bf16;
    void *workspace;
};

// The workspace begins with the chunk images; byte offsets of what follows.
struct DeltaBwdPlan {
    size_t off_e = 0, off_x = 0, off_s = 0, off_ds = 0;
    DeltaCut cut;
    size_t off_map = 0, off_init = 0, off_dmap = 0, off_dinit = 0;      // of the segments, and of their gradients
    size_t off_parts = 0, off_gate_parts = 0;   // sums of dq and dk, da and dbeta in `splits` parts, if more than 1
    int splits = 1;
    size_t total = 0;
};
DeltaBwdPlan plan_delta_bwd(int b, int L, int H, int P, int N, int G, bool bf16);
hipError_t launch_delta_bwd(const DeltaBwdArgs &a, const DeltaBwdPlan &plan, hipStream_t stream);

}  // namespace ssd
