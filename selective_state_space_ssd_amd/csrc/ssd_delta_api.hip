// ssd_delta_api.hip -- host-side checks and dispatch of the gated delta rule.
#include <limits.h>

#include "ssd_checks.h"
#include "ssd_delta.h"
#include "ssd_kernels.h"
#include "ssd_mi355x.h"

namespace {

using ssd::aligned;
using ssd::any_alias;
using ssd::Range;

bool known(ssd_dtype_t io) { return io == SSD_DTYPE_F32 || io == SSD_DTYPE_BF16; }

ssd_status_t check_dims(int b, int L, int H, int P, int N, int G, ssd_dtype_t io) {
    if (!known(io)) return SSD_ERR_UNSUPPORTED;
    if (b < 0 || L < 0 || H <= 0 || P <= 0 || N <= 0 || G <= 0) return SSD_ERR_BAD_DIM;
    if (H % G != 0) return SSD_ERR_GROUPS;
    if (!ssd::delta_step_supported_n(N) || H > 65535 || b > 65535) return SSD_ERR_UNSUPPORTED;
    // the kernels count tokens in 31 bits, up to a chunk past the last one, and a launch's
    // dimension holds fewer than 2^24 blocks of state rows
    if (L > INT_MAX - 64 || P > ssd::delta_step_most_rows(N)) return SSD_ERR_UNSUPPORTED;
    return SSD_OK;
}

// Sequences up to this length go token by token, in one launch that keeps no workspace.
// Both sides, us, token by token / in chunks, at P = 64 and one group:
//   bf16, N = 64:   32 x 80 heads, 16 tokens 53 / 73, 24 tokens 85 / 71;  8 heads, 24 tokens 16 / 20, 32 tokens 21 / 21
//   bf16, N = 128:  32 x 80 heads, 16 tokens 78 / 96, 24 tokens 108 / 95;  8 heads, 24 tokens 19 / 20, 32 tokens 23 / 20
//   fp32, N = 64:   32 x 80 heads, 32 tokens 91 / 102, 48 tokens 130 / 105;  8 heads, 32 tokens 17 / 20, 48 tokens 24 / 20
//   fp32, N = 128:  32 x 80 heads, 32 tokens 136 / 241;  8 heads, 32 tokens 21 / 20, 48 tokens 30 / 20
int most_by_token(ssd_dtype_t io) { return io == SSD_DTYPE_BF16 ? 24 : 32; }

// The chunked path of a sequence, unless it is short or no chunk kernel runs its shape.
ssd::DeltaChunkPlan sequence_plan(int b, int L, int H, int P, int N, int G, ssd_dtype_t io) {
    if (b == 0 || L <= most_by_token(io)) return {};
    return ssd::plan_delta_chunk(b, L, H, P, N, G, io == SSD_DTYPE_BF16);
}

ssd_status_t done(hipError_t e) { return e == hipSuccess ? SSD_OK : SSD_ERR_HIP; }

}  // namespace

extern "C" {

ssd_status_t ssd_gated_delta_step(const float *state_in, const void *q, const void *k,
                                  const void *v, const float *a, const float *beta,
                                  const int32_t *accept_len, void *y, float *state_out,
                                  int32_t *err_flag, int b, int K, int H, int P, int N, int G,
                                  float scale, ssd_dtype_t io, void *hip_stream) {
    if (const ssd_status_t st = check_dims(b, K, H, P, N, G, io); st != SSD_OK) return st;
    if (K < 1 || K > 16) return SSD_ERR_UNSUPPORTED;
    if (b == 0) return SSD_OK;
    if (!state_in || !q || !k || !v || !a || !beta || !y || !state_out) return SSD_ERR_NULL_ARG;
    const bool bf16 = io == SSD_DTYPE_BF16;
    const size_t esz = bf16 ? 2 : 4;
    if (!aligned(state_in, 16) || !aligned(state_out, 16) || !aligned(q, 16) || !aligned(k, 16) ||
        !aligned(v, esz) || !aligned(y, esz) || !aligned(a, 4) || !aligned(beta, 4) ||
        !aligned(accept_len, 4) || !aligned(err_flag, 4))
        return SSD_ERR_ALIGN;
    const size_t st = size_t(b) * H * P * N * 4, qk = size_t(b) * K * G * N * esz;
    const size_t vy = size_t(b) * K * H * P * esz, gt = size_t(b) * K * H * 4;
    const Range rin(state_in, st), rout(state_out, st);
    if (rin.overlaps(rout) && !rin.same(rout)) return SSD_ERR_ALIAS;
    const Range ins[] = {Range(q, qk), Range(k, qk), Range(v, vy), Range(a, gt), Range(beta, gt),
                         Range(accept_len, size_t(b) * 4)};
    const Range outs[] = {Range(y, vy), rout, Range(err_flag, 4)};
    if (any_alias(ins, outs) || outs[0].overlaps(rin) || outs[2].overlaps(rin)) return SSD_ERR_ALIAS;
    ssd::DeltaStepArgs s{};
    s.state_in = state_in; s.q = q; s.k = k; s.v = v; s.a = a; s.beta = beta;
    s.accept_len = accept_len; s.y = y; s.state_out = state_out; s.err_flag = err_flag;
    s.b = b; s.L = K; s.H = H; s.P = P; s.N = N; s.G = G; s.scale = scale; s.bf16 = bf16;
    return done(ssd::launch_delta_step(s, static_cast<hipStream_t>(hip_stream)));
}

size_t ssd_gated_delta_fwd_workspace_bytes(int b, int L, int H, int P, int N, int G,
                                           ssd_dtype_t io) {
    if (check_dims(b, L, H, P, N, G, io) != SSD_OK) return size_t(-1);
    return sequence_plan(b, L, H, P, N, G, io).total;
}

ssd_status_t ssd_gated_delta_fwd(const void *q, const void *k, const void *v, const float *a,
                                 const float *beta, const float *init_state, void *y,
                                 float *final_state, int b, int L, int H, int P, int N, int G,
                                 float scale, ssd_dtype_t io, void *workspace,
                                 size_t workspace_bytes, void *hip_stream) {
    if (const ssd_status_t st = check_dims(b, L, H, P, N, G, io); st != SSD_OK) return st;
    const hipStream_t stream = static_cast<hipStream_t>(hip_stream);
    const size_t st = size_t(b) * H * P * N * 4;
    const Range rinit(init_state, st), rfin(final_state, st);
    if (b == 0) return SSD_OK;
    if (!aligned(init_state, 16) || !aligned(final_state, 16)) return SSD_ERR_ALIGN;
    if (rinit.overlaps(rfin)) return SSD_ERR_ALIAS;
    if (L == 0) return final_state ? done(ssd::launch_copy_state(init_state, final_state, st / 4, stream)) : SSD_OK;
    if (!q || !k || !v || !a || !beta || !y) return SSD_ERR_NULL_ARG;
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(y, 16) || !aligned(a, 4) ||
        !aligned(beta, 4) || !aligned(workspace, 16))
        return SSD_ERR_ALIGN;
    const bool bf16 = io == SSD_DTYPE_BF16;
    const size_t esz = bf16 ? 2 : 4;
    const size_t qk = size_t(b) * L * G * N * esz, vy = size_t(b) * L * H * P * esz, gt = size_t(b) * L * H * 4;
    const Range ins[] = {Range(q, qk), Range(k, qk), Range(v, vy), Range(a, gt), Range(beta, gt), rinit};
    const ssd::DeltaChunkPlan plan = sequence_plan(b, L, H, P, N, G, io);
    if (plan.total > 0 && (!workspace || workspace_bytes < plan.total)) return SSD_ERR_WORKSPACE;
    const Range outs[] = {Range(y, vy), rfin, Range(workspace, plan.total)};
    if (any_alias(ins, outs)) return SSD_ERR_ALIAS;
    if (plan.supported) {
        ssd::DeltaChunkArgs c{};
        c.q = q; c.k = k; c.v = v; c.a = a; c.beta = beta; c.init_state = init_state;
        c.y = y; c.final_state = final_state; c.workspace = workspace;
        c.b = b; c.L = L; c.H = H; c.P = P; c.N = N; c.G = G; c.scale = scale; c.bf16 = bf16;
        return done(ssd::launch_delta_chunk(c, plan, stream));
    }
    ssd::DeltaStepArgs s{};
    s.state_in = init_state; s.q = q; s.k = k; s.v = v; s.a = a; s.beta = beta;
    s.y = y; s.state_out = final_state;
    s.b = b; s.L = L; s.H = H; s.P = P; s.N = N; s.G = G; s.scale = scale; s.bf16 = bf16;
    return done(ssd::launch_delta_step(s, stream));
}

size_t ssd_gated_delta_bwd_workspace_bytes(int b, int L, int H, int P, int N, int G,
                                           ssd_dtype_t io) {
    if (check_dims(b, L, H, P, N, G, io) != SSD_OK) return size_t(-1);
    if (!ssd::delta_chunk_supported(b, L, H, P, N, G, io == SSD_DTYPE_BF16)) return size_t(-1);
    return ssd::plan_delta_bwd(b, L, H, P, N, G, io == SSD_DTYPE_BF16).total;
}

ssd_status_t ssd_gated_delta_bwd(const void *q, const void *k, const void *v, const float *a,
                                 const float *beta, const float *init_state, const void *dy,
                                 const float *d_final, void *dq, void *dk, void *dv, float *da,
                                 float *dbeta, float *d_init, int b, int L, int H, int P, int N,
                                 int G, float scale, ssd_dtype_t io, void *workspace,
                                 size_t workspace_bytes, void *hip_stream) {
    if (const ssd_status_t st = check_dims(b, L, H, P, N, G, io); st != SSD_OK) return st;
    const bool bf16 = io == SSD_DTYPE_BF16;
    if (!ssd::delta_chunk_supported(b, L, H, P, N, G, bf16)) return SSD_ERR_UNSUPPORTED;
    const hipStream_t stream = static_cast<hipStream_t>(hip_stream);
    const size_t st = size_t(b) * H * P * N * 4;
    const Range rdf(d_final, st), rdi(d_init, st);
    if (b == 0) return SSD_OK;
    if (!aligned(d_final, 16) || !aligned(d_init, 16)) return SSD_ERR_ALIGN;
    if (rdi.overlaps(rdf)) return SSD_ERR_ALIAS;
    if (L == 0) return d_init ? done(ssd::launch_copy_state(d_final, d_init, st / 4, stream)) : SSD_OK;
    if (!q || !k || !v || !a || !beta || !dy || !dq || !dk || !dv || !da || !dbeta) return SSD_ERR_NULL_ARG;
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(dy, 16) || !aligned(dq, 16) ||
        !aligned(dk, 16) || !aligned(dv, 16) || !aligned(init_state, 16) || !aligned(a, 4) || !aligned(beta, 4) ||
        !aligned(da, 4) || !aligned(dbeta, 4) || !aligned(workspace, 16))
        return SSD_ERR_ALIGN;
    const ssd::DeltaBwdPlan plan = ssd::plan_delta_bwd(b, L, H, P, N, G, bf16);
    if (!workspace || workspace_bytes < plan.total) return SSD_ERR_WORKSPACE;
    const size_t esz = bf16 ? 2 : 4;
    const size_t qk = size_t(b) * L * G * N * esz, vy = size_t(b) * L * H * P * esz, gt = size_t(b) * L * H * 4;
    const Range ins[] = {Range(q, qk), Range(k, qk), Range(v, vy), Range(a, gt), Range(beta, gt),
                         Range(init_state, st), Range(dy, vy), rdf};
    const Range outs[] = {Range(dq, qk), Range(dk, qk), Range(dv, vy), Range(da, gt), Range(dbeta, gt), rdi,
                          Range(workspace, plan.total)};
    if (any_alias(ins, outs)) return SSD_ERR_ALIAS;
    ssd::DeltaBwdArgs c{};
    c.q = q; c.k = k; c.v = v; c.a = a; c.beta = beta; c.init_state = init_state; c.dy = dy; c.d_final = d_final;
    c.dq = dq; c.dk = dk; c.dv = dv; c.da = da; c.dbeta = dbeta; c.d_init = d_init; c.workspace = workspace;
    c.b = b; c.L = L; c.H = H; c.P = P; c.N = N; c.G = G; c.scale = scale; c.bf16 = bf16;
    return done(ssd::launch_delta_bwd(c, plan, stream));
}

}  // extern "C"
