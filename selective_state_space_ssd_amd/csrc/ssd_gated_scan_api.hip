// ssd_gated_scan_api.hip -- host-side checks and dispatch of the gated scan.
#include <algorithm>
#include <atomic>

#include "ssd_checks.h"
#include "ssd_gated_scan.h"
#include "ssd_kernels.h"
#include "ssd_mi355x.h"

namespace {

using ssd::aligned;
using ssd::any_alias;
using ssd::Range;

static_assert(SSD_GATED_SCAN_KEEP == ssd::kGatedScanKeep);

size_t elem(ssd_dtype_t io) { return io == SSD_DTYPE_BF16 ? 2 : 4; }

ssd_status_t check_dims(int b, int L, int D, ssd_dtype_t io, ssd_dtype_t a_io) {
    if ((io != SSD_DTYPE_F32 && io != SSD_DTYPE_BF16) || (a_io != SSD_DTYPE_F32 && a_io != io)) return SSD_ERR_UNSUPPORTED;
    if (b < 0 || L < 0 || D <= 0) return SSD_ERR_BAD_DIM;
    return ssd::gated_scan_supported(b, L, D) ? SSD_OK : SSD_ERR_UNSUPPORTED;
}

size_t kept_bytes(int b, int L, int D) {
    return size_t(b) * ((size_t(L) + SSD_GATED_SCAN_KEEP - 1) / SSD_GATED_SCAN_KEEP) * D * 4;
}

// Of the backward call without its kept states: the two passes that it may run use the same place.
size_t words_bytes(int b, int L, int D, ssd_dtype_t io) {
    const bool bf16 = io == SSD_DTYPE_BF16;
    const size_t n = std::max(ssd::gated_scan_workspace(b, L, D, bf16, false), ssd::gated_scan_workspace(b, L, D, bf16, true));
    return (n + 15) / 16 * 16;
}

// looks at another block's word before a wait gives up; 2^20 take about a second
std::atomic<int> wait_limit{1 << 20};

ssd_status_t done(hipError_t e) { return e == hipSuccess ? SSD_OK : SSD_ERR_HIP; }

}  // namespace

extern "C" {

ssd_status_t ssd_gated_scan_step(const float *state_in, const void *x, const void *a,
                                 const int32_t *accept_len, void *y, float *state_out,
                                 int32_t *err_flag, int b, int K, int D, int sigmoid, ssd_dtype_t io,
                                 ssd_dtype_t a_io, void *hip_stream) {
    if (const ssd_status_t st = check_dims(b, K, D, io, a_io); st != SSD_OK) return st;
    if (K < 1 || K > 16) return SSD_ERR_UNSUPPORTED;
    if (b == 0) return SSD_OK;
    if (!state_in || !x || !a || !y || !state_out) return SSD_ERR_NULL_ARG;
    if (!aligned(state_in, 16) || !aligned(x, 16) || !aligned(a, 16) || !aligned(y, 16) || !aligned(state_out, 16) ||
        !aligned(accept_len, 4) || !aligned(err_flag, 4))
        return SSD_ERR_ALIGN;
    const size_t n = size_t(b) * K * D, st = size_t(b) * D * 4;
    const Range rin(state_in, st), rout(state_out, st);
    if (rin.overlaps(rout) && !rin.same(rout)) return SSD_ERR_ALIAS;
    const Range ins[] = {Range(x, n * elem(io)), Range(a, n * elem(a_io)), Range(accept_len, size_t(b) * 4)};
    const Range outs[] = {Range(y, n * elem(io)), rout, Range(err_flag, 4)};
    if (any_alias(ins, outs) || outs[0].overlaps(rin) || outs[2].overlaps(rin)) return SSD_ERR_ALIAS;
    ssd::GatedStepArgs s{};
    s.state_in = state_in; s.x = x; s.a = a; s.accept_len = accept_len; s.y = y; s.state_out = state_out;
    s.err_flag = err_flag;
    s.b = b; s.K = K; s.D = D; s.sigmoid = sigmoid != 0; s.bf16 = io == SSD_DTYPE_BF16; s.a_bf16 = a_io == SSD_DTYPE_BF16;
    return done(ssd::launch_gated_scan_step(s, static_cast<hipStream_t>(hip_stream)));
}

size_t ssd_gated_scan_fwd_workspace_bytes(int b, int L, int D, ssd_dtype_t io, ssd_dtype_t a_io) {
    if (check_dims(b, L, D, io, a_io) != SSD_OK) return size_t(-1);
    return ssd::gated_scan_workspace(b, L, D, io == SSD_DTYPE_BF16, false);
}

ssd_status_t ssd_gated_scan_fwd(const void *x, const void *a, const float *init_state, void *y,
                                float *states, float *final_state, int b, int L, int D, int sigmoid,
                                ssd_dtype_t io, ssd_dtype_t a_io, void *workspace,
                                size_t workspace_bytes, void *hip_stream) {
    if (const ssd_status_t st = check_dims(b, L, D, io, a_io); st != SSD_OK) return st;
    if (b == 0) return SSD_OK;
    const hipStream_t stream = static_cast<hipStream_t>(hip_stream);
    const size_t n = size_t(b) * L * D, st = size_t(b) * D * 4;
    if (!aligned(init_state, 16) || !aligned(final_state, 16)) return SSD_ERR_ALIGN;
    const Range rinit(init_state, st), rfinal(final_state, st);
    if (rinit.overlaps(rfinal)) return SSD_ERR_ALIAS;
    if (L == 0) return final_state ? done(ssd::launch_copy_state(init_state, final_state, size_t(b) * D, stream)) : SSD_OK;
    if (!x || !a || !y) return SSD_ERR_NULL_ARG;
    if (!aligned(x, 16) || !aligned(a, 16) || !aligned(y, 16) || !aligned(states, 16) || !aligned(workspace, 16))
        return SSD_ERR_ALIGN;
    const size_t need = ssd::gated_scan_workspace(b, L, D, io == SSD_DTYPE_BF16, false);
    if (need && (!workspace || workspace_bytes < need)) return SSD_ERR_WORKSPACE;
    const Range ins[] = {Range(x, n * elem(io)), Range(a, n * elem(a_io)), rinit};
    const Range outs[] = {Range(y, n * elem(io)), Range(states, kept_bytes(b, L, D)), rfinal, Range(workspace, need)};
    if (any_alias(ins, outs)) return SSD_ERR_ALIAS;
    ssd::GatedScanArgs s{};
    s.looks = wait_limit.load(std::memory_order_relaxed);
    s.x = x; s.a = a; s.init_state = init_state; s.y = y; s.kept = states; s.final_state = final_state; s.workspace = workspace;
    s.b = b; s.L = L; s.D = D; s.sigmoid = sigmoid != 0; s.bf16 = io == SSD_DTYPE_BF16; s.a_bf16 = a_io == SSD_DTYPE_BF16;
    return done(ssd::launch_gated_scan_fwd(s, stream));
}

size_t ssd_gated_scan_bwd_workspace_bytes(int b, int L, int D, int with_states, ssd_dtype_t io,
                                          ssd_dtype_t a_io) {
    if (check_dims(b, L, D, io, a_io) != SSD_OK) return size_t(-1);
    return words_bytes(b, L, D, io) + (with_states ? 0 : kept_bytes(b, L, D));
}

ssd_status_t ssd_gated_scan_bwd(const void *x, const void *a, const float *init_state,
                                const float *states, const void *dy, const float *d_final, void *dx,
                                void *da, float *d_init, int b, int L, int D, int sigmoid,
                                ssd_dtype_t io, ssd_dtype_t a_io, void *workspace,
                                size_t workspace_bytes, void *hip_stream) {
    if (const ssd_status_t st = check_dims(b, L, D, io, a_io); st != SSD_OK) return st;
    if (b == 0) return SSD_OK;
    const hipStream_t stream = static_cast<hipStream_t>(hip_stream);
    const size_t n = size_t(b) * L * D, st = size_t(b) * D * 4;
    if (!aligned(d_final, 16) || !aligned(d_init, 16)) return SSD_ERR_ALIGN;
    const Range rfinal(d_final, st), rinit(d_init, st);
    if (rinit.overlaps(rfinal)) return SSD_ERR_ALIAS;
    if (L == 0) return d_init ? done(ssd::launch_copy_state(d_final, d_init, size_t(b) * D, stream)) : SSD_OK;
    if (!x || !a || !dy || !dx || !da) return SSD_ERR_NULL_ARG;
    if (!aligned(x, 16) || !aligned(a, 16) || !aligned(init_state, 16) || !aligned(states, 16) || !aligned(dy, 16) ||
        !aligned(dx, 16) || !aligned(da, 16) || !aligned(workspace, 16))
        return SSD_ERR_ALIGN;
    const size_t own = words_bytes(b, L, D, io), need = own + (states ? 0 : kept_bytes(b, L, D));
    if (need && (!workspace || workspace_bytes < need)) return SSD_ERR_WORKSPACE;
    const Range ins[] = {Range(x, n * elem(io)), Range(a, n * elem(a_io)), Range(states ? nullptr : init_state, st),
                         Range(states, kept_bytes(b, L, D)), Range(dy, n * elem(io)), rfinal};
    const Range outs[] = {Range(dx, n * elem(io)), Range(da, n * elem(a_io)), rinit, Range(workspace, need)};
    if (any_alias(ins, outs)) return SSD_ERR_ALIAS;
    ssd::GatedScanArgs s{};
    s.looks = wait_limit.load(std::memory_order_relaxed);
    s.x = x; s.a = a; s.init_state = init_state; s.workspace = workspace;
    s.b = b; s.L = L; s.D = D; s.sigmoid = sigmoid != 0; s.bf16 = io == SSD_DTYPE_BF16; s.a_bf16 = a_io == SSD_DTYPE_BF16;
    if (states) {
        s.kept = const_cast<float *>(states);       // read only
    } else {
        // the states of the forward pass once more, without its outputs
        s.kept = reinterpret_cast<float *>(static_cast<char *>(workspace) + own);
        if (const hipError_t e = ssd::launch_gated_scan_fwd(s, stream); e != hipSuccess) return SSD_ERR_HIP;
        s.keep_error = ssd::gated_scan_waits(L);
    }
    s.dy = dy; s.d_final = d_final; s.dx = dx; s.da = da; s.d_init = d_init;
    return done(ssd::launch_gated_scan_bwd(s, stream));
}

ssd_status_t ssd_gated_scan_workspace_error(const void *workspace, size_t workspace_bytes, int b, int L,
                                            int32_t *err_out, void *hip_stream) {
    if (b < 0 || L < 0) return SSD_ERR_BAD_DIM;
    if (!err_out) return SSD_ERR_NULL_ARG;
    if (!aligned(workspace, 16) || !aligned(err_out, 4)) return SSD_ERR_ALIGN;
    const bool waits = b > 0 && ssd::gated_scan_waits(L);
    if (waits && (!workspace || workspace_bytes < 16)) return SSD_ERR_WORKSPACE;
    if (Range(workspace, workspace_bytes).overlaps(Range(err_out, 4))) return SSD_ERR_ALIAS;
    return done(ssd::launch_gated_scan_error(waits ? workspace : nullptr, err_out, static_cast<hipStream_t>(hip_stream)));
}

int ssd_gated_scan_wait_limit(int looks) {
    return looks < 0 ? wait_limit.load(std::memory_order_relaxed) : wait_limit.exchange(looks, std::memory_order_relaxed);
}

}  // extern "C"
