// ssd_norm_api.hip -- host-side checks and dispatch of the norm entry points.
#include <limits.h>

#include "ssd_checks.h"
#include "ssd_kernels.h"
#include "ssd_mi355x.h"
#include "ssd_norm.h"

namespace {

using ssd::aligned;
using ssd::any_alias;
using ssd::Range;

bool known(ssd_dtype_t io) { return io == SSD_DTYPE_F32 || io == SSD_DTYPE_BF16; }

size_t elem(ssd_dtype_t io) { return io == SSD_DTYPE_BF16 ? 2 : 4; }

ssd_status_t check_dims(int rows, int D, int group) {
    if (rows < 0 || D <= 0 || group <= 0) return SSD_ERR_BAD_DIM;
    if (D % group != 0) return SSD_ERR_GROUPS;
    // the kernels count channels in 31 bits, up to a block past the last one
    if (D > INT_MAX - 256) return SSD_ERR_UNSUPPORTED;
    // segments counted in 31 bits (a launch's two dimensions hold as many blocks), groups of a row in 16
    if (int64_t(rows) * (D / group) > INT_MAX || D / group > 65535) return SSD_ERR_UNSUPPORTED;
    return SSD_OK;
}

ssd_status_t done(hipError_t e) { return e == hipSuccess ? SSD_OK : SSD_ERR_HIP; }

}  // namespace

extern "C" {

ssd_status_t ssd_norm_gate_fwd(const void *x, const void *z, const float *w, void *y, int rows,
                               int D, int group, float eps, int gate_first, ssd_dtype_t io,
                               void *hip_stream) {
    if (!known(io)) return SSD_ERR_UNSUPPORTED;
    if (const ssd_status_t st = check_dims(rows, D, group); st != SSD_OK) return st;
    if (rows == 0) return SSD_OK;
    if (!x || !w || !y) return SSD_ERR_NULL_ARG;
    if (!aligned(x, 16) || !aligned(z, 16) || !aligned(w, 16) || !aligned(y, 16)) return SSD_ERR_ALIGN;
    const size_t n = size_t(rows) * D * elem(io);
    const Range ins[] = {Range(x, n), Range(z, n), Range(w, size_t(D) * 4)};
    const Range outs[] = {Range(y, n)};
    if (any_alias(ins, outs)) return SSD_ERR_ALIAS;
    ssd::NormGateArgs a{};
    a.x = x; a.z = z; a.w = w; a.y = y;
    a.rows = rows; a.D = D; a.group = group; a.eps = eps;
    a.gate_first = gate_first != 0; a.bf16 = io == SSD_DTYPE_BF16;
    return done(ssd::launch_norm_gate_fwd(a, static_cast<hipStream_t>(hip_stream)));
}

size_t ssd_norm_bwd_workspace_bytes(int rows, int D, int group, int params, ssd_dtype_t io) {
    if (!known(io) || check_dims(rows, D, group) != SSD_OK || params < 1 || params > 2) return size_t(-1);
    return ssd::plan_norm_bwd(rows, D, group, params, io == SSD_DTYPE_BF16).total;
}

ssd_status_t ssd_norm_gate_bwd(const void *x, const void *z, const float *w, const void *dy,
                               void *dx, void *dz, float *dw, int rows, int D, int group,
                               float eps, int gate_first, ssd_dtype_t io, void *workspace,
                               size_t workspace_bytes, void *hip_stream) {
    if (!known(io)) return SSD_ERR_UNSUPPORTED;
    if (const ssd_status_t st = check_dims(rows, D, group); st != SSD_OK) return st;
    if (!dw) return SSD_ERR_NULL_ARG;
    if (!aligned(dw, 16)) return SSD_ERR_ALIGN;
    const hipStream_t stream = static_cast<hipStream_t>(hip_stream);
    if (rows == 0) return done(ssd::launch_copy_state(nullptr, dw, size_t(D), stream));
    if (!x || !w || !dy || !dx || (z == nullptr) != (dz == nullptr)) return SSD_ERR_NULL_ARG;
    if (!aligned(x, 16) || !aligned(z, 16) || !aligned(w, 16) || !aligned(dy, 16) || !aligned(dx, 16) ||
        !aligned(dz, 16) || !aligned(workspace, 16))
        return SSD_ERR_ALIGN;
    const ssd::NormBwdPlan plan = ssd::plan_norm_bwd(rows, D, group, 1, io == SSD_DTYPE_BF16);
    if (!workspace || workspace_bytes < plan.total) return SSD_ERR_WORKSPACE;
    const size_t n = size_t(rows) * D * elem(io);
    const Range ins[] = {Range(x, n), Range(z, n), Range(w, size_t(D) * 4), Range(dy, n)};
    const Range outs[] = {Range(dx, n), Range(dz, n), Range(dw, size_t(D) * 4), Range(workspace, plan.total)};
    if (any_alias(ins, outs)) return SSD_ERR_ALIAS;
    ssd::NormGateArgs a{};
    a.x = x; a.z = z; a.w = w; a.dy = dy; a.dx = dx; a.dz = dz; a.dw = dw; a.workspace = workspace;
    a.rows = rows; a.D = D; a.group = group; a.eps = eps;
    a.gate_first = gate_first != 0; a.bf16 = io == SSD_DTYPE_BF16;
    return done(ssd::launch_norm_gate_bwd(a, plan, stream));
}

ssd_status_t ssd_norm_add_fwd(const void *x, const void *residual, const float *scale,
                              const float *w, void *sum, void *y, int rows, int D, float eps,
                              ssd_dtype_t io, ssd_dtype_t res_io, void *hip_stream) {
    if (!known(io) || !known(res_io)) return SSD_ERR_UNSUPPORTED;
    if (res_io != SSD_DTYPE_F32 && res_io != io) return SSD_ERR_UNSUPPORTED;
    if (const ssd_status_t st = check_dims(rows, D, D); st != SSD_OK) return st;
    if (rows == 0) return SSD_OK;
    if (!x || !residual || !w || !sum || !y) return SSD_ERR_NULL_ARG;
    if (!aligned(x, 16) || !aligned(residual, 16) || !aligned(scale, 16) || !aligned(w, 16) || !aligned(sum, 16) ||
        !aligned(y, 16))
        return SSD_ERR_ALIGN;
    const size_t n = size_t(rows) * D * elem(io), m = size_t(rows) * D * elem(res_io);
    const Range rres(residual, m), rsum(sum, m);
    if (rres.overlaps(rsum) && !rres.same(rsum)) return SSD_ERR_ALIAS;
    const Range ins[] = {Range(x, n), Range(scale, size_t(D) * 4), Range(w, size_t(D) * 4)};
    const Range outs[] = {rsum, Range(y, n)};
    if (any_alias(ins, outs) || outs[1].overlaps(rres)) return SSD_ERR_ALIAS;
    ssd::NormAddArgs a{};
    a.x = x; a.residual = residual; a.scale = scale; a.w = w; a.sum = sum; a.y = y;
    a.rows = rows; a.D = D; a.eps = eps;
    a.bf16 = io == SSD_DTYPE_BF16; a.res_bf16 = res_io == SSD_DTYPE_BF16;
    return done(ssd::launch_norm_add_fwd(a, static_cast<hipStream_t>(hip_stream)));
}

ssd_status_t ssd_norm_add_bwd(const void *x, const void *sum, const float *scale, const float *w,
                              const void *dy, const void *d_sum, void *dx, void *d_residual,
                              float *d_scale, float *dw, int rows, int D, float eps,
                              ssd_dtype_t io, ssd_dtype_t res_io, void *workspace,
                              size_t workspace_bytes, void *hip_stream) {
    if (!known(io) || !known(res_io)) return SSD_ERR_UNSUPPORTED;
    if (res_io != SSD_DTYPE_F32 && res_io != io) return SSD_ERR_UNSUPPORTED;
    if (const ssd_status_t st = check_dims(rows, D, D); st != SSD_OK) return st;
    if (!dw || (scale == nullptr) != (d_scale == nullptr)) return SSD_ERR_NULL_ARG;
    if (!aligned(dw, 16) || !aligned(d_scale, 16)) return SSD_ERR_ALIGN;
    const hipStream_t stream = static_cast<hipStream_t>(hip_stream);
    const Range rdw(dw, size_t(D) * 4), rds(d_scale, size_t(D) * 4);
    if (rdw.overlaps(rds)) return SSD_ERR_ALIAS;
    if (rows == 0) {
        if (ssd::launch_copy_state(nullptr, dw, size_t(D), stream) != hipSuccess) return SSD_ERR_HIP;
        return d_scale ? done(ssd::launch_copy_state(nullptr, d_scale, size_t(D), stream)) : SSD_OK;
    }
    if (!sum || !w || !dy || !dx || !d_residual || (scale && !x)) return SSD_ERR_NULL_ARG;
    if (!aligned(x, 16) || !aligned(sum, 16) || !aligned(scale, 16) || !aligned(w, 16) || !aligned(dy, 16) ||
        !aligned(d_sum, 16) || !aligned(dx, 16) || !aligned(d_residual, 16) || !aligned(workspace, 16))
        return SSD_ERR_ALIGN;
    const ssd::NormBwdPlan plan = ssd::plan_norm_bwd(rows, D, D, scale ? 2 : 1, io == SSD_DTYPE_BF16);
    if (!workspace || workspace_bytes < plan.total) return SSD_ERR_WORKSPACE;
    const size_t n = size_t(rows) * D * elem(io), m = size_t(rows) * D * elem(res_io);
    const Range ins[] = {Range(scale ? x : nullptr, n), Range(sum, m), Range(scale, size_t(D) * 4),
                         Range(w, size_t(D) * 4), Range(dy, n), Range(d_sum, m)};
    const Range outs[] = {Range(dx, n), Range(d_residual, m), rds, rdw, Range(workspace, plan.total)};
    if (any_alias(ins, outs)) return SSD_ERR_ALIAS;
    ssd::NormAddArgs a{};
    a.x = x; a.sum = const_cast<void *>(sum); a.scale = scale; a.w = w; a.dy = dy; a.dsum = d_sum;
    a.dx = dx; a.dres = d_residual; a.dscale = d_scale; a.dw = dw; a.workspace = workspace;
    a.rows = rows; a.D = D; a.eps = eps;
    a.bf16 = io == SSD_DTYPE_BF16; a.res_bf16 = res_io == SSD_DTYPE_BF16;
    return done(ssd::launch_norm_add_bwd(a, plan, stream));
}

}  // extern "C"
