// ssd_norm_add.h -- the residual sum and the norm of the next block, with their gradients
// (formulas at the top of ssd_norm.hip), for what is added as it is and with dropout.
//
// DROP says what becomes of x on its way to the sum: NoDrop, or the dropout of
// ssd_norm_drop.hip.  It has
//   mask<VEC>(i)      bit j says whether element i + j of the flat array stays
//   factor()          what an element that stays is multiplied by
// and is asked again by the backward pass; no mask is stored.
#pragma once

#include "ssd_norm.h"
#include "ssd_norm_team.h"

namespace ssd {
namespace {

struct NoDrop {
    static constexpr bool kOn = false;
};

// x[j], or 0 where bit j of the mask is clear, whatever x[j] holds there.
template <class DROP, int VEC>
__device__ __forceinline__ void drop_vec(const DROP &drop, uint32_t mask, float (&x)[VEC]) {
    if constexpr (DROP::kOn) {
#pragma unroll
        for (int j = 0; j < VEC; ++j) x[j] = (mask >> j & 1) ? x[j] * drop.factor() : 0.f;
    }
}

template <typename IO, typename RES, class DROP, int VEC, int TPS, int NV>
__global__ __launch_bounds__(kBlock) void k_norm_add_fwd(const IO *__restrict__ x, const RES *residual,
                                                         const float *__restrict__ scale, const float *__restrict__ w,
                                                         RES *sum, IO *__restrict__ y, int64_t rows, int D, float eps,
                                                         DROP drop) {
    __shared__ float tmp[4];
    constexpr int kTeams = kBlock / TPS;
    const int lane = threadIdx.x % TPS;
    const int64_t row = block_index() * kTeams + threadIdx.x / TPS;
    const bool live = row < rows;
    const int64_t at = (live ? row : 0) * D;
    float s[NV][VEC], xv[NV][VEC];
    uint32_t stays[NV] = {};
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * TPS + lane) * VEC;
        if (live && c < D) {
            load_vec<RES, VEC>(residual + at + c, s[i]);
            load_vec<IO, VEC>(x + at + c, xv[i]);
        }
    }
    if constexpr (DROP::kOn) {      // while the loads are under way
#pragma unroll
        for (int i = 0; i < NV; ++i) stays[i] = drop.template mask<VEC>(at + (i * TPS + lane) * VEC);
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * TPS + lane) * VEC;
        if (!(live && c < D)) continue;
        float sc[VEC];
        if (scale) load_vec<float, VEC>(scale + c, sc);
        drop_vec(drop, stays[i], xv[i]);
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
            // the norm sees the sum as it is stored: the backward pass reads that one
            s[i][j] = to_f32<RES>(from_f32<RES>(s[i][j] + (scale ? sc[j] * xv[i][j] : xv[i][j])));
            ss += s[i][j] * s[i][j];
        }
        store_vec<RES, VEC>(sum + at + c, s[i]);
    }
    const float r = 1.f / sqrtf(team_sum<TPS>(ss, tmp) / float(D) + eps);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * TPS + lane) * VEC;
        if (!(live && c < D)) continue;
        float wv[VEC];
        load_vec<float, VEC>(w + c, wv);
#pragma unroll
        for (int j = 0; j < VEC; ++j) s[i][j] = s[i][j] * r * wv[j];
        store_vec<IO, VEC>(y + at + c, s[i]);
    }
}

// TPS = 0: the team is the block, of as many waves as the row fills with one vector a lane.
template <typename IO, typename RES, class DROP, int VEC, int TPS, int NV>
__global__ __launch_bounds__(TPS ? kBlock : kWideBlock, TPS ? 1 : 4) void k_norm_add_bwd(const IO *__restrict__ x, const RES *__restrict__ sum,
                                                         const float *__restrict__ scale, const float *__restrict__ w,
                                                         const IO *__restrict__ dy, const RES *__restrict__ dsum,
                                                         IO *__restrict__ dx, RES *__restrict__ dres,
                                                         float *__restrict__ dwp, float *__restrict__ dsp, int64_t rows,
                                                         int D, int slices, float eps, DROP drop) {
    __shared__ float tmp[TPS ? 4 : kWideBlock / 64];
    const int tps = TPS ? TPS : int(blockDim.x), lane = threadIdx.x % tps;
    const int64_t team = TPS ? int64_t(blockIdx.x) * (kBlock / (TPS ? TPS : 1)) + threadIdx.x / tps : blockIdx.x;
    const bool live = team < slices;
    const int slice = live ? int(team) : 0;
    float wv[NV][VEC], dw[NV][VEC], ds[NV][VEC];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * tps + lane) * VEC;
#pragma unroll
        for (int j = 0; j < VEC; ++j) dw[i][j] = ds[i][j] = wv[i][j] = 0.f;
        if (c < D) load_vec<float, VEC>(w + c, wv[i]);
    }
    for (int64_t row0 = 0; row0 < rows; row0 += slices) {
        const int64_t row = row0 + slice;
        const bool on = live && row < rows;
        const int64_t at = (on ? row : 0) * D;
        float s[NV][VEC], d[NV][VEC], e[NV][VEC], xv[NV][VEC];
        uint32_t stays[NV] = {};
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * tps + lane) * VEC;
#pragma unroll
            for (int j = 0; j < VEC; ++j) s[i][j] = d[i][j] = e[i][j] = xv[i][j] = 0.f;
            if (on && c < D) {
                load_vec<RES, VEC>(sum + at + c, s[i]);
                load_vec<IO, VEC>(dy + at + c, d[i]);
                if (dsum) load_vec<RES, VEC>(dsum + at + c, e[i]);
                if (scale) load_vec<IO, VEC>(x + at + c, xv[i]);
            }
            if constexpr (DROP::kOn) stays[i] = drop.template mask<VEC>(at + c);
#pragma unroll
            for (int j = 0; j < VEC; ++j) ss += s[i][j] * s[i][j];
        }
        const float sq = team_sum<TPS>(ss, tmp);
        const float r = on ? 1.f / sqrtf(sq / float(D) + eps) : 0.f;    // no row: its zeros add nothing, eps = 0 too
        float dot = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                s[i][j] *= r;                       // n
                dw[i][j] += d[i][j] * s[i][j];
                d[i][j] *= wv[i][j];                // dn
                dot += d[i][j] * s[i][j];
            }
        const float mean = team_sum<TPS>(dot, tmp) / float(D);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * tps + lane) * VEC;
            if (!(on && c < D)) continue;
            float sc[VEC], ox[VEC];
            if (scale) load_vec<float, VEC>(scale + c, sc);
            drop_vec(drop, stays[i], xv[i]);
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                const float g = e[i][j] + r * (d[i][j] - s[i][j] * mean);
                ds[i][j] += g * xv[i][j];
                ox[j] = scale ? g * sc[j] : g;
                e[i][j] = g;
            }
            drop_vec(drop, stays[i], ox);
            store_vec<IO, VEC>(dx + at + c, ox);
            store_vec<RES, VEC>(dres + at + c, e[i]);
        }
    }
    if (!live) return;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * tps + lane) * VEC;
        if (c >= D) continue;
        store_vec<float, VEC>(dwp + int64_t(slice) * D + c, dw[i]);
        if (dsp) store_vec<float, VEC>(dsp + int64_t(slice) * D + c, ds[i]);
    }
}

// One block per segment of any length: the segment is read once for the sum of squares
// and once more (from the caches) for the result.
template <typename IO, typename RES, class DROP>
__global__ __launch_bounds__(kBlock) void k_norm_add_fwd_loop(const IO *__restrict__ x, const RES *residual,
                                                              const float *__restrict__ scale,
                                                              const float *__restrict__ w, RES *sum, IO *__restrict__ y,
                                                              int64_t rows, int D, float eps, DROP drop) {
    __shared__ float tmp[4];
    if (block_index() >= rows) return;
    const int64_t at = block_index() * D;
    float ss = 0.f;
    for (int c = threadIdx.x; c < D; c += kBlock) {
        float xv[1] = {to_f32<IO>(x[at + c])};
        if constexpr (DROP::kOn) drop_vec(drop, drop.template mask<1>(at + c), xv);
        const RES held = from_f32<RES>(to_f32<RES>(residual[at + c]) + (scale ? scale[c] * xv[0] : xv[0]));
        sum[at + c] = held;     // read back below by the same thread
        const float s = to_f32<RES>(held);
        ss += s * s;
    }
    const float r = 1.f / sqrtf(team_sum<256>(ss, tmp) / float(D) + eps);
    for (int c = threadIdx.x; c < D; c += kBlock) y[at + c] = from_f32<IO>(to_f32<RES>(sum[at + c]) * r * w[c]);
}

template <typename IO, typename RES, class DROP>
__global__ __launch_bounds__(kBlock) void k_norm_add_bwd_loop(const IO *__restrict__ x, const RES *__restrict__ sum,
                                                              const float *__restrict__ scale,
                                                              const float *__restrict__ w, const IO *__restrict__ dy,
                                                              const RES *__restrict__ dsum, IO *__restrict__ dx,
                                                              RES *__restrict__ dres, float *__restrict__ dwp,
                                                              float *__restrict__ dsp, int64_t rows, int D, int slices,
                                                              float eps, DROP drop) {
    __shared__ float tmp[4];
    const int slice = blockIdx.x;
    float *dw = dwp + int64_t(slice) * D, *ds = dsp ? dsp + int64_t(slice) * D : nullptr;
    for (int c = threadIdx.x; c < D; c += kBlock) {
        dw[c] = 0.f;
        if (ds) ds[c] = 0.f;
    }
    for (int64_t row = slice; row < rows; row += slices) {
        const int64_t at = row * D;
        float ss = 0.f;
        for (int c = threadIdx.x; c < D; c += kBlock) {
            const float s = to_f32<RES>(sum[at + c]);
            ss += s * s;
        }
        const float r = 1.f / sqrtf(team_sum<256>(ss, tmp) / float(D) + eps);
        float dot = 0.f;
        for (int c = threadIdx.x; c < D; c += kBlock) {
            const float n = to_f32<RES>(sum[at + c]) * r, d = to_f32<IO>(dy[at + c]);
            dw[c] += d * n;
            dot += d * w[c] * n;
        }
        const float mean = team_sum<256>(dot, tmp) / float(D);
        for (int c = threadIdx.x; c < D; c += kBlock) {
            const float n = to_f32<RES>(sum[at + c]) * r, d = to_f32<IO>(dy[at + c]);
            const float g = (dsum ? to_f32<RES>(dsum[at + c]) : 0.f) + r * (d * w[c] - n * mean);
            float ox[1] = {scale ? g * scale[c] : g}, xv[1] = {ds ? to_f32<IO>(x[at + c]) : 0.f};
            if constexpr (DROP::kOn) {
                const uint32_t stays = drop.template mask<1>(at + c);
                drop_vec(drop, stays, ox);
                drop_vec(drop, stays, xv);
            }
            if (ds) ds[c] += g * xv[0];
            dx[at + c] = from_f32<IO>(ox[0]);
            dres[at + c] = from_f32<RES>(g);
        }
    }
}

template <typename IO, typename RES, class DROP>
hipError_t add_fwd(const NormAddArgs &a, const DROP &drop, hipStream_t stream) {
    const auto *x = static_cast<const IO *>(a.x);
    const auto *res = static_cast<const RES *>(a.residual);
    auto *sum = static_cast<RES *>(a.sum);
    auto *y = static_cast<IO *>(a.y);
    const Team t = pick_team(a.D, a.bf16);
    if (!t.nv) {
        hipLaunchKernelGGL((k_norm_add_fwd_loop<IO, RES, DROP>), grid_of(a.rows, 1), dim3(kBlock), 0, stream, x, res, a.scale, a.w, sum, y, a.rows, a.D, a.eps, drop);
        return hipGetLastError();
    }
    return with_team<IO>(t, [&](auto v, auto tps, auto nv) {
        hipLaunchKernelGGL((k_norm_add_fwd<IO, RES, DROP, v(), tps(), nv()>), grid_of(a.rows, kBlock / tps()), dim3(kBlock), 0, stream,
                           x, res, a.scale, a.w, sum, y, a.rows, a.D, a.eps, drop);
        return hipGetLastError();
    });
}

template <typename IO, typename RES, class DROP>
hipError_t add_bwd(const NormAddArgs &a, const NormBwdPlan &plan, const DROP &drop, hipStream_t stream) {
    const auto *x = static_cast<const IO *>(a.x), *dy = static_cast<const IO *>(a.dy);
    const auto *sum = static_cast<const RES *>(a.sum), *dsum = static_cast<const RES *>(a.dsum);
    auto *dx = static_cast<IO *>(a.dx);
    auto *dres = static_cast<RES *>(a.dres);
    auto *part = static_cast<float *>(a.workspace);
    float *dsp = a.scale ? part + size_t(plan.slices) * a.D : nullptr;
    const Team t = pick_team(a.D, a.bf16);
    if constexpr (DROP::kOn && std::is_same_v<IO, bf16_bits>) {
        // Rows of 257 to 512 vectors leave most of a 256-lane team idle at its second vectors, and
        // the others wait: 8192 rows of 2560 channels 92 us, one vector a lane 83, 3584 111 and 104.
        // Longer rows make blocks of which a CU holds one: 4096 rows of 5120 86 and 93 us.
        // (fp32 I/O, with half the channels a vector: 22 and 23 us of 2677 rows of 1288.)
        if (t.vec == 8 && a.D / 8 > kBlock && a.D / 8 <= kWideBlock) {
            hipLaunchKernelGGL((k_norm_add_bwd<IO, RES, DROP, 8, 0, 1>), dim3(plan.slices), dim3((a.D / 8 + 63) / 64 * 64), 0, stream,
                               x, sum, a.scale, a.w, dy, dsum, dx, dres, part, dsp, a.rows, a.D, plan.slices, a.eps, drop);
            return hipGetLastError();
        }
    }
    if (!t.nv) {
        hipLaunchKernelGGL((k_norm_add_bwd_loop<IO, RES, DROP>), dim3(plan.slices), dim3(kBlock), 0, stream, x, sum, a.scale, a.w, dy, dsum, dx, dres,
                           part, dsp, a.rows, a.D, plan.slices, a.eps, drop);
        return hipGetLastError();
    }
    return with_team<IO>(t, [&](auto v, auto tps, auto nv) {
        hipLaunchKernelGGL((k_norm_add_bwd<IO, RES, DROP, v(), tps(), nv()>), dim3(blocks_of(plan.slices, kBlock / tps())), dim3(kBlock), 0, stream,
                           x, sum, a.scale, a.w, dy, dsum, dx, dres, part, dsp, a.rows, a.D, plan.slices, a.eps, drop);
        return hipGetLastError();
    });
}

// By the types of x and of the residual.
template <class DROP>
hipError_t add_fwd_by_type(const NormAddArgs &a, const DROP &drop, hipStream_t stream) {
    if (!a.bf16) return add_fwd<float, float>(a, drop, stream);
    return a.res_bf16 ? add_fwd<bf16_bits, bf16_bits>(a, drop, stream) : add_fwd<bf16_bits, float>(a, drop, stream);
}

template <class DROP>
hipError_t add_bwd_by_type(const NormAddArgs &a, const NormBwdPlan &plan, const DROP &drop, hipStream_t stream) {
    NormBwdPlan p = plan;
    if constexpr (DROP::kOn) {
        // two blocks for every CU, which holds two: half the partial sums of 1024 blocks, and no
        // second round (8192 rows of 2560 channels 97 -> 92 us, of 1024 52 -> 39).  Nothing in this
        // rule or in the teams above needs dropout: without it both would spare as much (8192 rows
        // of 2560 channels 94 -> 77 us, of 1024 32 -> 24, 4096 of 5120 90 -> 83), but add the
        // parameters' gradients up in another order than norm_add_bwd's callers have had so far.
        const Team t = pick_team(a.D, a.bf16);
        p.slices = std::min(p.slices, 512 * (t.nv ? kBlock / t.tps : 1));
    }
    hipError_t e;
    if (!a.bf16) e = add_bwd<float, float>(a, p, drop, stream);
    else e = a.res_bf16 ? add_bwd<bf16_bits, bf16_bits>(a, p, drop, stream) : add_bwd<bf16_bits, float>(a, p, drop, stream);
    if (e != hipSuccess) return e;
    return launch_norm_reduce(static_cast<const float *>(a.workspace), a.dw, a.dscale, p.slices, a.D, stream);
}

}  // namespace
}  // namespace ssd
