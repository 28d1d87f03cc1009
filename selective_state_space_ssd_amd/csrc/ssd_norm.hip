// ssd_norm.hip -- the norms around a mixer block, each fused with what stands next to it.
//
// After the mixer, with its gate (act(z) = z / (1 + e^-z), one norm per group of
// channels, r = (mean u^2 + eps)^-1/2):
//   norm first:  u = x,         y = u r w act(z)
//   gate first:  u = x act(z),  y = u r w
// Before the next block, with the residual sum (scale per channel, or 1):
//   s = residual + scale x,     y = s r w,  r = (mean s^2 + eps)^-1/2
//
// Gradients, with n = u r, dn the gradient of n: du = r (dn - n mean(dn n)); the sums
// over rows (dw, dscale) are kept per thread in fp32, written once per row slice and
// added by a second kernel in a fixed order, so results do not change from run to run.
//
// All of it streams: every array is read or written once and the row is held in
// registers between the sum of squares and its use.  A team of TPS lanes holds one
// segment, NV vectors of VEC channels a lane (VEC elements = 16 bytes); teams of 16
// lanes serve the short groups of a per-head norm, one wave or one block the whole rows
// of a layer.  Segments whose length does not divide into vectors take VEC = 1 teams (all
// arrays are 16-byte aligned), and those that no team of their kind holds the loop kernels,
// which read the segment twice.
//
// Bound by the bytes: gate backward of 8192 x 4096, groups of 128, bf16 (336 MB) 70 us, 4.8
// TB/s; residual sum and norm of 8192 x 2560, bf16 with an fp32 residual (252 MB) 51 us, 4.9
// TB/s; its backward of 2677 x 1288 fp32 (83 MB) 17 us, and 5 for the sums of its
// parameters' gradients, 3.9 TB/s together; a copy reaches 5.2.  A forward call of 5 rows is
// its launch: 4.5 us of kernel in 9.
#include <algorithm>

#include "ssd_norm.h"
#include "ssd_norm_add.h"
#include "ssd_norm_team.h"

namespace ssd {
namespace {

constexpr int kBwdBlocks = 1024;    // blocks of a backward pass, at the most

// act(z) = z sigmoid(z).  e^-z overflows to inf for z below -88, where the gate is -0.
// With bf16 I/O the exponential is the hardware's of z log2(e) and the quotient its
// reciprocal (relative errors of a few 2^-24 (1 + |z|), against 2^-9 of the rounding to
// come).  That, one evaluation per element instead of three, and the order of gate and norm
// as a template argument took the backward pass of 8192 x 4096 from 114 to 70 us (336 MB).
template <typename IO>
__device__ __forceinline__ float sigmoid(float z) {
    if constexpr (std::is_same_v<IO, float>) return 1.f / (1.f + expf(-z));
    else return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-z * kLog2e));
}

// ------------------------------------------------------------------- after the mixer
template <typename IO, int VEC, int TPS, int NV>
__global__ __launch_bounds__(kBlock) void k_norm_gate_fwd(const IO *__restrict__ x, const IO *__restrict__ z,
                                                          const float *__restrict__ w, IO *__restrict__ y,
                                                          int64_t segments, int D, int group, float eps,
                                                          bool gate_first) {
    __shared__ float tmp[4];
    constexpr int kTeams = kBlock / TPS;
    const int lane = threadIdx.x % TPS;
    const int64_t seg = block_index() * kTeams + threadIdx.x / TPS;
    const bool live = seg < segments;           // the same for a whole team
    const int64_t at = (live ? seg : 0) * group;
    const int col = int(at % D);                // channel of the segment's first element
    float u[NV][VEC], g[NV][VEC];
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * TPS + lane) * VEC;
        if (live && c < group) {
            load_vec<IO, VEC>(x + at + c, u[i]);
            if (z) load_vec<IO, VEC>(z + at + c, g[i]);
        }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * TPS + lane) * VEC;
        if (!(live && c < group)) continue;
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
            const float act = z ? g[i][j] * sigmoid<IO>(g[i][j]) : 1.f;
            if (gate_first) u[i][j] *= act;
            g[i][j] = gate_first ? 1.f : act;
            ss += u[i][j] * u[i][j];
        }
    }
    const float r = 1.f / sqrtf(team_sum<TPS>(ss, tmp) / float(group) + eps);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * TPS + lane) * VEC;
        if (!(live && c < group)) continue;
        float wv[VEC];
        load_vec<float, VEC>(w + col + c, wv);
#pragma unroll
        for (int j = 0; j < VEC; ++j) u[i][j] = u[i][j] * r * wv[j] * g[i][j];
        store_vec<IO, VEC>(y + at + c, u[i]);
    }
}

// One team keeps one group of channels and walks the rows of its slice; its sums for dw
// stay in registers until the end.
template <typename IO, bool FIRST, int VEC, int TPS, int NV>
__global__ __launch_bounds__(kBlock) void k_norm_gate_bwd(const IO *__restrict__ x, const IO *__restrict__ z,
                                                          const float *__restrict__ w, const IO *__restrict__ dy,
                                                          IO *__restrict__ dx, IO *__restrict__ dz,
                                                          float *__restrict__ dwp, int64_t rows, int D, int group,
                                                          int slices, float eps) {
    __shared__ float tmp[4];
    constexpr int kTeams = kBlock / TPS;
    const int lane = threadIdx.x % TPS;
    const int ngroups = D / group;
    const int64_t team = int64_t(blockIdx.x) * kTeams + threadIdx.x / TPS;
    const bool live = team < int64_t(ngroups) * slices;
    const int gi = live ? int(team % ngroups) : 0;
    const int slice = live ? int(team / ngroups) : 0;
    const int col = gi * group;
    float wv[NV][VEC], dw[NV][VEC];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * TPS + lane) * VEC;
#pragma unroll
        for (int j = 0; j < VEC; ++j) dw[i][j] = wv[i][j] = 0.f;
        if (c < group) load_vec<float, VEC>(w + col + c, wv[i]);
    }
    // every team of a block takes the same number of turns (the block-wide sums hold
    // barriers): rows past the end are computed from zeros and not stored
    for (int64_t row0 = 0; row0 < rows; row0 += slices) {
        const int64_t row = row0 + slice;
        const bool on = live && row < rows;
        const int64_t at = (on ? row : 0) * D + col;
        float u[NV][VEC], g[NV][VEC], d[NV][VEC];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * TPS + lane) * VEC;
#pragma unroll
            for (int j = 0; j < VEC; ++j) u[i][j] = g[i][j] = d[i][j] = 0.f;
            if (on && c < group) {
                load_vec<IO, VEC>(x + at + c, u[i]);
                if (z) load_vec<IO, VEC>(z + at + c, g[i]);
                load_vec<IO, VEC>(dy + at + c, d[i]);
            }
        }
        float act[NV][VEC], ss = 0.f;       // the gate; g becomes its slope
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                const float sg = sigmoid<IO>(g[i][j]);
                act[i][j] = z ? g[i][j] * sg : 1.f;
                g[i][j] = sg + act[i][j] * (1.f - sg);
                const float v = FIRST ? u[i][j] * act[i][j] : u[i][j];
                ss += v * v;
            }
        const float sq = team_sum<TPS>(ss, tmp);
        const float r = on ? 1.f / sqrtf(sq / float(group) + eps) : 0.f;    // no row: its zeros add nothing, eps = 0 too
        float dot = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                const float n = (FIRST ? u[i][j] * act[i][j] : u[i][j]) * r;
                const float up = FIRST ? d[i][j] : d[i][j] * act[i][j];     // gradient of n w
                dw[i][j] += up * n;
                dot += up * wv[i][j] * n;
            }
        const float mean = team_sum<TPS>(dot, tmp) / float(group);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * TPS + lane) * VEC;
            if (!(on && c < group)) continue;
            float ox[VEC], oz[VEC];
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                const float n = (FIRST ? u[i][j] * act[i][j] : u[i][j]) * r;
                const float du = r * ((FIRST ? d[i][j] : d[i][j] * act[i][j]) * wv[i][j] - n * mean);
                ox[j] = FIRST ? du * act[i][j] : du;
                oz[j] = (FIRST ? du * u[i][j] : d[i][j] * n * wv[i][j]) * g[i][j];
            }
            store_vec<IO, VEC>(dx + at + c, ox);
            if (z) store_vec<IO, VEC>(dz + at + c, oz);
        }
    }
    if (!live) return;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * TPS + lane) * VEC;
        if (c < group) store_vec<float, VEC>(dwp + int64_t(slice) * D + col + c, dw[i]);
    }
}

// ------------------------------------------------------------------ loop kernels
// One block per segment of any length: the segment is read once for the sum of squares
// and once more (from the caches) for the result.
template <typename IO>
__global__ __launch_bounds__(kBlock) void k_norm_gate_fwd_loop(const IO *__restrict__ x, const IO *__restrict__ z,
                                                               const float *__restrict__ w, IO *__restrict__ y,
                                                               int64_t segments, int D, int group, float eps,
                                                               bool gate_first) {
    __shared__ float tmp[4];
    if (block_index() >= segments) return;
    const int64_t at = block_index() * group;
    const int col = int(at % D);
    float ss = 0.f;
    for (int c = threadIdx.x; c < group; c += kBlock) {
        float u = to_f32<IO>(x[at + c]);
        if (z && gate_first) {
            const float zz = to_f32<IO>(z[at + c]);
            u *= zz * sigmoid<IO>(zz);
        }
        ss += u * u;
    }
    const float r = 1.f / sqrtf(team_sum<256>(ss, tmp) / float(group) + eps);
    for (int c = threadIdx.x; c < group; c += kBlock) {
        const float zz = z ? to_f32<IO>(z[at + c]) : 0.f;
        const float act = z ? zz * sigmoid<IO>(zz) : 1.f;
        y[at + c] = from_f32<IO>(to_f32<IO>(x[at + c]) * act * r * w[col + c]);
    }
}

// Blocks x = group, y = row slice.  The block's sums for dw are added up in its own row
// of the partials, channel by channel by the thread that owns the channel.
template <typename IO>
__global__ __launch_bounds__(kBlock) void k_norm_gate_bwd_loop(const IO *__restrict__ x, const IO *__restrict__ z,
                                                               const float *__restrict__ w, const IO *__restrict__ dy,
                                                               IO *__restrict__ dx, IO *__restrict__ dz,
                                                               float *__restrict__ dwp, int64_t rows, int D, int group,
                                                               int slices, float eps, bool gate_first) {
    __shared__ float tmp[4];
    const int col = int(blockIdx.x) * group, slice = blockIdx.y;
    float *dw = dwp + int64_t(slice) * D + col;
    for (int c = threadIdx.x; c < group; c += kBlock) dw[c] = 0.f;
    for (int64_t row = slice; row < rows; row += slices) {
        const int64_t at = row * D + col;
        float ss = 0.f;
        for (int c = threadIdx.x; c < group; c += kBlock) {
            float u = to_f32<IO>(x[at + c]);
            if (z && gate_first) {
                const float zz = to_f32<IO>(z[at + c]);
                u *= zz * sigmoid<IO>(zz);
            }
            ss += u * u;
        }
        const float r = 1.f / sqrtf(team_sum<256>(ss, tmp) / float(group) + eps);
        float dot = 0.f;
        for (int c = threadIdx.x; c < group; c += kBlock) {
            const float zz = z ? to_f32<IO>(z[at + c]) : 0.f, act = z ? zz * sigmoid<IO>(zz) : 1.f;
            const float d = to_f32<IO>(dy[at + c]), u = to_f32<IO>(x[at + c]);
            const float n = u * (gate_first ? act : 1.f) * r, up = gate_first ? d : d * act;
            dw[c] += up * n;
            dot += up * w[col + c] * n;
        }
        const float mean = team_sum<256>(dot, tmp) / float(group);
        for (int c = threadIdx.x; c < group; c += kBlock) {
            const float zz = z ? to_f32<IO>(z[at + c]) : 0.f, sg = z ? sigmoid<IO>(zz) : 1.f;
            const float act = z ? zz * sg : 1.f, slope = sg * (1.f + zz * (1.f - sg));
            const float d = to_f32<IO>(dy[at + c]), u = to_f32<IO>(x[at + c]), wc = w[col + c];
            const float n = u * (gate_first ? act : 1.f) * r;
            const float du = r * ((gate_first ? d : d * act) * wc - n * mean);
            dx[at + c] = from_f32<IO>(gate_first ? du * act : du);
            if (z) dz[at + c] = from_f32<IO>((gate_first ? du * u : d * n * wc) * slope);
        }
    }
}

// out[p][c] = the sum over slices of part[p][slice][c] in a fixed order: 64 channels per
// block, 16 waves with every 16th slice each, 8 loads in flight.
constexpr int kReduceWaves = 16;
__global__ __launch_bounds__(64 * kReduceWaves) void k_norm_reduce(const float *__restrict__ part, float *out0, float *out1,
                                                                   int slices, int D) {
    __shared__ float tmp[kReduceWaves][64];
    const int lane = threadIdx.x & 63, c = blockIdx.x * 64 + lane, wv = threadIdx.x >> 6;
    const float *p = part + size_t(blockIdx.y) * slices * D + min(c, D - 1);
    float s[8] = {};
    int i = wv;
    for (; i + 7 * kReduceWaves < slices; i += 8 * kReduceWaves)
#pragma unroll
        for (int j = 0; j < 8; ++j) s[j] += p[size_t(i + j * kReduceWaves) * D];
    for (; i < slices; i += kReduceWaves) s[0] += p[size_t(i) * D];
    tmp[wv][lane] = ((s[0] + s[1]) + (s[2] + s[3])) + ((s[4] + s[5]) + (s[6] + s[7]));
    __syncthreads();
    if (wv == 0 && c < D) {
        float t = 0.f;
#pragma unroll
        for (int j = 0; j < kReduceWaves; ++j) t += tmp[j][lane];
        (blockIdx.y ? out1 : out0)[c] = t;
    }
}

// ------------------------------------------------------------------------ launches
template <typename IO>
hipError_t gate_fwd(const NormGateArgs &a, hipStream_t stream) {
    const auto *x = static_cast<const IO *>(a.x), *z = static_cast<const IO *>(a.z);
    auto *y = static_cast<IO *>(a.y);
    const int64_t segments = a.rows * (a.D / a.group);
    const Team t = pick_team(a.group, a.bf16);
    if (!t.nv) {
        hipLaunchKernelGGL((k_norm_gate_fwd_loop<IO>), grid_of(segments, 1), dim3(kBlock), 0, stream, x, z, a.w, y, segments, a.D, a.group, a.eps, a.gate_first);
        return hipGetLastError();
    }
    return with_team<IO>(t, [&](auto v, auto tps, auto nv) {
        hipLaunchKernelGGL((k_norm_gate_fwd<IO, v(), tps(), nv()>), grid_of(segments, kBlock / tps()), dim3(kBlock), 0, stream,
                           x, z, a.w, y, segments, a.D, a.group, a.eps, a.gate_first);
        return hipGetLastError();
    });
}

template <typename IO>
hipError_t gate_bwd(const NormGateArgs &a, const NormBwdPlan &plan, hipStream_t stream) {
    const auto *x = static_cast<const IO *>(a.x), *z = static_cast<const IO *>(a.z), *dy = static_cast<const IO *>(a.dy);
    auto *dx = static_cast<IO *>(a.dx), *dz = static_cast<IO *>(a.dz);
    auto *part = static_cast<float *>(a.workspace);
    const int ngroups = a.D / a.group;
    const Team t = pick_team(a.group, a.bf16);
    if (!t.nv) {
        hipLaunchKernelGGL((k_norm_gate_bwd_loop<IO>), dim3(ngroups, plan.slices), dim3(kBlock), 0, stream, x, z, a.w, dy, dx, dz, part,
                           a.rows, a.D, a.group, plan.slices, a.eps, a.gate_first);
        return hipGetLastError();
    }
    return with_team<IO>(t, [&](auto v, auto tps, auto nv) {
        const dim3 grid(blocks_of(int64_t(ngroups) * plan.slices, kBlock / tps()));
        if (a.gate_first)
            hipLaunchKernelGGL((k_norm_gate_bwd<IO, true, v(), tps(), nv()>), grid, dim3(kBlock), 0, stream, x, z, a.w, dy, dx, dz, part,
                               a.rows, a.D, a.group, plan.slices, a.eps);
        else
            hipLaunchKernelGGL((k_norm_gate_bwd<IO, false, v(), tps(), nv()>), grid, dim3(kBlock), 0, stream, x, z, a.w, dy, dx, dz, part,
                               a.rows, a.D, a.group, plan.slices, a.eps);
        return hipGetLastError();
    });
}

}  // namespace

hipError_t launch_norm_reduce(const float *part, float *out0, float *out1, int slices, int D, hipStream_t stream) {
    hipLaunchKernelGGL(k_norm_reduce, dim3((D + 63) / 64, out1 ? 2 : 1), dim3(64 * kReduceWaves), 0, stream, part, out0, out1, slices, D);
    return hipGetLastError();
}

NormBwdPlan plan_norm_bwd(int64_t rows, int D, int group, int params, bool bf16) {
    NormBwdPlan p;
    if (rows <= 0) return p;
    const Team t = pick_team(group, bf16);
    const int ngroups = D / group, teams = t.nv ? kBlock / t.tps : 1;
    // enough blocks for the loads in flight, few enough for the partials to add up
    const int64_t want = (int64_t(kBwdBlocks) * teams + ngroups - 1) / ngroups;
    p.slices = int(std::max<int64_t>(1, std::min<int64_t>(std::min<int64_t>(rows, 32768), want)));
    p.total = size_t(params) * p.slices * D * sizeof(float);
    return p;
}

hipError_t launch_norm_gate_fwd(const NormGateArgs &a, hipStream_t stream) {
    return a.bf16 ? gate_fwd<bf16_bits>(a, stream) : gate_fwd<float>(a, stream);
}

hipError_t launch_norm_gate_bwd(const NormGateArgs &a, const NormBwdPlan &plan, hipStream_t stream) {
    const hipError_t e = a.bf16 ? gate_bwd<bf16_bits>(a, plan, stream) : gate_bwd<float>(a, plan, stream);
    if (e != hipSuccess) return e;
    return launch_norm_reduce(static_cast<const float *>(a.workspace), a.dw, nullptr, plan.slices, a.D, stream);
}

hipError_t launch_norm_add_fwd(const NormAddArgs &a, hipStream_t stream) { return add_fwd_by_type(a, NoDrop{}, stream); }

hipError_t launch_norm_add_bwd(const NormAddArgs &a, const NormBwdPlan &plan, hipStream_t stream) {
    return add_bwd_by_type(a, plan, NoDrop{}, stream);
}

}  // namespace ssd
