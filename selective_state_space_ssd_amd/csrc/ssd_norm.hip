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

#include "ssd_device.h"
#include "ssd_norm.h"

namespace ssd {
namespace {

constexpr int kBlock = 256;

// Blocks of a forward pass: one dimension of a launch holds fewer than 2^32 threads, so that
// many blocks go into two.  The last row of them may be only begun.
__device__ __forceinline__ int64_t block_index() { return int64_t(blockIdx.y) * gridDim.x + blockIdx.x; }
constexpr int kBwdBlocks = 1024;    // blocks of a backward pass, at the most

// VEC elements of the I/O type, loaded and stored as one access.
template <typename IO, int VEC>
__device__ __forceinline__ void load_vec(const IO *p, float (&f)[VEC]) {
    if constexpr (VEC == 1) {
        f[0] = to_f32<IO>(p[0]);
    } else if constexpr (std::is_same_v<IO, float>) {
        const float4 v = *reinterpret_cast<const float4 *>(p);
        f[0] = v.x; f[1] = v.y; f[2] = v.z; f[3] = v.w;
        if constexpr (VEC == 8) {
            const float4 u = *reinterpret_cast<const float4 *>(p + 4);
            f[4] = u.x; f[5] = u.y; f[6] = u.z; f[7] = u.w;
        }
    } else {
        static_assert(VEC == 8);
        const uint4 v = *reinterpret_cast<const uint4 *>(p);
        f[0] = bf16_lo(v.x); f[1] = bf16_hi(v.x); f[2] = bf16_lo(v.y); f[3] = bf16_hi(v.y);
        f[4] = bf16_lo(v.z); f[5] = bf16_hi(v.z); f[6] = bf16_lo(v.w); f[7] = bf16_hi(v.w);
    }
}

template <typename IO, int VEC>
__device__ __forceinline__ void store_vec(IO *p, const float (&f)[VEC]) {
    if constexpr (VEC == 1) {
        p[0] = from_f32<IO>(f[0]);
    } else if constexpr (std::is_same_v<IO, float>) {
        *reinterpret_cast<float4 *>(p) = make_float4(f[0], f[1], f[2], f[3]);
        if constexpr (VEC == 8) *reinterpret_cast<float4 *>(p + 4) = make_float4(f[4], f[5], f[6], f[7]);
    } else {
        static_assert(VEC == 8);
        *reinterpret_cast<uint4 *>(p) = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]),
                                                   pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
    }
}

// Sum over a team of TPS lanes (16, 64 or the whole 256-thread block); every lane of the
// team ends with the total.  TPS = 256 holds two block barriers.
template <int TPS>
__device__ __forceinline__ float team_sum(float v, float *tmp) {
    v = row16_sum(v);
    if constexpr (TPS == 16) return v;
    v = xor32_sum(xor16_sum(v));
    if constexpr (TPS == 64) return v;
    if ((threadIdx.x & 63) == 0) tmp[threadIdx.x >> 6] = v;
    __syncthreads();
    v = (tmp[0] + tmp[1]) + (tmp[2] + tmp[3]);
    __syncthreads();
    return v;
}

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

// ------------------------------------------------------- before the next block
template <typename IO, typename RES, int VEC, int TPS, int NV>
__global__ __launch_bounds__(kBlock) void k_norm_add_fwd(const IO *__restrict__ x, const RES *residual,
                                                         const float *__restrict__ scale, const float *__restrict__ w,
                                                         RES *sum, IO *__restrict__ y, int64_t rows, int D, float eps) {
    __shared__ float tmp[4];
    constexpr int kTeams = kBlock / TPS;
    const int lane = threadIdx.x % TPS;
    const int64_t row = block_index() * kTeams + threadIdx.x / TPS;
    const bool live = row < rows;
    const int64_t at = (live ? row : 0) * D;
    float s[NV][VEC], xv[NV][VEC];
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * TPS + lane) * VEC;
        if (live && c < D) {
            load_vec<RES, VEC>(residual + at + c, s[i]);
            load_vec<IO, VEC>(x + at + c, xv[i]);
        }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * TPS + lane) * VEC;
        if (!(live && c < D)) continue;
        float sc[VEC];
        if (scale) load_vec<float, VEC>(scale + c, sc);
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

template <typename IO, typename RES, int VEC, int TPS, int NV>
__global__ __launch_bounds__(kBlock) void k_norm_add_bwd(const IO *__restrict__ x, const RES *__restrict__ sum,
                                                         const float *__restrict__ scale, const float *__restrict__ w,
                                                         const IO *__restrict__ dy, const RES *__restrict__ dsum,
                                                         IO *__restrict__ dx, RES *__restrict__ dres,
                                                         float *__restrict__ dwp, float *__restrict__ dsp, int64_t rows,
                                                         int D, int slices, float eps) {
    __shared__ float tmp[4];
    constexpr int kTeams = kBlock / TPS;
    const int lane = threadIdx.x % TPS;
    const int64_t team = int64_t(blockIdx.x) * kTeams + threadIdx.x / TPS;
    const bool live = team < slices;
    const int slice = live ? int(team) : 0;
    float wv[NV][VEC], dw[NV][VEC], ds[NV][VEC];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * TPS + lane) * VEC;
#pragma unroll
        for (int j = 0; j < VEC; ++j) dw[i][j] = ds[i][j] = wv[i][j] = 0.f;
        if (c < D) load_vec<float, VEC>(w + c, wv[i]);
    }
    for (int64_t row0 = 0; row0 < rows; row0 += slices) {
        const int64_t row = row0 + slice;
        const bool on = live && row < rows;
        const int64_t at = (on ? row : 0) * D;
        float s[NV][VEC], d[NV][VEC], e[NV][VEC], xv[NV][VEC];
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * TPS + lane) * VEC;
#pragma unroll
            for (int j = 0; j < VEC; ++j) s[i][j] = d[i][j] = e[i][j] = xv[i][j] = 0.f;
            if (on && c < D) {
                load_vec<RES, VEC>(sum + at + c, s[i]);
                load_vec<IO, VEC>(dy + at + c, d[i]);
                if (dsum) load_vec<RES, VEC>(dsum + at + c, e[i]);
                if (scale) load_vec<IO, VEC>(x + at + c, xv[i]);
            }
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
            const int c = (i * TPS + lane) * VEC;
            if (!(on && c < D)) continue;
            float sc[VEC], ox[VEC];
            if (scale) load_vec<float, VEC>(scale + c, sc);
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                const float g = e[i][j] + r * (d[i][j] - s[i][j] * mean);
                ds[i][j] += g * xv[i][j];
                ox[j] = scale ? g * sc[j] : g;
                e[i][j] = g;
            }
            store_vec<IO, VEC>(dx + at + c, ox);
            store_vec<RES, VEC>(dres + at + c, e[i]);
        }
    }
    if (!live) return;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * TPS + lane) * VEC;
        if (c >= D) continue;
        store_vec<float, VEC>(dwp + int64_t(slice) * D + c, dw[i]);
        if (dsp) store_vec<float, VEC>(dsp + int64_t(slice) * D + c, ds[i]);
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

template <typename IO, typename RES>
__global__ __launch_bounds__(kBlock) void k_norm_add_fwd_loop(const IO *__restrict__ x, const RES *residual,
                                                              const float *__restrict__ scale,
                                                              const float *__restrict__ w, RES *sum, IO *__restrict__ y,
                                                              int64_t rows, int D, float eps) {
    __shared__ float tmp[4];
    if (block_index() >= rows) return;
    const int64_t at = block_index() * D;
    float ss = 0.f;
    for (int c = threadIdx.x; c < D; c += kBlock) {
        const float xv = to_f32<IO>(x[at + c]);
        const RES held = from_f32<RES>(to_f32<RES>(residual[at + c]) + (scale ? scale[c] * xv : xv));
        sum[at + c] = held;     // read back below by the same thread
        const float s = to_f32<RES>(held);
        ss += s * s;
    }
    const float r = 1.f / sqrtf(team_sum<256>(ss, tmp) / float(D) + eps);
    for (int c = threadIdx.x; c < D; c += kBlock) y[at + c] = from_f32<IO>(to_f32<RES>(sum[at + c]) * r * w[c]);
}

template <typename IO, typename RES>
__global__ __launch_bounds__(kBlock) void k_norm_add_bwd_loop(const IO *__restrict__ x, const RES *__restrict__ sum,
                                                              const float *__restrict__ scale,
                                                              const float *__restrict__ w, const IO *__restrict__ dy,
                                                              const RES *__restrict__ dsum, IO *__restrict__ dx,
                                                              RES *__restrict__ dres, float *__restrict__ dwp,
                                                              float *__restrict__ dsp, int64_t rows, int D, int slices,
                                                              float eps) {
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
            if (ds) ds[c] += g * to_f32<IO>(x[at + c]);
            dx[at + c] = from_f32<IO>(scale ? g * scale[c] : g);
            dres[at + c] = from_f32<RES>(g);
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
// The team that holds a segment of `len` elements: vectors of `vec` elements over tps
// lanes, nv each; nv = 0: no team holds it.
struct Team {
    int vec = 0, tps = 0, nv = 0;
};

Team pick_team(int len, bool bf16) {
    const int full = bf16 ? 8 : 4;
    Team t;
    t.vec = len % full == 0 ? full : 1;
    const int vecs = len / t.vec;
    if (t.vec == 1) {
        if (vecs <= 64) { t.tps = 16; t.nv = 4; }
        else if (vecs <= 512) { t.tps = 64; t.nv = 8; }
        else if (vecs <= 2048) { t.tps = 256; t.nv = 8; }
        return t;
    }
    if (vecs <= 16) { t.tps = 16; t.nv = 1; }
    else if (vecs <= 32) { t.tps = 16; t.nv = 2; }
    else if (vecs <= 64) { t.tps = 64; t.nv = 1; }
    else if (vecs <= 128) { t.tps = 64; t.nv = 2; }
    else if (vecs <= 256) { t.tps = 256; t.nv = 1; }
    else if (vecs <= 512) { t.tps = 256; t.nv = 2; }
    else if (vecs <= 768) { t.tps = 256; t.nv = 3; }
    else if (vecs <= 1024) { t.tps = 256; t.nv = 4; }
    else if (vecs <= 1536) { t.tps = 256; t.nv = 6; }
    return t;
}

template <typename IO, class F>
hipError_t with_team(const Team &t, F &&f) {
    using std::integral_constant;
    constexpr int V = std::is_same_v<IO, float> ? 4 : 8;
#define SSD_TEAM(vec_, tps_, nv_) \
    if (t.vec == vec_ && t.tps == tps_ && t.nv == nv_) \
        return f(integral_constant<int, vec_>{}, integral_constant<int, tps_>{}, integral_constant<int, nv_>{});
    SSD_TEAM(1, 16, 4) SSD_TEAM(1, 64, 8) SSD_TEAM(1, 256, 8)
    SSD_TEAM(V, 16, 1) SSD_TEAM(V, 16, 2) SSD_TEAM(V, 64, 1) SSD_TEAM(V, 64, 2)
    SSD_TEAM(V, 256, 1) SSD_TEAM(V, 256, 2) SSD_TEAM(V, 256, 3) SSD_TEAM(V, 256, 4) SSD_TEAM(V, 256, 6)
#undef SSD_TEAM
    return hipErrorInvalidValue;
}

unsigned blocks_of(int64_t units, int per) { return unsigned((units + per - 1) / per); }

// The same in two dimensions (block_index).
dim3 grid_of(int64_t units, int per) {
    constexpr int64_t kRow = 1 << 20;
    const int64_t blocks = (units + per - 1) / per;
    return blocks <= kRow ? dim3(unsigned(blocks)) : dim3(unsigned(kRow), unsigned((blocks + kRow - 1) / kRow));
}

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

template <typename IO, typename RES>
hipError_t add_fwd(const NormAddArgs &a, hipStream_t stream) {
    const auto *x = static_cast<const IO *>(a.x);
    const auto *res = static_cast<const RES *>(a.residual);
    auto *sum = static_cast<RES *>(a.sum);
    auto *y = static_cast<IO *>(a.y);
    const Team t = pick_team(a.D, a.bf16);
    if (!t.nv) {
        hipLaunchKernelGGL((k_norm_add_fwd_loop<IO, RES>), grid_of(a.rows, 1), dim3(kBlock), 0, stream, x, res, a.scale, a.w, sum, y, a.rows, a.D, a.eps);
        return hipGetLastError();
    }
    return with_team<IO>(t, [&](auto v, auto tps, auto nv) {
        hipLaunchKernelGGL((k_norm_add_fwd<IO, RES, v(), tps(), nv()>), grid_of(a.rows, kBlock / tps()), dim3(kBlock), 0, stream,
                           x, res, a.scale, a.w, sum, y, a.rows, a.D, a.eps);
        return hipGetLastError();
    });
}

template <typename IO, typename RES>
hipError_t add_bwd(const NormAddArgs &a, const NormBwdPlan &plan, hipStream_t stream) {
    const auto *x = static_cast<const IO *>(a.x), *dy = static_cast<const IO *>(a.dy);
    const auto *sum = static_cast<const RES *>(a.sum), *dsum = static_cast<const RES *>(a.dsum);
    auto *dx = static_cast<IO *>(a.dx);
    auto *dres = static_cast<RES *>(a.dres);
    auto *part = static_cast<float *>(a.workspace);
    float *dsp = a.scale ? part + size_t(plan.slices) * a.D : nullptr;
    const Team t = pick_team(a.D, a.bf16);
    if (!t.nv) {
        hipLaunchKernelGGL((k_norm_add_bwd_loop<IO, RES>), dim3(plan.slices), dim3(kBlock), 0, stream, x, sum, a.scale, a.w, dy, dsum, dx, dres,
                           part, dsp, a.rows, a.D, plan.slices, a.eps);
        return hipGetLastError();
    }
    return with_team<IO>(t, [&](auto v, auto tps, auto nv) {
        hipLaunchKernelGGL((k_norm_add_bwd<IO, RES, v(), tps(), nv()>), dim3(blocks_of(plan.slices, kBlock / tps())), dim3(kBlock), 0, stream,
                           x, sum, a.scale, a.w, dy, dsum, dx, dres, part, dsp, a.rows, a.D, plan.slices, a.eps);
        return hipGetLastError();
    });
}

hipError_t reduce(const float *part, float *out0, float *out1, int slices, int D, hipStream_t stream) {
    hipLaunchKernelGGL(k_norm_reduce, dim3((D + 63) / 64, out1 ? 2 : 1), dim3(64 * kReduceWaves), 0, stream, part, out0, out1, slices, D);
    return hipGetLastError();
}

}  // namespace

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
    return reduce(static_cast<const float *>(a.workspace), a.dw, nullptr, plan.slices, a.D, stream);
}

hipError_t launch_norm_add_fwd(const NormAddArgs &a, hipStream_t stream) {
    if (!a.bf16) return add_fwd<float, float>(a, stream);
    return a.res_bf16 ? add_fwd<bf16_bits, bf16_bits>(a, stream) : add_fwd<bf16_bits, float>(a, stream);
}

hipError_t launch_norm_add_bwd(const NormAddArgs &a, const NormBwdPlan &plan, hipStream_t stream) {
    hipError_t e;
    if (!a.bf16) e = add_bwd<float, float>(a, plan, stream);
    else e = a.res_bf16 ? add_bwd<bf16_bits, bf16_bits>(a, plan, stream) : add_bwd<bf16_bits, float>(a, plan, stream);
    if (e != hipSuccess) return e;
    return reduce(static_cast<const float *>(a.workspace), a.dw, a.dscale, plan.slices, a.D, stream);
}

}  // namespace ssd
