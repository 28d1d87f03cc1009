// ssd_norm_q8.hip -- the residual sum and the norm of the next block, in 8 bits for the
// projection that reads it.
//
//   s = residual + scale x,   y = s r w,   r = (mean s^2 + eps)^-1/2
//   per group of channels:  d = max(max |y| / 448, 2^-126),   q = e4m3(y / d)
//
// 448 is the largest finite e4m3 value; the least d is the smallest normal number, so that
// a group of zeros has a scale to multiply by and to divide by.  y stays in 32 bits until it
// is rounded to e4m3.  A NaN in s leaves NaN in the whole row, an infinity (r = 0) NaN in its
// group and zeros in the others.
//
// The team of ssd_norm_team.h holds the row; a group's maximum is taken as the largest bit
// pattern of |y|, an order in which NaN is above infinity, so nothing of it depends on who
// comes first.  Groups that fill 2^k lanes of a wave (128 bf16 channels: 16) meet in the lanes'
// registers, others in LDS.
//
// Bound by the bytes: 8192 rows of 2560 bf16 channels, fp32 residual, a scale per 128 (232 MB)
// 44 us, 5.3 TB/s; one array into another reaches 6.1.  5 rows of 5120 are the call: 4.6 us of
// kernel in 13.  Not so for groups that vectors of 16 bytes would reach over (not a multiple of 8
// bf16 or 4 fp32 channels): their rows go element by element, up to 2048 channels at 3.3 to 4 TB/s
// (4096 rows of 2048, groups of 4 and 1: 31 us, of 8: 17), longer ones with a wave for a group at a
// time: 4096 rows of 5120 channels in groups of 20 173 us, of 4 635, where groups of 32 take 44.
#include "ssd_norm.h"
#include "ssd_norm_team.h"

namespace ssd {
namespace {

constexpr float kE4m3Max = 448.f, kLeastScale = 0x1p-126f;

__device__ __forceinline__ float scale_of(uint32_t amax_bits) {
    const float d = __uint_as_float(amax_bits) / kE4m3Max;
    return d < kLeastScale ? kLeastScale : d;       // NaN stays
}

template <int CTRL>
__device__ __forceinline__ uint32_t dpp_max(uint32_t v) {
    return max(v, uint32_t(__builtin_amdgcn_update_dpp(0, int(v), CTRL, 0xF, 0xF, false)));
}

// Largest value of 2^k consecutive lanes, lanes_per = 2^k <= 64 (the same for the whole launch).
__device__ __forceinline__ uint32_t lanes_max(uint32_t v, int lanes_per) {
    if (lanes_per > 1) v = dpp_max<0xB1>(v);
    if (lanes_per > 2) v = dpp_max<0x4E>(v);
    if (lanes_per > 4) v = dpp_max<0x141>(v);
    if (lanes_per > 8) v = dpp_max<0x140>(v);
    if (lanes_per > 16) {
        const auto s = __builtin_amdgcn_permlane16_swap(v, v, false, false);
        v = max(uint32_t(s[0]), uint32_t(s[1]));
    }
    if (lanes_per > 32) {
        const auto s = __builtin_amdgcn_permlane32_swap(v, v, false, false);
        v = max(uint32_t(s[0]), uint32_t(s[1]));
    }
    return v;
}

// VEC e4m3 bytes of y / d, one store.
template <int VEC>
__device__ __forceinline__ void store_q8(uint8_t *q, const float (&y)[VEC], float inv) {
    if constexpr (VEC == 1) {
        q[0] = uint8_t(__builtin_amdgcn_cvt_pk_fp8_f32(y[0] * inv, 0.f, 0, false) & 0xff);
    } else {
        uint32_t w[VEC / 4];
#pragma unroll
        for (int k = 0; k < VEC / 4; ++k) {
            int p = __builtin_amdgcn_cvt_pk_fp8_f32(y[4 * k] * inv, y[4 * k + 1] * inv, 0, false);
            w[k] = uint32_t(__builtin_amdgcn_cvt_pk_fp8_f32(y[4 * k + 2] * inv, y[4 * k + 3] * inv, p, true));
        }
        if constexpr (VEC == 4) *reinterpret_cast<uint32_t *>(q) = w[0];
        else *reinterpret_cast<uint2 *>(q) = make_uint2(w[0], w[1]);
    }
}

// Groups of a block: kBlock / TPS rows of at most TPS x NV x VEC channels, a group of VEC
// channels at the least.
template <int VEC, int TPS, int NV>
constexpr int most_groups() { return kBlock * NV; }

// GROUPS: 0 one group a row, 1 groups of VEC 2^k channels that fill 2^k lanes of one wave
// each, 2 any that are a multiple of VEC (their maxima meet in LDS).
template <typename IO, typename RES, int GROUPS, int VEC, int TPS, int NV>
__global__ __launch_bounds__(kBlock) void k_norm_add_q8(const IO *__restrict__ x, const RES *residual,
                                                        const float *__restrict__ scale, const float *__restrict__ w,
                                                        RES *sum, uint8_t *__restrict__ q, float *__restrict__ q_scale,
                                                        int64_t rows, int D, int group, float eps) {
    __shared__ float tmp[4];
    __shared__ uint32_t amax[GROUPS == 2 ? most_groups<VEC, TPS, NV>() : 4];
    constexpr int kTeams = kBlock / TPS;
    const int lane = threadIdx.x % TPS, team = threadIdx.x / TPS;
    const int64_t row = block_index() * kTeams + team;
    const bool live = row < rows;
    const int64_t at = (live ? row : 0) * D;
    const int ngroups = GROUPS ? D / group : 1;
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
    if constexpr (GROUPS == 2) {
        for (int g = threadIdx.x; g < kTeams * ngroups; g += kBlock) amax[g] = 0;
        __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * TPS + lane) * VEC;
        if (!(live && c < D)) continue;
        float sc[VEC];
        if (scale) load_vec<float, VEC>(scale + c, sc);
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
            // the norm sees the sum as it is stored
            s[i][j] = to_f32<RES>(from_f32<RES>(s[i][j] + (scale ? sc[j] * xv[i][j] : xv[i][j])));
            ss += s[i][j] * s[i][j];
        }
        store_vec<RES, VEC>(sum + at + c, s[i]);
    }
    const float r = 1.f / sqrtf(team_sum<TPS>(ss, tmp) / float(D) + eps);
    uint32_t m[NV], all = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * TPS + lane) * VEC;
        m[i] = 0;
        if (live && c < D) {
            float wv[VEC];
            load_vec<float, VEC>(w + c, wv);
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                s[i][j] = s[i][j] * r * wv[j];
                m[i] = max(m[i], __float_as_uint(s[i][j]) & 0x7fffffffu);
            }
            if constexpr (GROUPS == 2) atomicMax(&amax[team * ngroups + c / group], m[i]);
        }
        if constexpr (GROUPS == 1) m[i] = lanes_max(m[i], group / VEC);
        all = max(all, m[i]);
    }
    if constexpr (GROUPS == 0) {
        all = lanes_max(all, TPS < 64 ? TPS : 64);
        if constexpr (TPS == 256) {
            if ((threadIdx.x & 63) == 0) amax[threadIdx.x >> 6] = all;
            __syncthreads();
            all = max(max(amax[0], amax[1]), max(amax[2], amax[3]));
        }
    }
    if constexpr (GROUPS == 2) __syncthreads();
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * TPS + lane) * VEC;
        if (!(live && c < D)) continue;
        const int g = GROUPS ? c / group : 0;
        const float d = scale_of(GROUPS == 0 ? all : GROUPS == 1 ? m[i] : amax[team * ngroups + g]);
        store_q8<VEC>(q + at + c, s[i], 1.f / d);
        if (c == g * group) q_scale[row * ngroups + g] = d;
    }
}

// Rows that no team holds, one block each: the sum is read back, by the block for groups of
// many channels, by a wave each for the others.
template <typename IO, typename RES>
__global__ __launch_bounds__(kBlock) void k_norm_add_q8_loop(const IO *__restrict__ x, const RES *residual,
                                                             const float *__restrict__ scale,
                                                             const float *__restrict__ w, RES *sum,
                                                             uint8_t *__restrict__ q, float *__restrict__ q_scale,
                                                             int64_t rows, int D, int group, float eps) {
    __shared__ float tmp[4];
    __shared__ uint32_t amax[4];
    if (block_index() >= rows) return;
    const int64_t row = block_index(), at = row * D;
    float ss = 0.f;
    for (int c = threadIdx.x; c < D; c += kBlock) {
        const float xv = to_f32<IO>(x[at + c]);
        const RES held = from_f32<RES>(to_f32<RES>(residual[at + c]) + (scale ? scale[c] * xv : xv));
        sum[at + c] = held;     // read back below, behind the barriers of the sum
        const float s = to_f32<RES>(held);
        ss += s * s;
    }
    const float r = 1.f / sqrtf(team_sum<256>(ss, tmp) / float(D) + eps);
    const int ngroups = D / group, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const bool whole = group >= 4 * kBlock;     // a group for the block, or one for each wave
    for (int g = whole ? 0 : wave; g < ngroups; g += whole ? 1 : 4) {
        const int first = whole ? int(threadIdx.x) : lane, step = whole ? kBlock : 64;
        uint32_t m = 0;
        for (int c = first; c < group; c += step)
            m = max(m, __float_as_uint(to_f32<RES>(sum[at + int64_t(g) * group + c]) * r * w[g * group + c]) & 0x7fffffffu);
        m = lanes_max(m, 64);
        if (whole) {
            if (lane == 0) amax[wave] = m;
            __syncthreads();
            m = max(max(amax[0], amax[1]), max(amax[2], amax[3]));
            __syncthreads();
        }
        const float d = scale_of(m), inv = 1.f / d;
        for (int c = first; c < group; c += step) {
            const float y[1] = {to_f32<RES>(sum[at + int64_t(g) * group + c]) * r * w[g * group + c]};
            store_q8<1>(q + at + int64_t(g) * group + c, y, inv);
        }
        if (first == 0) q_scale[row * ngroups + g] = d;
    }
}

template <typename IO, typename RES>
hipError_t add_q8(const NormAddArgs &a, const NormQ8Args &o, hipStream_t stream) {
    const auto *x = static_cast<const IO *>(a.x);
    const auto *res = static_cast<const RES *>(a.residual);
    auto *sum = static_cast<RES *>(a.sum);
    constexpr int full = std::is_same_v<IO, float> ? 4 : 8;
    // vectors that would reach over a group's end go one by one
    const Team t = pick_team(a.D, a.bf16, o.group % full == 0);
    if (!t.nv) {
        hipLaunchKernelGGL((k_norm_add_q8_loop<IO, RES>), grid_of(a.rows, 1), dim3(kBlock), 0, stream, x, res, a.scale, a.w, sum, o.q, o.scale,
                           a.rows, a.D, o.group, a.eps);
        return hipGetLastError();
    }
    const int lanes = o.group / t.vec;
    const bool in_lanes = o.group % t.vec == 0 && (lanes & (lanes - 1)) == 0 && lanes <= (t.tps < 64 ? t.tps : 64);
    return with_team<IO>(t, [&](auto v, auto tps, auto nv) {
        auto run = [&](auto kernel) {
            hipLaunchKernelGGL(kernel, grid_of(a.rows, kBlock / tps()), dim3(kBlock), 0, stream, x, res, a.scale, a.w, sum, o.q, o.scale,
                               a.rows, a.D, o.group, a.eps);
            return hipGetLastError();
        };
        if (o.group == a.D) return run(k_norm_add_q8<IO, RES, 0, v(), tps(), nv()>);
        if (in_lanes) return run(k_norm_add_q8<IO, RES, 1, v(), tps(), nv()>);
        return run(k_norm_add_q8<IO, RES, 2, v(), tps(), nv()>);
    });
}

}  // namespace

hipError_t launch_norm_add_q8(const NormAddArgs &a, const NormQ8Args &o, hipStream_t stream) {
    if (!a.bf16) return add_q8<float, float>(a, o, stream);
    return a.res_bf16 ? add_q8<bf16_bits, bf16_bits>(a, o, stream) : add_q8<bf16_bits, float>(a, o, stream);
}

}  // namespace ssd
