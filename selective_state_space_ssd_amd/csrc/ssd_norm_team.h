// ssd_norm_team.h -- what the norm kernels share: a team of lanes holds one segment of a row
// in registers, vectors of VEC elements (16 bytes) a lane.
#pragma once

#include <algorithm>

#include "ssd_device.h"

namespace ssd {
namespace {

constexpr int kBlock = 256;
constexpr int kWideBlock = 512;     // at the most, of a team that is a block of its own size

// Blocks of a forward pass: one dimension of a launch holds fewer than 2^32 threads, so that
// many blocks go into two.  The last row of them may be only begun.
__device__ __forceinline__ int64_t block_index() { return int64_t(blockIdx.y) * gridDim.x + blockIdx.x; }

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

// Sum over a team of TPS lanes (16, 64, the whole 256-thread block, or 0: a block of any number
// of waves); every lane of the team ends with the total.  A block's holds two barriers.
template <int TPS>
__device__ __forceinline__ float team_sum(float v, float *tmp) {
    v = row16_sum(v);
    if constexpr (TPS == 16) return v;
    v = xor32_sum(xor16_sum(v));
    if constexpr (TPS == 64) return v;
    if ((threadIdx.x & 63) == 0) tmp[threadIdx.x >> 6] = v;
    __syncthreads();
    if constexpr (TPS == 0) {
        v = 0.f;
        for (unsigned i = 0; i < blockDim.x / 64; ++i) v += tmp[i];
    } else {
        v = (tmp[0] + tmp[1]) + (tmp[2] + tmp[3]);
    }
    __syncthreads();
    return v;
}

// ------------------------------------------------------------------------ launches
// The team that holds a segment of `len` elements: vectors of `vec` elements over tps
// lanes, nv each; nv = 0: no team holds it.  vectors = false: elements one by one.
struct Team {
    int vec = 0, tps = 0, nv = 0;
};

Team pick_team(int len, bool bf16, bool vectors = true) {
    const int full = bf16 ? 8 : 4;
    Team t;
    t.vec = vectors && len % full == 0 ? full : 1;
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

}  // namespace
}  // namespace ssd
