// ssd_gated_scan_gate.h -- the gate of the gated scan and one step of its state.
//
//   log decay:  alpha = e^a,             u = x
//   sigmoid:    alpha = 1 / (1 + e^-a),  u = (1 - alpha) x
//
// A decay near 1 is kept as beta = 1 - alpha, a smaller one as alpha, each to a few 2^-24 of
// itself (a log decay's series for beta to 1.1), and where exp2 makes it |a| 2^-24 more, the
// rounding of a log2 e: 9 2^-24 of a state that a gate of 1e-4 leaves.  Near 1, where long memories lie, alpha in 32 bits is off by up to 2^-25 however
// small beta is, and the same way at every token of a constant gate: at a = -1e-6 the
// memory's length would be off by 3 %, and a state decayed with it by 2^-25 a token.  Far
// from 1 it is beta that says too little of alpha, as after a gate that erases a large state.
// One float holds either: m = alpha with the sign bit clear, or m = -beta with the sign bit set.
#pragma once

#include "ssd_device.h"

namespace ssd {

// The same value, of which the compiler does not know that: what is made of it is made where
// it is used, and what it is made of is computed without a branch.
__device__ __forceinline__ float here(float v) {
    asm("" : "+v"(v));
    return v;
}

template <bool SIGMOID>
__device__ __forceinline__ float gate_of(float a) {
    const float na = -kLog2e * a;
    if constexpr (SIGMOID) {
        // 1 / (1 + e^|a|) is the smaller of alpha and beta: beta where a is not negative
        const uint32_t smaller = __float_as_uint(__builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(fabsf(na))));
        return __uint_as_float((smaller & 0x7fffffffu) | (__float_as_uint(na) & 0x80000000u));
    } else {
        // e^a - 1 for -1/16 < a < 0: the series, whose first term left out is 2^-29 of the sum.
        // (Further from 1, alpha's rounding is at most 2^-21 of beta.)  Both sides are cheaper
        // than a branch around either, which most waves would take twice.
        const float alpha = here(__builtin_amdgcn_exp2f(-na));
        float s = fmaf(1.f / 120.f, a, 1.f / 24.f);
        s = fmaf(s, a, 1.f / 6.f);
        s = fmaf(s, a, 0.5f);
        s = fmaf(s, a, 1.f);
        s = here(s * a);
        return a > -0.0625f && a < 0.f ? s : alpha;
    }
}

__device__ __forceinline__ bool near_one(float m) { return int32_t(__float_as_uint(m)) < 0; }
__device__ __forceinline__ float alpha_of(float m) { return near_one(m) ? 1.f + m : m; }
__device__ __forceinline__ float beta_of(float m) { return near_one(m) ? -m : 1.f - m; }

// alpha h + u.  What a token changes near alpha = 1, u - beta h, is formed before it meets h:
// one rounding of the state a token, and that of a sum with u, which varies.  (h - beta h
// first would be rounded the same way at every token of a constant gate: a state of 4000 with
// beta = 1e-7 was off by 1e-5 of itself after 4096 tokens.)
__device__ __forceinline__ float apply_pair(float m, float h, float u) { return fmaf(m, h, u) + (near_one(m) ? h : 0.f); }

// The state after a token.  sigmoid: alpha h + (1 - alpha) x is h - beta (h - x), or x +
// alpha (h - x).
template <bool SIGMOID>
__device__ __forceinline__ float step_state(float m, float h, float x) {
    if constexpr (SIGMOID) return fmaf(m, h - x, near_one(m) ? h : x);
    else return apply_pair(m, h, x);
}

// alpha h
__device__ __forceinline__ float decayed(float m, float h) { return fmaf(m, h, near_one(m) ? h : 0.f); }

}  // namespace ssd
