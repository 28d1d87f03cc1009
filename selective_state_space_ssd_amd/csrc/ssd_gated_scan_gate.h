// ssd_gated_scan_gate.h -- the gate of the gated scan and one step of its state.
//
//   log decay:  alpha = e^a,             u = x
//   sigmoid:    alpha = 1 / (1 + e^-a),  u = (1 - alpha) x
//
// A decay near 1 is kept as beta = 1 - alpha, a smaller one as alpha, each to a few 2^-24 of
// itself.  Near 1, where long memories lie, alpha in 32 bits is off by up to 2^-25 however
// small beta is, and the same way at every token of a constant gate: at a = -1e-6 the
// memory's length would be off by 3 %, and a state decayed with it by 2^-25 a token.  Far
// from 1 it is beta that says too little of alpha, as after a gate that erases a large state.
// One float holds either: m = alpha, or m = -beta where that is negative.
#pragma once

#include "ssd_device.h"

namespace ssd {

// 1 - e^a for -1/4 < a < 0: the series, whose first term left out is 2^-29 of the sum.
__device__ __forceinline__ float one_minus_exp(float a) {
    float s = 1.f / 5040.f;
    s = fmaf(s, a, 1.f / 720.f);
    s = fmaf(s, a, 1.f / 120.f);
    s = fmaf(s, a, 1.f / 24.f);
    s = fmaf(s, a, 1.f / 6.f);
    s = fmaf(s, a, 0.5f);
    s = fmaf(s, a, 1.f);
    return -a * s;
}

template <bool SIGMOID>
__device__ __forceinline__ float gate_of(float a) {
    if constexpr (SIGMOID) {
        // with t = e^-|a| <= 1: 1 / (1 + t) is the larger of alpha and beta, t / (1 + t) the smaller
        const float t = __builtin_amdgcn_exp2f(-fabsf(a) * kLog2e);
        const float smaller = t * __builtin_amdgcn_rcpf(1.f + t);
        // a = infinity leaves -0, which is no negative number: alpha = 1
        return a > 0.f ? (smaller > 0.f ? -smaller : 1.f) : smaller;
    } else {
        const float alpha = __builtin_amdgcn_exp2f(a * kLog2e);
        return a > -0.25f && a < 0.f ? -one_minus_exp(a) : alpha;
    }
}

__device__ __forceinline__ float alpha_of(float m) { return m < 0.f ? 1.f + m : m; }
__device__ __forceinline__ float beta_of(float m) { return m < 0.f ? -m : 1.f - m; }

// What a token puts into the state.
template <bool SIGMOID>
__device__ __forceinline__ float entering(float m, float x) {
    return SIGMOID ? beta_of(m) * x : x;
}

// alpha h + u.  What a token changes near alpha = 1, u - beta h, is formed before it meets h:
// one rounding of the state a token, and that of a sum with u, which varies.  (h - beta h
// first would be rounded the same way at every token of a constant gate: a state of 4000 with
// beta = 1e-7 was off by 1e-5 of itself after 4096 tokens.)
__device__ __forceinline__ float step_state(float m, float h, float u) { return fmaf(m, h, u) + (m < 0.f ? h : 0.f); }

}  // namespace ssd
