// ssd_gated_scan.hip -- the gated scan over whole sequences, and its gradients.
//
//   h_t = alpha_t h_{t-1} + u_t,  y_t = h_t       (the gate: ssd_gated_scan_gate.h)
//
// Gradients, with g_t what reaches h_t from later tokens (g_L = d_final) and lam_t = dy_t + g_t:
//   g_{t-1} = alpha_t lam_t,  d_init = g_0
//   log decay:  dx_t = lam_t,        da_t = lam_t alpha_t h_{t-1}
//   sigmoid:    dx_t = beta_t lam_t, da_t = lam_t alpha_t beta_t (h_{t-1} - x_t)
// The states come from those that were kept before every 32nd token.
#include <limits.h>

#include "ssd_gated_scan.h"
#include "ssd_gated_scan_gate.h"

namespace ssd {
namespace {

constexpr int kBlock = 64;

template <typename IO, typename AIO, bool SIGMOID>
__global__ __launch_bounds__(kBlock) void k_gated_scan_fwd(const IO *__restrict__ x, const AIO *__restrict__ a,
                                                           const float *__restrict__ init_state, IO *__restrict__ y,
                                                           float *__restrict__ kept, float *__restrict__ final_state,
                                                           int L, int D) {
    const int c = blockIdx.x * kBlock + threadIdx.x, bi = blockIdx.y;
    if (c >= D) return;
    const size_t chunks = (size_t(L) + kGatedScanKeep - 1) / kGatedScanKeep;
    float h = init_state ? init_state[size_t(bi) * D + c] : 0.f;
    for (int t = 0; t < L; ++t) {
        if (kept && t % kGatedScanKeep == 0) kept[(bi * chunks + t / kGatedScanKeep) * D + c] = h;
        const size_t at = (size_t(bi) * L + t) * D + c;
        const float m = gate_of<SIGMOID>(to_f32<AIO>(a[at]));
        h = step_state(m, h, entering<SIGMOID>(m, to_f32<IO>(x[at])));
        if (y) y[at] = from_f32<IO>(h);
    }
    if (final_state) final_state[size_t(bi) * D + c] = h;
}

template <typename IO, typename AIO, bool SIGMOID>
__global__ __launch_bounds__(kBlock) void k_gated_scan_bwd(const IO *__restrict__ x, const AIO *__restrict__ a,
                                                           const float *__restrict__ kept, const IO *__restrict__ dy,
                                                           const float *__restrict__ d_final, IO *__restrict__ dx,
                                                           AIO *__restrict__ da, float *__restrict__ d_init, int L, int D) {
    const int c = blockIdx.x * kBlock + threadIdx.x, bi = blockIdx.y;
    if (c >= D) return;
    const int chunks = (L + kGatedScanKeep - 1) / kGatedScanKeep;
    float g = d_final ? d_final[size_t(bi) * D + c] : 0.f;
    for (int k = chunks - 1; k >= 0; --k) {
        const int t0 = k * kGatedScanKeep;
        const size_t base = (size_t(bi) * L + t0) * D + c;
        float before[kGatedScanKeep], h = kept[(size_t(bi) * chunks + k) * D + c];
#pragma unroll
        for (int t = 0; t < kGatedScanKeep; ++t) {
            before[t] = h;
            if (t0 + t < L) {
                const float m = gate_of<SIGMOID>(to_f32<AIO>(a[base + size_t(t) * D]));
                h = step_state(m, h, entering<SIGMOID>(m, to_f32<IO>(x[base + size_t(t) * D])));
            }
        }
#pragma unroll
        for (int t = kGatedScanKeep - 1; t >= 0; --t) {
            if (t0 + t >= L) continue;
            const size_t at = base + size_t(t) * D;
            const float m = gate_of<SIGMOID>(to_f32<AIO>(a[at]));
            const float lam = to_f32<IO>(dy[at]) + g;
            g = step_state(m, lam, 0.f);
            dx[at] = from_f32<IO>(SIGMOID ? beta_of(m) * lam : lam);
            da[at] = from_f32<AIO>(SIGMOID ? g * beta_of(m) * (before[t] - to_f32<IO>(x[at])) : g * before[t]);
        }
    }
    if (d_init) d_init[size_t(bi) * D + c] = g;
}

template <typename IO, typename AIO>
hipError_t fwd(const GatedScanArgs &s, hipStream_t stream) {
    auto run = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, dim3((unsigned(s.D) + kBlock - 1) / kBlock, s.b), dim3(kBlock), 0, stream,
                           static_cast<const IO *>(s.x), static_cast<const AIO *>(s.a), s.init_state,
                           static_cast<IO *>(s.y), s.kept, s.final_state, s.L, s.D);
        return hipGetLastError();
    };
    return s.sigmoid ? run(k_gated_scan_fwd<IO, AIO, true>) : run(k_gated_scan_fwd<IO, AIO, false>);
}

template <typename IO, typename AIO>
hipError_t bwd(const GatedScanArgs &s, hipStream_t stream) {
    auto run = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, dim3((unsigned(s.D) + kBlock - 1) / kBlock, s.b), dim3(kBlock), 0, stream,
                           static_cast<const IO *>(s.x), static_cast<const AIO *>(s.a), s.kept,
                           static_cast<const IO *>(s.dy), s.d_final, static_cast<IO *>(s.dx), static_cast<AIO *>(s.da),
                           s.d_init, s.L, s.D);
        return hipGetLastError();
    };
    return s.sigmoid ? run(k_gated_scan_bwd<IO, AIO, true>) : run(k_gated_scan_bwd<IO, AIO, false>);
}

}  // namespace

// the kernels count tokens and channels in 31 bits, up to a block past the last one
bool gated_scan_supported(int b, int L, int D) { return b <= 65535 && L <= INT_MAX - 64 && D <= INT_MAX - 256; }

size_t gated_scan_workspace(int, int, int, bool) { return 0; }

hipError_t launch_gated_scan_fwd(const GatedScanArgs &a, hipStream_t stream) {
    if (!a.bf16) return fwd<float, float>(a, stream);
    return a.a_bf16 ? fwd<bf16_bits, bf16_bits>(a, stream) : fwd<bf16_bits, float>(a, stream);
}

hipError_t launch_gated_scan_bwd(const GatedScanArgs &a, hipStream_t stream) {
    if (!a.bf16) return bwd<float, float>(a, stream);
    return a.a_bf16 ? bwd<bf16_bits, bf16_bits>(a, stream) : bwd<bf16_bits, float>(a, stream);
}

}  // namespace ssd
