// ssd_gated_scan_step.hip -- the gated scan token by token on a kept state.
//
// A stream over the state and the tokens: a lane holds VEC consecutive channels of one batch
// row, steps them through the K tokens and writes the state after the accepted ones.  All
// loads of a call are independent of each other and issued first.
#include "ssd_gated_scan.h"
#include "ssd_gated_scan_gate.h"

namespace ssd {
namespace {

constexpr int kBlock = 256;


template <typename IO, typename AIO, bool SIGMOID>
__global__ __launch_bounds__(kBlock) void k_gated_scan_step(const float *state_in, const IO *__restrict__ x,
                                                            const AIO *__restrict__ a,
                                                            const int32_t *__restrict__ accept_len, IO *__restrict__ y,
                                                            float *state_out, int32_t *err_flag, int K, int D) {
    const int c = blockIdx.x * kBlock + threadIdx.x, bi = blockIdx.y;
    int acc = accept_len ? accept_len[bi] : K;
    if (acc < 0 || acc > K) {
        if (err_flag && blockIdx.x == 0 && threadIdx.x == 0) *err_flag = 1;
        acc = acc < 0 ? 0 : K;
    }
    if (c >= D) return;
    float h = state_in[size_t(bi) * D + c], kept = h;
    for (int t = 0; t < K; ++t) {
        const size_t at = (size_t(bi) * K + t) * D + c;
        const float m = gate_of<SIGMOID>(to_f32<AIO>(a[at]));
        h = step_state<SIGMOID>(m, h, to_f32<IO>(x[at]));
        y[at] = from_f32<IO>(h);
        if (t + 1 == acc) kept = h;
    }
    state_out[size_t(bi) * D + c] = kept;
}

template <typename IO, typename AIO>
hipError_t step(const GatedStepArgs &s, hipStream_t stream) {
    auto run = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, dim3((unsigned(s.D) + kBlock - 1) / kBlock, s.b), dim3(kBlock), 0, stream, s.state_in,
                           static_cast<const IO *>(s.x), static_cast<const AIO *>(s.a), s.accept_len,
                           static_cast<IO *>(s.y), s.state_out, s.err_flag, s.K, s.D);
        return hipGetLastError();
    };
    return s.sigmoid ? run(k_gated_scan_step<IO, AIO, true>) : run(k_gated_scan_step<IO, AIO, false>);
}

}  // namespace

hipError_t launch_gated_scan_step(const GatedStepArgs &s, hipStream_t stream) {
    if (!s.bf16) return step<float, float>(s, stream);
    return s.a_bf16 ? step<bf16_bits, bf16_bits>(s, stream) : step<bf16_bits, float>(s, stream);
}

}  // namespace ssd
