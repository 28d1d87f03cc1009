// ssd_gated_scan_step.hip -- the gated scan token by token on a kept state.
//
// A stream over the state and the tokens: a lane holds a channel of one batch row, steps it
// through the K tokens and writes the state after the accepted ones.  One token of 64 sequences
// of 5120 channels (4.6 MB) is 3.2 us of kernel, five tokens of 3 sequences 3.4: a call is its
// launch, 10 us from Python.
#include "ssd_gated_scan.h"
#include "ssd_gated_scan_gate.h"

namespace ssd {
namespace {

constexpr int kBlock = 256;
constexpr int kAhead = 4;       // tokens whose loads are under way together

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
    for (int t0 = 0; t0 < K; t0 += kAhead) {
        float xv[kAhead], m[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {      // past the last token: the last one's again
            const size_t at = (size_t(bi) * K + min(t0 + i, K - 1)) * D + c;
            m[i] = to_f32<AIO>(a[at]);
            xv[i] = to_f32<IO>(x[at]);
        }
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            if (t0 + i >= K) break;
            h = step_state<SIGMOID>(gate_of<SIGMOID>(m[i]), h, xv[i]);
            y[(size_t(bi) * K + t0 + i) * D + c] = from_f32<IO>(h);
            if (t0 + i + 1 == acc) kept = h;
        }
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
