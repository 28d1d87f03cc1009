// ssd_delta_step.hip -- the gated delta rule token by token on gfx950.
//
// Per (batch, head), state S [P x N], for each token
//   S <- e^a S;   u = beta (v - S k);   S <- S + u k^T;   y = scale S q.
// With the state before the token both products can be taken at once,
//   y = scale (e^a (S q) + u (k . q)),   u = beta (v - e^a (S k)),
// so the two sums over N, and k . q, leave one dependent step per token.
//
// For a few tokens the work is a stream over the state: read once, updated in registers,
// written once.  A row of the state is spread over LR consecutive lanes, J chunks of 4
// columns each, interleaved so that one load of the wave covers whole 128-byte pieces;
// rows never meet.  k and q of a block of tokens are shared by all rows and staged in
// LDS as fp32, v and the gates are read by the rows that use them.
//
// One token of 64 sequences, 32 heads of 128 x 128 (274 MB, nearly all of it the state in and
// out): 46 us, 5.8 TB/s; a copy of that size reaches 5.2.  With few rows a call is its
// launch: 5 tokens of 3 sequences, 16 heads of 64 x 128, take 12.5 us with the call's host
// side, the kernel itself under 5.
#include "ssd_delta.h"
#include "ssd_device.h"

namespace ssd {
namespace {

constexpr int kTok = 16;    // tokens staged at a time

template <int N>
struct StepShape {
    static constexpr int LR = (N >= 32) ? 8 : N / 4;   // lanes per state row
    static constexpr int J = N / (4 * LR);             // 4-column chunks per lane
    static constexpr int RW = 64 / LR;                 // rows per wave
    static constexpr int RB = 4 * RW;                  // rows per block
    static_assert(N == 16 ? RB == 64 : RB == 32);
};

// Sum over the LR (4 or 8) consecutive lanes of a row.
template <int LR>
__device__ __forceinline__ float lanes_sum(float v) {
    v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0xB1, 0xF, 0xF, false));
    v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x4E, 0xF, 0xF, false));
    if constexpr (LR == 8)
        v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x141, 0xF, 0xF, false));
    return v;
}

template <typename IO>
__device__ __forceinline__ float4 read4(const IO *p) {
    if constexpr (std::is_same_v<IO, float>) {
        return *reinterpret_cast<const float4 *>(p);
    } else {
        const uint2 v = *reinterpret_cast<const uint2 *>(p);
        return make_float4(bf16_lo(v.x), bf16_hi(v.x), bf16_lo(v.y), bf16_hi(v.y));
    }
}

template <typename IO, int N>
__global__ __launch_bounds__(256) void k_delta_step(const float *state_in, const IO *__restrict__ q,
                                                    const IO *__restrict__ k, const IO *__restrict__ v,
                                                    const float *__restrict__ a, const float *__restrict__ beta,
                                                    const int32_t *__restrict__ accept_len, IO *__restrict__ y,
                                                    float *state_out, int32_t *err_flag, int L, int H, int P, int G,
                                                    float scale) {
    using S = StepShape<N>;
    __shared__ __align__(16) float sk[kTok * N], sq[kTok * N];
    const int lr = (threadIdx.x & 63) % S::LR;
    const int p = blockIdx.x * S::RB + threadIdx.x / S::LR;
    const int h = blockIdx.y, bi = blockIdx.z, g = h / (H / G);
    const bool valid = p < P;
    const size_t row = ((size_t(bi) * H + h) * P + (valid ? p : 0)) * N;

    float4 s[S::J];
#pragma unroll
    for (int j = 0; j < S::J; ++j) {
        s[j] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (state_in && valid) {
            const f32x4 t = __builtin_nontemporal_load(
                reinterpret_cast<const f32x4 *>(state_in + row + j * 4 * S::LR + lr * 4));
            s[j] = make_float4(t.x, t.y, t.z, t.w);
        }
    }
    int acc = accept_len ? accept_len[bi] : L;
    if (acc < 0 || acc > L) {
        if (err_flag && blockIdx.x == 0 && h == 0 && threadIdx.x == 0) *err_flag = 1;
        acc = acc < 0 ? 0 : L;
    }
    auto store_state = [&]() {
#pragma unroll
        for (int j = 0; j < S::J; ++j)
            __builtin_nontemporal_store(f32x4{s[j].x, s[j].y, s[j].z, s[j].w},
                                        reinterpret_cast<f32x4 *>(state_out + row + j * 4 * S::LR + lr * 4));
    };
    if (acc == 0 && valid && state_out) store_state();

    for (int t0 = 0; t0 < L; t0 += kTok) {
        const int nt = min(kTok, L - t0);
        if (t0) __syncthreads();
        for (int i = 4 * int(threadIdx.x); i < nt * N; i += 1024) {
            const size_t src = ((size_t(bi) * L + t0 + i / N) * G + g) * N + i % N;
            *reinterpret_cast<float4 *>(sk + i) = read4<IO>(k + src);
            *reinterpret_cast<float4 *>(sq + i) = read4<IO>(q + src);
        }
        __syncthreads();
        for (int t = 0; t < nt; ++t) {
            const size_t bt = (size_t(bi) * L + t0 + t) * H + h;
            const float alpha = expf(a[bt]), bt_ = beta[bt];
            const float vv = valid ? to_f32<IO>(v[bt * P + p]) : 0.f;
            float ks = 0.f, qs = 0.f, kq = 0.f;
            float4 kk[S::J];
#pragma unroll
            for (int j = 0; j < S::J; ++j) {
                const int n = j * 4 * S::LR + lr * 4;
                kk[j] = *reinterpret_cast<const float4 *>(sk + t * N + n);
                const float4 qq = *reinterpret_cast<const float4 *>(sq + t * N + n);
                ks += s[j].x * kk[j].x + s[j].y * kk[j].y + s[j].z * kk[j].z + s[j].w * kk[j].w;
                qs += s[j].x * qq.x + s[j].y * qq.y + s[j].z * qq.z + s[j].w * qq.w;
                kq += kk[j].x * qq.x + kk[j].y * qq.y + kk[j].z * qq.z + kk[j].w * qq.w;
            }
            ks = lanes_sum<S::LR>(ks);
            qs = lanes_sum<S::LR>(qs);
            kq = lanes_sum<S::LR>(kq);
            const float u = bt_ * (vv - alpha * ks);
            if (valid && lr == 0) y[bt * P + p] = from_f32<IO>(scale * (alpha * qs + u * kq));
#pragma unroll
            for (int j = 0; j < S::J; ++j) {
                s[j].x = alpha * s[j].x + u * kk[j].x;
                s[j].y = alpha * s[j].y + u * kk[j].y;
                s[j].z = alpha * s[j].z + u * kk[j].z;
                s[j].w = alpha * s[j].w + u * kk[j].w;
            }
            if (t0 + t + 1 == acc && valid && state_out) store_state();
        }
    }
}

template <typename IO, int N>
hipError_t launch_n(const DeltaStepArgs &a, hipStream_t stream) {
    using S = StepShape<N>;
    hipLaunchKernelGGL((k_delta_step<IO, N>), dim3((a.P + S::RB - 1) / S::RB, a.H, a.b), dim3(256), 0, stream,
                       a.state_in, static_cast<const IO *>(a.q), static_cast<const IO *>(a.k),
                       static_cast<const IO *>(a.v), a.a, a.beta, a.accept_len, static_cast<IO *>(a.y), a.state_out,
                       a.err_flag, a.L, a.H, a.P, a.G, a.scale);
    return hipGetLastError();
}

template <typename IO>
hipError_t launch_io(const DeltaStepArgs &a, hipStream_t stream) {
    switch (a.N) {
        case 16: return launch_n<IO, 16>(a, stream);
        case 32: return launch_n<IO, 32>(a, stream);
        case 64: return launch_n<IO, 64>(a, stream);
        case 128: return launch_n<IO, 128>(a, stream);
        case 256: return launch_n<IO, 256>(a, stream);
        default: return hipErrorInvalidValue;
    }
}

}  // namespace

bool delta_step_supported_n(int N) { return N == 16 || N == 32 || N == 64 || N == 128 || N == 256; }

int delta_step_most_rows(int N) { return ((1 << 24) - 1) * (N == 16 ? StepShape<16>::RB : StepShape<32>::RB); }

hipError_t launch_delta_step(const DeltaStepArgs &a, hipStream_t stream) {
    return a.bf16 ? launch_io<bf16_bits>(a, stream) : launch_io<float>(a, stream);
}

}  // namespace ssd
