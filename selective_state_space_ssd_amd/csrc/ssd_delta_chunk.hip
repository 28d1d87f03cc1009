// ssd_delta_chunk.hip -- the chunked gated delta rule, forward: the part that does not
// depend on the state for all chunks (ssd_delta_prep.h), then the chain over the chunks
// (ssd_delta_chain.h).
#include <algorithm>

#include "ssd_delta.h"
#include "ssd_delta_chain.h"
#include "ssd_delta_prep.h"

namespace ssd {
namespace {

template <typename IO, int N>
hipError_t launch_n(const DeltaChunkArgs &a, hipStream_t stream) {
    using Pl = DeltaPlanes<false>;
    const int nc = (a.L + kC - 1) / kC;
    char *images = static_cast<char *>(a.workspace);
    const auto *q = static_cast<const IO *>(a.q), *k = static_cast<const IO *>(a.k), *v = static_cast<const IO *>(a.v);
    hipError_t e = launch_delta_prep<IO, N, Pl::kM, Pl::kQ>(q, k, a.a, a.beta, images, a.b, a.L, a.H, a.G, a.scale, stream);
    if (e != hipSuccess) return e;
    // waves per block and waves per tile of 16 rows
    auto chain = [&](auto w_, auto x_) {
        constexpr int W = decltype(w_)::value, X = decltype(x_)::value;
        using T = ChainLds<IO, N, W, X, Pl::kQ, true>;
        const int per = 16 * W / X, pblocks = (a.P + per - 1) / per;
        auto kern = k_delta_chain<IO, N, W, X, false>;
        e = hipFuncSetAttribute(reinterpret_cast<const void *>(kern), hipFuncAttributeMaxDynamicSharedMemorySize, T::kBytes);
        if (e != hipSuccess) return e;
        hipLaunchKernelGGL(kern, dim3(unsigned(a.b * a.H * pblocks)), dim3(64 * W), T::kBytes, stream, q, k, v, images, a.init_state,
                           static_cast<IO *>(a.y), a.final_state, nullptr, DeltaSaved{}, a.L, a.H, a.P, a.G, nc, pblocks, a.scale);
        return hipGetLastError();
    };
    return with_chain_shape<IO, N>(a.b, a.H, a.P, chain);
}

}  // namespace

bool delta_chunk_supported(int b, int L, int H, int P, int N, int G, bool bf16) {
    const bool n_ok = N == 32 || N == 64 || N == 128 || (bf16 && N == 256);
    if (!n_ok || P % 16 != 0) return false;
    // grids, and a chunk's extent in bytes, count in 31 bits
    const int64_t bh = int64_t(b) * H, nc = (int64_t(L) + kC - 1) / kC, most = 0x7fffffff;
    return bh * nc <= most && bh * (P / 16) <= most && int64_t(kC) * H * P * 4 <= most && int64_t(kC) * G * N * 4 <= most;
}

DeltaChunkPlan plan_delta_chunk(int b, int L, int H, int P, int N, int G, bool bf16) {
    DeltaChunkPlan pl;
    if (!delta_chunk_supported(b, L, H, P, N, G, bf16)) return pl;
    using Pl = DeltaPlanes<false>;
    pl.supported = true;
    pl.total = size_t(b) * H * ((L + kC - 1) / kC) * (bf16 ? ChunkImage<bf16_bits, Pl::kM, Pl::kQ>::kBytes : ChunkImage<float, Pl::kM, Pl::kQ>::kBytes);
    return pl;
}

hipError_t launch_delta_chunk(const DeltaChunkArgs &a, hipStream_t stream) {
    switch (a.N) {
        case 32: return a.bf16 ? launch_n<bf16_bits, 32>(a, stream) : launch_n<float, 32>(a, stream);
        case 64: return a.bf16 ? launch_n<bf16_bits, 64>(a, stream) : launch_n<float, 64>(a, stream);
        case 128: return a.bf16 ? launch_n<bf16_bits, 128>(a, stream) : launch_n<float, 128>(a, stream);
        case 256: return a.bf16 ? launch_n<bf16_bits, 256>(a, stream) : hipErrorInvalidValue;
        default: return hipErrorInvalidValue;
    }
}

}  // namespace ssd
