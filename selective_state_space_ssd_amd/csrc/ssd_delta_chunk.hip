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
hipError_t launch_n(const DeltaChunkArgs &a, const DeltaChunkPlan &pl, hipStream_t stream) {
    char *images = static_cast<char *>(a.workspace);
    auto *map = reinterpret_cast<float *>(images + pl.off_map), *init = reinterpret_cast<float *>(images + pl.off_init);
    const auto *q = static_cast<const IO *>(a.q), *k = static_cast<const IO *>(a.k), *v = static_cast<const IO *>(a.v);
    hipError_t e = launch_delta_prep<IO, N>(q, k, a.a, a.beta, images, a.b, a.L, a.H, a.G, a.scale, stream);
    if (e != hipSuccess) return e;
    if ((e = enter_segments<IO, N, false>(q, k, v, images, a.init_state, map, init, a.b, a.L, a.H, a.P, a.G, pl.cut, a.scale, stream)) != hipSuccess)
        return e;
    auto go = [&](auto w_, auto x_, auto one_) {
        constexpr int W = decltype(w_)::value, X = decltype(x_)::value;
        return launch_chain<IO, N, W, X, Chain::run, decltype(one_)::value>(q, k, v, images, pl.cut.segments > 1 ? init : a.init_state, static_cast<IO *>(a.y),
                                                             a.final_state, DeltaSaved{}, a.b, a.L, a.H, a.P, a.G, pl.cut.per,
                                                             pl.cut.segments, a.scale, stream);
    };
    return with_chain_shape<IO, N, false>(int64_t(a.b) * a.H * pl.cut.segments * (a.P / 16), go);
}

}  // namespace

// Chains wait for their own results, chunk after chunk; with few (batch, head)s most of the
// device is idle meanwhile.  A sequence cut into segments needs each chunk twice, once to see
// what its segment does to any state (P + N rows instead of P) and once with the state that
// enters it, but all segments run at once.  The cut is the cheapest by the measured cost of a
// chunk, in units of one step of a chain that has its SIMD to itself (3.4 us in bf16, N =
// 128).  One segment -> this rule -> the best of 1, 2, 3, 4, 5, 6, 8, 11, 16, 24, 32, 64, us, b = 1:
//   bf16, P = N = 128:  3 heads, 4096 tokens 210 -> 85 -> 83, 16384: 788 -> 161 -> 168;
//                       32 heads, 4096: 227 -> 192 -> 191, 16384: 874 -> 664 -> 631
//   fp32, P = N = 64:   24 heads, 1600 tokens 139 -> 85 -> 83, 16384: 1186 -> 432 -> 436
// and over 432 shapes of 1 to 192 heads and 256 to 16384 tokens 1.01 times as long as that best
// in the mean, 1.22 times at the most.  Backward, 216 shapes: 1.01, 1.14 at the most;
//   bf16, P = 64, N = 128:  24 heads, 2048 tokens 256 -> 200 -> 199, 6000: 712 -> 435 -> 436
//   fp32, P = N = 64:   4 heads, 777 tokens 152 -> 113 -> 112, 6000: 839 -> 190 -> 187
// More tiles than SIMDs go in rounds, forward cheaper ones, where two blocks a CU cover for
// each other (with_chain_shape).
DeltaCut cut_sequence(int64_t bh, int nc, int P, int N, bool bf16, bool back) {
    const bool wide = N * (bf16 ? 2 : 4) > 256;     // blocks of 8 waves for 2 tiles
    auto step = [&](int64_t tiles) {
        if (wide) return tiles <= kSimds / 4 ? 1.0 : 1.5 * double((tiles + kSimds / 2 - 1) / (kSimds / 2));
        if (tiles <= kSimds / 2) return tiles <= kSimds / 4 ? 0.8 : 0.85;       // shared by waves
        return tiles <= kSimds ? 1.0 : (back ? 1.0 : 0.85) * double((tiles + kSimds - 1) / kSimds);
    };
    const double carry = N == 256 ? 1.5 : N == 128 ? 0.35 : 0.2, launches = 2.0;
    DeltaCut best{1, nc};
    // a map costs a little less than a run; backward: a chain each way, and the chain back over
    // zeros for its map
    const double passes = back ? 2.0 : 1.0, extra = back ? 0.8 : 0.0, map = 0.75;
    double least = 0.95 * nc * passes * step(bh * (P / 16));      // no cut for less than a twentieth
    for (int s = 2; s <= std::min(nc / 2, 64); ++s) {
        const int per = (nc + s - 1) / s;
        if ((nc + per - 1) / per != s) continue;
        const double c = per * ((passes + extra) * step(bh * s * (P / 16)) + map * step(bh * (s - 1) * ((P + N) / 16))) + passes * (carry * s + launches);
        if (c < least) {
            least = c;
            best = {s, per};
        }
    }
    return best;
}

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
    pl.supported = true;
    const int nc = (L + kC - 1) / kC;
    const size_t bh = size_t(b) * H;
    pl.total = bh * nc * (bf16 ? ChunkImage<bf16_bits>::kBytes : ChunkImage<float>::kBytes);
    pl.cut = cut_sequence(int64_t(bh), nc, P, N, bf16, false);
    pl.off_map = pl.total;
    pl.off_init = pl.off_map + map_bytes(bh, P, N, pl.cut);
    pl.total = pl.off_init + entering_bytes(bh, P, N, pl.cut);
    return pl;
}

hipError_t launch_delta_chunk(const DeltaChunkArgs &a, const DeltaChunkPlan &pl, hipStream_t stream) {
    switch (a.N) {
        case 32: return a.bf16 ? launch_n<bf16_bits, 32>(a, pl, stream) : launch_n<float, 32>(a, pl, stream);
        case 64: return a.bf16 ? launch_n<bf16_bits, 64>(a, pl, stream) : launch_n<float, 64>(a, pl, stream);
        case 128: return a.bf16 ? launch_n<bf16_bits, 128>(a, pl, stream) : launch_n<float, 128>(a, pl, stream);
        case 256: return a.bf16 ? launch_n<bf16_bits, 256>(a, pl, stream) : hipErrorInvalidValue;
        default: return hipErrorInvalidValue;
    }
}

}  // namespace ssd
