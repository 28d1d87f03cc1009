// ssd_delta_chunk.hip -- the chunked gated delta rule, forward (see ssd_delta_chunk.h for
// the formulas and the tile layout, ssd_delta_prep.h for the first of its two kernels).
#include <algorithm>

#include "ssd_delta.h"
#include "ssd_delta_prep.h"

namespace ssd {
namespace {

// Planes of the values that stay 32-bit on their way through the bf16 matrix products:
// the state, what is added to it, M and the vectors M meets (3: 24 bits).  y is rounded to
// bf16 at the end, but its terms may be much larger than it is (keys that repeat: each U
// takes back most of the one before), so its operands keep 16 bits.
constexpr int kNS = 3, kNM = 3, kNQ = 2, kNY = 2;

template <typename IO, int N>
struct Tile {
    using Img = ChunkImage<IO, kNM, kNQ>;
    static constexpr int RB = N * int(sizeof(IO));          // bytes per row of k or q
    static constexpr int kRows = kC * RB;                   // bytes of a k or q tile
    static constexpr int kBytes = 2 * kRows + Img::kBytes;  // k, q, then the image
    static constexpr int kBufs = 2 * kBytes <= 160 * 1024 ? 2 : 1;
};

// The chain over the chunks: block = (batch, head, W * 16 rows of the state), one wave per
// 16 rows.  k, q and the chunk's image go through LDS, shared by the waves; the next
// chunk's are copied into the other buffer meanwhile (one buffer where two do not fit).
template <typename IO, int N, int W>
__global__ __launch_bounds__(64 * W) void k_delta_chain(const IO *__restrict__ qg, const IO *__restrict__ kg,
                                                        const IO *__restrict__ vg, const char *__restrict__ images,
                                                        const float *__restrict__ init, IO *__restrict__ yg,
                                                        float *__restrict__ fin, int L, int H, int P, int G, int nc,
                                                        int pblocks, float scale) {
    using T = Tile<IO, N>;
    using Img = typename T::Img;
    extern __shared__ __align__(16) char lds[];
    constexpr int kThreads = 64 * W, KS = N / 32;
    constexpr int kRowIt = T::kRows / 16 / kThreads;
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6, c = lane & 15, q = lane >> 4;
    const int pb = blockIdx.x % pblocks, bh = blockIdx.x / pblocks;
    const int h = bh % H, bi = bh / H, g = h / (H / G);
    const int p0 = (pb * W + w) * 16, p = p0 + c;
    const bool live = p0 < P;       // the same for a whole wave
    const size_t hp = size_t(H) * P, gn = size_t(G) * N;
    const char *img = images + size_t(bh) * nc * Img::kBytes;

    IO rv[16];
    // chunk ch into the LDS buffer `buf` (not waited for), and its v into registers
    auto fetch = [&](int ch, char *buf) {
        const int t0 = ch * kC, last = L - 1 - t0;
        const size_t base = (size_t(bi) * L + t0) * gn + size_t(g) * N;
#pragma unroll
        for (int i = 0; i < kRowIt; ++i) {
            const int at = i * kThreads + tid, r = at / (T::RB / 16), col = (at % (T::RB / 16)) ^ place<T::RB>(r);
            const size_t src = base + min(r, last) * gn + col * (16 / sizeof(IO));
            char *dst = buf + (i * kThreads + 64 * w) * 16;
            copy16(kg + src, dst);
            copy16(qg + src, dst + T::kRows);
        }
        for (int i = w; i < Img::kBytes / 1024; i += W)
            copy16(img + size_t(ch) * Img::kBytes + i * 1024 + lane * 16, buf + 2 * T::kRows + i * 1024);
        if (live)
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    rv[4 * t + r] = vg[(size_t(bi) * L + t0 + min(32 * (t >> 1) + 8 * q + 4 * (t & 1) + r, last)) * hp + size_t(h) * P + p];
    };

    f32x4 S[N / 16];
#pragma unroll
    for (int t = 0; t < N / 16; ++t) {
        S[t] = f32x4{0.f, 0.f, 0.f, 0.f};
        if (init && live)
            S[t] = *reinterpret_cast<const f32x4 *>(init + (size_t(bh) * P + p) * N + 32 * (t >> 1) + 8 * q + 4 * (t & 1));
    }
    fetch(0, lds);
    f32x4 V[4];
    auto take_v = [&]() {
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) V[t][r] = to_f32<IO>(rv[4 * t + r]);
    };
    take_v();
    copies_done();
    __syncthreads();

    for (int ch = 0; ch < nc; ++ch) {
        const char *buf = lds + (T::kBufs == 2 ? (ch & 1) * T::kBytes : 0);
        if (T::kBufs == 2 && ch + 1 < nc) fetch(ch + 1, lds + ((ch + 1) & 1) * T::kBytes);
        if (live) {
            const char *tk = buf, *tq = buf + T::kRows, *tm = buf + 2 * T::kRows + Img::kM, *ts = buf + 2 * T::kRows + Img::kQ;
            const float *gates = reinterpret_cast<const float *>(buf + 2 * T::kRows + Img::kGates);
            Op<IO, kNS> so[KS];
#pragma unroll
            for (int s = 0; s < KS; ++s) so[s] = to_op<IO, kNS>(S[2 * s], S[2 * s + 1]);
            // R = V - e^g K S^T, and beta R
            f32x4 E[4];
            Op<IO, kNM> br[2];
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                f32x4 b[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    f32x4 z = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int ks = 0; ks < KS; ++ks) z = mma(read_row<IO, 1, T::RB>(tk, 0, tile_row(s, e, c), ks, q), so[ks], z);
                    const f32x4 fs = *reinterpret_cast<const f32x4 *>(gates + 32 * s + 8 * q + 4 * e);
                    const f32x4 bt = *reinterpret_cast<const f32x4 *>(gates + 2 * kC + 32 * s + 8 * q + 4 * e);
                    E[2 * s + e] = V[2 * s + e] - fs * z;
                    b[e] = bt * E[2 * s + e];
                }
                br[s] = to_op<IO, kNM>(b[0], b[1]);
            }
            // E = R + M (beta R), U = beta E
            Op<IO, kNY> uy[2];
            Op<IO, kNS> ud[2];
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                f32x4 u[2], d[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    f32x4 z = E[2 * s + e];
#pragma unroll
                    for (int ks = 0; ks <= s; ++ks) z = mma(read_row<IO, kNM, Img::kRow>(tm, Img::kPlane, tile_row(s, e, c), ks, q), br[ks], z);
                    const f32x4 te = *reinterpret_cast<const f32x4 *>(gates + kC + 32 * s + 8 * q + 4 * e);
                    const f32x4 bt = *reinterpret_cast<const f32x4 *>(gates + 2 * kC + 32 * s + 8 * q + 4 * e);
                    u[e] = bt * z;
                    d[e] = te * u[e];
                }
                uy[s] = to_op<IO, kNY>(u[0], u[1]);
                ud[s] = to_op<IO, kNS>(d[0], d[1]);
            }
            // Y, its rows p in registers: 4 consecutive ones of one token per lane
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const int row = tile_row(t >> 1, t & 1, c);
                f32x4 y = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int ks = 0; ks < KS; ++ks) y = mma(first_planes<kNY>(so[ks]), read_row<IO, 1, T::RB>(tq, 0, row, ks, q), y);
                y *= scale * gates[row];
#pragma unroll
                for (int ks = 0; ks <= (t >> 1); ++ks) y = mma(uy[ks], read_row<IO, kNQ, Img::kRow>(ts, Img::kPlane, row, ks, q), y);
                if (ch * kC + row < L) {
                    IO *dst = yg + (size_t(bi) * L + ch * kC + row) * hp + size_t(h) * P + p0 + 4 * q;
                    if constexpr (std::is_same_v<IO, float>) *reinterpret_cast<f32x4 *>(dst) = y;
                    else *reinterpret_cast<uint2 *>(dst) = make_uint2(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]));
                }
            }
            // S <- e^{g_C} S + K^T (e^{g_C - g} U)
            const float alpha = gates[kC - 1];
#pragma unroll
            for (int t = 0; t < N / 16; ++t) {
                f32x4 z = S[t] * alpha;
#pragma unroll
                for (int ks = 0; ks < 2; ++ks) z = mma(read_col<IO, 1, T::RB>(tk, 0, 32 * ks, 32 * (t >> 1), t & 1, c, q), ud[ks], z);
                S[t] = z;
            }
        }
        if (ch + 1 < nc) {
            if constexpr (T::kBufs == 1) {
                __syncthreads();
                fetch(ch + 1, lds);
            }
            take_v();
            copies_done();
            __syncthreads();
        }
    }
    if (fin && live)
#pragma unroll
        for (int t = 0; t < N / 16; ++t)
            *reinterpret_cast<f32x4 *>(fin + (size_t(bh) * P + p) * N + 32 * (t >> 1) + 8 * q + 4 * (t & 1)) = S[t];
}

template <typename IO, int N>
hipError_t launch_n(const DeltaChunkArgs &a, hipStream_t stream) {
    using T = Tile<IO, N>;
    const int nc = (a.L + kC - 1) / kC;
    char *images = static_cast<char *>(a.workspace);
    const auto *q = static_cast<const IO *>(a.q), *k = static_cast<const IO *>(a.k), *v = static_cast<const IO *>(a.v);
    hipLaunchKernelGGL((k_delta_prep<IO, N, kNM, kNQ>), dim3(unsigned(a.b * a.H * nc)), dim3(256), 0, stream, q, k, a.a, a.beta, images,
                       a.L, a.H, a.G, nc, a.scale);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    constexpr int W = 4;
    constexpr int lds = T::kBufs * T::kBytes;
    const int pblocks = (a.P + 16 * W - 1) / (16 * W);
    auto kern = k_delta_chain<IO, N, W>;
    e = hipFuncSetAttribute(reinterpret_cast<const void *>(kern), hipFuncAttributeMaxDynamicSharedMemorySize, lds);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(kern, dim3(unsigned(a.b * a.H * pblocks)), dim3(64 * W), lds, stream, q, k, v, images, a.init_state,
                       static_cast<IO *>(a.y), a.final_state, a.L, a.H, a.P, a.G, nc, pblocks, a.scale);
    return hipGetLastError();
}

template <typename IO>
size_t image_bytes() {
    return ChunkImage<IO, kNM, kNQ>::kBytes;
}

}  // namespace

DeltaChunkPlan plan_delta_chunk(int b, int L, int H, int P, int N, bool bf16) {
    DeltaChunkPlan pl;
    const bool n_ok = N == 32 || N == 64 || N == 128 || (bf16 && N == 256);
    if (!n_ok || P % 16 != 0) return pl;
    const int64_t units = int64_t(b) * H * ((L + kC - 1) / kC);
    if (units > 0x7fffffff || int64_t(b) * H * ((P + 15) / 16) > 0x7fffffff) return pl;
    pl.supported = true;
    pl.total = size_t(units) * (bf16 ? image_bytes<bf16_bits>() : image_bytes<float>());
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
