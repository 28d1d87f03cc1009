// ssd_delta_chain.h -- the chain over the chunks of the gated delta rule, forward (see
// ssd_delta_chunk.h for the formulas and the tile layout).
#pragma once

#include "ssd_delta_chunk.h"

namespace ssd {

// What the forward chain leaves for the backward pass, per (batch, head):
//   E       [nc][P / 16][4][64] f32x4: a wave's accumulators of the brackets, as held
//   S       [nc][P][N] io: the state that enters each chunk
//   anchor  [P / 16][segments][N / 16][64] f32x4: the state after each segment of chunks
//   ydy     [nc][P / 16][64] fp32: y . dy of each token over the wave's 16 rows
// Chunks per segment.  The gate gradients' error grows with the root of it: da of the
// 4 x 2048-token layer 5.3e-7 of its norm with 1, 1.05e-6 with 4, which saves 47 of 725 us.
// In fp32 the anchors cost nothing measurable.
template <typename IO>
constexpr int kSegment = std::is_same_v<IO, float> ? 1 : 2;

struct DeltaSaved {
    float *E;
    void *S;
    float *anchor;
    float *ydy;
};

// Planes of the values that stay 32-bit on their way through the bf16 matrix products:
// the state, what is added to it, M and the vectors M meets (3: 24 bits).  y is rounded to
// bf16 at the end, but its terms may be much larger than it is (keys that repeat: each U
// takes back most of the one before), so its operands keep 16 bits; for the backward
// pass, whose gate gradients are differences of y . dy, all 24.
template <bool SAVE>
struct DeltaPlanes {
    static constexpr int kS = 3, kM = 3, kQ = SAVE ? 3 : 2;
};

// LDS buffer of one chunk: k, q, the block's 16 W columns of v, the image.
template <typename IO, int N, int W, bool SAVE>
struct ChainTile {
    using Pl = DeltaPlanes<SAVE>;
    using Img = ChunkImage<IO, Pl::kM, Pl::kQ>;
    static constexpr int kSz = int(sizeof(IO));
    static constexpr int RB = N * kSz;                      // bytes per row of k or q
    static constexpr int RV = 16 * W * kSz;                 // bytes per row of v
    static constexpr int kRows = kC * RB, kVals = kC * RV;  // bytes of the tiles
    static constexpr int kQt = kRows, kVt = 2 * kRows, kImg = 2 * kRows + kVals;
    static constexpr int kBytes = kImg + Img::kBytes;
    static constexpr int kBufs = 2 * kBytes <= 160 * 1024 ? 2 : 1;
    static constexpr int kLds = kBufs * kBytes;
};

// Start the copies of ROWS rows of RB bytes (row r at base + r * stride bytes; rows
// past `last`: that one; 16-byte chunks of a row past `chunks`: the last one) into a tile.
// The block's waves take 1 KiB in turn; this call starts part PART of PARTS.
template <int RB, int ROWS, int W, int PART, int PARTS>
__device__ __forceinline__ void copy_rows(const void *base, uint32_t stride, int last, int chunks, uint32_t dst) {
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    constexpr int kIt = ROWS * RB / 1024 / W, kPer = (kIt + PARTS - 1) / PARTS;
#pragma unroll
    for (int i = PART * kPer; i < (PART + 1) * kPer && i < kIt; ++i) {
        const int at = (i * W + w) * 64 + lane, r = at / (RB / 16), col = min((at % (RB / 16)) ^ place<RB>(r), chunks - 1);
        copy16(base, uint32_t(min(r, last)) * stride + uint32_t(col) * 16, dst + uint32_t(i * W + w) * 1024);
    }
}

// The same for an image, linear; a KiB past its end: its last one again.
template <int BYTES, int W, int PART, int PARTS>
__device__ __forceinline__ void copy_image(const char *img, uint32_t dst) {
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    constexpr int kIt = (BYTES / 1024 + W - 1) / W, kPer = (kIt + PARTS - 1) / PARTS;
#pragma unroll
    for (int i = PART * kPer; i < (PART + 1) * kPer && i < kIt; ++i) {
        const int at = min(i * W + w, BYTES / 1024 - 1) * 1024;
        copy16(img + at, uint32_t(lane) * 16, dst + uint32_t(at));
    }
}

// 4 consecutive elements of a range-checked view; past its end: 0.
template <typename IO>
using Raw4 = std::conditional_t<std::is_same_v<IO, float>, f32x4, u32x2>;
template <typename IO>
__device__ __forceinline__ Raw4<IO> load4_checked(__amdgpu_buffer_rsrc_t v, uint32_t off) {
    if constexpr (std::is_same_v<IO, float>) return __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(v, int(off), 0, 0));
    else return __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(v, int(off), 0, 0));
}
template <typename IO>
__device__ __forceinline__ f32x4 widen(Raw4<IO> v) {
    if constexpr (std::is_same_v<IO, float>) return v;
    else return f32x4{bf16_lo(v[0]), bf16_hi(v[0]), bf16_lo(v[1]), bf16_hi(v[1])};
}
template <typename IO>
__device__ __forceinline__ Raw4<IO> narrow(f32x4 v) {
    if constexpr (std::is_same_v<IO, float>) return v;
    else return u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
}

// block = (batch, head, W * 16 rows of the state), one wave per 16 rows.  k, q, v and the
// chunk's image go through LDS; the next chunk's are copied into the other buffer
// meanwhile, a part of them between any two steps (one buffer where two do not fit).
// SAVE: instead of y and the final state, what the backward pass needs (dyg is read).
template <typename IO, int N, int W, bool SAVE>
__global__ __launch_bounds__(64 * W, (SAVE && N * int(sizeof(IO)) > 256) ? 1 : 2) void k_delta_chain(const IO *__restrict__ qg, const IO *__restrict__ kg,
                                                        const IO *__restrict__ vg, const char *__restrict__ images,
                                                        const float *__restrict__ init, IO *__restrict__ yg,
                                                        float *__restrict__ fin, const IO *__restrict__ dyg,
                                                        DeltaSaved saved, int L, int H, int P, int G, int nc, int pblocks,
                                                        float scale) {
    using T = ChainTile<IO, N, W, SAVE>;
    using Img = typename T::Img;
    using Pl = DeltaPlanes<SAVE>;
    extern __shared__ __align__(16) char lds[];
    constexpr int KS = N / 32, kSz = int(sizeof(IO));
    const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6), c = lane & 15, q = lane >> 4;
    const int pb = blockIdx.x % pblocks, bh = blockIdx.x / pblocks;
    const int h = bh % H, bi = bh / H, g = h / (H / G);
    const int p0 = (pb * W + w) * 16, p = p0 + c, ptiles = P / 16;
    const bool live = p0 < P;       // the same for a whole wave
    const size_t hp = size_t(H) * P, gn = size_t(G) * N;
    const char *img = images + size_t(bh) * nc * Img::kBytes;
    const IO *k0 = kg + size_t(bi) * L * gn + size_t(g) * N, *q0 = qg + size_t(bi) * L * gn + size_t(g) * N;
    const IO *v0 = vg + size_t(bi) * L * hp + size_t(h) * P + size_t(pb) * W * 16;
    const int vchunks = min(16 * W, P - pb * W * 16) * kSz / 16;
    const uint32_t lds0 = lds_address(lds), tok = uint32_t(hp) * kSz;

    // the copies of chunk ch into the buffer at `buf`, in 4 parts
    auto fetch = [&](int ch, uint32_t buf, auto part) {
        constexpr int kPart = decltype(part)::value;
        const int t0 = ch * kC, last = min(kC, L - t0) - 1;
        copy_rows<T::RB, kC, W, kPart, 4>(k0 + size_t(t0) * gn, uint32_t(gn) * kSz, last, T::RB / 16, buf);
        copy_rows<T::RB, kC, W, kPart, 4>(q0 + size_t(t0) * gn, uint32_t(gn) * kSz, last, T::RB / 16, buf + T::kQt);
        copy_rows<T::RV, kC, W, kPart, 4>(v0 + size_t(t0) * hp, tok, last, vchunks, buf + T::kVt);
        copy_image<Img::kBytes, W, kPart, 4>(img + size_t(ch) * Img::kBytes, buf + T::kImg);
    };
    auto fetch_all = [&](int ch, uint32_t buf) {
        fetch(ch, buf, std::integral_constant<int, 0>{});
        fetch(ch, buf, std::integral_constant<int, 1>{});
        fetch(ch, buf, std::integral_constant<int, 2>{});
        fetch(ch, buf, std::integral_constant<int, 3>{});
    };

    f32x4 S[N / 16];
#pragma unroll
    for (int t = 0; t < N / 16; ++t) S[t] = f32x4{0.f, 0.f, 0.f, 0.f};
    if (init && live)
#pragma unroll
        for (int t = 0; t < N / 16; ++t)
            S[t] = *reinterpret_cast<const f32x4 *>(init + (size_t(bh) * P + p) * N + 32 * (t >> 1) + 8 * q + 4 * (t & 1));
    fetch_all(0, lds0);
    copies_done();
    __syncthreads();

    for (int ch = 0; ch < nc; ++ch) {
        const int t0 = ch * kC, rows = min(kC, L - t0);
        const char *buf = lds + (T::kBufs == 2 ? (ch & 1) * T::kBytes : 0);
        auto ahead = [&](auto part) {       // past the last chunk: that one again
            if constexpr (T::kBufs == 2) fetch(min(ch + 1, nc - 1), lds0 + ((ch + 1) & 1) * T::kBytes, part);
        };
        ahead(std::integral_constant<int, 0>{});
        Raw4<IO> yo[4];
        f32x4 E[4];
        if (live) {
            const char *tk = buf, *tq = buf + T::kQt, *tm = buf + T::kImg + Img::kM, *ts = buf + T::kImg + Img::kQ;
            const float *gates = reinterpret_cast<const float *>(buf + T::kImg + Img::kGates);
            if constexpr (SAVE) {
                const __amdgpu_buffer_rsrc_t view = buffer_rsrc(dyg + (size_t(bi) * L + t0) * hp + size_t(h) * P, uint32_t(rows - 1) * tok + uint32_t(P) * kSz);
#pragma unroll
                for (int t = 0; t < 4; ++t)
                    yo[t] = load4_checked<IO>(view, uint32_t(tile_row(t >> 1, t & 1, c)) * tok + uint32_t(p0 + 4 * q) * kSz);
            }
            Op<IO, Pl::kS> so[KS];
#pragma unroll
            for (int s = 0; s < KS; ++s) so[s] = to_op<IO, Pl::kS>(S[2 * s], S[2 * s + 1]);
            if constexpr (SAVE) {
                IO *dst = static_cast<IO *>(saved.S) + ((size_t(bh) * nc + ch) * P + p) * N + 8 * q;
#pragma unroll
                for (int s = 0; s < KS; ++s) {
                    if constexpr (kSz == 4) {
                        *reinterpret_cast<f32x4 *>(dst + 32 * s) = S[2 * s];
                        *reinterpret_cast<f32x4 *>(dst + 32 * s + 4) = S[2 * s + 1];
                    } else {
                        *reinterpret_cast<bf16x8 *>(dst + 32 * s) = so[s].p[0];
                    }
                }
            }
            auto gate_of = [&](int which, int t) {
                return *reinterpret_cast<const f32x4 *>(gates + which * kC + 32 * (t >> 1) + 8 * q + 4 * (t & 1));
            };
            // R = V - e^g K S^T, and the state's part of Y (its rows p in registers)
            f32x4 Y[4];
#pragma unroll
            for (int t = 0; t < 4; ++t) E[t] = Y[t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                Op<IO, 1> a[4];
#pragma unroll
                for (int t = 0; t < 4; ++t) a[t] = read_row<IO, 1, T::RB>(tk, 0, tile_row(t >> 1, t & 1, c), ks, q);
                mma(E, a, so[ks]);
            }
            ahead(std::integral_constant<int, 1>{});
            Op<IO, Pl::kM> br[2];
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                f32x4 b[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int t = 2 * s + e;
                    f32x4 V;
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int row = 32 * s + 8 * q + 4 * e + r, at = (16 * w + c) * kSz;
                        V[r] = to_f32<IO>(*reinterpret_cast<const IO *>(buf + T::kVt + row * T::RV + (((at >> 4) ^ place<T::RV>(row)) << 4) + (at & 15)));
                    }
                    E[t] = V - gate_of(0, t) * E[t];
                    b[e] = gate_of(2, t) * E[t];
                }
                br[s] = to_op<IO, Pl::kM>(b[0], b[1]);
            }
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                Op<IO, 1> a[4];
#pragma unroll
                for (int t = 0; t < 4; ++t) a[t] = read_row<IO, 1, T::RB>(tq, 0, tile_row(t >> 1, t & 1, c), ks, q);
                mma(Y, first_planes<Pl::kQ>(so[ks]), a);
            }
            ahead(std::integral_constant<int, 2>{});
            // E = R + M (beta R), U = beta E
            {
                Op<IO, Pl::kM> a[4];
#pragma unroll
                for (int t = 0; t < 4; ++t) a[t] = tri_row<IO, Pl::kM>(tm, t >> 1, t & 1, 0, c, q);
                mma(E, a, br[0]);
            }
            {
                f32x4 lower[2] = {E[2], E[3]};
                Op<IO, Pl::kM> a[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) a[e] = tri_row<IO, Pl::kM>(tm, 1, e, 1, c, q);
                mma(lower, a, br[1]);
                E[2] = lower[0];
                E[3] = lower[1];
            }
            Op<IO, Pl::kQ> uy[2];
            Op<IO, Pl::kS> ud[2];
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const f32x4 u0 = gate_of(2, 2 * s) * E[2 * s], u1 = gate_of(2, 2 * s + 1) * E[2 * s + 1];
                ud[s] = to_op<IO, Pl::kS>(gate_of(1, 2 * s) * u0, gate_of(1, 2 * s + 1) * u1);
                uy[s] = to_op<IO, Pl::kQ>(u0, u1);
            }
            ahead(std::integral_constant<int, 3>{});
            // S <- e^{g_C} S + K^T (e^{g_C - g} U)
            const float alpha = gates[kC - 1];
#pragma unroll
            for (int t = 0; t < N / 16; ++t) S[t] *= alpha;
#pragma unroll
            for (int ks = 0; ks < 2; ++ks)
#pragma unroll
                for (int t0 = 0; t0 < N / 16; t0 += 4) {     // 4 tiles a turn (N = 32 has 2)
                    constexpr int NT = N / 16 < 4 ? N / 16 : 4;
                    f32x4 z[NT];
                    Op<IO, 1> a[NT];
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        z[t] = S[t0 + t];
                        a[t] = read_col<IO, 1, T::RB>(tk, 0, 32 * ks, 32 * ((t0 + t) >> 1), t & 1, c, q);
                    }
                    mma(z, a, ud[ks]);
#pragma unroll
                    for (int t = 0; t < NT; ++t) S[t0 + t] = z[t];
                }
            // Y = scale e^g Q S^T + scores U: 4 consecutive rows p of one token per lane
#pragma unroll
            for (int t = 0; t < 4; ++t) Y[t] *= scale * gates[tile_row(t >> 1, t & 1, c)];
            {
                Op<IO, Pl::kQ> a[4];
#pragma unroll
                for (int t = 0; t < 4; ++t) a[t] = tri_row<IO, Pl::kQ>(ts, t >> 1, t & 1, 0, c, q);
                mma(Y, uy[0], a);
            }
            {
                f32x4 lower[2] = {Y[2], Y[3]};
                Op<IO, Pl::kQ> a[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) a[e] = tri_row<IO, Pl::kQ>(ts, 1, e, 1, c, q);
                mma(lower, uy[1], a);
                Y[2] = lower[0];
                Y[3] = lower[1];
            }
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                if constexpr (SAVE) {
                    const f32x4 d = widen<IO>(yo[t]);
                    const float dot = group4_sum(Y[t][0] * d[0] + Y[t][1] * d[1] + Y[t][2] * d[2] + Y[t][3] * d[3]);
                    if (q == 0) saved.ydy[((size_t(bh) * nc + ch) * ptiles + p0 / 16) * kC + tile_row(t >> 1, t & 1, c)] = dot;
                } else {
                    yo[t] = narrow<IO>(Y[t]);
                }
            }
        } else {
            ahead(std::integral_constant<int, 1>{});
            ahead(std::integral_constant<int, 2>{});
            ahead(std::integral_constant<int, 3>{});
        }
        if constexpr (T::kBufs == 1) {
            __syncthreads();
            if (ch + 1 < nc) fetch_all(ch + 1, lds0);
        }
        copies_done();
        __syncthreads();
        // stores last: nothing waits for them before the next chunk's copies
        if (live) {
            if constexpr (SAVE) {
                f32x4 *dst = reinterpret_cast<f32x4 *>(saved.E) + ((size_t(bh) * nc + ch) * ptiles + p0 / 16) * 256 + lane;
#pragma unroll
                for (int t = 0; t < 4; ++t) dst[64 * t] = E[t];
                if (ch % kSegment<IO> == kSegment<IO> - 1 || ch == nc - 1) {
                    const int segs = (nc + kSegment<IO> - 1) / kSegment<IO>;
                    f32x4 *at = reinterpret_cast<f32x4 *>(saved.anchor) +
                                ((size_t(bh) * ptiles + p0 / 16) * segs + ch / kSegment<IO>) * (N / 16) * 64 + lane;
#pragma unroll
                    for (int t = 0; t < N / 16; ++t) at[64 * t] = S[t];
                }
            } else {
                const __amdgpu_buffer_rsrc_t view = buffer_rsrc(yg + (size_t(bi) * L + t0) * hp + size_t(h) * P, uint32_t(rows - 1) * tok + uint32_t(P) * kSz);
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    const int off = int(uint32_t(tile_row(t >> 1, t & 1, c)) * tok + uint32_t(p0 + 4 * q) * kSz);
                    if constexpr (kSz == 4) __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, yo[t]), view, off, 0, 0);
                    else __builtin_amdgcn_raw_buffer_store_b64(yo[t], view, off, 0, 0);
                }
            }
        }
    }
    if (!SAVE && fin && live)
#pragma unroll
        for (int t = 0; t < N / 16; ++t)
            *reinterpret_cast<f32x4 *>(fin + (size_t(bh) * P + p) * N + 32 * (t >> 1) + 8 * q + 4 * (t & 1)) = S[t];
}

}  // namespace ssd
