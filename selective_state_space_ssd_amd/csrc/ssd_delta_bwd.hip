// ssd_delta_bwd.hip -- gradients of the gated delta rule, in chunks of 64 tokens (formulas,
// names and tile layout of the forward pass: ssd_delta_chunk.h).
//
// Nothing is kept from the forward pass; five kernels:
//   1 prep       M and the scores of every chunk (ssd_delta_prep.h)
//   2 chain      forward over the chunks: E, the entering states, y . dy (ssd_delta_chain.h)
//   3 chain back from d_final, with dS the gradient of the state a chunk leaves:
//        dU = scores^T dY + e^{g_C - g} (K dS^T),   X = dU + M^T (beta dU)
//        dv = beta X,   dbeta_i = X_i . E_i
//        dS <- e^{g_C} dS + (scale e^g dY)^T Q - (e^g dv)^T K
//   4 grads      per chunk; dq and dk are sums over a group's heads, taken in one block, or
//                in a few whose fp32 sums a further kernel adds:
//        dq = scale e^g dY S + W K,                      W_ij = scale (dy_i . u_j) D_ij, j <= i
//        dk = -e^g dv S + e^{g_C - g} U dS + W^T Q + G K,  G = F + F^T, F_ij = -(dv_i . u_j) D_ij, j < i
//      Both are differences where the chunk's updates erase a large state, or the gradient of
//      one: states, U, dv, W and G keep 32 bits here too, and dq and dk are rounded once.
//   5 gates      da.  The gates only scale v going in and y coming out of an ungated rule,
//        so the gradient of the gate sum at token t is y_t . dy_t - v_t . dv_t, and
//        da_t = sum of it from t to the end of a segment + <dS, S> at the segment's end.
// 2 and 3 are chains over the chunks whose waves keep 16 rows of the state each, as in the
// forward pass: 32-bit values throughout, since da and dbeta come out of differences.
//
// 4 x 2048 tokens, 32 heads of 128 x 128, bf16, us: prep 45, chain 216, chain back 287, grads
// 325, gates 9.  The chains are bound by a wave's steps (ssd_delta_chain.h) and write 805 MB
// (both states, E and X, in 32 bits); grads reads 870 MB, 2.7 TB/s.
#include <algorithm>

#include "ssd_delta.h"
#include "ssd_delta_chain.h"
#include "ssd_delta_prep.h"

namespace ssd {
namespace {

// Sums over 16 rows of the state, per token: fp32 [nc][P / 16][64] each.
struct BackSums {
    float *xe, *vdv;
    float *lam;         // [P / 16][segments][X]: <dS, S> at the end of each segment, in parts
};

// Kernel 3.  Waves, tiles and LDS as in the forward chain; dy is read by every wave.  One
// chain per (batch, head, segment of `per` chunks).  What leaves the last segment is d_final,
// what leaves the others is in `d_enter`.  MAP: of the segments 1 .. segs - 1, only the
// gradient of the state that enters each, into d_out [segs], with 0 for what leaves the
// others; the forward maps tell what d_enter adds to it.
template <typename IO, int N, int W, int X, bool MAP, bool ONE>
__global__ __launch_bounds__(64 * W) void k_delta_chain_back(const IO *__restrict__ qg, const IO *__restrict__ kg,
                                                             const IO *__restrict__ vg, const IO *__restrict__ dyg,
                                                             const char *__restrict__ images, const float *__restrict__ d_final,
                                                             const float *__restrict__ d_enter, const f32x4 *__restrict__ E,
                                                             const f32x4 *__restrict__ anchor, IO *__restrict__ dvg,
                                                             float *__restrict__ dSg, f32x4 *__restrict__ Xg, float *__restrict__ d_out, BackSums sums, int L,
                                                             int H, int P, int G, int nc, int per, int segs, int pblocks,
                                                             float scale) {
    using T = ChainLds<IO, N, W, X, false, ONE>;
    using Img = typename T::Img;
    extern __shared__ __align__(16) char lds[];
    constexpr int kSz = int(sizeof(IO)), KS = N / 32 / X, NT = 2 * KS;
    const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6), c = lane & 15, q = lane >> 4;
    const int x = w % X, n0 = x * KS;
    const int blk = xcd_neighbours(), pb = blk % pblocks, chain = blk / pblocks, skip = MAP ? 1 : 0;
    const int seg = chain % (segs - skip) + skip, bh = chain / (segs - skip), first = seg * per, last = min(first + per, nc) - 1;
    const int h = bh % H, bi = bh / H, g = h / (H / G);
    const int p0 = (pb * (W / X) + w / X) * 16, p = p0 + c, ptiles = P / 16, anchors = (nc + kSegment<IO> - 1) / kSegment<IO>;
    const bool live = p0 < P;
    const size_t hp = size_t(H) * P, gn = size_t(G) * N;
    const char *img = images + size_t(bh) * nc * Img::kBytes;
    const IO *k0 = kg + size_t(bi) * L * gn + size_t(g) * N, *q0 = qg + size_t(bi) * L * gn + size_t(g) * N;
    const size_t vy0 = size_t(bi) * L * hp + size_t(h) * P;
    const uint32_t lds0 = lds_address(lds), tok = uint32_t(hp) * kSz;
    char *xe = lds + T::kE + w * 4096;

    auto fetch = [&](int ch, uint32_t buf, auto part) {
        constexpr int kPart = decltype(part)::value;
        const int t0 = ch * kC, last = min(kC, L - t0) - 1;
        copy_rows<T::RB, kC, W, kPart, 4>(k0 + size_t(t0) * gn, uint32_t(gn) * kSz, last, T::RB / 16, buf);
        copy_image<Img::kBytes, W, kPart, 4>(img + size_t(ch) * Img::kBytes, buf + T::kImg);
        if constexpr (T::kQMain) copy_rows<T::RB, kC, W, kPart, 4>(q0 + size_t(t0) * gn, uint32_t(gn) * kSz, last, T::RB / 16, buf + T::kRows);
    };
    auto fetch_q = [&](int ch) {
        if constexpr (T::kQMain) return;
        const int t0 = ch * kC, last = min(kC, L - t0) - 1;
        copy_rows<T::RB, kC, W, 0, 1>(q0 + size_t(t0) * gn, uint32_t(gn) * kSz, last, T::RB / 16, lds0 + T::kQt);
    };
    auto fetch_main = [&](int ch, uint32_t buf) {
        fetch(ch, buf, std::integral_constant<int, 0>{});
        fetch(ch, buf, std::integral_constant<int, 1>{});
        fetch(ch, buf, std::integral_constant<int, 2>{});
        fetch(ch, buf, std::integral_constant<int, 3>{});
    };
    // dy of chunk ch, accumulator layout; 0 past the sequence
    IO ry[16];
    auto fetch_dy = [&](int ch) {
        if (!live) return;
        const int t0 = ch * kC;
        const __amdgpu_buffer_rsrc_t view = chunk_view(dyg + vy0 + size_t(t0) * hp, min(kC, L - t0), tok, P);
        const uint32_t off = uint32_t(8 * q) * tok + uint32_t(p) * kSz;
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) ry[4 * t + r] = load_checked<IO>(view, off + uint32_t(32 * (t >> 1) + 4 * (t & 1) + r) * tok);
    };
    auto dy_of = [&](int t) {
        return f32x4{to_f32<IO>(ry[4 * t]), to_f32<IO>(ry[4 * t + 1]), to_f32<IO>(ry[4 * t + 2]), to_f32<IO>(ry[4 * t + 3])};
    };
    // of the 4 token tiles this wave finishes kOwn, from its x'th on
    constexpr int kOwn = 4 / X;
    auto own = [&](const f32x4 (&a)[4], int i) {
        f32x4 v = a[i];
#pragma unroll
        for (int o = 1; o < X; ++o)
#pragma unroll
            for (int r = 0; r < 4; ++r) v[r] = x == o ? float(a[o * kOwn + i][r]) : float(v[r]);
        return v;
    };
    auto state_at = [&](int of, int t) { return (size_t(of) * P + p) * N + 32 * (n0 + (t >> 1)) + 8 * q + 4 * (t & 1); };

    f32x4 S[NT];        // dS
#pragma unroll
    for (int t = 0; t < NT; ++t) S[t] = f32x4{0.f, 0.f, 0.f, 0.f};
    const float *from = seg == segs - 1 ? d_final : MAP ? nullptr : d_enter;
    if (from && live)
#pragma unroll
        for (int t = 0; t < NT; ++t) S[t] = *reinterpret_cast<const f32x4 *>(from + state_at(seg == segs - 1 ? bh : bh * segs + seg, t));
#pragma unroll
    for (int i = 0; i < 16; ++i) ry[i] = IO(0);
    fetch_main(last, lds0);
    fetch_q(last);
    fetch_dy(last);
    copies_done();
    __syncthreads();

    for (int i = 0; i <= last - first; ++i) {
        const int ch = last - i, t0 = ch * kC, rows = min(kC, L - t0), next = max(ch - 1, first);     // past the first: that one again
        const char *buf = lds + (T::kBufs == 2 ? (i & 1) * T::kMain : 0);
        const char *tk = buf, *tq = T::kQMain ? buf + T::kRows : lds + T::kQt, *tm = buf + T::kImg + Img::kM, *ts = buf + T::kImg + Img::kQ;
        const float *gates = reinterpret_cast<const float *>(buf + T::kImg + Img::kGates);
        const size_t unit = size_t(bh) * nc + ch;
        auto ahead = [&](auto part) {
            if constexpr (T::kBufs == 2) fetch(next, lds0 + ((i + 1) & 1) * T::kMain, part);
        };
        auto gate_of = [&](int which, int t) {
            return *reinterpret_cast<const f32x4 *>(gates + which * kC + 32 * (t >> 1) + 8 * q + 4 * (t & 1));
        };
        if (!MAP && live) {
            if (ch % kSegment<IO> == kSegment<IO> - 1 || ch == nc - 1) {
                const size_t at = (size_t(bh) * ptiles + p0 / 16) * anchors + ch / kSegment<IO>;
                const f32x4 *a0 = anchor + (at * (N / 16) + x * NT) * 64 + lane;
                float dot = 0.f;
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    const f32x4 a = a0[64 * t];
                    dot += S[t][0] * a[0] + S[t][1] * a[1] + S[t][2] * a[2] + S[t][3] * a[3];
                }
                dot = wave_sum(dot);
                if (lane == 0) sums.lam[at * X + x] = dot;
            }
        }
        f32x4 dU[4], dv[4], xs[kOwn], vd[kOwn], Ev[kOwn];
        IO rv[4 * kOwn];
        if (live) {
            Op<IO, kPlanes> so[KS];
#pragma unroll
            for (int s = 0; s < KS; ++s) so[s] = to_op<IO, kPlanes>(S[2 * s], S[2 * s + 1]);
            if constexpr (!MAP) {
                float *dst = dSg + (unit * P + p) * N + 32 * n0 + 8 * q;
#pragma unroll
                for (int t = 0; t < NT; ++t) *reinterpret_cast<f32x4 *>(dst + 32 * (t >> 1) + 4 * (t & 1)) = S[t];
            }
            // this wave's part of dU = e^{g_C - g} K dS^T + scores^T dY: its columns of dS, and
            // token half x of dY (both halves with one wave, none for waves past the second)
#pragma unroll
            for (int t = 0; t < 4; ++t) dU[t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                Op<IO, 1> a[4];
#pragma unroll
                for (int t = 0; t < 4; ++t) a[t] = read_row<IO, 1, T::RB>(tk, 0, tile_row(t >> 1, t & 1, c), n0 + ks, q);
                mma(dU, a, so[ks]);
            }
#pragma unroll
            for (int t = 0; t < 4; ++t) dU[t] *= gate_of(1, t);
            if (X == 1 || x == 1) {
                Op<IO, kPlanes> a[4];
#pragma unroll
                for (int t = 0; t < 4; ++t) a[t] = tri_col<IO, kPlanes>(ts, 1, t >> 1, t & 1, c, q);
                mma(dU, a, to_op<IO, 1>(dy_of(2), dy_of(3)));
            }
            if (x == 0) {
                f32x4 upper[2] = {dU[0], dU[1]};
                Op<IO, kPlanes> a[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) a[e] = tri_col<IO, kPlanes>(ts, 0, 0, e, c, q);
                mma(upper, a, to_op<IO, 1>(dy_of(0), dy_of(1)));
                dU[0] = upper[0];
                dU[1] = upper[1];
            }
            if constexpr (X > 1)
#pragma unroll
                for (int t = 0; t < 4; ++t) reinterpret_cast<f32x4 *>(xe)[64 * t + lane] = dU[t];
        }
        if constexpr (X > 1) {
            copies_done();      // q, asked for at the chunk's beginning
            __syncthreads();    // and the parts are written
        }
        if (!MAP && live) {     // what the end of the chunk needs: E and v of this wave's token tiles
            const f32x4 *src = E + (unit * ptiles + p0 / 16) * 256 + lane;
            const __amdgpu_buffer_rsrc_t view = chunk_view(vg + vy0 + size_t(t0) * hp, rows, tok, P);
            const uint32_t off = uint32_t(8 * q) * tok + uint32_t(p) * kSz;
#pragma unroll
            for (int j = 0; j < kOwn; ++j) {
                const int t = x * kOwn + j;
                Ev[j] = src[64 * t];
#pragma unroll
                for (int r = 0; r < 4; ++r) rv[4 * j + r] = load_checked<IO>(view, off + uint32_t(32 * (t >> 1) + 4 * (t & 1) + r) * tok);
            }
        }
        ahead(std::integral_constant<int, 0>{});
        ahead(std::integral_constant<int, 1>{});
        if (live) {
            if constexpr (X > 1) sum_of_parts<X>(lds + T::kE + (w - x) * 4096, lane, dU);
            // X = dU + M^T (beta dU), in place
            const Op<IO, kPlanes> br0 = to_op<IO, kPlanes>(gate_of(2, 0) * dU[0], gate_of(2, 1) * dU[1]);
            const Op<IO, kPlanes> br1 = to_op<IO, kPlanes>(gate_of(2, 2) * dU[2], gate_of(2, 3) * dU[3]);
            {
                Op<IO, kPlanes> a[4];
#pragma unroll
                for (int t = 0; t < 4; ++t) a[t] = tri_col<IO, kPlanes>(tm, 1, t >> 1, t & 1, c, q);
                mma(dU, a, br1);
            }
            {
                f32x4 upper[2] = {dU[0], dU[1]};
                Op<IO, kPlanes> a[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) a[e] = tri_col<IO, kPlanes>(tm, 0, 0, e, c, q);
                mma(upper, a, br0);
                dU[0] = upper[0];
                dU[1] = upper[1];
            }
#pragma unroll
            for (int t = 0; t < 4; ++t) dv[t] = gate_of(2, t) * dU[t];
        }
        ahead(std::integral_constant<int, 2>{});
        ahead(std::integral_constant<int, 3>{});
        if (live) {
            // dS <- e^{g_C} dS + Q^T (scale e^g dY) - K^T (e^g dv)
            const float alpha = gates[kC - 1];
#pragma unroll
            for (int t = 0; t < NT; ++t) S[t] *= alpha;
#pragma unroll
            for (int ks = 0; ks < 2; ++ks) {
                const f32x4 f0 = gate_of(0, 2 * ks), f1 = gate_of(0, 2 * ks + 1);
                const Op<IO, kPlanes> oq = to_op<IO, kPlanes>(scale * f0 * dy_of(2 * ks), scale * f1 * dy_of(2 * ks + 1));
                const Op<IO, kPlanes> ok = to_op<IO, kPlanes>(-f0 * dv[2 * ks], -f1 * dv[2 * ks + 1]);
                if (ks == 1) fetch_dy(next);
#pragma unroll
                for (int u0 = 0; u0 < NT; u0 += 4) {
                    constexpr int M = NT < 4 ? NT : 4;
                    f32x4 z[M];
                    Op<IO, 1> a[M], b[M];
#pragma unroll
                    for (int t = 0; t < M; ++t) {
                        z[t] = S[u0 + t];
                        a[t] = read_col<IO, 1, T::RB>(tq, 0, 32 * ks, 32 * (n0 + ((u0 + t) >> 1)), t & 1, c, q);
                        b[t] = read_col<IO, 1, T::RB>(tk, 0, 32 * ks, 32 * (n0 + ((u0 + t) >> 1)), t & 1, c, q);
                    }
                    mma(z, a, oq);
                    mma(z, b, ok);
#pragma unroll
                    for (int t = 0; t < M; ++t) S[u0 + t] = z[t];
                    if constexpr (kSz == 4) __builtin_amdgcn_sched_barrier(0);     // no registers to read ahead
                }
            }
            // the sums over the 16 rows (the 16 lanes of a row group), of this wave's token tiles
#pragma unroll
            for (int j = 0; j < (MAP ? 0 : kOwn); ++j) {
                const f32x4 du = own(dU, j), dvj = own(dv, j);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    xs[j][r] = row16_sum(du[r] * Ev[j][r]);
                    vd[j][r] = row16_sum(dvj[r] * to_f32<IO>(rv[4 * j + r]));
                }
            }
        }
        if constexpr (T::kBufs == 1) {
            __syncthreads();
            if (ch > first) {
                fetch_main(ch - 1, lds0);
                fetch_q(ch - 1);
            }
        }
        copies_done();
        __syncthreads();
        if constexpr (T::kBufs == 2) fetch_q(next);     // this chunk's is read
        if (!MAP && live) {
            const size_t at = (unit * ptiles + p0 / 16) * kC + 8 * q;
            const __amdgpu_buffer_rsrc_t view = chunk_view(dvg + vy0 + size_t(t0) * hp, rows, tok, P);
            const uint32_t off = uint32_t(8 * q) * tok + uint32_t(p) * kSz;
#pragma unroll
            for (int j = 0; j < kOwn; ++j) {
                const int t = x * kOwn + j, row = 32 * (t >> 1) + 4 * (t & 1);
                const f32x4 dvj = own(dv, j);
                Xg[(unit * ptiles + p0 / 16) * 256 + 64 * t + lane] = own(dU, j);
                if (c == 0) {
                    *reinterpret_cast<f32x4 *>(sums.xe + at + row) = xs[j];
                    *reinterpret_cast<f32x4 *>(sums.vdv + at + row) = vd[j];
                }
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int o = int(off + uint32_t(row + r) * tok);
                    if constexpr (kSz == 4) __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(dvj[r]), view, o, 0, 0);
                    else __builtin_amdgcn_raw_buffer_store_b16(f32_to_bf16(dvj[r]), view, o, 0, 0);
                }
            }
        }
    }
    copies_done();      // of the last chunk's q, asked for once more
    if (d_out && live && (MAP || seg == 0))
#pragma unroll
        for (int t = 0; t < NT; ++t) *reinterpret_cast<f32x4 *>(d_out + state_at(MAP ? bh * segs + seg : bh, t)) = S[t];
}

// Kernel 4.  Block = (batch, chunk, group, one of `splits` parts of its heads' state rows).
// Wave w holds dq^T and dk^T of 16 tokens (tile columns; rows n in registers, 4 consecutive
// ones a tile), of one half of the N's: waves w and w + 4 share their tokens.  Per turn a
// head's 32 rows p: dY, dv, U and both states go through LDS, 32-bit ones split into kPlanes
// planes on the way there; the next turn's values are on their way into registers meanwhile.
template <typename IO, int N>
struct GradTile {
    static constexpr int kSz = int(sizeof(IO)), kP = kSz == 4 ? 1 : kPlanes;
    static constexpr int kRows = 32;                        // state rows a turn
    static constexpr int RP = kRows * kSz, RB = N * kSz;    // bytes per row of p's / of N
    static constexpr int kTok = kC * RP, kState = kRows * RB;       // bytes of a [64][32] / [32][N] tile
    static constexpr int kS = 0, kD = kP * kState, kU = 2 * kP * kState, kV = kU + kP * kTok, kY = kV + kP * kTok, kHead = kY + kTok;
    // after the heads: W and G (kP planes each), k, q
    static constexpr int RM = kC * kSz, kMat = kC * RM, kWm = 0, kGm = kP * kMat, kK = 2 * kP * kMat, kQ = kK + kC * RB, kTail = kQ + kC * RB;
    static constexpr int kLds = kHead > kTail ? kHead : kTail;
    static constexpr int kThreads = 512, kEights = kRows * N / 8, kLoads = (kEights + kThreads - 1) / kThreads;     // 8 values a thread and load
    static constexpr bool kTight = RB >= 512;       // as many accumulators as leave few registers
    static constexpr bool kAhead = N <= 128;        // a turn's values are asked for a turn ahead
    static_assert(kLds <= 159 * 1024);
};

template <typename IO, int N>
__global__ __launch_bounds__(512) void k_delta_grads(const IO *__restrict__ qg, const IO *__restrict__ kg,
                                                     const float *__restrict__ ag, const IO *__restrict__ dyg,
                                                     const char *__restrict__ images, const f32x4 *__restrict__ E,
                                                     const f32x4 *__restrict__ Xg, const float *__restrict__ Sg,
                                                     const float *__restrict__ dSg, IO *__restrict__ dqg, IO *__restrict__ dkg,
                                                     float *__restrict__ parts, int splits, int L, int H, int P, int G, int nc,
                                                     float scale) {
    using T = GradTile<IO, N>;
    using Img = ChunkImage<IO>;
    constexpr int kSz = T::kSz, kP = T::kP, NT = N / 32;    // column tiles of a wave
    extern __shared__ __align__(16) char lds[];
    __shared__ double gd[kC];
    const uint32_t lds0 = lds_address(lds);
    const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6), c = lane & 15, q = lane >> 4;
    const int split = blockIdx.x % splits, cell = blockIdx.x / splits, ch = cell % nc, bg = cell / nc, g = bg % G, bi = bg / G, r = H / G;
    const int t0 = ch * kC, rows = min(kC, L - t0), ptiles = P / 16;
    const size_t hp = size_t(H) * P, gn = size_t(G) * N;
    const int tw = w & 3, half = w >> 2, tok = tile_row(tw >> 1, tw & 1, c);    // this lane's token
    auto column = [&](int i) { return half * NT + i; };     // tile i of this wave, of the N / 16

    f32x4 dq[NT], dk[NT], Wm[2], Fm[2];
#pragma unroll
    for (int i = 0; i < NT; ++i) dq[i] = dk[i] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int e = 0; e < 2; ++e) Wm[e] = Fm[e] = f32x4{0.f, 0.f, 0.f, 0.f};

    const int pbs = (P + T::kRows - 1) / T::kRows, turns = r * pbs;
    const int first = int(int64_t(turns) * split / splits), end = int(int64_t(turns) * (split + 1) / splits);
    // one turn's values, as loaded: rows and tokens past the end are zeros
    struct {
        f32x4 s[T::kLoads][2], d[T::kLoads][2], e, x, bt;
        u32x4 y;
        float a, fs, te;
    } in;
    auto fetch = [&](int turn) {
        const int h = g * r + turn / pbs, pb = turn % pbs * T::kRows;
        const size_t unit = (size_t(bi) * H + h) * nc + ch;
        const float *gates = reinterpret_cast<const float *>(images + unit * Img::kBytes + Img::kGates);
        const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < T::kLoads; ++i) {
            const int u = i * T::kThreads + tid, row = u / (N / 8);
            const bool on = u < T::kEights && pb + row < P;
            const size_t at = (unit * P + pb + (on ? row : 0)) * N + u % (N / 8) * 8;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                in.s[i][e] = on ? *reinterpret_cast<const f32x4 *>(Sg + at + 4 * e) : zero;
                in.d[i][e] = on ? *reinterpret_cast<const f32x4 *>(dSg + at + 4 * e) : zero;
            }
        }
        // E and X: a chain wave's tile of 16 p's is 256 pieces, (tid & 255) >> 6 the token tile
        const int pt = pb / 16 + (tid >> 8), t = (tid >> 6) & 3;
        const size_t piece = (unit * ptiles + min(pt, ptiles - 1)) * 256 + (tid & 255);
        in.e = pt < ptiles ? E[piece] : zero;
        in.x = pt < ptiles ? Xg[piece] : zero;
        in.bt = *reinterpret_cast<const f32x4 *>(gates + 2 * kC + 32 * (t >> 1) + 8 * q + 4 * (t & 1));
        constexpr int kPer = T::RP / 16;        // 16-byte pieces of a token's row of dY
        const int ty = tid / kPer, py = pb + tid % kPer * (16 / kSz);
        const bool on = ty < rows && py < P;
        const IO *src = dyg + (size_t(bi) * L + t0 + (on ? ty : 0)) * hp + size_t(h) * P + (on ? py : 0);
        in.y = on ? *reinterpret_cast<const u32x4 *>(src) : u32x4{0, 0, 0, 0};
        in.a = lane < rows ? ag[(size_t(bi) * L + t0 + min(lane, rows - 1)) * H + h] : 0.f;
        in.fs = gates[tok];
        in.te = gates[kC + tok];
    };
    auto put = [&](char *tile, int stride, int row_bytes, int place_, int row, int col, float v) {
        char *dst = tile + row * row_bytes + (((col * kSz >> 4) ^ place_) << 4) + (col * kSz & 15);
        if constexpr (kSz == 4) {
            *reinterpret_cast<float *>(dst) = v;
        } else {
#pragma unroll
            for (int p = 0; p < kP; ++p) {
                const bf16_bits part = f32_to_bf16(v);
                *reinterpret_cast<bf16_bits *>(dst + p * stride) = part;
                v -= bf16_to_f32(part);
            }
        }
    };
    auto put_state = [&](char *tile, int row, int eight, const f32x4 (&v)[2]) {
        if constexpr (kSz == 4) {
#pragma unroll
            for (int e = 0; e < 2; ++e) *reinterpret_cast<f32x4 *>(tile + row * T::RB + (((2 * eight + e) ^ place<T::RB>(row)) * 16)) = v[e];
        } else {
            const Op<IO, kP> o = to_op<IO, kP>(v[0], v[1]);
#pragma unroll
            for (int p = 0; p < kP; ++p)
                *reinterpret_cast<uint4 *>(tile + p * T::kState + row * T::RB + ((eight ^ place<T::RB>(row)) * 16)) = __builtin_bit_cast(uint4, o.p[p]);
        }
    };
    float D[2][4] = {};         // decays from token j = 32 half + 8 q + 4 e + i to this lane's
    if (T::kAhead && first < end) fetch(first);
    for (int turn = first; turn < end; ++turn) {    // head h, rows pb .. pb + 31 of its state
        const bool new_head = turn == first || turn % pbs == 0;
        if constexpr (!T::kAhead) fetch(turn);
        const float fs = in.fs, te = in.te;
        __syncthreads();        // the tiles' last readers
        // a thread number the compiler does not know: addresses are formed here again rather
        // than kept over the turns, for which there may not be the registers
        int tid = threadIdx.x;
        if constexpr (T::kTight) asm volatile("" : "+v"(tid));
        const int lane = tid & 63, c = lane & 15, q = lane >> 4, tok = tile_row(tw >> 1, tw & 1, c);
        if (new_head && w == 0) {
            double s = lane < rows ? gate(in.a) : 0.0;
#pragma unroll
            for (int off = 1; off < 64; off <<= 1) {
                const double o = __shfl_up(s, off, 64);
                if (lane >= off) s += o;
            }
            gd[lane] = s;
        }
#pragma unroll
        for (int i = 0; i < T::kLoads; ++i) {
            const int u = i * T::kThreads + tid;
            if (u >= T::kEights) break;
            put_state(lds + T::kS, u / (N / 8), u % (N / 8), in.s[i]);
            put_state(lds + T::kD, u / (N / 8), u % (N / 8), in.d[i]);
            if constexpr (T::kTight) __builtin_amdgcn_sched_barrier(0);
        }
        {
            const int t = (tid >> 6) & 3, col = 16 * (tid >> 8) + c;
            const f32x4 u = in.bt * in.e, v = in.bt * in.x;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int row = 32 * (t >> 1) + 8 * q + 4 * (t & 1) + j;
                put(lds + T::kU, T::kTok, T::RP, place<T::RP>(row), row, col, u[j]);
                put(lds + T::kV, T::kTok, T::RP, place<T::RP>(row), row, col, v[j]);
                if constexpr (T::kTight) __builtin_amdgcn_sched_barrier(0);
            }
            constexpr int kPer = T::RP / 16;
            if (const int row = tid / kPer; row < kC)
                *reinterpret_cast<u32x4 *>(lds + T::kY + row * T::RP + (((tid % kPer) ^ place<T::RP>(row)) * 16)) = in.y;
        }
        if constexpr (T::kAhead) fetch(min(turn + 1, end - 1));
        __syncthreads();
        if (new_head) {
            const double gt = gd[tok];
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int j = 32 * half + 8 * q + 4 * e + i;
                    D[e][i] = expf(j <= tok ? float(gt - gd[j]) : 0.f);
                }
        }
        // the states' parts
        const Op<IO, 1> oy = read_row<IO, 1, T::RP>(lds + T::kY, 0, tok, 0, q);
        const Op<IO, kP> ov = read_row<IO, kP, T::RP>(lds + T::kV, T::kTok, tok, 0, q), ou = read_row<IO, kP, T::RP>(lds + T::kU, T::kTok, tok, 0, q);
        constexpr int M = NT < 2 || T::kTight ? 1 : 2;
#pragma unroll
        for (int i0 = 0; i0 < NT; i0 += M) {
            Op<IO, kP> as[M], ad[M];
            f32x4 zq[M], zv[M], zu[M];
#pragma unroll
            for (int i = 0; i < M; ++i) {
                const int t = column(i0 + i);
                as[i] = read_col<IO, kP, T::RB>(lds + T::kS, T::kState, 0, 32 * (t >> 1), t & 1, c, q);
                ad[i] = read_col<IO, kP, T::RB>(lds + T::kD, T::kState, 0, 32 * (t >> 1), t & 1, c, q);
                zq[i] = zv[i] = zu[i] = f32x4{0.f, 0.f, 0.f, 0.f};
            }
            mma(zq, as, oy);
            mma(zv, as, ov);
            mma(zu, ad, ou);
#pragma unroll
            for (int i = 0; i < M; ++i) {
                dq[i0 + i] += (scale * fs) * zq[i];
                dk[i0 + i] += te * zu[i] - fs * zv[i];
            }
            if constexpr (T::kTight) __builtin_amdgcn_sched_barrier(0);     // no registers to read ahead
        }
        // dY U^T and dv U^T (rows j, columns i: this lane's token), where some j <= i
        if (half <= (tw >> 1)) {
            Op<IO, kP> au[2];
            f32x4 zw[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}}, zf[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
            for (int e = 0; e < 2; ++e) au[e] = read_row<IO, kP, T::RP>(lds + T::kU, T::kTok, tile_row(half, e, c), 0, q);
            mma(zw, au, oy);
            mma(zf, au, ov);
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int j = 32 * half + 8 * q + 4 * e + i;
                    const float wv = scale * D[e][i] * zw[e][i], fv = -D[e][i] * zf[e][i];
                    Wm[e][i] += j <= tok && tok < rows ? wv : 0.f;
                    Fm[e][i] += j < tok && tok < rows ? fv : 0.f;
                }
        }
    }
    __syncthreads();
    // k and q into LDS, W [i][j] and G [i][j] = G [j][i] beside them
    const size_t src = (size_t(bi) * L + t0) * gn + size_t(g) * N;
    constexpr int kCopiers = kC * T::RB >= 8 * 1024 ? 8 : 4;    // waves: 1 KiB each at least
    if (w < kCopiers) {
        copy_rows<T::RB, kC, kCopiers, 0, 1>(kg + src, uint32_t(gn) * kSz, rows - 1, T::RB / 16, lds0 + T::kK);
        copy_rows<T::RB, kC, kCopiers, 0, 1>(qg + src, uint32_t(gn) * kSz, rows - 1, T::RB / 16, lds0 + T::kQ);
    }
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int j = 32 * half + 8 * q + 4 * e + i;
            put(lds + T::kWm, T::kMat, T::RM, place<T::RM>(tok), tok, j, Wm[e][i]);     // 0 above the diagonal
            if (j < tok) {
                put(lds + T::kGm, T::kMat, T::RM, place<T::RM>(tok), tok, j, Fm[e][i]);
                put(lds + T::kGm, T::kMat, T::RM, place<T::RM>(j), j, tok, Fm[e][i]);
            } else if (j == tok) {
                put(lds + T::kGm, T::kMat, T::RM, place<T::RM>(j), j, j, 0.f);
            }
        }
    copies_done();
    __syncthreads();
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
        int l = lane;
        if constexpr (T::kTight) asm volatile("" : "+v"(l));
        const int c = l & 15, q = l >> 4, tok = tile_row(tw >> 1, tw & 1, c);
        const Op<IO, kP> wr = read_row<IO, kP, T::RM>(lds + T::kWm, T::kMat, tok, ks, q);
        const Op<IO, kP> gr = read_row<IO, kP, T::RM>(lds + T::kGm, T::kMat, tok, ks, q);
        const Op<IO, kP> wc = read_col<IO, kP, T::RM>(lds + T::kWm, T::kMat, 32 * ks, 32 * (tw >> 1), tw & 1, c, q);
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            const int t = column(i);
            const Op<IO, 1> ak[1] = {read_col<IO, 1, T::RB>(lds + T::kK, 0, 32 * ks, 32 * (t >> 1), t & 1, c, q)};
            const Op<IO, 1> aq[1] = {read_col<IO, 1, T::RB>(lds + T::kQ, 0, 32 * ks, 32 * (t >> 1), t & 1, c, q)};
            f32x4 z[1] = {dq[i]};
            mma(z, ak, wr);
            dq[i] = z[0];
            z[0] = dk[i];
            mma(z, ak, gr);
            mma(z, aq, wc);
            dk[i] = z[0];
            if constexpr (T::kTight) __builtin_amdgcn_sched_barrier(0);
        }
    }
    if (tok < rows) {
        const size_t dst = (size_t(bi) * L + t0 + tok) * gn + size_t(g) * N + 8 * q;
        const size_t all = size_t(gridDim.x / (splits * nc * G)) * L * gn;
        float *pq = parts + 2 * split * all + dst, *pk = pq + all;
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            const int at = 32 * (column(i) >> 1) + 4 * (column(i) & 1);
            if (splits > 1) {
                *reinterpret_cast<f32x4 *>(pq + at) = dq[i];
                *reinterpret_cast<f32x4 *>(pk + at) = dk[i];
            } else {
                *reinterpret_cast<Raw4<IO> *>(dqg + dst + at) = narrow<IO>(dq[i]);
                *reinterpret_cast<Raw4<IO> *>(dkg + dst + at) = narrow<IO>(dk[i]);
            }
        }
    }
}

// The parts of dq and dk added in their order: parts [splits][dq, dk][all] fp32, 8 elements
// per thread.
template <typename IO>
__global__ __launch_bounds__(256) void k_delta_join(const float *__restrict__ parts, IO *__restrict__ dqg, IO *__restrict__ dkg,
                                                    int splits, size_t all) {
    const size_t at = (size_t(blockIdx.x) * 256 + threadIdx.x) * 8;
    if (at >= 2 * all) return;
    f32x4 s0 = {0.f, 0.f, 0.f, 0.f}, s1 = s0;
    for (int i = 0; i < splits; ++i) {
        const float *p = parts + 2 * i * all + at;
        s0 += *reinterpret_cast<const f32x4 *>(p);
        s1 += *reinterpret_cast<const f32x4 *>(p + 4);
    }
    IO *dst = at < all ? dqg + at : dkg + (at - all);
    if constexpr (sizeof(IO) == 4) {
        *reinterpret_cast<f32x4 *>(dst) = s0;
        *reinterpret_cast<f32x4 *>(dst + 4) = s1;
    } else {
        *reinterpret_cast<bf16x8 *>(dst) = to_op<IO, 1>(s0, s1).p[0];
    }
}

// Kernel 5.  Block = (batch, head, segment), one wave per chunk of it, lane = token.  The
// sum from a token to the segment's end is taken in 64 bits: it is the sum of up to 128
// terms that largely cancel.
template <int SEG>
__global__ __launch_bounds__(64 * SEG) void k_delta_gates(const float *__restrict__ ydy, const float *__restrict__ vdv,
                                                               const float *__restrict__ xe, const float *__restrict__ lam,
                                                               float *__restrict__ da, float *__restrict__ dbeta, int L, int H,
                                                               int nc, int ptiles, int segs, int parts) {
    __shared__ double total[SEG];
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    const int seg = blockIdx.x % segs, bh = blockIdx.x / segs, h = bh % H, bi = bh / H;
    const int ch = seg * SEG + w, t = ch * kC + lane;
    double d = 0.0;
    float b = 0.f;
    if (ch < nc) {
        const size_t unit = size_t(bh) * nc + ch, at = unit * ptiles * kC + lane;
        const float *y = ydy + unit * parts * ptiles * kC + lane;
#pragma unroll 8
        for (int i = 0; i < parts * ptiles; ++i) d += double(y[i * kC]);
#pragma unroll 8
        for (int i = 0; i < ptiles; ++i) {
            d -= double(vdv[at + i * kC]);
            b += xe[at + i * kC];
        }
    }
    if (t >= L) d = 0.0;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
        const double o = __shfl_down(d, off, 64);
        if (lane + off < 64) d += o;
    }
    if (lane == 0) total[w] = d;
    __syncthreads();
    for (int i = w + 1; i < SEG; ++i) d += total[i];
    double dot = 0.0;       // <dS, S>, lane i one part of it
    for (int i = lane; i < ptiles * parts; i += 64) dot += double(lam[((size_t(bh) * ptiles + i / parts) * segs + seg) * parts + i % parts]);
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) dot += __shfl_xor(dot, off, 64);
    d += dot;
    if (ch < nc && t < L) {
        const size_t at = (size_t(bi) * L + t) * H + h;
        da[at] = float(d);
        dbeta[at] = b;
    }
}

template <typename IO, int N>
hipError_t launch_n(const DeltaBwdArgs &a, const DeltaBwdPlan &pl, hipStream_t stream) {
    const int nc = (a.L + kC - 1) / kC, segs = (nc + kSegment<IO> - 1) / kSegment<IO>, ptiles = a.P / 16;
    char *ws = static_cast<char *>(a.workspace);
    char *images = ws;
    const auto *q = static_cast<const IO *>(a.q), *k = static_cast<const IO *>(a.k), *v = static_cast<const IO *>(a.v);
    const auto *dy = static_cast<const IO *>(a.dy);
    auto *dv = static_cast<IO *>(a.dv);
    DeltaSaved saved{reinterpret_cast<float *>(ws + pl.off_e), reinterpret_cast<float *>(ws + pl.off_s), reinterpret_cast<float *>(ws + pl.off_anchor),
                     reinterpret_cast<float *>(ws + pl.off_ydy)};
    BackSums sums{reinterpret_cast<float *>(ws + pl.off_xe), reinterpret_cast<float *>(ws + pl.off_vdv), reinterpret_cast<float *>(ws + pl.off_lam)};
    auto *dS = reinterpret_cast<float *>(ws + pl.off_ds);
    auto *kept_x = reinterpret_cast<f32x4 *>(ws + pl.off_x);
    auto *parts = reinterpret_cast<float *>(ws + pl.off_parts);

    hipError_t e = launch_delta_prep<IO, N>(q, k, a.a, a.beta, images, a.b, a.L, a.H, a.G, a.scale, stream);
    if (e != hipSuccess) return e;
    auto *map = reinterpret_cast<float *>(ws + pl.off_map), *init = reinterpret_cast<float *>(ws + pl.off_init);
    auto *dmap = reinterpret_cast<float *>(ws + pl.off_dmap), *dinit = reinterpret_cast<float *>(ws + pl.off_dinit);
    const DeltaCut &cut = pl.cut;
    e = enter_segments<IO, N, true>(q, k, v, images, a.init_state, map, init, a.b, a.L, a.H, a.P, a.G, cut, a.scale, stream);
    if (e != hipSuccess) return e;
    auto back = [&](auto w_, auto x_, auto one_, auto map_, float *to) {
        constexpr int W = decltype(w_)::value, X = decltype(x_)::value;
        constexpr bool MAP = decltype(map_)::value, ONE = decltype(one_)::value;
        constexpr int lds = ChainLds<IO, N, W, X, false, ONE>::kBytes;
        const int rows = 16 * W / X, pblocks = (a.P + rows - 1) / rows;
        auto kern = k_delta_chain_back<IO, N, W, X, MAP, ONE>;
        e = hipFuncSetAttribute(reinterpret_cast<const void *>(kern), hipFuncAttributeMaxDynamicSharedMemorySize, lds);
        if (e != hipSuccess) return e;
        hipLaunchKernelGGL(kern, dim3(unsigned(int64_t(a.b) * a.H * (cut.segments - (MAP ? 1 : 0)) * pblocks)), dim3(64 * W), lds, stream, q, k,
                           v, dy, images, a.d_final, dinit, reinterpret_cast<const f32x4 *>(saved.E),
                           reinterpret_cast<const f32x4 *>(saved.anchor), dv, dS, kept_x, to, sums, a.L, a.H, a.P, a.G, nc, cut.per, cut.segments,
                           pblocks, a.scale);
        return hipGetLastError();
    };
    const int64_t tiles = int64_t(a.b) * a.H * ptiles;
    if (cut.segments > 1) {
        auto go = [&](auto w, auto x, auto one) { return back(w, x, one, std::true_type{}, dmap); };
        if ((e = with_chain_shape<IO, N, true>(tiles * (cut.segments - 1), go)) != hipSuccess) return e;
        hipLaunchKernelGGL((k_delta_carry<N, true>), dim3(unsigned(tiles)), dim3(4 * N), 0, stream, map, dmap, nullptr, dinit, a.P, cut.segments);
        if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    int share = 1;      // waves per tile, each with its own part of the sums
    auto chains = [&](auto w_, auto x_, auto one_) {
        constexpr int W = decltype(w_)::value, X = decltype(x_)::value;
        share = X;
        e = launch_chain<IO, N, W, X, Chain::save, decltype(one_)::value>(q, k, v, images, cut.segments > 1 ? init : a.init_state, nullptr, nullptr, dy, saved,
                                                           a.b, a.L, a.H, a.P, a.G, cut.per, cut.segments, a.scale, stream);
        return e != hipSuccess ? e : back(w_, x_, one_, std::false_type{}, a.d_init);
    };
    if ((e = with_chain_shape<IO, N, true>(tiles * cut.segments, chains)) != hipSuccess) return e;
    auto grads = k_delta_grads<IO, N>;
    constexpr int lds = GradTile<IO, N>::kLds;
    e = hipFuncSetAttribute(reinterpret_cast<const void *>(grads), hipFuncAttributeMaxDynamicSharedMemorySize, lds);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(grads, dim3(unsigned(int64_t(a.b) * a.G * nc * pl.splits)), dim3(GradTile<IO, N>::kThreads), lds, stream, q, k, a.a, dy, images,
                       reinterpret_cast<const f32x4 *>(saved.E), kept_x, saved.S, dS, static_cast<IO *>(a.dq),
                       static_cast<IO *>(a.dk), parts, pl.splits, a.L, a.H, a.P, a.G, nc, a.scale);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    if (pl.splits > 1) {
        const size_t all = size_t(a.b) * a.L * a.G * N;
        hipLaunchKernelGGL(k_delta_join<IO>, dim3(unsigned((2 * all + 2047) / 2048)), dim3(256), 0, stream, parts,
                           static_cast<IO *>(a.dq), static_cast<IO *>(a.dk), pl.splits, all);
        if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    hipLaunchKernelGGL((k_delta_gates<kSegment<IO>>), dim3(unsigned(int64_t(a.b) * a.H * segs)), dim3(64 * kSegment<IO>), 0, stream, saved.ydy, sums.vdv, sums.xe,
                       sums.lam, a.da, a.dbeta, a.L, a.H, nc, ptiles, segs, share);
    return hipGetLastError();
}

// Parts to split a group's `turns` (of up to 32 state rows) into, where the chunks alone
// leave CUs idle: as many as give each CU a block.
int grad_splits(size_t cells, size_t turns) { return int(std::max<size_t>(1, std::min(turns, 256 / cells))); }

}  // namespace

DeltaBwdPlan plan_delta_bwd(int b, int L, int H, int P, int N, int G, bool bf16) {
    DeltaBwdPlan pl;
    if (b <= 0 || L <= 0 || !delta_chunk_supported(b, L, H, P, N, G, bf16)) return pl;
    const size_t nc = (size_t(L) + kC - 1) / kC, segs = bf16 ? (nc + kSegment<bf16_bits> - 1) / kSegment<bf16_bits> : (nc + kSegment<float> - 1) / kSegment<float>, bh = size_t(b) * H, units = bh * nc;
    const size_t state = size_t(P) * N, ptiles = size_t(P) / 16;
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t off = at;
        at += (bytes + 255) / 256 * 256;
        return off;
    };
    take(units * (bf16 ? ChunkImage<bf16_bits>::kBytes : ChunkImage<float>::kBytes));
    pl.off_e = take(units * kC * P * 4);
    pl.off_x = take(units * kC * P * 4);
    pl.off_s = take(units * state * 4);
    pl.off_ds = take(units * state * 4);
    pl.off_anchor = take(bh * segs * state * 4);
    pl.off_ydy = take(units * kMaxShare * ptiles * kC * 4);
    pl.off_xe = take(units * ptiles * kC * 4);
    pl.off_vdv = take(units * ptiles * kC * 4);
    pl.off_lam = take(bh * ptiles * segs * kMaxShare * 4);
    pl.splits = grad_splits(size_t(b) * G * nc, size_t(H / G) * ((P + 31) / 32));
    pl.cut = cut_sequence(int64_t(bh), int(nc), P, N, bf16, true);
    pl.off_map = take(map_bytes(bh, P, N, pl.cut));
    pl.off_init = take(entering_bytes(bh, P, N, pl.cut));
    pl.off_dmap = take(entering_bytes(bh, P, N, pl.cut));
    pl.off_dinit = take(entering_bytes(bh, P, N, pl.cut));
    pl.off_parts = take(pl.splits > 1 ? size_t(pl.splits) * 2 * b * L * G * N * 4 : 0);
    pl.total = at;
    pl.supported = true;
    return pl;
}

hipError_t launch_delta_bwd(const DeltaBwdArgs &a, const DeltaBwdPlan &pl, hipStream_t stream) {
    switch (a.N) {
        case 32: return a.bf16 ? launch_n<bf16_bits, 32>(a, pl, stream) : launch_n<float, 32>(a, pl, stream);
        case 64: return a.bf16 ? launch_n<bf16_bits, 64>(a, pl, stream) : launch_n<float, 64>(a, pl, stream);
        case 128: return a.bf16 ? launch_n<bf16_bits, 128>(a, pl, stream) : launch_n<float, 128>(a, pl, stream);
        case 256: return a.bf16 ? launch_n<bf16_bits, 256>(a, pl, stream) : hipErrorInvalidValue;
        default: return hipErrorInvalidValue;
    }
}

}  // namespace ssd
