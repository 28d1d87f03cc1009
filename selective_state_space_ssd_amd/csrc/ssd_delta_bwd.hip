// ssd_delta_bwd.hip -- gradients of the gated delta rule, in chunks of 64 tokens (formulas,
// names and tile layout of the forward pass: ssd_delta_chunk.h).
//
// Nothing is kept from the forward pass; four kernels:
//   1 prep       M and the scores of every chunk (ssd_delta_prep.h)
//   2 chain      forward over the chunks: E and the entering states (ssd_delta_chain.h)
//   3 chain back from d_final, with dS the gradient of the state a chunk leaves:
//        dU = scores^T dY + e^{g_C - g} (K dS^T),   X = dU + M^T (beta dU)
//        dv = beta X
//        dS <- e^{g_C} dS + (scale e^g dY)^T Q - (e^g dv)^T K
//   4 grads      per chunk; dq and dk are sums over a group's heads, taken in one block, or
//                in a few whose fp32 sums a further kernel adds:
//        dq = scale e^g dY S + W K,                      W_ij = scale (dy_i . u_j) D_ij, j <= i
//        dk = -e^g dv S + e^{g_C - g} U dS + W^T Q + G K,  G = F + F^T, F_ij = -(dv_i . u_j) D_ij, j < i
//      Both are differences where the chunk's updates erase a large state, or the gradient of
//      one: states, U, dv, W and G keep 32 bits here too, and dq and dk are rounded once.
//        dbeta_i = X_i . E_i
//      da_t is the sum of what passes the gate of token t: from tokens j < t to i >= t in the
//      chunk, from the entering state to i >= t, from j < t to the leaving state, and from
//      state to state.  Every such term holds e^{a_t}.  (The difference y . dy - v . dv summed
//      over the tokens from t on is the same number, with fewer products, but its terms do
//      not shrink with the gate: with a = -8 it was off by 2e-3 of da, with -16 by 3 times da.)
// 2 and 3 are chains over the chunks whose waves keep 16 rows of the state each, as in the
// forward pass: 32-bit values throughout.
//
// 4 x 2048 tokens, 32 heads of 128 x 128, bf16: 710 us a call; in calls back to back prep
// 46, chain 150, chain back 218, grads 300 (under a trace 46, 161, 231, 368).  The chains
// are bound by a wave's steps (ssd_delta_chain.h) and write 805 MB (both states, E and X,
// in 32 bits).  grads reads 870 MB at 2.9 TB/s, for which it is not waiting (every state
// from the caches: 265): a wave issues vector instructions 22 % of the time (a third of
// them splits values into planes), its SIMD's matrix unit is busy 23 %, and two waves a
// SIMD, all that the registers allow, leave gaps at LDS reads, barriers and the ends of
// heads (a head's gates take 30 us of the 300, a block's beginning and end 35).  With the
// states' planes in LDS, shared by all waves, it is the same time.
#include <algorithm>

#include "ssd_delta.h"
#include "ssd_delta_chain.h"
#include "ssd_delta_prep.h"

namespace ssd {
namespace {

// Kernel 3.  Waves, tiles and LDS as in the forward chain; dy is read by every wave.  One
// chain per (batch, head, segment of `per` chunks).  What leaves the last segment is d_final,
// what leaves the others is in `d_enter`.  MAP: of the segments 1 .. segs - 1, only the
// gradient of the state that enters each, into d_out [segs], with 0 for what leaves the
// others; the forward maps tell what d_enter adds to it.
template <typename IO, int N, int W, int X, bool MAP, bool ONE>
__global__ __launch_bounds__(64 * W) void k_delta_chain_back(const IO *__restrict__ qg, const IO *__restrict__ kg,
                                                             const IO *__restrict__ dyg, const char *__restrict__ images,
                                                             const float *__restrict__ d_final, const float *__restrict__ d_enter,
                                                             IO *__restrict__ dvg, float *__restrict__ dSg, f32x4 *__restrict__ Xg,
                                                             float *__restrict__ d_out, int L, int H, int P, int G, int nc, int per,
                                                             int segs, int pblocks, float scale) {
    using T = ChainLds<IO, N, W, X, true, false, ONE>;
    using Img = typename T::Img;
    extern __shared__ __align__(16) char lds[];
    constexpr int kSz = int(sizeof(IO)), KS = N / 32 / X, NT = 2 * KS;
    const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6), c = lane & 15, q = lane >> 4;
    const int x = w % X, n0 = x * KS;
    const int blk = xcd_neighbours(), pb = blk % pblocks, chain = blk / pblocks, skip = MAP ? 1 : 0;
    const int seg = chain % (segs - skip) + skip, bh = chain / (segs - skip), first = seg * per, last = min(first + per, nc) - 1;
    const int h = bh % H, bi = bh / H, g = h / (H / G);
    const int p0 = (pb * (W / X) + w / X) * 16, p = p0 + c, ptiles = P / 16;
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
        f32x4 dU[4], dv[4];
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
            const __amdgpu_buffer_rsrc_t view = chunk_view(dvg + vy0 + size_t(t0) * hp, rows, tok, P);
            const uint32_t off = uint32_t(8 * q) * tok + uint32_t(p) * kSz;
#pragma unroll
            for (int j = 0; j < kOwn; ++j) {
                const int t = x * kOwn + j, row = 32 * (t >> 1) + 4 * (t & 1);
                const f32x4 dvj = own(dv, j);
                Xg[(unit * ptiles + p0 / 16) * 256 + 64 * t + lane] = own(dU, j);
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

// Kernel 4.  Block = (batch, chunk, group, one of `splits` parts of its heads' state rows, NB
// of the N columns: more have no room in registers).  A turn takes 32 rows p of a head's
// state.  The states are operands as loaded: wave w holds 16 of the columns, of 16 NTT tokens
// dq^T and dk^T (rows n in registers, 4 consecutive ones; tile columns the tokens), and
// splits its part of S and dS into planes in registers, once for all its tokens.  dY, E and X
// go through LDS, the next turn's while this one is computed: one barrier a turn.
template <typename IO, int N>
struct GradTile {
    static constexpr int kSz = int(sizeof(IO)), kP = kSz == 4 ? 1 : kPlanes;
    static constexpr int kThreads = 512, kRows = 32;        // state rows a turn
    static constexpr int NB = N * kSz > 256 ? 256 / kSz : N, kCols = N / NB;
    static constexpr int CT = NB / 16, TH = 8 / CT, NTT = 4 / TH;           // column tiles, waves that share one, token tiles of each
    static constexpr int RT = kC * kSz, RP = kRows * kSz, RB = NB * kSz;    // bytes per row of tokens / of p's / of columns
    static constexpr int kTok = kRows * RT;                 // bytes of a tile of tokens
    // of a turn: E, X [32][64] (kP planes each); dY [64][32]; e^g, e^{g_C - g} and beta.  Two of them
    static constexpr int kE = 0, kV = kP * kTok, kY = 2 * kP * kTok, kGates = kY + kTok, kTurn = kGates + 1024;
    // after the heads, over them: W and F [64][64] (kP planes each); beside them k, q [64][NB]
    static constexpr int kMat = kC * RT, kWm = 0, kFm = kP * kMat, kTail = 2 * kP * kMat;
    static constexpr int kK = 2 * kTurn > kTail ? 2 * kTurn : kTail, kQ = kK + kC * RB, kEnd = kQ + kC * RB;
    // W and F, summed over the heads so far, as the 6 waves hold them that have any; the gates'
    // part: sums down T's columns [8][64]; A, B [CT][64], X . E [2][64].  T [64][65] lies over the
    // head's last turn.
    static constexpr int kW = kEnd, kSums = kW + 6 * 4096, kA = kSums + 8 * kC * 4, kB = kA + CT * kC * 4, kX = kB + CT * kC * 4;
    static constexpr int kLds = kX + 2 * kC * 4, LT = kC + 1;
    static_assert(kC * LT * 4 <= kGates && kLds <= 159 * 1024);
};

// Portions of a head's state rows that different blocks take, where a group's turns are split:
// block s takes the turns turns * s / splits .. turns * (s + 1) / splits - 1.
__host__ __device__ __forceinline__ int split_of(int64_t turn, int64_t turns, int splits) { return int(((turn + 1) * splits - 1) / turns); }

template <typename IO, int N>
__global__ __launch_bounds__(512) void k_delta_grads(const IO *__restrict__ qg, const IO *__restrict__ kg,
                                                     const float *__restrict__ ag, const IO *__restrict__ dyg,
                                                     const char *__restrict__ images, const f32x4 *__restrict__ E,
                                                     const f32x4 *__restrict__ Xg, const float *__restrict__ Sg,
                                                     const float *__restrict__ dSg, IO *__restrict__ dqg, IO *__restrict__ dkg,
                                                     float *__restrict__ dag, float *__restrict__ dbg, float *__restrict__ parts,
                                                     float *__restrict__ gate_parts, int splits, int b, int L, int H, int P,
                                                     int G, int nc, float scale) {
    using T = GradTile<IO, N>;
    using Img = ChunkImage<IO>;
    constexpr int kSz = T::kSz, kP = T::kP, NB = T::NB, kCols = T::kCols, NTT = T::NTT;
    extern __shared__ __align__(16) char lds[];
    __shared__ double gd[2][kC];        // this head's gate sums, in units of ln 2, and the next one's
    __shared__ float zs[8];
    const uint32_t lds0 = lds_address(lds);
    int tid = threadIdx.x, lane = tid & 63, c = lane & 15, q = lane >> 4;
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6), cb = blockIdx.x % kCols, split = blockIdx.x / kCols % splits, cell = blockIdx.x / kCols / splits, ch = cell % nc, bg = cell / nc, g = bg % G, bi = bg / G, r = H / G;
    const int t0 = ch * kC, rows = min(kC, L - t0), ptiles = P / 16;
    const size_t hp = size_t(H) * P, gn = size_t(G) * N;
    const int tw = w & 3, half = w >> 2;
    const bool below = half <= (tw >> 1);       // some of this wave's j's are not after its tokens
    // this wave's columns 32 (ct >> 1) + 8 (m >> 2) + 4 (ct & 1) + (m & 3), m = 0 .. 15, and token tiles th NTT ..
    const int ct = w % T::CT, th = w / T::CT, nq = 32 * (ct >> 1) + 4 * (ct & 1);
    auto tile_of = [&](int i) { return th * NTT + i; };
    const IO *k0 = kg + (size_t(bi) * L + t0) * gn + size_t(g) * N, *q0 = qg + (size_t(bi) * L + t0) * gn + size_t(g) * N;
    float *sums = reinterpret_cast<float *>(lds + T::kSums);
    float *As = reinterpret_cast<float *>(lds + T::kA), *Bs = reinterpret_cast<float *>(lds + T::kB), *Xs = reinterpret_cast<float *>(lds + T::kX);
    f32x4 *held = reinterpret_cast<f32x4 *>(lds + T::kW) + (half ? tw + 2 : tw) * 256 + lane;     // W, F [2][64] each of a wave

    f32x4 dq[NTT], dk[NTT];                 // sums over the heads
    f32x4 Wh[2], Fh[2], xe;                 // of one head: dY E^T and X E^T; X . E
    float accQ[NTT], accV[NTT], accU[NTT], accZ;    // this lane's part of dy S q, X S k, E dS k per token and <S, dS> of one head
    const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < NTT; ++i) dq[i] = dk[i] = zero;
    if (below)
#pragma unroll
        for (int e = 0; e < 4; ++e) held[64 * e] = zero;
    auto clear_head = [&]() {
        Wh[0] = Wh[1] = Fh[0] = Fh[1] = xe = zero;
        accZ = 0.f;
#pragma unroll
        for (int i = 0; i < NTT; ++i) accQ[i] = accV[i] = accU[i] = 0.f;
    };
    clear_head();

    constexpr int kCopiers = kC * T::RB >= 8 * 1024 ? 8 : 4;    // waves: 1 KiB each at least
    auto copy_keys = [&]() {
        if (w < kCopiers) {
            copy_rows<T::RB, kC, kCopiers, 0, 1>(k0 + cb * NB, uint32_t(gn) * kSz, rows - 1, T::RB / 16, lds0 + T::kK);
            copy_rows<T::RB, kC, kCopiers, 0, 1>(q0 + cb * NB, uint32_t(gn) * kSz, rows - 1, T::RB / 16, lds0 + T::kQ);
        }
    };
    const int pbs = (P + T::kRows - 1) / T::kRows, turns = r * pbs;
    const int first = int(int64_t(turns) * split / splits), end = int(int64_t(turns) * (split + 1) / splits);
    // a turn: head g r + hr, rows 32 pi .. of its state
    struct Turn {
        int hr, pi;
    };
    auto following = [&](const Turn &t) { return t.pi + 1 < pbs ? Turn{t.hr, t.pi + 1} : Turn{t.hr + 1, 0}; };
    // one turn's values, as loaded: rows and tokens past the end are zeros
    float in_s[8], in_d[8];         // column tile_row(0, 0, c) + nq, rows 8 q ..
    f32x4 in_e, in_x;
    u32x4 in_y;
    float in_a, in_gate;
    // range-checked views, so that a load's address is a scalar base and the thread's own offset
    auto view_of = [](const void *base, uint32_t bytes) { return buffer_rsrc(base, bytes); };
    auto load16 = [](__amdgpu_buffer_rsrc_t v, uint32_t off) { return __builtin_amdgcn_raw_buffer_load_b128(v, int(off), 0, 0); };
    const uint32_t off_state = (8 * q * N + tile_row(0, 0, c) + nq) * 4;
    auto fetch_states = [&](const Turn &t) {
        const int h = g * r + t.hr, pb = t.pi * T::kRows;
        const size_t at = (((size_t(bi) * H + h) * nc + ch) * P + pb) * N + cb * NB;
        const uint32_t bytes = (min(T::kRows, P - pb) * N - cb * NB) * 4, off = off_state;
        const __amdgpu_buffer_rsrc_t vs = view_of(Sg + at, bytes), vd = view_of(dSg + at, bytes);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            in_s[j] = load_checked<float>(vs, off + 4 * j * N);
            in_d[j] = load_checked<float>(vd, off + 4 * j * N);
        }
    };
    constexpr int kPer = T::RP / 16;            // 16-byte pieces of a token's row of dY
    const int at_y = tid % kPer * (16 / kSz);
    const uint32_t off_dy = tid / kPer * uint32_t(hp) * kSz + tid % kPer * 16;
    auto fetch_rest = [&](const Turn &t) {
        const int h = g * r + t.hr, pb = t.pi * T::kRows;
        const size_t unit = (size_t(bi) * H + h) * nc + ch;
        // E and X: a chain wave's tile of 16 p's is 256 pieces, (tid & 255) >> 6 the token tile
        const size_t piece = (unit * ptiles + pb / 16) * 256;
        const uint32_t bytes = min(T::kRows / 16, ptiles - pb / 16) * 4096;
        in_e = __builtin_bit_cast(f32x4, load16(view_of(E + piece, bytes), tid * 16));
        in_x = __builtin_bit_cast(f32x4, load16(view_of(Xg + piece, bytes), tid * 16));
        const uint32_t past = at_y < P - pb ? 0 : 0x80000000u;
        in_y = load16(chunk_view(dyg + (size_t(bi) * L + t0) * hp + size_t(h) * P + pb, rows, uint32_t(hp) * kSz, P - pb), off_dy | past);
        in_a = ag[(size_t(bi) * L + t0 + min(tid & 63, rows - 1)) * H + h];
        in_gate = reinterpret_cast<const float *>(images + unit * Img::kBytes + Img::kGates)[min(tid, 3 * kC - 1)];
    };
    auto sum_gates = [&](double (&to)[kC], int lane) {      // by one wave, of the head fetched last
        double s = lane < rows ? gate(in_a) : 0.0;
#pragma unroll
        for (int off = 1; off < 64; off <<= 1) {
            const double o = __shfl_up(s, off, 64);
            if (lane >= off) s += o;
        }
        to[lane] = s * kPerLn2;
    };
    auto put4 = [&](char *dst, int stride, f32x4 v) {       // 4 consecutive values, planes `stride` bytes apart
        if constexpr (kSz == 4) {
            *reinterpret_cast<f32x4 *>(dst) = v;
        } else {
#pragma unroll
            for (int p = 0; p < kP; ++p) {
                const u32x2 part = {pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
                *reinterpret_cast<u32x2 *>(dst + p * stride) = part;
                v = f32x4{minus_lo(v[0], part[0]), minus_hi(v[1], part[0]), minus_lo(v[2], part[1]), minus_hi(v[3], part[1])};
            }
        }
    };
    // Offsets formed once.  Chunks of a row lie at chunk ^ place(row), so that another token
    // tile's, whose chunk numbers differ in bits of their own, is an exclusive or away.
    constexpr int kJ = kSz == 4 ? 8 : 2;
    int off_col[kJ];        // of a tile of tokens: rows 8 q .., column tile_row(0, 0, c), as read_col takes them
#pragma unroll
    for (int j = 0; j < kJ; ++j) {
        const int row = kSz == 4 ? 8 * q + j : 8 * q + 4 * j + (c >> 2), n = tile_row(0, 0, c);
        off_col[j] = row * T::RT + (((kSz == 4 ? n >> 2 : c & 3) ^ place<T::RT>(row)) * 16) + (kSz == 4 ? (n & 3) * 4 : 0);
    }
    auto token_operand = [&](const char *tile, int s, int e) {      // columns tile_row(s, e, c)
        Op<IO, kP> o;
        if constexpr (kSz == 4) {
#pragma unroll
            for (int j = 0; j < 8; ++j) o.v[j >> 2][j & 3] = *reinterpret_cast<const float *>(tile + (off_col[j] ^ (128 * s + 16 * e)));
        } else {
#pragma unroll
            for (int i = 0; i < kP; ++i)
                o.p[i] = read_tr8(tile + i * T::kTok + (off_col[0] ^ (64 * s)) + 8 * e, tile + i * T::kTok + (off_col[1] ^ (64 * s)) + 8 * e);
        }
        return o;
    };
    const int row0 = tile_row(0, 0, c);     // token tile 0's row of this lane
    const int off_y = row0 * T::RP + ((kSz == 4 ? 0 : q ^ place<T::RP>(row0)) * 16);
    auto dy_operand = [&](const char *tile, int s, int e) {         // row tile_row(s, e, c), p's 8 q ..
        if constexpr (kSz == 4) {
            return read_row<IO, 1, T::RP>(tile, 0, row0 + 32 * s + 4 * e, 0, q);
        } else {
            Op<IO, 1> o;        // place<64> sees neither the bit of s nor that of e
            o.p[0] = as_bf16x8(*reinterpret_cast<const uint4 *>(tile + off_y + (32 * s + 4 * e) * T::RP));
            return o;
        }
    };
    // 4 values of row tile_row(s, e, c) of k or q, this lane's columns nq + 8 q ..
    const int at_key = (nq + 8 * q) * kSz, off_key = row0 * T::RB + (((at_key >> 4) ^ place<T::RB>(row0)) << 4) + (at_key & 15);
    auto four_of = [&](const char *tile, int s, int e) {
        constexpr int kFlip = place<T::RB>(4) << 4;
        return widen<IO>(*reinterpret_cast<const Raw4<IO> *>(tile + (e ? off_key ^ kFlip : off_key) + (32 * s + 4 * e) * T::RB));
    };
    const int put_row = 16 * (tid >> 8) + c, put_col = 32 * ((tid >> 7) & 1) + 8 * q + 4 * ((tid >> 6) & 1);
    const int off_put = put_row * T::RT + (((put_col * kSz >> 4) ^ place<T::RT>(put_row)) << 4) + (put_col * kSz & 15);
    const int off_puty = tid / (T::RP / 16) * T::RP + (((tid % (T::RP / 16)) ^ place<T::RP>(tid / (T::RP / 16))) * 16);
    auto put_rest = [&](char *to) {
        put4(to + T::kE + off_put, T::kTok, in_e);
        put4(to + T::kV + off_put, T::kTok, in_x);
        if (T::kTok == 16 * T::kThreads || tid < T::kTok / 16) *reinterpret_cast<u32x4 *>(to + T::kY + off_puty) = in_y;
        if (tid < 3 * kC) reinterpret_cast<float *>(to + T::kGates)[tid] = in_gate;
    };
    // row `tok` of k or q as an operand, columns 32 ks + 8 q .. of all N
    auto row_of = [&](const char *tile, const IO *src, int tok, int ks, int q) {
        if constexpr (kCols == 1) return read_row<IO, 1, T::RB>(tile, 0, tok, ks, q);
        else return load_row8<IO>(src + size_t(min(tok, rows - 1)) * gn + 32 * ks + 8 * q);
    };

    Turn now{first / pbs, first % pbs};
    const int portion = split - split_of(int64_t(now.hr) * pbs, turns, splits);     // of the first head
    int side = 0;
    copy_keys();
    fetch_rest(now);
    fetch_states(now);
    copies_done();
    if (w == 4) sum_gates(gd[0], lane);
    xe += in_e * in_x;
    put_rest(lds);
    fetch_rest(first + 1 < end ? following(now) : now);
    __syncthreads();
    for (int turn = first; turn < end; ++turn, now = following(now)) {
        // a thread number the compiler does not know: addresses are formed here again rather
        // than kept over the turns, for which there are not the registers
        tid = threadIdx.x;
        asm volatile("" : "+v"(tid));
        lane = tid & 63, c = lane & 15, q = lane >> 4;
        const bool last_of_head = turn == end - 1 || now.pi == pbs - 1;
        const Turn ahead = turn + 1 < end ? following(now) : now;
        char *buf = lds + (turn - first) % 2 * T::kTurn, *other = lds + (turn - first + 1) % 2 * T::kTurn;
        const float *gates = reinterpret_cast<const float *>(buf + T::kGates);
        float *Tm = reinterpret_cast<float *>(buf);
        // the states' parts; before them the next turn's rest into the other buffer, whose
        // readers have passed the last barrier
        f32x4 xe_next;
        {
            Op<IO, kP> as[1] = {to_op<IO, kP>(f32x4{in_s[0], in_s[1], in_s[2], in_s[3]}, f32x4{in_s[4], in_s[5], in_s[6], in_s[7]})};
            Op<IO, kP> ad[1] = {to_op<IO, kP>(f32x4{in_d[0], in_d[1], in_d[2], in_d[3]}, f32x4{in_d[4], in_d[5], in_d[6], in_d[7]})};
            if (th == 0)
#pragma unroll
                for (int j = 0; j < 8; ++j) accZ += in_s[j] * in_d[j];
            fetch_states(ahead);
            xe_next = in_e * in_x;
            put_rest(other);
            if (last_of_head && w == 4) sum_gates(gd[side ^ 1], lane);      // a wave with fewer products than others
            fetch_rest(turn + 2 < end ? following(ahead) : ahead);
            __builtin_amdgcn_sched_barrier(0);      // the loads first
#pragma unroll
            for (int i = 0; i < NTT; ++i) {
                const int tt = tile_of(i), ts = tt >> 1, te_ = tt & 1, tok = row0 + 32 * ts + 4 * te_;
                const float fs = gates[tok], bt = gates[2 * kC + tok], te = gates[kC + tok] * bt, fv = fs * bt, fq = scale * fs;
                const Op<IO, 1> oy = dy_operand(buf + T::kY, ts, te_);
                const Op<IO, kP> ov = token_operand(buf + T::kV, ts, te_), ou = token_operand(buf + T::kE, ts, te_);
                const f32x4 kv = four_of(lds + T::kK, ts, te_), qv = four_of(lds + T::kQ, ts, te_);
                f32x4 zq[1] = {zero}, zv[1] = {zero}, zu[1] = {zero};
                mma(zq, as, oy);
                mma(zv, as, ov);
                mma(zu, ad, ou);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    dq[i][j] += fq * zq[0][j];
                    dk[i][j] += te * zu[0][j];
                    dk[i][j] -= fv * zv[0][j];
                    accQ[i] += zq[0][j] * qv[j];
                    accV[i] += zv[0][j] * kv[j];
                    accU[i] += zu[0][j] * kv[j];
                }
            }
        }
        const int tok = tile_row(tw >> 1, tw & 1, c);       // this lane's token in what follows
        // dY E^T and X E^T (rows j, columns i: this lane's token)
        if (below) {
            const Op<IO, 1> oy = dy_operand(buf + T::kY, tw >> 1, tw & 1);
            const Op<IO, kP> ov = token_operand(buf + T::kV, tw >> 1, tw & 1);
            Op<IO, kP> au[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) au[e] = token_operand(buf + T::kE, half, e);
            mma(Wh, au, oy);
            mma(Fh, au, ov);
        }
        __syncthreads();
        if (!last_of_head) {
            xe += xe_next;
            continue;
        }

        // The head's W and F, and its gates' gradients:  with T_ij = W_ij (q_i . k_j) + F_ij (k_i . k_j),
        //   A_i = scale e^{g_i} dy_i . S q_i - dv_i . e^{g_i} S k_i,  B_j = u_j . e^{g_C - g_j} dS k_j,  Z = e^{g_C} <S, dS>
        //   da_t = sum of T_ij over j < t <= i + sum of A_i over i >= t + sum of B_j over j < t + Z
        // all terms that pass the gate of token t, and no others: each holds e^{a_t}, so that none
        // of them outgrows the result where that gate closes.
        {
            f32x4 kk[2] = {zero, zero}, qk[2] = {zero, zero};
            if (below && cb == 0) {     // T once, not per part of the columns
#pragma unroll
                for (int ks = 0; ks < N / 32; ++ks) {
                    Op<IO, 1> a[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) a[e] = row_of(lds + T::kK, k0, tile_row(half, e, c), ks, q);
                    mma(kk, a, row_of(lds + T::kK, k0, tok, ks, q));
                    mma(qk, a, row_of(lds + T::kQ, q0, tok, ks, q));
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
            const double *gs = gd[side], gt = gs[tok];
            const float bt = gates[2 * kC + tok];
            const int most = tok < rows ? tok : -1;     // no j is that small
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int j0 = 32 * half + 8 * q + 4 * e;
                const f32x4 bj = *reinterpret_cast<const f32x4 *>(gates + 2 * kC + j0);
                f32x4 wv, fv;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float d = decay(gt - gs[j0 + i]) * bj[i], x = scale * d * Wh[e][i], y = -bt * d * Fh[e][i];
                    wv[i] = j0 + i <= most ? x : 0.f;
                    fv[i] = j0 + i < most ? y : 0.f;
                    Tm[tok * T::LT + j0 + i] = j0 + i < most ? x * qk[e][i] + y * kk[e][i] : 0.f;
                }
                if (below) {
                    held[128 * e] += wv;
                    held[128 * e + 64] += fv;
                }
            }
        }
        // sums over the 4 lane groups; of 4 token tiles, each ends up in a group of its own
        float sa[NTT], sb[NTT];
#pragma unroll
        for (int i = 0; i < NTT; ++i) {
            const int tt = tile_of(i), at = row0 + 32 * (tt >> 1) + 4 * (tt & 1);
            const float fs = gates[at], bt = gates[2 * kC + at];
            sa[i] = scale * fs * accQ[i] - fs * bt * accV[i];
            sb[i] = gates[kC + at] * bt * accU[i];
        }
        if constexpr (NTT == 4) {
            const float a = two_sums16(two_sums32(sa[0], sa[2]), two_sums32(sa[1], sa[3])), b = two_sums16(two_sums32(sb[0], sb[2]), two_sums32(sb[1], sb[3]));
            const int at = row0 + 32 * (q >> 1) + 4 * (q & 1);
            As[ct * kC + at] = at < rows ? a : 0.f;
            Bs[ct * kC + at] = at < rows ? b : 0.f;
        } else {
#pragma unroll
            for (int i = 0; i < NTT; ++i) {
                const int tt = tile_of(i), at = row0 + 32 * (tt >> 1) + 4 * (tt & 1);
                const float a = group4_sum(sa[i]), b = group4_sum(sb[i]);
                if (q == 0) {
                    As[ct * kC + at] = at < rows ? a : 0.f;
                    Bs[ct * kC + at] = at < rows ? b : 0.f;
                }
            }
        }
        accZ = wave_sum(accZ);
        if (lane == 0) zs[w] = accZ;
#pragma unroll
        for (int j = 0; j < 4; ++j) xe[j] = row16_sum(xe[j]);
        if (c == 0) *reinterpret_cast<f32x4 *>(Xs + (tid >> 8) * kC + 32 * ((tid >> 7) & 1) + 8 * q + 4 * ((tid >> 6) & 1)) = xe;
        const float alpha = gates[kC - 1];      // (the next turn writes this buffer)
        clear_head();
        xe = xe_next;
        __syncthreads();
        // wave w: the sums down the columns of T, from rows 8 w .. 8 w + 7 on; lane = column j
        float v[8];
#pragma unroll
        for (int i = 7; i >= 0; --i) v[i] = Tm[(8 * w + i) * T::LT + lane] + (i < 7 ? v[i + 1] : 0.f);
        sums[w * kC + lane] = v[0];
        __syncthreads();
        float lower = 0.f;
#pragma unroll
        for (int i = 1; i < 8; ++i) lower += w + i < 8 ? sums[((w + i) & 7) * kC + lane] : 0.f;
        // row 8 w + i: its columns j < t; 8 sums over 64 lanes, two rows at a time ending up in
        // half of the lanes each
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = lane < 8 * w + i ? v[i] + lower : 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = two_sums32(v[i], v[i + 4]);
#pragma unroll
        for (int i = 0; i < 2; ++i) v[i] = row16_sum(two_sums16(v[i], v[i + 2]));
        const int t = 8 * w + 4 * (q >> 1) + 2 * (q & 1) + (c & 1);     // lane's row
        // A from the last token down, B from the first up to the one before
        float a = 0.f, bs = 0.f;
#pragma unroll
        for (int i = 0; i < T::CT; ++i) {
            a += As[i * kC + 63 - lane];
            bs += Bs[i * kC + lane];
        }
        const float after = __shfl(wave_inclusive_scan(a), 63 - t, 64), before = __shfl(wave_inclusive_scan(bs), max(t - 1, 0), 64);
        const float z = ((zs[0] + zs[1]) + (zs[2] + zs[3])) + ((zs[4] + zs[5]) + (zs[6] + zs[7]));
        const float da = (c & 1 ? v[1] : v[0]) + after + (t ? before : 0.f) + alpha * z;
        if (c < 2 && t < rows) {
            const size_t all = size_t(b) * L * H, at = (size_t(bi) * L + t0 + t) * H + g * r + now.hr;
            const float db = cb == 0 ? Xs[t] + Xs[kC + t] : 0.f;
            if (kCols > 1 || splits > 1) {
                float *to = gate_parts + 2 * all * ((turn - now.pi < first ? portion : 0) * kCols + cb) + at;
                to[0] = da;
                to[all] = db;
            } else {
                dag[at] = da;
                dbg[at] = db;
            }
        }
        side ^= 1;
    }
    __syncthreads();
    const int tok = tile_row(tw >> 1, tw & 1, c);
    // W [i][j] and F [i][j], 0 above the diagonal
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const int col = 32 * half + 8 * q + 4 * e, at = tok * T::RT + (((col * kSz >> 4) ^ place<T::RT>(tok)) << 4) + (col * kSz & 15);
        put4(lds + T::kWm + at, T::kMat, below ? held[128 * e] : zero);
        put4(lds + T::kFm + at, T::kMat, below ? held[128 * e + 64] : zero);
    }
    __syncthreads();
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
        const Op<IO, 1> ak[1] = {read_col<IO, 1, T::RB>(lds + T::kK, 0, 32 * ks, 32 * (ct >> 1), ct & 1, c, q)};
        const Op<IO, 1> aq[1] = {read_col<IO, 1, T::RB>(lds + T::kQ, 0, 32 * ks, 32 * (ct >> 1), ct & 1, c, q)};
#pragma unroll
        for (int i = 0; i < NTT; ++i) {
            const int tt = tile_of(i), at = tile_row(tt >> 1, tt & 1, c);
            f32x4 zq[1] = {dq[i]}, zk[1] = {dk[i]};
            if (ks <= (tt >> 1)) {          // rows i of the tile: j <= i
                mma(zq, ak, read_row<IO, kP, T::RT>(lds + T::kWm, T::kMat, at, ks, q));
                mma(zk, ak, read_row<IO, kP, T::RT>(lds + T::kFm, T::kMat, at, ks, q));
            }
            if (ks >= (tt >> 1)) {          // and as columns: i >= j
                mma(zk, ak, read_col<IO, kP, T::RT>(lds + T::kFm, T::kMat, 32 * ks, 32 * (tt >> 1), tt & 1, c, q));
                mma(zk, aq, read_col<IO, kP, T::RT>(lds + T::kWm, T::kMat, 32 * ks, 32 * (tt >> 1), tt & 1, c, q));
            }
            dq[i] = zq[0];
            dk[i] = zk[0];
        }
    }
    const size_t all = size_t(b) * L * gn;
#pragma unroll
    for (int i = 0; i < NTT; ++i) {
        const int tt = tile_of(i), at = tile_row(tt >> 1, tt & 1, c);
        if (at >= rows) continue;
        const size_t dst = (size_t(bi) * L + t0 + at) * gn + size_t(g) * N + cb * NB + nq + 8 * q;
        if (splits > 1) {
            *reinterpret_cast<f32x4 *>(parts + 2 * split * all + dst) = dq[i];
            *reinterpret_cast<f32x4 *>(parts + (2 * split + 1) * all + dst) = dk[i];
        } else {
            *reinterpret_cast<Raw4<IO> *>(dqg + dst) = narrow<IO>(dq[i]);
            *reinterpret_cast<Raw4<IO> *>(dkg + dst) = narrow<IO>(dk[i]);
        }
    }
}

// The parts added in their order: of dq and dk, parts [splits][dq, dk][all] fp32, 8 elements
// per thread; of da and dbeta, gate_parts [portions of a head][da, dbeta][b, L, H], one per
// thread of the blocks from `blocks` on (`cols` of them per portion).
template <typename IO>
__global__ __launch_bounds__(256) void k_delta_join(const float *__restrict__ parts, IO *__restrict__ dqg, IO *__restrict__ dkg,
                                                    const float *__restrict__ gate_parts, float *__restrict__ da,
                                                    float *__restrict__ dbeta, int splits, size_t all, unsigned blocks, size_t tokens,
                                                    int H, int r, int pbs, int cols) {
    if (blockIdx.x >= blocks) {
        const size_t i = size_t(blockIdx.x - blocks) * 256 + threadIdx.x, n = tokens * H;
        if (i >= 2 * n) return;
        const bool second = i >= n;
        const int hr = int((second ? i - n : i) % H) % r;
        const int64_t turn = int64_t(hr) * pbs, turns = int64_t(r) * pbs;
        const int portions = split_of(turn + pbs - 1, turns, splits) - split_of(turn, turns, splits) + 1;
        float s = 0.f;
        for (int j = 0; j < portions * cols; ++j) s += gate_parts[2 * n * j + i];
        (second ? dbeta : da)[second ? i - n : i] = s;
        return;
    }
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

// Turns of a head in k_delta_grads, and the parts its columns are taken in.
int grad_turns(int P) { return (P + 31) / 32; }
int grad_columns(int N, bool bf16) { return N * (bf16 ? 2 : 4) > 256 ? N * (bf16 ? 2 : 4) / 256 : 1; }

template <typename IO, int N>
hipError_t launch_n(const DeltaBwdArgs &a, const DeltaBwdPlan &pl, hipStream_t stream) {
    const int nc = (a.L + kC - 1) / kC, ptiles = a.P / 16;
    char *ws = static_cast<char *>(a.workspace);
    char *images = ws;
    const auto *q = static_cast<const IO *>(a.q), *k = static_cast<const IO *>(a.k), *v = static_cast<const IO *>(a.v);
    const auto *dy = static_cast<const IO *>(a.dy);
    auto *dv = static_cast<IO *>(a.dv);
    DeltaSaved saved{reinterpret_cast<float *>(ws + pl.off_e), reinterpret_cast<float *>(ws + pl.off_s)};
    auto *dS = reinterpret_cast<float *>(ws + pl.off_ds);
    auto *kept_x = reinterpret_cast<f32x4 *>(ws + pl.off_x);
    auto *parts = reinterpret_cast<float *>(ws + pl.off_parts), *gate_parts = reinterpret_cast<float *>(ws + pl.off_gate_parts);

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
        constexpr int lds = ChainLds<IO, N, W, X, true, false, ONE>::kBytes;
        const int rows = 16 * W / X, pblocks = (a.P + rows - 1) / rows;
        auto kern = k_delta_chain_back<IO, N, W, X, MAP, ONE>;
        e = hipFuncSetAttribute(reinterpret_cast<const void *>(kern), hipFuncAttributeMaxDynamicSharedMemorySize, lds);
        if (e != hipSuccess) return e;
        hipLaunchKernelGGL(kern, dim3(unsigned(int64_t(a.b) * a.H * (cut.segments - (MAP ? 1 : 0)) * pblocks)), dim3(64 * W), lds, stream, q, k,
                           dy, images, a.d_final, dinit, dv, dS, kept_x, to, a.L, a.H, a.P, a.G, nc, cut.per, cut.segments, pblocks, a.scale);
        return hipGetLastError();
    };
    const int64_t tiles = int64_t(a.b) * a.H * ptiles;
    if (cut.segments > 1) {
        auto go = [&](auto w, auto x, auto one) { return back(w, x, one, std::true_type{}, dmap); };
        if ((e = with_chain_shape<IO, N, true>(tiles * (cut.segments - 1), go)) != hipSuccess) return e;
        hipLaunchKernelGGL((k_delta_carry<N, true>), dim3(unsigned(tiles)), dim3(4 * N), 0, stream, map, dmap, nullptr, dinit, a.P, cut.segments);
        if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    auto chains = [&](auto w_, auto x_, auto one_) {
        constexpr int W = decltype(w_)::value, X = decltype(x_)::value;
        e = launch_chain<IO, N, W, X, Chain::save, decltype(one_)::value>(q, k, v, images, cut.segments > 1 ? init : a.init_state, nullptr, nullptr,
                                                           saved, a.b, a.L, a.H, a.P, a.G, cut.per, cut.segments, a.scale, stream);
        return e != hipSuccess ? e : back(w_, x_, one_, std::false_type{}, a.d_init);
    };
    if ((e = with_chain_shape<IO, N, true>(tiles * cut.segments, chains)) != hipSuccess) return e;
    auto grads = k_delta_grads<IO, N>;
    constexpr int lds = GradTile<IO, N>::kLds;
    e = hipFuncSetAttribute(reinterpret_cast<const void *>(grads), hipFuncAttributeMaxDynamicSharedMemorySize, lds);
    if (e != hipSuccess) return e;
    constexpr int kCols = GradTile<IO, N>::kCols;
    hipLaunchKernelGGL(grads, dim3(unsigned(int64_t(a.b) * a.G * nc * pl.splits * kCols)), dim3(GradTile<IO, N>::kThreads), lds, stream, q, k, a.a, dy, images,
                       reinterpret_cast<const f32x4 *>(saved.E), kept_x, saved.S, dS, static_cast<IO *>(a.dq), static_cast<IO *>(a.dk), a.da,
                       a.dbeta, parts, gate_parts, pl.splits, a.b, a.L, a.H, a.P, a.G, nc, a.scale);
    if ((e = hipGetLastError()) != hipSuccess || pl.splits * kCols == 1) return e;
    const size_t tokens = size_t(a.b) * a.L, all = tokens * a.G * N;
    const unsigned blocks = pl.splits > 1 ? unsigned((2 * all + 2047) / 2048) : 0;
    hipLaunchKernelGGL(k_delta_join<IO>, dim3(blocks + unsigned((2 * tokens * a.H + 255) / 256)), dim3(256), 0, stream, parts, static_cast<IO *>(a.dq),
                       static_cast<IO *>(a.dk), gate_parts, a.da, a.dbeta, pl.splits, all, blocks, tokens, a.H, a.H / a.G, grad_turns(a.P), kCols);
    return hipGetLastError();
}

// Parts to split a group's `turns` (of up to 32 state rows) into, where the chunks alone
// leave CUs idle: as many as give each CU a block.
int grad_splits(size_t cells, size_t turns) { return int(std::max<size_t>(1, std::min(turns, 256 / cells))); }

}  // namespace

DeltaBwdPlan plan_delta_bwd(int b, int L, int H, int P, int N, int G, bool bf16) {
    DeltaBwdPlan pl;
    if (b <= 0 || L <= 0 || !delta_chunk_supported(b, L, H, P, N, G, bf16)) return pl;
    const size_t nc = (size_t(L) + kC - 1) / kC, bh = size_t(b) * H, units = bh * nc;
    const size_t state = size_t(P) * N;
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
    const int cols = grad_columns(N, bf16);
    pl.splits = grad_splits(size_t(b) * G * nc * cols, size_t(H / G) * grad_turns(P));
    pl.cut = cut_sequence(int64_t(bh), int(nc), P, N, bf16, true);
    pl.off_map = take(map_bytes(bh, P, N, pl.cut));
    pl.off_init = take(entering_bytes(bh, P, N, pl.cut));
    pl.off_dmap = take(entering_bytes(bh, P, N, pl.cut));
    pl.off_dinit = take(entering_bytes(bh, P, N, pl.cut));
    pl.off_parts = take(pl.splits > 1 ? size_t(pl.splits) * 2 * b * L * G * N * 4 : 0);
    pl.off_gate_parts = take(pl.splits * cols > 1 ? size_t(pl.splits > 1 ? grad_turns(P) : 1) * cols * 2 * b * L * H * 4 : 0);
    pl.total = at;
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
