// ssd_delta_chain.h -- the chain over the chunks of the gated delta rule, forward (see
// ssd_delta_chunk.h for the formulas and the tile layout).
#pragma once

#include "ssd_delta.h"
#include "ssd_delta_chunk.h"

namespace ssd {

// What the forward chain leaves for the backward pass, fp32, per (batch, head):
//   E       [nc][P / 16][4][64] f32x4: a wave's accumulators of the brackets, as held
//   S       [nc][P][N]: the state that enters each chunk
struct DeltaSaved {
    float *E, *S;
};

// A block's W waves are W / X tiles of 16 state rows, each shared by X waves that hold
// N / X of its columns.  The sums over all columns (K S^T, Q S^T) are added up through LDS;
// what only depends on those is computed by every one of the X waves, bit for bit alike.
// Sharing shortens a chunk's steps where there are fewer tiles than SIMDs.
//
// LDS: k, M, the scores and gates of two chunks, the next one's copied in meanwhile (one
// chunk where two do not fit, or, ONE, where two blocks a CU gain more than copies ahead).
// Chains that read them (Q) have the scores, and q: with X = 1 beside them; with more, that of
// one chunk, which is done with halfway through it.  Then the exchanged sums (YX: those of
// Q S^T too).
template <typename IO, int N, int W, int X, bool Q, bool YX, bool ONE>
struct ChainLds {
    using Img = ChunkImage<IO>;
    static constexpr int kSz = int(sizeof(IO));
    static constexpr int RB = N * kSz;                      // bytes per row of k or q
    static constexpr int kRows = kC * RB;                   // bytes of such a tile
    static constexpr bool kQMain = Q && X == 1;             // q beside k, in both buffers
    static constexpr int kImg = kQMain ? 2 * kRows : kRows, kImgBytes = Q ? Img::kBytes : Img::kQ;
    static constexpr int kMain = kImg + kImgBytes, kQOwn = Q && X > 1 ? kRows : 0;
    static constexpr int kXe = X > 1 ? W * 4096 : 0, kXy = X > 1 && YX ? W * (4096 - 4096 / X) : 0;
    static constexpr int kBufs = !ONE && 2 * kMain + kQOwn + kXe + kXy <= 160 * 1024 ? 2 : 1;
    static constexpr int kQt = kBufs * kMain, kE = kQt + kQOwn, kY = kE + kXe, kBytes = kY + kXy;
    static_assert(kBytes <= 160 * 1024 && N / 32 % X == 0 && W % X == 0);
};

// Start the copies of ROWS rows of RB bytes (row r at base + r * stride bytes; rows
// past `last`: that one; 16-byte chunks of a row past `chunks`: the last one) into a tile.
// The block's waves take 1 KiB in turn; this call starts part PART of PARTS.
template <int RB, int ROWS, int W, int PART, int PARTS>
__device__ __forceinline__ void copy_rows(const void *base, uint32_t stride, int last, int chunks, uint32_t dst) {
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    constexpr int kIt = ROWS * RB / 1024 / W, kPer = (kIt + PARTS - 1) / PARTS;
    static_assert(kIt * W * 1024 == ROWS * RB);
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

// One element of a range-checked view; past its end: 0.
template <typename IO>
__device__ __forceinline__ IO load_checked(__amdgpu_buffer_rsrc_t v, uint32_t off) {
    if constexpr (std::is_same_v<IO, float>) return __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(v, int(off), 0, 0));
    else return __builtin_amdgcn_raw_buffer_load_b16(v, int(off), 0, 0);
}
// 4 elements of the I/O type.
template <typename IO>
using Raw4 = std::conditional_t<std::is_same_v<IO, float>, f32x4, u32x2>;
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

// Element r becomes a NaN.
template <typename IO>
__device__ __forceinline__ void set_nan(Raw4<IO> &v, int r) {
    if constexpr (std::is_same_v<IO, float>) v[r] = __builtin_nanf("");
    else v[r >> 1] |= 0x7fffu << (16 * (r & 1));
}

// A range-checked view of one chunk of a [b, L, H, P] tensor, from its first token's row of
// head h on (`base`), `rows` tokens.
template <typename IO>
__device__ __forceinline__ __amdgpu_buffer_rsrc_t chunk_view(const IO *base, int rows, uint32_t tok, int P) {
    return buffer_rsrc(base, uint32_t(rows - 1) * tok + uint32_t(P) * uint32_t(sizeof(IO)));
}

// The sum of the X waves' accumulators (16-byte pieces [4][64] per wave), in their order.
template <int X>
__device__ __forceinline__ void sum_of_parts(const char *first, int lane, f32x4 (&out)[4]) {
#pragma unroll
    for (int t = 0; t < 4; ++t) {
        out[t] = reinterpret_cast<const f32x4 *>(first)[64 * t + lane];
#pragma unroll
        for (int x = 1; x < X; ++x) out[t] += reinterpret_cast<const f32x4 *>(first + x * 4096)[64 * t + lane];
    }
}

// The first token of a chunk with a value that is not finite among this lane's column (p),
// kC if there is none; v and w become 0 from there on.  A matrix product multiplies the zeros
// above a triangle too: with them, such a value would reach the tokens before it.
__device__ __forceinline__ int stop_at(f32x4 (&v)[4], f32x4 (&w)[4], int q) {
    int first = kC;
#pragma unroll
    for (int t = 3; t >= 0; --t)
#pragma unroll
        for (int r = 3; r >= 0; --r)
            if (!__builtin_isfinite(v[t][r])) first = 32 * (t >> 1) + 8 * q + 4 * (t & 1) + r;
    first = min(first, __shfl_xor(first, 16, 64));
    first = min(first, __shfl_xor(first, 32, 64));
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r)
            if (32 * (t >> 1) + 8 * q + 4 * (t & 1) + r >= first) v[t][r] = w[t][r] = 0.f;
    return first;
}

// What bounds it: one wave's steps, not the matrix cores.  A chunk of a bf16 tile at N = 128
// is 216 matrix instructions (3500 cycles) and 7400 cycles in between, of which splitting
// values into planes and the accumulators' scaling issue for 3300; the waves of the only
// block that fits a CU find nobody to fill the rest.  4 x 2048 tokens, 32 heads of 128 x 128,
// a wave on every SIMD: 168 us for 32 chunks in turn, 168 MB of inputs and outputs.  Tried
// without gain on an earlier, 141 us form: 8 waves in lockstep, copies in two groups with half
// a chunk each to arrive, products interleaved by hand, two blocks a CU (spills).

// What a chain is run for.
//   run   y and the final state
//   save  what the backward pass needs
//   map   what a segment of the sequence does to the state that enters it, S -> S A + B: the
//         states after it of P rows that enter as 0 (B) and, with v = 0, of the N rows of the
//         identity (A).  The first segment's P rows enter as they are, without the others.
enum class Chain { run, save, map };

// One chain per (batch, head, segment of `per` chunks); `init` has a state for each, `fin`
// for each (map: [P + N][N]) or for each (batch, head).
template <typename IO, int N, int W, int X, Chain MODE, bool ONE>
__global__ __launch_bounds__(64 * W) void k_delta_chain(const IO *__restrict__ qg, const IO *__restrict__ kg,
                                                        const IO *__restrict__ vg, const char *__restrict__ images,
                                                        const float *__restrict__ init, IO *__restrict__ yg,
                                                        float *__restrict__ fin, DeltaSaved saved, int L, int H, int P, int G, int nc, int per, int segs,
                                                        int pblocks, float scale) {
    constexpr bool RUN = MODE == Chain::run, SAVE = MODE == Chain::save, MAP = MODE == Chain::map;
    using T = ChainLds<IO, N, W, X, RUN, RUN, ONE>;
    using Img = typename T::Img;
    extern __shared__ __align__(16) char lds[];
    constexpr int kSz = int(sizeof(IO)), KS = N / 32 / X, NT = 2 * KS;  // this wave's column blocks and tiles
    const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6), c = lane & 15, q = lane >> 4;
    const int x = w % X, n0 = x * KS;           // first column block
    const int blk = xcd_neighbours(), pb = blk % pblocks, unit = blk / pblocks, seg = unit % segs, bh = unit / segs;
    const int h = bh % H, bi = bh / H, g = h / (H / G);
    const int p0 = (pb * (W / X) + w / X) * 16, p = p0 + c, ptiles = P / 16;
    const int first = seg * per, end = min(first + per, nc), prows = MAP && seg > 0 ? P + N : P;
    if (pb * (W / X) * 16 >= prows) return;
    const bool live = p0 < prows;   // the same for a whole wave, and for the waves of a tile
    const size_t hp = size_t(H) * P, gn = size_t(G) * N;
    const char *img = images + size_t(bh) * nc * Img::kBytes;
    const IO *k0 = kg + size_t(bi) * L * gn + size_t(g) * N, *q0 = qg + size_t(bi) * L * gn + size_t(g) * N;
    const size_t vy0 = size_t(bi) * L * hp + size_t(h) * P;
    const uint32_t lds0 = lds_address(lds), tok = uint32_t(hp) * kSz;
    char *xe = lds + T::kE + w * 4096;

    // the copies of chunk ch: k and the image into the buffer at `buf` in 4 parts; q
    // (with it or alone)
    auto fetch = [&](int ch, uint32_t buf, auto part) {
        constexpr int kPart = decltype(part)::value;
        const int t0 = ch * kC, last = min(kC, L - t0) - 1;
        copy_rows<T::RB, kC, W, kPart, 4>(k0 + size_t(t0) * gn, uint32_t(gn) * kSz, last, T::RB / 16, buf);
        copy_image<T::kImgBytes, W, kPart, 4>(img + size_t(ch) * Img::kBytes, buf + T::kImg);
        if constexpr (T::kQMain) copy_rows<T::RB, kC, W, kPart, 4>(q0 + size_t(t0) * gn, uint32_t(gn) * kSz, last, T::RB / 16, buf + T::kRows);
    };
    auto fetch_q = [&](int ch) {
        if constexpr (T::kQMain || !RUN) return;
        const int t0 = ch * kC, last = min(kC, L - t0) - 1;
        copy_rows<T::RB, kC, W, 0, 1>(q0 + size_t(t0) * gn, uint32_t(gn) * kSz, last, T::RB / 16, lds0 + T::kQt);
    };
    auto fetch_main = [&](int ch, uint32_t buf) {
        fetch(ch, buf, std::integral_constant<int, 0>{});
        fetch(ch, buf, std::integral_constant<int, 1>{});
        fetch(ch, buf, std::integral_constant<int, 2>{});
        fetch(ch, buf, std::integral_constant<int, 3>{});
    };
    // v of chunk ch, by one wave of a tile: accumulator layout
    IO rv[16];
    auto fetch_v = [&](int ch) {
        if (!live || x != 0 || (MAP && p0 >= P)) return;
        const int t0 = ch * kC;
        const __amdgpu_buffer_rsrc_t view = chunk_view(vg + vy0 + size_t(t0) * hp, min(kC, L - t0), tok, P);
        const uint32_t off = uint32_t(8 * q) * tok + uint32_t(p) * kSz;
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) rv[4 * t + r] = load_checked<IO>(view, off + uint32_t(32 * (t >> 1) + 4 * (t & 1) + r) * tok);
    };
    f32x4 V[4];
    auto take_v = [&]() {
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) V[t][r] = x == 0 ? to_f32<IO>(rv[4 * t + r]) : 0.f;
    };
    // row p of the state, this wave's columns 32 (n0 + t / 2) + 8 q + 4 (t & 1) ..
    auto state_at = [&](size_t of, int rows, int t) { return (of * rows + p) * N + 32 * (n0 + (t >> 1)) + 8 * q + 4 * (t & 1); };

    f32x4 S[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) S[t] = f32x4{0.f, 0.f, 0.f, 0.f};
    if (MAP && p0 >= P) {
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) S[t][r] = p - P == 32 * (n0 + (t >> 1)) + 8 * q + 4 * (t & 1) + r ? 1.f : 0.f;
    } else if (init && live && (!MAP || seg == 0)) {
#pragma unroll
        for (int t = 0; t < NT; ++t) S[t] = *reinterpret_cast<const f32x4 *>(init + state_at(MAP ? bh : unit, P, t));
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) rv[i] = IO(0);
    fetch_main(first, lds0);
    fetch_q(first);
    fetch_v(first);
    copies_done();
    take_v();
    __syncthreads();

    for (int ch = first; ch < end; ++ch) {
        const int t0 = ch * kC, rows = min(kC, L - t0), next = min(ch + 1, end - 1);    // past the last: that one again
        const char *buf = lds + (T::kBufs == 2 ? ((ch - first) & 1) * T::kMain : 0);
        const char *tk = buf, *tq = T::kQMain ? buf + T::kRows : lds + T::kQt, *tm = buf + T::kImg + Img::kM, *ts = buf + T::kImg + Img::kQ;
        const float *gates = reinterpret_cast<const float *>(buf + T::kImg + Img::kGates);
        auto ahead = [&](auto part) {
            if constexpr (T::kBufs == 2) fetch(next, lds0 + ((ch - first + 1) & 1) * T::kMain, part);
        };
        auto gate_of = [&](int which, int t) {
            return *reinterpret_cast<const f32x4 *>(gates + which * kC + 32 * (t >> 1) + 8 * q + 4 * (t & 1));
        };
        Raw4<IO> yo[4];
        f32x4 E[4], Y[4];
        bool stop = false;      // the same for a whole wave
        int bad = kC;
        fetch_v(next);
        ahead(std::integral_constant<int, 0>{});
        if (live) {
            Op<IO, kPlanes> so[KS];
#pragma unroll
            for (int s = 0; s < KS; ++s) so[s] = to_op<IO, kPlanes>(S[2 * s], S[2 * s + 1]);
            if constexpr (SAVE) {
                float *dst = saved.S + ((size_t(bh) * nc + ch) * P + p) * N + 32 * n0 + 8 * q;
#pragma unroll
                for (int t = 0; t < NT; ++t) *reinterpret_cast<f32x4 *>(dst + 32 * (t >> 1) + 4 * (t & 1)) = S[t];
            }
            // this wave's part of R = V - e^g K S^T, and of the state's part of Y (rows p in
            // registers: 4 consecutive ones of one token per lane)
#pragma unroll
            for (int t = 0; t < 4; ++t) E[t] = Y[t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                Op<IO, 1> a[4];
#pragma unroll
                for (int t = 0; t < 4; ++t) a[t] = read_row<IO, 1, T::RB>(tk, 0, tile_row(t >> 1, t & 1, c), n0 + ks, q);
                mma(E, a, so[ks]);
            }
#pragma unroll
            for (int ks = 0; ks < (RUN ? KS : 0); ++ks) {
                Op<IO, 1> a[4];
#pragma unroll
                for (int t = 0; t < 4; ++t) a[t] = read_row<IO, 1, T::RB>(tq, 0, tile_row(t >> 1, t & 1, c), n0 + ks, q);
                mma(Y, so[ks], a);
            }
#pragma unroll
            for (int t = 0; t < 4; ++t) E[t] = V[t] - gate_of(0, t) * E[t];
            if constexpr (X > 1) {
#pragma unroll
                for (int t = 0; t < 4; ++t) reinterpret_cast<f32x4 *>(xe)[64 * t + lane] = E[t];
                if constexpr (RUN) {     // token tiles t of Y go to wave t / (4 / X)
                    f32x4 *xy = reinterpret_cast<f32x4 *>(lds + T::kY + w * (T::kXy / W));
#pragma unroll
                    for (int t = 0; t < 4; ++t) {
                        const int to = t / (4 / X);
                        if (to != x) xy[64 * (to < x ? t : t - 4 / X) + lane] = Y[t];
                    }
                }
            }
        }
        if constexpr (X > 1) __syncthreads();       // the parts are written, q is read
        if constexpr (T::kBufs == 2) fetch_q(next);
        ahead(std::integral_constant<int, 1>{});
        if (live) {
            if constexpr (X > 1) sum_of_parts<X>(lds + T::kE + (w - x) * 4096, lane, E);
            // E = R + M (beta R), U = beta E
            f32x4 B[4];
            f32x4 probe = {0.f, 0.f, 0.f, 0.f};     // NaN if any bracket is not finite
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                B[t] = gate_of(2, t) * E[t];
#pragma unroll
                for (int r = 0; r < 4; ++r) probe[r] = __builtin_fmaf(E[t][r], 0.f, probe[r]);
            }
            const float any = (probe[0] + probe[1]) + (probe[2] + probe[3]);
            stop = __any(any != any);
            if (stop) bad = stop_at(E, B, q);
            Op<IO, kPlanes> br[2];
#pragma unroll
            for (int s = 0; s < 2; ++s) br[s] = to_op<IO, kPlanes>(B[2 * s], B[2 * s + 1]);
            {
                Op<IO, kPlanes> a[4];
#pragma unroll
                for (int t = 0; t < 4; ++t) a[t] = tri_row<IO, kPlanes>(tm, t >> 1, t & 1, 0, c, q);
                mma(E, a, br[0]);
            }
            {
                f32x4 lower[2] = {E[2], E[3]};
                Op<IO, kPlanes> a[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) a[e] = tri_row<IO, kPlanes>(tm, 1, e, 1, c, q);
                mma(lower, a, br[1]);
                E[2] = lower[0];
                E[3] = lower[1];
            }
            Op<IO, kPlanes> uy[2];
            Op<IO, kPlanes> ud[2];
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const f32x4 u0 = gate_of(2, 2 * s) * E[2 * s], u1 = gate_of(2, 2 * s + 1) * E[2 * s + 1];
                ud[s] = to_op<IO, kPlanes>(gate_of(1, 2 * s) * u0, gate_of(1, 2 * s + 1) * u1);
                uy[s] = to_op<IO, kPlanes>(u0, u1);
            }
            ahead(std::integral_constant<int, 2>{});
            // S <- e^{g_C} S + K^T (e^{g_C - g} U)
            const float alpha = gates[kC - 1];
#pragma unroll
            for (int t = 0; t < NT; ++t) S[t] *= alpha;
#pragma unroll
            for (int ks = 0; ks < 2; ++ks)
#pragma unroll
                for (int u0 = 0; u0 < NT; u0 += 4) {     // 4 tiles a turn (or all 2)
                    constexpr int M = NT < 4 ? NT : 4;
                    f32x4 z[M];
                    Op<IO, 1> a[M];
#pragma unroll
                    for (int t = 0; t < M; ++t) {
                        z[t] = S[u0 + t];
                        a[t] = read_col<IO, 1, T::RB>(tk, 0, 32 * ks, 32 * (n0 + ((u0 + t) >> 1)), t & 1, c, q);
                    }
                    mma(z, a, ud[ks]);
#pragma unroll
                    for (int t = 0; t < M; ++t) S[u0 + t] = z[t];
                }
            ahead(std::integral_constant<int, 3>{});
            // Y = scale e^g Q S^T + scores U; wave x finishes the token tiles t of t / (4 / X) = x
#pragma unroll
            for (int t = 0; t < (RUN ? 4 : 0); ++t) {
                const bool mine = t / (4 / X) == x;     // the same for a whole wave
                if constexpr (X > 1) {
                    if (!mine) continue;
#pragma unroll
                    for (int o = 1; o < X; ++o) {
                        const int from = (x + o) % X;   // any order: two parts only, or a fixed rotation
                        Y[t] += reinterpret_cast<const f32x4 *>(lds + T::kY + (w - x + from) * (T::kXy / W))[64 * (x < from ? t : t - 4 / X) + lane];
                    }
                }
                f32x4 z[1] = {(scale * gates[tile_row(t >> 1, t & 1, c)]) * Y[t]};
#pragma unroll
                for (int ks = 0; ks <= (t >> 1); ++ks) {
                    const Op<IO, kPlanes> a[1] = {tri_row<IO, kPlanes>(ts, t >> 1, t & 1, ks, c, q)};
                    mma(z, uy[ks], a);
                }
                yo[t] = narrow<IO>(z[0]);
            }
            if (stop) {     // NaN from that token on, and in the row's state
                const float nan = __builtin_nanf("");
#pragma unroll
                for (int t = 0; t < NT; ++t)
                    if (bad < kC) S[t] = f32x4{nan, nan, nan, nan};
#pragma unroll
                for (int t = 0; t < 4; ++t)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        if (32 * (t >> 1) + 8 * q + 4 * (t & 1) + r >= bad) E[t][r] = nan;
                        if constexpr (RUN)      // y: rows p in registers, 4 q + r
                            if (tile_row(t >> 1, t & 1, c) >= __shfl(bad, 4 * q + r, 64)) set_nan<IO>(yo[t], r);
                    }
            }
        } else {
            ahead(std::integral_constant<int, 2>{});
            ahead(std::integral_constant<int, 3>{});
        }
        if constexpr (T::kBufs == 1) {
            __syncthreads();
            if (ch + 1 < end) {
                fetch_main(ch + 1, lds0);
                fetch_q(ch + 1);
            }
        }
        copies_done();
        take_v();
        __syncthreads();
        // stores last: nothing waits for them before the next chunk's copies
        if (live) {
            if constexpr (SAVE) {
                f32x4 *dst = reinterpret_cast<f32x4 *>(saved.E) + ((size_t(bh) * nc + ch) * ptiles + p0 / 16) * 256 + lane;
#pragma unroll
                for (int t = 0; t < 4; ++t)
                    if (t / (4 / X) == x) dst[64 * t] = E[t];
            } else if constexpr (RUN) {
                const __amdgpu_buffer_rsrc_t view = chunk_view(yg + vy0 + size_t(t0) * hp, rows, tok, P);
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    if (t / (4 / X) != x) continue;
                    const int off = int(uint32_t(tile_row(t >> 1, t & 1, c)) * tok + uint32_t(p0 + 4 * q) * kSz);
                    if constexpr (kSz == 4) __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, yo[t]), view, off, 0, 0);
                    else __builtin_amdgcn_raw_buffer_store_b64(yo[t], view, off, 0, 0);
                }
            }
        }
    }
    if (!SAVE && fin && live && (MAP || seg == segs - 1))
#pragma unroll
        for (int t = 0; t < NT; ++t) *reinterpret_cast<f32x4 *>(fin + state_at(MAP ? unit : bh, MAP ? P + N : P, t)) = S[t];
}

constexpr int kSimds = 1024;

// Calls f(W, X) with the waves per block and per tile for `tiles` chains of 16 state rows.
// A tile is shared by X waves as long as each wave still has one of the 1024 SIMDs to itself
// (the chain waits for its own results, so that two waves on a SIMD cost one of them little,
// but more waves than SIMDs cost every block its exchange).  512 tokens, one group, waves per
// tile before -> after, us of the backward pass at 128, 256, 384, 512 and 640 tiles:
//   bf16, N = 64,  1 -> 2:  86 -> 85, 101 -> 94, 112 -> 105, 124 -> 115, 136 -> 158
//   fp32, N = 64,  1 -> 2:  115 -> 107, 159 -> 136, 177 -> 154, 193 -> 170, 211 -> 241
//   bf16, N = 128, 1 -> 2:  117 -> 105, 132 -> 118, 145 -> 132, 159 -> 147, 173 -> 215
//   bf16, N = 128, 1 -> 4:  117 -> 100, 132 -> 111, 145 -> 173
// and with one tile per block (4, 4) for two (8, 4) at 128, 256 and 384 tiles:
//   fp32, N = 128:  177 -> 145, 217 -> 186, 258 -> 299;   bf16, N = 256:  148 -> 128, 184 -> 165, 220 -> 260
// The forward pass goes the same way (bf16, N = 128, 512 tiles: 70 -> 63, 640: 76 -> 98).
//
// With more tiles than SIMDs, one chunk's buffer instead of two lets a second block onto a CU,
// whose waves fill the waits, where the registers allow it too (the backward pass of wide
// rows has none).  2048 tokens, two buffers -> one, us at 1024, 1280, 2048 and 4096 tiles:
//   bf16, N = 32,  forward:   205 -> 226, 301 -> 281, 406 -> 395, 729 -> 743
//   bf16, N = 64,  forward:   218 -> 240, 331 -> 320, 419 -> 405, 795 -> 760
//   bf16, N = 64,  backward:  669 -> 691, 934 -> 902, 1309 -> 1293, 2547 -> 2571
//   bf16, N = 128, forward:   253 -> 277, 410 -> 383, 513 -> 470, 968 -> 901
//   bf16, N = 128, backward:  842 -> 900, 1210 -> 1189, 1643 -> 1645, 3222 -> 3223 (not done)
//   fp32, N = 64,  forward:   312 -> 338, 522 -> 453, 576 -> 515, 1131 -> 1001
//   fp32, N = 64,  backward:  973 -> 1042, 1425 -> 1341, 1853 -> 1774, 3685 -> 3560 (not done)
template <typename IO, int N, bool BACK, class F>
hipError_t with_chain_shape(int64_t tiles, F &&f) {
    using std::integral_constant;
    constexpr integral_constant<int, 1> one{};
    constexpr integral_constant<int, 2> two{};
    constexpr integral_constant<int, 4> four{};
    [[maybe_unused]] constexpr integral_constant<int, 8> eight{};
    constexpr int kRow = N * int(sizeof(IO));
    [[maybe_unused]] auto alone = [&]() {       // a wave per tile
        constexpr bool kGains = 4 * ChainLds<IO, N, 4, 1, true, false, false>::kMain > 160 * 1024 && (!BACK || kRow <= 128);
        if constexpr (kGains)
            if (tiles > kSimds) return f(four, one, std::true_type{});
        return f(four, one, std::false_type{});
    };
    if constexpr (N == 32) {
        return alone();
    } else if constexpr (N == 64) {
        return tiles <= kSimds / 2 ? f(four, two, std::false_type{}) : alone();
    } else if constexpr (kRow == 256) {
        return tiles <= kSimds / 4 ? f(four, four, std::false_type{}) : tiles <= kSimds / 2 ? f(four, two, std::false_type{}) : alone();
    } else {
        return tiles <= kSimds / 4 ? f(four, four, std::false_type{}) : f(eight, four, std::false_type{});
    }
}

template <typename IO, int N, int W, int X, Chain MODE, bool ONE>
hipError_t launch_chain(const IO *q, const IO *k, const IO *v, const char *images, const float *init, IO *y, float *fin,
                        const DeltaSaved &saved, int b, int L, int H, int P, int G, int per, int segs, float scale, hipStream_t stream) {
    constexpr bool RUN = MODE == Chain::run;
    constexpr int lds = ChainLds<IO, N, W, X, RUN, RUN, ONE>::kBytes;
    const int rows = 16 * W / X, pblocks = ((MODE == Chain::map ? P + N : P) + rows - 1) / rows, nc = (L + kC - 1) / kC;
    auto kern = k_delta_chain<IO, N, W, X, MODE, ONE>;
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void *>(kern), hipFuncAttributeMaxDynamicSharedMemorySize, lds);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(kern, dim3(unsigned(int64_t(b) * H * segs * pblocks)), dim3(64 * W), lds, stream, q, k, v, images, init, y, fin,
                       saved, L, H, P, G, nc, per, segs, pblocks, scale);
    return hipGetLastError();
}

namespace {

// The states at the segments' borders, one after the other.  Block = (batch, head, 16 rows
// of the state), wave w = 16 of its columns, on the fp32 matrix instruction; A is read ahead
// by one segment where there are registers for it.
//   !BACK  S_0 = init_state, S_1 = the first segment's rows, S_{i+1} = S_i A_i + B_i
//   BACK   from the last segment down: dS that leaves segment i - 1 = dS_i A_i^T + D_i; `map`
//          holds the A's as before, `add` the D's [segments][P][N] and `init` is unused
template <int N, bool BACK>
__global__ __launch_bounds__(4 * N) void k_delta_carry(const float *__restrict__ map, const float *__restrict__ add,
                                                       const float *__restrict__ init_state, float *__restrict__ out, int P, int segs) {
    __shared__ __align__(16) float rows[16][N + 4];
    constexpr bool kAhead = N <= 128;
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, c = lane & 15, q = lane >> 4;
    const int pt = blockIdx.x % (P / 16), bh = blockIdx.x / (P / 16), col = 16 * w + c;
    const size_t pn = size_t(P) * N, step = pn + size_t(N) * N, at = size_t(16 * pt + 4 * q) * N + col;
    const float *m = map + size_t(bh) * (segs - 1) * step;
    float *o = out + size_t(bh) * segs * pn + at;
    f32x4 s, a[N / 16], an[kAhead ? N / 16 : 1];
    // a product's k = 16 j + 4 q + r, r = 0 .. 3 in the elements of a[j]
    auto fetch = [&](f32x4 (&to)[N / 16], int seg) {
        const float *A = m + size_t(seg) * step + pn;
#pragma unroll
        for (int j = 0; j < N / 16; ++j) {
            if constexpr (BACK) {
                to[j] = *reinterpret_cast<const f32x4 *>(A + size_t(col) * N + 16 * j + 4 * q);
            } else {
#pragma unroll
                for (int r = 0; r < 4; ++r) to[j][r] = A[(16 * j + 4 * q + r) * N + col];
            }
        }
    };
    auto added = [&](int seg) {     // B or D of a segment
        f32x4 v;
#pragma unroll
        for (int r = 0; r < 4; ++r) v[r] = BACK ? add[(size_t(bh) * segs + seg) * pn + at + r * N] : m[size_t(seg) * step + at + r * N];
        return v;
    };
    auto put = [&](int seg, const f32x4 &v) {
#pragma unroll
        for (int r = 0; r < 4; ++r) o[seg * pn + r * N] = v[r];
    };
    if constexpr (!BACK) {
        f32x4 v = {0.f, 0.f, 0.f, 0.f};
        if (init_state)
#pragma unroll
            for (int r = 0; r < 4; ++r) v[r] = init_state[size_t(bh) * pn + at + r * N];
        put(0, v);
    }
    const int turns = segs - 2;         // the segments 1 .. segs - 2 that are passed through
    auto segment = [&](int i) { return BACK ? segs - 2 - i : i + 1; };
    s = added(BACK ? segs - 1 : 0);
    put(BACK ? segs - 2 : 1, s);
    if (turns > 0) fetch(a, segment(0));
    for (int i = 0; i < turns; ++i) {
        __syncthreads();                // the last product's readers
#pragma unroll
        for (int r = 0; r < 4; ++r) rows[4 * q + r][col] = s[r];
        s = added(segment(i));
        if constexpr (kAhead) fetch(an, segment(min(i + 1, turns - 1)));
        __syncthreads();
        f32x4 odd = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < N / 16; ++j) {
            const f32x4 row = *reinterpret_cast<const f32x4 *>(&rows[c][16 * j + 4 * q]);
            s = mfma_f32(row[0], a[j][0], s);
            odd = mfma_f32(row[1], a[j][1], odd);
            s = mfma_f32(row[2], a[j][2], s);
            odd = mfma_f32(row[3], a[j][3], odd);
        }
        s += odd;
        put(BACK ? segment(i) - 1 : segment(i) + 1, s);
        if constexpr (kAhead) {
#pragma unroll
            for (int j = 0; j < N / 16; ++j) a[j] = an[j];
        } else {
            fetch(a, segment(min(i + 1, turns - 1)));
        }
    }
}

// The states that enter the segments, if there are more than one.
template <typename IO, int N, bool BACK>
hipError_t enter_segments(const IO *q, const IO *k, const IO *v, const char *images, const float *init_state, float *map, float *init, int b,
                          int L, int H, int P, int G, const DeltaCut &cut, float scale, hipStream_t stream) {
    if (cut.segments == 1) return hipSuccess;
    const int64_t bh = int64_t(b) * H;
    auto go = [&](auto w_, auto x_, auto one_) {
        constexpr int W = decltype(w_)::value, X = decltype(x_)::value;
        return launch_chain<IO, N, W, X, Chain::map, decltype(one_)::value>(q, k, v, images, init_state, static_cast<IO *>(nullptr), map, DeltaSaved{}, b,
                                                         L, H, P, G, cut.per, cut.segments - 1, scale, stream);
    };
    const hipError_t e = with_chain_shape<IO, N, BACK>(bh * (cut.segments - 1) * ((P + N) / 16), go);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((k_delta_carry<N, false>), dim3(unsigned(bh * (P / 16))), dim3(4 * N), 0, stream, map, nullptr, init_state, init, P,
                       cut.segments);
    return hipGetLastError();
}

}  // namespace
}  // namespace ssd
