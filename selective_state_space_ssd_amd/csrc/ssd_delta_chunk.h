// ssd_delta_chunk.h -- device building blocks of the chunked gated delta rule.
//
// The rule over a chunk of C = 64 tokens, with g_i the running sum of a inside the chunk
// and S the state that enters it (per head; rows p of S never meet):
//   D_ij = e^{g_i - g_j},  Lo = the strictly lower part of (k_i . k_j) D_ij
//   M = -(I + Lo diag(beta))^-1 Lo                       (strictly lower)
//   R = V - e^g (K S^T),   E = R + M (beta R),   U = beta E
//   Y = scale (e^g Q S^T + [(q_i . k_j) D_ij, j <= i] U)
//   S <- e^{g_C} S + U^T (e^{g_C - g} K)
// E holds the bracket v - S' k of every token, U what each token adds.  M and the scores
// do not depend on the state: one kernel forms them for all chunks at once.  What is left
// is a chain over the chunks, which each wave runs for 16 rows p of its own.
//
// Matrix tiles (16 x 16, wave64; lane l: c = l & 15, q = l >> 4).  The columns of a chain
// wave's tiles are its 16 rows p.  An accumulator element r of lane (q, c) is row 4 q + r;
// an operand holds 8 consecutive values of the summed index, 8 q .. 8 q + 7, per block of
// 32.  So that an accumulator can be the next product's operand without leaving its lanes,
// the rows of the two tiles (e = 0, 1) of a block of 32 are numbered
//   row m of tile e  <->  index 8 (m >> 2) + 4 e + (m & 3),
// whence lane q's accumulators of the two tiles are exactly indices 8 q .. 8 q + 7.  The
// other operand's rows are read from LDS in that order, which costs nothing.
#pragma once

#include "ssd_device.h"

namespace ssd {

constexpr int kC = 64;      // tokens per chunk

// A gate sum of -infinity would make differences of sums NaN; from -1e5 on a decay is 0
// in any case, and the sums (in 64 bits) keep the digits of the small ones beside it.
__device__ __forceinline__ double gate(float a) { return a < -1e5f ? -1e5 : double(a); }

// The decay of a difference of gate sums that are kept in units of ln 2: one exp2 of the
// hardware (one unit in the last place) where e^x takes a dozen instructions; the difference
// loses what it loses in rounding to 32 bits either way.  Below 2^-126 it is 0.
constexpr double kPerLn2 = 1.4426950408889634;
__device__ __forceinline__ float decay(double x) { return __builtin_amdgcn_exp2f(float(x)); }

// LDS tiles: rows of RB bytes in chunks of 16; chunk `ch` of row r lies at ch ^ place(r).
// A 128-bit read serves 16 lanes a cycle, lanes {0-3, 12-15, 20-27} and {4-11, 16-19,
// 28-31} and the same 32 further on, from 64 banks; a 64-bit read the 32 lanes of a half.
// These placements, found by a search over the maps that are linear in the row's bits,
// give 16 different 16-byte columns to each such group of a row read (rows tile_row(.),
// or consecutive ones) and at most two lanes a column to a transposing read, which only
// ever uses one half of each column.
template <int RB>
__host__ __device__ constexpr __forceinline__ int place(int r) {
    if constexpr (RB >= 256) return (r & 1) ^ ((r & 2) << 1) ^ ((r & 4) >> 1) ^ ((r & 8) | ((r & 8) >> 3)) ^ ((r & 16) >> 3);
    else if constexpr (RB == 128) return ((r & 2) >> 1) ^ ((r & 4) >> 1) ^ ((r & 8) >> 1) ^ ((r & 16) >> 3);
    else return (r & 8) >> 2;
}

// Workgroups go round the 8 XCDs in launch order; this numbers them so that neighbours run
// on one XCD and find what they share in its L2.
__device__ __forceinline__ int xcd_neighbours() {
    constexpr int kXcds = 8;
    const int n = gridDim.x, x = blockIdx.x % kXcds;
    return x * (n / kXcds) + min(x, n % kXcds) + blockIdx.x / kXcds;
}

// The tile row of lane c: index 32 s + 8 (c >> 2) + 4 e + (c & 3).
__device__ __forceinline__ int tile_row(int s, int e, int c) { return 32 * s + 8 * (c >> 2) + 4 * e + (c & 3); }

// An operand: 8 consecutive values of the summed index per lane.  Matrix products run on
// bf16; a 32-bit value goes in as NP planes, each the rounding of what the ones before it
// left (8 bits a plane).  Products of planes i + j >= max planes are below the last
// plane's rounding and left out.  fp32 I/O uses the fp32 matrix instruction instead.
template <typename IO, int NP>
struct Op {
    bf16x8 p[NP];
};
template <int NP>
struct Op<float, NP> {
    f32x4 v[2];
};

// acc[t] += A[t] B for the NT tiles of a step (or A B[t]: products commute lane by lane).
// Tiles innermost: a product waits for the one before it in the same accumulator, so the
// tiles take turns.  Small terms first.
template <int NT, int NA, int NB>
__device__ __forceinline__ void mma(f32x4 (&acc)[NT], const Op<bf16_bits, NA> (&a)[NT], const Op<bf16_bits, NB> &b) {
    constexpr int NM = NA > NB ? NA : NB;
#pragma unroll
    for (int i = NA - 1; i >= 0; --i)
#pragma unroll
        for (int j = NB - 1; j >= 0; --j)
            if (i + j < NM)
#pragma unroll
                for (int t = 0; t < NT; ++t) acc[t] = mfma_bf16(a[t].p[i], b.p[j], acc[t]);
}
template <int NT, int NA, int NB>
__device__ __forceinline__ void mma(f32x4 (&acc)[NT], const Op<float, NA> (&a)[NT], const Op<float, NB> &b) {
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int t = 0; t < NT; ++t) acc[t] = mfma_f32(a[t].v[e][r], b.v[e][r], acc[t]);
}
template <int NT, int NA, int NB>
__device__ __forceinline__ void mma(f32x4 (&acc)[NT], const Op<bf16_bits, NA> &a, const Op<bf16_bits, NB> (&b)[NT]) {
    constexpr int NM = NA > NB ? NA : NB;
#pragma unroll
    for (int i = NA - 1; i >= 0; --i)
#pragma unroll
        for (int j = NB - 1; j >= 0; --j)
            if (i + j < NM)
#pragma unroll
                for (int t = 0; t < NT; ++t) acc[t] = mfma_bf16(a.p[i], b[t].p[j], acc[t]);
}
template <int NT, int NA, int NB>
__device__ __forceinline__ void mma(f32x4 (&acc)[NT], const Op<float, NA> &a, const Op<float, NB> (&b)[NT]) {
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int t = 0; t < NT; ++t) acc[t] = mfma_f32(a.v[e][r], b[t].v[e][r], acc[t]);
}

// A constant in a scalar register.  The bf16 pair (0, -1) has the bits of fp32 -1, which
// the compiler takes for an inline constant that the instruction reads as (-1, 0).
__device__ __forceinline__ bf16x2 pair_constant(uint32_t bits) {
    uint32_t v;
    asm("s_mov_b32 %0, %1" : "=s"(v) : "n"(bits));
    return __builtin_bit_cast(bf16x2, v);
}

// v minus the low / high bf16 of a packed pair, exact (the pair holds v's own rounding in
// that half): one two-term dot product instead of a widening and a subtraction.
__device__ __forceinline__ float minus_lo(float v, uint32_t pair) {
    return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, pair), pair_constant(0x0000bf80u), v, false);
}
__device__ __forceinline__ float minus_hi(float v, uint32_t pair) {
    return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, pair), pair_constant(0xbf800000u), v, false);
}

// The operand of 8 fp32 values (indices 8 q .. 8 q + 7: two accumulators).
template <typename IO, int NP>
__device__ __forceinline__ Op<IO, NP> to_op(f32x4 lo, f32x4 hi) {
    Op<IO, NP> o;
    if constexpr (std::is_same_v<IO, float>) {
        o.v[0] = lo;
        o.v[1] = hi;
    } else {
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            const uint4 w = make_uint4(pack_bf16x2(lo[0], lo[1]), pack_bf16x2(lo[2], lo[3]),
                                       pack_bf16x2(hi[0], hi[1]), pack_bf16x2(hi[2], hi[3]));
            o.p[i] = as_bf16x8(w);
            if (i + 1 < NP) {
                lo = f32x4{minus_lo(lo[0], w.x), minus_hi(lo[1], w.x), minus_lo(lo[2], w.y), minus_hi(lo[3], w.y)};
                hi = f32x4{minus_lo(hi[0], w.z), minus_hi(hi[1], w.z), minus_lo(hi[2], w.w), minus_hi(hi[3], w.w)};
            }
        }
    }
    return o;
}

// Row `row` of a tile, values 8 (4 ks + q) .. + 7, from NP planes `stride` bytes apart.
template <typename IO, int NP, int RB>
__device__ __forceinline__ Op<IO, NP> read_row(const char *tile, int stride, int row, int ks, int q) {
    Op<IO, NP> o;
    const int x = place<RB>(row);
    const char *r = tile + row * RB;
    if constexpr (std::is_same_v<IO, float>) {
#pragma unroll
        for (int e = 0; e < 2; ++e) o.v[e] = *reinterpret_cast<const f32x4 *>(r + (((8 * ks + 2 * q + e) ^ x) * 16));
    } else {
#pragma unroll
        for (int i = 0; i < NP; ++i) o.p[i] = as_bf16x8(*reinterpret_cast<const uint4 *>(r + i * stride + (((4 * ks + q) ^ x) * 16)));
    }
    return o;
}

// Two transposing reads of 4 values each.
__device__ __forceinline__ bf16x8 read_tr8(const char *lo, const char *hi) {
    typedef short s16x4 __attribute__((ext_vector_type(4)));
    const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4 *)(lo));
    const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4 *)(hi));
    return __builtin_bit_cast(bf16x8, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
}

// Column n0 + tile_row(0, e, c) of a tile (n0 a multiple of 32), rows k0 + 8 q .. + 7:
// for bf16 two transposing reads of a 4 x 16 block each, in which lane c of a group of 16
// addresses row c >> 2, columns 4 (c & 3) .. + 3, and receives column c of the 4 rows.
template <typename IO, int NP, int RB>
__device__ __forceinline__ Op<IO, NP> read_col(const char *tile, int stride, int k0, int n0, int e, int c, int q) {
    Op<IO, NP> o;
    if constexpr (std::is_same_v<IO, float>) {
        const int n = n0 + tile_row(0, e, c);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int row = k0 + 8 * q + j;
            o.v[j >> 2][j & 3] = *reinterpret_cast<const float *>(tile + row * RB + (((n >> 2) ^ place<RB>(row)) * 16) + (n & 3) * 4);
        }
    } else {
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            const char *at[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int row = k0 + 8 * q + 4 * j + (c >> 2);
                at[j] = tile + i * stride + row * RB + (((n0 / 8 + (c & 3)) ^ place<RB>(row)) * 16) + 8 * e;
            }
            o.p[i] = read_tr8(at[0], at[1]);
        }
    }
    return o;
}

// Copy 16 bytes per lane from global memory (base + off, base the same for the whole wave)
// into LDS without passing through registers: lane l's go to LDS byte dst + 16 l.  Written
// in assembly because the compiler waits for every such copy at the next LDS read,
// whichever buffer that reads; here the copy into the other buffer stays in flight until
// copies_done().  It has no output register; the wait states cover an M0 or an address
// pair written just before.  M0 is a reserved register, which a list of clobbers cannot
// name: nothing else in the kernels that copy this way uses it.
__device__ __forceinline__ void copy16(const void *base, uint32_t off, uint32_t dst) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tglobal_load_lds_dwordx4 %1, %2"
                 :: "s"(dst), "v"(off), "s"(base) : "memory");
}

// Every copy16 (and load and store) of this wave has arrived: vmcnt 0, the other counters
// left alone.  A block barrier after it makes the copies of all waves readable.
__device__ __forceinline__ void copies_done() { __builtin_amdgcn_s_waitcnt(0x0f70); }

__device__ __forceinline__ uint32_t lds_address(const char *p) {
    return uint32_t(reinterpret_cast<uintptr_t>((const __attribute__((address_space(3))) char *)p));
}

// Planes of the values that stay 32-bit on their way through the bf16 matrix products (24
// bits): the state, what is added to it, M, the vectors M meets, and the scores.  y too, though
// it is rounded to bf16 in the end: where the chunk's updates erase a large state, or keys
// repeat, its terms are much larger than it is.  With 16 bits of state, scores and updates y
// was off by 2^-18 of those terms, and 1.2e-4 of the layer's y (2-norm) fell on the other side
// of a rounding border than the exact value.
constexpr int kPlanes = 3;

// One chunk's image in the workspace and in LDS:
//   M in kPlanes planes (fp32 I/O: one fp32 plane), lower triangular: a plane holds rows
//   0 .. 31 of columns 0 .. 31, then rows 32 .. 63 whole; then [3][64] fp32: e^g,
//   e^{g_C - g}, beta; then the scores, like M.
template <typename IO>
struct ChunkImage {
    static constexpr int kSz = int(sizeof(IO));
    static constexpr int kTop = 32 * 32 * kSz, kPlane = kTop + 32 * 64 * kSz;
    static constexpr int kOf = kSz == 4 ? 1 : kPlanes;      // planes a matrix has
    static constexpr int kM = 0, kGates = kOf * kPlane, kQ = kGates + 1024;     // the gates rounded up to 1 KiB
    static constexpr int kBytes = kQ + kOf * kPlane;
};

// Operands from a lower triangular matrix of an image, blocks of 32: rows tile_row(s, e, c),
// columns 32 ks + 8 q .. (ks <= s);
template <typename IO, int NP>
__device__ __forceinline__ Op<IO, NP> tri_row(const char *m, int s, int e, int ks, int c, int q) {
    using Img = ChunkImage<IO>;
    if (s == 0) return read_row<IO, NP, 32 * Img::kSz>(m, Img::kPlane, tile_row(0, e, c), 0, q);
    return read_row<IO, NP, 64 * Img::kSz>(m + Img::kTop, Img::kPlane, tile_row(0, e, c), ks, q);
}
// columns tile_row(s, e, c), rows 32 ks + 8 q .. (ks >= s).
template <typename IO, int NP>
__device__ __forceinline__ Op<IO, NP> tri_col(const char *m, int ks, int s, int e, int c, int q) {
    using Img = ChunkImage<IO>;
    if (ks == 0) return read_col<IO, NP, 32 * Img::kSz>(m, Img::kPlane, 0, 0, e, c, q);
    return read_col<IO, NP, 64 * Img::kSz>(m + Img::kTop, Img::kPlane, 0, 32 * s, e, c, q);
}

}  // namespace ssd
