// ssd_delta_prep.h -- the part of the chunked gated delta rule that does not depend on the
// state: M and the scores of every chunk (see ssd_delta_chunk.h for the formulas).
//
// One block per chunk and a few heads of a group.  k_i . k_j and q_i . k_j are matrix products (exact
// operands, fp32 sums).  M solves (I + Lo diag(beta)) M = -Lo: row by row inside the four
// diagonal blocks of 16 (one lane per column), and from there by
//   M21 = -(I + M22 b2) Lo21 (I + b1 M11)
// for the blocks below the diagonal, 16 then 32 wide, on the fp32 matrix instruction.  No
// power of Lo is formed, so keys that repeat do not make the terms grow.
//
// 4096 chunks of a head (4 x 2048 tokens, 32 heads in 8 groups, bf16, N = 128) take 45 to
// 48 us and write 154 MB of images, 3.3 TB/s (a fill reaches 7): a head is seven steps between
// barriers, 4 blocks a CU cover for each other, and the waves wait for LDS and barriers 60 % of
// their time.  With registers for 3 blocks it is the same (the forward call 193 us against 196).
#pragma once

#include <algorithm>

#include "ssd_delta_chunk.h"

namespace ssd {

constexpr int kLd = kC + 4;     // LDS row of the fp32 work matrices: 16-byte pieces, rows 4 banks apart

template <typename IO>
__device__ __forceinline__ Op<IO, 1> load_row8(const IO *p) {
    Op<IO, 1> o;
    if constexpr (std::is_same_v<IO, float>) {
        o.v[0] = *reinterpret_cast<const f32x4 *>(p);
        o.v[1] = *reinterpret_cast<const f32x4 *>(p + 4);
    } else {
        o.p[0] = as_bf16x8(*reinterpret_cast<const uint4 *>(p));
    }
    return o;
}

// A value that is not finite comes from a token that spoils all after it, whatever stands
// here, and none before: where it meets the zeros of a triangle it counts as 0.
__device__ __forceinline__ float finite_or_0(float v) { return __builtin_isfinite(v) ? v : 0.f; }

// Copy an fp32 lower triangular [64][64] matrix from LDS into its image: NP planes,
// 16-byte chunks placed as the chain's LDS tiles hold them; by `threads` threads, this one
// the `first`.  FINITE: see finite_or_0.
template <typename IO, int NP, bool FINITE>
__device__ __forceinline__ void write_image(const float *m, char *dst, int first, int threads) {
    using Img = ChunkImage<IO>;
    constexpr int kRowTop = 32 * Img::kSz, kRow = 64 * Img::kSz, E = 16 / Img::kSz;
    for (int i = first; i < Img::kPlane / 16; i += threads) {
        const bool top = i < Img::kTop / 16;
        const int at = top ? i : i - Img::kTop / 16, per_row = (top ? kRowTop : kRow) / 16;
        const int r = at / per_row, pos = at % per_row;
        const int col = (pos ^ (top ? place<kRowTop>(r) : place<kRow>(r))) * E;
        const float *s = m + (top ? r : 32 + r) * kLd + col;
        auto four = [&](int e) {
            f32x4 v = *reinterpret_cast<const f32x4 *>(s + 4 * e);
            if constexpr (FINITE)
#pragma unroll
                for (int j = 0; j < 4; ++j) v[j] = finite_or_0(v[j]);
            return v;
        };
        if constexpr (std::is_same_v<IO, float>) {
            *reinterpret_cast<f32x4 *>(dst + i * 16) = four(0);
        } else {
            const Op<IO, NP> o = to_op<IO, NP>(four(0), four(1));
#pragma unroll
            for (int p = 0; p < NP; ++p)
                *reinterpret_cast<uint4 *>(dst + p * Img::kPlane + i * 16) = __builtin_bit_cast(uint4, o.p[p]);
        }
    }
}

// Heads of a group that one block takes, sharing the products of the group's keys.
constexpr int kPrepHeads = 4;

template <typename IO, int N>
__global__ __launch_bounds__(256, 4) void k_delta_prep(const IO *__restrict__ qg, const IO *__restrict__ kg,
                                                    const float *__restrict__ a, const float *__restrict__ beta,
                                                    char *__restrict__ images, int L, int H, int G, int nc, int hb,
                                                    float scale) {
    using Img = ChunkImage<IO>;
    __shared__ double gd[kPrepHeads][kC];
    __shared__ float sbs[kPrepHeads][kC];
    __shared__ __align__(16) float mm[kC * kLd], sc[kC * kLd];  // Lo, then M over it; scores
    float *yt = sc;                                             // later [32][33] of it
    const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6), c = lane & 15, q = lane >> 4;
    const int r = H / G, hblocks = (r + hb - 1) / hb;
    const int ch = blockIdx.x % nc, hblk = blockIdx.x / nc % hblocks, bg = blockIdx.x / nc / hblocks;
    const int g = bg % G, bi = bg / G;
    const int h0 = g * r + hblk * hb, nh = min(hb, r - hblk * hb);
    const int t0 = ch * kC, valid = min(kC, L - t0);
    auto image = [&](int j) { return images + (size_t(bi * H + h0 + j) * nc + ch) * Img::kBytes; };

    if (w < nh) {       // wave w: the gates of head h0 + w
        const size_t at = (size_t(bi) * L + t0 + min(lane, valid - 1)) * H + h0 + w;
        double s = lane < valid ? gate(a[at]) : 0.0;
        const float bt = lane < valid ? beta[at] : 0.f;
#pragma unroll
        for (int off = 1; off < 64; off <<= 1) {
            const double o = __shfl_up(s, off, 64);
            if (lane >= off) s += o;
        }
        const double end = __shfl(s, 63, 64);
        // a beta that is not finite counts as 0 and makes e^g a NaN: the token's bracket is one then
        const bool ok = __builtin_isfinite(bt);
        gd[w][lane] = s * kPerLn2;
        sbs[w][lane] = ok ? bt : 0.f;
        float *gates = reinterpret_cast<float *>(image(w) + Img::kGates);
        gates[lane] = ok ? expf(float(s)) : __builtin_nanf("");
        gates[kC + lane] = expf(float(end - s));
        gates[2 * kC + lane] = ok ? bt : 0.f;
    }
    // wave w: row tile w of k k^T and row tile 3 - w of q k^T, up to the diagonal (5 tiles)
    f32x4 kk[4], qk[4];
    const int wq = 3 - w;
    {
        const size_t ts = size_t(G) * N;
        const size_t base = (size_t(bi) * L + t0) * ts + size_t(g) * N + 8 * q;
#pragma unroll
        for (int j = 0; j < 4; ++j) kk[j] = qk[j] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int ks = 0; ks < N / 32; ++ks) {
            const Op<IO, 1> ak = load_row8<IO>(kg + base + min(16 * w + c, valid - 1) * ts + 32 * ks);
            const Op<IO, 1> aq = load_row8<IO>(qg + base + min(16 * wq + c, valid - 1) * ts + 32 * ks);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (j > w && j > wq) continue;
                const Op<IO, 1> bk[1] = {load_row8<IO>(kg + base + min(16 * j + c, valid - 1) * ts + 32 * ks)};
                f32x4 one[1];
                if (j <= w) {
                    one[0] = kk[j];
                    mma(one, ak, bk);
                    kk[j] = one[0];
                }
                if (j <= wq) {
                    one[0] = qk[j];
                    mma(one, aq, bk);
                    qk[j] = one[0];
                }
            }
        }
    }
    for (int j = 0; j < nh; ++j) {
        const float *sb = sbs[j];
        char *img = image(j);
        __syncthreads();            // the gates; the last head's matrices are written out
        double gk[4], gq[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            gk[i] = gd[j][16 * w + 4 * q + i];
            gq[i] = gd[j][16 * wq + 4 * q + i];
        }
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const int col = 16 * t + c;
            const double gc = gd[j][col];
            // above the diagonal: zeros, and no decay is taken in the tiles there
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int rk = 16 * w + 4 * q + i;
                mm[rk * kLd + col] = t <= w ? col < rk ? kk[t][i] * decay(gk[i] - gc) : 0.f : 0.f;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int rq = 16 * wq + 4 * q + i;
                sc[rq * kLd + col] = t <= wq ? col <= rq ? scale * qk[t][i] * decay(gq[i] - gc) : 0.f : 0.f;
            }
        }
        __syncthreads();
        if (w > 0) {    // the other waves write the scores out meanwhile
            write_image<IO, kPlanes, false>(sc, img + Img::kQ, tid - 64, 192);
        } else {        // diagonal blocks of 16, lane = (block q, column c): each row found
                        // is taken out of all later ones
            float *l0 = mm + 16 * q * kLd + 16 * q;
            float m[16];
#pragma unroll
            for (int i = 1; i < 16; ++i) m[i] = -l0[i * kLd + c];
#pragma unroll
            for (int k0 = 0; k0 < 16; k0 += 2) {    // 2 columns of Lo in registers at a time
                f32x2 lo[16];
#pragma unroll
                for (int i = k0 + 1; i < 16; ++i) lo[i] = *reinterpret_cast<const f32x2 *>(l0 + i * kLd + k0);
                asm volatile("" ::: "memory");
#pragma unroll
                for (int k = k0 == 0 ? 1 : 0; k < 2; ++k) {
                    const float bm = m[k0 + k] * sb[16 * q + k0 + k];
#pragma unroll
                    for (int i = k0 + k + 1; i < 16; ++i) m[i] -= lo[i][k] * bm;
                }
            }
#pragma unroll
            for (int i = 1; i < 16; ++i) l0[i * kLd + c] = m[i];
        }
        __syncthreads();
        if (w < 2) {    // blocks (1, 0) and (3, 2)
            const int r0 = 32 * w + 16, c0 = 32 * w;
            f32x4 y;
#pragma unroll
            for (int i = 0; i < 4; ++i) y[i] = mm[(r0 + 4 * q + i) * kLd + c0 + c];
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const int k = c0 + 4 * t + q;
                y = mfma_f32(mm[(r0 + c) * kLd + k], sb[k] * mm[k * kLd + c0 + c], y);
            }
            f32x4 z = y;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int k = r0 + 4 * q + i;
                z = mfma_f32(mm[(r0 + c) * kLd + k], finite_or_0(sb[k] * y[i]), z);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) mm[(r0 + 4 * q + i) * kLd + c0 + c] = -z[i];
        }
        __syncthreads();
        {               // rows 32 .. 63, columns 0 .. 31: one tile per wave
            const int r0 = 32 + 16 * (w >> 1), c0 = 16 * (w & 1);
            f32x4 y;
#pragma unroll
            for (int i = 0; i < 4; ++i) y[i] = mm[(r0 + 4 * q + i) * kLd + c0 + c];
#pragma unroll
            for (int t = 0; t < 8; ++t) {
                const int k = 4 * t + q;
                y = mfma_f32(mm[(r0 + c) * kLd + k], sb[k] * mm[k * kLd + c0 + c], y);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) yt[(r0 - 32 + 4 * q + i) * 33 + c0 + c] = y[i];
            __syncthreads();
            f32x4 z = y;
#pragma unroll
            for (int t = 0; t < 8; ++t) {
                const int k = 4 * t + q;
                z = mfma_f32(mm[(r0 + c) * kLd + 32 + k], finite_or_0(sb[32 + k] * yt[k * 33 + c0 + c]), z);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) mm[(r0 + 4 * q + i) * kLd + c0 + c] = -z[i];
        }
        __syncthreads();
        write_image<IO, kPlanes, true>(mm, img + Img::kM, tid, 256);
    }
}

// One launch over all chunks.  A block per chunk, group and kPrepHeads heads where that
// fills the device, per head where it does not.
template <typename IO, int N>
hipError_t launch_delta_prep(const IO *q, const IO *k, const float *a, const float *beta, char *images, int b, int L, int H,
                             int G, float scale, hipStream_t stream) {
    const int nc = (L + kC - 1) / kC, r = H / G;
    const int hb = int64_t(b) * nc * G * ((r + kPrepHeads - 1) / kPrepHeads) >= 512 ? std::min(r, kPrepHeads) : 1;
    const unsigned blocks = unsigned(int64_t(b) * nc * G * ((r + hb - 1) / hb));
    hipLaunchKernelGGL((k_delta_prep<IO, N>), dim3(blocks), dim3(256), 0, stream, q, k, a, beta, images, L, H, G, nc, hb, scale);
    return hipGetLastError();
}

}  // namespace ssd
