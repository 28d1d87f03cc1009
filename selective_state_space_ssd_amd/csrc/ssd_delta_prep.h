// ssd_delta_prep.h -- the part of the chunked gated delta rule that does not depend on the
// state: M and the scores of every chunk (see ssd_delta_chunk.h for the formulas).
//
// One block per (batch, head, chunk).  k_i . k_j and q_i . k_j are matrix products (exact
// operands, fp32 sums).  M solves (I + Lo diag(beta)) M = -Lo: row by row inside the four
// diagonal blocks of 16 (one lane per column), and from there by
//   M21 = -(I + M22 b2) Lo21 (I + b1 M11)
// for the blocks below the diagonal, 16 then 32 wide, on the fp32 matrix instruction.  No
// power of Lo is formed, so keys that repeat do not make the terms grow.
#pragma once

#include "ssd_delta_chunk.h"

namespace ssd {

constexpr int kLd = kC + 1;     // LDS row of the fp32 work matrices

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

// Copy an fp32 lower triangular [64][64] matrix from LDS into its image: NP planes,
// 16-byte chunks placed as the chain's LDS tiles hold them.
template <typename IO, int NP>
__device__ __forceinline__ void write_image(const float *m, char *dst) {
    using Img = ChunkImage<IO, 1, 1>;
    constexpr int kRowTop = 32 * Img::kSz, kRow = 64 * Img::kSz, E = 16 / Img::kSz;
    for (int i = threadIdx.x; i < Img::kPlane / 16; i += 256) {
        const bool top = i < Img::kTop / 16;
        const int at = top ? i : i - Img::kTop / 16, per_row = (top ? kRowTop : kRow) / 16;
        const int r = at / per_row, pos = at % per_row;
        const int col = (pos ^ (top ? place<kRowTop>(r) : place<kRow>(r))) * E;
        const float *s = m + (top ? r : 32 + r) * kLd + col;
        if constexpr (std::is_same_v<IO, float>) {
            *reinterpret_cast<float4 *>(dst + i * 16) = make_float4(s[0], s[1], s[2], s[3]);
        } else {
            const Op<IO, NP> o = to_op<IO, NP>(f32x4{s[0], s[1], s[2], s[3]}, f32x4{s[4], s[5], s[6], s[7]});
#pragma unroll
            for (int p = 0; p < NP; ++p)
                *reinterpret_cast<uint4 *>(dst + p * Img::kPlane + i * 16) = __builtin_bit_cast(uint4, o.p[p]);
        }
    }
}

template <typename IO, int N, int NM, int NQ>
__global__ __launch_bounds__(256) void k_delta_prep(const IO *__restrict__ qg, const IO *__restrict__ kg,
                                                    const float *__restrict__ a, const float *__restrict__ beta,
                                                    char *__restrict__ images, int L, int H, int G, int nc, float scale) {
    using Img = ChunkImage<IO, NM, NQ>;
    __shared__ double gd[kC];
    __shared__ float sb[kC];
    __shared__ float lo[kC * kLd], mm[kC * kLd], sc[kC * kLd], yt[32 * 33];
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6, c = lane & 15, q = lane >> 4;
    const int ch = blockIdx.x % nc, bh = blockIdx.x / nc;
    const int h = bh % H, bi = bh / H, g = h / (H / G);
    const int t0 = ch * kC, valid = min(kC, L - t0);
    char *img = images + size_t(blockIdx.x) * Img::kBytes;

    for (int i = tid; i < kC * kLd; i += 256) lo[i] = mm[i] = sc[i] = 0.f;
    if (w == 0) {
        const size_t at = (size_t(bi) * L + t0 + min(lane, valid - 1)) * H + h;
        double s = lane < valid ? gate(a[at]) : 0.0;
        const float bt = lane < valid ? beta[at] : 0.f;
#pragma unroll
        for (int off = 1; off < 64; off <<= 1) {
            const double o = __shfl_up(s, off, 64);
            if (lane >= off) s += o;
        }
        const double end = __shfl(s, 63, 64);
        gd[lane] = s;
        sb[lane] = bt;
        float *gates = reinterpret_cast<float *>(img + Img::kGates);
        gates[lane] = expf(float(s));
        gates[kC + lane] = expf(float(end - s));
        gates[2 * kC + lane] = bt;
    }
    __syncthreads();

    {   // wave w: rows 16 w .. of both products, columns up to the diagonal
        const size_t ts = size_t(G) * N;
        const size_t base = (size_t(bi) * L + t0) * ts + size_t(g) * N + 8 * q;
        const size_t arow = base + min(16 * w + c, valid - 1) * ts;
        f32x4 kk[4], qk[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) kk[j] = qk[j] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int ks = 0; ks < N / 32; ++ks) {
            const Op<IO, 1> ak = load_row8<IO>(kg + arow + 32 * ks), aq = load_row8<IO>(qg + arow + 32 * ks);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (j > w) break;
                const Op<IO, 1> bk = load_row8<IO>(kg + base + min(16 * j + c, valid - 1) * ts + 32 * ks);
                kk[j] = mma(ak, bk, kk[j]);
                qk[j] = mma(aq, bk, qk[j]);
            }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (j > w) break;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int i = 16 * w + 4 * q + r, jj = 16 * j + c;
                if (jj > i) continue;
                const float d = expf(float(gd[i] - gd[jj]));
                sc[i * kLd + jj] = scale * qk[j][r] * d;
                if (jj < i) lo[i * kLd + jj] = kk[j][r] * d;
            }
        }
    }
    __syncthreads();

    if (w == 0) {   // diagonal blocks of 16: lane = (block q, column c)
        float m[16], bm[16];
        const float *l0 = lo + 16 * q * kLd + 16 * q;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            float v = -l0[i * kLd + c];
#pragma unroll
            for (int k = 0; k < i; ++k) v -= l0[i * kLd + k] * bm[k];
            m[i] = v;
            bm[i] = v * sb[16 * q + i];
        }
#pragma unroll
        for (int i = 1; i < 16; ++i) mm[(16 * q + i) * kLd + 16 * q + c] = m[i];
    }
    __syncthreads();
    if (w < 2) {    // blocks (1, 0) and (3, 2)
        const int r0 = 32 * w + 16, c0 = 32 * w;
        f32x4 y;
#pragma unroll
        for (int r = 0; r < 4; ++r) y[r] = lo[(r0 + 4 * q + r) * kLd + c0 + c];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const int k = c0 + 4 * t + q;
            y = mfma_f32(lo[(r0 + c) * kLd + k], sb[k] * mm[k * kLd + c0 + c], y);
        }
        f32x4 z = y;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int k = r0 + 4 * q + r;
            z = mfma_f32(mm[(r0 + c) * kLd + k], sb[k] * y[r], z);
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) mm[(r0 + 4 * q + r) * kLd + c0 + c] = -z[r];
    }
    write_image<IO, Img::kPlanesQ>(sc, img + Img::kQ);
    __syncthreads();
    {               // rows 32 .. 63, columns 0 .. 31: tile (ti, tj) of wave w
        const int r0 = 32 + 16 * (w >> 1), c0 = 16 * (w & 1);
        f32x4 y;
#pragma unroll
        for (int r = 0; r < 4; ++r) y[r] = lo[(r0 + 4 * q + r) * kLd + c0 + c];
#pragma unroll
        for (int t = 0; t < 8; ++t) {
            const int k = 4 * t + q;
            y = mfma_f32(lo[(r0 + c) * kLd + k], sb[k] * mm[k * kLd + c0 + c], y);
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) yt[(r0 - 32 + 4 * q + r) * 33 + c0 + c] = y[r];
        __syncthreads();
        f32x4 z = y;
#pragma unroll
        for (int t = 0; t < 8; ++t) {
            const int k = 4 * t + q;
            z = mfma_f32(mm[(r0 + c) * kLd + 32 + k], sb[32 + k] * yt[k * 33 + c0 + c], z);
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) mm[(r0 + 4 * q + r) * kLd + c0 + c] = -z[r];
    }
    __syncthreads();
    write_image<IO, Img::kPlanesM>(mm, img + Img::kM);
}

}  // namespace ssd
