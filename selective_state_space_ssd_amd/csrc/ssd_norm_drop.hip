// ssd_norm_drop.hip -- the residual sum with dropout on what is added, and its norm.
//
//   s = residual + scale m x / (1 - p),   y = s r w,   m = 1 with probability 1 - p, else 0
//
// The mask is a function of the element's place and of the generator's state, so neither
// pass stores it: the kernels of ssd_norm_add.h ask for it where they use x, the backward
// pass once more.  Element i of the flat array takes word i mod 4 of Philox4x32-10 (J.
// Salmon, M. Moraes, R. Dror, D. Shaw, "Parallel random numbers: as easy as 1, 2, 3", SC
// 2011) of the counter (i / 4, offset) under the key `seed`, 64 bits each, and stays where
// that word is at least p 2^32.  Seed and offset are read on the device: a captured step
// that counts the offset on draws another mask in each replay.
//
// The generator hides behind the loads: 8192 rows of 2560 bf16 channels with an fp32 residual
// (252 MB) take 42 us forward, 5.9 TB/s, as without dropout, and 77 backward (377 MB and 11 of
// partial sums), 5.0 TB/s, and 5 more for adding those up; medians of a trace.  (20 wide products
// and about as many other instructions a counter, four elements: 5.3 us of the vector ALU's time
// forward.)
#include "ssd_norm_add.h"

namespace ssd {
namespace {

struct Philox {
    uint32_t c[4];
};

// Ten rounds of two 32 x 32-bit products whose halves cross over.
__device__ __forceinline__ Philox philox(uint64_t counter, uint64_t offset, uint64_t seed) {
    constexpr uint32_t kMul0 = 0xD2511F53u, kMul1 = 0xCD9E8D57u, kKey0 = 0x9E3779B9u, kKey1 = 0xBB67AE85u;
    uint32_t c0 = uint32_t(counter), c1 = uint32_t(counter >> 32), c2 = uint32_t(offset), c3 = uint32_t(offset >> 32);
    uint32_t k0 = uint32_t(seed), k1 = uint32_t(seed >> 32);
#pragma unroll
    for (int r = 0; r < 10; ++r) {
        const uint64_t p = uint64_t(kMul0) * c0, q = uint64_t(kMul1) * c2;
        c0 = uint32_t(q >> 32) ^ c1 ^ k0;
        c2 = uint32_t(p >> 32) ^ c3 ^ k1;
        c1 = uint32_t(q);
        c3 = uint32_t(p);
        k0 += kKey0;
        k1 += kKey1;
    }
    return {{c0, c1, c2, c3}};
}

struct Dropout {
    static constexpr bool kOn = true;
    const uint64_t *rng;        // seed, offset
    uint32_t threshold;         // p 2^32
    float up;                   // 1 / (1 - p)

    __device__ __forceinline__ float factor() const { return up; }

    // VEC = 4 or 8: i is a multiple of VEC, as rows whose length is one begin there.
    template <int VEC>
    __device__ __forceinline__ uint32_t mask(int64_t i) const {
        const uint64_t seed = rng[0], offset = rng[1];
        if constexpr (VEC == 1) {
            const Philox w = philox(uint64_t(i) >> 2, offset, seed);
            const uint32_t lo = (i & 1) ? w.c[1] : w.c[0], hi = (i & 1) ? w.c[3] : w.c[2];
            return ((i & 2) ? hi : lo) >= threshold ? 1u : 0u;
        } else {
            uint32_t bits = 0;
#pragma unroll
            for (int q = 0; q < VEC / 4; ++q) {
                const Philox w = philox((uint64_t(i) >> 2) + q, offset, seed);
#pragma unroll
                for (int j = 0; j < 4; ++j) bits |= (w.c[j] >= threshold ? 1u : 0u) << (4 * q + j);
            }
            return bits;
        }
    }
};

Dropout dropout_of(const NormDropArgs &d) {
    // p < 1 in 32 bits: p 2^32 and 1 - p are exact in 64
    return {d.rng, uint32_t(double(d.p) * 4294967296.0), float(1.0 / (1.0 - double(d.p)))};
}

}  // namespace

hipError_t launch_norm_add_drop_fwd(const NormAddArgs &a, const NormDropArgs &d, hipStream_t stream) {
    return add_fwd_by_type(a, dropout_of(d), stream);
}

hipError_t launch_norm_add_drop_bwd(const NormAddArgs &a, const NormDropArgs &d, const NormBwdPlan &plan, hipStream_t stream) {
    return add_bwd_by_type(a, plan, dropout_of(d), stream);
}

}  // namespace ssd
