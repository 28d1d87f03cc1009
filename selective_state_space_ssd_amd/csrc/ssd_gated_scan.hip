// ssd_gated_scan.hip -- the gated scan over whole sequences, and its gradients.
//
//   h_t = alpha_t h_{t-1} + u_t,  y_t = h_t       (the gate: ssd_gated_scan_gate.h)
//
// Gradients, with g_t what reaches h_t from later tokens (g_L = d_final) and lam_t = dy_t + g_t:
//   g_{t-1} = alpha_t lam_t,  d_init = g_0
//   log decay:  dx_t = lam_t,        da_t = lam_t alpha_t h_{t-1}
//   sigmoid:    dx_t = beta_t lam_t, da_t = lam_t alpha_t beta_t (h_{t-1} - x_t)
// h_{t-1} is stepped again from the states that the forward pass kept.
//
// Each pass reads its inputs once.  A wave holds T tokens of 64 V channels, a lane V
// neighbouring channels; a block's W waves follow each other in time (the gradient's the
// other way round), and so do the blocks of a strip of channels.  What a stretch of tokens
// does to a state is one pair, h -> P h + S, per channel: a wave forms its pair, folds those
// of the waves before it, and steps its tokens a second time from the state that enters.
// From block to block:
//   - the last wave publishes the block's pair as soon as it has it,
//   - every wave waits for the pair of one of the W blocks before, and looks whether that
//     block's outgoing state is there too,
//   - all fold the pairs behind the nearest such state, one by one, into the entering state
//     (the same operations in the same order whichever block that was, so results repeat),
//   - the last wave publishes the outgoing state.
// Blocks take their places from a counter, earlier stretches first, so whatever a block
// waits for belongs to a block that is running already.  A pair or a state is one 8-byte
// word, written at once and never zero; zero means not there yet.
#include <limits.h>

#include "ssd_gated_scan.h"
#include "ssd_gated_scan_gate.h"
#include "ssd_kernels.h"

namespace ssd {
namespace {

constexpr int kT = kGatedScanKeep;  // tokens of a wave
constexpr int kW = 8;               // waves of a block
constexpr int kSpins = 1 << 20;     // looks at a word before a wait gives up (about a second)

// ------------------------------------------------------------- V channels of a lane
template <typename T, int V>
struct Raw;
template <> struct Raw<bf16_bits, 1> { uint16_t r; __device__ float get(int) const { return bf16_to_f32(r); } };
template <> struct Raw<bf16_bits, 2> { uint32_t r; __device__ float get(int j) const { return j ? bf16_hi(r) : bf16_lo(r); } };
template <> struct Raw<float, 1> { float r; __device__ float get(int) const { return r; } };
template <> struct Raw<float, 2> { float2 r; __device__ float get(int j) const { return j ? r.y : r.x; } };

template <typename T, int V>
__device__ __forceinline__ Raw<T, V> raw_of(const float (&f)[V]) {
    Raw<T, V> o;
    if constexpr (V == 1) o.r = from_f32<T>(f[0]);
    else if constexpr (std::is_same_v<T, float>) o.r = make_float2(f[0], f[1]);
    else o.r = pack_bf16x2(f[0], f[1]);
    return o;
}

template <typename T, int V>
__device__ __forceinline__ Raw<T, V> raw_same(float f) {
    const float v[2] = {f, f};
    return raw_of<T, V>(reinterpret_cast<const float (&)[V]>(v));
}

// Rows [0, kT) of a stretch of n tokens; those past it repeat the last.  `p` is at the lane's
// channels of the first row.
template <typename T, int V>
__device__ __forceinline__ void load_rows(const T *p, size_t D, int n, Raw<T, V> (&out)[kT]) {
#pragma unroll
    for (int t = 0; t < kT; ++t)
        out[t] = *reinterpret_cast<const Raw<T, V> *>(p + size_t(n == kT ? t : min(t, n - 1)) * D);
}

// ----------------------------------------------------------------- pairs and their words
// The decay of two stretches after each other, in the form of ssd_gated_scan_gate.h.
__device__ __forceinline__ float both_decays(float m1, float m2) {
    const float a = alpha_of(m1) * alpha_of(m2), b1 = beta_of(m1), b2 = beta_of(m2);
    const float b = fmaf(b1, 1.f - b2, b2);
    return a > 0.5f && b > 0.f ? -b : a;
}

// The decay of the tokens of a stretch, taken one by one.  Near 1 from the sum of what each
// takes away (log decay: of a itself), below from the product: the sum of a log decay that
// erases with many small ones rounds those to the erasing one's last bits.
template <bool SIGMOID>
struct Decay {
    float alpha = 1.f, lost = 0.f;      // lost: 1 - alpha (sigmoid), the sum of a (log decay)
    __device__ __forceinline__ void token(float m, float a) {
        alpha *= alpha_of(m);
        if constexpr (SIGMOID) lost = fmaf(beta_of(m), 1.f - lost, lost);
        else lost += a;
    }
    __device__ __forceinline__ float m() const {
        if constexpr (SIGMOID) return alpha > 0.5f && lost > 0.f ? -lost : alpha;
        else return lost > -1.f ? gate_of<false>(lost) : alpha;
    }
};

typedef unsigned long long word_t;

// Never zero: the complement of two floats of which the first is not all ones.
__device__ __forceinline__ word_t word_of(float first, float second) {
    const uint32_t f = first == first ? __float_as_uint(first) : 0x7fc00000u;
    return ~(word_t(f) << 32 | __float_as_uint(second));
}
__device__ __forceinline__ float first_of(word_t w) { return __uint_as_float(uint32_t(~w >> 32)); }
__device__ __forceinline__ float second_of(word_t w) { return __uint_as_float(uint32_t(~w)); }

__device__ __forceinline__ word_t look(const word_t *p) { return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); }
__device__ __forceinline__ void publish(word_t *p, word_t w) { __hip_atomic_store(p, w, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); }

// Workspace: the counter (16 bytes), then per block 64 V words of its pair and 64 V of its
// outgoing state.
struct Tiles {
    word_t *words;          // null: one block a strip, nothing to wait for
    unsigned *counter;
    int strips, segs, b;
};

template <int V>
__device__ __forceinline__ word_t *words_of(const Tiles &s, int bi, int seg, int strip) {
    return s.words + ((size_t(seg) * s.b + bi) * s.strips + strip) * (2 * 64 * V);
}

// Whether all V words of every lane are there.
template <int V>
__device__ __forceinline__ bool all_there(const word_t (&w)[V]) {
    bool there = true;
#pragma unroll
    for (int j = 0; j < V; ++j) there = there && w[j] != 0;
    return __all(there);
}

template <int V>
__device__ __forceinline__ bool look_all(const word_t *p, word_t (&w)[V]) {
#pragma unroll
    for (int j = 0; j < V; ++j) w[j] = look(p + j);
    return all_there<V>(w);
}

template <int V>
struct ChainLds {
    float2 pair[kW][64 * V];        // of the block's waves
    float2 before[kW][64 * V];      // of the blocks before: pair, or (., outgoing state)
    int state[kW];                  // whether it is a state
    unsigned place;
};

// The state that enters a wave's tokens.  `wave` counts in the order of the scan; m and s are
// the pair of the wave's tokens, `start` the state before the first block.
template <int V>
__device__ __forceinline__ void enter(const Tiles &tiles, ChainLds<V> &lds, int bi, int seg, int strip, int wave, int lane,
                                      const float (&m)[V], const float (&s)[V], const float (&start)[V], float (&h)[V]) {
#pragma unroll
    for (int j = 0; j < V; ++j) lds.pair[wave][lane * V + j] = make_float2(m[j], s[j]);
    __syncthreads();
    float pm[V], ps[V];             // of the waves before
#pragma unroll
    for (int j = 0; j < V; ++j) { pm[j] = 1.f; ps[j] = 0.f; }
    for (int k = 0; k < wave; ++k)
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const float2 p = lds.pair[k][lane * V + j];
            pm[j] = both_decays(pm[j], p.x);
            ps[j] = step_state(p.x, ps[j], p.y);
        }
    if (tiles.segs == 1) {
#pragma unroll
        for (int j = 0; j < V; ++j) h[j] = step_state(pm[j], start[j], ps[j]);
        return;
    }
    word_t *own = words_of<V>(tiles, bi, seg, strip) + lane * V;
    float bm[V], bs[V];             // of the block
    if (wave == kW - 1) {
#pragma unroll
        for (int j = 0; j < V; ++j) {
            bm[j] = both_decays(pm[j], m[j]);
            bs[j] = step_state(m[j], ps[j], s[j]);
            publish(own + j, word_of(bm[j], bs[j]));
        }
    }
    const int n = min(kW, seg);     // blocks before that are looked at
    const int back = kW - wave;     // this wave's: 1 is the nearest
    bool lost = false;
    if (back <= n) {
        const word_t *p = words_of<V>(tiles, bi, seg - back, strip) + lane * V;
        word_t w[V], o[V];
        int spins = 0;
        while (!look_all<V>(p, w) && ++spins < kSpins) __builtin_amdgcn_s_sleep(1);
        const bool state = look_all<V>(p + 64 * V, o);
        lost = spins >= kSpins;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const word_t v = state ? o[j] : w[j];
            lds.before[back - 1][lane * V + j] = make_float2(first_of(v), lost ? __uint_as_float(0x7fc00000u) : second_of(v));
        }
        if (lane == 0) lds.state[back - 1] = state;
    }
    __syncthreads();
    float in[V];
    int k = 0;                      // the nearest state
    while (k < n && !lds.state[k]) ++k;
    if (seg == 0) {
#pragma unroll
        for (int j = 0; j < V; ++j) in[j] = start[j];
    } else if (k < n) {
#pragma unroll
        for (int j = 0; j < V; ++j) in[j] = lds.before[k][lane * V + j].y;
    } else {                        // none yet: the furthest one's
        const word_t *p = words_of<V>(tiles, bi, seg - n, strip) + 64 * V + lane * V;
        word_t o[V];
        int spins = 0;
        while (!look_all<V>(p, o) && ++spins < kSpins) __builtin_amdgcn_s_sleep(1);
        k = n - 1;
#pragma unroll
        for (int j = 0; j < V; ++j) in[j] = spins < kSpins ? second_of(o[j]) : __uint_as_float(0x7fc00000u);
    }
    for (int i = k - 1; i >= 0; --i)
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const float2 p = lds.before[i][lane * V + j];
            in[j] = step_state(p.x, in[j], p.y);
        }
    if (wave == kW - 1)
#pragma unroll
        for (int j = 0; j < V; ++j) publish(own + 64 * V + j, word_of(0.f, step_state(bm[j], in[j], bs[j])));
#pragma unroll
    for (int j = 0; j < V; ++j) h[j] = step_state(pm[j], in[j], ps[j]);
}

// A block's place: strip fastest, then the batch row, then the stretch of the sequence.
template <int V>
__device__ __forceinline__ void place_of(const Tiles &tiles, ChainLds<V> &lds, int &bi, int &seg, int &strip) {
    unsigned p = blockIdx.x;
    if (tiles.segs > 1) {
        if (threadIdx.x == 0) lds.place = atomicAdd(tiles.counter, 1u);
        __syncthreads();
        p = __builtin_amdgcn_readfirstlane(lds.place);
    }
    strip = int(p % unsigned(tiles.strips));
    const unsigned q = p / unsigned(tiles.strips);
    bi = int(q % unsigned(tiles.b));
    seg = int(q / unsigned(tiles.b));
}

// --------------------------------------------------------------------------- forward
template <typename IO, typename AIO, bool SIGMOID, int V>
__global__ __launch_bounds__(64 * kW) void k_gated_scan_fwd(const IO *__restrict__ x, const AIO *__restrict__ a,
                                                            const float *__restrict__ init_state, IO *__restrict__ y,
                                                            float *__restrict__ kept, float *__restrict__ final_state,
                                                            int L, int D, Tiles tiles) {
    __shared__ ChainLds<V> lds;
    int bi, seg, strip;
    place_of<V>(tiles, lds, bi, seg, strip);
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int c = strip * 64 * V + lane * V;
    const bool on = c < D;                  // V divides D
    const int cl = on ? c : 0;
    const int t0 = (seg * kW + wave) * kT, n = min(kT, L - t0);     // n <= 0: past the end
    const size_t row = size_t(bi) * L + t0;

    Raw<IO, V> xr[kT];
    float m[kT][V], pm[V], ps[V];
    if (n > 0) {
        Raw<AIO, V> ar[kT];
        load_rows<AIO, V>(a + row * D + cl, D, n, ar);
        load_rows<IO, V>(x + row * D + cl, D, n, xr);
        if (n < kT) {                       // tokens that leave the state as it is
#pragma unroll
            for (int t = 0; t < kT; ++t)
                if (t >= n) {
                    ar[t] = raw_same<AIO, V>(SIGMOID ? __builtin_inff() : 0.f);
                    xr[t] = raw_same<IO, V>(0.f);
                }
        }
#pragma unroll
        for (int j = 0; j < V; ++j) {
            Decay<SIGMOID> d;
            float s = 0.f;
#pragma unroll
            for (int t = 0; t < kT; ++t) {
                const float av = ar[t].get(j);
                m[t][j] = gate_of<SIGMOID>(av);
                d.token(m[t][j], av);
                s = step_state(m[t][j], s, entering<SIGMOID>(m[t][j], xr[t].get(j)));
            }
            pm[j] = d.m();
            ps[j] = s;
        }
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j) { pm[j] = 1.f; ps[j] = 0.f; }
    }
    float start[V], h[V];
#pragma unroll
    for (int j = 0; j < V; ++j) start[j] = init_state ? init_state[size_t(bi) * D + cl + j] : 0.f;
    enter<V>(tiles, lds, bi, seg, strip, wave, lane, pm, ps, start, h);
    if (n <= 0 || !on) return;
    if (kept) {
        float *k = kept + (size_t(bi) * ((unsigned(L) + kT - 1) / kT) + t0 / kT) * D + c;
#pragma unroll
        for (int j = 0; j < V; ++j) k[j] = h[j];
    }
#pragma unroll
    for (int t = 0; t < kT; ++t) {
#pragma unroll
        for (int j = 0; j < V; ++j) h[j] = step_state(m[t][j], h[j], entering<SIGMOID>(m[t][j], xr[t].get(j)));
        if (y && t < n) *reinterpret_cast<Raw<IO, V> *>(y + (row + t) * D + c) = raw_of<IO, V>(h);
    }
    if (final_state && t0 + n == L)
#pragma unroll
        for (int j = 0; j < V; ++j) final_state[size_t(bi) * D + c + j] = h[j];
}

// -------------------------------------------------------------------------- backward
// The order of the scan is that of the tokens backwards: segment and wave 0 are the last.
template <typename IO, typename AIO, bool SIGMOID, int V>
__global__ __launch_bounds__(64 * kW) void k_gated_scan_bwd(const IO *__restrict__ x, const AIO *__restrict__ a,
                                                            const float *__restrict__ kept, const IO *__restrict__ dy,
                                                            const float *__restrict__ d_final, IO *__restrict__ dx,
                                                            AIO *__restrict__ da, float *__restrict__ d_init, int L,
                                                            int D, Tiles tiles) {
    __shared__ ChainLds<V> lds;
    int bi, seg, strip;
    place_of<V>(tiles, lds, bi, seg, strip);
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int c = strip * 64 * V + lane * V;
    const bool on = c < D;
    const int cl = on ? c : 0;
    const int t0 = ((tiles.segs - 1 - seg) * kW + kW - 1 - wave) * kT, n = min(kT, L - t0);
    const size_t row = size_t(bi) * L + t0;

    Raw<IO, V> xr[kT], gr[kT];
    float m[kT][V], before[kT][V], pm[V], ps[V];
    if (n > 0) {
        Raw<AIO, V> ar[kT];
        load_rows<AIO, V>(a + row * D + cl, D, n, ar);
        load_rows<IO, V>(dy + row * D + cl, D, n, gr);
        load_rows<IO, V>(x + row * D + cl, D, n, xr);
        if (n < kT) {
#pragma unroll
            for (int t = 0; t < kT; ++t)
                if (t >= n) {
                    ar[t] = raw_same<AIO, V>(SIGMOID ? __builtin_inff() : 0.f);
                    gr[t] = xr[t] = raw_same<IO, V>(0.f);
                }
        }
        const float *k = kept + (size_t(bi) * ((unsigned(L) + kT - 1) / kT) + t0 / kT) * D + cl;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            Decay<SIGMOID> d;
            float g = 0.f;
#pragma unroll
            for (int t = kT - 1; t >= 0; --t) {
                const float av = ar[t].get(j);
                m[t][j] = gate_of<SIGMOID>(av);
                d.token(m[t][j], av);
                g = step_state(m[t][j], gr[t].get(j) + g, 0.f);
            }
            pm[j] = d.m();
            ps[j] = g;
            float h = k[j];
#pragma unroll
            for (int t = 0; t < kT; ++t) {
                before[t][j] = h;
                h = step_state(m[t][j], h, entering<SIGMOID>(m[t][j], xr[t].get(j)));
            }
        }
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j) { pm[j] = 1.f; ps[j] = 0.f; }
    }
    float start[V], g[V];
#pragma unroll
    for (int j = 0; j < V; ++j) start[j] = d_final ? d_final[size_t(bi) * D + cl + j] : 0.f;
    enter<V>(tiles, lds, bi, seg, strip, wave, lane, pm, ps, start, g);
    if (n <= 0 || !on) return;
#pragma unroll
    for (int t = kT - 1; t >= 0; --t) {
        if (t >= n) continue;
        float ox[V], oa[V];
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const float lam = gr[t].get(j) + g[j];
            g[j] = step_state(m[t][j], lam, 0.f);
            ox[j] = SIGMOID ? beta_of(m[t][j]) * lam : lam;
            oa[j] = SIGMOID ? g[j] * beta_of(m[t][j]) * (before[t][j] - xr[t].get(j)) : g[j] * before[t][j];
        }
        *reinterpret_cast<Raw<IO, V> *>(dx + (row + t) * D + c) = raw_of<IO, V>(ox);
        *reinterpret_cast<Raw<AIO, V> *>(da + (row + t) * D + c) = raw_of<AIO, V>(oa);
    }
    if (d_init && t0 == 0)
#pragma unroll
        for (int j = 0; j < V; ++j) d_init[size_t(bi) * D + c + j] = g[j];
}

// ---------------------------------------------------------------------------- launches
// Channels of a lane: two bf16 in one 4-byte access where the rows allow it.
int lane_channels(int D, bool bf16) { return bf16 && D % 2 == 0 ? 2 : 1; }

struct Shape {
    int V;
    int64_t strips, segs, blocks;
};

Shape shape_of(int b, int L, int D, bool bf16) {
    Shape s;
    s.V = lane_channels(D, bf16);
    s.strips = (int64_t(D) + 64 * s.V - 1) / (64 * s.V);
    s.segs = (int64_t(L) + kT * kW - 1) / (kT * kW);
    s.blocks = s.strips * s.segs * b;
    return s;
}

hipError_t tiles_of(const GatedScanArgs &a, const Shape &s, Tiles &t, hipStream_t stream) {
    t.strips = int(s.strips);
    t.segs = int(s.segs);
    t.b = a.b;
    t.words = nullptr;
    t.counter = nullptr;
    if (s.segs <= 1) return hipSuccess;
    t.counter = static_cast<unsigned *>(a.workspace);
    t.words = reinterpret_cast<word_t *>(static_cast<char *>(a.workspace) + 16);
    return launch_copy_state(nullptr, static_cast<float *>(a.workspace), gated_scan_workspace(a.b, a.L, a.D, a.bf16) / 4, stream);
}

template <typename IO, typename AIO, int V>
hipError_t fwd(const GatedScanArgs &s, const Shape &shape, const Tiles &tiles, hipStream_t stream) {
    auto run = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, dim3(unsigned(shape.blocks)), dim3(64 * kW), 0, stream, static_cast<const IO *>(s.x),
                           static_cast<const AIO *>(s.a), s.init_state, static_cast<IO *>(s.y), s.kept, s.final_state, s.L, s.D, tiles);
        return hipGetLastError();
    };
    return s.sigmoid ? run(k_gated_scan_fwd<IO, AIO, true, V>) : run(k_gated_scan_fwd<IO, AIO, false, V>);
}

template <typename IO, typename AIO, int V>
hipError_t bwd(const GatedScanArgs &s, const Shape &shape, const Tiles &tiles, hipStream_t stream) {
    auto run = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, dim3(unsigned(shape.blocks)), dim3(64 * kW), 0, stream, static_cast<const IO *>(s.x),
                           static_cast<const AIO *>(s.a), s.kept, static_cast<const IO *>(s.dy), s.d_final,
                           static_cast<IO *>(s.dx), static_cast<AIO *>(s.da), s.d_init, s.L, s.D, tiles);
        return hipGetLastError();
    };
    return s.sigmoid ? run(k_gated_scan_bwd<IO, AIO, true, V>) : run(k_gated_scan_bwd<IO, AIO, false, V>);
}

}  // namespace

// the kernels count tokens and channels in 31 bits, up to a block past the last one, and
// blocks in 31
bool gated_scan_supported(int b, int L, int D) {
    return b <= 65535 && L <= INT_MAX - kT * kW && D <= INT_MAX - 256 && shape_of(b, L, D, false).blocks <= (1 << 22);
}

size_t gated_scan_workspace(int b, int L, int D, bool bf16) {
    const Shape s = shape_of(b, L, D, bf16);
    return s.segs <= 1 ? 0 : 16 + size_t(s.blocks) * 64 * s.V * 2 * sizeof(word_t);
}

hipError_t launch_gated_scan_fwd(const GatedScanArgs &a, hipStream_t stream) {
    const Shape s = shape_of(a.b, a.L, a.D, a.bf16);
    Tiles t;
    if (const hipError_t e = tiles_of(a, s, t, stream); e != hipSuccess) return e;
    if (!a.bf16) return fwd<float, float, 1>(a, s, t, stream);
    if (s.V == 2) return a.a_bf16 ? fwd<bf16_bits, bf16_bits, 2>(a, s, t, stream) : fwd<bf16_bits, float, 2>(a, s, t, stream);
    return a.a_bf16 ? fwd<bf16_bits, bf16_bits, 1>(a, s, t, stream) : fwd<bf16_bits, float, 1>(a, s, t, stream);
}

hipError_t launch_gated_scan_bwd(const GatedScanArgs &a, hipStream_t stream) {
    const Shape s = shape_of(a.b, a.L, a.D, a.bf16);
    Tiles t;
    if (const hipError_t e = tiles_of(a, s, t, stream); e != hipSuccess) return e;
    if (!a.bf16) return bwd<float, float, 1>(a, s, t, stream);
    if (s.V == 2) return a.a_bf16 ? bwd<bf16_bits, bf16_bits, 2>(a, s, t, stream) : bwd<bf16_bits, float, 2>(a, s, t, stream);
    return a.a_bf16 ? bwd<bf16_bits, bf16_bits, 1>(a, s, t, stream) : bwd<bf16_bits, float, 1>(a, s, t, stream);
}

}  // namespace ssd
