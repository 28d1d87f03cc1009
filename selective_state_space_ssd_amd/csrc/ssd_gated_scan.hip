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
//   - eight of the waves (four of a block of four) wait for one block before each, until its
//     pair or already its outgoing state is there; where there is no state among them, as in
//     long sequences of few channels, they look at three blocks more each,
//   - all fold the pairs behind the nearest such state, one by one, into the entering state
//     (the same operations in the same order whichever block that was, so results repeat),
//   - the last wave publishes the outgoing state in the pair's place.
// Blocks take their places from a counter, earlier stretches first, so whatever a block
// waits for belongs to a block that is running already.  A pair or a state is one 8-byte
// word, written at once and never zero; zero means not there yet.  A wait that gives up all
// the same sets the workspace's error word and goes on with NaN.
//
// Tiles of 256 tokens (8 waves of 32) by 128 bf16 channels put 131 KB of loads under way per
// block, two blocks a CU; a token's gate takes the place of its value in registers, so that the
// second walk starts from what the first left (122 registers forward, 193 backward).
//
// bf16, medians of kernel times: 4 x 2048 tokens of 5120 channels behind gates, forward 252 MB in
// 58 us, 4.3 TB/s; 16384 tokens of 2560 with fp32 decays, 335 MB in 78, 4.3 TB/s; backward of the
// former 425 MB in 88, 4.8 TB/s (with an fp32 gate 593 MB in 106, 5.6), without kept states 47 more
// for a forward pass that stores nothing else, its second walk included.  One array into
// another reaches 6.1 TB/s on this card.  24 vector instructions an element forward (36 backward)
// keep the vector ALU busy for 60 % of that time, which loads do not wholly cover.  Blocks come
// in rounds of two a CU, 1280 forward and 2560 backward for 5120 channels, 2.5 and 5 rounds.  The
// fewer the rounds, the more a part-filled last one counts: 2560 channels, 1.25 and 2.5 rounds,
// take 35 us, 3.6 TB/s, and 51, 4.2.  Not better: tiles of half and of twice the tokens, four
// channels a lane (fewer waves a CU: 74 us), loads in the order of their use, all looks further
// back at once (spills).
// fp32, 2 x 1337 tokens of 1288: 41 MB in 15 us, one block a CU, whose latencies add up;
// backward of 2 x 777 tokens of 645: 11 us.
#include "ssd_gated_scan.h"
#include "ssd_gated_scan_gate.h"

namespace ssd {
namespace {

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

// As here(float): what is made of r (unpacked values, products, signs) is made again where it is
// used again.  Kept from one use to the other they would take more registers than there are.
template <typename T, int V>
__device__ __forceinline__ Raw<T, V> again(Raw<T, V> r) {
    if constexpr (sizeof(r) == 2) {
        uint32_t v = r.r;
        asm("" : "+v"(v));
        r.r = uint16_t(v);
    } else if constexpr (sizeof(r) == 8) {
        asm("" : "+v"(r.r.x), "+v"(r.r.y));
    } else {
        asm("" : "+v"(r.r));
    }
    return r;
}

// Rows of a stretch of n tokens, through a buffer view of them: a row's place is a scalar
// register's, the channels' place in it the lane's.  What is read is read once: it does not stay
// in the caches (the layer of 4 x 2048 tokens, 5120 channels 100 -> 92 us backward, 16384 tokens 85
// -> 80; stores marked so gained nothing).
struct Rows {
    __amdgpu_buffer_rsrc_t view;
    uint32_t lane, row;     // bytes

    template <typename T, int V>
    __device__ __forceinline__ Raw<T, V> load(int t) const {
        if constexpr (sizeof(Raw<T, V>) == 2) return __builtin_bit_cast(Raw<T, V>, __builtin_amdgcn_raw_buffer_load_b16(view, lane, t * row, kBufNonTemporal));
        else if constexpr (sizeof(Raw<T, V>) == 4) return __builtin_bit_cast(Raw<T, V>, __builtin_amdgcn_raw_buffer_load_b32(view, lane, t * row, kBufNonTemporal));
        else return __builtin_bit_cast(Raw<T, V>, __builtin_amdgcn_raw_buffer_load_b64(view, lane, t * row, kBufNonTemporal));
    }
    // Rows [0, TOK); those past the n-th repeat it.
    template <typename T, int V, int TOK>
    __device__ __forceinline__ void load_all(int n, Raw<T, V> (&out)[TOK]) const {
#pragma unroll
        for (int t = 0; t < TOK; ++t) out[t] = load<T, V>(n == TOK ? t : min(t, n - 1));
    }
    template <typename T, int V>
    __device__ __forceinline__ void store(int t, Raw<T, V> r) const {
        if constexpr (sizeof(r) == 2) __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(uint16_t, r), view, lane, t * row, 0);
        else if constexpr (sizeof(r) == 4) __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, r), view, lane, t * row, 0);
        else __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(u32x2, r), view, lane, t * row, 0);
    }
};

// n > 0 rows of D <= 2^24 channels from `first` on.
template <typename T>
__device__ __forceinline__ Rows rows_at(const T *first, int n, int D, int channel) {
    const uint32_t row = uint32_t(D) * uint32_t(sizeof(T));
    return {buffer_rsrc(first, uint32_t(n) * row), uint32_t(channel) * uint32_t(sizeof(T)), row};
}

// ----------------------------------------------------------------- pairs and their words
// The decay of two stretches after each other, in the form of ssd_gated_scan_gate.h.
__device__ __forceinline__ float both_decays(float m1, float m2) {
    const float a = alpha_of(m1) * alpha_of(m2), b1 = beta_of(m1), b2 = beta_of(m2);
    const float b = fmaf(b1, 1.f - b2, b2);
    return a > 0.5f && b >= 0.f ? -b : a;
}

// The decay of the tokens of a stretch, taken one by one.  Near 1 from the sum of what each
// takes away (log decay: of a itself), below from the product: the sum of a log decay that
// erases with many small ones rounds those to the erasing one's last bits.
template <bool SIGMOID>
struct Decay {
    float alpha = 1.f, lost = 0.f;      // lost: 1 - alpha (sigmoid), the sum of a (log decay)
    __device__ __forceinline__ void token(float m, float a) {
        alpha = decayed(m, alpha);
        // (a token far from 1 makes the product what counts: lost may be anything then)
        if constexpr (SIGMOID) lost = fmaf(-m, 1.f - lost, lost);
        else lost += a;
    }
    __device__ __forceinline__ float m() const {
        // here(): the product is not put off into a branch on the sum
        const float product = here(alpha), near = here(SIGMOID ? -lost : gate_of<false>(lost));
        if constexpr (SIGMOID) return alpha > 0.5f && lost >= 0.f ? near : product;
        else return lost > -1.f ? near : product;
    }
};

typedef unsigned long long word_t;

// A pair (m, S), or a state behind a mark that no m is.  Never zero: the complement of two floats
// of which the first is not all ones.
constexpr uint32_t kNan = 0x7fc00000u, kState = 0x7fc00001u;
__device__ __forceinline__ word_t word_of(uint32_t first, float second) { return ~(word_t(first) << 32 | __float_as_uint(second)); }
__device__ __forceinline__ word_t pair_word(float m, float s) { return word_of(m == m ? __float_as_uint(m) : kNan, s); }
__device__ __forceinline__ word_t state_word(float h) { return word_of(kState, h); }
__device__ __forceinline__ uint32_t first_of(word_t w) { return uint32_t(~w >> 32); }
__device__ __forceinline__ float second_of(word_t w) { return __uint_as_float(uint32_t(~w)); }

__device__ __forceinline__ word_t look(const word_t *p) { return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); }
__device__ __forceinline__ void publish(word_t *p, word_t w) { __hip_atomic_store(p, w, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); }

// Workspace: 16 bytes with the counter of places and the error word, then per block 64 V words.
struct Tiles {
    word_t *words;          // null: one block a strip, nothing to wait for
    unsigned *counter;      // the error word behind it
    int strips, segs, b;
    int looks;              // at a word, before a wait gives up
};

template <int V>
__device__ __forceinline__ word_t *words_of(const Tiles &s, int bi, int seg, int strip) {
    return s.words + ((size_t(seg) * s.b + bi) * s.strips + strip) * (64 * V);
}

enum Seen { kNothing, kPairs, kStates };

// What all V words of every lane are; kNothing while they differ.
template <int V>
__device__ __forceinline__ Seen look_all(const word_t *p, word_t (&w)[V]) {
    bool there = true, state = true, pair = true;
#pragma unroll
    for (int j = 0; j < V; ++j) w[j] = look(p + j);
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const bool is_state = first_of(w[j]) == kState;
        there = there && w[j] != 0;
        state = state && is_state;
        pair = pair && !is_state;
    }
    if (!__all(there)) return kNothing;
    return __all(state) ? kStates : __all(pair) ? kPairs : kNothing;
}

// Looks at a block's words until they are there, or until all are states if `states` says so.
// A wait that gives up leaves kNothing, and the error word set.
template <int V>
__device__ __forceinline__ Seen wait_for(const Tiles &tiles, const word_t *p, bool states, int lane, word_t (&w)[V]) {
#pragma unroll
    for (int j = 0; j < V; ++j) w[j] = 0;
#pragma unroll 1
    for (int n = 0; n < tiles.looks; ++n) {
        const Seen seen = look_all<V>(p, w);
        if (seen == kStates || (seen == kPairs && !states)) return seen;
        __builtin_amdgcn_s_sleep(1);
    }
    if (lane == 0) __hip_atomic_store(tiles.counter + 1, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    return kNothing;
}

template <int V, int W>
struct ChainLds {
    // blocks before that are looked at: one for each of the last kNear waves, and kFar more
    // for each where none of those has a state yet
    static constexpr int kNear = W < 8 ? W : 8, kFar = 3;
    float2 pair[W][64 * V];         // of the block's waves
    float2 before[kNear * (1 + kFar)][64 * V];      // of the blocks before: pair, or (., outgoing state)
    int state[kNear * (1 + kFar)];  // whether it is a state
    unsigned place;
};

// The state that enters a wave's tokens.  `wave` counts in the order of the scan; m and s are
// the pair of the wave's tokens, `start` the state before the first block.
template <int V, int W>
__device__ __forceinline__ void enter(const Tiles &tiles, ChainLds<V, W> &lds, int bi, int seg, int strip, int wave, int lane,
                                      const float (&m)[V], const float (&s)[V], const float (&start)[V], float (&h)[V]) {
#pragma unroll
    for (int j = 0; j < V; ++j) lds.pair[wave][lane * V + j] = make_float2(m[j], s[j]);
    __syncthreads();
    float pm[V], ps[V];             // of the waves before
#pragma unroll
    for (int j = 0; j < V; ++j) { pm[j] = 1.f; ps[j] = 0.f; }
#pragma unroll 2
    for (int k = 0; k < wave; ++k)
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const float2 p = lds.pair[k][lane * V + j];
            pm[j] = both_decays(pm[j], p.x);
            ps[j] = apply_pair(p.x, ps[j], p.y);
        }
    if (tiles.segs == 1) {
#pragma unroll
        for (int j = 0; j < V; ++j) h[j] = apply_pair(pm[j], start[j], ps[j]);
        return;
    }
    word_t *own = words_of<V>(tiles, bi, seg, strip) + lane * V;
    float bm[V], bs[V];             // of the block
    if (wave == W - 1) {
#pragma unroll
        for (int j = 0; j < V; ++j) {
            bm[j] = both_decays(pm[j], m[j]);
            bs[j] = apply_pair(m[j], ps[j], s[j]);
            publish(own + j, pair_word(bm[j], bs[j]));
        }
    }
    constexpr int kNear = ChainLds<V, W>::kNear, kFar = ChainLds<V, W>::kFar;
    const int back = W - wave;      // this wave's of the blocks before: 1 is the nearest
    const float nan = __uint_as_float(kNan);
    // the words of the block `at` before, into its place
    auto gather = [&](int at) {
        const word_t *p = words_of<V>(tiles, bi, seg - at, strip) + lane * V;
        word_t w[V];
        const Seen seen = wait_for<V>(tiles, p, false, lane, w);
#pragma unroll
        for (int j = 0; j < V; ++j)
            lds.before[at - 1][lane * V + j] = make_float2(__uint_as_float(first_of(w[j])), seen != kNothing ? second_of(w[j]) : nan);
        if (lane == 0) lds.state[at - 1] = seen == kStates;
    };
    // the nearest state among the first n places; n: none
    auto nearest = [&](int n) {
        const unsigned long long have = __ballot(lane < n && lds.state[lane < n ? lane : 0]);
        return have ? int(__builtin_ctzll(have)) : n;
    };
    int n = min(kNear, seg), k = 0;
    if (back <= n) gather(back);
    __syncthreads();
    float in[V];
    if (seg == 0) {
#pragma unroll
        for (int j = 0; j < V; ++j) in[j] = start[j];
    } else {
        k = nearest(n);
        if (k == n && seg > n) {    // the block runs far ahead of the states
            n = min(kNear * (1 + kFar), seg);
            if (back <= kNear)
#pragma unroll 1
                for (int at = back + kNear; at <= n; at += kNear) gather(at);
            __syncthreads();
            k = nearest(n);
        }
        if (k < n) {
#pragma unroll
            for (int j = 0; j < V; ++j) in[j] = lds.before[k][lane * V + j].y;
        } else {                    // none yet: the furthest one's
            const word_t *p = words_of<V>(tiles, bi, seg - n, strip) + lane * V;
            word_t w[V];
            const bool there = wait_for<V>(tiles, p, true, lane, w) == kStates;
            k = n - 1;
#pragma unroll
            for (int j = 0; j < V; ++j) in[j] = there ? second_of(w[j]) : nan;
        }
    }
#pragma unroll 2
    for (int i = k - 1; i >= 0; --i)
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const float2 p = lds.before[i][lane * V + j];
            in[j] = apply_pair(p.x, in[j], p.y);
        }
    if (wave == W - 1)
#pragma unroll
        for (int j = 0; j < V; ++j) publish(own + j, state_word(apply_pair(bm[j], in[j], bs[j])));
#pragma unroll
    for (int j = 0; j < V; ++j) h[j] = apply_pair(pm[j], in[j], ps[j]);
}

// A block's place: strip fastest, then the batch row, then the stretch of the sequence.
template <int V, int W>
__device__ __forceinline__ void place_of(const Tiles &tiles, ChainLds<V, W> &lds, int &bi, int &seg, int &strip) {
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
template <typename IO, typename AIO, bool SIGMOID, int V, int T, int W>
__global__ __launch_bounds__(64 * W, 4) void k_gated_scan_fwd(const IO *__restrict__ x, const AIO *__restrict__ a,
                                                            const float *__restrict__ init_state, IO *__restrict__ y,
                                                            float *__restrict__ kept, float *__restrict__ final_state,
                                                            int L, int D, Tiles tiles) {
    __shared__ ChainLds<V, W> lds;
    int bi, seg, strip;
    place_of<V, W>(tiles, lds, bi, seg, strip);
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int c = strip * 64 * V + lane * V;
    const bool on = c < D;                  // V divides D
    const int cl = on ? c : 0;
    const int t0 = (seg * W + wave) * T, n = min(T, L - t0);     // n <= 0: past the end
    const size_t row = size_t(bi) * L + t0;

    Raw<IO, V> xr[T];
    float m[T][V], pm[V], ps[V];
    if (n > 0) {
        Raw<AIO, V> ar[T];
        rows_at(a + row * D, n, D, cl).template load_all<AIO, V, T>(n, ar);
        rows_at(x + row * D, n, D, cl).template load_all<IO, V, T>(n, xr);
        if (n < T) {                       // tokens that leave the state as it is
#pragma unroll
            for (int t = 0; t < T; ++t)
                if (t >= n) {
                    ar[t] = raw_same<AIO, V>(SIGMOID ? __builtin_inff() : 0.f);
                    xr[t] = raw_same<IO, V>(0.f);
                }
        }
        // token by token: a gate takes the place of the values that it comes from
        Decay<SIGMOID> d[V];
#pragma unroll
        for (int j = 0; j < V; ++j) ps[j] = 0.f;
#pragma unroll
        for (int t = 0; t < T; ++t) {
            ar[t] = again<AIO, V>(ar[t]);
            xr[t] = again<IO, V>(xr[t]);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float av = ar[t].get(j);
                m[t][j] = gate_of<SIGMOID>(av);
                d[j].token(m[t][j], av);
                ps[j] = step_state<SIGMOID>(m[t][j], ps[j], xr[t].get(j));
            }
        }
#pragma unroll
        for (int j = 0; j < V; ++j) pm[j] = d[j].m();
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j) { pm[j] = 1.f; ps[j] = 0.f; }
    }
    float start[V], h[V];
#pragma unroll
    for (int j = 0; j < V; ++j) start[j] = init_state ? init_state[size_t(bi) * D + cl + j] : 0.f;
    enter<V, W>(tiles, lds, bi, seg, strip, wave, lane, pm, ps, start, h);
    if (n <= 0 || !on) return;
    if (kept && t0 % kGatedScanKeep == 0) {
        float *k = kept + (size_t(bi) * ((unsigned(L) + kGatedScanKeep - 1) / kGatedScanKeep) + t0 / kGatedScanKeep) * D + c;
#pragma unroll
        for (int j = 0; j < V; ++j) k[j] = h[j];
    }
    const Rows out = rows_at(y ? y + row * D : y, n, D, c);
#pragma unroll
    for (int t = 0; t < T; ++t) {
        if (t >= n) continue;       // the last token's state as it is, also where it is infinite
        xr[t] = again<IO, V>(xr[t]);
#pragma unroll
        for (int j = 0; j < V; ++j) h[j] = step_state<SIGMOID>(here(m[t][j]), h[j], xr[t].get(j));
        if (y) out.template store<IO, V>(t, raw_of<IO, V>(h));
    }
    if (final_state && t0 + n == L)
#pragma unroll
        for (int j = 0; j < V; ++j) final_state[size_t(bi) * D + c + j] = h[j];
}

// -------------------------------------------------------------------------- backward
// The order of the scan is that of the tokens backwards: segment and wave 0 are the last.
template <typename IO, typename AIO, bool SIGMOID, int V, int T, int W>
__global__ __launch_bounds__(64 * W, T == kGatedScanKeep ? 2 : 4) void k_gated_scan_bwd(const IO *__restrict__ x, const AIO *__restrict__ a,
                                                            const float *__restrict__ kept, const IO *__restrict__ dy,
                                                            const float *__restrict__ d_final, IO *__restrict__ dx,
                                                            AIO *__restrict__ da, float *__restrict__ d_init, int L,
                                                            int D, Tiles tiles) {
    // waves of a kept state's stretch, and what each does to the state (forward)
    constexpr int kParts = kGatedScanKeep / T;
    static_assert(W % kParts == 0);
    __shared__ float2 ahead[kParts > 1 ? W : 1][64 * V];
    __shared__ ChainLds<V, W> lds;
    int bi, seg, strip;
    place_of<V, W>(tiles, lds, bi, seg, strip);
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int c = strip * 64 * V + lane * V;
    const bool on = c < D;
    const int cl = on ? c : 0;
    const int t0 = ((tiles.segs - 1 - seg) * W + W - 1 - wave) * T, n = min(T, L - t0);
    const size_t row = size_t(bi) * L + t0;

    Raw<IO, V> xr[T], gr[T];
    float m[T][V], slope[T][V], pm[V], ps[V], h[V];
    // what da_t is g_{t-1} times: h_{t-1}, or beta_t (h_{t-1} - x_t); x is done with then
    auto slopes = [&]() {
#pragma unroll
        for (int t = 0; t < T; ++t) {
            xr[t] = again<IO, V>(xr[t]);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float xv = xr[t].get(j), hb = h[j], mt = here(m[t][j]);
                h[j] = step_state<SIGMOID>(mt, hb, xv);
                slope[t][j] = SIGMOID ? beta_of(mt) * (hb - xv) : hb;
            }
        }
    };
    if (n > 0) {
        Raw<AIO, V> ar[T];
        rows_at(a + row * D, n, D, cl).template load_all<AIO, V, T>(n, ar);
        rows_at(dy + row * D, n, D, cl).template load_all<IO, V, T>(n, gr);
        rows_at(x + row * D, n, D, cl).template load_all<IO, V, T>(n, xr);
        if (n < T) {
#pragma unroll
            for (int t = 0; t < T; ++t)
                if (t >= n) {
                    ar[t] = raw_same<AIO, V>(SIGMOID ? __builtin_inff() : 0.f);
                    gr[t] = xr[t] = raw_same<IO, V>(0.f);
                }
        }
        const float *k = kept + (size_t(bi) * ((unsigned(L) + kGatedScanKeep - 1) / kGatedScanKeep) + t0 / kGatedScanKeep) * D + cl;
        Decay<SIGMOID> d[V];
#pragma unroll
        for (int j = 0; j < V; ++j) { ps[j] = 0.f; h[j] = k[j]; }
#pragma unroll
        for (int t = T - 1; t >= 0; --t) {
            ar[t] = again<AIO, V>(ar[t]);
            gr[t] = again<IO, V>(gr[t]);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float av = ar[t].get(j);
                m[t][j] = gate_of<SIGMOID>(av);
                d[j].token(m[t][j], av);
                ps[j] = decayed(m[t][j], gr[t].get(j) + ps[j]);
            }
        }
#pragma unroll
        for (int j = 0; j < V; ++j) pm[j] = d[j].m();
        if constexpr (kParts == 1) {
            slopes();
        } else {
#pragma unroll
            for (int j = 0; j < V; ++j) {
                float sf = 0.f;
#pragma unroll
                for (int t = 0; t < T; ++t) sf = step_state<SIGMOID>(m[t][j], sf, xr[t].get(j));
                ahead[wave][lane * V + j] = make_float2(pm[j], sf);
            }
        }
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j) { pm[j] = 1.f; ps[j] = 0.f; }
    }
    float start[V], g[V];
#pragma unroll
    for (int j = 0; j < V; ++j) start[j] = d_final ? d_final[size_t(bi) * D + cl + j] : 0.f;
    enter<V, W>(tiles, lds, bi, seg, strip, wave, lane, pm, ps, start, g);
    if (n <= 0 || !on) return;
    if constexpr (kParts > 1) {
        // from the kept state over the waves between it and this one's tokens
        const int part = t0 / T % kParts;
#pragma unroll 1
        for (int k = part; k > 0; --k)
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float2 p = ahead[wave + k][lane * V + j];
                h[j] = apply_pair(p.x, h[j], p.y);
            }
        slopes();
    }
    const Rows outx = rows_at(dx + row * D, n, D, c), outa = rows_at(da + row * D, n, D, c);
#pragma unroll
    for (int t = T - 1; t >= 0; --t) {
        if (t >= n) continue;
        float ox[V], oa[V];
        gr[t] = again<IO, V>(gr[t]);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const float lam = gr[t].get(j) + g[j], mt = here(m[t][j]);
            g[j] = decayed(mt, lam);
            ox[j] = SIGMOID ? beta_of(mt) * lam : lam;
            oa[j] = g[j] * slope[t][j];
        }
        outx.template store<IO, V>(t, raw_of<IO, V>(ox));
        outa.template store<AIO, V>(t, raw_of<AIO, V>(oa));
    }
    if (d_init && t0 == 0)
#pragma unroll
        for (int j = 0; j < V; ++j) d_init[size_t(bi) * D + c + j] = g[j];
}

// ---------------------------------------------------------------------------- launches
// keep: the error word stays, of a pass before this one in the same call.
__global__ __launch_bounds__(256) void k_gated_scan_clear(uint4 *p, size_t n, bool keep) {
    const size_t i = size_t(blockIdx.x) * 256 + threadIdx.x;
    if (i < n) p[i] = make_uint4(0, i == 0 && keep ? p[0].y : 0, 0, 0);
}

__global__ void k_gated_scan_error(const unsigned *header, int32_t *err_out) {
    *err_out = header ? int32_t(__hip_atomic_load(header + 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT)) : 0;
}

// Channels of a lane: two bf16 in one 4-byte access where the rows allow it.  (Four, in 8 bytes,
// leave a CU half the waves: 4 x 2048 tokens of 5120 channels 74 instead of 58 us.)
int lane_channels(int D, bool bf16) { return bf16 && D % 2 == 0 ? 2 : 1; }

// Tokens of a block: W waves of T tokens.  Much work takes long stretches, fewer pairs to hand on
// for as many bytes: forward 8 x 32 tokens, backward 4 x 32 with two channels a lane (193
// registers, of which a SIMD holds two waves) and 16 x 16 with one (68 registers).  Where 128
// tokens a block make no more blocks than there are CUs, and for sequences that end within
// one, 8 x 16.  The long way / the short way in us, both launches:
//   blocks of 8 x 16   154 (2 x 777 tokens)  304 (2 x 1024)  464          704          1008         1504         2560 (4 x 2048)
//   forward, fp32      13.1 / 11.4           14.1 / 14.9     16.1 / 18.1  21.5 / 24.6  26.1 / 33.3  37.6 / 43.8  51.8 / 59.9
//   forward, bf16                            16.6 / 17.5     19.0 / 20.7  25.1 / 27.8  29.1 / 39.2  41.6 / 45.2  59.6 / 63.3
//   backward, fp32     17.2 / 13.4           17.3 / 17.8     19.7 / 21.6  31.1 / 34.3  39.8 / 44.6  55.3 / 56.5  84.2 / 82.3
//   backward, bf16                           21.7 / 21.4     25.2 / 25.1  36.9 / 35.5  46.3 / 46.5  58.9 / 58.1  90.6 / 87.3
// (The gradients in bf16 hardly depend on it.  16 x 16 would take 20.8, 22.8, 36.3, 42.1, 60.7 and
// 101.4 there; forward, in bf16, 16.8, 18.9, 28.8, 31.5, 43.6 and 67.6.)  Sequences that end within
// a block, 32 x 100 tokens of 2560 channels: forward bf16 15.8 / 13.9, fp32 19.8 / 17.1, backward
// 23.1 / 20.7 and 33.0 / 28.5.
// A chain of more than 32 of the short blocks costs more than their latency spares.  One sequence,
// forward: 16384 tokens, bf16, 64, 128 and 256 channels 19.5 / 22.0, 19.9 / 22.7, 21.6 / 24.8, fp32, half
// as many channels, 14.6 / 16.3, 15.1 / 16.5, 16.6 / 18.5; 8192 tokens of 256 or 128 channels 17.7 / 18.1
// and 14.1 / 13.8, 5000 of 512 or 256 17.5 / 17.4 and 14.0 / 14.0; 60000 of 64 or 32 34.0 / 55.6 and
// 23.8 / 36.4.  (Backward, at 5000, 8192, 16384 and 60000 tokens, bf16 19.8 / 19.7, 20.5 / 19.9,
// 26.2 / 24.6, 60.8 / 58.4, fp32 17.4 / 15.7, 17.2 / 15.1, 18.1 / 17.8, 28.4 / 37.8.)
//
// Sequences of 129 to 256 tokens take one block of 16 x 16: no words to clear, one launch instead
// of two.  Two blocks of 8 x 16 / this, kernel times and, of the first, call times: forward, bf16
// 4 x 200 of 640 9.7 / 8.6 (15.0 / 10.6), fp32 8.9 / 6.4; backward, bf16 12.0 / 12.1 (17.8 / 13.1),
// fp32 10.4 / 7.7.  Where that makes many blocks, 4 x 32 / this, backward, bf16: 32 x 256 of 2560
// 52.0 / 48.4, 64 x 256 of 1024 44.9 / 37.8; but 8 x 32 / this, forward, bf16: 27.6 / 33.7, 20.3 /
// 27.4 (fp32 the same).
struct Shape {
    int V, T, W;
    int64_t strips, segs, blocks;
};

constexpr int kFwdT = 32, kFwdW = 8;
template <int V> constexpr int kBwdT = V == 2 ? 32 : 16;
template <int V> constexpr int kBwdW = V == 2 ? 4 : 16;
constexpr int kShortT = 16, kShortW = 8, kShort = kShortT * kShortW, kPairW = 16, kCus = 256, kLongChain = 32;

Shape shape_of(int b, int L, int D, bool bf16, bool backward) {
    Shape s;
    s.V = lane_channels(D, bf16);
    s.strips = (int64_t(D) + 64 * s.V - 1) / (64 * s.V);
    s.segs = (int64_t(L) + kShort - 1) / kShort;
    s.T = kShortT;
    s.W = kShortW;
    const bool much = s.strips * s.segs * b > kCus || s.segs > kLongChain;
    if (s.segs == 2 && (backward || !much)) {
        s.W = kPairW;
        s.segs = 1;
    } else if (s.segs > 1 && much) {
        s.T = !backward ? kFwdT : s.V == 2 ? kBwdT<2> : kBwdT<1>;
        s.W = !backward ? kFwdW : s.V == 2 ? kBwdW<2> : kBwdW<1>;
        s.segs = (int64_t(L) + s.T * s.W - 1) / (s.T * s.W);
    }
    s.blocks = s.strips * s.segs * b;
    return s;
}

size_t words_bytes(const Shape &s) { return s.segs <= 1 ? 0 : 16 + size_t(s.blocks) * 64 * s.V * sizeof(word_t); }

hipError_t tiles_of(const GatedScanArgs &a, const Shape &s, Tiles &t, hipStream_t stream) {
    t.strips = int(s.strips);
    t.segs = int(s.segs);
    t.b = a.b;
    t.looks = a.looks;
    t.words = nullptr;
    t.counter = nullptr;
    if (s.segs <= 1) return hipSuccess;
    t.counter = static_cast<unsigned *>(a.workspace);
    t.words = reinterpret_cast<word_t *>(static_cast<char *>(a.workspace) + 16);
    const size_t n = words_bytes(s) / 16;
    hipLaunchKernelGGL(k_gated_scan_clear, dim3(unsigned((n + 255) / 256)), dim3(256), 0, stream, static_cast<uint4 *>(a.workspace), n, a.keep_error);
    return hipGetLastError();
}

template <typename IO, typename AIO, int V, int T, int W>
hipError_t fwd(const GatedScanArgs &s, const Shape &shape, const Tiles &tiles, hipStream_t stream) {
    auto run = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, dim3(unsigned(shape.blocks)), dim3(64 * W), 0, stream, static_cast<const IO *>(s.x),
                           static_cast<const AIO *>(s.a), s.init_state, static_cast<IO *>(s.y), s.kept, s.final_state, s.L, s.D, tiles);
        return hipGetLastError();
    };
    return s.sigmoid ? run(k_gated_scan_fwd<IO, AIO, true, V, T, W>) : run(k_gated_scan_fwd<IO, AIO, false, V, T, W>);
}

template <typename IO, typename AIO, int V, int T, int W>
hipError_t bwd(const GatedScanArgs &s, const Shape &shape, const Tiles &tiles, hipStream_t stream) {
    auto run = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, dim3(unsigned(shape.blocks)), dim3(64 * W), 0, stream, static_cast<const IO *>(s.x),
                           static_cast<const AIO *>(s.a), s.kept, static_cast<const IO *>(s.dy), s.d_final,
                           static_cast<IO *>(s.dx), static_cast<AIO *>(s.da), s.d_init, s.L, s.D, tiles);
        return hipGetLastError();
    };
    return s.sigmoid ? run(k_gated_scan_bwd<IO, AIO, true, V, T, W>) : run(k_gated_scan_bwd<IO, AIO, false, V, T, W>);
}

// f(IO{}, AIO{}, V) for the call's types and channels of a lane.
template <class F>
hipError_t by_types(const GatedScanArgs &a, int V, F &&f) {
    using std::integral_constant;
    if (!a.bf16) return f(float{}, float{}, integral_constant<int, 1>{});
    if (V == 2) return a.a_bf16 ? f(bf16_bits{}, bf16_bits{}, integral_constant<int, 2>{}) : f(bf16_bits{}, float{}, integral_constant<int, 2>{});
    return a.a_bf16 ? f(bf16_bits{}, bf16_bits{}, integral_constant<int, 1>{}) : f(bf16_bits{}, float{}, integral_constant<int, 1>{});
}

}  // namespace

// The bytes of a wave's rows are counted in 32 bits.  One bound on the blocks for every type, pass
// and tile, counted with the smallest tile at one channel a lane: as many take 2^30 of a launch's
// 2^32 threads, and two channels a lane or longer tiles a quarter of that or less, so it is not
// the launch's own.  It keeps L below 2^28 + 1 and with it the kernels' token counters.
bool gated_scan_supported(int b, int L, int D) {
    return b <= 65535 && D <= (1 << 24) && b * ((int64_t(L) + 127) / 128) * ((int64_t(D) + 63) / 64) <= (1 << 21);
}

// shape_of: up to kPairW short waves of tokens are one block's, and any more are several blocks'
bool gated_scan_waits(int L) { return L > kPairW * kShortT; }

hipError_t launch_gated_scan_error(const void *workspace, int32_t *err_out, hipStream_t stream) {
    hipLaunchKernelGGL(k_gated_scan_error, dim3(1), dim3(1), 0, stream, static_cast<const unsigned *>(workspace), err_out);
    return hipGetLastError();
}

size_t gated_scan_workspace(int b, int L, int D, bool bf16, bool backward) { return words_bytes(shape_of(b, L, D, bf16, backward)); }

hipError_t launch_gated_scan_fwd(const GatedScanArgs &a, hipStream_t stream) {
    const Shape s = shape_of(a.b, a.L, a.D, a.bf16, false);
    Tiles t;
    if (const hipError_t e = tiles_of(a, s, t, stream); e != hipSuccess) return e;
    return by_types(a, s.V, [&](auto io, auto aio, auto v) {
        using IO = decltype(io);
        using AIO = decltype(aio);
        if (s.T == kFwdT) return fwd<IO, AIO, v(), kFwdT, kFwdW>(a, s, t, stream);
        if (s.W == kPairW) return fwd<IO, AIO, v(), kShortT, kPairW>(a, s, t, stream);
        return fwd<IO, AIO, v(), kShortT, kShortW>(a, s, t, stream);
    });
}

hipError_t launch_gated_scan_bwd(const GatedScanArgs &a, hipStream_t stream) {
    const Shape s = shape_of(a.b, a.L, a.D, a.bf16, true);
    Tiles t;
    if (const hipError_t e = tiles_of(a, s, t, stream); e != hipSuccess) return e;
    return by_types(a, s.V, [&](auto io, auto aio, auto v) {
        using IO = decltype(io);
        using AIO = decltype(aio);
        constexpr int V = v(), T = kBwdT<V>, W = kBwdW<V>;
        if (s.T == T && s.W == W) return bwd<IO, AIO, V, T, W>(a, s, t, stream);
        if (s.W == kPairW) return bwd<IO, AIO, V, kShortT, kPairW>(a, s, t, stream);
        return bwd<IO, AIO, V, kShortT, kShortW>(a, s, t, stream);
    });
}

}  // namespace ssd
