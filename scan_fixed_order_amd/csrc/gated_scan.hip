// gated_scan.hip -- the gated linear recurrence over [batch][steps][d], channel by channel, and its
// backward pass.
//
// Mathematics:  h[t] = a[t] h[t-1] + b[t], h[-1] the given state or 0;  a = gate, b = x, or with
// sigmoid gates a = 1 / (1 + e^-gate), b = (1 - a) x.  Backwards, with E the gradient that reaches
// h[t] from behind (the final state's, or 0, at the last step):
//   G[t] = dh[t] + E[t+1];  E[t] = a[t] G[t];  the first state's gradient is E[0]
//   dx = G, dgate = G h[t-1];  sigmoid gates: dx = (1 - a) G, dgate = a (1 - a) (h[t-1] - x) G
// The backward pass takes h as it was stored, rounded to the storage type once: the unrounded one would be a
// second recurrence, or 32 bits a step kept.  dgate is off by that half step of h times G (or a (1 - a) G).
// Steps at or past a sequence's length keep the state and have h, dx and dgate 0.
//
// Order, fixed by a step's own position: a span of 8 steps is a chain of fused multiply-adds from the
// state that reaches its first step; 16 neighbouring spans (backwards 8) make a chunk.  A span's effect
// on a state is (A, H): h -> A h + H, its chain from 0 and its product of a.  The effects of a chunk's
// spans are composed from the first on, applied to the state that reaches the chunk, and give what
// reaches each span and the next chunk.  (Backwards the same from the last step, span and chunk on.)
// The same bits come out whether one workgroup walks all chunks of its channels or several take a
// part each.
#include "det_internal.h"
#include "lm_device.h"

namespace det {
namespace {

// By measurement of calls, 8 x 2048 x 4096 bf16 forward and backward, then 3 x 10007 x 2500 f32, ragged: 93
// and 148, 194 and 332 us; 8 spans forward 92, 206; 16 backward 348 (spilled registers), 308; spans of 16
// steps with 8 of them 96 and 321, 196 and 316.
constexpr int kSteps = 8;              // steps of a span: a lane's share of a chunk
constexpr int kSpans = 16;             // spans of a chunk
constexpr int kBackSpans = 8;          // the same backwards, where a step has twice the words

// Channels of a lane: one 32-bit word of a row, so a wave's load of a step takes 256 neighbouring bytes.
// Rows of one 16-bit channel (Lone) have no word of their own.
template <typename T>
struct Lone {};
template <typename T>
struct Elem {
    typedef T type;
    static constexpr int kCh = 4 / sizeof(T);
};
template <typename T>
struct Elem<Lone<T>> {
    typedef T type;
    static constexpr int kCh = 1;
};
template <typename T>
constexpr int kCh = Elem<T>::kCh;
template <typename T>
using elem = typename Elem<T>::type;

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

typedef uint32_t u32_a2 __attribute__((aligned(2)));

// The word at `off` bytes from `base`, which is uniform.
template <typename T>
__device__ __forceinline__ uint32_t load_word(const elem<T>* base, uint32_t off) {
    const char* at = reinterpret_cast<const char*>(base) + off;
    if constexpr (sizeof(elem<T>) == 4)
        return *reinterpret_cast<const uint32_t*>(at);
    else if constexpr (kCh<T> == 1)
        return (uint32_t)*reinterpret_cast<const uint16_t*>(at);
    else
        return *reinterpret_cast<const u32_a2*>(at);
}

template <typename T>
__device__ __forceinline__ void word_of(uint32_t r, bool last, float (&v)[kCh<T>]) {
    if constexpr (sizeof(elem<T>) == 4) {
        v[0] = __uint_as_float(r);
    } else {
        if (last) r >>= 16;      // the row's last channel, alone
        if constexpr (__is_same(elem<T>, _Float16)) {
            v[0] = (float)__builtin_bit_cast(_Float16, (uint16_t)r);
            if constexpr (kCh<T> == 2) v[1] = (float)__builtin_bit_cast(_Float16, (uint16_t)(r >> 16));
        } else {
            v[0] = __uint_as_float(r << 16);
            if constexpr (kCh<T> == 2) v[1] = __uint_as_float(r & 0xFFFF0000u);
        }
    }
}

// The value as the float it is.  Some kernels' last multiply-add would be folded into its conversion
// to f16, and round once where the others round twice.
__device__ __forceinline__ float as_float(float v) {
    asm("" : "+v"(v));
    return v;
}

// n: channels from this one to the row's end
template <typename T>
__device__ __forceinline__ void store_word(elem<T>* p, int n, const float (&v)[kCh<T>]) {
    if constexpr (kCh<T> == 1) {
        if (n > 0) *p = (elem<T>)as_float(v[0]);
    } else {
        const T first = (T)as_float(v[0]);
        const uint32_t lo = __builtin_bit_cast(uint16_t, first);
        const uint32_t hi = __builtin_bit_cast(uint16_t, (T)as_float(v[1]));
        if (n >= 2)
            *reinterpret_cast<u32_a2*>(p) = lo | hi << 16;
        else if (n == 1)
            *p = first;
    }
}

// the first n of N floats of a state, zeros behind them
template <int N>
__device__ __forceinline__ void load_state(const float* p, int64_t n, float (&v)[N]) {
    typedef float floats __attribute__((ext_vector_type(N), aligned(4)));
    if (n >= N) {
        const floats f = *reinterpret_cast<const floats*>(p);
#pragma unroll
        for (int e = 0; e < N; ++e) v[e] = f[e];
    } else {
#pragma unroll
        for (int e = 0; e < N; ++e) v[e] = e < n ? p[e] : 0.0f;
    }
}

template <int N>
__device__ __forceinline__ void store_state(float* p, int64_t n, const float (&v)[N]) {
    typedef float floats __attribute__((ext_vector_type(N), aligned(4)));
    if (n >= N) {
        floats f;
#pragma unroll
        for (int e = 0; e < N; ++e) f[e] = v[e];
        *reinterpret_cast<floats*>(p) = f;
    } else {
#pragma unroll
        for (int e = 0; e < N; ++e)
            if (e < n) p[e] = v[e];
    }
}

// (1 / (1 + e^-x), 1 / (1 + e^x)) by one exponential and one reciprocal, both within (4 + |x|) 2^-23
// relative to themselves; the smaller one is 0 past |x| = 88.
__device__ __forceinline__ void sigmoids(float x, float& keep, float& take) {
    const float e = exp_fast(-fabsf(x));
    const float large = __builtin_amdgcn_rcpf(1.0f + e), small = e * large;
    keep = x >= 0.0f ? large : small;
    take = x >= 0.0f ? small : large;
}

// A state c after a span of effect (A, H).  The product of a span's linear gates may overflow although
// each is finite: a state of 0 leaves H.  (A gate that is not finite itself is in H: from_zero.)
template <bool SIG>
__device__ __forceinline__ float after_span(float A, float c, float H) {
    return !SIG && c == 0.0f ? H : fmaf(A, c, H);
}

// A span's chain begins at a state of 0, which a linear gate multiplies all the same: one of infinity or
// NaN makes the chain NaN, as it makes every state behind it.
template <bool SIG>
__device__ __forceinline__ float from_zero(float a, float b) {
    return SIG ? b : fmaf(a, 0.0f, b);
}

// what a span of steps does to a state: h -> A h + H
struct Effect {
    float A, H;
};

struct ScanArgs {
    const void *gate, *x;
    const float* state0;
    const int32_t* lengths;
    void* h;
    float* state;
    Effect* effects;      // of every chunk, where several workgroups share a sequence
    int64_t batch, steps, d, tiles, chunks, per;      // per: chunks a workgroup walks
    bool runs;            // item_of's
};

struct ScanBackArgs {
    const void *dh, *gate, *x, *h;
    const float *state0, *dstate;
    const int32_t* lengths;
    void *dgate, *dx;
    float* dstate0;
    Effect* effects;
    int64_t batch, steps, d, tiles, chunks, per;
    bool runs;
};

// steps of sequence b that count
template <typename ARGS>
__device__ __forceinline__ int64_t length_of(const ARGS& a, int64_t b) {
    if (!a.lengths) return a.steps;
    const int64_t n = a.lengths[b];
    return n < 0 ? 0 : n < a.steps ? n : a.steps;
}

// The workgroup's tile; -1 past the last one.  Workgroup b runs on XCD b % 8: with `runs` each XCD takes
// a run of neighbouring tiles, which share lines where a row is no whole number of 128-byte lines
// (3 x 10007 x 2500 f32 194 us so, 247 tile by tile; where rows are whole lines tile by tile is
// a little faster: 32 x 1024 x 2048 f16 92 us, 94 in runs).
__device__ __forceinline__ int64_t item_of(int64_t items, bool runs) {
    if (!runs) return blockIdx.x < items ? (int64_t)blockIdx.x : -1;
    const int64_t per = (items + 7) / 8, at = (int64_t)(blockIdx.x & 7) * per + (blockIdx.x >> 3);
    return (blockIdx.x >> 3) < per && at < items ? at : -1;
}

// the wave's number, known to be uniform
__device__ __forceinline__ int wave_of() { return __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); }

// What a workgroup's lane works on.  A wave takes 64 words of channels of one span, or (LANES 32) 32
// words of two neighbouring spans.  The addresses of a step are uniform but for 32-bit offsets.
struct Place {
    int64_t item, b, row0;   // tile and sequence, its first row
    int64_t load_c, c0;      // where the workgroup's part of a row begins, for loads and for stores
    uint32_t off, at;        // the lane's word in it (bytes), and its first channel
    int left;                // channels from there to the row's end
    int word, sub, span;     // the lane's word, its span in the wave and in the chunk
    bool last, whole;        // the row's last channel is alone in its word; every lane's word is whole
};

// Lanes at the row's end load its last word, whose element `word_of` moves to the front.
template <typename T, int LANES>
__device__ __forceinline__ Place place_of(int64_t item, int64_t tiles, int64_t steps, int64_t d) {
    constexpr int E = kCh<T>;
    Place p;
    p.item = item;
    p.b = item / tiles;
    p.row0 = p.b * steps;
    p.c0 = item % tiles * LANES * E;
    p.load_c = p.c0 + E <= d ? p.c0 : d < E ? 0 : d - E;
    p.word = threadIdx.x & (LANES - 1);
    p.sub = LANES == 64 ? 0 : (threadIdx.x & 63) / LANES;
    p.span = wave_of() * (64 / LANES) + p.sub;
    p.at = p.word * E;
    const int64_t left = d - p.c0 - p.at, most = d - E - p.load_c;      // the last word's place
    p.left = left < 0 ? 0 : left < E ? (int)left : E;
    p.off = (most <= 0 ? 0 : p.at < most ? p.at : (uint32_t)most) * (uint32_t)sizeof(elem<T>);
    p.last = E == 2 && p.left == 1;
    p.whole = p.c0 + LANES * E <= d;
    return p;
}

// (a, b) of one step's word
template <typename T, bool SIG>
__device__ __forceinline__ void terms(uint32_t g, uint32_t x, bool last, float (&a)[kCh<T>],
                                      float (&b)[kCh<T>]) {
    word_of<T>(g, last, a);
    word_of<T>(x, last, b);
    if constexpr (SIG) {
#pragma unroll
        for (int e = 0; e < kCh<T>; ++e) {
            float keep, take;
            sigmoids(a[e], keep, take);
            b[e] *= take;
            a[e] = keep;
        }
    }
}

// The terms of a span's steps that lie past the length: they keep the state.  (A branch of its own: a
// choice a step costs as much as the recurrence.)
template <int E>
__device__ __forceinline__ void keep_past(bool full, int64_t inside, float (&a)[kSteps][E],
                                          float (&b)[kSteps][E]) {
    if (full) return;
#pragma unroll
    for (int i = 0; i < kSteps; ++i)
        if (i >= inside) {
#pragma unroll
            for (int e = 0; e < E; ++e) {
                a[i][e] = 1.0f;
                b[i][e] = 0.0f;
            }
        }
}

// the two words of each of a span's steps
struct SpanWords {
    uint32_t g[kSteps], x[kSteps];
};

// Bytes from a span's first row to the row of step i, the row `rest` steps on from where that lies past
// it: what is loaded there is not used.  (No branch: the words of a chunk ahead would be copied, and
// waited for, where two paths of loads meet.)
__device__ __forceinline__ uint32_t row_bytes(const Place& p, int i, int rest, uint32_t pitch) {
    const int at = p.sub * kSteps + i;
    return __umul24((uint32_t)(at < rest ? at : rest), pitch);      // at most 15 times less than 2^24
}

__device__ __forceinline__ int rest_of(int64_t begin, int64_t most) {
    return most - begin < 2 * kSteps ? (int)(most - begin) : 2 * kSteps;
}

// at: the first step of the wave's spans; rows past `most` are that row again
template <typename T>
__device__ __forceinline__ void read_span(const elem<T>* gate, const elem<T>* x, const Place& p,
                                          int64_t at, int64_t most, int64_t d, SpanWords& r) {
    if (at > most) at = most;
    const int rest = rest_of(at, most);
    const int64_t row = (p.row0 + at) * d + p.load_c;
    gate += row;
    x += row;
    const uint32_t pitch = (uint32_t)d * sizeof(elem<T>);
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
        const uint32_t off = p.off + row_bytes(p, i, rest, pitch);
        r.g[i] = load_word<T>(gate, off);
        r.x[i] = load_word<T>(x, off);
    }
}

// The effects of a chunk's spans on CH channels, and the states that reach the spans.
template <int SPANS, int CH>
struct ChunkState {
    Effect eff[SPANS][CH];
    float in[SPANS][CH];
};

// One channel's effects composed, from the first span on (backwards from the last): `in` gets the
// state that reaches each, for the one that reaches the chunk; that becomes the next chunk's.
template <bool SIG, bool BACK, int SPANS, int CH>
__device__ __forceinline__ void compose(ChunkState<SPANS, CH>& s, int ch, float& carry) {
    Effect all = {};
    float in[SPANS];
#pragma unroll
    for (int k = 0; k < SPANS; ++k) {
        const Effect one = s.eff[BACK ? SPANS - 1 - k : k][ch];
        in[k] = k ? after_span<SIG>(all.A, carry, all.H) : carry;
        all.H = k ? after_span<SIG>(one.A, all.H, one.H) : one.H;
        all.A = k ? all.A * one.A : one.A;
    }
#pragma unroll
    for (int k = 0; k < SPANS; ++k) s.in[BACK ? SPANS - 1 - k : k][ch] = in[k];
    carry = after_span<SIG>(all.A, carry, all.H);
}

// place of a chunk's effect on a channel: [chunk][sequence][tile][channel]
template <int CH, typename ARGS>
__device__ __forceinline__ int64_t effect_at(const ARGS& a, int64_t item, int64_t chunk, int ch) {
    return (chunk * a.batch * a.tiles + item) * CH + ch;
}

// The state that reaches the workgroup's first chunk on channel ch (of CH, `inside` the row).
template <int CH, bool SIG, bool BACK, typename ARGS>
__device__ __forceinline__ float enter(const ARGS& a, const Place& p, const float* from,
                                       int64_t chunk, int ch, bool inside) {
    float carry = from && inside ? from[p.b * a.d + p.c0 + ch] : 0.0f;
    const int64_t count = BACK ? a.chunks - 1 - chunk : chunk;
    const Effect* at = a.effects + effect_at<CH>(a, p.item, BACK ? a.chunks - 1 : 0, ch);
    const int64_t step = (BACK ? -1 : 1) * a.batch * a.tiles * CH;
#pragma unroll 8
    for (int64_t i = 0; i < count; ++i) {
        const Effect one = at[i * step];
        carry = after_span<SIG>(one.A, carry, one.H);
    }
    return carry;
}

// A workgroup walks chunks of 64 (or 32) words of channels, the next two chunks' words in flight while
// this one's effects go round.  One pass over gate and x: bound by HBM.  8 x 2048 x 4096 bf16 89 us (403 MB,
// 4.5 TB/s), 3 x 10007 x 2500 f32, ragged, 183 (847 MB, 4.6; rows are no whole number of lines).
template <typename T, bool SIG, int LANES>
__global__ __launch_bounds__(LANES * kSpans) void k_gated_scan(ScanArgs a) {
    constexpr int E = kCh<T>, CH = LANES * E, kChunkSteps = kSteps * kSpans, kMine = kSteps * 64 / LANES;
    __shared__ ChunkState<kSpans, CH> s;
    const int wave = wave_of(), ch = threadIdx.x;      // the threads below CH compose a channel each
    const int64_t item = item_of(a.batch * a.tiles, a.runs);
    if (item < 0) return;
    const Place p = place_of<T, LANES>(item, a.tiles, a.steps, a.d);
    const int64_t len = length_of(a, p.b);
    const elem<T>* gate = static_cast<const elem<T>*>(a.gate);
    const elem<T>* x = static_cast<const elem<T>*>(a.x);
    const int64_t first = (int64_t)blockIdx.y * a.per;
    const int64_t behind = first + a.per < a.chunks ? first + a.per : a.chunks;
    SpanWords even, odd;      // the words of two chunks, both in flight
    int64_t begin = first * kChunkSteps + wave * kMine;      // the wave's first step
    const int64_t limit = len < behind * kChunkSteps ? len : behind * kChunkSteps;
    const int64_t most = limit > 0 ? limit - 1 : 0;      // the last row that is read
    read_span<T>(gate, x, p, begin, most, a.d, even);
    read_span<T>(gate, x, p, begin + kChunkSteps, most, a.d, odd);
    float carry = 0.0f;
    if (ch < CH) {
        const bool inside = p.c0 + ch < a.d;
        carry = enter<CH, SIG, false>(a, p, a.state0, first, ch, inside);
        if (first == 0 && len == 0 && inside) a.state[p.b * a.d + p.c0 + ch] = carry;
    }
    const auto walk = [&](SpanWords& words) {
        const int64_t t0 = begin + p.sub * kSteps;
        float av[kSteps][E], bv[kSteps][E];
#pragma unroll
        for (int i = 0; i < kSteps; ++i) terms<T, SIG>(words.g[i], words.x[i], p.last, av[i], bv[i]);
        read_span<T>(gate, x, p, begin + 2 * kChunkSteps, most, a.d, words);
        keep_past(begin + kMine <= len, len - t0, av, bv);
#pragma unroll
        for (int e = 0; e < E; ++e) {
            Effect own{av[0][e], from_zero<SIG>(av[0][e], bv[0][e])};
#pragma unroll
            for (int i = 1; i < kSteps; ++i) {
                own.H = fmaf(av[i][e], own.H, bv[i][e]);
                own.A *= av[i][e];
            }
            s.eff[p.span][p.at + e] = own;
        }
        __syncthreads();
        if (ch < CH) compose<SIG, false>(s, ch, carry);
        __syncthreads();
        float h[E];
#pragma unroll
        for (int e = 0; e < E; ++e) h[e] = s.in[p.span][p.at + e];
        elem<T>* out = static_cast<elem<T>*>(a.h) + (p.row0 + begin) * a.d + p.c0;
        const uint32_t at = p.at + (uint32_t)(p.sub * kSteps) * (uint32_t)a.d;
        if (p.whole && begin + kMine < len) {      // not the last step, whose state is kept
#pragma unroll
            for (int i = 0; i < kSteps; ++i) {
#pragma unroll
                for (int e = 0; e < E; ++e) h[e] = fmaf(av[i][e], h[e], bv[i][e]);
                store_word<T>(out + at, E, h);
                out += a.d;
            }
        } else {
#pragma unroll
            for (int i = 0; i < kSteps; ++i) {
                const int64_t t = t0 + i;
#pragma unroll
                for (int e = 0; e < E; ++e) h[e] = fmaf(av[i][e], h[e], bv[i][e]);
                if (t < len) {
                    store_word<T>(out + at, p.left, h);
                    if (t == len - 1) store_state(a.state + p.b * a.d + p.c0 + p.at, p.left, h);
                } else if (t < a.steps) {
                    const float zero[E] = {};
                    store_word<T>(out + at, p.left, zero);
                }
                out += a.d;
            }
        }
        begin += kChunkSteps;
    };
    for (int64_t k = first; k < behind; k += 2) {
        walk(even);
        if (k + 1 < behind) walk(odd);
    }
}

// The effect of every chunk but the last one (backwards: but the first), for workgroups that begin
// in the middle of a sequence.
template <typename T, bool SIG, bool BACK, int LANES, typename ARGS>
__device__ __forceinline__ void chunk_effect(const ARGS& a, const elem<T>* gate, const elem<T>* other,
                                             int64_t chunk) {
    constexpr int E = kCh<T>, SPANS = BACK ? kBackSpans : kSpans;
    constexpr int CH = LANES * E, kMine = kSteps * 64 / LANES;
    __shared__ Effect s_eff[SPANS][CH];
    const int wave = wave_of(), ch = threadIdx.x;
    const int64_t item = item_of(a.batch * a.tiles, a.runs);
    if (item < 0) return;
    const Place p = place_of<T, LANES>(item, a.tiles, a.steps, a.d);
    const int64_t len = length_of(a, p.b), begin = chunk * SPANS * kSteps + wave * kMine;
    SpanWords r;
    read_span<T>(gate, other, p, begin, len > 0 ? len - 1 : 0, a.d, r);
    float av[kSteps][E], bv[kSteps][E];
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
        if constexpr (BACK) {
            word_of<T>(r.g[i], p.last, av[i]);
            word_of<T>(r.x[i], p.last, bv[i]);
            if constexpr (SIG) {
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    float take;
                    sigmoids(av[i][e], av[i][e], take);
                }
            }
        } else {
            terms<T, SIG>(r.g[i], r.x[i], p.last, av[i], bv[i]);
        }
    }
    keep_past(begin + kMine <= len, len - begin - p.sub * kSteps, av, bv);
#pragma unroll
    for (int e = 0; e < E; ++e) {
        Effect own;
#pragma unroll
        for (int j = 0; j < kSteps; ++j) {
            const int i = BACK ? kSteps - 1 - j : j;
            if constexpr (BACK)      // E -> a (dh + E)
                own.H = av[i][e] * (j ? bv[i][e] + own.H : bv[i][e]);
            else
                own.H = j ? fmaf(av[i][e], own.H, bv[i][e]) : from_zero<SIG>(av[i][e], bv[i][e]);
            own.A = j ? own.A * av[i][e] : av[i][e];
        }
        s_eff[p.span][p.at + e] = own;
    }
    __syncthreads();
    if (ch >= CH) return;
    Effect all;
#pragma unroll
    for (int k = 0; k < SPANS; ++k) {
        const Effect one = s_eff[BACK ? SPANS - 1 - k : k][ch];
        all.H = k ? after_span<SIG>(one.A, all.H, one.H) : one.H;
        all.A = k ? all.A * one.A : one.A;
    }
    a.effects[effect_at<CH>(a, item, chunk, ch)] = all;
}

template <typename T, bool SIG, int LANES>
__global__ __launch_bounds__(LANES * kSpans) void k_gated_scan_chunks(ScanArgs a, int64_t chunk0) {
    chunk_effect<T, SIG, false, LANES>(a, static_cast<const elem<T>*>(a.gate), static_cast<const elem<T>*>(a.x),
                                chunk0 + blockIdx.y);
}

template <typename T, bool SIG, int LANES>
__global__ __launch_bounds__(LANES * kBackSpans) void k_gated_scan_chunks_back(ScanBackArgs a, int64_t chunk0) {
    chunk_effect<T, SIG, true, LANES>(a, static_cast<const elem<T>*>(a.gate), static_cast<const elem<T>*>(a.dh),
                               chunk0 + blockIdx.y);
}

// At most kSteps steps: no spans to compose, a lane takes a vector of channels.  One step of 64 x 4096 bf16
// 3.5 us, a load's latency and a store's.
template <typename T, bool SIG>
__global__ __launch_bounds__(256) void k_gated_scan_steps(ScanArgs a) {
    constexpr int V = kVec<T>;
    const int64_t vectors = (a.d + V - 1) / V;
    const int64_t item = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (item >= a.batch * vectors) return;
    const int64_t b = item / vectors, c = item % vectors * V, left = a.d - c;
    const int64_t len = length_of(a, b);
    float h[V] = {};
    if (a.state0) load_state(a.state0 + b * a.d + c, left, h);
    for (int64_t t = 0; t < a.steps; ++t) {
        const int64_t at = (b * a.steps + t) * a.d + c;
        float g[V], x[V], o[V];
        read_vec(static_cast<const T*>(a.gate) + at, left, 0.0f, g);
        read_vec(static_cast<const T*>(a.x) + at, left, 0.0f, x);
#pragma unroll
        for (int e = 0; e < V; ++e) {
            if constexpr (SIG) {
                float keep, take;
                sigmoids(g[e], keep, take);
                x[e] *= take;
                g[e] = keep;
            }
            if (t < len) h[e] = fmaf(g[e], h[e], x[e]);
            o[e] = t < len ? as_float(h[e]) : 0.0f;
        }
        write_vec(static_cast<T*>(a.h) + at, left, o);
    }
    store_state(a.state + b * a.d + c, left, h);
}

// ---------------------------------------------------------------- backward

// the words of each of a span's steps: gate and dh; h one step before and x (sigmoid gates)
struct BackWords {
    SpanWords in;      // gate, dh
    uint32_t h[kSteps], x[kSteps];
};

// as read_span; of h the rows before (before the sequence's first that itself, which is not used)
template <typename T, bool SIG>
__device__ __forceinline__ void read_before(const ScanBackArgs& a, const Place& p, int64_t at,
                                            int64_t most, BackWords& r) {
    if (at > most) at = most;
    const int rest = rest_of(at, most), back = at > 0 ? 0 : 1;
    const int64_t row = (p.row0 + at) * a.d + p.load_c;
    const elem<T>* x = static_cast<const elem<T>*>(a.x) + row;
    const elem<T>* h = static_cast<const elem<T>*>(a.h) + (back ? row : row - a.d);
    const uint32_t pitch = (uint32_t)a.d * sizeof(elem<T>);
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
        const uint32_t off = row_bytes(p, i, rest, pitch);
        if constexpr (SIG) r.x[i] = load_word<T>(x, p.off + off);
        r.h[i] = load_word<T>(h, p.off + (back && off ? off - pitch : off));
    }
}

// As k_gated_scan from the last step on.  8 x 2048 x 4096 bf16 159 us: 821 MB at 5.2 TB/s, h read a step before
// dh, gate and x.
template <typename T, bool SIG, int LANES>
__global__ __launch_bounds__(LANES * kBackSpans) void k_gated_scan_backward(ScanBackArgs a) {
    constexpr int E = kCh<T>, CH = LANES * E, kChunkSteps = kSteps * kBackSpans;
    constexpr int kMine = kSteps * 64 / LANES;
    __shared__ ChunkState<kBackSpans, CH> s;
    const int wave = wave_of(), ch = threadIdx.x;      // the threads below CH compose a channel each
    const int64_t item = item_of(a.batch * a.tiles, a.runs);
    if (item < 0) return;
    const Place p = place_of<T, LANES>(item, a.tiles, a.steps, a.d);
    const int64_t len = length_of(a, p.b);
    const int64_t first = (int64_t)blockIdx.y * a.per;
    const int64_t behind = first + a.per < a.chunks ? first + a.per : a.chunks;
    const elem<T>* gate = static_cast<const elem<T>*>(a.gate);
    const elem<T>* dh = static_cast<const elem<T>*>(a.dh);
    BackWords even, odd;      // the words of two chunks, both in flight
    int64_t begin = (behind - 1) * kChunkSteps + wave * kMine;      // the wave's first step
    const int64_t least = first * kChunkSteps + wave * kMine, most = len > 0 ? len - 1 : 0;
    // chunks before the workgroup's first: that one again
    const auto read_in = [&](int64_t at, BackWords& r) {
        read_span<T>(gate, dh, p, at > least ? at : least, most, a.d, r.in);
    };
    const auto read_rest = [&](int64_t at, BackWords& r) {
        read_before<T, SIG>(a, p, at > least ? at : least, most, r);
    };
    read_in(begin, even);
    read_rest(begin, even);
    read_in(begin - kChunkSteps, odd);
    read_rest(begin - kChunkSteps, odd);
    float carry = 0.0f, start[E] = {};
    if (ch < CH) carry = enter<CH, SIG, true>(a, p, a.dstate, behind - 1, ch, p.c0 + ch < a.d);
    if (a.state0) load_state(a.state0 + p.b * a.d + p.c0 + p.at, p.left, start);
    const auto walk = [&](BackWords& words) {
        const int64_t t0 = begin + p.sub * kSteps;
        const bool full = begin + kMine <= len;
        float av[kSteps][E], dv[kSteps][E], take[kSteps][E];
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            word_of<T>(words.in.g[i], p.last, av[i]);
            word_of<T>(words.in.x[i], p.last, dv[i]);
            if constexpr (SIG) {
#pragma unroll
                for (int e = 0; e < E; ++e) sigmoids(av[i][e], av[i][e], take[i][e]);
            }
        }
        keep_past(full, len - t0, av, dv);
        read_in(begin - 2 * kChunkSteps, words);
#pragma unroll
        for (int e = 0; e < E; ++e) {
            Effect own{av[kSteps - 1][e], av[kSteps - 1][e] * dv[kSteps - 1][e]};
#pragma unroll
            for (int i = kSteps - 2; i >= 0; --i) {
                own.H = av[i][e] * (dv[i][e] + own.H);
                own.A *= av[i][e];
            }
            s.eff[p.span][p.at + e] = own;
        }
        __syncthreads();
        if (ch < CH) compose<SIG, true>(s, ch, carry);
        __syncthreads();
        float back[E];
#pragma unroll
        for (int e = 0; e < E; ++e) back[e] = s.in[p.span][p.at + e];
        const auto step = [&](int i, float (&dg)[E], float (&dx)[E], const float (&before)[E]) {
            float x[E];
            if constexpr (SIG) word_of<T>(words.x[i], p.last, x);
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const float total = dv[i][e] + back[e];
                if constexpr (SIG) {
                    dx[e] = take[i][e] * total;
                    dg[e] = av[i][e] * (before[e] - x[e]) * dx[e];
                } else {
                    dx[e] = total;
                    dg[e] = before[e] * total;
                }
                back[e] = av[i][e] * total;
            }
        };
        const int64_t row = (p.row0 + begin + kSteps - 1) * a.d + p.c0;
        elem<T>* dg_at = static_cast<elem<T>*>(a.dgate) + row;
        elem<T>* dx_at = static_cast<elem<T>*>(a.dx) + row;
        const uint32_t at = p.at + (uint32_t)(p.sub * kSteps) * (uint32_t)a.d;
        if (p.whole && begin > 0 && full) {
#pragma unroll
            for (int i = kSteps - 1; i >= 0; --i) {
                float h[E], dg[E], dx[E];
                word_of<T>(words.h[i], p.last, h);
                step(i, dg, dx, h);
                store_word<T>(dg_at + at, E, dg);
                store_word<T>(dx_at + at, E, dx);
                dg_at -= a.d;
                dx_at -= a.d;
            }
        } else {
#pragma unroll
            for (int i = kSteps - 1; i >= 0; --i) {
                const int64_t t = t0 + i;
                float h[E], dg[E], dx[E];
                word_of<T>(words.h[i], p.last, h);
                if (t == 0) {
#pragma unroll
                    for (int e = 0; e < E; ++e) h[e] = start[e];
                }
                step(i, dg, dx, h);
                if (t >= len) {
#pragma unroll
                    for (int e = 0; e < E; ++e) dg[e] = dx[e] = 0.0f;
                }
                if (t < a.steps) {
                    store_word<T>(dg_at + at, p.left, dg);
                    store_word<T>(dx_at + at, p.left, dx);
                }
                if (t == 0 && a.dstate0) store_state(a.dstate0 + p.b * a.d + p.c0 + p.at, p.left, back);
                dg_at -= a.d;
                dx_at -= a.d;
            }
        }
        read_rest(begin - 2 * kChunkSteps, words);
        begin -= kChunkSteps;
    };
    for (int64_t k = behind - 1; k >= first; k -= 2) {
        walk(even);
        if (k - 1 >= first) walk(odd);
    }
}

// ---------------------------------------------------------------- launches

struct ScanPlan {
    int64_t tiles, chunks, parts, per;
    int lanes;
    bool runs;
};

// One workgroup a tile of channels: of 64 words, or of 32 where twice as many tiles still have a compute
// unit each.  Forward and backward, us: 120 tiles of 64 (3 x 10007 x 2500 f32) 306 and 487, 240 of 32 194
// and 332; 128 (16 x 1024 x 1024 bf16) 38 and 46, 256 of 32 23 and 38; but 144 (9 x 2048 x 2048 bf16) 52 and
// 109, 288 of 32 53 and 124; 192 (6 x 2048 x 4096 bf16) 64 and 118, 384 of 32 74 and 144.  Where those are
// still few, the chunks' effects are taken first (gate and x read twice) and 512 workgroups share the
// sequences: 32 tiles of 32 (1 x 32768 x 2048 bf16) 133 and 211, a workgroup a tile 464 and 942; 128 (2 x
// 4096 x 4096 bf16) 58 and 94, a workgroup a tile 60 and 129; but 240 (3 x 10007 x 2500 f32) 194 and 332
// without it, 330 and 508 with it.
ScanPlan scan_plan(int64_t batch, int64_t steps, int64_t d, det_dtype dtype, int spans) {
    ScanPlan p;
    const int64_t es = (int64_t)lm_size(dtype), ch = 4 / es;
    p.lanes = d == 1 || cdiv(d, 64 * ch) * batch <= 128 ? 32 : 64;
    p.tiles = cdiv(d, p.lanes * (d == 1 ? 1 : ch));
    p.chunks = cdiv(steps, kSteps * spans);
    p.parts = 1;
    p.runs = d * es % 128 != 0;
    const int64_t wgs = p.tiles * batch;
    if (wgs <= 128 && p.chunks >= 4) {
        p.parts = cdiv(512, wgs);
        if (p.parts > p.chunks) p.parts = p.chunks;
    }
    p.per = cdiv(p.chunks, p.parts);
    p.parts = cdiv(p.chunks, p.per);
    return p;
}

// A grid holds fewer than 2^32 threads, and 65535 along y.  Workgroups have up to 1024 threads, and a
// launch a multiple of 8 of them (item_of), so the most that fits is one too.
constexpr int64_t kGridTiles = 4194296, kGridChunks = 65535;
static_assert(kGridTiles % 8 == 0 && kGridTiles * 64 * kSpans < (int64_t)1 << 32, "threads of a grid");

template <typename T>
void from_sequence(ScanArgs& a, int64_t b) {
    const int64_t n = b * a.steps * a.d * (int64_t)sizeof(T);
    a.gate = static_cast<const char*>(a.gate) + n;
    a.x = static_cast<const char*>(a.x) + n;
    a.h = static_cast<char*>(a.h) + n;
    if (a.state0) a.state0 += b * a.d;
    if (a.state) a.state += b * a.d;
    if (a.lengths) a.lengths += b;
}

template <typename T>
void from_sequence(ScanBackArgs& a, int64_t b) {
    const int64_t n = b * a.steps * a.d * (int64_t)sizeof(T);
    a.dh = static_cast<const char*>(a.dh) + n;
    a.gate = static_cast<const char*>(a.gate) + n;
    a.x = static_cast<const char*>(a.x) + n;
    a.h = static_cast<const char*>(a.h) + n;
    a.dgate = static_cast<char*>(a.dgate) + n;
    a.dx = static_cast<char*>(a.dx) + n;
    if (a.state0) a.state0 += b * a.d;
    if (a.dstate) a.dstate += b * a.d;
    if (a.dstate0) a.dstate0 += b * a.d;
    if (a.lengths) a.lengths += b;
}

template <typename T, bool SIG, int LANES>
det_status scan_as(const ScanArgs& all, const ScanPlan& p, hipStream_t s) {
    const dim3 block(LANES * kSpans);
    const int64_t most = kGridTiles / p.tiles;      // sequences of a launch
    for (int64_t b = 0; b < all.batch; b += most) {
        ScanArgs a = all;
        from_sequence<elem<T>>(a, b);
        a.batch = all.batch - b < most ? all.batch - b : most;
        const unsigned wgs = (unsigned)(cdiv(p.tiles * a.batch, 8) * 8);
        for (int64_t k = 0; p.parts > 1 && k < p.chunks - 1; k += kGridChunks) {
            const int64_t n = p.chunks - 1 - k < kGridChunks ? p.chunks - 1 - k : kGridChunks;
            KernelTimer kt("k_gated_scan_chunks", s);
            k_gated_scan_chunks<T, SIG, LANES><<<dim3(wgs, (unsigned)n), block, 0, s>>>(a, k);
        }
        KernelTimer kt("k_gated_scan", s);
        k_gated_scan<T, SIG, LANES><<<dim3(wgs, (unsigned)p.parts), block, 0, s>>>(a);
        const det_status st = launch_status();
        if (st != DET_SUCCESS) return st;
    }
    return DET_SUCCESS;
}

template <typename T, bool SIG>
det_status scan_typed(const ScanArgs& a, const ScanPlan& p, hipStream_t s) {
    if (a.steps <= kSteps) {
        const int64_t items = a.batch * cdiv(a.d, kVec<T>);
        KernelTimer kt("k_gated_scan_steps", s);
        k_gated_scan_steps<T, SIG><<<dim3((unsigned)cdiv(items, 256)), dim3(256), 0, s>>>(a);
        return launch_status();
    }
    if constexpr (sizeof(T) == 2) {
        if (a.d == 1) return scan_as<Lone<T>, SIG, 32>(a, p, s);
    }
    return p.lanes == 32 ? scan_as<T, SIG, 32>(a, p, s) : scan_as<T, SIG, 64>(a, p, s);
}

template <typename T, bool SIG, int LANES>
det_status scan_back_as(const ScanBackArgs& all, const ScanPlan& p, hipStream_t s) {
    const dim3 block(LANES * kBackSpans);
    const int64_t most = kGridTiles / p.tiles;
    for (int64_t b = 0; b < all.batch; b += most) {
        ScanBackArgs a = all;
        from_sequence<elem<T>>(a, b);
        a.batch = all.batch - b < most ? all.batch - b : most;
        const unsigned wgs = (unsigned)(cdiv(p.tiles * a.batch, 8) * 8);
        for (int64_t k = 1; p.parts > 1 && k < p.chunks; k += kGridChunks) {
            const int64_t n = p.chunks - k < kGridChunks ? p.chunks - k : kGridChunks;
            KernelTimer kt("k_gated_scan_chunks_back", s);
            k_gated_scan_chunks_back<T, SIG, LANES><<<dim3(wgs, (unsigned)n), block, 0, s>>>(a, k);
        }
        KernelTimer kt("k_gated_scan_backward", s);
        k_gated_scan_backward<T, SIG, LANES><<<dim3(wgs, (unsigned)p.parts), block, 0, s>>>(a);
        const det_status st = launch_status();
        if (st != DET_SUCCESS) return st;
    }
    return DET_SUCCESS;
}

template <typename T, bool SIG>
det_status scan_back_typed(const ScanBackArgs& a, const ScanPlan& p, hipStream_t s) {
    if constexpr (sizeof(T) == 2) {
        if (a.d == 1) return scan_back_as<Lone<T>, SIG, 32>(a, p, s);
    }
    return p.lanes == 32 ? scan_back_as<T, SIG, 32>(a, p, s) : scan_back_as<T, SIG, 64>(a, p, s);
}

}  // namespace

namespace {

size_t effect_bytes(const ScanPlan& p, int64_t batch, det_dtype dtype) {
    const size_t ch = 4 / lm_size(dtype);      // channels of a word
    return p.parts > 1 ? round_up((size_t)p.chunks * batch * p.tiles * p.lanes * ch * 8, 256) : 256;
}

}  // namespace

size_t gated_scan_workspace(int64_t batch, int64_t steps, int64_t d, det_dtype dtype) {
    const ScanPlan p = scan_plan(batch, steps, d, dtype, kSpans);
    return effect_bytes(p, batch, dtype);
}

size_t gated_scan_backward_workspace(int64_t batch, int64_t steps, int64_t d, det_dtype dtype) {
    const ScanPlan p = scan_plan(batch, steps, d, dtype, kBackSpans);
    return effect_bytes(p, batch, dtype);
}

det_status gated_scan_launch(const ScanCall& c, void* ws, hipStream_t s) {
    const ScanPlan p = scan_plan(c.batch, c.steps, c.d, c.dtype, kSpans);
    const ScanArgs a{c.gate, c.x, c.state0, c.lengths, c.h, c.state, static_cast<Effect*>(ws),
                     c.batch, c.steps, c.d, p.tiles, p.chunks, p.per, p.runs};
    switch (c.dtype) {
        case DET_F32: return c.sigmoid ? scan_typed<float, true>(a, p, s) : scan_typed<float, false>(a, p, s);
        case DET_F16:
            return c.sigmoid ? scan_typed<_Float16, true>(a, p, s) : scan_typed<_Float16, false>(a, p, s);
        default:
            return c.sigmoid ? scan_typed<__bf16, true>(a, p, s) : scan_typed<__bf16, false>(a, p, s);
    }
}

det_status gated_scan_backward_launch(const ScanBackCall& c, void* ws, hipStream_t s) {
    const ScanPlan p = scan_plan(c.batch, c.steps, c.d, c.dtype, kBackSpans);
    const ScanBackArgs a{c.dh, c.gate, c.x, c.h, c.state0, c.dstate, c.lengths, c.dgate, c.dx,
                         c.dstate0, static_cast<Effect*>(ws), c.batch, c.steps, c.d, p.tiles,
                         p.chunks, p.per, p.runs};
    switch (c.dtype) {
        case DET_F32:
            return c.sigmoid ? scan_back_typed<float, true>(a, p, s) : scan_back_typed<float, false>(a, p, s);
        case DET_F16:
            return c.sigmoid ? scan_back_typed<_Float16, true>(a, p, s)
                             : scan_back_typed<_Float16, false>(a, p, s);
        default:
            return c.sigmoid ? scan_back_typed<__bf16, true>(a, p, s)
                             : scan_back_typed<__bf16, false>(a, p, s);
    }
}

}  // namespace det
