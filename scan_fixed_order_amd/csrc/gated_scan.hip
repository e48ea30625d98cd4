// gated_scan.hip -- the gated linear recurrence over [batch][steps][d], channel by channel, and its
// backward pass.
//
// Mathematics:  h[t] = a[t] h[t-1] + b[t], h[-1] the given state or 0;  a = gate, b = x, or with
// sigmoid gates a = 1 / (1 + e^-gate), b = (1 - a) x.  Backwards, with E the gradient that reaches
// h[t] from behind (the final state's, or 0, at the last step):
//   G[t] = dh[t] + E[t+1];  E[t] = a[t] G[t];  the first state's gradient is E[0]
//   dx = G, dgate = G h[t-1];  sigmoid gates: dx = (1 - a) G, dgate = a (1 - a) (h[t-1] - x) G
// Steps at or past a sequence's length keep the state and have h, dx and dgate 0.
//
// Order, fixed by a step's own position: a span of kSteps steps is a chain of fused multiply-adds
// from its first step's incoming state; kSpans neighbouring spans make a chunk.  A span's
// effect on a state is (A, H): h -> A h + H, its chain from 0 and its product of a.  The effects of
// a chunk's spans are composed from the first on, applied to the chunk's incoming state, and give
// each span's; a chunk's whole effect gives the next chunk's.  (Backwards the same from the last
// step, span and chunk on.)  The same bits come out whether one workgroup walks all chunks of its
// channels or several take a part each.
#include "det_internal.h"
#include "lm_device.h"

namespace det {
namespace {

constexpr int kSteps = 8;                     // steps of a span: a wave's share of a chunk
constexpr int kSpans = 16;                    // spans of a chunk: waves of a workgroup
constexpr int kChunkSteps = kSteps * kSpans;

// Channels of a lane: one 32-bit word of a row, so a wave's load of a step takes 256 neighbouring bytes.
template <typename T>
constexpr int kCh = 4 / sizeof(T);

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

typedef uint32_t u32_a2 __attribute__((aligned(2)));

// The word of channels c .. of a row of d: the row's last word where it reaches past the end, whose
// element `word_of` moves to the front.  Any c.
template <typename T>
__device__ __forceinline__ uint32_t load_word(const T* row, int64_t c, int64_t d) {
    if constexpr (sizeof(T) == 4) {
        return __float_as_uint(row[c < d ? c : d - 1]);
    } else {
        if (d < 2) return (uint32_t)__builtin_bit_cast(uint16_t, row[0]);
        return *reinterpret_cast<const u32_a2*>(row + (c + 2 <= d ? c : d - 2));
    }
}

template <typename T>
__device__ __forceinline__ void word_of(uint32_t r, bool last, float (&v)[kCh<T>]) {
    if constexpr (sizeof(T) == 4) {
        v[0] = __uint_as_float(r);
    } else {
        if (last) r >>= 16;      // the row's last channel, alone
        if constexpr (__is_same(T, _Float16)) {
            v[0] = (float)__builtin_bit_cast(_Float16, (uint16_t)r);
            v[1] = (float)__builtin_bit_cast(_Float16, (uint16_t)(r >> 16));
        } else {
            v[0] = __uint_as_float(r << 16);
            v[1] = __uint_as_float(r & 0xFFFF0000u);
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
__device__ __forceinline__ void store_word(T* p, int64_t n, const float (&v)[kCh<T>]) {
    if constexpr (sizeof(T) == 4) {
        if (n > 0) *p = v[0];
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

template <int N>
__device__ __forceinline__ void load_state(const float* p, int64_t n, float (&v)[N]) {
#pragma unroll
    for (int e = 0; e < N; ++e) v[e] = e < n ? p[e] : 0.0f;
}

template <int N>
__device__ __forceinline__ void store_state(float* p, int64_t n, const float (&v)[N]) {
#pragma unroll
    for (int e = 0; e < N; ++e)
        if (e < n) p[e] = v[e];
}

// 1 / (1 + e^-x), within (3 + |x|) 2^-23 relative to it; 0 below -88
__device__ __forceinline__ float sigmoid_of(float x) {
    return __builtin_amdgcn_rcpf(1.0f + exp_fast(-x));
}

// a state c after a span of effect (A, H): a state of 0 leaves H also where A is infinite
__device__ __forceinline__ float after_span(float A, float c, float H) {
    return c == 0.0f ? H : fmaf(A, c, H);
}

struct ScanArgs {
    const void *gate, *x;
    const float* state0;
    const int32_t* lengths;
    void* h;
    float* state;
    float* effects;       // [chunk][A, H][batch * d], where several workgroups share a sequence
    int64_t batch, steps, d, tiles, chunks, per;      // per: chunks a workgroup walks
};

struct ScanBackArgs {
    const void *dh, *gate, *x, *h;
    const float *state0, *dstate;
    const int32_t* lengths;
    void *dgate, *dx;
    float* dstate0;
    float* effects;
    int64_t batch, steps, d, tiles, chunks, per;
};

// steps of sequence b that count
template <typename ARGS>
__device__ __forceinline__ int64_t length_of(const ARGS& a, int64_t b) {
    if (!a.lengths) return a.steps;
    const int64_t n = a.lengths[b];
    return n < 0 ? 0 : n < a.steps ? n : a.steps;
}

// what a workgroup's lane works on
struct Place {
    int64_t b, c, left, row0;      // sequence, first channel, channels to the row's end, first row
    bool last;                     // the row's last channel, alone in its word
};

template <typename T>
__device__ __forceinline__ Place place_of(int64_t item, int64_t tiles, int64_t steps, int64_t d) {
    Place p;
    p.b = item / tiles;
    p.c = (item % tiles * 64 + (threadIdx.x & 63)) * kCh<T>;
    p.left = d - p.c;
    p.row0 = p.b * steps;
    p.last = kCh<T> == 2 && p.left == 1 && d >= 2;
    return p;
}

// (a, b) of one step's word
template <typename T, bool SIG>
__device__ __forceinline__ void terms(uint32_t g, uint32_t x, bool last, bool inside,
                                      float (&a)[kCh<T>], float (&b)[kCh<T>]) {
    word_of<T>(g, last, a);
    word_of<T>(x, last, b);
#pragma unroll
    for (int e = 0; e < kCh<T>; ++e) {
        if constexpr (SIG) {
            b[e] = sigmoid_of(-a[e]) * b[e];
            a[e] = sigmoid_of(a[e]);
        }
        if (!inside) {
            a[e] = 1.0f;
            b[e] = 0.0f;
        }
    }
}

// the two words of each of a span's steps
struct SpanWords {
    uint32_t g[kSteps], x[kSteps];
};

template <typename T>
__device__ __forceinline__ void read_span(const T* gate, const T* x, const Place& p, int64_t t0,
                                          int64_t len, int64_t d, SpanWords& r) {
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
        // past the length the last step again: what lies there is not used
        const int64_t t = t0 + i < len ? t0 + i : len > 0 ? len - 1 : 0;
        r.g[i] = load_word(gate + (p.row0 + t) * d, p.c, d);
        r.x[i] = load_word(x + (p.row0 + t) * d, p.c, d);
    }
}

template <int E>
struct Effect {
    float A[E], H[E];
};

// the effects of spans in LDS, composed: of the spans before mine, and of all
template <int E, bool BACK>
__device__ __forceinline__ void compose(const Effect<E> (*s)[64], int wave, Effect<E>& mine,
                                        Effect<E>& all) {
    const int lane = threadIdx.x & 63;
    all = s[BACK ? kSpans - 1 : 0][lane];
#pragma unroll
    for (int k = 1; k < kSpans; ++k) {
        const int v = BACK ? kSpans - 1 - k : k;
        if (v == wave) mine = all;
        const Effect<E> one = s[v][lane];
#pragma unroll
        for (int e = 0; e < E; ++e) {
            all.H[e] = after_span(one.A[e], all.H[e], one.H[e]);
            all.A[e] *= one.A[e];
        }
    }
}

// the state that reaches the workgroup's first chunk
template <int E, typename ARGS, bool BACK>
__device__ __forceinline__ void enter(const ARGS& a, const Place& p, const float* from,
                                      int64_t chunk, float (&carry)[E]) {
#pragma unroll
    for (int e = 0; e < E; ++e) carry[e] = 0.0f;
    if (from) load_state(from + p.b * a.d + p.c, p.left, carry);
    const int64_t cells = a.batch * a.d;
    const int64_t count = BACK ? a.chunks - 1 - chunk : chunk;
#pragma unroll 4
    for (int64_t i = 0; i < count; ++i) {
        const float* at = a.effects + (BACK ? a.chunks - 1 - i : i) * 2 * cells + p.b * a.d + p.c;
        Effect<E> one;
        load_state(at, p.left, one.A);
        load_state(at + cells, p.left, one.H);
#pragma unroll
        for (int e = 0; e < E; ++e) carry[e] = after_span(one.A[e], carry[e], one.H[e]);
    }
}

// A workgroup walks chunks of 64 words of channels, a wave per span, the next chunk's words in
// flight while this one's effects go round.  One pass over gate and x: bound by HBM.
template <typename T, bool SIG>
__global__ __launch_bounds__(64 * kSpans) void k_gated_scan(ScanArgs a) {
    constexpr int E = kCh<T>;
    __shared__ Effect<E> s_eff[2][kSpans][64];
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const Place p = place_of<T>(blockIdx.x, a.tiles, a.steps, a.d);
    const int64_t len = length_of(a, p.b);
    const T* gate = static_cast<const T*>(a.gate);
    const T* x = static_cast<const T*>(a.x);
    const int64_t first = (int64_t)blockIdx.y * a.per;
    const int64_t behind = first + a.per < a.chunks ? first + a.per : a.chunks;
    SpanWords cur, next;
    read_span(gate, x, p, first * kChunkSteps + wave * kSteps, len, a.d, cur);
    float carry[E];
    enter<E, ScanArgs, false>(a, p, a.state0, first, carry);
    if (first == 0 && len == 0 && wave == 0) store_state(a.state + p.b * a.d + p.c, p.left, carry);
    for (int64_t k = first; k < behind; ++k) {
        const int64_t t0 = k * kChunkSteps + wave * kSteps;
        if (k + 1 < behind) read_span(gate, x, p, t0 + kChunkSteps, len, a.d, next);
        float av[kSteps][E], bv[kSteps][E];
        Effect<E> own;
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            terms<T, SIG>(cur.g[i], cur.x[i], p.last, t0 + i < len, av[i], bv[i]);
#pragma unroll
            for (int e = 0; e < E; ++e) {
                own.H[e] = i ? fmaf(av[i][e], own.H[e], bv[i][e]) : bv[i][e];
                own.A[e] = i ? own.A[e] * av[i][e] : av[i][e];
            }
        }
        s_eff[k & 1][wave][lane] = own;
        __syncthreads();
        Effect<E> mine, all;
        compose<E, false>(s_eff[k & 1], wave, mine, all);
        float h[E];
#pragma unroll
        for (int e = 0; e < E; ++e) {
            h[e] = wave ? after_span(mine.A[e], carry[e], mine.H[e]) : carry[e];
            carry[e] = after_span(all.A[e], carry[e], all.H[e]);
        }
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            const int64_t t = t0 + i;
#pragma unroll
            for (int e = 0; e < E; ++e) h[e] = fmaf(av[i][e], h[e], bv[i][e]);
            if (t < len) {
                store_word(static_cast<T*>(a.h) + (p.row0 + t) * a.d + p.c, p.left, h);
                if (t == len - 1) store_state(a.state + p.b * a.d + p.c, p.left, h);
            } else if (t < a.steps) {
                const float zero[E] = {};
                store_word(static_cast<T*>(a.h) + (p.row0 + t) * a.d + p.c, p.left, zero);
            }
        }
        cur = next;
    }
}

// The effect of every chunk but the last one (backwards: but the first), for workgroups that begin
// in the middle of a sequence.
template <typename T, bool SIG, bool BACK, typename ARGS>
__device__ __forceinline__ void chunk_effect(const ARGS& a, const T* gate, const T* other,
                                             int64_t chunk) {
    constexpr int E = kCh<T>;
    __shared__ Effect<E> s_eff[kSpans][64];
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const Place p = place_of<T>(blockIdx.x, a.tiles, a.steps, a.d);
    const int64_t len = length_of(a, p.b), t0 = chunk * kChunkSteps + wave * kSteps;
    SpanWords r;
    read_span(gate, other, p, t0, len, a.d, r);
    Effect<E> own;
#pragma unroll
    for (int j = 0; j < kSteps; ++j) {
        const int i = BACK ? kSteps - 1 - j : j;
        float av[E], bv[E];
        if constexpr (BACK) {
            word_of<T>(r.g[i], p.last, av);
            word_of<T>(r.x[i], p.last, bv);
#pragma unroll
            for (int e = 0; e < E; ++e) {
                if constexpr (SIG) av[e] = sigmoid_of(av[e]);
                if (t0 + i >= len) {
                    av[e] = 1.0f;
                    bv[e] = 0.0f;
                }
                // E -> a (dh + E)
                own.H[e] = av[e] * (j ? bv[e] + own.H[e] : bv[e]);
                own.A[e] = j ? own.A[e] * av[e] : av[e];
            }
        } else {
            terms<T, SIG>(r.g[i], r.x[i], p.last, t0 + i < len, av, bv);
#pragma unroll
            for (int e = 0; e < E; ++e) {
                own.H[e] = j ? fmaf(av[e], own.H[e], bv[e]) : bv[e];
                own.A[e] = j ? own.A[e] * av[e] : av[e];
            }
        }
    }
    s_eff[wave][lane] = own;
    __syncthreads();
    if (wave) return;
    Effect<E> mine, all;
    compose<E, BACK>(s_eff, -1, mine, all);
    const int64_t cells = a.batch * a.d;
    float* at = a.effects + chunk * 2 * cells + p.b * a.d + p.c;
    store_state(at, p.left, all.A);
    store_state(at + cells, p.left, all.H);
}

template <typename T, bool SIG>
__global__ __launch_bounds__(64 * kSpans) void k_gated_scan_chunks(ScanArgs a) {
    chunk_effect<T, SIG, false>(a, static_cast<const T*>(a.gate), static_cast<const T*>(a.x),
                                blockIdx.y);
}

template <typename T, bool SIG>
__global__ __launch_bounds__(64 * kSpans) void k_gated_scan_chunks_back(ScanBackArgs a) {
    chunk_effect<T, SIG, true>(a, static_cast<const T*>(a.gate), static_cast<const T*>(a.dh),
                               blockIdx.y + 1);
}

// At most kSteps steps: no spans to compose, a lane takes a vector of channels.
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
                x[e] = sigmoid_of(-g[e]) * x[e];
                g[e] = sigmoid_of(g[e]);
            }
            if (t < len) h[e] = fmaf(g[e], h[e], x[e]);
            o[e] = t < len ? as_float(h[e]) : 0.0f;
        }
        write_vec(static_cast<T*>(a.h) + at, left, o);
    }
    store_state(a.state + b * a.d + c, left, h);
}

// ---------------------------------------------------------------- backward

// the words of each of a span's steps: gate, dh, h one step before, x (sigmoid gates)
struct BackWords {
    uint32_t g[kSteps], dh[kSteps], h[kSteps], x[kSteps];
};

template <typename T, bool SIG>
__device__ __forceinline__ void read_back(const ScanBackArgs& a, const Place& p, int64_t t0,
                                          int64_t len, BackWords& r) {
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
        const int64_t t = t0 + i < len ? t0 + i : len > 0 ? len - 1 : 0;
        const int64_t row = (p.row0 + t) * a.d;
        r.g[i] = load_word(static_cast<const T*>(a.gate) + row, p.c, a.d);
        r.dh[i] = load_word(static_cast<const T*>(a.dh) + row, p.c, a.d);
        r.h[i] = load_word(static_cast<const T*>(a.h) + (t > 0 ? row - a.d : row), p.c, a.d);
        if constexpr (SIG) r.x[i] = load_word(static_cast<const T*>(a.x) + row, p.c, a.d);
    }
}

// As k_gated_scan from the last step on.
template <typename T, bool SIG>
__global__ __launch_bounds__(64 * kSpans) void k_gated_scan_backward(ScanBackArgs a) {
    constexpr int E = kCh<T>;
    __shared__ Effect<E> s_eff[2][kSpans][64];
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const Place p = place_of<T>(blockIdx.x, a.tiles, a.steps, a.d);
    const int64_t len = length_of(a, p.b);
    const int64_t first = (int64_t)blockIdx.y * a.per;
    const int64_t behind = first + a.per < a.chunks ? first + a.per : a.chunks;
    BackWords cur, next;
    read_back<T, SIG>(a, p, (behind - 1) * kChunkSteps + wave * kSteps, len, cur);
    float carry[E], start[E] = {};
    enter<E, ScanBackArgs, true>(a, p, a.dstate, behind - 1, carry);
    if (a.state0) load_state(a.state0 + p.b * a.d + p.c, p.left, start);
    for (int64_t k = behind - 1; k >= first; --k) {
        const int64_t t0 = k * kChunkSteps + wave * kSteps;
        if (k > first) read_back<T, SIG>(a, p, t0 - kChunkSteps, len, next);
        float av[kSteps][E], dv[kSteps][E];
        Effect<E> own;
#pragma unroll
        for (int i = kSteps - 1; i >= 0; --i) {
            word_of<T>(cur.g[i], p.last, av[i]);
            word_of<T>(cur.dh[i], p.last, dv[i]);
#pragma unroll
            for (int e = 0; e < E; ++e) {
                float keep = SIG ? sigmoid_of(av[i][e]) : av[i][e];
                if (t0 + i >= len) {
                    keep = 1.0f;
                    dv[i][e] = 0.0f;
                }
                const bool begins = i == kSteps - 1;
                own.H[e] = keep * (begins ? dv[i][e] : dv[i][e] + own.H[e]);
                own.A[e] = begins ? keep : own.A[e] * keep;
                if constexpr (!SIG) av[i][e] = keep;
            }
        }
        s_eff[k & 1][wave][lane] = own;
        __syncthreads();
        Effect<E> mine, all;
        compose<E, true>(s_eff[k & 1], wave, mine, all);
        float back[E];
#pragma unroll
        for (int e = 0; e < E; ++e) {
            back[e] = wave < kSpans - 1 ? after_span(mine.A[e], carry[e], mine.H[e]) : carry[e];
            carry[e] = after_span(all.A[e], carry[e], all.H[e]);
        }
#pragma unroll
        for (int i = kSteps - 1; i >= 0; --i) {
            const int64_t t = t0 + i;
            float h[E], x[E], dg[E], dx[E];
            word_of<T>(cur.h[i], p.last, h);
            if constexpr (SIG) word_of<T>(cur.x[i], p.last, x);
            const bool inside = t < len;
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const float before = t > 0 ? h[e] : start[e];
                const float total = dv[i][e] + back[e];
                if constexpr (SIG) {
                    const float keep = sigmoid_of(av[i][e]), take = sigmoid_of(-av[i][e]);
                    dx[e] = take * total;
                    dg[e] = keep * (before - x[e]) * dx[e];
                    if (inside) back[e] = keep * total;
                } else {
                    dx[e] = total;
                    dg[e] = before * total;
                    if (inside) back[e] = av[i][e] * total;
                }
                if (!inside) dx[e] = dg[e] = 0.0f;
            }
            if (t < a.steps) {
                const int64_t at = (p.row0 + t) * a.d + p.c;
                store_word(static_cast<T*>(a.dgate) + at, p.left, dg);
                store_word(static_cast<T*>(a.dx) + at, p.left, dx);
            }
            if (t == 0 && a.dstate0) store_state(a.dstate0 + p.b * a.d + p.c, p.left, back);
        }
        cur = next;
    }
}

// ---------------------------------------------------------------- launches

struct ScanPlan {
    int64_t tiles, chunks, parts, per;
};

// One workgroup a tile of channels, unless that leaves most compute units without one: then the
// chunks' effects are taken first (gate and x read twice) and several share a sequence.
ScanPlan scan_plan(int64_t batch, int64_t steps, int64_t d, det_dtype dtype) {
    ScanPlan p;
    p.tiles = cdiv(d, 64 * (4 / (int64_t)lm_size(dtype)));
    p.chunks = cdiv(steps, kChunkSteps);
    p.parts = 1;
    const int64_t wgs = p.tiles * batch;
    if (wgs <= 128 && p.chunks >= 4) {
        p.parts = cdiv(512, wgs);
        if (p.parts > p.chunks) p.parts = p.chunks;
    }
    p.per = cdiv(p.chunks, p.parts);
    p.parts = cdiv(p.chunks, p.per);
    return p;
}

template <typename T, bool SIG>
det_status scan_typed(const ScanArgs& a, const ScanPlan& p, hipStream_t s) {
    if (a.steps <= kSteps) {
        const int64_t items = a.batch * cdiv(a.d, kVec<T>);
        KernelTimer kt("k_gated_scan_steps", s);
        k_gated_scan_steps<T, SIG><<<dim3((unsigned)cdiv(items, 256)), dim3(256), 0, s>>>(a);
        return launch_status();
    }
    const unsigned wgs = (unsigned)(p.tiles * a.batch);
    if (p.parts > 1) {
        KernelTimer kt("k_gated_scan_chunks", s);
        k_gated_scan_chunks<T, SIG><<<dim3(wgs, (unsigned)(p.chunks - 1)), dim3(64 * kSpans), 0, s>>>(a);
        const det_status st = launch_status();
        if (st != DET_SUCCESS) return st;
    }
    KernelTimer kt("k_gated_scan", s);
    k_gated_scan<T, SIG><<<dim3(wgs, (unsigned)p.parts), dim3(64 * kSpans), 0, s>>>(a);
    return launch_status();
}

template <typename T, bool SIG>
det_status scan_back_typed(const ScanBackArgs& a, const ScanPlan& p, hipStream_t s) {
    const unsigned wgs = (unsigned)(p.tiles * a.batch);
    if (p.parts > 1) {
        KernelTimer kt("k_gated_scan_chunks_back", s);
        k_gated_scan_chunks_back<T, SIG><<<dim3(wgs, (unsigned)(p.chunks - 1)), dim3(64 * kSpans), 0, s>>>(a);
        const det_status st = launch_status();
        if (st != DET_SUCCESS) return st;
    }
    KernelTimer kt("k_gated_scan_backward", s);
    k_gated_scan_backward<T, SIG><<<dim3(wgs, (unsigned)p.parts), dim3(64 * kSpans), 0, s>>>(a);
    return launch_status();
}

}  // namespace

size_t gated_scan_workspace(int64_t batch, int64_t steps, int64_t d, det_dtype dtype) {
    const ScanPlan p = scan_plan(batch, steps, d, dtype);
    return p.parts > 1 ? round_up((size_t)p.chunks * 2 * batch * d * 4, 256) : 256;
}

size_t gated_scan_backward_workspace(int64_t batch, int64_t steps, int64_t d, det_dtype dtype) {
    return gated_scan_workspace(batch, steps, d, dtype);
}

det_status gated_scan_launch(const ScanCall& c, void* ws, hipStream_t s) {
    const ScanPlan p = scan_plan(c.batch, c.steps, c.d, c.dtype);
    const ScanArgs a{c.gate, c.x, c.state0, c.lengths, c.h, c.state, static_cast<float*>(ws),
                     c.batch, c.steps, c.d, p.tiles, p.chunks, p.per};
    switch (c.dtype) {
        case DET_F32: return c.sigmoid ? scan_typed<float, true>(a, p, s) : scan_typed<float, false>(a, p, s);
        case DET_F16:
            return c.sigmoid ? scan_typed<_Float16, true>(a, p, s) : scan_typed<_Float16, false>(a, p, s);
        default:
            return c.sigmoid ? scan_typed<__bf16, true>(a, p, s) : scan_typed<__bf16, false>(a, p, s);
    }
}

det_status gated_scan_backward_launch(const ScanBackCall& c, void* ws, hipStream_t s) {
    const ScanPlan p = scan_plan(c.batch, c.steps, c.d, c.dtype);
    const ScanBackArgs a{c.dh, c.gate, c.x, c.h, c.state0, c.dstate, c.lengths, c.dgate, c.dx,
                         c.dstate0, static_cast<float*>(ws), c.batch, c.steps, c.d, p.tiles,
                         p.chunks, p.per};
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
