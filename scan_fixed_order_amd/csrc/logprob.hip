// logprob.hip -- log probabilities of given tokens with the entropy and the best alternatives,
// and the logits' gradient.
//
// Mathematics, per row of logits x, z = scale * x, everything after the load in f32:
//   lse = log(sum exp z);  logp = z[target] - lse (0 where the target is not a token);
//   entropy = -sum p log p, p = exp(z - lse);  top: the largest logits, ties to the lower index;
//   dlogits = scale * (dlogp (hit - p) - dentropy * p * (log p + entropy)).
// One pass forward: s = sum exp(d) and w = sum exp(d) d with d = scale * (x - ref) against a running
// maximum ref of the logits give lse = scale * ref + log s and entropy = log s - w / s.  d is the
// difference times the scale, not scale * x less a scaled reference: where a mask has put -1e30 into
// a row, the rounding of that product alone is 1e22, far more than exp takes.  A term whose p is 0
// adds 0 to the entropy also where its logit is -inf.  A row without any mass (all logits -inf) has
// lse = -inf, entropy 0, logp -inf and gradient 0.
//
// Order: 1024 lanes share a row, lane L holding elements V (L + 1024 j) .. + V for j = 0, 1, ...
// (V = 8, 4 of f32);
// each adds its own in that order, then 64 neighbouring lanes join by the adjacent-lanes tree,
// then the 16 groups by the same tree.  How many threads play those lanes does not enter the
// order, nor do the other rows: a row's bits depend on its logits and the scale alone.
#include <float.h>

#include "det_internal.h"
#include "lm_device.h"

namespace det {
namespace {

constexpr int kLanes = 1024;              // lanes that share a row, in the order above
template <typename T>
constexpr int kTile = kLanes * kVec<T>;   // elements they take at a time
constexpr int kGroup = 32;                // neighbouring elements whose largest is kept for top
constexpr int kShort = 512;               // candidates of the short way to the top
constexpr float kFar = -1e30f;            // differences of references stop here (never -inf)
constexpr float kLn2 = 0.69314718055994531f;

// the largest of three; a quiet NaN loses (a signalling one takes what it was compared with along:
// the instruction answers it with a quiet NaN, which the next comparison drops)
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("v_max3_f32 %0, %1, %2, %3" : "=v"(r) : "v"(a), "v"(b), "v"(c));
    return r;
}

// whole numbers that order like the values, both zeros alike, from 1 on; NaN like -inf
__device__ __forceinline__ uint32_t order_key(float x) {
    x = x >= -INFINITY ? x + 0.0f : -INFINITY;
    const uint32_t u = __float_as_uint(x);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float key_value(uint32_t k) {
    return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}

struct LogpArgs {
    const void* logits;
    const int64_t* targets;
    float *logp, *entropy, *lse, *top_logp;
    int64_t* top_ids;
    int64_t stride, rows, vocab;
    int top;
    float scale, scale2;       // scale2 = scale * log2(e)
};

// One lane's running sums against its reference, the largest of its values so far.  (A reference
// that values may pass by 8 spares most lanes the rescaling, 3 % of 2048 x 131072 bf16 with
// alternatives, but then log(sum) and the target cancel in a row of one likely token: its log
// probability was off by 20 times 2^-24, where 1.4 times is what a float sum costs.)
struct Part {
    float ref, s, w;      // w in units of 2^x: times log(2) at the end
};

__device__ __forceinline__ void rebase(Part& p, float ref, float scale2) {
    const float dm = fmaxf((p.ref - ref) * scale2, kFar);
    const float f = __builtin_amdgcn_exp2f(dm);
    p.w = fmaf(p.s, dm, p.w) * f;
    p.s = p.s * f;
    p.ref = ref;
}

// over 16 neighbouring lanes, by the adjacent-lanes tree
__device__ __forceinline__ float sum16(float v) {
    v = v + xor_partner<1>(v);
    v = v + xor_partner<2>(v);
    v = v + xor_partner<4>(v);
    return v + xor_partner<8>(v);
}

// adds a vector of N logits; `largest`: their maximum (NaN ignored)
template <int N>
__device__ __forceinline__ void take(Part& p, const float (&x)[N], float largest, float scale2) {
    if (largest > p.ref) rebase(p, largest, scale2);
    float e[N], d[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        d[i] = (x[i] - p.ref) * scale2;
        e[i] = __builtin_amdgcn_exp2f(d[i]);
    }
    float w0 = e[0] * d[0], w1 = e[1] * d[1];
#pragma unroll
    for (int i = 2; i < N; i += 2) {
        w0 = fmaf(e[i], d[i], w0);
        w1 = fmaf(e[i + 1], d[i + 1], w1);
    }
    float w = w0 + w1;
    if (w != w) {      // 0 * -inf among them: such a term counts as 0
        w = 0.0f;
#pragma unroll
        for (int i = 0; i < N; ++i) w += e[i] == 0.0f ? 0.0f : e[i] * d[i];
    }
    float s = (e[0] + e[1]) + (e[2] + e[3]);
    if constexpr (N == 8) s += (e[4] + e[5]) + (e[6] + e[7]);
    p.s += s;
    p.w += w;
}

template <int N>
__device__ __forceinline__ float largest_of(const float (&x)[N]) {
    if constexpr (N == 4) return max3(max3(x[0], x[1], x[2]), x[3], -INFINITY);
    else return max3(max3(x[0], x[1], x[2]), max3(x[3], x[4], x[5]), max3(x[6], x[7], -INFINITY));
}

// groups of a super-group: 64 of them cover the row; odd, so that lanes that read one group of
// each fall on different LDS banks
__host__ __device__ constexpr int64_t super_len(int64_t vocab) {
    return ((vocab + kGroup - 1) / kGroup + 63) / 64 | 1;
}

// LDS of the top logits' search
struct Search {
    uint32_t super[64];                     // largest key of each super-group
    uint32_t pick[kShort];                  // groups whose logits may be candidates
    unsigned long long cand[kShort];        // candidates: key, then the lower index first
    uint32_t bound;                         // a key that at least `top` logits reach
    int picks, cands;
};

// Ranks n candidates (their places differ from run to run, their ranks do not) and writes the
// first `top`; 8 lanes a candidate.
template <int BLOCK>
__device__ __forceinline__ void rank_candidates(const LogpArgs& a, int64_t row,
                                                const unsigned long long* cand, int n, float ref,
                                                float log_s) {
    const int part = threadIdx.x & 7;
#pragma unroll 1
    for (int i0 = 0; i0 < n; i0 += BLOCK / 8) {
        const int i = i0 + (threadIdx.x >> 3);
        const unsigned long long c = i < n ? cand[i] : 0;
        uint32_t rank = 0;
#pragma unroll 2
        for (int j = part; j < n; j += 8) rank += cand[j] > c;
        rank += xor_partner<1>(rank);
        rank += xor_partner<2>(rank);
        rank += xor_partner<4>(rank);
        if (part == 0 && i < n && (int)rank < a.top) {
            a.top_ids[row * a.top + rank] = (int64_t)(uint32_t)~(uint32_t)c;
            a.top_logp[row * a.top + rank] =
                fmaf(key_value((uint32_t)(c >> 32)) - ref, a.scale, -log_s);
        }
    }
}

// Candidates among the logits of groups pick[0 .. n): those whose key reaches `bound`, as far as
// `room` goes (*count counts all).
template <typename T, int BLOCK>
__device__ __forceinline__ void gather_candidates(const LogpArgs& a, const T* x,
                                                  const uint32_t* pick, int n, uint32_t bound,
                                                  unsigned long long* cand, int room, int* count) {
#pragma unroll 1
    for (int i = threadIdx.x; i < n * kGroup; i += BLOCK) {
        const uint32_t id = pick[i / kGroup] * kGroup + i % kGroup;
        if (id >= a.vocab) continue;
        const uint32_t k = order_key((float)x[id]);
        if (k < bound) continue;
        const int at = atomicAdd(count, 1);
        if (at < room) cand[at] = (unsigned long long)k << 32 | (uint32_t)~id;
    }
}

// largest key of a group's logits, one by one
template <typename T>
__device__ __forceinline__ uint32_t group_key(const LogpArgs& a, const T* x, int group) {
    const int64_t first = (int64_t)group * kGroup, n = a.vocab - first;
    uint32_t k = 0;
#pragma unroll 1
    for (int i = 0; i < kGroup && i < n; ++i) k = umax(k, order_key((float)x[first + i]));
    return k;
}

// The `top` largest logits of a row.  On entry s_key holds every group's largest logit, which are
// not to be trusted where the row holds a NaN (`suspect`); they are replaced by their order keys (0
// behind the last group), in 64 super-groups of super_len groups.
//
// The top-th largest of the super-groups' maxima is a bound that at least `top` logits reach, and
// few more do in most rows: these are ranked against each other.  Where too many reach it (long
// runs of equal logits, logits in ascending order), one wave picks the top groups one by one
// through a tournament of the super-groups instead, and their logits are the candidates: the
// top logits lie in the top groups, since each of these holds one that beats every logit of the
// others.
template <typename T, int BLOCK>
__device__ void pick_top(const LogpArgs& a, int64_t row, const T* x, uint32_t* s_key, Search& s,
                         float ref, float log_s, bool suspect) {
    const int groups = (int)((a.vocab + kGroup - 1) / kGroup);
    const int len = (int)super_len(a.vocab);
    const int lane = threadIdx.x & 63;
    // kParts neighbouring lanes a super-group
    constexpr int kParts = BLOCK / 64, kOthers = 64 / kParts;
    const int sg = threadIdx.x / kParts, part = threadIdx.x % kParts;
    {
        uint32_t m = 0;
#pragma unroll 4
        for (int i = part; i < len; i += kParts) {
            const int at = sg * len + i;
            const uint32_t k = at >= groups ? 0
                               : suspect    ? group_key(a, x, at)
                                            : order_key(__uint_as_float(s_key[at]));
            s_key[at] = k;
            m = umax(m, k);
        }
        m = umax(m, xor_partner<1>(m));
        m = umax(m, xor_partner<2>(m));
        if constexpr (kParts >= 8) m = umax(m, xor_partner<4>(m));
        if constexpr (kParts >= 16) m = umax(m, xor_partner<8>(m));
        if (part == 0) s.super[sg] = m;
        if (threadIdx.x == 0) s.picks = s.cands = 0;
    }
    __syncthreads();
    {
        const uint32_t mine = s.super[sg];
        uint32_t rank = 0;
#pragma unroll 4
        for (int i = 0; i < kOthers; ++i) {
            const int j = part * kOthers + i;
            const uint32_t k = s.super[j];
            rank += k > mine || (k == mine && j < sg);
        }
        rank += xor_partner<1>(rank);
        rank += xor_partner<2>(rank);
        if constexpr (kParts >= 8) rank += xor_partner<4>(rank);
        if constexpr (kParts >= 16) rank += xor_partner<8>(rank);
        // 0: a super-group behind the row's end, so that every logit counts
        if (part == 0 && (int)rank == a.top - 1) s.bound = umax(mine, 1u);
    }
    __syncthreads();
    const uint32_t bound = s.bound;
#pragma unroll 1
    for (int i = threadIdx.x; i < groups; i += BLOCK)
        if (s_key[i] >= bound) {
            const int at = atomicAdd(&s.picks, 1);
            if (at < kShort) s.pick[at] = (uint32_t)i;
        }
    __syncthreads();
    bool done = s.picks <= kShort;
    if (done) {
        gather_candidates<T, BLOCK>(a, x, s.pick, s.picks, bound, s.cand, kShort, &s.cands);
        __syncthreads();
        done = s.cands <= kShort;
        if (done) rank_candidates<BLOCK>(a, row, s.cand, s.cands, ref, log_s);
    }
    if (!done) {
        const int picks = a.top < groups ? a.top : groups;
        __syncthreads();      // s.picks and s.cands are read
        if (threadIdx.x < 64) {
            uint32_t mine = s.super[lane], best = 0;
            for (int r = 0; r < picks; ++r) {
                best = wave_max(mine);
                const int from = __ffsll((unsigned long long)__ballot(mine == best)) - 1;
                // the first group of that super-group with this key, and the largest other key
                uint32_t rest = 0;
                int at = -1;
                for (int i = 0; i < len; i += 64) {
                    uint32_t k = i + lane < len ? s_key[from * len + i + lane] : 0;
                    const unsigned long long hits = __ballot(k == best);
                    if (at < 0 && hits) {
                        const int l = __ffsll(hits) - 1;
                        at = i + l;
                        if (lane == l) k = 0;
                    }
                    rest = umax(rest, k);
                }
                rest = wave_max(rest);
                if (lane == from) mine = rest;
                if (lane == 0) {
                    s.pick[r] = from * len + at;
                    s_key[from * len + at] = 0;
                }
                wave_sync();
            }
            // with fewer groups than places every logit is a candidate
            if (lane == 0) {
                s.bound = picks < a.top ? 1u : best;
                s.cands = 0;
            }
        }
        __syncthreads();
        unsigned long long* cand = reinterpret_cast<unsigned long long*>(s_key);
        gather_candidates<T, BLOCK>(a, x, s.pick, picks, s.bound, cand, picks * kGroup, &s.cands);
        __syncthreads();
        rank_candidates<BLOCK>(a, row, cand, s.cands, ref, log_s);
    }
    __syncthreads();      // s_key and s are written again
}

// One row per workgroup, each logit read once; 1024 or 512 threads for few rows, where a compute
// unit's vector rate bounds (about 17 logits a nanosecond), 256 for many.  2048 x 131072 bf16: 89 us
// (6.0 TB/s, bound by HBM), with 5 alternatives 97 us (5.5 TB/s: 11 vector instructions and an
// exponential a logit fill the vector units, and a row's search runs for 2 us).  256 x 131072 with
// 5 alternatives 17 us with 1024 threads a row, 512 rows 31 us with 512.
template <typename T, int BLOCK, bool TOP, bool ONCE>
__global__ __launch_bounds__(BLOCK) void k_token_logprobs(LogpArgs a) {
    constexpr int kSets = kLanes / BLOCK;       // lanes a thread plays
    constexpr int kSteps = 32 / kVec<T> / kSets;   // tiles whose loads are in flight together
    extern __shared__ __align__(16) uint32_t s_key[];
    __shared__ Part s_part[2][kLanes / 64];      // rows take turns: no second barrier a row
    __shared__ Search s_search;      // not laid out where nothing is searched
    const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
    int parity = 0;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const T* x = static_cast<const T*>(a.logits) + row * a.stride;
        const int64_t target = a.targets[row];
        const bool scored = target >= 0 && target < a.vocab;
        const float picked = scored ? (float)x[target] : 0.0f;
        Part p[kSets];
#pragma unroll
        for (int u = 0; u < kSets; ++u) p[u] = Part{-FLT_MAX, 0.0f, 0.0f};
        const auto one = [&](int64_t c, int u, const float(&v)[kVec<T>], bool keep) {
            const float largest = largest_of(v);
            if constexpr (TOP) {
                // (fmaxf would quiet its operands first, an instruction each)
                float g = largest, other = xor_partner<1>(g);
                g = max3(g, other, other);
                other = xor_partner<2>(g);
                g = max3(g, other, other);
                if constexpr (kGroup / kVec<T> == 8) {
                    other = xor_partner<4>(g);
                    g = max3(g, other, other);
                }
                if (keep && lane % (kGroup / kVec<T>) == 0) s_key[c / kGroup] = __float_as_uint(g);
            }
            if (keep) take(p[u], v, largest, a.scale2);
        };
        const int64_t whole = a.vocab / (kTile<T> * kSteps);
        for (int64_t i = 0; i < whole; ++i) {
            u32x4 raw[kSteps][kSets];
#pragma unroll
            for (int q = 0; q < kSteps; ++q)
#pragma unroll
                for (int u = 0; u < kSets; ++u)
                    raw[q][u] = load_vec<ONCE>(x + (i * kSteps + q) * kTile<T> + kVec<T> * (t + u * BLOCK));
#pragma unroll
            for (int q = 0; q < kSteps; ++q)
#pragma unroll
                for (int u = 0; u < kSets; ++u) {
                    float v[kVec<T>];
                    unpack<T>(raw[q][u], v);
                    one((i * kSteps + q) * kTile<T> + kVec<T> * (t + u * BLOCK), u, v, true);
                }
        }
        for (int64_t base = whole * kSteps * kTile<T>; base < a.vocab; base += kTile<T>) {
#pragma unroll
            for (int u = 0; u < kSets; ++u) {
                if (base + kVec<T> * u * BLOCK >= a.vocab) break;
                const int64_t c = base + kVec<T> * (t + u * BLOCK);
                float v[kVec<T>];
                unpack<T>(settle<T>(load_row(x, c, a.vocab), c, a.vocab), v);
#pragma unroll
                for (int i = 0; i < kVec<T>; ++i)
                    if (c + i >= a.vocab) v[i] = -INFINITY;
                one(c, u, v, c < a.vocab);
            }
        }
        // 64 neighbouring lanes against their own largest reference, then those 16 groups
#pragma unroll
        for (int u = 0; u < kSets; ++u) {
            const float ref = wave_max(p[u].ref);
            rebase(p[u], ref, a.scale2);
            const float s = wave_pw(p[u].s), w = wave_pw(p[u].w);
            if (lane == 0) s_part[parity][wave + u * (BLOCK / 64)] = Part{ref, s, w};
        }
        __syncthreads();
        Part g = s_part[parity][lane & 15];      // every wave joins them for itself
        parity ^= 1;
        float ref = g.ref;
        ref = fmaxf(ref, xor_partner<1>(ref));
        ref = fmaxf(ref, xor_partner<2>(ref));
        ref = fmaxf(ref, xor_partner<4>(ref));
        ref = fmaxf(ref, xor_partner<8>(ref));
        rebase(g, ref, a.scale2);
        const float s = sum16(g.s), w = sum16(g.w), log_s = logf(s);
        const bool none = s == 0.0f;
        if (t == 0) {
            a.lse[row] = fmaf(ref, a.scale, log_s);
            a.entropy[row] = none ? 0.0f : log_s - w * kLn2 / s;
            a.logp[row] = !scored ? 0.0f : none ? -INFINITY : fmaf(picked - ref, a.scale, -log_s);
        }
        if constexpr (TOP)
            pick_top<T, BLOCK>(a, row, x, s_key, s_search, none ? 0.0f : ref, none ? 0.0f : log_s,
                               s != s);
    }
}

// ---------------------------------------------------------------- backward

struct LogpBackArgs {
    const void* logits;
    const int64_t* targets;
    const float *lse, *dlogp, *entropy, *dentropy;      // the last two NULL: no entropy term
    void* dlogits;
    int64_t stride, dstride, rows, vocab, tiles;
    float scale;
};

constexpr int kBackTile = 8192;                           // elements a workgroup takes at a time

// lse is a float: beyond this its rounding moves every p = exp(z - lse) by more than 2^-16, in a row of
// the type's lowest values nothing of log(sum) is left in it, and with a scale it may be infinite.
// Such a row's sum is taken again.
constexpr float kFarLse = 256.0f;

// What a row's gradient takes besides its logits
struct BackTerms {
    int64_t target;               // -1: not scored
    float dlogp, dent, both;      // both = dlogp + dentropy * entropy
};

__device__ __forceinline__ float logit_gradient(float log, const BackTerms& r, bool hit) {
    const float p = exp_fast(log);
    // below -1000 p is 0 and -inf must not meet it
    const float d = -p * fmaf(r.dent, fmaxf(log, -1000.0f), r.both);
    return hit ? d + r.dlogp : d;
}

// A row whose lse is far from zero, by one workgroup: its maximum, its sum against that, and only
// then the gradient (which may replace the logits); 0 where all logits are -inf.  Order of the sum:
// a lane's vectors, the adjacent-lanes tree, the four waves.
template <typename T>
__device__ void far_row(const LogpBackArgs& a, const T* x, T* out, const BackTerms& r) {
    __shared__ float s_max[4], s_sum[4];
    const int wave = threadIdx.x >> 6;
    float v[kVec<T>], top = -INFINITY;
    for (int64_t c = kVec<T> * threadIdx.x; c < a.vocab; c += 256 * kVec<T>) {
        read_vec(x + c, a.vocab - c, -INFINITY, v);
#pragma unroll
        for (int i = 0; i < kVec<T>; ++i) top = fmaxf(top, v[i]);
    }
    top = wave_max(top);
    if ((threadIdx.x & 63) == 0) s_max[wave] = top;
    __syncthreads();
    top = fmaxf(fmaxf(s_max[0], s_max[1]), fmaxf(s_max[2], s_max[3]));
    const bool none = top == -INFINITY;
    float sum = 0.0f;
    for (int64_t c = kVec<T> * threadIdx.x; c < a.vocab; c += 256 * kVec<T>) {
        read_vec(x + c, a.vocab - c, -INFINITY, v);
#pragma unroll
        for (int i = 0; i < kVec<T>; ++i) sum += exp_fast((v[i] - top) * a.scale);
    }
    sum = wave_pw(sum);
    if ((threadIdx.x & 63) == 0) s_sum[wave] = sum;
    __syncthreads();
    const float log_s = logf(((s_sum[0] + s_sum[1]) + s_sum[2]) + s_sum[3]);
    for (int64_t c = kVec<T> * threadIdx.x; c < a.vocab; c += 256 * kVec<T>) {
        read_vec(x + c, a.vocab - c, -INFINITY, v);
        const int64_t hit = r.target - c;
#pragma unroll
        for (int i = 0; i < kVec<T>; ++i) {
            const float d = logit_gradient(fmaf(v[i] - top, a.scale, -log_s), r, i == hit);
            v[i] = none ? 0.0f : d * a.scale;
        }
        write_vec(out + c, a.vocab - c, v);
    }
    __syncthreads();      // the LDS slots are written again
}

// Each logit read once, each gradient written once; nothing is summed (but in far_row).  A lane's
// loads are all on their way before its first value is used.  Bound by HBM: 4096 x 65536 bf16 178
// us (6.0 TB/s; 176 without far rows, 182 with them told apart before the loads, 189 after; 190
// with a branch between whole and partial vectors at each load), 517 x 50021 f32 with the forward
// pass 64 us (4.8 TB/s; rows there start off 16 bytes), 69 with such a branch.
template <typename T, bool ONCE>
__global__ __launch_bounds__(256) void k_token_logprobs_backward(LogpBackArgs a) {
    for (int64_t tile = blockIdx.x; tile < a.rows * a.tiles; tile += gridDim.x) {
        const int64_t row = tile / a.tiles, c0 = tile % a.tiles * kBackTile;
        const T* x = static_cast<const T*>(a.logits) + row * a.stride;
        T* out = static_cast<T*>(a.dlogits) + row * a.dstride;
        const float lse = a.lse[row];
        const int64_t at = a.targets[row];
        const bool scored = at >= 0 && at < a.vocab;
        BackTerms r;
        r.target = scored ? at : -1;
        r.dlogp = scored ? a.dlogp[row] : 0.0f;
        r.dent = a.dentropy ? a.dentropy[row] : 0.0f;
        r.both = a.dentropy ? fmaf(r.dent, a.entropy[row], r.dlogp) : r.dlogp;
        const bool far = fabsf(lse) > kFarLse;
        const int64_t end = far ? 0 : a.vocab;      // far rows come below
        constexpr int kVecs = kBackTile / (256 * kVec<T>);
        u32x4 raw[kVecs];
#pragma unroll
        for (int j = 0; j < kVecs; ++j)
            raw[j] = load_row<ONCE>(x, c0 + kVec<T> * (threadIdx.x + 256 * j), a.vocab);
#pragma unroll
        for (int j = 0; j < kVecs; ++j) {
            const int64_t c = c0 + kVec<T> * (threadIdx.x + 256 * j), n = end - c;
            float v[kVec<T>];
            unpack<T>(settle<T>(raw[j], c, a.vocab), v);
            if (n <= 0) continue;
            const int64_t hit = r.target - c;
#pragma unroll
            for (int i = 0; i < kVec<T>; ++i)
                v[i] = logit_gradient(fmaf(v[i], a.scale, -lse), r, i == hit) * a.scale;
            write_vec(out + c, n, v);
        }
        if (far && c0 == 0) far_row<T>(a, x, out, r);
    }
}

template <typename T, int BLOCK, bool ONCE>
void logp_block(const LogpArgs& a, hipStream_t s) {
    const dim3 grid((unsigned)(a.rows < (1 << 21) ? a.rows : (1 << 21))), block(BLOCK);
    KernelTimer kt("k_token_logprobs", s);
    if (a.top > 0) {
        const int64_t keys = 64 * super_len(a.vocab) * 4, cand = (int64_t)a.top * kGroup * 8;
        const int lds = (int)(keys > cand ? keys : cand);
        k_token_logprobs<T, BLOCK, true, ONCE><<<grid, block, lds, s>>>(a);
    } else {
        k_token_logprobs<T, BLOCK, false, ONCE><<<grid, block, 0, s>>>(a);
    }
}

template <typename T>
bool once(int64_t rows, int64_t vocab) {
    return (double)rows * (double)vocab * sizeof(T) >= (double)kOnceBytes;
}

// Threads for the rows at hand, as many as still leave each row a place on the 256 units (the order
// is the same): 256 x 131072 bf16 with 5 alternatives 17 us with 1024, 28 with 256; 512 rows 30
// with 512, 38 with 256; 700 rows 45 with 512, 41 with 256.
template <typename T>
void logp_typed(const LogpArgs& a, hipStream_t s) {
    const bool wide = a.vocab > kTile<T>, past = once<T>(a.rows, a.vocab);
    if (wide && a.rows <= 256)
        logp_block<T, 1024, false>(a, s);
    else if (wide && a.rows <= 512)
        past ? logp_block<T, 512, true>(a, s) : logp_block<T, 512, false>(a, s);
    else
        past ? logp_block<T, 256, true>(a, s) : logp_block<T, 256, false>(a, s);
}

template <typename T>
void logp_back_typed(const LogpBackArgs& a, hipStream_t s) {
    const int64_t wgs = a.rows * a.tiles;
    const dim3 grid((unsigned)(wgs < (1 << 22) ? wgs : (1 << 22))), block(256);
    KernelTimer kt("k_token_logprobs_backward", s);
    if (once<T>(a.rows, a.vocab))
        k_token_logprobs_backward<T, true><<<grid, block, 0, s>>>(a);
    else
        k_token_logprobs_backward<T, false><<<grid, block, 0, s>>>(a);
}

}  // namespace

det_status logprob_launch(const LogpCall& c, hipStream_t s) {
    const LogpArgs a{c.logits, c.targets, c.logp, c.entropy, c.lse, c.top_logp, c.top_ids,
                     c.stride, c.rows, c.vocab, c.top, c.scale,
                     (float)(c.scale * 1.4426950408889634)};
    switch (c.dtype) {
        case DET_F32: logp_typed<float>(a, s); break;
        case DET_F16: logp_typed<_Float16>(a, s); break;
        default: logp_typed<__bf16>(a, s); break;
    }
    return launch_status();
}

det_status logprob_backward_launch(const LogpBackCall& c, hipStream_t s) {
    const LogpBackArgs a{c.logits, c.targets, c.lse, c.dlogp, c.entropy, c.dentropy, c.dlogits,
                         c.stride, c.dstride, c.rows, c.vocab,
                         (c.vocab + kBackTile - 1) / kBackTile, c.scale};
    switch (c.dtype) {
        case DET_F32: logp_back_typed<float>(a, s); break;
        case DET_F16: logp_back_typed<_Float16>(a, s); break;
        default: logp_back_typed<__bf16>(a, s); break;
    }
    return launch_status();
}

}  // namespace det
