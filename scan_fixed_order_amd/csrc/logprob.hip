// logprob.hip -- log probabilities of given tokens with the entropy and the best alternatives,
// and the logits' gradient.
//
// Mathematics, per row of logits x, z = scale * x, everything after the load in f32:
//   lse = log(sum exp z);  logp = z[target] - lse (0 where the target is not a token);
//   entropy = -sum p log p, p = exp(z - lse);  top: the largest logits, ties to the lower index;
//   dlogits = scale * (dlogp (hit - p) - dentropy * p * (log p + entropy)).
// One pass forward: s = sum exp(z - ref) and w = sum exp(z - ref) (z - ref) against a running
// reference give lse = ref + log s and entropy = log s - w / s.  A term whose p is 0 adds 0 to
// the entropy also where its logit is -inf.  A row without any mass (all logits -inf) has
// lse = -inf, entropy 0, logp -inf and gradient 0.
//
// Order: 1024 lanes share a row, lane L holding elements 8 L + 8192 j .. + 8 for j = 0, 1, ...;
// each adds its own in that order, then 64 neighbouring lanes join by the adjacent-lanes tree,
// then the 16 groups in ascending order.  How many threads play those lanes does not enter the
// order, nor do the other rows: a row's bits depend on its logits and the scale alone.
#include <float.h>

#include "det_internal.h"
#include "lm_device.h"

namespace det {
namespace {

constexpr int kLanes = 1024;              // lanes that share a row, in the order above
constexpr int kTile = kLanes * kVec;      // elements they take at a time
constexpr int kGroup = 32;                // neighbouring elements whose largest is kept for top
// A lane's reference is one of its own values, replaced when a value exceeds it by more than
// this: sums against it stay far from overflow, terms are off by at most the rounding of a
// difference of that size, and a lane rarely rescales.
constexpr float kSlack = 8.0f;
constexpr float kFar = -1e30f;            // differences of references stop here (never -inf)

// the largest of three; a quiet NaN loses
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
    float scale;
};

// One lane's running sums against its reference
struct Part {
    float ref, s, w;
};

__device__ __forceinline__ void rebase(Part& p, float ref) {
    const float dm = fmaxf(p.ref - ref, kFar);
    const float f = exp_fast(dm);
    p.w = fmaf(p.s, dm, p.w) * f;
    p.s = p.s * f;
    p.ref = ref;
}

// adds 8 logits; `largest`: their maximum (NaN ignored)
__device__ __forceinline__ void take(Part& p, const float (&x)[kVec], float largest, float scale) {
    const float top = largest * scale;
    if (top > p.ref + kSlack) rebase(p, top);
    float e[kVec], d[kVec];
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
        d[i] = fmaf(x[i], scale, -p.ref);
        e[i] = exp_fast(d[i]);
    }
    float w0 = e[0] * d[0], w1 = e[1] * d[1];
#pragma unroll
    for (int i = 2; i < kVec; i += 2) {
        w0 = fmaf(e[i], d[i], w0);
        w1 = fmaf(e[i + 1], d[i + 1], w1);
    }
    float w = w0 + w1;
    if (w != w) {      // 0 * -inf among them: such a term counts as 0
        w = 0.0f;
#pragma unroll
        for (int i = 0; i < kVec; ++i) w += e[i] == 0.0f ? 0.0f : e[i] * d[i];
    }
    p.s += ((e[0] + e[1]) + (e[2] + e[3])) + ((e[4] + e[5]) + (e[6] + e[7]));
    p.w += w;
}

__device__ __forceinline__ float max8(const float (&x)[kVec]) {
    return max3(max3(x[0], x[1], x[2]), max3(x[3], x[4], x[5]), max3(x[6], x[7], -INFINITY));
}

// orders LDS accesses of one wave's lanes among each other
__device__ __forceinline__ void wave_sync() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// groups of a super-group: 64 of them cover the row; odd, so that lanes that read one group of
// each fall on different LDS banks
__host__ __device__ constexpr int64_t super_len(int64_t vocab) {
    return ((vocab + kGroup - 1) / kGroup + 63) / 64 | 1;
}

// The `top` largest logits of a row.  On entry s_key holds the order key of every group's
// largest logit (0 behind the last group).  The top logits lie in the top groups (each of these
// holds one that beats every logit of the others), so one wave picks the groups through a
// tournament of 64 super-groups, and the workgroup ranks the picked groups' logits that reach
// the last picked group's largest.
template <typename T, int BLOCK>
__device__ void pick_top(const LogpArgs& a, int64_t row, const T* x, uint32_t* s_key,
                         uint32_t* s_super, uint32_t* s_pick, int* s_count, uint32_t* s_least,
                         float ref, float log_s) {
    const int groups = (int)((a.vocab + kGroup - 1) / kGroup);
    const int len = (int)super_len(a.vocab);
    const int lane = threadIdx.x & 63;
    constexpr int kParts = BLOCK / 64;
    {
        const int sg = threadIdx.x / kParts, part = threadIdx.x % kParts;
        uint32_t m = 0;
        for (int i = part; i < len; i += kParts) m = umax(m, s_key[sg * len + i]);
        m = umax(m, xor_partner<1>(m));
        m = umax(m, xor_partner<2>(m));
        if constexpr (kParts == 16) {
            m = umax(m, xor_partner<4>(m));
            m = umax(m, xor_partner<8>(m));
        }
        if (part == 0) s_super[sg] = m;
        if (threadIdx.x == 0) *s_count = 0;
    }
    __syncthreads();
    const int picks = a.top < groups ? a.top : groups;
    if (threadIdx.x < 64) {
        uint32_t mine = s_super[lane], best = 0;
        for (int r = 0; r < picks; ++r) {
            best = wave_max(mine);
            const int sg = __ffsll((unsigned long long)__ballot(mine == best)) - 1;
            // the first group of that super-group with this key, and the largest of the others
            uint32_t rest = 0;
            int at = -1;
            for (int i = 0; i < len; i += 64) {
                uint32_t k = i + lane < len ? s_key[sg * len + i + lane] : 0;
                const unsigned long long hits = __ballot(k == best);
                if (at < 0 && hits) {
                    const int l = __ffsll(hits) - 1;
                    at = i + l;
                    if (lane == l) k = 0;
                }
                rest = umax(rest, k);
            }
            rest = wave_max(rest);
            if (lane == sg) mine = rest;
            if (lane == 0) {
                s_pick[r] = sg * len + at;
                s_key[sg * len + at] = 0;
            }
            wave_sync();
        }
        // with fewer groups than places every logit is a candidate
        if (lane == 0) *s_least = picks < a.top ? 1u : best;
    }
    __syncthreads();
    unsigned long long* s_cand = reinterpret_cast<unsigned long long*>(s_key);
    const uint32_t least = *s_least;
    for (int i = threadIdx.x; i < picks * kGroup; i += BLOCK) {
        const int64_t id = (int64_t)s_pick[i / kGroup] * kGroup + i % kGroup;
        if (id >= a.vocab) continue;
        const uint32_t k = order_key((float)x[id]);
        if (k < least) continue;
        s_cand[atomicAdd(s_count, 1)] = (unsigned long long)k << 32 | (uint32_t)~(uint32_t)id;
    }
    __syncthreads();
    // the candidates' places differ from run to run, their ranks do not
    const int n = *s_count;
    for (int i = threadIdx.x; i < n; i += BLOCK) {
        const unsigned long long c = s_cand[i];
        int rank = 0;
        for (int j = 0; j < n; ++j) rank += s_cand[j] > c;
        if (rank < a.top) {
            const float z = fmaf(key_value((uint32_t)(c >> 32)), a.scale, -ref);
            a.top_ids[row * a.top + rank] = (int64_t)(uint32_t)~(uint32_t)c;
            a.top_logp[row * a.top + rank] = z - log_s;
        }
    }
    __syncthreads();      // s_key is written again
}

// One row per workgroup, each logit read once.
template <typename T, int BLOCK, bool TOP>
__global__ __launch_bounds__(BLOCK) void k_token_logprobs(LogpArgs a) {
    constexpr int kSets = kLanes / BLOCK;       // lanes a thread plays
    constexpr int kSteps = 4 / kSets;           // tiles whose loads are in flight together
    extern __shared__ __align__(16) uint32_t s_key[];
    __shared__ float s_max[BLOCK / 64], s_s[kLanes / 64], s_w[kLanes / 64];
    __shared__ uint32_t s_super[64], s_pick[DET_LOGPROB_MAX_TOP], s_least;
    __shared__ int s_count;
    const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
    const int64_t key_slots = TOP ? 64 * super_len(a.vocab) : 0;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const T* x = static_cast<const T*>(a.logits) + row * a.stride;
        Part p[kSets];
#pragma unroll
        for (int u = 0; u < kSets; ++u) p[u] = Part{-FLT_MAX, 0.0f, 0.0f};
        if constexpr (TOP) {
            // slots behind the last whole tile's groups
            for (int64_t i = a.vocab / kTile * (kTile / kGroup) + t; i < key_slots; i += BLOCK)
                s_key[i] = 0;
            __syncthreads();
        }
        const auto one = [&](int64_t c, int u, const float(&v)[kVec], bool keep) {
            const float largest = max8(v);
            if constexpr (TOP) {
                float g = largest;
                g = fmaxf(g, xor_partner<1>(g));
                g = fmaxf(g, xor_partner<2>(g));
                if (keep && (lane & 3) == 0) s_key[c / kGroup] = order_key(g);
            }
            if (keep) take(p[u], v, largest, a.scale);
        };
        const int64_t whole = a.vocab / (kTile * kSteps);
        for (int64_t i = 0; i < whole; ++i) {
            Raw8<T> raw[kSteps][kSets];
#pragma unroll
            for (int q = 0; q < kSteps; ++q)
#pragma unroll
                for (int u = 0; u < kSets; ++u)
                    raw[q][u] = load8(x + (i * kSteps + q) * kTile + kVec * (t + u * BLOCK));
#pragma unroll
            for (int q = 0; q < kSteps; ++q)
#pragma unroll
                for (int u = 0; u < kSets; ++u) {
                    float v[kVec];
                    unpack8<T>(raw[q][u], v);
                    one((i * kSteps + q) * kTile + kVec * (t + u * BLOCK), u, v, true);
                }
        }
        for (int64_t base = whole * kSteps * kTile; base < a.vocab; base += kTile) {
#pragma unroll
            for (int u = 0; u < kSets; ++u) {
                const int64_t c = base + kVec * (t + u * BLOCK);
                float v[kVec];
                read8(x + c, a.vocab - c, -INFINITY, v);
                one(c, u, v, c < a.vocab);
            }
        }
        // the row's reference, then every lane's sums against it
        float ref = p[0].ref;
#pragma unroll
        for (int u = 1; u < kSets; ++u) ref = fmaxf(ref, p[u].ref);
        ref = wave_max(ref);
        if (lane == 0) s_max[wave] = ref;
        __syncthreads();
        ref = s_max[0];
#pragma unroll
        for (int w = 1; w < BLOCK / 64; ++w) ref = fmaxf(ref, s_max[w]);
#pragma unroll
        for (int u = 0; u < kSets; ++u) {
            rebase(p[u], ref);
            const float s = wave_pw(p[u].s), w = wave_pw(p[u].w);
            if (lane == 0) {
                s_s[wave + u * (BLOCK / 64)] = s;
                s_w[wave + u * (BLOCK / 64)] = w;
            }
        }
        __syncthreads();
        float s = s_s[0], w = s_w[0];
#pragma unroll
        for (int i = 1; i < kLanes / 64; ++i) {
            s += s_s[i];
            w += s_w[i];
        }
        const float log_s = logf(s);
        if (t == 0) {
            const int64_t at = a.targets[row];
            const bool none = s == 0.0f;
            a.lse[row] = ref + log_s;
            a.entropy[row] = none ? 0.0f : log_s - w / s;
            float lp = 0.0f;
            if (at >= 0 && at < a.vocab)
                lp = none ? -INFINITY : fmaf((float)x[at], a.scale, -ref) - log_s;
            a.logp[row] = lp;
        }
        if constexpr (TOP)
            pick_top<T, BLOCK>(a, row, x, s_key, s_super, s_pick, &s_count, &s_least,
                               s == 0.0f ? 0.0f : ref, s == 0.0f ? 0.0f : log_s);
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

constexpr int kBackVecs = 4;                              // vectors a thread
constexpr int kBackTile = 256 * kVec * kBackVecs;

// Each logit read once, each gradient written once; nothing is summed.
template <typename T>
__global__ __launch_bounds__(256) void k_token_logprobs_backward(LogpBackArgs a) {
    for (int64_t tile = blockIdx.x; tile < a.rows * a.tiles; tile += gridDim.x) {
        const int64_t row = tile / a.tiles, c0 = tile % a.tiles * kBackTile;
        const T* x = static_cast<const T*>(a.logits) + row * a.stride;
        T* out = static_cast<T*>(a.dlogits) + row * a.dstride;
        const float lse = a.lse[row];
        const int64_t at = a.targets[row];
        const bool scored = at >= 0 && at < a.vocab;
        const float dlogp = scored ? a.dlogp[row] : 0.0f;
        const float dent = a.dentropy ? a.dentropy[row] : 0.0f;
        const float both = a.dentropy ? fmaf(dent, a.entropy[row], dlogp) : dlogp;
        const bool none = lse == -INFINITY;
#pragma unroll
        for (int j = 0; j < kBackVecs; ++j) {
            const int64_t c = c0 + kVec * (threadIdx.x + 256 * j), n = a.vocab - c;
            if (n <= 0) continue;
            float v[kVec];
            read8(x + c, n, 0.0f, v);
            const int64_t hit = scored ? at - c : -1;
#pragma unroll
            for (int i = 0; i < kVec; ++i) {
                const float log = fmaf(v[i], a.scale, -lse);
                const float p = exp_fast(log);
                // below -1000 p is 0 and -inf must not meet it
                float d = -p * fmaf(dent, fmaxf(log, -1000.0f), both);
                if (i == hit) d += dlogp;
                v[i] = none ? 0.0f : d * a.scale;
            }
            write8(out + c, n, v);
        }
    }
}

template <typename T, int BLOCK>
void logp_block(const LogpArgs& a, hipStream_t s) {
    const dim3 grid((unsigned)(a.rows < (1 << 21) ? a.rows : (1 << 21))), block(BLOCK);
    KernelTimer kt("k_token_logprobs", s);
    if (a.top > 0) {
        const int64_t keys = 64 * super_len(a.vocab) * 4, cand = (int64_t)a.top * kGroup * 8;
        const int lds = (int)(keys > cand ? keys : cand);
        k_token_logprobs<T, BLOCK, true><<<grid, block, lds, s>>>(a);
    } else {
        k_token_logprobs<T, BLOCK, false><<<grid, block, 0, s>>>(a);
    }
}

template <typename T>
void logp_typed(const LogpArgs& a, hipStream_t s) {
    if (a.rows <= 256 && a.vocab > kTile)
        logp_block<T, 1024>(a, s);
    else
        logp_block<T, 256>(a, s);
}

template <typename T>
void logp_back_typed(const LogpBackArgs& a, hipStream_t s) {
    const int64_t wgs = a.rows * a.tiles;
    KernelTimer kt("k_token_logprobs_backward", s);
    k_token_logprobs_backward<T><<<dim3((unsigned)(wgs < (1 << 22) ? wgs : (1 << 22))), dim3(256),
                                   0, s>>>(a);
}

}  // namespace

det_status logprob_launch(const LogpCall& c, hipStream_t s) {
    const LogpArgs a{c.logits, c.targets, c.logp, c.entropy, c.lse, c.top_logp, c.top_ids,
                     c.stride, c.rows, c.vocab, c.top, c.scale};
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
