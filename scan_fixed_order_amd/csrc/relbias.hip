// relbias.hip -- a learned relative position bias by buckets, added to scores or alone, and its
// table's gradient.
//
// Mathematics, for head h, query position i and key position j, r = j - i:
//   out[h, i, j] = (scores[h, i, j] +) table[bucket(r)][h], -inf where the masks leave nothing;
//   dtable[b][h] = sum of dout[h, i, j] over the unmasked places with bucket(r) = b.
// bucket(r) is a step function of r: a side has n buckets and the host computes the first
// distance of each in whole numbers (relbias_starts), so a distance on a border falls on the
// same side everywhere.  Both directions use that a value depends on j - i alone: a row of the
// output is the row above it moved by one place, and the gradient's sums run along diagonals.
#include <math.h>

#include "det_internal.h"
#include "lm_device.h"

namespace det {
namespace {

constexpr int kBlock = 256;

struct Map {
    int starts[kBiasMaxSide];      // first distance of bucket j of a side, ascending
    int side;                      // buckets a side
    bool two_sided, causal;
    int64_t q, k, q_offset;
    const int32_t* q_offsets;      // NULL: q_offset for every sequence
    const int32_t* lengths;        // NULL: no padding
};

__device__ __forceinline__ int bucket_of(const Map& m, const int* starts, int64_t r) {
    int64_t far = r < 0 ? -r : (m.two_sided ? r : 0);
    int lo = m.side - 1;
    if (far < starts[m.side - 1]) {
        // the last bucket whose start is not beyond the distance (starts[0] = 0)
        lo = 0;
        int hi = m.side - 1;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (starts[mid] <= far) lo = mid; else hi = mid;
        }
    }
    return m.two_sided && r > 0 ? lo + m.side : lo;
}

__device__ __forceinline__ int64_t offset_of(const Map& m, int64_t b) {
    return m.q_offsets ? (int64_t)m.q_offsets[b] : m.q_offset;
}

// keys and query positions below this are inside sequence b
__device__ __forceinline__ int64_t length_of(const Map& m, int64_t b) {
    return m.lengths ? (int64_t)m.lengths[b] : INT64_MAX / 4;
}

struct BiasArgs {
    const void* table;      // [buckets][heads]; NULL: the scores alone, masked
    const void* scores;     // NULL: none
    void* out;              // [batch][heads][q][k]
    int64_t sb, sh, sq;     // strides of scores
    int64_t heads, batch;
    int lanes_log2;         // lanes across the keys: 2^lanes_log2 of the workgroup's 256
    int rows;               // query rows a lane walks
    float fill;             // what a masked place gets
    int64_t kt, qt;         // tiles along the keys and the queries
};

// A workgroup covers `width` = 8 * 2^lanes_log2 keys and (256 >> lanes_log2) * rows queries of
// one head.  The values of all its diagonals are laid out once in LDS; a lane then walks down
// its rows, and each next row is the last one moved by one element, with one new element read.
template <typename T, bool SCORES>
__global__ __launch_bounds__(kBlock) void k_relative_bias(Map m, BiasArgs a) {
    extern __shared__ float s_diag[];           // value of diagonal (first + i)
    __shared__ int s_starts[kBiasMaxSide];
    const int lanes = 1 << a.lanes_log2, teams = kBlock >> a.lanes_log2;
    const int width = kVec * lanes, height = teams * a.rows;
    for (int i = threadIdx.x; i < m.side; i += kBlock) s_starts[i] = m.starts[i];
    for (int64_t tile = blockIdx.x; tile < a.batch * a.heads * a.qt * a.kt; tile += gridDim.x) {
        const int64_t kt = tile % a.kt, qt = tile / a.kt % a.qt, bh = tile / (a.kt * a.qt);
        const int64_t b = bh / a.heads, h = bh % a.heads;
        const int64_t k0 = kt * width, q0 = qt * height;
        const int64_t off = offset_of(m, b), len = length_of(m, b);
        const T* table = static_cast<const T*>(a.table);
        __syncthreads();      // s_starts is there; the last tile's diagonals are read
        // diagonal index i holds r = (k0 - (q0 + height - 1)) + i - off
        const int64_t r0 = k0 - (q0 + height - 1) - off;
        for (int i = threadIdx.x; i < width + height - 1; i += kBlock)
            s_diag[i] = table ? (float)table[bucket_of(m, s_starts, r0 + i) * a.heads + h] : 0.0f;
        __syncthreads();
        const int lane = threadIdx.x & (lanes - 1), team = threadIdx.x >> a.lanes_log2;
        const int64_t c = k0 + kVec * lane, row0 = q0 + (int64_t)team * a.rows;
        const int64_t n = m.k - c;                       // keys from c on
        if (n <= 0) continue;
        float v[kVec];
        int at = kVec * lane + (height - 1 - team * a.rows);   // diagonal of (row0, c)
#pragma unroll
        for (int i = 1; i < kVec; ++i) v[i - 1] = s_diag[at + i];   // moved into place by the first row
        const int64_t end = row0 + a.rows < m.q ? row0 + a.rows : m.q;
        for (int64_t row = row0; row < end; ++row, --at) {
#pragma unroll
            for (int i = kVec - 1; i > 0; --i) v[i] = v[i - 1];
            v[0] = s_diag[at];
            // keys that the masks leave this row; a masked place is never read
            int64_t left = row + off < len ? len : 0;
            if (m.causal && row + off + 1 < left) left = row + off + 1;
            left -= c;
            float o[kVec];
            if constexpr (SCORES) {
                const T* sc = static_cast<const T*>(a.scores) + b * a.sb + h * a.sh + row * a.sq + c;
                read8(sc, left < n ? left : n, 0.0f, o);
#pragma unroll
                for (int i = 0; i < kVec; ++i) o[i] += v[i];
            } else {
#pragma unroll
                for (int i = 0; i < kVec; ++i) o[i] = v[i];
            }
            if (left < kVec) {
#pragma unroll
                for (int i = 0; i < kVec; ++i)
                    if (i >= left) o[i] = a.fill;
            }
            write8(static_cast<T*>(a.out) + (bh * m.q + row) * m.k + c, n, o);
        }
    }
}

// ---------------------------------------------------------------- the table's gradient

struct BiasBackArgs {
    const void* dout;
    float* part;              // [batch * heads][row strips][diagonal tiles][buckets]
    int64_t sb, sh, sq, heads, batch;
    int strip;                // query rows a workgroup walks
    int64_t qt, dt;           // row strips and diagonal tiles
    int buckets;
};

constexpr int kWaves = kBlock / 64;
constexpr int kDiags = 64 * kVec;          // diagonals a wave covers

// A lane owns 8 neighbouring diagonals and walks down the strip's rows: its 8 elements of a row
// lie together in memory, one place further along with every row.  The wave then adds its
// diagonals up by buckets, which are runs of neighbouring diagonals.
template <typename T>
__global__ __launch_bounds__(kBlock) void k_relative_bias_backward(Map m, BiasBackArgs a) {
    __shared__ float s_sums[kWaves][kDiags];
    __shared__ int s_starts[kBiasMaxSide];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    for (int i = threadIdx.x; i < m.side; i += kBlock) s_starts[i] = m.starts[i];
    const int64_t tiles = a.batch * a.heads * a.qt * a.dt;
    float* s_sum = s_sums[wave];
    for (int64_t first = (int64_t)blockIdx.x * kWaves; first < tiles;
         first += (int64_t)gridDim.x * kWaves) {
        const bool live = first + wave < tiles;
        const int64_t tile = live ? first + wave : tiles - 1;
        const int64_t dt = tile % a.dt, qt = tile / a.dt % a.qt, bh = tile / (a.dt * a.qt);
        const int64_t b = bh / a.heads, h = bh % a.heads;
        const int64_t off = offset_of(m, b), len = length_of(m, b);
        const int64_t q0 = qt * a.strip;
        int64_t q1 = q0 + a.strip < m.q ? q0 + a.strip : m.q;
        if (q1 > len - off) q1 = len - off;               // rows past the sequence hold nothing
        const int64_t keys = len < m.k ? len : m.k;       // keys past it neither
        // diagonal d of the strip, from 0: key = row + d - shift
        const int64_t shift = q0 + a.strip - 1;
        const int64_t d0 = dt * kDiags + kVec * lane - shift;    // key = row + d0 + i
        float acc[kVec] = {};
        const T* p = static_cast<const T*>(a.dout) + b * a.sb + h * a.sh + q0 * a.sq + q0 + d0;
        // a diagonal after the query is masked as a whole when causal
        const bool some = !m.causal || d0 - off <= 0;
        if (__all(some && q0 + d0 >= 0 && q1 + d0 + kVec - 1 <= keys)) {
#pragma unroll 8
            for (int64_t row = q0; row < q1; ++row, p += a.sq + 1) {
                float v[kVec];
                unpack8<T>(load8(p), v);
#pragma unroll
                for (int i = 0; i < kVec; ++i) acc[i] += v[i];
            }
        } else if (some) {
#pragma unroll 4
            for (int64_t row = q0; row < q1; ++row, p += a.sq + 1) {
                const int64_t c = row + d0;
                if (c >= 0 && c + kVec <= keys) {
                    float v[kVec];
                    unpack8<T>(load8(p), v);
#pragma unroll
                    for (int i = 0; i < kVec; ++i) acc[i] += v[i];
                } else if (c > -kVec && c < keys) {
#pragma unroll
                    for (int i = 0; i < kVec; ++i)
                        if (c + i >= 0 && c + i < keys) acc[i] += (float)p[i];
                }
            }
        }
        __syncthreads();      // s_starts is there; the last tile's sums are read
#pragma unroll
        for (int i = 0; i < kVec; ++i)
            s_sum[kVec * lane + i] = m.causal && d0 + i - off > 0 ? 0.0f : acc[i];
        __syncthreads();
        if (!live) continue;
        const int64_t r0 = dt * kDiags - shift - off;     // r of the tile's diagonal 0
        for (int bk = 0; bk < a.buckets; ++bk) {
            // diagonals r in [lo, hi) of this bucket
            int64_t lo = 0, hi = 0;
            if (bk < m.side) {
                lo = bk + 1 < m.side ? 1 - (int64_t)s_starts[bk + 1] : INT64_MIN / 2;
                hi = bk == 0 && !m.two_sided ? INT64_MAX / 2 : 1 - (int64_t)s_starts[bk];
            } else if (m.two_sided && bk < 2 * m.side) {
                const int j = bk - m.side;
                lo = s_starts[j] > 0 ? s_starts[j] : 1;
                hi = j + 1 < m.side ? s_starts[j + 1] : INT64_MAX / 2;
            }
            lo -= r0;
            hi -= r0;
            const int from = (int)(lo < 0 ? 0 : lo > kDiags ? kDiags : lo);
            const int to = (int)(hi < 0 ? 0 : hi > kDiags ? kDiags : hi);
            float v = 0.0f;
            for (int i = from + lane; i < to; i += 64) v += s_sum[i];
            if (from < to) v = wave_pw(v);
            if (lane == 0) a.part[tile * a.buckets + bk] = v;
        }
    }
}

// dtable[bk][h] = the tiles' sums of every sequence, added in 64 bits: thread t adds items t,
// t + 256, ... in that order, then the threads join by a halving tree.
template <typename T>
__global__ __launch_bounds__(kBlock) void k_bias_table_sums(const float* part, int64_t batch,
                                                            int64_t heads, int64_t per_head,
                                                            int buckets, T* out) {
    __shared__ double s[kBlock];
    const int bk = blockIdx.x % buckets;
    const int64_t h = blockIdx.x / buckets;
    double v = 0.0;
    for (int64_t i = threadIdx.x; i < batch * per_head; i += kBlock) {
        const int64_t b = i / per_head, t = i % per_head;
        v += (double)part[((b * heads + h) * per_head + t) * buckets + bk];
    }
    s[threadIdx.x] = v;
    __syncthreads();
    for (int n = kBlock / 2; n > 0; n >>= 1) {
        if ((int)threadIdx.x < n) s[threadIdx.x] += s[threadIdx.x + n];
        __syncthreads();
    }
    if (threadIdx.x == 0) out[bk * heads + h] = (T)s[0];
}

// ---------------------------------------------------------------- the buckets' borders

// A natural number as 32-bit limbs, lowest first; room for the products of 2 * kBiasMaxSide
// 32-bit factors.
struct Big {
    uint32_t limb[2 * kBiasMaxSide];
    int n;
};

void times(Big& v, uint32_t by, int power) {
    for (; power > 0; --power) {
        uint64_t carry = 0;
        for (int i = 0; i < v.n; ++i) {
            carry += (uint64_t)v.limb[i] * by;
            v.limb[i] = (uint32_t)carry;
            carry >>= 32;
        }
        if (carry) v.limb[v.n++] = (uint32_t)carry;
    }
}

// (a / near)^power >= (distance / near)^j, in whole numbers
bool reaches(uint32_t a, uint32_t near, uint32_t distance, int power, int j) {
    Big l{{1}, 1}, r{{1}, 1};
    times(l, a, power);
    times(l, near, j);
    times(r, distance, j);
    times(r, near, power);
    if (l.n != r.n) return l.n > r.n;
    for (int i = l.n; i-- > 0;)
        if (l.limb[i] != r.limb[i]) return l.limb[i] > r.limb[i];
    return true;
}

}  // namespace

// A side of n buckets: the first `near` = n / 2 hold one distance each; bucket near + j starts at
// the least a with log(a / near) / log(distance / near) * (n - near) >= j.
void relbias_starts(int n, int64_t distance, int* starts) {
    const int near = n / 2, power = n - near;
    for (int i = 0; i < near; ++i) starts[i] = i;
    int64_t prev = near;
    for (int j = 0; j < power; ++j) {
        const double est = near * pow((double)distance / near, (double)j / power);
        const double whole = nearbyint(est);
        int64_t a = (int64_t)ceil(est);
        // the estimate is good to far better than 1e-9; next to a whole number ask that number
        if (fabs(est - whole) <= 1e-9 * est)
            a = (int64_t)whole + (reaches((uint32_t)whole, (uint32_t)near, (uint32_t)distance,
                                          power, j) ? 0 : 1);
        if (a < prev) a = prev;
        starts[near + j] = (int)a;
        prev = a;
    }
}

namespace {

Map map_of(const BiasCall& c) {
    Map m;
    m.side = c.bidirectional ? c.buckets / 2 : c.buckets;
    relbias_starts(m.side, c.max_distance, m.starts);
    for (int i = m.side; i < kBiasMaxSide; ++i) m.starts[i] = 0;
    m.two_sided = c.bidirectional;
    m.causal = c.causal;
    m.q = c.q;
    m.k = c.k;
    m.q_offset = c.q_offset;
    m.q_offsets = c.q_offsets;
    m.lengths = c.lengths;
    return m;
}

unsigned grid_of(int64_t tiles) { return (unsigned)(tiles < (1 << 22) ? tiles : (1 << 22)); }

template <typename T>
void bias_typed(const BiasCall& c, hipStream_t s) {
    const Map m = map_of(c);
    BiasArgs a{c.table, c.scores, c.out, c.sb, c.sh, c.sq, c.heads, c.batch, 8, 1, c.fill, 0, 0};
    // as many lanes across the keys as the row has vectors (at most the workgroup), the rest of
    // the workgroup on further rows
    while (a.lanes_log2 > 3 && ((int64_t)kVec << (a.lanes_log2 - 1)) >= c.k) --a.lanes_log2;
    const int teams = kBlock >> a.lanes_log2;
    while (a.rows < 64 && (int64_t)a.rows * teams < c.q) a.rows *= 2;
    const int64_t width = (int64_t)kVec << a.lanes_log2, height = (int64_t)teams * a.rows;
    a.kt = (c.k + width - 1) / width;
    a.qt = (c.q + height - 1) / height;
    const int lds = (int)(width + height) * (int)sizeof(float);
    const dim3 grid(grid_of(a.batch * a.heads * a.kt * a.qt));
    KernelTimer kt("k_relative_bias", s);
    if (c.scores)
        k_relative_bias<T, true><<<grid, dim3(kBlock), lds, s>>>(m, a);
    else
        k_relative_bias<T, false><<<grid, dim3(kBlock), lds, s>>>(m, a);
}

struct BackShape {
    int strip;
    int64_t qt, dt;
};

// Rows a strip and the diagonals' tiles, from (q, k) alone: the order of the sums.
BackShape back_shape(int64_t q, int64_t k) {
    BackShape r;
    r.strip = q < 128 ? (int)(q > 0 ? q : 1) : 128;
    r.qt = (q + r.strip - 1) / r.strip;
    r.dt = (k + r.strip - 1 + kDiags - 1) / kDiags;
    return r;
}

template <typename T>
det_status back_typed(const BiasCall& c, const void* dout, void* dtable, void* ws, hipStream_t s) {
    const Map m = map_of(c);
    const BackShape sh = back_shape(c.q, c.k);
    BiasBackArgs a{dout, static_cast<float*>(ws), c.sb, c.sh, c.sq, c.heads, c.batch, sh.strip,
                   sh.qt, sh.dt, c.buckets};
    const int64_t tiles = c.q > 0 && c.k > 0 ? c.batch * c.heads * sh.qt * sh.dt : 0;
    if (tiles > 0) {
        KernelTimer kt("k_relative_bias_backward", s);
        k_relative_bias_backward<T><<<dim3(grid_of((tiles + kWaves - 1) / kWaves)), dim3(kBlock), 0, s>>>(m, a);
        const det_status st = launch_status();
        if (st != DET_SUCCESS) return st;
    }
    KernelTimer kt("k_bias_table_sums", s);
    k_bias_table_sums<T><<<dim3((unsigned)(c.heads * c.buckets)), dim3(kBlock), 0, s>>>(
        a.part, tiles > 0 ? c.batch : 0, c.heads, sh.qt * sh.dt, c.buckets,
        static_cast<T*>(dtable));
    return launch_status();
}

}  // namespace

size_t bias_backward_workspace(int64_t batch, int64_t heads, int64_t q, int64_t k, int buckets) {
    const BackShape s = back_shape(q, k);
    return round_up((size_t)batch * heads * s.qt * s.dt * buckets * sizeof(float), 256) + 256;
}

det_status bias_launch(const BiasCall& c, hipStream_t s) {
    switch (c.dtype) {
        case DET_F32: bias_typed<float>(c, s); break;
        case DET_F16: bias_typed<_Float16>(c, s); break;
        default: bias_typed<__bf16>(c, s); break;
    }
    return launch_status();
}

det_status bias_backward_launch(const BiasCall& c, const void* dout, void* dtable, void* ws,
                                hipStream_t s) {
    switch (c.dtype) {
        case DET_F32: return back_typed<float>(c, dout, dtable, ws, s);
        case DET_F16: return back_typed<_Float16>(c, dout, dtable, ws, s);
        default: return back_typed<__bf16>(c, dout, dtable, ws, s);
    }
}

}  // namespace det
