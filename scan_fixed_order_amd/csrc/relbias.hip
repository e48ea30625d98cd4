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
    int side, top;                 // buckets a side, the largest power of two below that
    bool two_sided, causal;
    int64_t q, k, q_offset;
    const int32_t* q_offsets;      // NULL: q_offset for every sequence
    const int32_t* lengths;        // NULL: no padding
};

// Bucket of a relative position: the last of the side's whose start is not beyond the distance
// (starts[0] = 0).  top: the largest power of two below the number of buckets a side.
__device__ __forceinline__ int bucket_of(const Map& m, const int* starts, int top, int64_t r) {
    const int64_t far = r < 0 ? -r : (m.two_sided ? r : 0);
    int lo = m.side - 1;
    if (far < starts[lo]) {
        lo = 0;
        for (int step = top; step > 0; step >>= 1) {
            const int next = lo + step, at = next < m.side ? next : m.side - 1;
            lo = starts[at] <= far ? at : lo;
        }
    }
    return m.two_sided && r > 0 ? lo + m.side : lo;
}

// Buckets of N neighbouring relative positions from r on, their searches side by side.
template <int N>
__device__ __forceinline__ void buckets_of(const Map& m, const int* starts, int64_t r,
                                           int (&bucket)[N]) {
    const int border = starts[m.side - 1];
    int far[N];
    bool near = false;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int64_t a = r + i < 0 ? -(r + i) : (m.two_sided ? r + i : 0);
        far[i] = a < border ? (int)a : border;
        near |= far[i] < border;
        bucket[i] = m.side - 1;
    }
    if (near) {
#pragma unroll
        for (int i = 0; i < N; ++i) bucket[i] = 0;
        for (int step = m.top; step > 0; step >>= 1) {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                // read in any case: a branch around the load would make the searches take turns
                const int next = bucket[i] + step, at = next < m.side ? next : m.side - 1;
                bucket[i] = starts[at] <= far[i] ? at : bucket[i];
            }
        }
    }
#pragma unroll
    for (int i = 0; i < N; ++i)
        if (m.two_sided && r + i > 0) bucket[i] += m.side;
}

// a / b, in 32 bits where both fit
__device__ __forceinline__ int64_t split(int64_t a, int64_t b) {
    return ((a | b) >> 32) == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
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
    int64_t extent;         // elements from scores' first to behind its last
    int64_t heads, batch;
    int lanes_log2;         // lanes across the keys: 2^lanes_log2 of the workgroup's 256
    int rows;               // query rows a lane walks, a multiple of kRows
    int buckets;
    float fill;             // what a masked place gets
    int64_t qt;             // tiles along the queries
};

constexpr int kRows = 8;

// A vector from place `at` of a tensor whose elements lie in [0, extent), of which the first n
// count; the others are unspecified.  Those may lie past the row's end but never outside the
// tensor, whose two ends alone are read one by one.
template <typename T>
__device__ __forceinline__ u32x4 load_inside(const T* p, int64_t at, int64_t n, int64_t extent) {
    u32x4 r = {};
    if (n > 0) {
        if (at + kVec<T> <= extent) {
            r = load_vec(p + at);
        } else {
            float v[kVec<T>];
            load_tail(p + at, n, 0.0f, v);
            r = pack<T>(v);
        }
    }
    return r;
}

// A workgroup covers `width` = 2^lanes_log2 vectors of keys and (256 >> lanes_log2) * rows queries of
// one head.  The values of all its diagonals are laid out once in LDS; a lane then walks down
// its rows, and each next row is the last one moved by one element, with one new element read.
// Bound by HBM's writes: 16 x 4096 x 4096 bf16 alone 97 us (5.5 TB/s; any height, width or order of
// the tiles measured gives 96 to 100, without the bucket search too), added to 4 x 16 x 512 x 1024
// scores under a causal mask 21 us (4.9 TB/s).
template <typename T, bool SCORES>
__global__ __launch_bounds__(kBlock) void k_relative_bias(Map m, BiasArgs a) {
    extern __shared__ float s_diag[];           // value of diagonal (first + i)
    __shared__ int s_starts[kBiasMaxSide];
    __shared__ float s_table[DET_BIAS_MAX_BUCKETS];
    constexpr int kStep = SCORES ? kRows / 2 : kRows;
    const int lanes = 1 << a.lanes_log2, teams = kBlock >> a.lanes_log2;
    const int width = kVec<T> * lanes, height = teams * a.rows;
    for (int i = threadIdx.x; i < m.side; i += kBlock) s_starts[i] = m.starts[i];
    const int64_t kt = blockIdx.x;
    for (int64_t bh = blockIdx.z; bh < a.batch * a.heads; bh += gridDim.z)
    for (int64_t qt = blockIdx.y; qt < a.qt; qt += gridDim.y) {
        const int64_t b = split(bh, a.heads), h = bh - b * a.heads;
        const int64_t k0 = kt * width, q0 = qt * height;
        const int64_t off = offset_of(m, b), len = length_of(m, b);
        const T* table = static_cast<const T*>(a.table);
        for (int i = threadIdx.x; i < a.buckets; i += kBlock)
            s_table[i] = table ? (float)table[(int64_t)i * a.heads + h] : 0.0f;
        __syncthreads();      // the last tile's diagonals are read
        // diagonal index i holds r = (k0 - (q0 + height - 1)) + i - off
        const int64_t r0 = k0 - (q0 + height - 1) - off;
#pragma unroll 3
        for (int i = threadIdx.x; i < width + height - 1; i += kBlock)
            s_diag[i] = s_table[bucket_of(m, s_starts, m.top, r0 + i)];
        __syncthreads();
        const int lane = threadIdx.x & (lanes - 1), team = threadIdx.x >> a.lanes_log2;
        const int64_t c = k0 + kVec<T> * lane, row0 = q0 + (int64_t)team * a.rows;
        const int64_t n = m.k - c;                       // keys from c on
        if (n <= 0) continue;
        float v[kVec<T>];
        int at = kVec<T> * lane + (height - 1 - team * a.rows);   // diagonal of (row0, c)
#pragma unroll
        for (int i = 1; i < kVec<T>; ++i) v[i - 1] = s_diag[at + i];   // moved into place by the first row
        const int64_t end = row0 + a.rows < m.q ? row0 + a.rows : m.q;
        const int64_t base = SCORES ? b * a.sb + h * a.sh + c : 0;
        const T* scores = static_cast<const T*>(a.scores);
        // kStep rows at a time, their loads in flight together
        for (int64_t row = row0; row < end; row += kStep, at -= kStep) {
            u32x4 raw[kStep];
            int left[kStep];          // of the vector's keys, those that the masks leave
#pragma unroll
            for (int j = 0; j < kStep; ++j) {
                const int64_t pos = row + j + off;
                const int64_t keys = (m.causal && pos + 1 < len ? pos + 1 : len) - c;
                left[j] = pos >= len || row + j >= end || keys < 0 ? 0 : keys < kVec<T> ? (int)keys : kVec<T>;
                if constexpr (SCORES)
                    raw[j] = load_inside(scores, base + (row + j) * a.sq,
                                          left[j] < n ? left[j] : n, a.extent);
            }
#pragma unroll
            for (int j = 0; j < kStep; ++j) {
                if (row + j >= end) break;
#pragma unroll
                for (int i = kVec<T> - 1; i > 0; --i) v[i] = v[i - 1];
                v[0] = s_diag[at - j];
                float o[kVec<T>];
                if constexpr (SCORES) {
                    unpack<T>(raw[j], o);
#pragma unroll
                    for (int i = 0; i < kVec<T>; ++i) o[i] += v[i];
                } else {
#pragma unroll
                    for (int i = 0; i < kVec<T>; ++i) o[i] = v[i];
                }
                if (left[j] < kVec<T>) {
#pragma unroll
                    for (int i = 0; i < kVec<T>; ++i)
                        if (i >= left[j]) o[i] = a.fill;
                }
                write_vec(static_cast<T*>(a.out) + (bh * m.q + row + j) * m.k + c, n, o);
            }
        }
    }
}

// Few queries: nothing to share between rows, so every lane finds its 8 keys' buckets by itself.
// A workgroup's teams of 2^lanes_log2 lanes take neighbouring rows of the output.  A batch of 32
// x 16 rows of 4097 keys 6.5 us a call; 8.3 between events, 14.9 through the diagonals' layout, of
// which a row uses each value once.  Bound by latency: of the 8.3, 5.4 remain without the buckets.
template <typename T, bool SCORES>
__global__ __launch_bounds__(kBlock) void k_relative_bias_row(Map m, BiasArgs a) {
    __shared__ int s_starts[kBiasMaxSide];
    const int lanes = 1 << a.lanes_log2, teams = kBlock >> a.lanes_log2;
    for (int i = threadIdx.x; i < m.side; i += kBlock) s_starts[i] = m.starts[i];
    __syncthreads();
    const int64_t c = (int64_t)blockIdx.x * kVec<T> * lanes + kVec<T> * (threadIdx.x & (lanes - 1));
    const int64_t n = m.k - c;
    if (n <= 0) return;
    const T* table = static_cast<const T*>(a.table);
    for (int64_t r = (int64_t)blockIdx.y * teams + (threadIdx.x >> a.lanes_log2);
         r < a.batch * a.heads * m.q; r += (int64_t)gridDim.y * teams) {
        const int64_t bh = split(r, m.q), row = r - bh * m.q;
        const int64_t b = split(bh, a.heads), h = bh - b * a.heads;
        const int64_t off = offset_of(m, b), len = length_of(m, b);
        const int64_t keys = (m.causal && row + off + 1 < len ? row + off + 1 : len) - c;
        const int left = row + off >= len || keys < 0 ? 0 : keys < kVec<T> ? (int)keys : kVec<T>;
        float o[kVec<T>];
        u32x4 raw;
        if constexpr (SCORES)
            raw = load_inside(static_cast<const T*>(a.scores),
                               b * a.sb + h * a.sh + row * a.sq + c, left < n ? left : n, a.extent);
        const int64_t r0 = c - row - off;
#pragma unroll
        for (int i = 0; i < kVec<T>; ++i) o[i] = a.fill;
        if (left > 0) {
            int bucket[kVec<T>];
            buckets_of(m, s_starts, r0, bucket);
            float v[kVec<T>];
#pragma unroll
            for (int i = 0; i < kVec<T>; ++i)
                v[i] = table ? (float)table[(int64_t)bucket[i] * a.heads + h] : 0.0f;
            if constexpr (SCORES) {
                float sc[kVec<T>];
                unpack<T>(raw, sc);
#pragma unroll
                for (int i = 0; i < kVec<T>; ++i) v[i] += sc[i];
            }
#pragma unroll
            for (int i = 0; i < kVec<T>; ++i)
                if (i < left) o[i] = v[i];
        }
        write_vec(static_cast<T*>(a.out) + r * m.k + c, n, o);
    }
}

// ---------------------------------------------------------------- the table's gradient

struct BiasBackArgs {
    const void* dout;
    double* part;             // [batch * heads][tiles / kWaves][buckets]
    int64_t sb, sh, sq, extent, heads, batch;
    int strip;                // query rows a workgroup walks
    int64_t qt, dt;           // row strips and diagonal tiles
    int buckets;
};

constexpr int kWaves = kBlock / 64;
constexpr int kShortRun = 16;              // diagonals
template <typename T>
constexpr int kDiags = 64 * kVec<T>;       // diagonals a wave covers

// What kRows rows of a diagonal are added in.  A gradient of 16 bits does not show the 7 float
// roundings (2^-24 each, of the summed magnitudes), and sums in double cost it 3 to 20 % (2 x 16 x
// 1024 x 1024 f16 20.5 us, 25.1 in double); one of f32 shows them, and pays 0.1 to 2.5 %.
template <typename T>
struct RowSum {
    typedef float type;
};
template <>
struct RowSum<float> {
    typedef double type;
};

// A lane owns a vector's neighbouring diagonals and walks down the strip's rows: its elements of
// a row lie together in memory, one place further along with every row.  kRows rows are added in
// RowSum, their sums in f64.  The wave then adds its diagonals up by buckets, which are runs of
// neighbouring diagonals, and the workgroup its waves.  Bound by HBM: 4 x 16 x 2048 x 2048 bf16
// 98 us with the last sums (5.5 TB/s); 107 while the edges' rows were masked in 64 bits.  Its loads
// start at any element, which fetches a tenth more than the tensor holds.  Strips of 32 rows: 64
// took 4 % longer, 128 12 % (fewer waves than fill the GPU evenly).
template <typename T, bool ONCE>
__global__ __launch_bounds__(kBlock) void k_relative_bias_backward(Map m, BiasBackArgs a) {
    __shared__ double s_sums[kWaves][kDiags<T>];
    __shared__ double s_part[kWaves][DET_BIAS_MAX_BUCKETS];
    __shared__ int s_starts[kBiasMaxSide];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    for (int i = threadIdx.x; i < m.side; i += kBlock) s_starts[i] = m.starts[i];
    // a workgroup takes kWaves neighbouring tiles (diagonals, then strips) of one head
    const int64_t per_head = (a.qt * a.dt + kWaves - 1) / kWaves;
    double* s_sum = s_sums[wave];
    __syncthreads();
    for (int64_t group = blockIdx.x; group < a.batch * a.heads * per_head; group += gridDim.x) {
        const int64_t bh = split(group, per_head), tile = (group - bh * per_head) * kWaves + wave;
        const bool live = tile < a.qt * a.dt;
        const int64_t qt = split(tile, a.dt), dt = tile - qt * a.dt;
        const int64_t b = split(bh, a.heads), h = bh - b * a.heads;
        const int64_t off = offset_of(m, b), len = length_of(m, b);
        const int64_t q0 = qt * a.strip;
        int64_t q1 = !live ? q0 : q0 + a.strip < m.q ? q0 + a.strip : m.q;
        if (q1 > len - off) q1 = len - off;               // rows past the sequence hold nothing
        const int64_t keys = len < m.k ? len : m.k;       // keys past it neither
        // diagonal d of the strip, from 0: key = row + d - shift
        const int64_t shift = q0 + a.strip - 1;
        const int64_t d0 = dt * kDiags<T> + kVec<T> * lane - shift;    // key = row + d0 + i
        double acc[kVec<T>] = {};
        const T* p = static_cast<const T*>(a.dout);
        const int64_t base = b * a.sb + h * a.sh + d0;
        const bool some = !m.causal || d0 - off <= 0;
        const bool whole = some && q0 + d0 >= 0 && q1 + d0 + kVec<T> - 1 <= keys;
        const bool inner = __all(whole);
        // the blocks of rows that meet the wave's diagonals
        const int64_t w0 = dt * kDiags<T> - shift;
        const int64_t lo = -(w0 + kDiags<T> - 1), hi = keys - w0;
        const int64_t from = lo > q0 ? q0 + (lo - q0) / kRows * kRows : q0;
        const int64_t to = m.causal && w0 - off > 0 ? from : hi < q1 ? hi : q1;
        for (int64_t row = from; row < to; row += kRows) {
            u32x4 raw[kRows];
            typename RowSum<T>::type sum[kVec<T>] = {};
            // of the vector in the first row: its place, its key, clipped, and the keys from it on
            const int64_t at = base + row * (a.sq + 1), key = row + d0, rest = keys - key;
            const int c = key < -64 ? -64 : key > 0 ? 0 : (int)key;
            const int n = rest < 0 ? 0 : rest > 64 ? 64 : (int)rest;
            const int rows = q1 - row < kRows ? (int)(q1 - row) : kRows;
            if (inner && rows == kRows) {
#pragma unroll
                for (int j = 0; j < kRows; ++j) raw[j] = load_vec<ONCE>(p + at + j * (a.sq + 1));
#pragma unroll
                for (int j = 0; j < kRows; ++j) {
                    float v[kVec<T>];
                    unpack<T>(raw[j], v);
#pragma unroll
                    for (int i = 0; i < kVec<T>; ++i) sum[i] += v[i];
                }
            } else if (!some || c + kRows + kVec<T> <= 1 || n == 0) {
                // none of these rows has a place on the lane's diagonals
            } else if (at >= 0 && at + (kRows - 1) * (a.sq + 1) + kVec<T> <= a.extent) {
                // whole vectors inside the tensor, what lies outside the row dropped
#pragma unroll
                for (int j = 0; j < kRows; ++j) {
                    raw[j] = u32x4{};
                    if (j < rows && c + j + kVec<T> > 0 && j < n)
                        raw[j] = load_vec<ONCE>(p + at + j * (a.sq + 1));
                }
#pragma unroll
                for (int j = 0; j < kRows; ++j) {
                    float v[kVec<T>];
                    unpack<T>(raw[j], v);
#pragma unroll
                    for (int i = 0; i < kVec<T>; ++i) sum[i] += i + j >= -c && i + j < n ? v[i] : 0.0f;
                }
            } else {
                // at the tensor's very ends, one by one; what does not count is read from the
                // nearest place inside (branches would make the loads wait for each other)
#pragma unroll 2
                for (int j = 0; j < rows; ++j) {
                    T v[kVec<T>];
#pragma unroll
                    for (int i = 0; i < kVec<T>; ++i) {
                        int64_t place = at + j * (a.sq + 1) + i;
                        place = place < 0 ? 0 : place < a.extent ? place : a.extent - 1;
                        v[i] = p[place];
                    }
#pragma unroll
                    for (int i = 0; i < kVec<T>; ++i)
                        sum[i] += i + j >= -c && i + j < n ? (float)v[i] : 0.0f;
                }
            }
#pragma unroll
            for (int i = 0; i < kVec<T>; ++i) acc[i] += (double)sum[i];
        }
        // a diagonal after the query is masked as a whole when causal
#pragma unroll
        for (int i = 0; i < kVec<T>; ++i)
            if (m.causal && d0 + i - off > 0) acc[i] = 0.0;
        const int64_t r0 = dt * kDiags<T> - shift - off;     // r of the tile's diagonal 0
        // lane by lane the buckets' runs of diagonals [first, last)
        bool laid_out = false;
        for (int bk0 = 0; bk0 < a.buckets; bk0 += 64) {
            const int bk = bk0 + lane;
            int64_t lo = 0, hi = 0;                       // r in [lo, hi)
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
            const int first = (int)(lo < 0 ? 0 : lo > kDiags<T> ? kDiags<T> : lo);
            const int last = (int)(hi < 0 ? 0 : hi > kDiags<T> ? kDiags<T> : hi);
            const bool wide = last - first > kShortRun;
            double mine = 0.0;
            // long runs (far from the diagonal one covers the tile): by the whole wave
            for (uint64_t runs = __ballot(wide); runs; runs &= runs - 1) {
                const int l = __ffsll((unsigned long long)runs) - 1;
                const int f = __builtin_amdgcn_readlane(first, l) - kVec<T> * lane;
                const int t = __builtin_amdgcn_readlane(last, l) - kVec<T> * lane;
                double v = 0.0;
#pragma unroll
                for (int i = 0; i < kVec<T>; ++i)
                    if (i >= f && i < t) v += acc[i];
                v = wave_pw(v);
                if (lane == l) mine = v;
            }
            // short ones: each by one lane, the diagonals laid out in LDS
            if (__ballot(!wide && first < last)) {
                if (!laid_out) {
                    wave_sync();
#pragma unroll
                    for (int i = 0; i < kVec<T>; ++i) s_sum[kVec<T> * lane + i] = acc[i];
                    wave_sync();
                    laid_out = true;
                }
                if (!wide) {
#pragma unroll 4
                    for (int i = first; i < last; ++i) mine += s_sum[i];
                }
            }
            if (bk < a.buckets) s_part[wave][bk] = mine;
        }
        __syncthreads();
        for (int bk = threadIdx.x; bk < a.buckets; bk += kBlock) {
            double v = s_part[0][bk];
#pragma unroll
            for (int w = 1; w < kWaves; ++w) v += s_part[w][bk];
            a.part[group * a.buckets + bk] = v;
        }
        __syncthreads();      // s_part is written again
    }
}

constexpr int kSumBuckets = 8;      // buckets a workgroup of the last sums takes (64 bytes)
constexpr int kSumBlock = 512;

// dtable[bk][h] = the workgroups' sums of every sequence: row g of 64 adds items g, g + 64, ...
// (sequence by sequence) in that order, then the rows join by a halving tree.
template <typename T>
__global__ __launch_bounds__(kSumBlock) void k_bias_table_sums(const double* part, int64_t batch,
                                                               int64_t heads, int64_t per_head,
                                                               int buckets, T* out) {
    constexpr int kGroups = kSumBlock / kSumBuckets;
    __shared__ double s[kGroups][kSumBuckets];
    const int blocks = (buckets + kSumBuckets - 1) / kSumBuckets;
    const int x = threadIdx.x % kSumBuckets, g = threadIdx.x / kSumBuckets;
    const int bk = blockIdx.x % blocks * kSumBuckets + x;
    const int64_t h = blockIdx.x / blocks, items = batch * per_head;
    double v = 0.0;
    if (bk < buckets) {
#pragma unroll 4
        for (int64_t i = g; i < items; i += kGroups) {
            const int64_t b = i / per_head, t = i - b * per_head;
            v += part[((b * heads + h) * per_head + t) * buckets + bk];
        }
    }
    s[g][x] = v;
    __syncthreads();
    for (int n = kGroups / 2; n > 0; n >>= 1) {
        if (g < n) s[g][x] += s[g + n][x];
        __syncthreads();
    }
    if (g == 0 && bk < buckets) out[bk * heads + h] = (T)s[0][x];
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
    for (m.top = 1; 2 * m.top < m.side;) m.top *= 2;
    m.two_sided = c.bidirectional;
    m.causal = c.causal;
    m.q = c.q;
    m.k = c.k;
    m.q_offset = c.q_offset;
    m.q_offsets = c.q_offsets;
    m.lengths = c.lengths;
    return m;
}

// elements from the strided tensor's first to behind its last
int64_t extent_of(const BiasCall& c) {
    if (c.batch == 0 || c.q == 0 || c.k == 0) return 0;
    return (c.batch - 1) * c.sb + (c.heads - 1) * c.sh + (c.q - 1) * c.sq + c.k;
}

unsigned grid_of(int64_t tiles) { return (unsigned)(tiles < (1 << 22) ? tiles : (1 << 22)); }

template <typename T>
void bias_typed(const BiasCall& c, hipStream_t s) {
    const Map m = map_of(c);
    BiasArgs a{c.table, c.scores, c.out, c.sb, c.sh, c.sq, extent_of(c), c.heads, c.batch, 8,
               kRows, c.buckets, c.fill, 0};
    // as many lanes across the keys as the row has vectors (at most the workgroup), the rest of
    // the workgroup on further rows
    while (a.lanes_log2 > 3 && ((int64_t)kVec<T> << (a.lanes_log2 - 1)) >= c.k) --a.lanes_log2;
    const int teams = kBlock >> a.lanes_log2;
    const int64_t width = (int64_t)kVec<T> << a.lanes_log2;
    const int64_t kt = (c.k + width - 1) / width, bh = a.batch * a.heads;
    if (c.q < kRows) {
        const int64_t rows = (bh * c.q + teams - 1) / teams;
        const dim3 grid((unsigned)kt, (unsigned)(rows < 65535 ? rows : 65535));
        KernelTimer timer("k_relative_bias_row", s);
        if (c.scores)
            k_relative_bias_row<T, true><<<grid, dim3(kBlock), 0, s>>>(m, a);
        else
            k_relative_bias_row<T, false><<<grid, dim3(kBlock), 0, s>>>(m, a);
        return;
    }
    // long walks share one layout of the diagonals among more rows, as long as workgroups enough
    // to fill the GPU are left
    while (a.rows < 64 && (int64_t)a.rows * teams < c.q &&
           bh * kt * ((c.q + 2 * a.rows * teams - 1) / (2 * a.rows * teams)) >= 2048)
        a.rows *= 2;
    const int64_t height = (int64_t)teams * a.rows;
    a.qt = (c.q + height - 1) / height;
    const int lds = (int)(width + height) * (int)sizeof(float);
    const dim3 grid((unsigned)kt, (unsigned)(a.qt < 65535 ? a.qt : 65535),
                    (unsigned)(bh < 65535 ? bh : 65535));
    KernelTimer timer("k_relative_bias", s);
    if (c.scores)
        k_relative_bias<T, true><<<grid, dim3(kBlock), lds, s>>>(m, a);
    else
        k_relative_bias<T, false><<<grid, dim3(kBlock), lds, s>>>(m, a);
}

struct BackShape {
    int strip;
    int64_t qt, dt;
};

// Rows a strip and the diagonals' tiles, from the sizes alone: the order of the sums.  Strips of
// 32 rows, halved down to 8 while that leaves fewer than 2048 waves (4096: 3 x 5 x 777 x 1003 f32,
// causal and ragged, 13.7 us instead of 11.6, 4 x 16 x 700 x 800 bf16 17.3 instead of 15.9).
BackShape back_shape(int64_t batch, int64_t heads, int64_t q, int64_t k, int64_t diags) {
    BackShape r;
    for (r.strip = 32;; r.strip /= 2) {
        r.qt = (q + r.strip - 1) / r.strip;
        r.dt = (k + r.strip - 1 + diags - 1) / diags;
        if (r.strip == kRows || (double)batch * heads * r.qt * r.dt >= 2048.0) return r;
    }
}

template <typename T>
det_status back_typed(const BiasCall& c, const void* dout, void* dtable, void* ws, hipStream_t s) {
    const Map m = map_of(c);
    const BackShape sh = back_shape(c.batch, c.heads, c.q, c.k, kDiags<T>);
    BiasBackArgs a{dout, static_cast<double*>(ws), c.sb, c.sh, c.sq, extent_of(c), c.heads,
                   c.batch, sh.strip, sh.qt, sh.dt, c.buckets};
    const int64_t per_head = (sh.qt * sh.dt + kWaves - 1) / kWaves;
    const int64_t groups = c.q > 0 && c.k > 0 ? c.batch * c.heads * per_head : 0;
    if (groups > 0) {
        KernelTimer kt("k_relative_bias_backward", s);
        if ((double)c.batch * c.heads * c.q * c.k * sizeof(T) >= (double)kOnceBytes)
            k_relative_bias_backward<T, true><<<dim3(grid_of(groups)), dim3(kBlock), 0, s>>>(m, a);
        else
            k_relative_bias_backward<T, false><<<dim3(grid_of(groups)), dim3(kBlock), 0, s>>>(m, a);
        const det_status st = launch_status();
        if (st != DET_SUCCESS) return st;
    }
    KernelTimer kt("k_bias_table_sums", s);
    const int64_t wgs = c.heads * ((c.buckets + kSumBuckets - 1) / kSumBuckets);
    k_bias_table_sums<T><<<dim3((unsigned)wgs), dim3(kSumBlock), 0, s>>>(
        a.part, groups > 0 ? c.batch : 0, c.heads, per_head, c.buckets, static_cast<T*>(dtable));
    return launch_status();
}

}  // namespace

size_t bias_backward_workspace(int64_t batch, int64_t heads, int64_t q, int64_t k, int buckets,
                               det_dtype dtype) {
    const BackShape s = back_shape(batch, heads, q, k,
                                   dtype == DET_F32 ? kDiags<float> : kDiags<_Float16>);
    const int64_t per_head = (s.qt * s.dt + kWaves - 1) / kWaves;
    return round_up((size_t)batch * heads * per_head * buckets * sizeof(double), 256) + 256;
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
