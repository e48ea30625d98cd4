// xent.hip -- cross entropy of softmax(scale * x weight^T) without keeping the logits, and its
// gradients, in pieces of the vocabulary.
//
// Mathematics, per row of x:  z = scale * x weight^T;  lse = log(sum exp z);  loss = lse - z[target]
//   D = exp(z - lse) - hit;  dx = scale * dloss * (D weight);  dweight = scale * (dloss D)^T x
// A row whose target lies outside the vocabulary has loss 0 and adds to no gradient.
//
// Every product is C[i][j] = sum over k of A[i][k] B[j][k], one kernel with four endings:
//   stats    i vocabulary, j rows of x, k width:  largest logit and sum of a tile's logits per row
//   dlogits  the same product again: D by rows (for dx) and by columns (for dweight), rounded to the
//            storage type once, as the matrix instructions take both their factors in it: the gradients of
//            4096 x 65536 x 4096 bf16 are off by 1.45 times what a D of 32 bits gives
//   dx       i width, j rows, k a piece of the vocabulary: weight transposed, D
//   dweight  i width, j vocabulary, k rows: x transposed, D's columns times dloss (f32: x times dloss)
// f32 goes through the matrix units in three bfloat16 parts of 8 bits each (exact together) and six
// products of parts; the three left out are within 2^-22 of the whole one, to either side, and an infinite
// factor may give NaN.
//
// Order: k ascending in steps of 16 inside the matrix instruction's own order, f32 accumulators (in tiles
// of 32 columns several in turn, joined in pairs: chains_of); a tile's logits, then the tiles of a row by
// lanes and the adjacent-lanes tree; dx adds pieces of the vocabulary in ascending order, then the parts
// that share a piece.  All of it fixed by (rows, vocab, d, dtype).
#include "det_internal.h"
#include "lm_device.h"

namespace det {
namespace {

constexpr int kDepth = 64, kDepthF32 = 32;    // elements of k a step: 128 bytes of a row
constexpr int64_t kPieceUnit = 256;           // a piece's entries are a multiple of every tile's
constexpr int64_t kPieceCells = 1 << 26;      // elements of D that a piece holds, up to 16384 rows
constexpr int64_t kPieceMin = 4096;           // above them a piece's entries: D has 4096 elements a row
constexpr int64_t kPieceMax = 65536;

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
int64_t up(int64_t a, int64_t b) { return cdiv(a, b) * b; }

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(3))) void* lds_ptr;

// one operand: rows of k elements, ld bytes apart
struct Operand {
    const char* p;
    int64_t rows, ld;
};

struct GemmArgs {
    Operand A, B;
    int64_t k;            // elements of a row that count
    int64_t ni, nj;       // tiles along i and j
    int64_t parts, per_part;      // of k, and the steps of one
    float scale;
    // stats, dlogits
    const int64_t* targets;
    int64_t v0, vocab, tile0, tiles;      // the piece's first entry, its first of `tiles` tiles
    u32x2* stats;                         // [row][tile]: largest logit, sum (two floats)
    float* hit;                           // [row]: the target's logit
    const float *lse, *dloss, *unit;      // unit: f16, the largest |dloss|
    char *d, *dt;                         // D by rows and by columns
    int64_t d_ld, dt_ld, rows_up, piece_up;      // bytes; D's rows and columns with their zeros
    // dx, dweight
    void* out;
    int64_t out_ld;       // elements
    bool add;
};

__device__ __forceinline__ f32x16 mma(u32x4 a, u32x4 b, f32x16 c, __bf16) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}
__device__ __forceinline__ f32x16 mma(u32x4 a, u32x4 b, f32x16 c, _Float16) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a),
                                                  __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

// Two floats in three parts each, 8 bits a part: parts n of a and b side by side in p[n].  The first is cut
// off, so that the largest floats stay finite, the second is rounded to nearest, and the third is all that
// is left.  Their bounds are 1, 2^-7 and 2^-16 of the value, and the third has either sign: the products left
// out reach 2^-22 of the whole one and cancel in long sums.  (With every part cut off they reach 2^-21, all
// of one sign; with the first rounded too, 2^-24, but it has to be kept from infinity: 8 rows x 30000 x 1000
// 42.4 us, 44.5 so, 47.7.)  The rest of an infinity is NaN.
__device__ __forceinline__ void parts_of(uint32_t a, uint32_t b, uint32_t (&p)[3]) {
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
#pragma unroll
    for (int n = 0; n < 3; ++n) {
        if (n == 1)
            p[n] = __builtin_bit_cast(
                uint32_t,
                __builtin_convertvector(f32x2{__uint_as_float(a), __uint_as_float(b)}, bf16x2));
        else
            p[n] = __builtin_amdgcn_perm(b, a, 0x07060302u);      // their upper halves
        a = __float_as_uint(__uint_as_float(a) - __uint_as_float(p[n] << 16));
        b = __float_as_uint(__uint_as_float(b) - __uint_as_float(p[n] & 0xFFFF0000u));
    }
}

// D's factor in storage: f16 has few exponents, and |D| <= 1
template <typename T>
constexpr float kUnit = __is_same(T, _Float16) ? 16384.0f : 1.0f;

template <typename H>
__device__ __forceinline__ uint16_t half_bits(float v) {
    return __builtin_bit_cast(uint16_t, (H)v);
}

// A vector of a row, in `load_row`'s and `settle`'s two steps where it may reach past the row's end.
template <bool WHOLE, typename T>
__device__ __forceinline__ u32x4 fetch_vec(const T* row, int64_t c, int64_t n) {
    if constexpr (WHOLE)
        return load_vec(row + c);
    else
        return load_row(row, c, n);
}
template <bool WHOLE, typename T>
__device__ __forceinline__ u32x4 settle_vec(u32x4 raw, int64_t c, int64_t n) {
    if constexpr (WHOLE)
        return raw;
    else
        return settle<T>(raw, c, n);
}
struct Whole {
    static constexpr bool value = true;
};
struct Partial {
    static constexpr bool value = false;
};

enum Ending { kStats, kLogits, kDx, kDw };

// Accumulators of a wave's tile of 32 x 32, which take the steps of 16 in turn: a tile of 32 columns has one
// such tile a wave and room for more, and its sums are four (f32: two) times as short.  Larger tiles have
// none to spare.
template <int MI, int MJ>
constexpr int chains_of(int depth) {
    return MI * MJ == 1 ? depth / 16 : 1;
}

// joined in pairs into the first
template <int CHAINS, int MI, int MJ>
__device__ __forceinline__ void join_chains(f32x16 (&acc)[CHAINS][MI][MJ]) {
#pragma unroll
    for (int step = 1; step < CHAINS; step *= 2)
#pragma unroll
        for (int c = 0; c < CHAINS; c += 2 * step)
#pragma unroll
            for (int i = 0; i < MI; ++i)
#pragma unroll
                for (int j = 0; j < MJ; ++j) acc[c][i][j] += acc[c + step][i][j];
}

// Columns of a tile on their way to rows in memory: a lane holds four elements of a column, whose rows in
// memory it would write 8 or 16 bytes at a time; through LDS a row's elements leave side by side.
// (dweight of 30000 entries x 1000 f32, 8 rows: 54 us, in pieces of 16 bytes 306: the rows that the
// chip has begun and not ended are as large as its caches.)  The 16-byte chunks of a column lie turned by it,
// so that lanes, a column each, write to different banks.
template <typename T, int BI>
__device__ __forceinline__ void column_put(char* lds, int col, int e, const float (&v)[4]) {
    if constexpr (sizeof(T) == 4) {
        *reinterpret_cast<f32x4*>(lds + col * BI * 4 + ((e / 4) ^ (col & 15)) * 16) =
            f32x4{v[0], v[1], v[2], v[3]};
    } else {
        uint32_t w[2];
#pragma unroll
        for (int r = 0; r < 2; ++r)
            w[r] = half_bits<T>(v[2 * r]) | (uint32_t)half_bits<T>(v[2 * r + 1]) << 16;
        *reinterpret_cast<u32x2*>(lds + col * BI * 2 + ((e / 8) ^ (col & 7)) * 16 + (e & 4) * 2) =
            u32x2{w[0], w[1]};
    }
}

// The columns j * 32 .. of every wave along j, elements below `left`, columns below `cols_left`.
template <typename T, int BI, int WJ, int MJ, int THREADS>
__device__ __forceinline__ void columns_out(const char* lds, int j, int left, int cols_left, T* out,
                                            int64_t ld) {
    constexpr int kChunks = BI / kVec<T>, kTurn = sizeof(T) == 4 ? 15 : 7;
    __syncthreads();
    for (int n = threadIdx.x; n < WJ * 32 * kChunks; n += THREADS) {
        const int in = n / kChunks, c = n % kChunks, col = (in / 32 * MJ + j) * 32 + in % 32;
        if (col >= cols_left || c * kVec<T> >= left) continue;
        const u32x4 w = *reinterpret_cast<const u32x4*>(lds + in * BI * (int)sizeof(T) + (c ^ (in & kTurn)) * 16);
        T* at = out + (int64_t)col * ld + c * kVec<T>;
        if (c * kVec<T> + kVec<T> <= left) {
            store_vec(at, w);
        } else {
#pragma unroll
            for (int i = 0; i < kVec<T>; ++i)
                if (c * kVec<T> + i < left) {
                    if constexpr (sizeof(T) == 4)
                        at[i] = __uint_as_float(w[i]);
                    else
                        at[i] = __builtin_bit_cast(T, (uint16_t)(w[i / 2] >> (16 * (i & 1))));
                }
        }
    }
    __syncthreads();
}

// What becomes of a tile at (i0, j0): wave (wi, wj)'s sums.  `lds` is free.
template <typename T, int WI, int WJ, int MI, int MJ, int END>
__device__ __forceinline__ void xent_ending(const GemmArgs& a, f32x16 (&acc)[MI][MJ], int64_t i0,
                                            int64_t j0, int part, int wi, int wj, char* lds) {
    constexpr int BI = WI * MI * 32, BJ = WJ * MJ * 32, NW = WI * WJ;
    const int lane = threadIdx.x & 63;
    // a lane's values: column wj.. + lane % 32, rows wi.. + 8 (r / 4) + 4 (lane / 32) + r % 4 of the tile
    const int row_base = wi * MI * 32 + 4 * (lane >> 5), col_base = wj * MJ * 32 + (lane & 31);
    const int col_in = wj * 32 + (lane & 31);      // among the columns of one j
    const auto row_of = [&](int i, int r) { return row_base + i * 32 + 8 * (r / 4) + r % 4; };
    const int rows_left = (int)(a.A.rows - i0 < BI ? a.A.rows - i0 : BI);
    const int cols_left = (int)(a.B.rows - j0 < BJ ? a.B.rows - j0 : BJ);
    // the place of a column's target among the lane's rows (row_of less row_base), -1 elsewhere
    const auto target_at = [&](int64_t target) {
        const int64_t at = target - a.v0 - i0;
        return at >= 0 && at < rows_left ? (int)at - row_base : -1;
    };

    if constexpr (END == kStats) {
        float* s_top = reinterpret_cast<float*>(lds);      // [WI][BJ], then the sums
        float* s_sum = s_top + WI * BJ;
#pragma unroll
        for (int j = 0; j < MJ; ++j) {
            const int col = col_base + j * 32;
            const int at = col < cols_left ? target_at(a.targets[j0 + col]) : -1;
            float top = -INFINITY;
            if (rows_left < BI) {
#pragma unroll
                for (int i = 0; i < MI; ++i)
#pragma unroll
                    for (int r = 0; r < 16; ++r)
                        if (row_of(i, r) >= rows_left) acc[i][j][r] = -INFINITY;
            }
#pragma unroll
            for (int i = 0; i < MI; ++i)
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    acc[i][j][r] *= a.scale;
                    top = fmaxf(top, acc[i][j][r]);
                }
            if (at >= 0) {      // the lane may hold it
                float hit = 0.0f;
                bool mine = false;
#pragma unroll
                for (int i = 0; i < MI; ++i)
#pragma unroll
                    for (int r = 0; r < 16; ++r)
                        if (at == i * 32 + 8 * (r / 4) + r % 4) {
                            hit = acc[i][j][r];
                            mine = true;
                        }
                if (mine) a.hit[j0 + col] = hit;
            }
            const float ref = top > -INFINITY ? top : 0.0f;
            float sum = 0.0f;
#pragma unroll
            for (int i = 0; i < MI; ++i)
#pragma unroll
                for (int r = 0; r < 16; ++r) sum += exp_fast(acc[i][j][r] - ref);
            // the other half of the wave has the same column
            const float other_top = __shfl_xor(top, 32), other_sum = __shfl_xor(sum, 32);
            const float both = fmaxf(top, other_top), from = both > -INFINITY ? both : 0.0f;
            if (lane < 32) {
                s_top[wi * BJ + col] = both;
                s_sum[wi * BJ + col] = sum * exp_fast(top - from) + other_sum * exp_fast(other_top - from);
            }
        }
        __syncthreads();
        for (int c = threadIdx.x; c < cols_left; c += NW * 64) {
            float top = s_top[c];
#pragma unroll
            for (int w = 1; w < WI; ++w) top = fmaxf(top, s_top[w * BJ + c]);
            const float from = top > -INFINITY ? top : 0.0f;
            float sum = 0.0f;
#pragma unroll
            for (int w = 0; w < WI; ++w) sum += s_sum[w * BJ + c] * exp_fast(s_top[w * BJ + c] - from);
            a.stats[(j0 + c) * a.tiles + a.tile0 + i0 / BI] =
                u32x2{__float_as_uint(top), __float_as_uint(sum)};
        }
    } else if constexpr (END == kLogits) {
        const int d_left = (int)(a.piece_up - i0 < BI ? a.piece_up - i0 : BI);      // of D's rows
        const int dt_left = (int)(a.rows_up - j0 < BJ ? a.rows_up - j0 : BJ);       // of its columns'
#pragma unroll
        for (int j = 0; j < MJ; ++j) {
            const int col = col_base + j * 32;
            const bool real = col < cols_left;
            const int64_t target = real ? a.targets[j0 + col] : -1;
            const bool scored = target >= 0 && target < a.vocab;
            const int at = target_at(target);
            const float lse = scored ? a.lse[j0 + col] : 0.0f;
            const float unit = scored ? kUnit<T> : 0.0f;
            float weight = scored ? a.dloss[j0 + col] : 0.0f;
            if constexpr (__is_same(T, _Float16)) weight = *a.unit > 0.0f ? weight / *a.unit : 0.0f;
            char* const dt_at = a.dt + (i0 + row_base) * a.dt_ld + (j0 + col) * (int64_t)sizeof(T);
#pragma unroll
            for (int i = 0; i < MI; ++i)
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    const int in_lane = i * 32 + 8 * g, v = row_base + in_lane;      // and three behind it
                    float d[4];
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const float p = exp_fast(acc[i][j][4 * g + r] * a.scale - lse);
                        d[r] = at == in_lane + r ? p - 1.0f : p;
                        d[r] = scored && v + r < rows_left ? d[r] * unit : 0.0f;
                    }
                    column_put<T, BI>(lds, col_in, v, d);
                    if constexpr (sizeof(T) == 2) {
#pragma unroll
                        for (int r = 0; r < 4; ++r)
                            if (v + r < rows_left && col < dt_left)
                                *reinterpret_cast<uint16_t*>(dt_at + (in_lane + r) * a.dt_ld) =
                                    half_bits<T>(d[r] * weight);
                    }
                }
            columns_out<T, BI, WJ, MJ, NW * 64>(lds, j, d_left, cols_left,
                                                reinterpret_cast<T*>(a.d + j0 * a.d_ld) + i0,
                                                a.d_ld / (int64_t)sizeof(T));
        }
    } else {
        // dx: f32 sums of a part; dweight: the gradient in its type
#pragma unroll
        for (int j = 0; j < MJ; ++j) {
            const int col = col_base + j * 32;
            float f = 1.0f;
            if constexpr (END == kDw) {
                f = a.scale / kUnit<T>;
                if constexpr (__is_same(T, _Float16)) f *= *a.unit;
            }
#pragma unroll
            for (int i = 0; i < MI; ++i)
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    const int e = row_of(i, 4 * g);
                    float v[4];
#pragma unroll
                    for (int r = 0; r < 4; ++r) v[r] = acc[i][j][4 * g + r] * f;
                    if constexpr (END == kDw) {
                        column_put<T, BI>(lds, col_in, e, v);
                    } else if (col < cols_left && e < rows_left) {
                        float* at = static_cast<float*>(a.out) + part * a.B.rows * a.out_ld +
                                    (j0 + col) * a.out_ld + i0 + e;      // out_ld: a multiple of 4, room for 4
                        if (a.add) {
                            const f32x4 old = *reinterpret_cast<const f32x4*>(at);
#pragma unroll
                            for (int r = 0; r < 4; ++r) v[r] = old[r] + v[r];
                        }
                        *reinterpret_cast<f32x4*>(at) = f32x4{v[0], v[1], v[2], v[3]};
                    }
                }
            if constexpr (END == kDw)
                columns_out<T, BI, WJ, MJ, NW * 64>(lds, j, rows_left, cols_left,
                                                    static_cast<T*>(a.out) + j0 * a.out_ld + i0, a.out_ld);
        }
    }
}

// Place of the workgroup's tile and its part of k.  Workgroup b runs on XCD b % 8: each takes a run of
// tiles, four along j by as many as follow along i, of one part of k and then the next, so that what
// an XCD holds at a time shares its rows in its L2.
template <int BI, int BJ>
__device__ __forceinline__ bool tile_of(const GemmArgs& a, int64_t& i0, int64_t& j0, int& part) {
    const int64_t tiles = a.ni * a.nj, all = tiles * a.parts, per = (all + 7) / 8;
    int64_t q = (int64_t)(blockIdx.x & 7) * per + (blockIdx.x >> 3);
    if ((blockIdx.x >> 3) >= per || q >= all) return false;
    part = a.parts > 1 ? (int)(q / tiles) : 0;
    q -= part * tiles;
    const int64_t band = q / (4 * a.ni), in_band = q % (4 * a.ni);
    const int64_t wide = a.nj - 4 * band < 4 ? a.nj - 4 * band : 4;
    i0 = in_band / wide * BI;
    j0 = (4 * band + in_band % wide) * BJ;
    return true;
}

// 16-bit types.  Wave grid WI x WJ, a wave has MI x MJ tiles of 32 x 32.  A step's rows go from memory
// straight to LDS, two steps in turn: 8 rows of 128 bytes a load, whose 16-byte chunks lie in the order
// chunk ^ (row / 2 % 8), so that the 16 rows that a read of the operands takes at a time lie in
// different banks.  What lies past an operand's rows or k reads as zero (the buffer's bounds).
//
// Bound by the matrix units and the clock that their power leaves: 4096 rows x 65536 entries x 4096 bf16
// takes 1.79 ms (1.23 PFLOP/s) for the sums of the softmax, 460 us for a quarter of dx or of dweight (1.2) and
// 518 for a quarter of D, which is stored twice; of the cycles (1.7 GHz over the sums) the matrix units work
// 70, 63 and 56 %, LDS has no bank conflicts in the products.  (Another card: 1.71 ms, 445 and 502 us.)  A row
// takes 42 us (268 MB, 6.4 TB/s).  Slower by 3 and 10 %: steps of half the depth, four in turn; four waves
// with tiles of 128 x 128.
// STAGED: rows that do not lie on 16 bytes go through registers instead (517 x 50021 f16: 1003 elements a row 113
// us, 1004 100, 1008 80; a vector off 16 bytes spans two lines).
template <typename T, int WI, int WJ, int MI, int MJ, bool STAGED, int END>
__device__ __forceinline__ void xent_product(const GemmArgs& a) {
    constexpr int BI = WI * MI * 32, BJ = WJ * MJ * 32, NW = WI * WJ;
    constexpr int kRow = kDepth * 2, kRows = 8;                    // rows of a load
    constexpr int LA = BI / kRows / NW, LB = BJ / kRows / NW;      // loads of a wave a step
    static_assert(BI % (kRows * NW) == 0 && BJ % (kRows * NW) == 0, "rows of a step per wave");
    constexpr int kStage = (BI + BJ) * kRow;
    __shared__ __attribute__((aligned(16))) char s_0[kStage];
    __shared__ __attribute__((aligned(16))) char s_1[kStage];
    // the places of a row's chunks are turned by this much
    const auto turn_of = [](int row) { return row >> 1 & 7; };
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int wi = wave / WJ, wj = wave % WJ;
    int64_t i0, j0;
    int part;
    if (!tile_of<BI, BJ>(a, i0, j0, part)) return;
    // a load's 8 rows are half of what the turn goes by: every other load's chunks differ
    const int in_load = lane >> 3;
    const int chunk[2] = {(lane & 7) ^ turn_of(in_load), (lane & 7) ^ turn_of(kRows + in_load)};
    const int first = (int)(part * a.per_part), steps = (int)((a.k + kDepth - 1) / kDepth);
    const int behind = first + a.per_part < steps ? (int)(first + a.per_part) : steps;
    constexpr int kChains = chains_of<MI, MJ>(kDepth);
    f32x16 acc[kChains][MI][MJ] = {};
    const auto products = [&](const char* s) {
        const char* pa = s + (wi * MI * 32 + (lane & 31)) * kRow;
        const char* pb = s + (BI + wj * MJ * 32 + (lane & 31)) * kRow;
        constexpr int kSteps = kDepth / 16;
        u32x4 av[2][MI], bv[2][MJ];
        const auto read = [&](int kk) {
            const int slot = ((kk * 2 + (lane >> 5)) ^ turn_of(lane & 31)) * 16;
#pragma unroll
            for (int j = 0; j < MJ; ++j)
                bv[kk & 1][j] = *reinterpret_cast<const u32x4*>(pb + j * 32 * kRow + slot);
#pragma unroll
            for (int i = 0; i < MI; ++i)
                av[kk & 1][i] = *reinterpret_cast<const u32x4*>(pa + i * 32 * kRow + slot);
        };
        read(0);
#pragma unroll
        for (int kk = 0; kk < kSteps; ++kk) {
            if (kk + 1 < kSteps) read(kk + 1);
#pragma unroll
            for (int i = 0; i < MI; ++i)
#pragma unroll
                for (int j = 0; j < MJ; ++j)
                    acc[kk % kChains][i][j] =
                        mma(av[kk & 1][i], bv[kk & 1][j], acc[kk % kChains][i][j], T{});
        }
        // In this order: the first operands, the next step's loads, and the operands behind them one by one
        // between matrix instructions.  (Left to the compiler each is waited for where it is read: forward of
        // 4096 x 65536 x 4096 bf16 1.86 ms, 1.75 so, backward 5.99 and 5.89; loads between the matrix
        // instructions too 1.82 and 6.03 to 6.11.)
        __builtin_amdgcn_sched_group_barrier(0x100, MI + MJ, 0);
        if constexpr (!STAGED) __builtin_amdgcn_sched_group_barrier(0x20, LA + LB, 0);
#pragma unroll
        for (int kk = 0; kk + 1 < kSteps; ++kk) {
#pragma unroll
            for (int n = 0; n < MI * MJ; ++n) {
                __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
                if (n < MI + MJ) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
            }
        }
        __builtin_amdgcn_sched_group_barrier(0x8, MI * MJ, 0);
    };
    if constexpr (STAGED) {
        // Rows that lie at any element: through registers, a step ahead (a tile of few columns, which waits
        // for memory, two), rows past the last one as that.  dx reads weight with k along its columns: a
        // lane takes four elements of k by eight rows of A and writes a row's four side by side.
        constexpr bool kAcross = END == kDx;
        constexpr int kSets = NW == 8 ? 1 : 2;
        static_assert(!kAcross || (BI == 64 && NW == 2), "a wave takes half of a step's k");
        const int rows_a = (int)(a.A.rows - i0 < BI ? a.A.rows - i0 : BI);
        const int rows_b = (int)(a.B.rows - j0 < BJ ? a.B.rows - j0 : BJ);
        const char* at_a[kAcross ? 1 : LA];
        const char* at_b[LB];
        if constexpr (!kAcross) {
#pragma unroll
            for (int u = 0; u < LA; ++u) {
                const int r = (wave * LA + u) * kRows + in_load;
                at_a[u] = a.A.p + i0 * a.A.ld + (r < rows_a ? r : rows_a - 1) * a.A.ld;
            }
        }
#pragma unroll
        for (int u = 0; u < LB; ++u) {
            const int r = (wave * LB + u) * kRows + in_load;
            at_b[u] = a.B.p + j0 * a.B.ld + (r < rows_b ? r : rows_b - 1) * a.B.ld;
        }
        u32x4 ga[kSets][LA], gb[kSets][LB];
        const int in_k = (wave * 8 + in_load) * 4, in_a = (lane & 7) * 8;      // kAcross
        const int64_t col = i0 + in_a < a.A.rows ? i0 + in_a : a.A.rows;
        const auto column = [&](int step, int load) {      // past the last step: k
            return step < behind ? (int64_t)step * kDepth + chunk[load & 1] * 8 : a.k;
        };
        // nearly every step is whole, and its vectors need no care (517 x 50021 x 1002 f16 107 -> 100 us; with k
        // along the columns the second form of it costs more than it gives, 77 -> 80 for 8 x 30000 x 1000)
        const auto whole = [&](int step) {
            return !kAcross && step < behind && (int64_t)(step + 1) * kDepth <= a.k;
        };
        const auto fetch_as = [&](auto as, int set, int step) {
            constexpr bool W = decltype(as)::value;
#pragma unroll
            for (int u = 0; u < LA; ++u) {
                if constexpr (kAcross) {
                    const int64_t k = (int64_t)step * kDepth + in_k + u, row = k < a.k ? k : a.k - 1;
                    ga[set][u] = load_row(reinterpret_cast<const T*>(a.A.p + row * a.A.ld), col, a.A.rows);
                } else {
                    ga[set][u] =
                        fetch_vec<W>(reinterpret_cast<const T*>(at_a[u]), column(step, wave * LA + u), a.k);
                }
            }
#pragma unroll
            for (int u = 0; u < LB; ++u)
                gb[set][u] = fetch_vec<W>(reinterpret_cast<const T*>(at_b[u]), column(step, wave * LB + u), a.k);
        };
        const auto fetch = [&](int set, int step) {
            if (whole(step))
                fetch_as(Whole{}, set, step);
            else
                fetch_as(Partial{}, set, step);
        };
        const auto put_as = [&](auto as, char* s, int set, int step) {
            constexpr bool W = decltype(as)::value;
            if constexpr (kAcross) {
                const int64_t k = step < behind ? (int64_t)step * kDepth + in_k : a.k;
                u32x4 r[4];
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    r[u] = settle<T>(ga[set][u], col, a.A.rows);
                    if (k + u >= a.k) r[u] = u32x4{0, 0, 0, 0};
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const uint32_t half = i & 1 ? 0x07060302u : 0x05040100u;
                    *reinterpret_cast<u32x2*>(s + (in_a + i) * kRow + ((in_k >> 3) ^ turn_of(in_a + i)) * 16 +
                                              (in_k & 4) * 2) =
                        u32x2{__builtin_amdgcn_perm(r[1][i / 2], r[0][i / 2], half),
                              __builtin_amdgcn_perm(r[3][i / 2], r[2][i / 2], half)};
                }
            } else {
#pragma unroll
                for (int u = 0; u < LA; ++u)
                    *reinterpret_cast<u32x4*>(s + (wave * LA + u) * 1024 + lane * 16) =
                        settle_vec<W, T>(ga[set][u], column(step, wave * LA + u), a.k);
            }
#pragma unroll
            for (int u = 0; u < LB; ++u)
                *reinterpret_cast<u32x4*>(s + BI * kRow + (wave * LB + u) * 1024 + lane * 16) =
                    settle_vec<W, T>(gb[set][u], column(step, wave * LB + u), a.k);
        };
        const auto put = [&](char* s, int set, int step) {
            if (whole(step))
                put_as(Whole{}, s, set, step);
            else
                put_as(Partial{}, s, set, step);
        };
        const auto one = [&](const char* now, char* next, int set, int step) {
            products(now);
            put(next, set, step + 1);
            fetch(set, step + 1 + kSets);
            __syncthreads();
        };
        fetch(0, first);
        put(s_0, 0, first);
        fetch(1 % kSets, first + 1);
        if constexpr (kSets == 2) fetch(0, first + 2);
        __syncthreads();
        // past the last step: zeros (settle)
#pragma unroll 1
        for (int step = first; step < behind; step += 2) {
            one(s_0, s_1, 1 % kSets, step);
            one(s_1, s_0, 0, step + 1);
        }
    } else {
        const auto records = [&](const Operand& o, int64_t from, int64_t most) {
            const int64_t rows = o.rows - from < most ? o.rows - from : most;
            return (uint32_t)((rows - 1) * o.ld + a.k * 2);
        };
        const auto ra = __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(a.A.p + i0 * a.A.ld), 0,
                                                          records(a.A, i0, BI), 0x00020000);
        const auto rb = __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(a.B.p + j0 * a.B.ld), 0,
                                                          records(a.B, j0, BJ), 0x00020000);
        const uint32_t lda = (uint32_t)a.A.ld, ldb = (uint32_t)a.B.ld;
        const uint32_t oa = (uint32_t)(wave * LA * kRows + in_load) * lda;
        const uint32_t ob = (uint32_t)(wave * LB * kRows + in_load) * ldb;
        const auto issue = [&](char* s, int step) {
            constexpr uint32_t kOut = 0x80000000u;      // past every row
            const uint32_t at = (uint32_t)step * kRow;
            const int left = step < behind ? (int)a.k - step * kDepth : 0;      // elements of k
#pragma unroll
            for (int u = 0; u < LA; ++u) {
                const int c = chunk[(wave * LA + u) & 1];
                __builtin_amdgcn_raw_ptr_buffer_load_lds(
                    ra, (lds_ptr)(s + (wave * LA + u) * 1024), 16,
                    c * 8 < left ? oa + u * kRows * lda + at + c * 16 : kOut, 0, 0, 0);
            }
#pragma unroll
            for (int u = 0; u < LB; ++u) {
                const int c = chunk[(wave * LB + u) & 1];
                __builtin_amdgcn_raw_ptr_buffer_load_lds(
                    rb, (lds_ptr)(s + BI * kRow + (wave * LB + u) * 1024), 16,
                    c * 8 < left ? ob + u * kRows * ldb + at + c * 16 : kOut, 0, 0, 0);
            }
        };
        // The step's loads are done (every wave waits for its own) and so are the reads of the other buffer.
        const auto turn = [&] {
            asm volatile("" ::: "memory");
            __builtin_amdgcn_s_waitcnt(0x0070);      // vmcnt(0) lgkmcnt(0)
            __builtin_amdgcn_s_barrier();
            asm volatile("" ::: "memory");
            __builtin_amdgcn_sched_barrier(0);
        };
        issue(s_0, first);
        // past the last step: zeros
#pragma unroll 1
        for (int step = first; step < behind; step += 2) {
            turn();
            issue(s_1, step + 1);
            products(s_0);
            turn();
            issue(s_0, step + 2);
            products(s_1);
        }
        turn();
    }
    join_chains(acc);
    xent_ending<T, WI, WJ, MI, MJ, END>(a, acc[0], i0, j0, part, wi, wj, s_0);
}

// f32.  A step's rows go through registers, are cut into their three parts and lie in LDS part by
// part; the product of the first parts has sums of its own, the five smaller ones theirs, so that few
// of the additions round at the result's size.
//
// An operand may lie with k along its columns (weight for dx, D for dweight): lanes take blocks of
// elements, H along k by four, and write a row's H side by side.
//
// Row r of an operand of B rows has slot r % 4 * (B / 4) + r / 4 of 64 bytes and its chunks turned by r % 4:
// 16 lanes that read rows one behind the other reach different banks, and so do 8 lanes that write
// rows r, r + 4, ..., in either form.
//
// Cutting a step into parts takes the vector units about as long as its products the matrix units: half
// of the eight waves do the one while the others do the other.  A tile of few columns waits for
// memory instead and has two steps on their way.  1024 rows x 20000 x 1024: 250 us (168 TFLOP/s, six times as
// many in bfloat16; the library's f32 product reaches 152); 8 rows x 30000 x 1000 42 to 45 us, 2.8 TB/s.
template <int WI, int WJ, int MI, int MJ, bool AK, bool BK, int END>
__device__ __forceinline__ void xent_product_f32(const GemmArgs& a) {
    constexpr int BI = WI * MI * 32, BJ = WJ * MJ * 32, NW = WI * WJ;
    constexpr int kRow = kDepthF32 * 2, kPart = (BI + BJ) * kRow;
    constexpr int LA = BI / 8 / NW, LB = BJ / 8 / NW, kSets = NW == 8 ? 1 : 2;
    static_assert(!AK || LA == 4, "blocks of four along k");
    static_assert(!BK || (LB == 2 && NW == 8 && BJ == 128), "blocks of two along k");
    __shared__ __attribute__((aligned(16))) char s_0[3 * kPart];
    __shared__ __attribute__((aligned(16))) char s_1[3 * kPart];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int wi = wave / WJ, wj = wave % WJ, hi = lane >> 3, lo = lane & 7;
    int64_t i0, j0;
    int part;
    if (!tile_of<BI, BJ>(a, i0, j0, part)) return;
    const int first = (int)(part * a.per_part), steps = (int)((a.k + kDepthF32 - 1) / kDepthF32);
    const int behind = first + a.per_part < steps ? (int)(first + a.per_part) : steps;
    // load u of a wave: rows q / 4 * 32 + q % 4 + 4 hi with q = wave * L + u, four elements of k from 4 lo;
    // k along the columns: element H hi + u of k (and 16 for the other half of the waves), rows 32 t + 4 lo
    const auto row_at = [&](const Operand& o, int64_t from, int most, int q) {      // past the last as that
        const int r = q / 4 * 32 + q % 4 + 4 * hi, rows = (int)(o.rows - from < most ? o.rows - from : most);
        return o.p + (from + (r < rows ? r : rows - 1)) * o.ld;
    };
    const char* at_a[AK ? 1 : LA];
    const char* at_b[BK ? 1 : LB];
    if constexpr (!AK) {
#pragma unroll
        for (int u = 0; u < LA; ++u) at_a[u] = row_at(a.A, i0, BI, wave * LA + u);
    }
    if constexpr (!BK) {
#pragma unroll
        for (int u = 0; u < LB; ++u) at_b[u] = row_at(a.B, j0, BJ, wave * LB + u);
    }
    const int64_t col_a = i0 + wave * 32 + 4 * lo, col_b = j0 + wave / 2 * 32 + 4 * lo;
    const int in_a = 4 * hi, in_b = (wave & 1) * 16 + 2 * hi;
    u32x4 ga[kSets][LA], gb[kSets][LB];
    // nearly every step is whole, and its vectors need no care (8 x 30000 x 1000 50 -> 42 us, 600 rows 265 ->
    // 242; with k along the columns nothing gained)
    const auto whole = [&](int step) {
        return !AK && !BK && step < behind && (int64_t)(step + 1) * kDepthF32 <= a.k;
    };
    const auto load_k = [&](const Operand& o, int64_t col, int64_t k) {
        const int64_t row = k < a.k ? k : a.k - 1;
        return load_row(reinterpret_cast<const float*>(o.p + row * o.ld), col < o.rows ? col : o.rows, o.rows);
    };
    const auto fetch_as = [&](auto as, int set, int step) {
        constexpr bool W = decltype(as)::value;
        const int64_t k = (int64_t)step * kDepthF32;
#pragma unroll
        for (int u = 0; u < LA; ++u) {
            if constexpr (AK)
                ga[set][u] = load_k(a.A, col_a, k + in_a + u);
            else
                ga[set][u] = fetch_vec<W>(reinterpret_cast<const float*>(at_a[u]), k + 4 * lo, a.k);
        }
#pragma unroll
        for (int u = 0; u < LB; ++u) {
            if constexpr (BK)
                gb[set][u] = load_k(a.B, col_b, k + in_b + u);
            else
                gb[set][u] = fetch_vec<W>(reinterpret_cast<const float*>(at_b[u]), k + 4 * lo, a.k);
        }
    };
    const auto fetch = [&](int set, int step) {
        if (whole(step))
            fetch_as(Whole{}, set, step);
        else
            fetch_as(Partial{}, set, step);
    };
    const auto put_row = [&](auto as, char* s, int rows, int q, u32x4 raw, int64_t k) {
        const u32x4 r = settle_vec<decltype(as)::value, float>(raw, k, a.k);
        uint32_t p[3], h[3];
        parts_of(r[0], r[1], p);
        parts_of(r[2], r[3], h);
        char* at = s + (q % 4 * (rows / 4) + q / 4 * 8 + hi) * kRow + ((lo >> 1) ^ (q & 3)) * 16 + (lo & 1) * 8;
#pragma unroll
        for (int n = 0; n < 3; ++n) *reinterpret_cast<u32x2*>(at + n * kPart) = u32x2{p[n], h[n]};
    };
    const auto put_as = [&](auto as, char* s, int set, int step) {      // past the last step: zeros
        constexpr bool W = decltype(as)::value;
        const int64_t k = W || step < behind ? (int64_t)step * kDepthF32 : a.k;
        if constexpr (AK) {
            u32x4 r[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                r[u] = settle<float>(ga[set][u], col_a < a.A.rows ? col_a : a.A.rows, a.A.rows);
                if (k + in_a + u >= a.k) r[u] = u32x4{0, 0, 0, 0};
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint32_t p[3], h[3];
                parts_of(r[0][i], r[1][i], p);
                parts_of(r[2][i], r[3][i], h);
                char* at = s + (i * (BI / 4) + wave * 8 + lo) * kRow + ((hi >> 1) ^ i) * 16 + (hi & 1) * 8;
#pragma unroll
                for (int n = 0; n < 3; ++n) *reinterpret_cast<u32x2*>(at + n * kPart) = u32x2{p[n], h[n]};
            }
        } else {
#pragma unroll
            for (int u = 0; u < LA; ++u) put_row(as, s, BI, wave * LA + u, ga[set][u], k + 4 * lo);
        }
        if constexpr (BK) {
            u32x4 r[2];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                r[u] = settle<float>(gb[set][u], col_b < a.B.rows ? col_b : a.B.rows, a.B.rows);
                if (k + in_b + u >= a.k) r[u] = u32x4{0, 0, 0, 0};
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint32_t p[3];
                parts_of(r[0][i], r[1][i], p);
                char* at = s + (BI + i * (BJ / 4) + wave / 2 * 8 + lo) * kRow + ((in_b >> 3) ^ i) * 16 + (hi & 3) * 4;
#pragma unroll
                for (int n = 0; n < 3; ++n) *reinterpret_cast<uint32_t*>(at + n * kPart) = p[n];
            }
        } else {
#pragma unroll
            for (int u = 0; u < LB; ++u) put_row(as, s + BI * kRow, BJ, wave * LB + u, gb[set][u], k + 4 * lo);
        }
    };
    const auto put = [&](char* s, int set, int step) {
        if (whole(step))
            put_as(Whole{}, s, set, step);
        else
            put_as(Partial{}, s, set, step);
    };
    constexpr int kChains = chains_of<MI, MJ>(kDepthF32);
    f32x16 acc[kChains][MI][MJ] = {}, small[MI][MJ] = {};
    const auto products = [&](const char* s) {
        const char* pa = s + ((lane & 3) * (BI / 4) + wi * MI * 8 + (lane & 31) / 4) * kRow;
        const char* pb = s + (BI + (lane & 3) * (BJ / 4) + wj * MJ * 8 + (lane & 31) / 4) * kRow;
#pragma unroll
        for (int kk = 0; kk < kDepthF32 / 16; ++kk) {
            const int slot = ((kk * 2 + (lane >> 5)) ^ (lane & 3)) * 16;
            u32x4 av[3][MI], bv[3][MJ];
#pragma unroll
            for (int n = 0; n < 3; ++n) {
#pragma unroll
                for (int i = 0; i < MI; ++i)
                    av[n][i] = *reinterpret_cast<const u32x4*>(pa + n * kPart + i * 8 * kRow + slot);
#pragma unroll
                for (int j = 0; j < MJ; ++j)
                    bv[n][j] = *reinterpret_cast<const u32x4*>(pb + n * kPart + j * 8 * kRow + slot);
            }
#pragma unroll
            for (int i = 0; i < MI; ++i)
#pragma unroll
                for (int j = 0; j < MJ; ++j) {
                    acc[kk % kChains][i][j] = mma(av[0][i], bv[0][j], acc[kk % kChains][i][j], __bf16{});
                    small[i][j] = mma(av[2][i], bv[0][j], small[i][j], __bf16{});
                    small[i][j] = mma(av[1][i], bv[1][j], small[i][j], __bf16{});
                    small[i][j] = mma(av[0][i], bv[2][j], small[i][j], __bf16{});
                    small[i][j] = mma(av[1][i], bv[0][j], small[i][j], __bf16{});
                    small[i][j] = mma(av[0][i], bv[1][j], small[i][j], __bf16{});
                }
        }
    };
    const bool early = NW == 8 && wave < 4;      // of the two waves of a SIMD one
    const auto one = [&](const char* now, char* next, int set, int step) {
        if (early) {
            put(next, set, step + 1);
            fetch(set, step + 1 + kSets);
        }
        products(now);
        if (!early) {
            put(next, set, step + 1);
            fetch(set, step + 1 + kSets);
        }
        __syncthreads();
    };
    fetch(0, first);
    put(s_0, 0, first);
    fetch(1 % kSets, first + 1);
    if constexpr (kSets == 2) fetch(0, first + 2);
    __syncthreads();
#pragma unroll 1
    for (int step = first; step < behind; step += 2) {
        one(s_0, s_1, 1 % kSets, step);
        one(s_1, s_0, 0, step + 1);
    }
    join_chains(acc);
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < MJ; ++j) acc[0][i][j] += small[i][j];
    xent_ending<float, WI, WJ, MI, MJ, END>(a, acc[0], i0, j0, part, wi, wj, s_0);
}

// (The kernel's body is a device function: it uses types that the host's compiler pass lacks.)
template <typename T, int WI, int WJ, int MI, int MJ, bool STAGED, int END>
__global__ __launch_bounds__(WI * WJ * 64) void k_xent_product(GemmArgs a) {
    if constexpr (sizeof(T) == 4)
        xent_product_f32<WI, WJ, MI, MJ, END == kDx, END == kDw, END>(a);
    else
        xent_product<T, WI, WJ, MI, MJ, STAGED, END>(a);
}

// ---------------------------------------------------------------- operands laid out

// rows of d elements -> d rows of `wide` (the number of rows rounded up), ld apart, zeros behind and
// for the rows that have no target in [0, vocab) (targets NULL: none); f32: times the row's dloss
template <typename T>
__global__ __launch_bounds__(256) void k_xent_transpose(const T* src, int64_t stride, int64_t rows,
                                                        int64_t d, int64_t wide, int64_t ld, T* dst,
                                                        const int64_t* targets, int64_t vocab,
                                                        const float* dloss) {
    constexpr int kSide = 64;
    __shared__ T s[kSide][kSide + 2];
    const int64_t r0 = (int64_t)blockIdx.x * kSide, c0 = (int64_t)blockIdx.y * kSide;
    constexpr int kPer = kSide / kVec<T>;      // vectors of a row
    u32x4 raw[kSide * kPer / 256];
#pragma unroll
    for (int u = 0; u < kSide * kPer / 256; ++u) {
        const int n = threadIdx.x + u * 256;
        const int64_t r = r0 + n / kPer < rows ? r0 + n / kPer : rows - 1;
        raw[u] = load_row(src + r * stride, c0 + n % kPer * kVec<T>, d);
    }
#pragma unroll
    for (int u = 0; u < kSide * kPer / 256; ++u) {
        const int n = threadIdx.x + u * 256, c = n % kPer * kVec<T>;
        const int64_t r = r0 + n / kPer;
        bool kept = r < rows;
        if (kept && targets) kept = targets[r] >= 0 && targets[r] < vocab;
        const u32x4 w = settle<T>(raw[u], c0 + c, d);
        const float f = sizeof(T) == 4 && kept ? dloss[r] : 1.0f;
#pragma unroll
        for (int i = 0; i < kVec<T>; ++i) {
            if constexpr (sizeof(T) == 4)
                s[c + i][n / kPer] = kept ? __uint_as_float(w[i]) * f : 0.0f;
            else
                s[c + i][n / kPer] =
                    __builtin_bit_cast(T, (uint16_t)(kept ? w[i / 2] >> (16 * (i & 1)) : 0));
        }
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < kSide * kPer / 256; ++u) {
        const int n = threadIdx.x + u * 256, c = n / kPer, r = n % kPer * kVec<T>;
        if (c0 + c >= d || r0 + r >= wide) continue;
        u32x4 w;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (sizeof(T) == 4)
                w[i] = __float_as_uint(s[c][r + i]);
            else
                w[i] = __builtin_bit_cast(uint16_t, s[c][r + 2 * i]) |
                       (uint32_t)__builtin_bit_cast(uint16_t, s[c][r + 2 * i + 1]) << 16;
        }
        *reinterpret_cast<u32x4*>(dst + (c0 + c) * ld + r0 + r) = w;
    }
}

// ---------------------------------------------------------------- rows' results

// A row's tiles joined: a wave a row, lanes the tiles l, l + 64, ... in that order.
__global__ __launch_bounds__(256) void k_xent_rows(const u32x2* stats, const float* hit,
                                                   const int64_t* targets, int64_t rows,
                                                   int64_t tiles, int64_t vocab, float* loss,
                                                   float* lse) {
    const int lane = threadIdx.x & 63;
    for (int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); row < rows;
         row += (int64_t)gridDim.x * 4) {
        float top = -INFINITY, sum = 0.0f;
#pragma unroll 4
        for (int64_t t = lane; t < tiles; t += 64) {
            const u32x2 one = stats[row * tiles + t];
            const float m = __uint_as_float(one[0]), s = __uint_as_float(one[1]);
            const float both = fmaxf(top, m), at = both > -INFINITY ? both : 0.0f;
            sum = sum * exp_fast(top - at) + s * exp_fast(m - at);
            top = both;
        }
        const float most = wave_max(top), at = most > -INFINITY ? most : 0.0f;
        const float total = wave_pw(sum * exp_fast(top - at));
        if (lane == 0) {
            const int64_t target = targets[row];
            const float log_total = logf(total);
            const bool none = total == 0.0f;      // every logit is -infinity
            lse[row] = none ? -INFINITY : most + log_total;
            loss[row] = target < 0 || target >= vocab ? 0.0f
                        : none                        ? INFINITY
                                                      : log_total + (most - hit[row]);
        }
    }
}

__global__ __launch_bounds__(256) void k_xent_zero(uint16_t* p, int64_t n) {
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256)
        p[i] = 0;
}

// the largest |dloss| of the rows that count (f16); infinite where one is NaN, so that dweight is NaN
__global__ __launch_bounds__(1024) void k_xent_unit(const float* dloss, const int64_t* targets,
                                                    int64_t rows, int64_t vocab, float* unit) {
    __shared__ float s[16];
    float m = 0.0f;
    for (int64_t r = threadIdx.x; r < rows; r += 1024)
        if (targets[r] >= 0 && targets[r] < vocab) m = fmaxf(m, dloss[r] != dloss[r] ? INFINITY : fabsf(dloss[r]));
    m = wave_max(m);
    if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = m;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < 16; ++w) m = fmaxf(m, s[w]);
        *unit = m;
    }
}

// dx of the parts' sums: parts added in their order, times scale and the row's dloss
template <typename T>
__global__ __launch_bounds__(256) void k_xent_dx(const float* sums, int64_t parts, int64_t rows,
                                                 int64_t d, int64_t ld, const int64_t* targets,
                                                 int64_t vocab, const float* dloss, float scale,
                                                 T* dx) {
    const int64_t per = ld / 4, total = rows * per;
    for (int64_t n = (int64_t)blockIdx.x * 256 + threadIdx.x; n < total; n += (int64_t)gridDim.x * 256) {
        const int64_t row = n / per, c = n % per * 4;
        f32x4 v = *reinterpret_cast<const f32x4*>(sums + row * ld + c);
#pragma unroll 8
        for (int64_t p = 1; p < parts; ++p)
            v += *reinterpret_cast<const f32x4*>(sums + (p * rows + row) * ld + c);
        const int64_t target = targets[row];
        const bool scored = target >= 0 && target < vocab;
        const float f = scored ? scale * dloss[row] / kUnit<T> : 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (c + i < d) dx[row * d + c + i] = scored ? (T)(v[i] * f) : (T)0.0f;
    }
}

// ---------------------------------------------------------------- launches

unsigned lanes_grid(int64_t items) {
    const int64_t g = cdiv(items, 256);
    return (unsigned)(g < 1 ? 1 : g < 65536 ? g : 65536);
}

template <typename T, int WI, int WJ, int MI, int MJ, bool STAGED, int END>
void product_as(GemmArgs a, int parts, hipStream_t s) {
    constexpr int64_t BI = WI * MI * 32, BJ = WJ * MJ * 32;
    a.ni = cdiv(a.A.rows, BI);
    a.nj = cdiv(a.B.rows, BJ);
    a.parts = parts;
    a.per_part = cdiv(cdiv(a.k, sizeof(T) == 4 ? kDepthF32 : kDepth), parts);
    k_xent_product<T, WI, WJ, MI, MJ, STAGED, END>
        <<<dim3((unsigned)(cdiv(a.ni * a.nj * parts, 8) * 8)), dim3(WI * WJ * 64), 0, s>>>(a);
}

// Columns (rows of x) of a tile.  Up to 64 rows 32 (with 64 entries): such tiles are many and wait for memory
// together, and dx takes weight as it lies.  bf16, 32768 entries x 4096: 1 row 45 us, in tiles of 256 x 128
// 63; 64 rows 55 and 74; 128 rows 92 and 83; 96 rows of 100000 x 1000 70 and 51; forward and backward of 64
// rows x 32768 x 2048 140 and 241, f32 407 and 517.
// More rows: the width whose rounds of workgroups (256 at a time with 256 entries, or 512 with 128) cost
// least, a tile about its width and 120 more.  bf16, 32768 entries x 4096, in widths of 128, 192 and 256: 129
// rows 70, 90, 96 us; 300 rows 130, 96, 102; 600 rows 191, 173, 190; 4096 rows x 65536 x 2048 both ways 5.05,
// 4.69, 4.05 ms.  f32, whose parts take three times the room, 128 (with 256 entries).
int tile_columns(int64_t rows, int64_t vocab, bool f32) {
    if (rows <= 64) return 32;
    if (f32) return 128;
    int best = 0;
    int64_t least = 0;
    for (const int w : {128, 192, 256}) {
        const int64_t cost = cdiv(cdiv(vocab, 256) * cdiv(rows, w), 256) * (w + 120);
        if (best == 0 || cost <= least) {
            best = w;
            least = cost;
        }
    }
    return best;
}

// Rows (vocabulary entries) of such a tile.  Width 128 with 128 of them, two workgroups a unit: 96 rows x 32768 x
// 4096 bf16 68 us, with 256 81; 128 rows x 8000 47 and 57.  The rule does not look at d: with five steps of k
// the larger tile would be the better one (128 rows x 100001 x 257 42 us, with 256 36).
int64_t tile_rows(int columns, bool f32) { return columns == 32 ? 64 : columns == 128 && !f32 ? 128 : 256; }

template <typename T, bool STAGED, int END>
void product_of(const GemmArgs& a, int columns, int parts, hipStream_t s) {
    if constexpr (sizeof(T) == 4 || END != kDx) {
        if (columns == 32) return product_as<T, 2, 1, 1, 1, STAGED, END>(a, parts, s);
    }
    if constexpr (sizeof(T) == 2) {
        if (columns == 256) return product_as<T, 2, 4, 4, 2, STAGED, END>(a, parts, s);
        if (columns == 192) return product_as<T, 4, 2, 2, 3, STAGED, END>(a, parts, s);
    }
    if constexpr (sizeof(T) == 2)
        product_as<T, 2, 2, 2, 2, STAGED, END>(a, parts, s);
    else
        product_as<T, 4, 2, 2, 2, STAGED, END>(a, parts, s);
}

template <typename T, int END>
void product(const GemmArgs& a, int columns, int parts, bool lies, hipStream_t s) {
    static const char* const names[] = {"k_xent_stats", "k_xent_logits", "k_xent_dx", "k_xent_dweight"};
    KernelTimer kt(names[END], s);
    constexpr bool f32 = sizeof(T) == 4;
    if constexpr (END == kDw) {      // columns are vocabulary entries, of which there are many
        if constexpr (f32)
            product_as<T, 4, 2, 2, 2, false, END>(a, parts, s);
        else
            product_as<T, 2, 4, 4, 2, false, END>(a, parts, s);
    } else {
        if constexpr (!f32 && END == kDx) {
            if (columns == 32) return product_as<T, 2, 1, 1, 1, true, END>(a, parts, s);
        } else if constexpr (!f32) {
            if (!lies) return product_of<T, true, END>(a, columns, parts, s);
        }
        product_of<T, false, END>(a, columns, parts, s);
    }
}

struct XentPlan {
    int64_t piece;
    int64_t wide_r;              // rows rounded up: zeros behind them
    int64_t ld_v, ld_r;          // rows of a piece and of the rows, in elements
    int columns;                 // of a tile
    int64_t parts, dx_ld, tile_i, tiles;
    int64_t wt_rows;             // weight transposed for dx: its d rows, 0: read as it lies
};

// Vocabulary entries of a piece: D of a piece takes about kPieceCells elements (kPieceMin a row where that
// is more), in 16-bit types twice.
XentPlan xent_plan(int64_t rows, int64_t vocab, int64_t d, det_dtype dtype) {
    XentPlan p;
    int64_t piece = kPieceCells / (rows > 0 ? rows : 1) / kPieceUnit * kPieceUnit;
    piece = piece < kPieceMin ? kPieceMin : piece > kPieceMax ? kPieceMax : piece;
    p.piece = piece < vocab ? piece : vocab;
    p.wide_r = up(rows, 32);      // what the narrowest tile writes of D's columns
    // rows a power of two apart would meet in the same channels of the memory
    const auto apart = [](int64_t n) { return n % 512 == 0 ? n + kDepth : n; };
    p.ld_v = apart(up(p.piece, kDepth));
    p.ld_r = apart(p.wide_r);
    p.dx_ld = up(d, 4);
    const int columns = tile_columns(rows, vocab, dtype == DET_F32);
    p.columns = columns;
    p.tile_i = tile_rows(columns, dtype == DET_F32);
    p.wt_rows = dtype == DET_F32 || columns == 32 ? 0 : d;
    p.tiles = cdiv(vocab, p.tile_i);
    // workgroups that share dx's sum over a piece where its tiles are few
    const int64_t tiles = cdiv(d, p.tile_i) * cdiv(rows, columns);
    // (256 of them run at a time, of the narrow tiles 1024)
    p.parts = (columns == 32 ? 1024 : p.tile_i == 128 ? 512 : 256) / tiles;
    const int64_t steps = cdiv(p.piece, dtype == DET_F32 ? kDepthF32 : kDepth);
    if (p.parts > cdiv(steps, 8)) p.parts = cdiv(steps, 8);
    if (p.parts < 1) p.parts = 1;
    return p;
}

struct XentLayout {
    size_t stats, hit, xt, wt, d, dt, sums, unit, total;
};

XentLayout xent_layout(int64_t rows, int64_t vocab, int64_t d, det_dtype dtype, bool back) {
    const XentPlan p = xent_plan(rows, vocab, d, dtype);
    const int64_t n = (int64_t)lm_size(dtype);
    XentLayout L = {};
    size_t o = 0;
    const auto take = [&](size_t bytes) {
        const size_t at = o;
        o += round_up(bytes > 0 ? bytes : 1, 256);
        return at;
    };
    if (!back) {
        L.stats = take((size_t)rows * p.tiles * 8);
        L.hit = take((size_t)rows * 4);
    } else {
        L.xt = take((size_t)d * p.ld_r * n);
        L.wt = take((size_t)p.wt_rows * p.ld_v * n);
        L.d = take((size_t)rows * p.ld_v * n);
        if (n == 2) L.dt = take((size_t)p.piece * p.ld_r * n);
        L.sums = take((size_t)p.parts * rows * p.dx_ld * 4);
        L.unit = take(4);
    }
    L.total = o;
    return L;
}

// whether a 16-bit operand's rows can go straight to LDS (a tile's 256 rows within 2^30 bytes)
bool lies_on_16(const void* p, int64_t stride, int64_t d) {
    return d % 8 == 0 && stride % 8 == 0 && stride <= (1 << 21) && reinterpret_cast<uintptr_t>(p) % 16 == 0;
}

template <typename T>
det_status xent_typed(const XentCall& c, char* ws, hipStream_t s) {
    const T* x = static_cast<const T*>(c.x);
    const T* w = static_cast<const T*>(c.weight);
    const bool lies = lies_on_16(x, c.x_stride, c.d) && lies_on_16(w, c.w_stride, c.d);
    const XentPlan p = xent_plan(c.rows, c.vocab, c.d, c.dtype);
    const XentLayout L = xent_layout(c.rows, c.vocab, c.d, c.dtype, false);
    GemmArgs a = {};
    a.B = Operand{reinterpret_cast<const char*>(x), c.rows, c.x_stride * (int64_t)sizeof(T)};
    a.k = c.d;
    a.scale = c.scale;
    a.targets = c.targets;
    a.vocab = c.vocab;
    a.stats = reinterpret_cast<u32x2*>(ws + L.stats);
    a.hit = reinterpret_cast<float*>(ws + L.hit);
    // one piece, up to what a grid holds
    const int64_t most = up(cdiv((int64_t)1 << 28, up(c.rows, kPieceUnit)), kPieceUnit) * kPieceUnit;
    const int64_t piece = c.vocab < most ? c.vocab : most;
    a.tiles = p.tiles;
    for (int64_t v0 = 0; v0 < c.vocab; v0 += piece) {
        const int64_t n = c.vocab - v0 < piece ? c.vocab - v0 : piece;
        a.A = Operand{reinterpret_cast<const char*>(w + v0 * c.w_stride), n, c.w_stride * (int64_t)sizeof(T)};
        a.v0 = v0;
        product<T, kStats>(a, p.columns, 1, lies, s);
        a.tile0 += cdiv(n, p.tile_i);
    }
    det_status st = launch_status();
    if (st != DET_SUCCESS) return st;
    KernelTimer kt("k_xent_rows", s);
    int64_t g = cdiv(c.rows, 4);
    if (g > 65536) g = 65536;
    k_xent_rows<<<dim3((unsigned)g), dim3(256), 0, s>>>(a.stats, a.hit, c.targets, c.rows, a.tiles,
                                                        c.vocab, c.loss, c.lse);
    return launch_status();
}

template <typename T>
det_status xent_back_typed(const XentBackCall& c, char* ws, hipStream_t s) {
    constexpr int64_t es = sizeof(T);
    const T* x = static_cast<const T*>(c.x);
    const T* w = static_cast<const T*>(c.weight);
    const bool lies = lies_on_16(x, c.x_stride, c.d) && lies_on_16(w, c.w_stride, c.d);
    const XentPlan p = xent_plan(c.rows, c.vocab, c.d, c.dtype);
    const XentLayout L = xent_layout(c.rows, c.vocab, c.d, c.dtype, true);
    float* unit = reinterpret_cast<float*>(ws + L.unit);
    if constexpr (__is_same(T, _Float16)) {
        KernelTimer kt("k_xent_unit", s);
        k_xent_unit<<<dim3(1), dim3(1024), 0, s>>>(c.dloss, c.targets, c.rows, c.vocab, unit);
    }
    T* xt = reinterpret_cast<T*>(ws + L.xt);
    {
        KernelTimer kt("k_xent_transpose", s);
        k_xent_transpose<T><<<dim3((unsigned)cdiv(p.wide_r, 64), (unsigned)cdiv(c.d, 64)), dim3(256), 0, s>>>(
            x, c.x_stride, c.rows, c.d, p.wide_r, p.ld_r, xt, c.targets, c.vocab, c.dloss);
    }
    for (int64_t v0 = 0; v0 < c.vocab; v0 += p.piece) {
        const int64_t n = c.vocab - v0 < p.piece ? c.vocab - v0 : p.piece, wide = up(n, kDepth);
        const T* rows = w + v0 * c.w_stride;
        GemmArgs a = {};
        a.scale = c.scale;
        a.targets = c.targets;
        a.vocab = c.vocab;
        a.v0 = v0;
        a.lse = c.lse;
        a.dloss = c.dloss;
        a.unit = unit;
        // D of the piece
        a.A = Operand{reinterpret_cast<const char*>(rows), n, c.w_stride * es};
        a.B = Operand{reinterpret_cast<const char*>(x), c.rows, c.x_stride * es};
        a.k = c.d;
        a.d = ws + L.d;
        a.dt = ws + L.dt;
        a.d_ld = p.ld_v * es;
        a.dt_ld = p.ld_r * es;
        a.rows_up = p.wide_r;
        a.piece_up = wide;
        product<T, kLogits>(a, p.columns, 1, lies, s);
        // dx += D weight
        GemmArgs b = a;
        b.out = ws + L.sums;
        b.out_ld = p.dx_ld;
        b.add = v0 > 0;
        b.B = Operand{ws + L.d, c.rows, a.d_ld};
        if (p.wt_rows == 0) {
            b.A = Operand{reinterpret_cast<const char*>(rows), c.d, c.w_stride * es};
            b.k = n;
        } else {
            T* wt = reinterpret_cast<T*>(ws + L.wt);
            KernelTimer kt("k_xent_transpose", s);
            k_xent_transpose<T><<<dim3((unsigned)(wide / 64), (unsigned)cdiv(c.d, 64)), dim3(256), 0, s>>>(
                rows, c.w_stride, n, c.d, wide, p.ld_v, wt, nullptr, 1, nullptr);
            b.A = Operand{ws + L.wt, c.d, p.ld_v * es};
            b.k = wide;
        }
        product<T, kDx>(b, p.columns, (int)p.parts, true, s);
        // dweight of the piece
        b.A = Operand{ws + L.xt, c.d, p.ld_r * es};
        b.B = es == 4 ? Operand{ws + L.d, n, a.d_ld} : Operand{ws + L.dt, n, a.dt_ld};
        b.k = es == 4 ? c.rows : p.wide_r;
        b.out = static_cast<T*>(c.dweight) + v0 * c.d;
        b.out_ld = c.d;
        product<T, kDw>(b, p.columns, 1, true, s);
        const det_status st = launch_status();
        if (st != DET_SUCCESS) return st;
    }
    KernelTimer kt("k_xent_dx_rows", s);
    k_xent_dx<T><<<dim3(lanes_grid(c.rows * (p.dx_ld / 4))), dim3(256), 0, s>>>(
        reinterpret_cast<const float*>(ws + L.sums), p.parts, c.rows, c.d, p.dx_ld, c.targets, c.vocab,
        c.dloss, c.scale, static_cast<T*>(c.dx));
    return launch_status();
}

}  // namespace

size_t xent_workspace(int64_t rows, int64_t vocab, int64_t d, det_dtype dtype) {
    return rows > 0 && vocab > 0 && d > 0 ? xent_layout(rows, vocab, d, dtype, false).total : 256;
}

size_t xent_backward_workspace(int64_t rows, int64_t vocab, int64_t d, det_dtype dtype) {
    return rows > 0 && vocab > 0 && d > 0 ? xent_layout(rows, vocab, d, dtype, true).total : 256;
}

det_status xent_launch(const XentCall& c, void* ws, hipStream_t s) {
    char* w = static_cast<char*>(ws);
    switch (c.dtype) {
        case DET_F32: return xent_typed<float>(c, w, s);
        case DET_F16: return xent_typed<_Float16>(c, w, s);
        default: return xent_typed<__bf16>(c, w, s);
    }
}

det_status xent_backward_launch(const XentBackCall& c, void* ws, hipStream_t s) {
    char* w = static_cast<char*>(ws);
    if (c.rows == 0) {      // no rows: dweight is 0
        const int64_t n = c.vocab * c.d * (int64_t)lm_size(c.dtype) / 2;
        KernelTimer kt("k_xent_zero", s);
        k_xent_zero<<<dim3(lanes_grid(n)), dim3(256), 0, s>>>(static_cast<uint16_t*>(c.dweight), n);
        return launch_status();
    }
    switch (c.dtype) {
        case DET_F32: return xent_back_typed<float>(c, w, s);
        case DET_F16: return xent_back_typed<_Float16>(c, w, s);
        default: return xent_back_typed<__bf16>(c, w, s);
    }
}

}  // namespace det
