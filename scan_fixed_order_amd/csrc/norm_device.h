// norm_device.h -- what the root-mean-square norm and layer norm share: teams of lanes that hold a row
// in registers, their sums in a fixed order, and the column sums of the weights' gradients.
#pragma once

#include "det_internal.h"
#include "lm_device.h"

namespace det {
namespace {

// A team of lanes per row, the row in registers between the sum and the output.  Teams by
// measurement (norm_sized): 8192 x 8192 bf16 with codes 76 us with 512 lanes of two vectors, 122
// with 1024 of one; 8192 x 2914 with codes 33 us with 256 of two, 39 with 512 of one, 37 with 128
// of four, 48 with 64 of eight; 8192 x 5000 f16 55 us with 256 of three, 60 with 768 of one; 2048 x
// 16384 with codes 46 us with 512 of four, 58 with 1024 of two.
template <int TEAM>
struct Team {
    static constexpr int kBlock = TEAM < 256 ? 256 : TEAM;
    static constexpr int kRows = kBlock / TEAM;      // rows a workgroup holds at a time
    static constexpr int kWaves = TEAM / 64;
};

// Sum over the team in the fixed order above; uniform over the team.  `slots`: kWaves floats of
// LDS.  Every thread of the workgroup calls it.
template <int TEAM>
__device__ __forceinline__ float team_sum(float v, float* slots) {
    v = wave_pw(v);
    if constexpr (TEAM > 64) {
        if ((threadIdx.x & 63) == 0) slots[threadIdx.x % TEAM >> 6] = v;
        __syncthreads();
        v = slots[0];
#pragma unroll
        for (int w = 1; w < TEAM / 64; ++w) v = v + slots[w];
    }
    return v;
}

// 1 / sqrt(x) within 2^-23: the hardware's estimate and a Newton step, a quarter of the
// instructions of a rounded root and division, which every wave of a row runs.
__device__ __forceinline__ float inv_sqrt(float x) {
    const bool tiny = x < 0x1p-100f;      // the estimate takes no subnormal numbers
    const float s = tiny ? x * 0x1p100f : x;
    const float r = __builtin_amdgcn_rsqf(s);
    const float y = fmaf(0.5f * r, fmaf(-(s * r), r, 1.0f), r);
    const float z = s > 0.0f && s < INFINITY ? y : r;      // 0, infinity and NaN need no step
    return tiny ? z * 0x1p50f : z;
}

// Lanes of a team that takes rows of up to d elements in the backward pass: one vector of 8 a lane
// to 512 elements, then two (11093 rows without dh, f32: 518 elements 19 us, 31 with 256 lanes of
// one; 2560 elements 65 us, 78 with 512 of one), 1024 lanes of one and two past 4096.
constexpr int back_team(int64_t d) {
    return d <= 1024 ? 64 : d <= 2048 ? 128 : d <= 4096 ? 256 : 1024;
}
// rows that a workgroup of such teams holds at a time
constexpr int back_rows(int64_t d) { return back_team(d) < 256 ? 256 / back_team(d) : 1; }

// dweight[c] = the strips' sums added: row k of 256 adds strips k, k + 256, ... in that order,
// then the 256 join by a halving tree.  4 lanes x 4 columns a workgroup: 64 bytes of a strip.
// Columns from first_of_2 on go to out2 (two weights' sums side by side).
constexpr int kSumCols = 16, kSumRows = 256;

template <typename T>
__global__ __launch_bounds__(1024) void k_col_sums(const float* part, int64_t strips, int64_t d,
                                                   T* out, int64_t first_of_2, T* out2) {
    __shared__ float s[kSumRows][kSumCols];
    const int quad = threadIdx.x & 3, grp = threadIdx.x >> 2;
    for (int64_t first = (int64_t)blockIdx.x * kSumCols, step = (int64_t)gridDim.x * kSumCols;;
         first += step) {
    const int64_t c = first + 4 * quad;
    float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (c + 4 <= d) {
#pragma unroll 4
        for (int64_t k = grp; k < strips; k += kSumRows) {
            const f32x4 q = *reinterpret_cast<const f32x4_a4*>(part + k * d + c);
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] += q[i];
        }
    } else {
        for (int64_t k = grp; k < strips; k += kSumRows)
            for (int i = 0; i < 4; ++i)
                if (c + i < d) v[i] += part[k * d + c + i];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) s[grp][4 * quad + i] = v[i];
    __syncthreads();
    const int col = threadIdx.x % kSumCols, row = threadIdx.x / kSumCols;     // 64 rows at a time
    for (int n = kSumRows / 2; n > 0; n >>= 1) {
        for (int r = row; r < n; r += 1024 / kSumCols) s[r][col] += s[r + n][col];
        __syncthreads();
    }
    const int64_t o = first + threadIdx.x;
    if (threadIdx.x < kSumCols && o < d)
        (o < first_of_2 ? out + o : out2 + (o - first_of_2))[0] = (T)s[0][threadIdx.x];
    if (first + step >= d) return;
    __syncthreads();      // s is written again
    }
}

// Rows a strip: 2^17 lanes at work (512 a compute unit), 256 teams at least; at least 4 rows each
// so that the strips' sums stay small beside the rows, or 2 where the next row's loads are not
// ahead: 967 x 1664 f32 with dh 13.5 us so, 19 with 4; 1000 x 4096 bf16 13.6 with 4, 15.3 with 2.
int64_t strip_rows(int64_t rows, int64_t d, det_dtype dtype) {
    const int64_t teams = d <= 4096 ? (1 << 17) / back_team(d) : 256;
    const int64_t r = (rows + teams - 1) / teams;
    const int64_t least = dtype == DET_F32 && d > 512 ? 2 : 4;
    return r < least ? least : r;
}

// strips whose sums reach k_col_sums
int64_t strip_sums(int64_t rows, int64_t d, int64_t strip) {
    const int64_t strips = (rows + strip - 1) / strip;
    return (strips + back_rows(d) - 1) / back_rows(d);
}

// workgroups a launch starts at most (a grid holds fewer than 2^32 threads); each walks the rows,
// or the columns
unsigned grid_of(int64_t wgs) { return (unsigned)(wgs < (1 << 21) ? wgs : (1 << 21)); }

}  // namespace
}  // namespace det
