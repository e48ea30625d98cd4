// norm.hip -- root-mean-square norm of rows, with the residual's addition before it, 8-bit
// output with scales behind it, and its backward pass.
//
// Mathematics, per row of d elements, everything between the load and the last rounding in f32:
//   h = x + residual;  rstd = 1 / sqrt(sum(h^2) / d + eps);  y = h * rstd * weight
//   8 bits: m = max |y| of a group (at least 2^-100); code = e4m3(y * (448 / m)); scale = m / 448
//   dx = rstd * (dy w - xhat * sum(dy w xhat) / d) + dh,  xhat = h * rstd;  dweight = sum of
//   dy * xhat over the rows.
//
// Order: lane t of the row's team holds elements V (t + j * team) .. + V for j = 0, 1, ... (V = 8,
// 4 of f32); it adds its own in that order, the wave adds its lanes by the adjacent-lanes tree, and the wave
// sums are added in wave order.  The team's size depends on d alone, so a row's bits depend
// neither on the other rows nor on their number.  dweight: a team's strip of rows in ascending order,
// the strips of a workgroup's teams in theirs, then the workgroups (k_col_sums); the strip length
// depends on (rows, d, dtype) alone.
#include "det_internal.h"
#include "lm_device.h"

namespace det {
namespace {

constexpr float kE4m3Max = 448.0f;
constexpr float kTinyMax = 0x1p-100f;

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

template <int TEAM>
__device__ __forceinline__ uint32_t team_max(uint32_t v, uint32_t* slots) {
    v = wave_max(v);
    if constexpr (TEAM > 64) {
        if ((threadIdx.x & 63) == 0) slots[threadIdx.x % TEAM >> 6] = v;
        __syncthreads();
        v = slots[0];
#pragma unroll
        for (int w = 1; w < TEAM / 64; ++w) v = umax(v, slots[w]);
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

// Largest |y| of a vector as its bits: they order like the magnitudes, and a NaN's lie above
// infinity's, so a NaN reaches its group's scale.
template <int N>
__device__ __forceinline__ uint32_t max_bits(const float (&y)[N]) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) m = umax(m, __float_as_uint(y[i]) & 0x7FFFFFFFu);
    return m;
}

template <int N>
__device__ __forceinline__ void store_codes(uint8_t* p, int64_t n, const float (&y)[N], float f) {
    uint32_t code[N / 4];
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
        int c = __builtin_amdgcn_cvt_pk_fp8_f32(y[4 * i] * f, y[4 * i + 1] * f, 0, false);
        c = __builtin_amdgcn_cvt_pk_fp8_f32(y[4 * i + 2] * f, y[4 * i + 3] * f, c, true);
        code[i] = (uint32_t)c;
    }
    if (n >= N) {
        typedef uint32_t codes __attribute__((ext_vector_type(N / 4), aligned(1)));
        codes v;
#pragma unroll
        for (int i = 0; i < N / 4; ++i) v[i] = code[i];
        *reinterpret_cast<codes*>(p) = v;
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (i < n) p[i] = (uint8_t)(code[i / 4] >> (8 * (i & 3)));
    }
}

struct NormArgs {
    const void* x;
    const void* res;      // NULL: none
    const void* w;
    void* h;              // written when res is given
    void* y;              // of the input's type, or codes
    float* scales;
    float* rstd;          // NULL: not written
    int64_t x_stride, res_stride, rows, d;
    int64_t groups;       // scales a row
    int group_log2;       // 8 bits: 5, 6, 7, or 0 for the row
    float len, eps;       // d
};

// y or codes of one vector; m: the row's largest |y| bits where the group is the row
template <typename T, bool Q8>
__device__ __forceinline__ void put(const NormArgs& a, int64_t row, int64_t c, int64_t n,
                                    const float (&y)[kVec<T>], uint32_t m) {
    if constexpr (!Q8) {
        if (n > 0) write_vec(static_cast<T*>(a.y) + row * a.d + c, n, y);
    } else {
        if (a.group_log2) {
            m = max_bits(y);      // every lane of the wave takes part; lanes past the row hold 0
            m = umax(m, xor_partner<1>(m));
            m = umax(m, xor_partner<2>(m));
            const int lanes = (1 << a.group_log2) / kVec<T>;      // 4 or more
            if (lanes >= 8) m = umax(m, xor_partner<4>(m));
            if (lanes >= 16) m = umax(m, xor_partner<8>(m));
            if (lanes >= 32) m = umax(m, xor_partner<16>(m));
        }
        const float top = __uint_as_float(umax(m, __float_as_uint(kTinyMax)));
        if (n > 0) {
            store_codes(static_cast<uint8_t*>(a.y) + row * a.d + c, n, y, kE4m3Max / top);
            const int64_t g = a.group_log2 ? c >> a.group_log2 : 0;
            if (g << a.group_log2 == c) a.scales[row * a.groups + g] = top / kE4m3Max;
        }
    }
}

// One row per team, the row in registers: NV vectors a lane.  Bound by HBM: every element is
// read once and written once.  8192 x 8192 bf16 with residual: 79 us (6.8 TB/s), with 8-bit codes
// 76 us (6.2 TB/s); one row of 4096 2.6 us.  Rows that start off 16 bytes cost more: 8192 x 5001
// f16 64 us (5.1 TB/s), 8192 x 5000 55 us.
template <typename T, int TEAM, int NV, bool RES, bool Q8, bool ONCE>
__global__ __launch_bounds__(Team<TEAM>::kBlock) void k_rms_norm(NormArgs a) {
    constexpr int kRows = Team<TEAM>::kRows, kWaves = Team<TEAM>::kWaves;
    constexpr bool kWeightAhead = NV * kVec<T> <= 16;      // registers for it
    __shared__ float s_sum[kRows][kWaves];
    __shared__ uint32_t s_max[kRows][kWaves];
    const int team = threadIdx.x / TEAM, t = threadIdx.x % TEAM;
    for (int64_t first = (int64_t)blockIdx.x * kRows; first < a.rows;
         first += (int64_t)gridDim.x * kRows) {
    const bool live = first + team < a.rows;
    const int64_t row = live ? first + team : a.rows - 1;   // a spare team repeats the last row, unwritten
    const T* x = static_cast<const T*>(a.x) + row * a.x_stride;
    const T* res = static_cast<const T*>(a.res) + (RES ? row * a.res_stride : 0);
    const T* w = static_cast<const T*>(a.w);

    u32x4 raw[NV], raw_res[NV], raw_w[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int64_t c = (int64_t)kVec<T> * (t + j * TEAM);
        raw[j] = load_row<ONCE>(x, c, a.d);
        if constexpr (RES) raw_res[j] = load_row<ONCE>(res, c, a.d);
    }
    if constexpr (kWeightAhead) {
#pragma unroll
        for (int j = 0; j < NV; ++j) raw_w[j] = load_row(w, (int64_t)kVec<T> * (t + j * TEAM), a.d);
    }
    float h[NV][kVec<T>];
    float sum = 0.0f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int64_t c = (int64_t)kVec<T> * (t + j * TEAM);
        unpack<T>(settle<T>(raw[j], c, a.d), h[j]);
        if constexpr (RES) {
            float r[kVec<T>];
            unpack<T>(settle<T>(raw_res[j], c, a.d), r);
#pragma unroll
            for (int i = 0; i < kVec<T>; ++i) h[j][i] += r[i];
            if (live && a.d > c) write_vec(static_cast<T*>(a.h) + row * a.d + c, a.d - c, h[j]);
        }
#pragma unroll
        for (int i = 0; i < kVec<T>; ++i) sum = fmaf(h[j][i], h[j][i], sum);
    }
    sum = team_sum<TEAM>(sum, s_sum[team % kRows]);
    const float rstd = inv_sqrt(sum / a.len + a.eps);
    if (a.rstd && live && t == 0) a.rstd[row] = rstd;

    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int64_t c = (int64_t)kVec<T> * (t + j * TEAM);
        float g[kVec<T>];
        if constexpr (!kWeightAhead) raw_w[j] = load_row(w, c, a.d);
        unpack<T>(settle<T>(raw_w[j], c, a.d), g);
#pragma unroll
        for (int i = 0; i < kVec<T>; ++i) h[j][i] = (h[j][i] * rstd) * g[i];
        if constexpr (Q8) m = umax(m, max_bits(h[j]));
    }
    if constexpr (Q8) {
        if (!a.group_log2) m = team_max<TEAM>(m, s_max[team % kRows]);
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int64_t c = (int64_t)kVec<T> * (t + j * TEAM);
        put<T, Q8>(a, row, c, live ? a.d - c : 0, h[j], m);
    }
    if constexpr (TEAM > 64) __syncthreads();      // the LDS slots are written again
    }
}

// Rows longer than the registers hold: the same order in a loop, the row read again for the
// output (and for a whole row's scale).
template <typename T, bool RES, bool Q8>
__global__ __launch_bounds__(1024) void k_rms_norm_long(NormArgs a) {
    constexpr int TEAM = 1024;
    __shared__ float s_sum[16];
    __shared__ uint32_t s_max[16];
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const T* x = static_cast<const T*>(a.x) + row * a.x_stride;
    const T* res = static_cast<const T*>(a.res) + (RES ? row * a.res_stride : 0);
    const T* w = static_cast<const T*>(a.w);
    const int64_t steps = (a.d + TEAM * kVec<T> - 1) / (TEAM * kVec<T>);
    const auto sums = [&](int64_t c, float (&h)[kVec<T>]) {
        read_vec(x + c, a.d - c, 0.0f, h);
        if constexpr (RES) {
            float r[kVec<T>];
            read_vec(res + c, a.d - c, 0.0f, r);
#pragma unroll
            for (int i = 0; i < kVec<T>; ++i) h[i] += r[i];
        }
    };
    float sum = 0.0f;
    for (int64_t j = 0; j < steps; ++j) {
        const int64_t c = kVec<T> * (threadIdx.x + j * TEAM);
        float h[kVec<T>];
        sums(c, h);
#pragma unroll
        for (int i = 0; i < kVec<T>; ++i) sum = fmaf(h[i], h[i], sum);
    }
    sum = team_sum<TEAM>(sum, s_sum);
    const float rstd = inv_sqrt(sum / a.len + a.eps);
    if (a.rstd && threadIdx.x == 0) a.rstd[row] = rstd;
    const auto outputs = [&](int64_t c, float (&h)[kVec<T>], bool last) {
        sums(c, h);
        float g[kVec<T>];
        read_vec(w + c, a.d - c, 0.0f, g);
        if constexpr (RES) {
            // only now: h may be x itself
            if (last && a.d > c) write_vec(static_cast<T*>(a.h) + row * a.d + c, a.d - c, h);
        }
#pragma unroll
        for (int i = 0; i < kVec<T>; ++i) h[i] = (h[i] * rstd) * g[i];
    };
    uint32_t m = 0;
    if constexpr (Q8) {
        if (!a.group_log2) {
            for (int64_t j = 0; j < steps; ++j) {
                float h[kVec<T>];
                outputs(kVec<T> * (threadIdx.x + j * TEAM), h, false);
                m = umax(m, max_bits(h));
            }
            m = team_max<TEAM>(m, s_max);
        }
    }
    for (int64_t j = 0; j < steps; ++j) {
        const int64_t c = kVec<T> * (threadIdx.x + j * TEAM);
        float h[kVec<T>];
        outputs(c, h, true);
        put<T, Q8>(a, row, c, a.d - c, h, m);
    }
    __syncthreads();      // the LDS slots are written again
    }
}

// ---------------------------------------------------------------- backward

struct NormBackArgs {
    const void* dy;
    const void* h;
    const void* w;
    const void* dh;       // NULL: none
    const float* rstd;
    void* dx;
    float* part;          // [strips][d], the strips' sums of dy * xhat
    int64_t dy_stride, h_stride, dh_stride, rows, d, strip;
    float len;            // d
};

// Lanes of a team that takes rows of up to d elements in the backward pass: one vector of 8 a lane
// to 512 elements, then two (11093 rows without dh, f32: 518 elements 19 us, 31 with 256 lanes of
// one; 2560 elements 65 us, 78 with 512 of one), 1024 lanes of one and two past 4096.
constexpr int back_team(int64_t d) {
    return d <= 1024 ? 64 : d <= 2048 ? 128 : d <= 4096 ? 256 : 1024;
}
// rows that a workgroup of such teams holds at a time
constexpr int back_rows(int64_t d) { return back_team(d) < 256 ? 256 / back_team(d) : 1; }

// One row's vectors of a lane as they lie in memory
template <typename T, int NV>
struct BackRow {
    u32x4 h[NV], dy[NV], dh[NV];
    float rstd;
};

// A team walks its strip of rows and keeps the strip's column sums in registers; the next row's
// loads are in flight while this one's sum goes round the team (16 elements of f32 a lane leave no
// registers for that).  With 1024 lanes of 16 elements the column sums are kept in LDS: 2048 rows
// of 16384 bf16 take 58 us so, 98 with them in registers (spilled).  The teams of a workgroup join
// their sums.  Bound by HBM: 16384 x 4096 bf16 with dh 98 us with k_col_sums (5.5 TB/s), 116
// without the loads ahead and past the caches.
template <typename T, int TEAM, int NV, bool DH, bool ONCE>
__global__ __launch_bounds__(Team<TEAM>::kBlock) void k_rms_norm_backward(NormBackArgs a) {
    constexpr int kRows = Team<TEAM>::kRows, kWaves = Team<TEAM>::kWaves;
    constexpr int kElems = NV * kVec<T>;      // a lane's share of a row
    constexpr bool kAhead = sizeof(T) == 2 || kElems <= 8, kLdsSums = kElems > 8 && TEAM == 1024;
    // kLdsSums: the lane's column sums, [vector][element][lane]
    extern __shared__ float s_cols[];
    __shared__ float s_sum[2][kRows][kWaves];
    __shared__ float s_acc[kRows > 1 ? kRows - 1 : 1][kRows > 1 ? TEAM * NV * kVec<T> : 1];
    const int team = threadIdx.x / TEAM, t = threadIdx.x % TEAM;
    const int64_t strip = (int64_t)blockIdx.x * kRows + team;
    const int64_t begin = strip * a.strip;
    const T* w = static_cast<const T*>(a.w);
    const auto read = [&](int64_t row, BackRow<T, NV>& r) {
        if (row >= a.rows) row = a.rows - 1;
        r.rstd = a.rstd[row];
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int64_t c = (int64_t)kVec<T> * (t + j * TEAM);
            r.h[j] = load_row<ONCE>(static_cast<const T*>(a.h) + row * a.h_stride, c, a.d);
            r.dy[j] = load_row<ONCE>(static_cast<const T*>(a.dy) + row * a.dy_stride, c, a.d);
            if constexpr (DH && kAhead)
                r.dh[j] = load_row<ONCE>(static_cast<const T*>(a.dh) + row * a.dh_stride, c, a.d);
        }
    };
    BackRow<T, NV> cur, next;
    read(begin, cur);
    u32x4 wraw[NV];
    float acc[NV][kVec<T>];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int64_t c = (int64_t)kVec<T> * (t + j * TEAM);
        wraw[j] = settle<T>(load_row(w, c, a.d), c, a.d);
#pragma unroll
        for (int i = 0; i < kVec<T>; ++i) {
            acc[j][i] = 0.0f;
            if constexpr (kLdsSums) s_cols[(j * kVec<T> + i) * TEAM + t] = 0.0f;
        }
    }
    // every team of the workgroup takes the steps of the first one (barriers)
    const int64_t rest = a.rows - (int64_t)blockIdx.x * kRows * a.strip;
    const int64_t steps = rest < a.strip ? rest : a.strip;
    for (int64_t k = 0; k < steps; ++k) {
        const bool live = begin + k < a.rows;
        if constexpr (kAhead) {
            if (k + 1 < steps) read(begin + k + 1, next);
        }
        const float rstd = cur.rstd;
        float h[NV][kVec<T>], dy[NV][kVec<T>];
        float sum = 0.0f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int64_t c = (int64_t)kVec<T> * (t + j * TEAM);
            unpack<T>(settle<T>(cur.h[j], c, a.d), h[j]);
            unpack<T>(settle<T>(cur.dy[j], c, a.d), dy[j]);
            float g[kVec<T>];
            unpack<T>(wraw[j], g);
#pragma unroll
            for (int i = 0; i < kVec<T>; ++i) {
                h[j][i] *= rstd;
                const float p = dy[j][i] * h[j][i];
                if (live) {
                    if constexpr (kLdsSums)
                        s_cols[(j * kVec<T> + i) * TEAM + t] += p;
                    else
                        acc[j][i] += p;
                }
                dy[j][i] *= g[i];
                sum = fmaf(dy[j][i], h[j][i], sum);
            }
        }
        const float mean = team_sum<TEAM>(sum, s_sum[k & 1][team % kRows]) / a.len;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int64_t c = (int64_t)kVec<T> * (t + j * TEAM);
            float o[kVec<T>], e[kVec<T>];
            if constexpr (DH && kAhead) unpack<T>(settle<T>(cur.dh[j], c, a.d), e);
            if constexpr (DH && !kAhead)
                read_vec<ONCE>(static_cast<const T*>(a.dh) + (live ? begin + k : a.rows - 1) * a.dh_stride + c,
                      a.d - c, 0.0f, e);
#pragma unroll
            for (int i = 0; i < kVec<T>; ++i) {
                o[i] = rstd * fmaf(-h[j][i], mean, dy[j][i]);
                if constexpr (DH) o[i] += e[i];
            }
            if (live && a.d > c)
                write_vec(static_cast<T*>(a.dx) + (begin + k) * a.d + c, a.d - c, o);
        }
        if constexpr (kAhead)
            cur = next;
        else if (k + 1 < steps)
            read(begin + k + 1, cur);
    }
    if constexpr (kRows > 1) {
        if (team > 0) {
#pragma unroll
            for (int j = 0; j < NV; ++j)
#pragma unroll
                for (int i = 0; i < kVec<T>; ++i) s_acc[team - 1][kVec<T> * (t + j * TEAM) + i] = acc[j][i];
        }
        __syncthreads();
        if (team > 0) return;
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int i = 0; i < kVec<T>; ++i)
                for (int r = 0; r < kRows - 1; ++r) acc[j][i] += s_acc[r][kVec<T> * (t + j * TEAM) + i];
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int64_t c = (int64_t)kVec<T> * (t + j * TEAM);
        if constexpr (kLdsSums) {
#pragma unroll
            for (int i = 0; i < kVec<T>; ++i) acc[j][i] = s_cols[(j * kVec<T> + i) * TEAM + t];
        }
        if (a.d > c) write_floats(a.part + blockIdx.x * a.d + c, a.d - c, acc[j]);
    }
}

// The dx of rows longer than the registers hold (the row read twice); the strips' sums are
// k_rms_norm_strips's.
template <typename T, bool DH>
__global__ __launch_bounds__(1024) void k_rms_norm_backward_long(NormBackArgs a) {
    constexpr int TEAM = 1024;
    __shared__ float s_sum[16];
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const T* w = static_cast<const T*>(a.w);
    const T* hp = static_cast<const T*>(a.h) + row * a.h_stride;
    const T* dyp = static_cast<const T*>(a.dy) + row * a.dy_stride;
    const T* dhp = static_cast<const T*>(a.dh) + (DH ? row * a.dh_stride : 0);
    const float rstd = a.rstd[row];
    const int64_t steps = (a.d + TEAM * kVec<T> - 1) / (TEAM * kVec<T>);
    const auto both = [&](int64_t c, float (&h)[kVec<T>], float (&dy)[kVec<T>]) {
        float g[kVec<T>];
        read_vec(hp + c, a.d - c, 0.0f, h);
        read_vec(dyp + c, a.d - c, 0.0f, dy);
        read_vec(w + c, a.d - c, 0.0f, g);
#pragma unroll
        for (int i = 0; i < kVec<T>; ++i) {
            h[i] *= rstd;
            dy[i] *= g[i];
        }
    };
    float sum = 0.0f;
    for (int64_t j = 0; j < steps; ++j) {
        float h[kVec<T>], dy[kVec<T>];
        both(kVec<T> * (threadIdx.x + j * TEAM), h, dy);
#pragma unroll
        for (int i = 0; i < kVec<T>; ++i) sum = fmaf(dy[i], h[i], sum);
    }
    const float mean = team_sum<TEAM>(sum, s_sum) / a.len;
    for (int64_t j = 0; j < steps; ++j) {
        const int64_t c = kVec<T> * (threadIdx.x + j * TEAM);
        float h[kVec<T>], dy[kVec<T>], e[kVec<T>];
        both(c, h, dy);
        if constexpr (DH) read_vec(dhp + c, a.d - c, 0.0f, e);
#pragma unroll
        for (int i = 0; i < kVec<T>; ++i) {
            dy[i] = rstd * fmaf(-h[i], mean, dy[i]);
            if constexpr (DH) dy[i] += e[i];
        }
        if (a.d > c) write_vec(static_cast<T*>(a.dx) + row * a.d + c, a.d - c, dy);
    }
    __syncthreads();      // the LDS slots are written again
    }
}

// The strips' sums of dy * xhat for long rows: a lane owns a vector of columns of one strip.
template <typename T>
__global__ __launch_bounds__(256) void k_rms_norm_strips(NormBackArgs a) {
    const int64_t c = kVec<T> * ((int64_t)blockIdx.x * 256 + threadIdx.x);
    const int64_t strip = blockIdx.y, begin = strip * a.strip;
    if (c >= a.d) return;
    const int64_t end = begin + a.strip < a.rows ? begin + a.strip : a.rows;
    float acc[kVec<T>] = {};
    for (int64_t row = begin; row < end; ++row) {
        float h[kVec<T>], dy[kVec<T>];
        read_vec(static_cast<const T*>(a.h) + row * a.h_stride + c, a.d - c, 0.0f, h);
        read_vec(static_cast<const T*>(a.dy) + row * a.dy_stride + c, a.d - c, 0.0f, dy);
        const float rstd = a.rstd[row];
#pragma unroll
        for (int i = 0; i < kVec<T>; ++i) {
            const float p = dy[i] * (h[i] * rstd);
            acc[i] += p;
        }
    }
    write_floats(a.part + strip * a.d + c, a.d - c, acc);
}

// dweight[c] = the strips' sums added: row k of 256 adds strips k, k + 256, ... in that order,
// then the 256 join by a halving tree.  4 lanes x 4 columns a workgroup: 64 bytes of a strip.
constexpr int kSumCols = 16, kSumRows = 256;

template <typename T>
__global__ __launch_bounds__(1024) void k_col_sums(const float* part, int64_t strips, int64_t d,
                                                   T* out) {
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
    if (threadIdx.x < kSumCols && o < d) out[o] = (T)s[0][threadIdx.x];
    if (first + step >= d) return;
    __syncthreads();      // s is written again
    }
}

// ---------------------------------------------------------------- launches

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

constexpr int64_t kRowInRegs = 16384;        // forward: 512 lanes of 32 elements

// NV: 8 elements of a row a lane
template <typename T, int TEAM, int NV, bool RES, bool Q8>
void norm_in_regs(const NormArgs& a, hipStream_t s) {
    const dim3 grid(grid_of((a.rows + Team<TEAM>::kRows - 1) / Team<TEAM>::kRows));
    const dim3 block(Team<TEAM>::kBlock);
    KernelTimer kt("k_rms_norm", s);
    if ((size_t)a.rows * a.d * sizeof(T) * (RES ? 2 : 1) >= kOnceBytes)
        k_rms_norm<T, TEAM, NV * 8 / kVec<T>, RES, Q8, true><<<grid, block, 0, s>>>(a);
    else
        k_rms_norm<T, TEAM, NV * 8 / kVec<T>, RES, Q8, false><<<grid, block, 0, s>>>(a);
}

template <typename T, bool RES, bool Q8>
void norm_sized(const NormArgs& a, hipStream_t s) {
    if (a.d <= 512) {
        norm_in_regs<T, 64, 1, RES, Q8>(a, s);
    } else if (a.d <= 1024) {
        norm_in_regs<T, 64, 2, RES, Q8>(a, s);
    } else if (a.d <= 2048) {
        norm_in_regs<T, 256, 1, RES, Q8>(a, s);
    } else if (a.d <= 4096) {
        norm_in_regs<T, 256, 2, RES, Q8>(a, s);
    } else if (a.d <= 6144) {
        norm_in_regs<T, 256, 3, RES, Q8>(a, s);
    } else if (a.d <= 8192) {
        norm_in_regs<T, 512, 2, RES, Q8>(a, s);
    } else if (a.d <= kRowInRegs) {
        norm_in_regs<T, 512, 4, RES, Q8>(a, s);
    } else {
        KernelTimer kt("k_rms_norm_long", s);
        k_rms_norm_long<T, RES, Q8><<<dim3(grid_of(a.rows)), dim3(1024), 0, s>>>(a);
    }
}

template <typename T>
void norm_typed(const NormArgs& a, bool q8, hipStream_t s) {
    if (a.res) {
        if (q8)
            norm_sized<T, true, true>(a, s);
        else
            norm_sized<T, true, false>(a, s);
    } else {
        if (q8)
            norm_sized<T, false, true>(a, s);
        else
            norm_sized<T, false, false>(a, s);
    }
}

template <typename T, int NV, int TEAM, bool DH>
void back_in_regs(const NormBackArgs& a, int64_t wgs, hipStream_t s) {
    const dim3 grid((unsigned)wgs), block(Team<TEAM>::kBlock);
    const int lds = NV > 1 && TEAM == 1024 ? TEAM * NV * 8 * 4 : 0;      // NV vectors of 8 (f32: twice as many of 4)
    KernelTimer kt("k_rms_norm_backward", s);
    if ((size_t)a.rows * a.d * sizeof(T) * (DH ? 3 : 2) >= kOnceBytes)
        k_rms_norm_backward<T, TEAM, NV * 8 / kVec<T>, DH, true><<<grid, block, lds, s>>>(a);
    else
        k_rms_norm_backward<T, TEAM, NV * 8 / kVec<T>, DH, false><<<grid, block, lds, s>>>(a);
}

template <typename T, bool DH>
void back_sized(const NormBackArgs& a, int64_t sums, hipStream_t s) {
    if (a.d <= 512) {
        back_in_regs<T, 1, back_team(512), DH>(a, sums, s);
    } else if (a.d <= 1024) {
        back_in_regs<T, 2, back_team(1024), DH>(a, sums, s);
    } else if (a.d <= 2048) {
        back_in_regs<T, 2, back_team(2048), DH>(a, sums, s);
    } else if (a.d <= 4096) {
        back_in_regs<T, 2, back_team(4096), DH>(a, sums, s);
    } else if (a.d <= 8192) {
        back_in_regs<T, 1, back_team(8192), DH>(a, sums, s);
    } else if (a.d <= kRowInRegs) {
        back_in_regs<T, 2, back_team(kRowInRegs), DH>(a, sums, s);
    } else {
        {
            KernelTimer kt("k_rms_norm_backward_long", s);
            k_rms_norm_backward_long<T, DH><<<dim3(grid_of(a.rows)), dim3(1024), 0, s>>>(a);
        }
        KernelTimer kt("k_rms_norm_strips", s);
        const dim3 grid((unsigned)((a.d + 256 * kVec<T> - 1) / (256 * kVec<T>)), (unsigned)sums);
        k_rms_norm_strips<T><<<grid, dim3(256), 0, s>>>(a);
    }
}

template <typename T>
det_status back_typed(const NormBackArgs& a, void* dw, hipStream_t s) {
    const int64_t sums = strip_sums(a.rows, a.d, a.strip);
    if (a.rows > 0) {
        if (a.dh)
            back_sized<T, true>(a, sums, s);
        else
            back_sized<T, false>(a, sums, s);
        const det_status st = launch_status();
        if (st != DET_SUCCESS) return st;
    }
    KernelTimer kt("k_col_sums", s);
    k_col_sums<T><<<dim3(grid_of((a.d + kSumCols - 1) / kSumCols)), dim3(1024), 0, s>>>(
        a.part, sums, a.d, static_cast<T*>(dw));
    return launch_status();
}

}  // namespace

size_t norm_backward_workspace(int64_t rows, int64_t d, det_dtype dtype) {
    const int64_t sums = strip_sums(rows, d, strip_rows(rows, d, dtype));
    return round_up((size_t)sums * (size_t)d * sizeof(float), 256) + 256;
}

det_status norm_launch(const NormCall& c, hipStream_t s) {
    const NormArgs a{c.x, c.residual, c.weight, c.h, c.y, c.scales, c.rstd, c.x_stride,
                     c.residual_stride, c.rows, c.d,
                     c.group ? (c.d + c.group - 1) / c.group : 1,
                     c.group ? __builtin_ctz((unsigned)c.group) : 0, (float)c.d, c.eps};
    switch (c.dtype) {
        case DET_F32: norm_typed<float>(a, c.codes, s); break;
        case DET_F16: norm_typed<_Float16>(a, c.codes, s); break;
        default: norm_typed<__bf16>(a, c.codes, s); break;
    }
    return launch_status();
}

det_status norm_backward_launch(const NormBackCall& c, void* ws, hipStream_t s) {
    const NormBackArgs a{c.dy, c.h, c.weight, c.dh, c.rstd, c.dx, static_cast<float*>(ws),
                         c.dy_stride, c.h_stride, c.dh_stride, c.rows, c.d,
                         strip_rows(c.rows, c.d, c.dtype), (float)c.d};
    switch (c.dtype) {
        case DET_F32: return back_typed<float>(a, c.dweight, s);
        case DET_F16: return back_typed<_Float16>(a, c.dweight, s);
        default: return back_typed<__bf16>(a, c.dweight, s);
    }
}

}  // namespace det
