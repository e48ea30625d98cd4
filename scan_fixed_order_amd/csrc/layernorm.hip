// layernorm.hip -- layer norm of rows, with the residual's addition before it, and its backward
// pass.
//
// Mathematics, per row of d elements, everything between the load and the one rounding in f32:
//   h = x + residual;  mean = sum(h) / d;  rstd = 1 / sqrt(sum((h - mean)^2) / d + eps)
//   y = (h - mean) * rstd * weight + bias
//   dx = rstd * (g - sum(g) / d - xhat * sum(g xhat) / d) + dh,  g = dy weight,  xhat = (h - mean) rstd
//   dweight = sum over the rows of dy * xhat;  dbias = sum over the rows of dy
// The variance is taken about the mean, from the registers, not as a difference of two large sums.
//
// Order: as the root-mean-square norm's (norm.hip): lane t of the row's team holds elements V (t + j
// * team) .. + V for j = 0, 1, ... and adds its own in that order, the wave adds its lanes by the
// adjacent-lanes tree, the wave sums are added in wave order.  The team's size depends on d alone.
// dweight and dbias: a team's strip of rows in ascending order, the strips of a workgroup's teams,
// then the workgroups (k_col_sums); the strip length depends on (rows, d, dtype) alone.
#include "norm_device.h"

namespace det {
namespace {

struct LayerArgs {
    const void* x;
    const void* res;      // NULL: none
    const void* w;
    const void* b;        // NULL: none
    void* h;              // written when res is given
    void* y;
    float* mean;          // NULL: not written
    float* rstd;          // NULL: not written
    int64_t x_stride, res_stride, rows, d;
    float len, eps;       // d
};

// zeros behind the first `rest` elements (the distances of what lies past a row's end)
template <int N>
__device__ __forceinline__ void cut(float (&v)[N], int64_t rest) {
    const int left = rest < 0 ? 0 : rest < N ? (int)rest : N;
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = i < left ? v[i] : 0.0f;
}

// Sums of two values over the team with one barrier.  `slots`: 2 x kWaves floats of LDS.
template <int TEAM>
__device__ __forceinline__ void team_sums(float& u, float& v, float (*slots)[2]) {
    u = wave_pw(u);
    v = wave_pw(v);
    if constexpr (TEAM > 64) {
        if ((threadIdx.x & 63) == 0) {
            slots[threadIdx.x % TEAM >> 6][0] = u;
            slots[threadIdx.x % TEAM >> 6][1] = v;
        }
        __syncthreads();
        u = slots[0][0];
        v = slots[0][1];
#pragma unroll
        for (int w = 1; w < TEAM / 64; ++w) {
            u += slots[w][0];
            v += slots[w][1];
        }
    }
}

// One row per team, the row in registers: NV vectors a lane, between the two sums and the output.
// Bound by HBM, which is read once and written once: 16384 x 4096 bf16 with residual and bias 95 us (537
// MB, 5.6 TB/s), 2048 x 16384 52 (5.2); one row 3 us, a chain of two loads, two sums and a store.  The teams
// are the root-mean-square norm's: fewer lanes with more vectors each lose more loads in flight than
// the second sum's barrier costs.
template <typename T, int TEAM, int NV, bool RES, bool ONCE>
__global__ __launch_bounds__(Team<TEAM>::kBlock) void k_layer_norm(LayerArgs a) {
    constexpr int kRows = Team<TEAM>::kRows, kWaves = Team<TEAM>::kWaves;
    constexpr bool kWeightAhead = NV * kVec<T> <= 16;      // registers for it
    __shared__ float s_sum[2][kRows][kWaves];
    const int team = threadIdx.x / TEAM, t = threadIdx.x % TEAM;
    for (int64_t first = (int64_t)blockIdx.x * kRows; first < a.rows;
         first += (int64_t)gridDim.x * kRows) {
    const bool live = first + team < a.rows;
    const int64_t row = live ? first + team : a.rows - 1;   // a spare team repeats the last row, unwritten
    const T* x = static_cast<const T*>(a.x) + row * a.x_stride;
    const T* res = static_cast<const T*>(a.res) + (RES ? row * a.res_stride : 0);
    const T* w = static_cast<const T*>(a.w);
    const T* b = static_cast<const T*>(a.b);

    u32x4 raw[NV], raw_res[NV], raw_w[NV], raw_b[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int64_t c = (int64_t)kVec<T> * (t + j * TEAM);
        raw[j] = load_row<ONCE>(x, c, a.d);
        if constexpr (RES) raw_res[j] = load_row<ONCE>(res, c, a.d);
    }
    if constexpr (kWeightAhead) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            raw_w[j] = load_row(w, (int64_t)kVec<T> * (t + j * TEAM), a.d);
            raw_b[j] = u32x4{0, 0, 0, 0};
            if (b) raw_b[j] = load_row(b, (int64_t)kVec<T> * (t + j * TEAM), a.d);
        }
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
        for (int i = 0; i < kVec<T>; ++i) sum += h[j][i];
    }
    const float mean = team_sum<TEAM>(sum, s_sum[0][team % kRows]) / a.len;
    float square = 0.0f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int64_t rest = a.d - (int64_t)kVec<T> * (t + j * TEAM);
#pragma unroll
        for (int i = 0; i < kVec<T>; ++i) h[j][i] -= mean;
        if (__any(rest < kVec<T>)) cut(h[j], rest);
#pragma unroll
        for (int i = 0; i < kVec<T>; ++i) square = fmaf(h[j][i], h[j][i], square);
    }
    square = team_sum<TEAM>(square, s_sum[1][team % kRows]);
    const float rstd = inv_sqrt(square / a.len + a.eps);
    if (live && t == 0) {
        if (a.mean) a.mean[row] = mean;
        if (a.rstd) a.rstd[row] = rstd;
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int64_t c = (int64_t)kVec<T> * (t + j * TEAM);
        float g[kVec<T>], o[kVec<T>];
        if constexpr (!kWeightAhead) {
            raw_w[j] = load_row(w, c, a.d);
            raw_b[j] = u32x4{0, 0, 0, 0};
            if (b) raw_b[j] = load_row(b, c, a.d);
        }
        unpack<T>(settle<T>(raw_w[j], c, a.d), g);
        unpack<T>(settle<T>(raw_b[j], c, a.d), o);
#pragma unroll
        for (int i = 0; i < kVec<T>; ++i) h[j][i] = fmaf(h[j][i] * rstd, g[i], o[i]);
        if (live && a.d > c) write_vec(static_cast<T*>(a.y) + row * a.d + c, a.d - c, h[j]);
    }
    if constexpr (TEAM > 64) __syncthreads();      // the LDS slots are written again
    }
}

// Rows longer than the registers hold: the same order in loops, the row read again for the
// variance and for the output (1024 x 32768 bf16 with residual and bias 75 us, 3.6 TB/s of what one pass
// needs; the later reads come from the caches).
template <typename T, bool RES>
__global__ __launch_bounds__(1024) void k_layer_norm_long(LayerArgs a) {
    constexpr int TEAM = 1024;
    __shared__ float s_sum[2][16];
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const T* x = static_cast<const T*>(a.x) + row * a.x_stride;
    const T* res = static_cast<const T*>(a.res) + (RES ? row * a.res_stride : 0);
    const T* w = static_cast<const T*>(a.w);
    const T* b = static_cast<const T*>(a.b);
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
        float h[kVec<T>];
        sums(kVec<T> * (threadIdx.x + j * TEAM), h);
#pragma unroll
        for (int i = 0; i < kVec<T>; ++i) sum += h[i];
    }
    const float mean = team_sum<TEAM>(sum, s_sum[0]) / a.len;
    float square = 0.0f;
    for (int64_t j = 0; j < steps; ++j) {
        const int64_t c = kVec<T> * (threadIdx.x + j * TEAM);
        float h[kVec<T>];
        sums(c, h);
#pragma unroll
        for (int i = 0; i < kVec<T>; ++i) h[i] -= mean;
        if (__any(a.d - c < kVec<T>)) cut(h, a.d - c);
#pragma unroll
        for (int i = 0; i < kVec<T>; ++i) square = fmaf(h[i], h[i], square);
    }
    square = team_sum<TEAM>(square, s_sum[1]);
    const float rstd = inv_sqrt(square / a.len + a.eps);
    if (threadIdx.x == 0) {
        if (a.mean) a.mean[row] = mean;
        if (a.rstd) a.rstd[row] = rstd;
    }
    for (int64_t j = 0; j < steps; ++j) {
        const int64_t c = kVec<T> * (threadIdx.x + j * TEAM);
        float h[kVec<T>], g[kVec<T>], o[kVec<T>] = {};
        sums(c, h);
        read_vec(w + c, a.d - c, 0.0f, g);
        if (b) read_vec(b + c, a.d - c, 0.0f, o);
        if (a.d <= c) continue;
        if constexpr (RES) {
            // only now: h may be x itself
            write_vec(static_cast<T*>(a.h) + row * a.d + c, a.d - c, h);
        }
#pragma unroll
        for (int i = 0; i < kVec<T>; ++i) h[i] = fmaf((h[i] - mean) * rstd, g[i], o[i]);
        write_vec(static_cast<T*>(a.y) + row * a.d + c, a.d - c, h);
    }
    __syncthreads();      // the LDS slots are written again
    }
}

// ---------------------------------------------------------------- backward

struct LayerBackArgs {
    const void* dy;
    const void* h;
    const void* w;
    const void* dh;       // NULL: none
    const float* mean;
    const float* rstd;
    void* dx;
    float* part;          // [strips][width]: the strips' sums of dy * xhat, behind them those of dy
    int64_t dy_stride, h_stride, dh_stride, rows, d, strip, width;
    float len;            // d
};

// One row's vectors of a lane as they lie in memory
template <typename T, int NV>
struct LayerRow {
    u32x4 h[NV], dy[NV], dh[NV];
    float mean, rstd;
};

// A team walks its strip of rows and keeps the strip's column sums in registers (with 1024 lanes of
// 16 elements in LDS); the next row's loads are in flight while this one's sums go round the team.
// The teams of a workgroup join their sums.  Bound by HBM: 16384 x 4096 bf16 with dh, dweight and dbias 88 us
// (537 MB and 17 MB of strips, 6.2 TB/s); 1003 x 5001 f32 15 us, one round of rows a workgroup.  Rows of
// 16384 keep one workgroup of 1024 lanes a unit, whose loads do not cover the sums (2048 rows 89 us, 4.5
// TB/s).
template <typename T, int TEAM, int NV, bool DH, bool BIAS, bool ONCE>
__global__ __launch_bounds__(Team<TEAM>::kBlock) void k_layer_norm_backward(LayerBackArgs a) {
    constexpr int kRows = Team<TEAM>::kRows, kWaves = Team<TEAM>::kWaves;
    constexpr int kElems = NV * kVec<T>;      // a lane's share of a row
    constexpr int kSums = BIAS ? 2 : 1;       // of dy * xhat, of dy
    constexpr bool kAhead = sizeof(T) == 2 || kElems <= 8, kLdsSums = kElems > 8 && TEAM == 1024;
    // kLdsSums: the lane's column sums, [sum][element][lane]
    __shared__ float s_cols[kLdsSums ? kSums * kElems * TEAM : 1];
    __shared__ float s_sum[2][kRows][kWaves][2];
    __shared__ float s_acc[kRows > 1 ? kRows - 1 : 1][kRows > 1 ? kSums * TEAM * kElems : 1];
    const int team = threadIdx.x / TEAM, t = threadIdx.x % TEAM;
    const int64_t strip = (int64_t)blockIdx.x * kRows + team;
    const int64_t begin = strip * a.strip;
    const T* w = static_cast<const T*>(a.w);
    const auto read = [&](int64_t row, LayerRow<T, NV>& r) {
        if (row >= a.rows) row = a.rows - 1;
        r.mean = a.mean[row];
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
    LayerRow<T, NV> cur, next;
    read(begin, cur);
    u32x4 wraw[NV];
    float acc[kSums][kElems];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int64_t c = (int64_t)kVec<T> * (t + j * TEAM);
        wraw[j] = settle<T>(load_row(w, c, a.d), c, a.d);
    }
#pragma unroll
    for (int q = 0; q < kSums; ++q)
#pragma unroll
        for (int i = 0; i < kElems; ++i) {
            acc[q][i] = 0.0f;
            if constexpr (kLdsSums) s_cols[(q * kElems + i) * TEAM + t] = 0.0f;
        }
    // every team of the workgroup takes the steps of the first one (barriers)
    const int64_t rest = a.rows - (int64_t)blockIdx.x * kRows * a.strip;
    const int64_t steps = rest < a.strip ? rest : a.strip;
    for (int64_t k = 0; k < steps; ++k) {
        const bool live = begin + k < a.rows;
        if constexpr (kAhead) {
            if (k + 1 < steps) read(begin + k + 1, next);
        }
        const float rstd = cur.rstd, mean = cur.mean;
        float h[NV][kVec<T>], dy[NV][kVec<T>];
        float sum = 0.0f, inner = 0.0f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int64_t c = (int64_t)kVec<T> * (t + j * TEAM);
            // past the row's end dy and the weight are 0, and so is what they multiply
            unpack<T>(settle<T>(cur.h[j], c, a.d), h[j]);
            unpack<T>(settle<T>(cur.dy[j], c, a.d), dy[j]);
            float g[kVec<T>];
            unpack<T>(wraw[j], g);
#pragma unroll
            for (int i = 0; i < kVec<T>; ++i) {
                h[j][i] = (h[j][i] - mean) * rstd;
                const float p = dy[j][i] * h[j][i];
                if (live) {
                    const int e = j * kVec<T> + i;
                    if constexpr (kLdsSums) {
                        s_cols[e * TEAM + t] += p;
                        if constexpr (BIAS) s_cols[(kElems + e) * TEAM + t] += dy[j][i];
                    } else {
                        acc[0][e] += p;
                        if constexpr (BIAS) acc[kSums - 1][e] += dy[j][i];
                    }
                }
                dy[j][i] *= g[i];
                sum += dy[j][i];
                inner = fmaf(dy[j][i], h[j][i], inner);
            }
        }
        team_sums<TEAM>(sum, inner, s_sum[k & 1][team % kRows]);
        const float off = sum / a.len, along = inner / a.len;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int64_t c = (int64_t)kVec<T> * (t + j * TEAM);
            float o[kVec<T>], e[kVec<T>];
            if constexpr (kLdsSums) {
                // from the words again, which take half of the registers across the sums (the empty asm keeps
                // the compiler from holding the floats all the same, 24 registers of a lane in memory: 106 us)
                asm("" : "+v"(cur.h[j]), "+v"(cur.dy[j]));
                float g[kVec<T>];
                unpack<T>(settle<T>(cur.h[j], c, a.d), h[j]);
                unpack<T>(settle<T>(cur.dy[j], c, a.d), dy[j]);
                unpack<T>(wraw[j], g);
#pragma unroll
                for (int i = 0; i < kVec<T>; ++i) {
                    h[j][i] = (h[j][i] - mean) * rstd;
                    dy[j][i] *= g[i];
                }
            }
            if constexpr (DH && kAhead) unpack<T>(settle<T>(cur.dh[j], c, a.d), e);
            if constexpr (DH && !kAhead)
                read_vec<ONCE>(static_cast<const T*>(a.dh) +
                                   (live ? begin + k : a.rows - 1) * a.dh_stride + c,
                               a.d - c, 0.0f, e);
#pragma unroll
            for (int i = 0; i < kVec<T>; ++i) {
                o[i] = rstd * fmaf(-h[j][i], along, dy[j][i] - off);
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
        // lane by lane: [sum][element][lane]
        if (team > 0) {
#pragma unroll
            for (int q = 0; q < kSums; ++q)
#pragma unroll
                for (int i = 0; i < kElems; ++i) s_acc[team - 1][(q * kElems + i) * TEAM + t] = acc[q][i];
        }
        __syncthreads();
        if (team > 0) return;
#pragma unroll
        for (int q = 0; q < kSums; ++q)
#pragma unroll
            for (int i = 0; i < kElems; ++i)
                for (int r = 0; r < kRows - 1; ++r) acc[q][i] += s_acc[r][(q * kElems + i) * TEAM + t];
    }
#pragma unroll
    for (int q = 0; q < kSums; ++q)
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int64_t c = (int64_t)kVec<T> * (t + j * TEAM);
            float v[kVec<T>];
#pragma unroll
            for (int i = 0; i < kVec<T>; ++i) {
                const int e = j * kVec<T> + i;
                if constexpr (kLdsSums)
                    v[i] = s_cols[(q * kElems + e) * TEAM + t];
                else
                    v[i] = acc[q][e];
            }
            if (a.d > c) write_floats(a.part + blockIdx.x * a.width + q * a.d + c, a.d - c, v);
        }
}

// The dx of rows longer than the registers hold (the row read twice); the strips' sums are
// k_layer_norm_strips's.  (1024 x 32768 bf16, both and the sums: 125 us.)
template <typename T, bool DH>
__global__ __launch_bounds__(1024) void k_layer_norm_backward_long(LayerBackArgs a) {
    constexpr int TEAM = 1024;
    __shared__ float s_sum[16][2];
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const T* w = static_cast<const T*>(a.w);
    const T* hp = static_cast<const T*>(a.h) + row * a.h_stride;
    const T* dyp = static_cast<const T*>(a.dy) + row * a.dy_stride;
    const T* dhp = static_cast<const T*>(a.dh) + (DH ? row * a.dh_stride : 0);
    const float rstd = a.rstd[row], mean = a.mean[row];
    const int64_t steps = (a.d + TEAM * kVec<T> - 1) / (TEAM * kVec<T>);
    const auto both = [&](int64_t c, float (&h)[kVec<T>], float (&dy)[kVec<T>]) {
        float g[kVec<T>];
        read_vec(hp + c, a.d - c, 0.0f, h);
        read_vec(dyp + c, a.d - c, 0.0f, dy);
        read_vec(w + c, a.d - c, 0.0f, g);
#pragma unroll
        for (int i = 0; i < kVec<T>; ++i) {
            h[i] = (h[i] - mean) * rstd;
            dy[i] *= g[i];
        }
    };
    float sum = 0.0f, inner = 0.0f;
    for (int64_t j = 0; j < steps; ++j) {
        float h[kVec<T>], dy[kVec<T>];
        both(kVec<T> * (threadIdx.x + j * TEAM), h, dy);
#pragma unroll
        for (int i = 0; i < kVec<T>; ++i) {
            sum += dy[i];
            inner = fmaf(dy[i], h[i], inner);
        }
    }
    team_sums<TEAM>(sum, inner, s_sum);
    const float off = sum / a.len, along = inner / a.len;
    for (int64_t j = 0; j < steps; ++j) {
        const int64_t c = kVec<T> * (threadIdx.x + j * TEAM);
        float h[kVec<T>], dy[kVec<T>], e[kVec<T>];
        both(c, h, dy);
        if constexpr (DH) read_vec(dhp + c, a.d - c, 0.0f, e);
#pragma unroll
        for (int i = 0; i < kVec<T>; ++i) {
            dy[i] = rstd * fmaf(-h[i], along, dy[i] - off);
            if constexpr (DH) dy[i] += e[i];
        }
        if (a.d > c) write_vec(static_cast<T*>(a.dx) + row * a.d + c, a.d - c, dy);
    }
    __syncthreads();      // the LDS slots are written again
    }
}

// The strips' column sums for long rows: a lane owns a vector of columns of one strip.
template <typename T, bool BIAS>
__global__ __launch_bounds__(256) void k_layer_norm_strips(LayerBackArgs a) {
    const int64_t c = kVec<T> * ((int64_t)blockIdx.x * 256 + threadIdx.x);
    const int64_t strip = blockIdx.y, begin = strip * a.strip;
    if (c >= a.d) return;
    const int64_t end = begin + a.strip < a.rows ? begin + a.strip : a.rows;
    float dw[kVec<T>] = {}, db[kVec<T>] = {};
    for (int64_t row = begin; row < end; ++row) {
        float h[kVec<T>], dy[kVec<T>];
        read_vec(static_cast<const T*>(a.h) + row * a.h_stride + c, a.d - c, 0.0f, h);
        read_vec(static_cast<const T*>(a.dy) + row * a.dy_stride + c, a.d - c, 0.0f, dy);
        const float rstd = a.rstd[row], mean = a.mean[row];
#pragma unroll
        for (int i = 0; i < kVec<T>; ++i) {
            const float p = dy[i] * ((h[i] - mean) * rstd);
            dw[i] += p;
            if constexpr (BIAS) db[i] += dy[i];
        }
    }
    write_floats(a.part + strip * a.width + c, a.d - c, dw);
    if constexpr (BIAS) write_floats(a.part + strip * a.width + a.d + c, a.d - c, db);
}

// ---------------------------------------------------------------- launches

constexpr int64_t kRowInRegs = 16384;        // 512 lanes of 32 elements; backward 1024 of 16

// NV: 8 elements of a row a lane
template <typename T, int TEAM, int NV, bool RES>
void layer_in_regs(const LayerArgs& a, hipStream_t s) {
    const dim3 grid(grid_of((a.rows + Team<TEAM>::kRows - 1) / Team<TEAM>::kRows));
    const dim3 block(Team<TEAM>::kBlock);
    KernelTimer kt("k_layer_norm", s);
    if ((size_t)a.rows * a.d * sizeof(T) * (RES ? 2 : 1) >= kOnceBytes)
        k_layer_norm<T, TEAM, NV * 8 / kVec<T>, RES, true><<<grid, block, 0, s>>>(a);
    else
        k_layer_norm<T, TEAM, NV * 8 / kVec<T>, RES, false><<<grid, block, 0, s>>>(a);
}

// the teams of the root-mean-square norm (norm_sized there)
template <typename T, bool RES>
void layer_sized(const LayerArgs& a, hipStream_t s) {
    if (a.d <= 512) {
        layer_in_regs<T, 64, 1, RES>(a, s);
    } else if (a.d <= 1024) {
        layer_in_regs<T, 64, 2, RES>(a, s);
    } else if (a.d <= 2048) {
        layer_in_regs<T, 256, 1, RES>(a, s);
    } else if (a.d <= 4096) {
        layer_in_regs<T, 256, 2, RES>(a, s);
    } else if (a.d <= 6144) {
        layer_in_regs<T, 256, 3, RES>(a, s);
    } else if (a.d <= 8192) {
        layer_in_regs<T, 512, 2, RES>(a, s);
    } else if (a.d <= kRowInRegs) {
        layer_in_regs<T, 512, 4, RES>(a, s);
    } else {
        KernelTimer kt("k_layer_norm_long", s);
        k_layer_norm_long<T, RES><<<dim3(grid_of(a.rows)), dim3(1024), 0, s>>>(a);
    }
}

template <typename T>
void layer_typed(const LayerArgs& a, hipStream_t s) {
    if (a.res)
        layer_sized<T, true>(a, s);
    else
        layer_sized<T, false>(a, s);
}

template <typename T, int NV, int TEAM, bool DH, bool BIAS>
void layer_back_in_regs(const LayerBackArgs& a, int64_t wgs, hipStream_t s) {
    const dim3 grid((unsigned)wgs), block(Team<TEAM>::kBlock);
    KernelTimer kt("k_layer_norm_backward", s);
    if ((size_t)a.rows * a.d * sizeof(T) * (DH ? 3 : 2) >= kOnceBytes)
        k_layer_norm_backward<T, TEAM, NV * 8 / kVec<T>, DH, BIAS, true><<<grid, block, 0, s>>>(a);
    else
        k_layer_norm_backward<T, TEAM, NV * 8 / kVec<T>, DH, BIAS, false><<<grid, block, 0, s>>>(a);
}

template <typename T, bool DH, bool BIAS>
void layer_back_sized(const LayerBackArgs& a, int64_t sums, hipStream_t s) {
    if (a.d <= 512) {
        layer_back_in_regs<T, 1, back_team(512), DH, BIAS>(a, sums, s);
    } else if (a.d <= 1024) {
        layer_back_in_regs<T, 2, back_team(1024), DH, BIAS>(a, sums, s);
    } else if (a.d <= 2048) {
        layer_back_in_regs<T, 2, back_team(2048), DH, BIAS>(a, sums, s);
    } else if (a.d <= 4096) {
        layer_back_in_regs<T, 2, back_team(4096), DH, BIAS>(a, sums, s);
    } else if (a.d <= 8192) {
        layer_back_in_regs<T, 1, back_team(8192), DH, BIAS>(a, sums, s);
    } else if (a.d <= kRowInRegs) {
        layer_back_in_regs<T, 2, back_team(kRowInRegs), DH, BIAS>(a, sums, s);
    } else {
        {
            KernelTimer kt("k_layer_norm_backward_long", s);
            k_layer_norm_backward_long<T, DH><<<dim3(grid_of(a.rows)), dim3(1024), 0, s>>>(a);
        }
        KernelTimer kt("k_layer_norm_strips", s);
        const dim3 grid((unsigned)((a.d + 256 * kVec<T> - 1) / (256 * kVec<T>)), (unsigned)sums);
        k_layer_norm_strips<T, BIAS><<<grid, dim3(256), 0, s>>>(a);
    }
}

template <typename T>
det_status layer_back_typed(const LayerBackArgs& a, void* dw, void* db, hipStream_t s) {
    const int64_t sums = strip_sums(a.rows, a.d, a.strip);
    if (a.rows > 0) {
        if (a.dh) {
            if (db)
                layer_back_sized<T, true, true>(a, sums, s);
            else
                layer_back_sized<T, true, false>(a, sums, s);
        } else {
            if (db)
                layer_back_sized<T, false, true>(a, sums, s);
            else
                layer_back_sized<T, false, false>(a, sums, s);
        }
        const det_status st = launch_status();
        if (st != DET_SUCCESS) return st;
    }
    KernelTimer kt("k_col_sums", s);
    k_col_sums<T><<<dim3(grid_of((a.width + kSumCols - 1) / kSumCols)), dim3(1024), 0, s>>>(
        a.part, sums, a.width, static_cast<T*>(dw), a.d, static_cast<T*>(db));
    return launch_status();
}

}  // namespace

size_t layer_norm_backward_workspace(int64_t rows, int64_t d, det_dtype dtype) {
    const int64_t sums = strip_sums(rows, d, strip_rows(rows, d, dtype));
    return round_up((size_t)sums * (size_t)d * 2 * sizeof(float), 256) + 256;
}

det_status layer_norm_launch(const LayerCall& c, hipStream_t s) {
    const LayerArgs a{c.x, c.residual, c.weight, c.bias, c.h, c.y, c.mean, c.rstd, c.x_stride,
                      c.residual_stride, c.rows, c.d, (float)c.d, c.eps};
    switch (c.dtype) {
        case DET_F32: layer_typed<float>(a, s); break;
        case DET_F16: layer_typed<_Float16>(a, s); break;
        default: layer_typed<__bf16>(a, s); break;
    }
    return launch_status();
}

det_status layer_norm_backward_launch(const LayerBackCall& c, void* ws, hipStream_t s) {
    const LayerBackArgs a{c.dy, c.h, c.weight, c.dh, c.mean, c.rstd, c.dx, static_cast<float*>(ws),
                          c.dy_stride, c.h_stride, c.dh_stride, c.rows, c.d,
                          strip_rows(c.rows, c.d, c.dtype), c.dbias ? 2 * c.d : c.d, (float)c.d};
    switch (c.dtype) {
        case DET_F32: return layer_back_typed<float>(a, c.dweight, c.dbias, s);
        case DET_F16: return layer_back_typed<_Float16>(a, c.dweight, c.dbias, s);
        default: return layer_back_typed<__bf16>(a, c.dweight, c.dbias, s);
    }
}

}  // namespace det
