// lm_device.h -- device helpers of the language-model operators: 16-byte vectors of the three
// storage types, their conversion to and from f32, and fixed-order reductions over a wave.
//
// Every lane owns 16 bytes of consecutive elements at a time (8 of f16 or bf16, 4 of f32), and
// neighbouring lanes neighbouring vectors, so a wave's load or store covers 1024 bytes without a
// gap, and which lane sums which element depends on the element's position and the type alone.
// (8 elements of f32 a lane, two loads apart by 32 bytes a lane, took 231 us where this takes 192:
// gradient of 8192 x 16385 f32 logits.)  The vectors are declared with the element's alignment:
// gfx950 takes 16-byte global loads and stores at any address, so rows of odd length and views
// with an offset run the same code and the same order as aligned ones.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "det_device.h"

namespace det {

template <typename T>
constexpr int kVec = 16 / sizeof(T);   // elements a lane loads or stores at a time

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef u32x4 u32x4_a2 __attribute__((aligned(2)));
typedef u32x4 u32x4_a4 __attribute__((aligned(4)));
typedef f32x4 f32x4_a4 __attribute__((aligned(4)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

// a vector at any address of an element
template <typename T>
struct VecAt {
    typedef u32x4_a2 type;
};
template <>
struct VecAt<float> {
    typedef u32x4_a4 type;
};

// A vector as it lies in memory.  ONCE: past the caches, for data that is read once and would push
// out what the caches hold.
template <bool ONCE = false, typename T>
__device__ __forceinline__ u32x4 load_vec(const T* p) {
    const auto* q = reinterpret_cast<const typename VecAt<T>::type*>(p);
    if constexpr (ONCE)
        return __builtin_nontemporal_load(q);
    else
        return *q;
}

template <typename T>
__device__ __forceinline__ void store_vec(T* p, u32x4 r) {
    *reinterpret_cast<typename VecAt<T>::type*>(p) = r;
}

template <typename T>
__device__ __forceinline__ void unpack(u32x4 r, float (&v)[kVec<T>]) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = __uint_as_float(r[i]);
    } else if constexpr (__is_same(T, _Float16)) {
        const f16x8 h = __builtin_bit_cast(f16x8, r);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = (float)h[i];
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(r[i] << 16);
            v[2 * i + 1] = __uint_as_float(r[i] & 0xFFFF0000u);
        }
    }
}

// one rounding to nearest even
template <typename T>
__device__ __forceinline__ u32x4 pack(const float (&v)[kVec<T>]) {
    if constexpr (sizeof(T) == 4) {
        return u32x4{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                     __float_as_uint(v[3])};
    } else if constexpr (__is_same(T, _Float16)) {
        f16x8 h;
#pragma unroll
        for (int i = 0; i < 8; ++i) h[i] = (_Float16)v[i];
        return __builtin_bit_cast(u32x4, h);
    } else {
        bf16x8 h;
#pragma unroll
        for (int i = 0; i < 8; ++i) h[i] = (__bf16)v[i];
        return __builtin_bit_cast(u32x4, h);
    }
}

// The first n elements at p, `fill` behind them.  n < 1 reads nothing.
template <typename T>
__device__ __forceinline__ void load_tail(const T* p, int64_t n, float fill, float (&v)[kVec<T>]) {
#pragma unroll
    for (int i = 0; i < kVec<T>; ++i) v[i] = i < n ? (float)p[i] : fill;
}

// a vector of which n elements lie inside the row (unpacked, `fill` behind them)
template <bool ONCE = false, typename T>
__device__ __forceinline__ void read_vec(const T* p, int64_t n, float fill, float (&v)[kVec<T>]) {
    if (n >= kVec<T>)
        unpack<T>(load_vec<ONCE>(p), v);
    else
        load_tail(p, n, fill, v);
}

// the same as it lies in memory, zeros behind them
template <typename T>
__device__ __forceinline__ u32x4 read_raw(const T* p, int64_t n) {
    if (n >= kVec<T>) return load_vec(p);
    float v[kVec<T>];
    load_tail(p, n, 0.0f, v);
    return pack<T>(v);
}

// The vector from element c of a row of d elements, in two steps that keep every lane on one
// path: the load takes the row's last vector where this one reaches past the end, and `settle`,
// at the use, moves its elements to the front and zeros behind them.  (A branch between whole
// and partial vectors makes a wave wait for its loads where it takes them: the norm's backward
// over 8192 x 4992 f16 took 95 us so, over 8192 x 5120, without partial waves, 67.)
template <bool ONCE = false, typename T>
__device__ __forceinline__ u32x4 load_row(const T* row, int64_t c, int64_t d) {
    if (d < kVec<T>) return read_raw(row + c, d - c);
    return load_vec<ONCE>(row + (c + kVec<T> <= d ? c : d - kVec<T>));
}

// (In 32-bit words.  A 64-bit shift whose amount the compiler had put in the last register that a
// wave owns gave wrong elements now and then, in the gradient of f32 logits.)
template <typename T>
__device__ __forceinline__ u32x4 settle(u32x4 r, int64_t c, int64_t d) {
    const int64_t past = c + kVec<T> - d;      // elements past the end
    if (d >= kVec<T> && __any(past > 0)) {
        const uint32_t n = past <= 0 ? 0 : past < kVec<T> ? (uint32_t)past : kVec<T>;
        if constexpr (sizeof(T) == 2) {
            const uint32_t half = n % 2 * 16;
            r = u32x4{__builtin_amdgcn_alignbit(r[1], r[0], half),
                      __builtin_amdgcn_alignbit(r[2], r[1], half),
                      __builtin_amdgcn_alignbit(r[3], r[2], half), r[3] >> half};
        }
        const uint32_t words = sizeof(T) == 2 ? n / 2 : n;
        if (words & 1) r = u32x4{r[1], r[2], r[3], 0};
        if (words & 2) r = u32x4{r[2], r[3], 0, 0};
        if (words & 4) r = u32x4{0, 0, 0, 0};
    }
    return r;
}

template <typename T>
__device__ __forceinline__ void write_vec(T* p, int64_t n, const float (&v)[kVec<T>]) {
    if (n >= kVec<T>) {
        store_vec(p, pack<T>(v));
    } else {
#pragma unroll
        for (int i = 0; i < kVec<T>; ++i)
            if (i < n) p[i] = (T)v[i];
    }
}

// the first n of N floats
template <int N>
__device__ __forceinline__ void write_floats(float* p, int64_t n, const float (&v)[N]) {
    if (n >= N) {
#pragma unroll
        for (int i = 0; i < N; i += 4)
            *reinterpret_cast<f32x4_a4*>(p + i) = f32x4{v[i], v[i + 1], v[i + 2], v[i + 3]};
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (i < n) p[i] = v[i];
    }
}

// ---------------------------------------------------------------- reductions over a wave

// Sums take the adjacent-lanes-first tree of wave_pw; maxima do not depend on the order.
__device__ __forceinline__ float wave_max(float v) {
    v = fmaxf(v, xor_partner<1>(v));
    v = fmaxf(v, xor_partner<2>(v));
    v = fmaxf(v, xor_partner<4>(v));
    v = fmaxf(v, xor_partner<8>(v));
    v = fmaxf(v, xor_partner<16>(v));
    return fmaxf(readlane(v, 0), readlane(v, 32));
}

__device__ __forceinline__ uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }

__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
    v = umax(v, xor_partner<1>(v));
    v = umax(v, xor_partner<2>(v));
    v = umax(v, xor_partner<4>(v));
    v = umax(v, xor_partner<8>(v));
    v = umax(v, xor_partner<16>(v));
    return umax(readlane(v, 0), readlane(v, 32));
}

// orders LDS accesses of one wave's lanes among each other
__device__ __forceinline__ void wave_sync() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

constexpr float kLog2e = 1.4426950408889634f;

// e^x with the hardware's 2^x, off by up to (1 + |x|) 2^-23: the constant and the product are rounded
// to float, which moves the exponent by as much relative to it, and 2^x is good to a last place.
// Results below 2^-126 become 0.
__device__ __forceinline__ float exp_fast(float x) { return __builtin_amdgcn_exp2f(x * kLog2e); }

}  // namespace det
