// lm_device.h -- device helpers of the language-model operators: 8-element vectors of the three
// storage types, their conversion to and from f32, and fixed-order reductions over a wave.
//
// Every lane owns 8 consecutive elements at a time, whatever the type (16 bytes of f16 or bf16,
// two 16-byte loads of f32), so which lane sums which element depends on the element's position
// alone.  The vectors are declared with the element's alignment: gfx950 takes 16-byte global
// loads and stores at any address, so rows of odd length and views with an offset run the same
// code and the same order as aligned ones.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "det_device.h"

namespace det {

constexpr int kVec = 8;   // elements a lane loads or stores at a time

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef u32x4 u32x4_a2 __attribute__((aligned(2)));
typedef f32x4 f32x4_a4 __attribute__((aligned(4)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

// 8 elements as they lie in memory
template <typename T>
struct Raw8 {
    u32x4 a;
};
template <>
struct Raw8<float> {
    f32x4 a, b;
};

// ONCE: past the caches, for data that is read once and would push out what the caches hold
template <bool ONCE = false, typename T>
__device__ __forceinline__ Raw8<T> load8(const T* p) {
    Raw8<T> r;
    if constexpr (sizeof(T) == 4) {
        const f32x4_a4* q = reinterpret_cast<const f32x4_a4*>(p);
        const f32x4_a4* q1 = reinterpret_cast<const f32x4_a4*>(p + 4);
        if constexpr (ONCE) {
            r.a = __builtin_nontemporal_load(q);
            r.b = __builtin_nontemporal_load(q1);
        } else {
            r.a = *q;
            r.b = *q1;
        }
    } else {
        const u32x4_a2* q = reinterpret_cast<const u32x4_a2*>(p);
        if constexpr (ONCE)
            r.a = __builtin_nontemporal_load(q);
        else
            r.a = *q;
    }
    return r;
}

template <typename T>
__device__ __forceinline__ void store8(T* p, const Raw8<T>& r) {
    if constexpr (sizeof(T) == 4) {
        *reinterpret_cast<f32x4_a4*>(p) = r.a;
        *reinterpret_cast<f32x4_a4*>(p + 4) = r.b;
    } else {
        *reinterpret_cast<u32x4_a2*>(p) = r.a;
    }
}

template <typename T>
__device__ __forceinline__ void unpack8(const Raw8<T>& r, float (&v)[kVec]) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[i] = r.a[i];
            v[4 + i] = r.b[i];
        }
    } else if constexpr (__is_same(T, _Float16)) {
        const f16x8 h = __builtin_bit_cast(f16x8, r.a);
#pragma unroll
        for (int i = 0; i < kVec; ++i) v[i] = (float)h[i];
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(r.a[i] << 16);
            v[2 * i + 1] = __uint_as_float(r.a[i] & 0xFFFF0000u);
        }
    }
}

// one rounding to nearest even
template <typename T>
__device__ __forceinline__ Raw8<T> pack8(const float (&v)[kVec]) {
    Raw8<T> r;
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            r.a[i] = v[i];
            r.b[i] = v[4 + i];
        }
    } else if constexpr (__is_same(T, _Float16)) {
        f16x8 h;
#pragma unroll
        for (int i = 0; i < kVec; ++i) h[i] = (_Float16)v[i];
        r.a = __builtin_bit_cast(u32x4, h);
    } else {
        bf16x8 h;
#pragma unroll
        for (int i = 0; i < kVec; ++i) h[i] = (__bf16)v[i];
        r.a = __builtin_bit_cast(u32x4, h);
    }
    return r;
}

// The first n (at most 8) elements at p, `fill` behind them.  n < 1 reads nothing.
template <typename T>
__device__ __forceinline__ void load_tail(const T* p, int64_t n, float fill, float (&v)[kVec]) {
#pragma unroll
    for (int i = 0; i < kVec; ++i) v[i] = i < n ? (float)p[i] : fill;
}

template <typename T>
__device__ __forceinline__ void store_tail(T* p, int64_t n, const float (&v)[kVec]) {
#pragma unroll
    for (int i = 0; i < kVec; ++i)
        if (i < n) p[i] = (T)v[i];
}

// 8 elements of which n lie inside the row (unpacked, `fill` behind them)
template <bool ONCE = false, typename T>
__device__ __forceinline__ void read8(const T* p, int64_t n, float fill, float (&v)[kVec]) {
    if (n >= kVec)
        unpack8<T>(load8<ONCE>(p), v);
    else
        load_tail(p, n, fill, v);
}

// the same as it lies in memory, zeros behind them
template <bool ONCE = false, typename T>
__device__ __forceinline__ Raw8<T> read_raw8(const T* p, int64_t n) {
    if (n >= kVec) return load8<ONCE>(p);
    float v[kVec];
    load_tail(p, n, 0.0f, v);
    return pack8<T>(v);
}

template <typename T>
__device__ __forceinline__ void write8(T* p, int64_t n, const float (&v)[kVec]) {
    if (n >= kVec)
        store8<T>(p, pack8<T>(v));
    else
        store_tail(p, n, v);
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

// e^x with the hardware's 2^x (about 1 ulp; results below 2^-126 become 0)
__device__ __forceinline__ float exp_fast(float x) { return __builtin_amdgcn_exp2f(x * kLog2e); }

}  // namespace det
