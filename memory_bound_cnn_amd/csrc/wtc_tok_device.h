// Device helpers of the token operators: 16-byte rows of float32 or bfloat16
// elements to and from float registers, and sums over groups of lanes.
#pragma once

#include <hip/hip_runtime.h>

#include "wtc_numeric.h"

namespace wtc {

typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));   // 16 bytes at any element address

// Elements in 16 bytes of a storage type (bfloat16 is held as its bits).
template <typename T>
constexpr int kVec = 16 / (int)sizeof(T);

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(uint16_t v) { return __builtin_bit_cast(float, (uint32_t)v << 16); }
template <typename T>
__device__ __forceinline__ T from_f32(float v) {
    if constexpr (sizeof(T) == 2)
        return bf16_rne(v);
    else
        return v;
}

// 16 bytes of elements as they lie in memory: half the registers of their
// float32 values when they are bfloat16, for loads that are on their way.
template <typename T>
struct Raw {
    u32x4_any u;
};
template <typename T>
__device__ __forceinline__ void unpack(const Raw<T>& r, float (&v)[kVec<T>]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t e = r.u[i];   // a value of its own: a vector's element is no object to cast the bits of
        if constexpr (sizeof(T) == 2) {
            v[2 * i] = __builtin_bit_cast(float, e << 16);
            v[2 * i + 1] = __builtin_bit_cast(float, e & 0xFFFF0000u);
        } else {
            v[i] = __builtin_bit_cast(float, e);
        }
    }
}

// 16 bytes at any element address: gfx950 reads and writes them with one
// instruction whatever their alignment.
template <typename T>
__device__ __forceinline__ void load16(const T* p, float (&v)[kVec<T>]) {
    unpack(Raw<T>{*reinterpret_cast<const u32x4_any*>(p)}, v);
}

template <typename T>
__device__ __forceinline__ void store16(T* p, const float (&v)[kVec<T>]) {
    u32x4_any u;
    if constexpr (sizeof(T) == 2) {
#pragma unroll
        for (int i = 0; i < 4; ++i) u[i] = bf16x2_rne(v[2 * i], v[2 * i + 1]);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) u[i] = __builtin_bit_cast(uint32_t, v[i]);
    }
    *reinterpret_cast<u32x4_any*>(p) = u;
}

// The first n (0 .. kVec) elements; the others are zero, and not touched in memory.
template <typename T>
__device__ __forceinline__ Raw<T> load_raw(const T* p, int n) {
    if (n >= kVec<T>) return {*reinterpret_cast<const u32x4_any*>(p)};
    Raw<T> r = {{0u, 0u, 0u, 0u}};
#pragma unroll
    for (int i = 0; i < kVec<T>; ++i)
        if (i < n) {
            if constexpr (sizeof(T) == 2)
                r.u[i / 2] |= (uint32_t)p[i] << (16 * (i % 2));
            else
                r.u[i] = __builtin_bit_cast(uint32_t, p[i]);
        }
    return r;
}
template <typename T>
__device__ __forceinline__ void load_part(const T* p, int n, float (&v)[kVec<T>]) {
    if (n >= kVec<T>) {
        load16(p, v);
    } else {
#pragma unroll
        for (int i = 0; i < kVec<T>; ++i) v[i] = i < n ? to_f32(p[i]) : 0.f;
    }
}
template <typename T>
__device__ __forceinline__ void store_part(T* p, int n, const float (&v)[kVec<T>]) {
    if (n >= kVec<T>) {
        store16(p, v);
    } else {
#pragma unroll
        for (int i = 0; i < kVec<T>; ++i)
            if (i < n) p[i] = from_f32<T>(v[i]);
    }
}

// What a value becomes when it is stored.
template <typename T>
__device__ __forceinline__ float as_stored(float v) {
    return to_f32(from_f32<T>(v));
}

}  // namespace wtc
