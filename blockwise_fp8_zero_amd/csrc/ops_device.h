// Element types of the operators' tensors: bf16 and fp16 as their 16-bit
// patterns, conversions with one rounding (to nearest, ties to even).
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

namespace bfz {

typedef __bf16 bf16_t;
typedef _Float16 f16_t;

template <class T>
struct Elem {
    static __device__ __forceinline__ float get(T x) { return (float)x; }
    static __device__ __forceinline__ T to(float x) {
        // keeps a product's own binary32 rounding: without it the compiler
        // folds product and conversion to fp16 into one operation
        if constexpr (__is_same(T, f16_t)) __asm__("" : "+v"(x));
        return (T)x;
    }
    // element l of a 16-byte block
    static __device__ __forceinline__ float from_block(const uint32_t __attribute__((ext_vector_type(4))) & raw, int l) {
        if constexpr (sizeof(T) == 4) {
            return __uint_as_float(raw[l]);
        } else {
            const uint16_t h = (uint16_t)(raw[l >> 1] >> (16 * (l & 1)));
            return (float)__builtin_bit_cast(T, h);
        }
    }
};

// 8 consecutive elements at a 16-byte boundary.
template <class T>
__device__ __forceinline__ void load8(const T* p, float (&x)[8]) {
    typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
    if constexpr (sizeof(T) == 4) {
        const u32x4 a = *reinterpret_cast<const u32x4*>(p), b = *(reinterpret_cast<const u32x4*>(p) + 1);
#pragma unroll
        for (int l = 0; l < 4; ++l) {
            x[l] = __uint_as_float(a[l]);
            x[4 + l] = __uint_as_float(b[l]);
        }
    } else {
        const u32x4 a = *reinterpret_cast<const u32x4*>(p);
#pragma unroll
        for (int l = 0; l < 8; ++l) x[l] = Elem<T>::from_block(a, l);
    }
}

template <class T>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    const uint16_t lo = __builtin_bit_cast(uint16_t, Elem<T>::to(a)), hi = __builtin_bit_cast(uint16_t, Elem<T>::to(b));
    return (uint32_t)lo | ((uint32_t)hi << 16);
}

template <class T>
__device__ __forceinline__ void store8(T* p, const float (&x)[8]) {
    typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
    if constexpr (sizeof(T) == 4) {
        u32x4 a, b;
#pragma unroll
        for (int l = 0; l < 4; ++l) {
            a[l] = __float_as_uint(x[l]);
            b[l] = __float_as_uint(x[4 + l]);
        }
        *reinterpret_cast<u32x4*>(p) = a;
        *(reinterpret_cast<u32x4*>(p) + 1) = b;
    } else {
        u32x4 a;
#pragma unroll
        for (int l = 0; l < 4; ++l) a[l] = pack2<T>(x[2 * l], x[2 * l + 1]);
        *reinterpret_cast<u32x4*>(p) = a;
    }
}

// An id outside [0, vocab) names no row: -1.
__device__ __forceinline__ int64_t row_of(const void* ids, int ids64, int64_t i, int64_t vocab) {
    const int64_t id = ids64 ? static_cast<const int64_t*>(ids)[i] : (int64_t) static_cast<const int32_t*>(ids)[i];
    return id >= 0 && id < vocab ? id : -1;
}

}  // namespace bfz
