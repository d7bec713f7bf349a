// E4M3 quantization of groups of values with one scale: the rules of the step's
// tiles, for kernels that quantize as they go.
#pragma once

#include <type_traits>

#include "ops_device.h"

namespace bfz {

// 2^T, the smallest with 448 2^T >= amax, T >= -149 (amax finite, > 0).  With
// amax = f 2^e, f in [0.5, 1), and 448 = 0.875 2^9: T = e - 9, one more where
// f > 0.875.
__device__ __forceinline__ float pow2_scale_of(float amax) {
    const int e = __builtin_amdgcn_frexp_expf(amax);
    const float f = __builtin_amdgcn_frexp_mantf(amax);
    const int T = max(e - 9 + (f > 0.875f ? 1 : 0), -149);
    return __builtin_amdgcn_ldexpf(1.0f, T);
}

// x / by, correctly rounded, from the rounded reciprocal of `by`: see Quotient.
__device__ __forceinline__ float quotient_of(float x, float by, float back) {
    float q = x * back;
    q = __builtin_fmaf(-__builtin_fmaf(q, by, -x), back, q);
    return __builtin_fmaf(-__builtin_fmaf(q, by, -x), back, q);
}

// Quotients x / scale, correctly rounded, from one division for the group: with
// y the rounded reciprocal, q = x y is within two units of the last place, and
// each q - (q scale - x) y, the remainder exact in one fused operation, brings it
// to the correctly rounded one (written so that -0 stays -0).  That holds while nothing leaves the normal
// range, which the scale decides: |x| <= 448 scale (1 + 2^-23), and quotients
// that underflow are far below E4M3's smallest value.  Other scales (below
// 2^-60, above 2^60, infinite or NaN) divide.
struct Quotient {
    float scale, back;
    bool direct;
    __device__ __forceinline__ explicit Quotient(float s) : scale(s), back(1.0f / s), direct(!(s >= 0x1p-60f && s <= 0x1p60f)) {}
    __device__ __forceinline__ float fast(float x) const { return quotient_of(x, scale, back); }
    // kept within +-448, since scales of few bits (subnormal) may lie below
    // amax / 448; a NaN stays one
    __device__ __forceinline__ float slow(float x) const {
        const float q = x / scale;
        return q > 448.0f ? 448.0f : q < -448.0f ? -448.0f : q;
    }
};

// Scale of a group from the largest |x| of its numbers (NaN aside).
__device__ __forceinline__ float scale_of(float amax, bool pow2) {
    if (pow2 && amax > 0.0f && amax < INFINITY) return pow2_scale_of(amax);
    if (__builtin_expect(amax >= 0x1p-60f && amax <= 0x1p100f, 1)) return quotient_of(amax, 448.0f, 1.0f / 448.0f);
    if (amax == 0.0f) return 1.0f;
    const float s = amax / 448.0f;
    return s == 0.0f ? 0x1p-149f : s;
}

// Codes of four values, the first in the lowest byte: to the nearest, ties to
// even (the conversion's own rounding; quotients beyond 448 round to 448 since
// they lie within 2^-23 of it).
__device__ __forceinline__ uint32_t codes_of(float a, float b, float c, float d) {
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
}

// Codes of 8 values of a group.
__device__ __forceinline__ void quantize8(const float (&x)[8], const Quotient& q, uint32_t (&words)[2]) {
    float y[8];
    if (__builtin_expect(q.direct, 0)) {
#pragma unroll
        for (int l = 0; l < 8; ++l) y[l] = q.slow(x[l]);
    } else {
#pragma unroll
        for (int l = 0; l < 8; ++l) y[l] = q.fast(x[l]);
    }
#pragma unroll
    for (int w = 0; w < 2; ++w) words[w] = codes_of(y[4 * w], y[4 * w + 1], y[4 * w + 2], y[4 * w + 3]);
}

// Largest value over 16 lanes that stand in a row, in all of them.
__device__ __forceinline__ float row_max(float x) {
    x = fmaxf(x, __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(x), 0x128, 0xf, 0xf, false)));  // rotated by 8
    x = fmaxf(x, __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(x), 0x124, 0xf, 0xf, false)));
    x = fmaxf(x, __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(x), 0x122, 0xf, 0xf, false)));
    return fmaxf(x, __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(x), 0x121, 0xf, 0xf, false)));
}

// Largest value over a wave, in all its lanes.
__device__ __forceinline__ float wave_max(float x) {
    x = row_max(x);
    const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    x = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
    const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}

// The first `count` of 8 elements, zeros for the others.  Loads of 16 bytes take any
// element's boundary on this hardware (1013 x 1001 floats, element by element, 10 us;
// so 5).
template <class T>
__device__ __forceinline__ void load8_any(const T* p, int count, float (&x)[8]) {
    if (count >= 8) {
        typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
        typedef uint32_t on_words __attribute__((ext_vector_type(4), aligned(4)));
        typedef uint32_t on_halves __attribute__((ext_vector_type(4), aligned(2)));
        typedef std::conditional_t<sizeof(T) == 4, on_words, on_halves> loose;
        const u32x4 a = *reinterpret_cast<const loose*>(p);
        if constexpr (sizeof(T) == 4) {
            const u32x4 b = *(reinterpret_cast<const loose*>(p) + 1);
#pragma unroll
            for (int l = 0; l < 8; ++l) x[l] = __uint_as_float(l < 4 ? a[l & 3] : b[l & 3]);
        } else {
#pragma unroll
            for (int l = 0; l < 8; ++l) x[l] = Elem<T>::from_block(a, l);
        }
        return;
    }
#pragma unroll
    for (int l = 0; l < 8; ++l) x[l] = l < count ? Elem<T>::get(p[l]) : 0.0f;
}

__device__ __forceinline__ float abs_max8(const float (&x)[8]) {
    float a = 0.0f;
#pragma unroll
    for (int l = 0; l < 8; ++l) a = fmaxf(a, fabsf(x[l]));
    return a;
}

}  // namespace bfz
