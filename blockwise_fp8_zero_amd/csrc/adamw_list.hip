// AdamW over many tensors at once, states in 32 or 8 bits.
//
//   m' = b1 m + (1-b1) g,  v' = b2 v + (1-b2) g g
//   p' = p - lr/(1-b1^t) m' / (sqrt(v') / sqrt(1-b2^t) + eps),  p' -= lr wd p'
//
// 8-bit states: E4M3 codes of m and of r = sqrt(v), which has half of v's range of
// exponents, one scale for each 256 elements, made anew from m' and r' in the pass
// that reads the old ones.  r rather than v also keeps a small root away from zero:
// a positive one has a code.
//
// Bound by memory with 32-bit states: 256M elements, f32 parameters and bf16
// gradients, 1.15 ms (6.0 TB/s); with 8-bit ones by memory and the four divisions
// and the root an element has left, 0.69 ms (5.5 TB/s).  Few small tensors: 56 of
// 100 elements 6 us, most of it the launch and fetching code.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "layer_internal.h"
#include "quant_device.h"

#pragma clang fp contract(off)

namespace bfz {
namespace {

constexpr int kThreads = 256;
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// Each byte is touched once: nothing is kept in the caches.
template <class T>
__device__ __forceinline__ T load_stream(const char* p) {
    return __builtin_nontemporal_load(reinterpret_cast<const T*>(p));
}
template <class T>
__device__ __forceinline__ void store_stream(char* p, const T& x) {
    __builtin_nontemporal_store(x, reinterpret_cast<T*>(p));
}

// 4 elements of an array as they lie there, converted only when they are used, so
// that all loads are under way together.
typedef u32x4 Raw;

__device__ __forceinline__ int size_of(int type) { return type == kF32 ? 4 : type == kE4M3 ? 1 : 2; }

__device__ __forceinline__ Raw load_raw(const void* p, int type, int64_t e, int count, bool vec) {
    Raw r = {0u, 0u, 0u, 0u};
    const char* at = static_cast<const char*>(p) + e * size_of(type);
    if (vec && count == 4) {
        if (type == kF32) {
            r = load_stream<u32x4>(at);
        } else if (type == kE4M3) {
            r[0] = load_stream<uint32_t>(at);
        } else {
            const u32x2 x = load_stream<u32x2>(at);
            r[0] = x[0];
            r[1] = x[1];
        }
        return r;
    }
#pragma unroll
    for (int l = 0; l < 4; ++l) {
        if (l >= count) continue;
        if (type == kF32) r[l] = reinterpret_cast<const uint32_t*>(at)[l];
        else if (type == kE4M3) r[0] |= (uint32_t) reinterpret_cast<const uint8_t*>(at)[l] << (8 * l);
        else r[l >> 1] |= (uint32_t) reinterpret_cast<const uint16_t*>(at)[l] << (16 * (l & 1));
    }
    return r;
}

__device__ __forceinline__ void values(const Raw& r, int type, float (&x)[4]) {
#pragma unroll
    for (int l = 0; l < 4; ++l) {
        const uint32_t h = r[l >> 1] >> (16 * (l & 1));
        x[l] = type == kF32 ? __uint_as_float(r[l]) : type == kBF16 ? __uint_as_float(h << 16) : (float)__builtin_bit_cast(f16_t, (uint16_t)h);
    }
}

__device__ __forceinline__ void store_raw(void* p, int type, int64_t e, int count, bool vec, const Raw& r) {
    char* at = static_cast<char*>(p) + e * size_of(type);
    if (vec && count == 4) {
        if (type == kF32) store_stream(at, r);
        else if (type == kE4M3) store_stream(at, (uint32_t)r[0]);
        else store_stream(at, u32x2{r[0], r[1]});
        return;
    }
#pragma unroll
    for (int l = 0; l < 4; ++l) {
        if (l >= count) continue;
        if (type == kF32) reinterpret_cast<uint32_t*>(at)[l] = r[l];
        else if (type == kE4M3) reinterpret_cast<uint8_t*>(at)[l] = (uint8_t)(r[0] >> (8 * l));
        else reinterpret_cast<uint16_t*>(at)[l] = (uint16_t)(r[l >> 1] >> (16 * (l & 1)));
    }
}

__device__ __forceinline__ Raw raw_of(const float (&x)[4], int type) {
    if (type == kF32) return Raw{__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3])};
    if (type == kBF16) return Raw{pack2<bf16_t>(x[0], x[1]), pack2<bf16_t>(x[2], x[3]), 0u, 0u};
    return Raw{pack2<f16_t>(x[0], x[1]), pack2<f16_t>(x[2], x[3]), 0u, 0u};
}

__device__ __forceinline__ void decode(const Raw& r, float scale, float (&x)[4]) {
    x[0] = __builtin_amdgcn_cvt_f32_fp8((int)r[0], 0) * scale;
    x[1] = __builtin_amdgcn_cvt_f32_fp8((int)r[0], 1) * scale;
    x[2] = __builtin_amdgcn_cvt_f32_fp8((int)r[0], 2) * scale;
    x[3] = __builtin_amdgcn_cvt_f32_fp8((int)r[0], 3) * scale;
}

// Codes of a block's values, a wave to a block, and its scale.
__device__ __forceinline__ Raw encode(const float (&x)[4], bool positive, float& scale) {
    scale = scale_of(wave_max(fmaxf(fmaxf(fabsf(x[0]), fabsf(x[1])), fmaxf(fabsf(x[2]), fabsf(x[3])))), false);
    const Quotient q(scale);
    float y[4];
#pragma unroll
    for (int l = 0; l < 4; ++l) y[l] = q.direct ? q.slow(x[l]) : q.fast(x[l]);
    uint32_t w = codes_of(y[0], y[1], y[2], y[3]);
    if (positive && scale < INFINITY) {  // a block with an infinity is NaN, zeros of it times its scale
#pragma unroll
        for (int l = 0; l < 4; ++l)
            if (x[l] > 0.0f && ((w >> (8 * l)) & 0xFFu) == 0u) w |= 1u << (8 * l);
    }
    return Raw{w, 0u, 0u, 0u};
}

__device__ __forceinline__ int find_tensor(const AdamwList& list, uint32_t c) {
    int lo = 0, hi = list.count - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (list.chunk0[mid] <= c) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

__device__ __forceinline__ bool on_fours(const void* p, int type) {
    return (reinterpret_cast<uintptr_t>(p) & (uintptr_t)(4 * size_of(type) - 1)) == 0;
}

// A chunk a workgroup.  A wave takes a state block of 256 elements at a time, 4 a
// lane, so that each load and store is contiguous whatever its type.
constexpr int kPieces = (int)(kAdamwChunk / (4 * kThreads));
static_assert(kStateBlock == 4 * 64 && kPieces * kThreads * 4 == kAdamwChunk, "a wave to a block");

// From element e0 on, a wave's blocks.  kWhole: all of them lie in the tensor, on boundaries of 4 elements.  Without those
// checks, and with the types known, it is a third of the instructions: 256M
// elements with f32 parameters, bf16 gradients and 8-bit states 690 us, with them
// 797.
template <bool kCodes, bool kWhole>
__device__ __forceinline__ void adamw_chunk(const AdamwList& list, const StepScalars& s, int k, int64_t e0, int pt, int gt) {
    constexpr int kMany = kWhole ? kPieces : 1;
    const int64_t n = list.n[k];
    constexpr int st = kCodes ? kE4M3 : kF32;
    void* param = list.param[k];
    const void* grad = list.grad[k];
    void* m = list.m[k];
    void* v = list.v[k];
    const bool vec = kWhole || (on_fours(param, pt) && on_fours(grad, gt) && on_fours(m, st) && on_fours(v, st));
    const float factor = s.grad_scale ? *s.grad_scale : 1.0f;
    // sbc2 = sqrt(1 - beta2^t) lies between 2^-27 and 1 (beta2 is a double)
    // and a root between 2^-75 and 2^64: their quotients need no scaling, only
    // infinities and zeros putting right
    const float back = 1.0f / s.sbc2;
    const int lane = threadIdx.x & 63;
    const int64_t b0 = e0 + 4 * lane;
    Raw rp[kMany], rg[kMany], rm[kMany], rv[kMany];
    float ms[kMany], vs[kMany];
#pragma unroll
    for (int i = 0; i < kMany; ++i) {
        const int64_t e = b0 + i * kStateBlock, left = n - e;
        const int count = kWhole || left >= 4 ? 4 : left <= 0 ? 0 : (int)left;
        rp[i] = load_raw(param, pt, e, count, vec);
        rg[i] = load_raw(grad, gt, e, count, vec);
        rm[i] = load_raw(m, st, e, count, vec);
        rv[i] = load_raw(v, st, e, count, vec);
        ms[i] = vs[i] = 0.0f;
        if (kCodes && count > 0) {
            ms[i] = list.m_scale[k][e / kStateBlock];
            vs[i] = list.v_scale[k][e / kStateBlock];
        }
    }
#pragma unroll
    for (int i = 0; i < kMany; ++i) {
        const int64_t e = b0 + i * kStateBlock, left = n - e;
        const int count = kWhole || left >= 4 ? 4 : left <= 0 ? 0 : (int)left;
        float p[4], g[4], mm[4], vv[4], root[4];
        values(rp[i], pt, p);
        values(rg[i], gt, g);
        if constexpr (kCodes) {
            decode(rm[i], ms[i], mm);
            decode(rv[i], vs[i], vv);
        } else {
            values(rm[i], kF32, mm);
            values(rv[i], kF32, vv);
        }
#pragma unroll
        for (int l = 0; l < 4; ++l) {
            if constexpr (kCodes) vv[l] *= vv[l];
            const float x = s.grad_scale ? g[l] * factor : g[l];
            mm[l] = s.b1 * mm[l] + s.c1 * x;
            vv[l] = s.b2 * vv[l] + s.c2 * (x * x);
            root[l] = sqrtf(vv[l]);
            const float den = __builtin_amdgcn_div_fixupf(quotient_of(root[l], s.sbc2, back), s.sbc2, root[l]) + s.eps;
            float pp = p[l] - s.step_size * (mm[l] / den);
            if (s.has_decay) pp = pp - s.decay * pp;
            p[l] = pp;
            if (kCodes && l >= count) mm[l] = root[l] = 0.0f;  // beyond the tensor nothing enters a scale
        }
        store_raw(param, pt, e, count, vec, raw_of(p, pt));
        if constexpr (kCodes) {
            const Raw mc = encode(mm, false, ms[i]), vc = encode(root, true, vs[i]);
            store_raw(m, kE4M3, e, count, vec, mc);
            store_raw(v, kE4M3, e, count, vec, vc);
            if (lane == 0 && count > 0) {
                list.m_scale[k][e / kStateBlock] = ms[i];
                list.v_scale[k][e / kStateBlock] = vs[i];
            }
        } else {
            store_raw(m, kF32, e, count, vec, raw_of(mm, kF32));
            store_raw(v, kF32, e, count, vec, raw_of(vv, kF32));
        }
    }
}

template <bool kCodes>
__device__ __forceinline__ void adamw_tensor(const AdamwList& list, const StepScalars& s, int k, int64_t e0) {
    const int pt = list.param_type[k], gt = list.grad_type[k];
    constexpr int st = kCodes ? kE4M3 : kF32;
    const bool whole = e0 + kAdamwChunk <= list.n[k] && on_fours(list.param[k], pt) && on_fours(list.grad[k], gt) && on_fours(list.m[k], st) &&
                       on_fours(list.v[k], st);
    if (!whole) {
        // a block at a time, in turn over the waves: little code, which a small
        // tensor's time goes into fetching
#pragma unroll 1
        for (int64_t e = e0 + (threadIdx.x >> 6) * kStateBlock; e < min(e0 + kAdamwChunk, list.n[k]); e += kThreads / 64 * kStateBlock)
            adamw_chunk<kCodes, false>(list, s, k, e, pt, gt);
        return;
    }
    const int64_t mine = e0 + (int64_t)(threadIdx.x >> 6) * (kPieces * kStateBlock);
    const auto with_grad = [&](auto param) {
        if (gt == kF32) adamw_chunk<kCodes, true>(list, s, k, mine, decltype(param)::value, kF32);
        else if (gt == kBF16) adamw_chunk<kCodes, true>(list, s, k, mine, decltype(param)::value, kBF16);
        else adamw_chunk<kCodes, true>(list, s, k, mine, decltype(param)::value, kF16);
    };
    if (pt == kF32) with_grad(std::integral_constant<int, kF32>{});
    else if (pt == kBF16) with_grad(std::integral_constant<int, kBF16>{});
    else with_grad(std::integral_constant<int, kF16>{});
}

__global__ __launch_bounds__(kThreads) void adamw_list_kernel(AdamwList list, StepScalars s) {
    const uint32_t c = blockIdx.x;
    const int k = find_tensor(list, c);
    const int64_t e0 = (int64_t)(c - list.chunk0[k]) * kAdamwChunk;
    if (list.state_type[k] == kE4M3) adamw_tensor<true>(list, s, k, e0);
    else adamw_tensor<false>(list, s, k, e0);
}

}  // namespace

int launch_adamw_list(const AdamwList& list, const StepScalars& s, void* stream) {
    if (list.chunks == 0) return hipSuccess;
    hipLaunchKernelGGL(adamw_list_kernel, dim3(list.chunks), dim3(kThreads), 0, (hipStream_t)stream, list, s);
    return hipGetLastError();
}

}  // namespace bfz
