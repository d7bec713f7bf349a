// AdamW over many tensors at once, states in 32 or 8 bits.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "layer_internal.h"
#include "quant_device.h"

#pragma clang fp contract(off)

namespace bfz {
namespace {

constexpr int kThreads = 256;
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ void load8_typed(const void* p, int type, int64_t e, int count, bool vec, float (&x)[8]) {
    switch (type) {
        case kF32: load8_any(static_cast<const float*>(p) + e, count, vec, x); break;
        case kBF16: load8_any(static_cast<const bf16_t*>(p) + e, count, vec, x); break;
        default: load8_any(static_cast<const f16_t*>(p) + e, count, vec, x); break;
    }
}

template <class T>
__device__ __forceinline__ void store8_any(T* p, int count, bool vec, const float (&x)[8]) {
    if (vec && count >= 8) {
        store8(p, x);
        return;
    }
#pragma unroll
    for (int l = 0; l < 8; ++l)
        if (l < count) p[l] = Elem<T>::to(x[l]);
}

__device__ __forceinline__ void store8_typed(void* p, int type, int64_t e, int count, bool vec, const float (&x)[8]) {
    switch (type) {
        case kF32: store8_any(static_cast<float*>(p) + e, count, vec, x); break;
        case kBF16: store8_any(static_cast<bf16_t*>(p) + e, count, vec, x); break;
        default: store8_any(static_cast<f16_t*>(p) + e, count, vec, x); break;
    }
}

__device__ __forceinline__ u32x2 load_codes(const uint8_t* p, int count, bool vec) {
    if (vec && count >= 8) return *reinterpret_cast<const u32x2*>(p);
    u32x2 w = {0u, 0u};
#pragma unroll
    for (int l = 0; l < 8; ++l)
        if (l < count) w[l >> 2] |= (uint32_t)p[l] << (8 * (l & 3));
    return w;
}

__device__ __forceinline__ void store_codes(uint8_t* p, int count, bool vec, const u32x2& w) {
    if (vec && count >= 8) {
        *reinterpret_cast<u32x2*>(p) = w;
        return;
    }
#pragma unroll
    for (int l = 0; l < 8; ++l)
        if (l < count) p[l] = (uint8_t)(w[l >> 2] >> (8 * (l & 3)));
}

__device__ __forceinline__ void decode(const u32x2& w, float scale, float (&x)[8]) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        x[4 * k] = __builtin_amdgcn_cvt_f32_fp8((int)w[k], 0) * scale;
        x[4 * k + 1] = __builtin_amdgcn_cvt_f32_fp8((int)w[k], 1) * scale;
        x[4 * k + 2] = __builtin_amdgcn_cvt_f32_fp8((int)w[k], 2) * scale;
        x[4 * k + 3] = __builtin_amdgcn_cvt_f32_fp8((int)w[k], 3) * scale;
    }
}

// Codes of a block's values, 32 lanes to a block, and its scale.
__device__ __forceinline__ u32x2 encode(const float (&x)[8], bool positive, float& scale) {
    float top = row_max(abs_max8(x));
    top = fmaxf(top, __shfl_xor(top, 16, 64));
    scale = scale_of(top, false);
    uint32_t w[2];
    quantize8(x, Quotient(scale), w);
    if (positive) {
#pragma unroll
        for (int l = 0; l < 8; ++l)
            if (x[l] > 0.0f && ((w[l >> 2] >> (8 * (l & 3))) & 0xFFu) == 0u) w[l >> 2] |= 1u << (8 * (l & 3));
    }
    return u32x2{w[0], w[1]};
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

// A chunk a workgroup; a thread takes 8 elements at a time, 32 lanes a block.
__global__ __launch_bounds__(kThreads) void adamw_list_kernel(AdamwList list, StepScalars s) {
    const uint32_t c = blockIdx.x;
    const int k = find_tensor(list, c);
    const int64_t n = list.n[k];
    const bool codes = list.state_type[k] == kE4M3;
    const int pt = list.param_type[k], gt = list.grad_type[k];
    void* param = list.param[k];
    const void* grad = list.grad[k];
    void* m = list.m[k];
    void* v = list.v[k];
    const bool vec = ((reinterpret_cast<uintptr_t>(param) | reinterpret_cast<uintptr_t>(grad)) & 15u) == 0 &&
                     ((reinterpret_cast<uintptr_t>(m) | reinterpret_cast<uintptr_t>(v)) & (codes ? 7u : 15u)) == 0;
    const float factor = s.grad_scale ? *s.grad_scale : 1.0f;
    const int64_t e0 = (int64_t)(c - list.chunk0[k]) * kAdamwChunk;
    for (int64_t e = e0 + 8 * threadIdx.x; e - 8 * (int64_t)threadIdx.x < min(e0 + kAdamwChunk, n); e += 8 * kThreads) {
        const int64_t left = n - e;
        const int count = left <= 0 ? 0 : left >= 8 ? 8 : (int)left;
        const int64_t block = e / kStateBlock;
        float p[8], g[8], mm[8], vv[8];
        load8_typed(param, pt, e, count, vec, p);
        load8_typed(grad, gt, e, count, vec, g);
        if (codes) {
            const bool there = count > 0;
            decode(load_codes(static_cast<const uint8_t*>(m) + e, count, vec), there ? list.m_scale[k][block] : 0.0f, mm);
            decode(load_codes(static_cast<const uint8_t*>(v) + e, count, vec), there ? list.v_scale[k][block] : 0.0f, vv);
#pragma unroll
            for (int l = 0; l < 8; ++l) vv[l] *= vv[l];
        } else {
            load8_typed(m, kF32, e, count, vec, mm);
            load8_typed(v, kF32, e, count, vec, vv);
        }
        float root[8];
#pragma unroll
        for (int l = 0; l < 8; ++l) {
            const float x = s.grad_scale ? g[l] * factor : g[l];
            mm[l] = s.b1 * mm[l] + s.c1 * x;
            vv[l] = s.b2 * vv[l] + s.c2 * (x * x);
            root[l] = sqrtf(vv[l]);
            const float den = root[l] / s.sbc2 + s.eps;
            float pp = p[l] - s.step_size * (mm[l] / den);
            if (s.has_decay) pp = pp - s.decay * pp;
            p[l] = l < count ? pp : 0.0f;
            if (l >= count) mm[l] = root[l] = 0.0f;
        }
        store8_typed(param, pt, e, count, vec, p);
        if (codes) {
            float ms, vs;
            const u32x2 mc = encode(mm, false, ms), vc = encode(root, true, vs);
            store_codes(static_cast<uint8_t*>(m) + e, count, vec, mc);
            store_codes(static_cast<uint8_t*>(v) + e, count, vec, vc);
            if ((threadIdx.x & 31) == 0 && count > 0) {
                list.m_scale[k][block] = ms;
                list.v_scale[k][block] = vs;
            }
        } else {
            store8_typed(m, kF32, e, count, vec, mm);
            store8_typed(v, kF32, e, count, vec, vv);
        }
    }
}

}  // namespace

int launch_adamw_list(const AdamwList& list, const StepScalars& s, void* stream) {
    if (list.chunks == 0) return hipSuccess;
    hipLaunchKernelGGL(adamw_list_kernel, dim3(list.chunks), dim3(kThreads), 0, (hipStream_t)stream, list, s);
    return hipGetLastError();
}

}  // namespace bfz
