// Layer norm and its gradient.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "layer_internal.h"
#include "ops_device.h"

namespace bfz {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float get_any(const void* p, int type, int64_t i) {
    return type == kF32 ? static_cast<const float*>(p)[i]
                        : type == kBF16 ? Elem<bf16_t>::get(static_cast<const bf16_t*>(p)[i]) : Elem<f16_t>::get(static_cast<const f16_t*>(p)[i]);
}

__device__ __forceinline__ void put_any(void* p, int type, int64_t i, float x) {
    if (type == kF32) static_cast<float*>(p)[i] = x;
    else if (type == kBF16) static_cast<bf16_t*>(p)[i] = Elem<bf16_t>::to(x);
    else static_cast<f16_t*>(p)[i] = Elem<f16_t>::to(x);
}

__device__ __forceinline__ float wave_sum(float x) {
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) x += __shfl_xor(x, off, 64);
    return x;
}

__device__ __forceinline__ float block_sum(float x, float* lds) {
    x = wave_sum(x);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = x;
    __syncthreads();
    return (lds[0] + lds[1]) + (lds[2] + lds[3]);
}

__global__ __launch_bounds__(kThreads) void layer_norm_kernel(LayerNormArgs a) {
    __shared__ float lds[4];
    for (int64_t r = blockIdx.x; r < a.n; r += gridDim.x) {
        float sum = 0.0f;
        for (int64_t c = threadIdx.x; c < a.dim; c += kThreads) sum += get_any(a.x, a.x_type, r * a.x_ld + c);
        const float mean = block_sum(sum, lds) / (float)a.dim;
        float square = 0.0f;
        for (int64_t c = threadIdx.x; c < a.dim; c += kThreads) {
            const float d = get_any(a.x, a.x_type, r * a.x_ld + c) - mean;
            square += d * d;
        }
        const float rstd = 1.0f / sqrtf(block_sum(square, lds) / (float)a.dim + a.eps);
        for (int64_t c = threadIdx.x; c < a.dim; c += kThreads) {
            const float h = (get_any(a.x, a.x_type, r * a.x_ld + c) - mean) * rstd;
            const float w = a.weight ? get_any(a.weight, a.param_type, c) : 1.0f;
            const float b = a.bias ? get_any(a.bias, a.param_type, c) : 0.0f;
            put_any(a.out, a.out_type, r * a.out_ld + c, __builtin_fmaf(h, w, b));
        }
        if (threadIdx.x == 0) {
            if (a.mean) a.mean[r] = mean;
            if (a.rstd) a.rstd[r] = rstd;
        }
    }
}

__global__ __launch_bounds__(kThreads) void layer_norm_dx_kernel(LayerNormGradArgs a) {
    __shared__ float lds[4];
    for (int64_t r = blockIdx.x; r < a.n; r += gridDim.x) {
        const float mean = a.mean[r], rstd = a.rstd[r];
        float s1 = 0.0f, s2 = 0.0f;
        for (int64_t c = threadIdx.x; c < a.dim; c += kThreads) {
            const float h = (get_any(a.x, a.x_type, r * a.x_ld + c) - mean) * rstd;
            const float g = get_any(a.dout, a.dout_type, r * a.dout_ld + c) * (a.weight ? get_any(a.weight, a.param_type, c) : 1.0f);
            s1 += g;
            s2 += g * h;
        }
        s1 = block_sum(s1, lds) / (float)a.dim;
        s2 = block_sum(s2, lds) / (float)a.dim;
        for (int64_t c = threadIdx.x; c < a.dim; c += kThreads) {
            const float h = (get_any(a.x, a.x_type, r * a.x_ld + c) - mean) * rstd;
            const float g = get_any(a.dout, a.dout_type, r * a.dout_ld + c) * (a.weight ? get_any(a.weight, a.param_type, c) : 1.0f);
            put_any(a.dx, a.dx_type, r * a.dx_ld + c, rstd * (g - s1 - h * s2));
        }
    }
}

// A thread a column.
__global__ __launch_bounds__(64) void layer_norm_dw_kernel(LayerNormGradArgs a) {
    const int64_t c = (int64_t)blockIdx.x * 64 + threadIdx.x;
    if (c >= a.dim) return;
    float dw = 0.0f, db = 0.0f;
    for (int64_t r = 0; r < a.n; ++r) {
        const float d = get_any(a.dout, a.dout_type, r * a.dout_ld + c);
        dw += d * ((get_any(a.x, a.x_type, r * a.x_ld + c) - a.mean[r]) * a.rstd[r]);
        db += d;
    }
    if (a.dweight) put_any(a.dweight, a.dparam_type, c, a.accumulate ? get_any(a.dweight, a.dparam_type, c) + dw : dw);
    if (a.dbias) put_any(a.dbias, a.dparam_type, c, a.accumulate ? get_any(a.dbias, a.dparam_type, c) + db : db);
}

}  // namespace

int launch_layer_norm(const LayerNormArgs& a, void* stream) {
    hipLaunchKernelGGL(layer_norm_kernel, dim3((uint32_t)std::min<int64_t>(a.n, 65536)), dim3(kThreads), 0, (hipStream_t)stream, a);
    return hipGetLastError();
}

int64_t layer_norm_work_bytes(int64_t, int64_t) { return 256; }

int launch_layer_norm_grad(const LayerNormGradArgs& a, void*, void* stream) {
    // the columns first: dx may be dout itself
    if (a.dweight || a.dbias)
        hipLaunchKernelGGL(layer_norm_dw_kernel, dim3((uint32_t)((a.dim + 63) / 64)), dim3(64), 0, (hipStream_t)stream, a);
    if (a.dx && a.n > 0)
        hipLaunchKernelGGL(layer_norm_dx_kernel, dim3((uint32_t)std::min<int64_t>(a.n, 65536)), dim3(kThreads), 0, (hipStream_t)stream, a);
    return hipGetLastError();
}

}  // namespace bfz
