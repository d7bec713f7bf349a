// The linear layer in E4M3: quantizer of activations, and the three products.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "layer_internal.h"
#include "quant_device.h"

namespace bfz {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

constexpr int kThreads = 256;

// ---- quantizer ------------------------------------------------------------------

// Row groups: 16 lanes hold a group, 8 columns each; a wave 4 groups of a row.
constexpr int kRowsOfWg = 32, kGroupsOfWave = 4;

template <class T>
__global__ __launch_bounds__(kThreads) void quantize_rows_kernel(QuantizeArgs a, int32_t col_wgs, int32_t vec) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t block = blockIdx.x;
    const int64_t c = (block % col_wgs) * (kGroupsOfWave * kTileDim) + 8 * lane;
    const int64_t r0 = block / col_wgs * kRowsOfWg;
    const int64_t left = a.dim - c;
    const int count = left <= 0 ? 0 : left >= 8 ? 8 : (int)left;
    const int64_t width = (a.dim + 15) / 16 * 16;
    for (int64_t r = r0 + wave; r < min(r0 + kRowsOfWg, a.n); r += kThreads / 64) {
        float x[8];
        load8_any(static_cast<const T*>(a.x) + r * a.x_ld + c, count, vec, x);
        const float scale = scale_of(row_max(abs_max8(x)), a.pow2);
        uint32_t w[2];
        quantize8(x, Quotient(scale), w);
        if (c < width) *reinterpret_cast<u32x2*>(a.codes + r * a.codes_ld + c) = u32x2{w[0], w[1]};
        if ((lane & 15) == 0 && c < a.dim) a.scales[c / kTileDim * a.scales_ld + r] = scale;
    }
}

// Tiles: 16 lanes a row, 16 rows at a time, the whole tile in registers.
template <class T>
__global__ __launch_bounds__(kThreads) void quantize_tiles_kernel(QuantizeArgs a, int32_t col_tiles, int32_t vec) {
    __shared__ float tops[kThreads / 64];
    const int64_t i = blockIdx.x / col_tiles, j = blockIdx.x % col_tiles;
    const int64_t c = j * kTileDim + 8 * (threadIdx.x & 15);
    const int64_t left = a.dim - c;
    const int count = left <= 0 ? 0 : left >= 8 ? 8 : (int)left;
    const int64_t r0 = i * kTileDim + (threadIdx.x >> 4);
    const int64_t width = (a.dim + 15) / 16 * 16;
    float x[8][8];
    float top = 0.0f;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const int64_t r = r0 + 16 * k;
        load8_any(static_cast<const T*>(a.x) + r * a.x_ld + c, r < a.n ? count : 0, vec, x[k]);
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) top = fmaxf(top, abs_max8(x[k]));
    top = row_max(top);
    top = fmaxf(top, __shfl_xor(top, 16, 64));
    top = fmaxf(top, __shfl_xor(top, 32, 64));
    if ((threadIdx.x & 63) == 0) tops[threadIdx.x >> 6] = top;
    __syncthreads();
    const float scale = scale_of(fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3])), a.pow2);
    const Quotient q(scale);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const int64_t r = r0 + 16 * k;
        uint32_t w[2];
        quantize8(x[k], q, w);
        if (r < a.n && c < width) *reinterpret_cast<u32x2*>(a.codes + r * a.codes_ld + c) = u32x2{w[0], w[1]};
    }
    if (threadIdx.x == 0) a.scales[i * a.scales_ld + j] = scale;
}

template <class T>
int quantize(const QuantizeArgs& a, hipStream_t stream) {
    const int32_t vec = ((reinterpret_cast<uintptr_t>(a.x) | (uint64_t)(a.x_ld * sizeof(T))) & 15u) == 0;
    if (a.tiles) {
        const int64_t wide = (a.dim + kTileDim - 1) / kTileDim, high = (a.n + kTileDim - 1) / kTileDim;
        hipLaunchKernelGGL((quantize_tiles_kernel<T>), dim3((uint32_t)(wide * high)), dim3(kThreads), 0, stream, a, (int32_t)wide, vec);
    } else {
        const int64_t wide = (a.dim + kGroupsOfWave * kTileDim - 1) / (kGroupsOfWave * kTileDim), high = (a.n + kRowsOfWg - 1) / kRowsOfWg;
        hipLaunchKernelGGL((quantize_rows_kernel<T>), dim3((uint32_t)(wide * high)), dim3(kThreads), 0, stream, a, (int32_t)wide, vec);
    }
    return hipGetLastError();
}

// ---- products -------------------------------------------------------------------

// D[t][m] = sum_k scale_b(t, k) scale_a(m, k) B[t][k] A[m][k], one wave for 16 by
// 16 of D, operands read byte by byte: right for every stride and size.
struct SimpleArgs {
    const uint8_t* a;
    const uint8_t* b;
    int64_t a_m, a_k, b_n, b_k;  // strides, bytes
    const float* sa;
    const float* sb;
    int64_t sa_m, sa_k, sb_n, sb_k;  // of scales, by 128 m and 128 k; n by tile or each
    int32_t sb_shift;
    int64_t m, n, k;
    void* out;
    int32_t out_type, accumulate;
    int64_t out_ld;
};

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

// 8 codes as bf16, which holds them exactly.
__device__ __forceinline__ bf16x8 codes_to_bf16(int w0, int w1) {
    bf16x8 r;
    const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w0, 1.0f, false), b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w0, 1.0f, true);
    const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w1, 1.0f, false), d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w1, 1.0f, true);
    r[0] = a[0];
    r[1] = a[1];
    r[2] = b[0];
    r[3] = b[1];
    r[4] = c[0];
    r[5] = c[1];
    r[6] = d[0];
    r[7] = d[1];
    return r;
}

__device__ __forceinline__ i32x8 gather(const uint8_t* p, int64_t stride, bool there, int64_t k0, int64_t k, int g) {
    i32x8 r;
#pragma unroll
    for (int w = 0; w < 8; ++w) {
        uint32_t x = 0;
#pragma unroll
        for (int l = 0; l < 4; ++l) {
            const int64_t at = k0 + (w < 4 ? 16 * g + 4 * w : 64 + 16 * g + 4 * (w - 4)) + l;
            if (there && at < k) x |= (uint32_t)p[at * stride] << (8 * l);
        }
        r[w] = (int)x;
    }
    return r;
}

__device__ __forceinline__ float get_any(const void* p, int type, int64_t i) {
    return type == kF32 ? static_cast<const float*>(p)[i]
                        : type == kBF16 ? Elem<bf16_t>::get(static_cast<const bf16_t*>(p)[i]) : Elem<f16_t>::get(static_cast<const f16_t*>(p)[i]);
}

__device__ __forceinline__ void put_any(void* p, int type, int64_t i, float x) {
    if (type == kF32) static_cast<float*>(p)[i] = x;
    else if (type == kBF16) static_cast<bf16_t*>(p)[i] = Elem<bf16_t>::to(x);
    else static_cast<f16_t*>(p)[i] = Elem<f16_t>::to(x);
}

__global__ __launch_bounds__(64) void simple_product_kernel(SimpleArgs s, int32_t m_tiles) {
    const int lane = threadIdx.x, g = lane >> 4;
    const int64_t m0 = (int64_t)(blockIdx.x % m_tiles) * 16, n0 = (int64_t)(blockIdx.x / m_tiles) * 16;
    const int64_t m = m0 + (lane & 15), n = n0 + (lane & 15);
    f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int64_t k0 = 0; k0 < s.k; k0 += kTileDim) {
        const i32x8 a = gather(s.a + min(m, s.m - 1) * s.a_m, s.a_k, m < s.m, k0, s.k, g);
        const i32x8 b = gather(s.b + min(n, s.n - 1) * s.b_n, s.b_k, n < s.n, k0, s.k, g);
        f32x4 part = {0.0f, 0.0f, 0.0f, 0.0f};
        if (s.out_type == kF32) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                part = __builtin_amdgcn_mfma_f32_16x16x32_bf16(codes_to_bf16(a[2 * j], a[2 * j + 1]), codes_to_bf16(b[2 * j], b[2 * j + 1]), part, 0, 0, 0);
        } else {
            part = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, part, 0, 0, 0, 0, 0, 0);
        }
        const float scale = s.sa[m0 / kTileDim * s.sa_m + k0 / kTileDim * s.sa_k] *
                            s.sb[(min(n, s.n - 1) >> s.sb_shift) * s.sb_n + k0 / kTileDim * s.sb_k];
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[i] = __builtin_fmaf(part[i], scale, acc[i]);
    }
    if (n >= s.n) return;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t at = m0 + 4 * g + i;
        if (at >= s.m) continue;
        const int64_t e = n * s.out_ld + at;
        put_any(s.out, s.out_type, e, s.accumulate ? get_any(s.out, s.out_type, e) + acc[i] : acc[i]);
    }
}

int simple_product(const SimpleArgs& s, void* stream) {
    const int64_t m_tiles = (s.m + 15) / 16, n_tiles = (s.n + 15) / 16;
    hipLaunchKernelGGL(simple_product_kernel, dim3((uint32_t)(m_tiles * n_tiles)), dim3(64), 0, (hipStream_t)stream, s, (int32_t)m_tiles);
    return hipGetLastError();
}

void token_scales(SimpleArgs& s, const Codes& c) {
    s.sb = c.scales;
    s.sb_n = c.tiles ? c.scales_ld : 1;
    s.sb_k = c.tiles ? 1 : c.scales_ld;
    s.sb_shift = c.tiles ? 7 : 0;
}

int64_t round_up(int64_t n, int64_t to) { return (n + to - 1) / to * to; }

}  // namespace

int launch_quantize(const QuantizeArgs& a, void* stream) {
    const hipStream_t s = (hipStream_t)stream;
    return a.x_type == kF32 ? quantize<float>(a, s) : a.x_type == kBF16 ? quantize<bf16_t>(a, s) : quantize<f16_t>(a, s);
}

int64_t linear_work_bytes(int64_t n, int64_t rows, int64_t cols, int copy, int quantize) {
    return 256 + (quantize ? round_up(n * round_up(cols, 16), 256) + round_up((cols + 127) / 128 * n * 4, 256) : 0);
}

void linear_work_codes(void* work, int64_t n, int64_t cols, uint8_t** codes, int64_t* ld, float** scales) {
    *ld = round_up(cols, 16);
    *codes = static_cast<uint8_t*>(work);
    *scales = reinterpret_cast<float*>(*codes + round_up(n * *ld, 256));
}

int launch_linear(const LinearArgs& a, void*, void* stream) {
    SimpleArgs s{};
    s.a = a.weight;
    s.a_m = a.weight_ld;
    s.a_k = 1;
    s.b = a.x.p;
    s.b_n = a.x.ld;
    s.b_k = 1;
    s.sa = a.grid;
    s.sa_m = (a.cols + 127) / 128;
    s.sa_k = 1;
    token_scales(s, a.x);
    s.m = a.rows;
    s.n = a.n;
    s.k = a.cols;
    s.out = a.out;
    s.out_type = a.out_type;
    s.out_ld = a.out_ld;
    s.accumulate = a.accumulate;
    return simple_product(s, stream);
}

int launch_linear_grad_input(const LinearArgs& a, void*, void* stream) {
    SimpleArgs s{};
    s.a = a.weight;
    s.a_m = 1;
    s.a_k = a.weight_ld;
    s.b = a.x.p;
    s.b_n = a.x.ld;
    s.b_k = 1;
    s.sa = a.grid;
    s.sa_m = 1;
    s.sa_k = (a.cols + 127) / 128;
    token_scales(s, a.x);
    s.m = a.cols;
    s.n = a.n;
    s.k = a.rows;
    s.out = a.out;
    s.out_type = a.out_type;
    s.out_ld = a.out_ld;
    s.accumulate = a.accumulate;
    return simple_product(s, stream);
}

int launch_linear_grad_weight(const LinearArgs& a, void*, void* stream) {
    SimpleArgs s{};
    s.a = a.other.p;
    s.a_m = 1;
    s.a_k = a.other.ld;
    s.b = a.x.p;
    s.b_n = 1;
    s.b_k = a.x.ld;
    s.sa = a.other.scales;
    s.sa_m = 1;
    s.sa_k = a.other.scales_ld;
    s.sb = a.x.scales;
    s.sb_n = 1;
    s.sb_k = a.x.scales_ld;
    s.sb_shift = 7;
    s.m = a.cols;
    s.n = a.rows;
    s.k = a.n;
    s.out = a.out;
    s.out_type = a.out_type;
    s.out_ld = a.out_ld;
    s.accumulate = a.accumulate;
    return simple_product(s, stream);
}

}  // namespace bfz
