// Layer norm and its gradient.
//
//   h = (x - mean) rstd,  out = h weight + bias,  g = dout weight
//   dx = rstd (g - mean(g) - h mean(g h)),  dweight = sum dout h,  dbias = sum dout
//
// Bound by memory: a row is read once, kept in registers while its sums are made,
// and written once.  The sums take two steps, so that a large common offset costs
// nothing but its own rounding in the mean that is kept: the mean; then the mean of
// what is left, by which the first one was off (up to 52 roundings of the offset:
// a constant row of 16321.2 in 11008 columns came out as 0.88 instead of 0), and of
// its square, less the square of that.  A row belongs to 64 to 1024 threads
// with 8 or 16 (32 beyond 16384 columns) of its elements each; workgroups walk
// rows, the next row's loads under way while one is summed, and keep weight and
// bias, and in the gradient their columns' sums for dweight and dbias, in
// registers.  Those leave as one partial row a workgroup, which a second kernel
// adds: sums in an order that the sizes fix.
//
// 32768 x 4096 bf16: 100 us (5.3 TB/s), the gradient 152 (5.3, a copy reaches 4.8);
// 3001 x 1001 floats 7.3 and 15.7 us, one row 3.4 of a 7.3 us call.  16384 x 1024: 15
// and 24.  Taking the first mean's error off costs 1% of the largest, 3% of 16384 x
// 1024.  Beyond 16384 columns a thread's 32 elements spill, in the gradient most
// (2000 x 20000: 131 and 436 us, 2000 x 20001: 128 and 449).  (Back-to-back calls.)
#include <hip/hip_runtime.h>

#include <algorithm>
#include <type_traits>

#include "layer_internal.h"
#include "ops_device.h"

namespace bfz {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

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

// 16 bytes on any element's boundary, which this hardware's loads and stores take.
typedef uint32_t on_words __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t on_halves __attribute__((ext_vector_type(4), aligned(2)));

// A thread's elements of a row: pieces of 8 side by side, of which those within the
// row are the first.  kWide: an array may hold 4-byte elements.
template <int kLanes, int kPieces, bool kWide>
struct Row {
    static constexpr int kWords = kWide ? 8 : 4;
    struct Raw {
        uint32_t w[kPieces][kWords];
    };
    int lane, count[kPieces];
    __device__ __forceinline__ Row(int lane, int dim) : lane(lane) {
#pragma unroll
        for (int j = 0; j < kPieces; ++j) {
            const int left = dim - column(j, 0);
            count[j] = left < 0 ? 0 : left > 8 ? 8 : left;
        }
    }
    __device__ __forceinline__ int column(int j, int l) const { return (j * kLanes + lane) * 8 + l; }
    // loads only: what is loaded is converted when it is used
    // (the last piece's elements are selected, not branched to: that took 8% of
    // 32768 x 4096 bf16, which has no such piece)
    __device__ __forceinline__ void load(const void* row, int type, Raw& r) const {
#pragma unroll
        for (int j = 0; j < kPieces; ++j) {
            if (count[j] == 8) {
                const char* p = static_cast<const char*>(row) + (int64_t)column(j, 0) * (kWide && type == kF32 ? 4 : 2);
                if constexpr (kWide) {
                    if (type != kF32) {
                        const u32x4 a = *reinterpret_cast<const on_halves*>(p);
#pragma unroll
                        for (int i = 0; i < 4; ++i) r.w[j][i] = a[i];
                        continue;
                    }
                }
                typedef std::conditional_t<kWide, on_words, on_halves> Read;
                const u32x4 a = *reinterpret_cast<const Read*>(p);
#pragma unroll
                for (int i = 0; i < 4; ++i) r.w[j][i] = a[i];
                if constexpr (kWide) {
                    const u32x4 b = reinterpret_cast<const Read*>(p)[1];
#pragma unroll
                    for (int i = 0; i < 4; ++i) r.w[j][4 + i] = b[i];
                }
                continue;
            }
#pragma unroll
            for (int i = 0; i < kWords; ++i) r.w[j][i] = 0;
#pragma unroll
            for (int l = 0; l < 8; ++l) {
                const int c = column(j, l);
                uint32_t x = 0;
                if (l < count[j]) {
                    if (kWide && type == kF32) x = static_cast<const uint32_t*>(row)[c];
                    else x = static_cast<const uint16_t*>(row)[c];
                }
                if (kWide && type == kF32) r.w[j][l & (kWords - 1)] = x;
                else r.w[j][l >> 1] |= x << (16 * (l & 1));
            }
        }
    }
    __device__ __forceinline__ void values(const Raw& r, int type, float (&x)[kPieces][8]) const {
        if (kWide && type == kF32) {
#pragma unroll
            for (int j = 0; j < kPieces; ++j)
#pragma unroll
                for (int l = 0; l < 8; ++l) x[j][l] = __uint_as_float(r.w[j][l & (kWords - 1)]);
            return;
        }
#pragma unroll
        for (int j = 0; j < kPieces; ++j)
#pragma unroll
            for (int l = 0; l < 8; ++l) {
                const uint32_t h = r.w[j][l >> 1] >> (16 * (l & 1));
                if (type == kBF16) x[j][l] = __uint_as_float(h << 16);
                else x[j][l] = (float)__builtin_bit_cast(f16_t, (uint16_t)h);
            }
    }
    __device__ __forceinline__ void store(void* row, int type, const float (&x)[kPieces][8]) const {
#pragma unroll
        for (int j = 0; j < kPieces; ++j) {
            const int c = column(j, 0);
            if (count[j] == 8) {
                if (type == kF32) {
                    on_words* p = reinterpret_cast<on_words*>(static_cast<float*>(row) + c);
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        p[h] = u32x4{__float_as_uint(x[j][4 * h]), __float_as_uint(x[j][4 * h + 1]), __float_as_uint(x[j][4 * h + 2]),
                                     __float_as_uint(x[j][4 * h + 3])};
                } else {
                    u32x4 a;
#pragma unroll
                    for (int i = 0; i < 4; ++i) a[i] = type == kBF16 ? pack2<bf16_t>(x[j][2 * i], x[j][2 * i + 1]) : pack2<f16_t>(x[j][2 * i], x[j][2 * i + 1]);
                    *reinterpret_cast<on_halves*>(static_cast<uint16_t*>(row) + c) = a;
                }
            } else {
#pragma unroll
                for (int l = 0; l < 8; ++l)
                    if (l < count[j]) put_any(row, type, column(j, l), x[j][l]);
            }
        }
    }
    // elements of a vector of parameters, `none` where there is none, from piece
    // j0 on
    template <int kMany>
    __device__ __forceinline__ void params(const void* p, int type, float none, float (&x)[kMany][8], int j0 = 0) const {
#pragma unroll
        for (int j = 0; j < kMany; ++j) {
            const int c = column(j0 + j, 0);
            if (p && count[j0 + j] == 8 && (reinterpret_cast<uintptr_t>(p) & 15u) == 0) {
                if (type == kF32) load8(static_cast<const float*>(p) + c, x[j]);
                else if (type == kBF16) load8(static_cast<const bf16_t*>(p) + c, x[j]);
                else load8(static_cast<const f16_t*>(p) + c, x[j]);
                continue;
            }
#pragma unroll
            for (int l = 0; l < 8; ++l) x[j][l] = p && l < count[j0 + j] ? get_any(p, type, column(j0 + j, l)) : none;
        }
    }
};

// Sums over the kLanes threads of a row, the same in all of them; slot: LDS of
// the row, kLanes / 64 floats for each of the sums.
template <int kLanes, int kSums>
__device__ __forceinline__ void row_sums(float (&s)[kSums], float* slot, int lane) {
#pragma unroll
    for (int k = 0; k < kSums; ++k) s[k] = wave_sum(s[k]);
    if constexpr (kLanes > 64) {
        constexpr int kWaves = kLanes / 64;
        if ((lane & 63) == 0) {
#pragma unroll
            for (int k = 0; k < kSums; ++k) slot[k * kWaves + (lane >> 6)] = s[k];
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kSums; ++k) {
            s[k] = slot[k * kWaves];
#pragma unroll
            for (int w = 1; w < kWaves; ++w) s[k] += slot[k * kWaves + w];
        }
    }
}

__device__ __forceinline__ const char* row_of(const void* p, int type, int64_t r, int64_t ld) {
    return static_cast<const char*>(p) + r * ld * (type == kF32 ? 4 : 2);
}

constexpr int most(int a, int b) { return a > b ? a : b; }

template <int kLanes, int kPieces, bool kWide>
__global__ __launch_bounds__(most(kLanes, 256)) void layer_norm_kernel(LayerNormArgs a) {
    constexpr int kRows = most(kLanes, 256) / kLanes;
    __shared__ float lds[kRows][3 * (kLanes / 64)];
    const int lane = threadIdx.x % kLanes, group = threadIdx.x / kLanes;
    typedef Row<kLanes, kPieces, kWide> Mine;
    const Mine row(lane, (int)a.dim);
    const int64_t step = (int64_t)gridDim.x * kRows;
    const float scale = 1.0f / (float)a.dim;
    int64_t r = (int64_t)blockIdx.x * kRows + group;
    constexpr bool kKeep = kPieces <= 2;  // parameters, and the next row's loads, in registers
    typename Mine::Raw raw;
    if constexpr (kKeep) row.load(row_of(a.x, a.x_type, min(r, a.n - 1), a.x_ld), a.x_type, raw);
    float w[kKeep ? kPieces : 1][8], b[kKeep ? kPieces : 1][8];
    if constexpr (kKeep) {
        row.params(a.weight, a.param_type, 1.0f, w);
        row.params(a.bias, a.param_type, 0.0f, b);
    }
    // the same number of turns for all rows of a workgroup, which share barriers
    for (int64_t r0 = (int64_t)blockIdx.x * kRows; r0 < a.n; r0 += step, r += step) {
        float x[kPieces][8];
        Mine now = row;
        // four pieces' addresses, made anew in each turn: kept from one to the next,
        // they spill, with them the row (2000 x 20000 bf16: 219 us instead of 131)
        if constexpr (!kKeep) __asm__ volatile("" : "+v"(now.lane));
        if constexpr (!kKeep) now.load(row_of(a.x, a.x_type, min(r, a.n - 1), a.x_ld), a.x_type, raw);
        now.values(raw, a.x_type, x);
        if constexpr (kKeep) {
            if (r0 + step < a.n) now.load(row_of(a.x, a.x_type, min(r + step, a.n - 1), a.x_ld), a.x_type, raw);
        }
        float sum[1] = {0.0f};
#pragma unroll
        for (int j = 0; j < kPieces; ++j)
#pragma unroll
            for (int l = 0; l < 8; ++l) sum[0] += x[j][l];
        row_sums<kLanes>(sum, lds[group], lane);
        const float first = sum[0] * scale;
        // of x - first, and of its square
        float rest[2] = {0.0f, 0.0f};
#pragma unroll
        for (int j = 0; j < kPieces; ++j)
#pragma unroll
            for (int l = 0; l < 8; ++l) {
                x[j][l] -= first;
                const float mine = l < now.count[j] ? x[j][l] : 0.0f;
                rest[0] += mine;
                rest[1] = __builtin_fmaf(mine, mine, rest[1]);
            }
        row_sums<kLanes>(rest, lds[group] + kLanes / 64, lane);
        const float off = rest[0] * scale, mean = first + off, square = rest[1] * scale;
        // an infinite square (or NaN) stays
        const float var = square < INFINITY ? fmaxf(__builtin_fmaf(-off, off, square), 0.0f) : square;
        const float rstd = 1.0f / sqrtf(var + a.eps), shift = -off * rstd;
#pragma unroll
        for (int j = 0; j < kPieces; ++j) {
            if constexpr (!kKeep) {
                now.params(a.weight, a.param_type, 1.0f, w, j);
                now.params(a.bias, a.param_type, 0.0f, b, j);
            }
#pragma unroll
            for (int l = 0; l < 8; ++l) x[j][l] = __builtin_fmaf(__builtin_fmaf(x[j][l], rstd, shift), w[kKeep ? j : 0][l], b[kKeep ? j : 0][l]);
        }
        if (r < a.n) {
            now.store(const_cast<char*>(row_of(a.out, a.out_type, r, a.out_ld)), a.out_type, x);
            if (lane == 0) {
                if (a.mean) a.mean[r] = mean;
                if (a.rstd) a.rstd[r] = rstd;
            }
        }
    }
}

// dweight (k = 0) or dbias of column c.
__device__ __forceinline__ void put_param(const LayerNormGradArgs& a, int k, int64_t c, float sum) {
    void* out = k ? a.dbias : a.dweight;
    if (out) put_any(out, a.dparam_type, c, a.accumulate ? get_any(out, a.dparam_type, c) + sum : sum);
}

// Threads of a workgroup of the gradient: as many rows at a time as fit, so that
// few partial rows leave.
constexpr int kGradThreads = 1024;

template <int kLanes, int kPieces, bool kWide>
__global__ __launch_bounds__(kGradThreads) void layer_norm_grad_kernel(LayerNormGradArgs a, float* partial) {
    constexpr int kRows = kGradThreads / kLanes, kWaves = kLanes / 64;
    constexpr bool kAhead = kPieces == 1 || (kPieces == 2 && !kWide);  // the next row's loads under way: where registers allow
    __shared__ float lds[2][kRows][2 * kWaves];
    __shared__ float sums[kRows][8][kLanes];
    const int lane = threadIdx.x % kLanes, group = threadIdx.x / kLanes;
    typedef Row<kLanes, kPieces, kWide> Mine;
    const Mine row(lane, (int)a.dim);
    const int64_t step = (int64_t)gridDim.x * kRows;
    const float scale = 1.0f / (float)a.dim;
    int64_t r = (int64_t)blockIdx.x * kRows + group;
    typename Mine::Raw raw_x, raw_d;
    float mean = 0.0f, rstd = 0.0f;
    auto load = [&](int64_t at) {
        at = min(at, a.n - 1);
        row.load(row_of(a.x, a.x_type, at, a.x_ld), a.x_type, raw_x);
        row.load(row_of(a.dout, a.dout_type, at, a.dout_ld), a.dout_type, raw_d);
        mean = a.mean[at];
        rstd = a.rstd[at];
    };
    constexpr bool kKeep = kPieces <= 2;
    float dw[kPieces][8] = {}, db[kPieces][8] = {}, w[kKeep ? kPieces : 1][8];
    if constexpr (kAhead) {
        if ((int64_t)blockIdx.x * kRows < a.n) load(r);
    }
    if constexpr (kKeep) row.params(a.weight, a.param_type, 1.0f, w);
    int turn = 0;
    for (int64_t r0 = (int64_t)blockIdx.x * kRows; r0 < a.n; r0 += step, r += step, turn ^= 1) {
        if constexpr (!kAhead) load(r);
        float h[kPieces][8], d[kPieces][8];
        const float m = mean, q = rstd;
        row.values(raw_x, a.x_type, h);
        row.values(raw_d, a.dout_type, d);
        if constexpr (kAhead) {
            if (r0 + step < a.n) load(r + step);
        }
        const bool there = r < a.n;
        float s[2] = {0.0f, 0.0f};
#pragma unroll
        for (int j = 0; j < kPieces; ++j) {
            if constexpr (!kKeep) row.params(a.weight, a.param_type, 1.0f, w, j);
#pragma unroll
            for (int l = 0; l < 8; ++l) {
                // beyond the row's end d is zero; h there does not count (0 times it
                // may be NaN)
                h[j][l] = l < row.count[j] ? (h[j][l] - m) * q : 0.0f;
                const float g = d[j][l] * w[kKeep ? j : 0][l];
                s[0] += g;
                s[1] = __builtin_fmaf(g, h[j][l], s[1]);
                if (there) {
                    dw[j][l] = __builtin_fmaf(d[j][l], h[j][l], dw[j][l]);
                    db[j][l] += d[j][l];
                }
            }
        }
        if (a.dx) {
            row_sums<kLanes>(s, lds[turn][group], lane);
            const float m1 = s[0] * scale, m2 = s[1] * scale;
#pragma unroll
            for (int j = 0; j < kPieces; ++j) {
                if constexpr (!kKeep) row.params(a.weight, a.param_type, 1.0f, w, j);
#pragma unroll
                for (int l = 0; l < 8; ++l) d[j][l] = q * (__builtin_fmaf(d[j][l], w[kKeep ? j : 0][l], -m1) - h[j][l] * m2);
            }
            if (there) row.store(const_cast<char*>(row_of(a.dx, a.dx_type, r, a.dx_ld)), a.dx_type, d);
        }
    }
    if (!a.dweight && !a.dbias) return;
    // the workgroup's rows added, in their order, 8 columns of each thread at a time
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int j = 0; j < kPieces; ++j) {
            const float(&x)[8] = k ? db[j] : dw[j];
            __syncthreads();
#pragma unroll
            for (int l = 0; l < 8; ++l) sums[group][l][lane] = x[l];
            __syncthreads();
            for (int i = threadIdx.x; i < 8 * kLanes; i += kGradThreads) {
                const int of = i >> 3, l = i & 7;
                float sum = 0.0f;
#pragma unroll
                for (int g = 0; g < kRows; ++g) sum += sums[g][l][of];
                const int64_t c = (j * kLanes + of) * 8 + l;
                if (c >= a.dim) continue;
                if (gridDim.x == 1) put_param(a, k, c, sum);
                else partial[(int64_t)blockIdx.x * 2 * a.dim + k * a.dim + c] = sum;
            }
        }
}

// dweight and dbias from the workgroups' partial rows: 32 columns a workgroup, 8
// threads to a column.
constexpr int kJoinColumns = 32, kJoinSlices = 8;
__global__ __launch_bounds__(kJoinColumns* kJoinSlices) void join_params_kernel(const float* __restrict__ partial, int64_t rows, LayerNormGradArgs a) {
    __shared__ float lds[kJoinSlices][kJoinColumns];
    const int x = threadIdx.x % kJoinColumns, y = threadIdx.x / kJoinColumns;
    const int64_t c = (int64_t)blockIdx.x * kJoinColumns + x;
    float sum = 0.0f;
    if (c < 2 * a.dim) {
        int64_t r = y;
        for (; r + 7 * kJoinSlices < rows; r += 8 * kJoinSlices) {
            float p[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) p[u] = partial[(r + u * kJoinSlices) * 2 * a.dim + c];
            sum += ((p[0] + p[1]) + (p[2] + p[3])) + ((p[4] + p[5]) + (p[6] + p[7]));
        }
        for (; r < rows; r += kJoinSlices) sum += partial[r * 2 * a.dim + c];
    }
    lds[y][x] = sum;
    __syncthreads();
    if (y != 0 || c >= 2 * a.dim) return;
#pragma unroll
    for (int k = 1; k < kJoinSlices; ++k) sum += lds[k][x];
    put_param(a, c >= a.dim, c < a.dim ? c : c - a.dim, sum);
}

// ---- host -------------------------------------------------------------------------

// Calls f(threads of a row, pieces of 8 elements a thread) with the first of
// these that hold dim columns.
template <class F>
int with_shape(int64_t dim, F&& f) {
    using std::integral_constant;
    if (dim <= 512) return f(integral_constant<int, 64>{}, integral_constant<int, 1>{});
    if (dim <= 1024) return f(integral_constant<int, 64>{}, integral_constant<int, 2>{});
    if (dim <= 2048) return f(integral_constant<int, 256>{}, integral_constant<int, 1>{});
    if (dim <= 4096) return f(integral_constant<int, 256>{}, integral_constant<int, 2>{});
    if (dim <= 8192) return f(integral_constant<int, 512>{}, integral_constant<int, 2>{});
    if (dim <= 16384) return f(integral_constant<int, 1024>{}, integral_constant<int, 2>{});
    return f(integral_constant<int, 1024>{}, integral_constant<int, 4>{});
}

// The same for the gradient, which has 16 waves' registers for twice the arrays.
template <class F>
int with_grad_shape(int64_t dim, F&& f) {
    using std::integral_constant;
    if (dim <= 512) return f(integral_constant<int, 64>{}, integral_constant<int, 1>{});
    if (dim <= 1024) return f(integral_constant<int, 128>{}, integral_constant<int, 1>{});
    if (dim <= 2048) return f(integral_constant<int, 256>{}, integral_constant<int, 1>{});
    if (dim <= 4096) return f(integral_constant<int, 512>{}, integral_constant<int, 1>{});
    if (dim <= 8192) return f(integral_constant<int, 1024>{}, integral_constant<int, 1>{});
    if (dim <= 16384) return f(integral_constant<int, 1024>{}, integral_constant<int, 2>{});
    return f(integral_constant<int, 1024>{}, integral_constant<int, 4>{});
}

template <class F>
int with_width(bool wide, F&& f) {
    return wide ? f(std::true_type{}) : f(std::false_type{});
}

// Workgroups of the gradient: one a CU, or one for every row of each thread group
// where there are fewer.
constexpr int64_t kGradWgs = 256;
int64_t grad_wgs(int64_t n, int64_t rows) { return std::max<int64_t>(1, std::min<int64_t>(kGradWgs, (n + rows - 1) / rows)); }

}  // namespace

int launch_layer_norm(const LayerNormArgs& a, void* stream) {
    return with_shape(a.dim, [&](auto lanes, auto pieces) {
        return with_width(a.x_type == kF32, [&](auto wide) {
            constexpr int kLanes = decltype(lanes)::value, kPieces = decltype(pieces)::value, kThreads = most(kLanes, 256);
            constexpr int64_t kRows = kThreads / kLanes;
            const int64_t wgs = std::min<int64_t>((a.n + kRows - 1) / kRows, 256 * 2048 / kThreads);
            hipLaunchKernelGGL((layer_norm_kernel<kLanes, kPieces, decltype(wide)::value>), dim3((uint32_t)wgs),
                               dim3(kThreads), 0, (hipStream_t)stream, a);
            return (int)hipGetLastError();
        });
    });
}

int64_t layer_norm_work_bytes(int64_t n, int64_t dim) {
    int64_t wgs = 0;
    with_grad_shape(dim, [&](auto lanes, auto) {
        wgs = grad_wgs(n, kGradThreads / decltype(lanes)::value);
        return 0;
    });
    return wgs * 2 * dim * 4;
}

int launch_layer_norm_grad(const LayerNormGradArgs& a, void* work, void* stream) {
    float* partial = a.dweight || a.dbias ? static_cast<float*>(work) : nullptr;
    if (!partial && !a.dx) return hipSuccess;
    int64_t wgs = 0;
    const int rc = with_grad_shape(a.dim, [&](auto lanes, auto pieces) {
        return with_width(a.x_type == kF32 || a.dout_type == kF32, [&](auto wide) {
            constexpr int kLanes = decltype(lanes)::value, kPieces = decltype(pieces)::value;
            wgs = grad_wgs(a.n, kGradThreads / kLanes);
            hipLaunchKernelGGL((layer_norm_grad_kernel<kLanes, kPieces, decltype(wide)::value>), dim3((uint32_t)wgs),
                               dim3(kGradThreads), 0, (hipStream_t)stream, a, partial);
            return (int)hipGetLastError();
        });
    });
    if (rc || !partial || wgs == 1) return rc;
    hipLaunchKernelGGL(join_params_kernel, dim3((uint32_t)((2 * a.dim + kJoinColumns - 1) / kJoinColumns)), dim3(kJoinColumns * kJoinSlices), 0,
                       (hipStream_t)stream, partial, wgs, a);
    return hipGetLastError();
}

}  // namespace bfz
