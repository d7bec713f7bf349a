// Softmax cross entropy over a large vocabulary, and its gradient, without
// the logits in memory.
//
//   z = h W^T,  lse[n] = log sum_v exp z[n][v],  loss[n] = lse[n] - z[n][t[n]]
//   dz[n][v] = dloss[n] (exp(z[n][v] - lse[n]) - [v = t[n]])
//   dh = dz W,  dW = dz^T h
//
// Forward: one product whose epilogue reduces a wave's 64 (32 in narrow tiles)
// logits of a token to their maximum and sum of exponentials; a small kernel
// joins those.  The work is 2 N V d operations, bound by the matrix cores once
// N is a few hundred, by reading W below that.
//
// Gradient: 6 N V d operations in three products over pieces of the
// vocabulary.  A piece's logits are computed again and leave the product as
// dz, rounded to bf16 (the matrix cores' input type: each dz is off by at
// most 2^-8 of itself, which the sums over v and n average out); then
// dz W adds onto dh's binary32 sums and dz^T h gives the piece's rows of dW.
// A float32 dW would show that rounding (1.4e-3 of it at 512 x 4000 x 128 with
// a dloss of each token's own), so what bf16 left of dz follows as a second
// bf16 part, 2^-16 off at most, and dW's product runs over the tokens twice:
// dz's rows, and h's, stand one part below the other.  An f32 dW of 512 x 4000 x
// 128 is then 2.2e-6 off.  The caller may waive it: loss and gradients of 8192 x
// 131072 x 4096 E4M3 with an f32 dW take 35.2 ms, with dz rounded once 27.4.
// dz is rounded in units of the largest dloss, by which the results are
// multiplied in binary32: where dloss is the same for all tokens, as in a
// mean, the target's p - 1 then rounds by what p holds, not by an error of
// dloss that all tokens share (at 1013 tokens the gradients' error went from
// 0.0035 to 0.0018, that of rounding them to bf16 alone).  A piece is as large as its dz may be, so that the products stay long.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <atomic>

#include "vocab_gemm.h"

namespace bfz {
namespace {

constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;

__device__ __forceinline__ int64_t target_of(const void* targets, int wide, int64_t n, int64_t vocab) {
    return row_of(targets, wide, n, vocab);
}

// What exponentials are taken relative to: the maximum, or 0 where that is
// infinite.  -inf logits, also where there is no other, then add 0, and a +inf
// one makes the sum +inf.
__device__ __forceinline__ float base_of(float top) { return fabsf(top) < INFINITY ? top : 0.0f; }

// Softmax statistics of the tile's rows for each token: maximum and sum of
// exponentials over the wave's rows, and the target's logit.
struct StatsEpilogue {
    float2* partial;  // [slot][token]
    float* target_logit;
    const void* targets;
    int32_t targets64;
    int64_t first, vocab, n, slots0;  // first: vocabulary row of m = 0
    int32_t waves_m;
    template <int kTM, int kTN>
    __device__ __forceinline__ void run(const f32x4 (&acc)[kTM][kTN], const WaveTile& w) const {
        const int64_t v0 = first + w.m0 + 4 * (w.lane >> 4);
        const int64_t slot = slots0 + (int64_t)w.tile_m * waves_m + w.wave_m;
        const bool whole = first + w.m0 + 16 * kTM <= vocab;  // all rows are in the vocabulary
#pragma unroll
        for (int u = 0; u < kTN; ++u) {
            const int64_t token = w.n0 + 16 * u + (w.lane & 15);
            const bool there = token < n;
            const int64_t t = there ? target_of(targets, targets64, token, vocab) : -1;
            float top = -INFINITY, sum = 0.0f;
            if (whole) {
#pragma unroll
                for (int r = 0; r < kTM; ++r)
#pragma unroll
                    for (int i = 0; i < 4; ++i) top = fmaxf(top, acc[r][u][i]);
            } else {
#pragma unroll
                for (int r = 0; r < kTM; ++r)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (v0 + 16 * r + i < vocab) top = fmaxf(top, acc[r][u][i]);
            }
            top = fmaxf(top, __shfl_xor(top, 16, 64));
            top = fmaxf(top, __shfl_xor(top, 32, 64));
            const float base = base_of(top);
            if (whole) {
#pragma unroll
                for (int r = 0; r < kTM; ++r)
#pragma unroll
                    for (int i = 0; i < 4; ++i) sum += __builtin_amdgcn_exp2f((acc[r][u][i] - base) * kLog2e);
            } else {
#pragma unroll
                for (int r = 0; r < kTM; ++r)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (v0 + 16 * r + i < vocab) sum += __builtin_amdgcn_exp2f((acc[r][u][i] - base) * kLog2e);
            }
            sum += __shfl_xor(sum, 16, 64);
            sum += __shfl_xor(sum, 32, 64);
            if (there && w.lane < 16) partial[slot * n + token] = make_float2(top, sum);
            // a target among these rows: for one token in a thousand
            const int64_t at = t - v0;
            if (__any(t >= 0 && at >= 0 && at < 16 * kTM)) {
#pragma unroll
                for (int r = 0; r < kTM; ++r)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (t >= 0 && at == 16 * r + i) target_logit[token] = acc[r][u][i];
            }
        }
    }
};

// dz of the piece, bf16 [token][width]; zero beyond the vocabulary.  rest, where
// there is one: what the rounding left, in the same layout.
struct LogitGradEpilogue {
    bf16_t* dz;
    bf16_t* rest;
    int64_t width, first, vocab, n;
    const float* lse;
    const float* dloss;
    const float* unit;
    const void* targets;
    int32_t targets64;
    template <int kTM, int kTN>
    __device__ __forceinline__ void run(const f32x4 (&acc)[kTM][kTN], const WaveTile& w) const {
        const int64_t m0 = w.m0 + 4 * (w.lane >> 4);
        const float most = *unit;
        const bool whole = first + w.m0 + 16 * kTM <= vocab;  // all rows are in the vocabulary
#pragma unroll
        for (int u = 0; u < kTN; ++u) {
            const int64_t token = w.n0 + 16 * u + (w.lane & 15);
            const bool there = token < n;
            const int64_t t = there ? target_of(targets, targets64, token, vocab) : -1;
            const float up = t < 0 ? 0.0f : dloss[token] / most;
            // p = 2^(z log2e - lse log2e), as 2^64 p and a factor, since the
            // instruction gives zero for subnormal results; a token without a
            // target gets p = 0
            const float turned = t < 0 ? INFINITY : lse[token] * kLog2e;
            const float shift = 64.0f - turned;
            // the roundings of both, which all the token's p share, go into the
            // factor: of the product, and of the difference
            const float back = shift - 64.0f;
            const float lost = (64.0f - (shift - back)) + (-turned - back) - __builtin_fmaf(t < 0 ? 0.0f : lse[token], kLog2e, -turned);
            const float factor = up * 0x1p-64f * (fabsf(lost) < 1.0f ? __builtin_fmaf(lost, kLn2, 1.0f) : 1.0f);
            const int64_t at = t - first - m0;
            float x[kTM][4];
#pragma unroll
            for (int r = 0; r < kTM; ++r)
#pragma unroll
                for (int i = 0; i < 4; ++i) x[r][i] = __builtin_amdgcn_exp2f(__builtin_fmaf(acc[r][u][i], kLog2e, shift)) * factor;
            // a target among these rows: for one token in a thousand
            if (__any(t >= 0 && at >= 0 && at < 16 * kTM)) {
#pragma unroll
                for (int r = 0; r < kTM; ++r)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (t >= 0 && at == 16 * r + i) x[r][i] -= up;
            }
            if (!whole) {
#pragma unroll
                for (int r = 0; r < kTM; ++r)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (first + m0 + 16 * r + i >= vocab) x[r][i] = 0.0f;
            }
            // a token without a target, whatever its logits are
            if (__any(there && t < 0)) {
#pragma unroll
                for (int r = 0; r < kTM; ++r)
#pragma unroll
                    for (int i = 0; i < 4; ++i) x[r][i] = t < 0 ? 0.0f : x[r][i];
            }
            if (!there) continue;
            bf16_t* row = dz + token * width + m0;
#pragma unroll
            for (int r = 0; r < kTM; ++r) {
                const u32x2 y = {pack2<bf16_t>(x[r][0], x[r][1]), pack2<bf16_t>(x[r][2], x[r][3])};
                *reinterpret_cast<u32x2*>(row + 16 * r) = y;
                if (rest) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) x[r][i] -= __uint_as_float((i & 1) ? (y[i >> 1] & 0xFFFF0000u) : (y[i >> 1] << 16));
                    *reinterpret_cast<u32x2*>(rest + token * width + m0 + 16 * r) =
                        u32x2{pack2<bf16_t>(x[r][0], x[r][1]), pack2<bf16_t>(x[r][2], x[r][3])};
                }
            }
        }
    }
};

// dh's binary32 sums, [split][token][ld]: written or added to.
struct SumEpilogue {
    float* sums;
    int64_t ld, slab, extent, n;  // extent: valid m, a multiple of 4
    int32_t add;
    template <int kTM, int kTN>
    __device__ __forceinline__ void run(const f32x4 (&acc)[kTM][kTN], const WaveTile& w) const {
        const int64_t m0 = w.m0 + 4 * (w.lane >> 4);
#pragma unroll
        for (int u = 0; u < kTN; ++u) {
            const int64_t token = w.n0 + 16 * u + (w.lane & 15);
            if (token >= n) continue;
            float* row = sums + w.split * slab + token * ld + m0;
#pragma unroll
            for (int r = 0; r < kTM; ++r) {
                if (m0 + 16 * r >= extent) continue;
                f32x4 x = acc[r][u];
                f32x4* p = reinterpret_cast<f32x4*>(row + 16 * r);
                if (add) x += *p;
                *p = x;
            }
        }
    }
};

// Rows of dW: column n of the product is vocabulary row first + n.
template <class O>
struct WeightGradEpilogue {
    O* dw;
    int64_t ld, dim, first, vocab;
    const float* unit;
    int32_t add, vec;  // vec: 4 elements at a time are aligned
    template <int kTM, int kTN>
    __device__ __forceinline__ void run(const f32x4 (&acc)[kTM][kTN], const WaveTile& w) const {
        const int64_t m0 = w.m0 + 4 * (w.lane >> 4);
        const float most = *unit;
#pragma unroll
        for (int u = 0; u < kTN; ++u) {
            const int64_t v = first + w.n0 + 16 * u + (w.lane & 15);
            if (v >= vocab) continue;
            O* row = dw + v * ld + m0;
#pragma unroll
            for (int r = 0; r < kTM; ++r) {
                put(row + 16 * r, m0 + 16 * r, acc[r][u] * most);
            }
        }
    }
    // 4 elements of a row from column c on
    __device__ __forceinline__ void put(O* p, int64_t c, f32x4 x) const {
        if (vec && c + 4 <= dim) {
            if constexpr (sizeof(O) == 4) {
                if (add) x += *reinterpret_cast<const f32x4*>(p);
                *reinterpret_cast<f32x4*>(p) = x;
            } else {
                if (add) {
                    const u32x2 o = *reinterpret_cast<const u32x2*>(p);
#pragma unroll
                    for (int i = 0; i < 4; ++i) x[i] += __uint_as_float((i & 1) ? (o[i >> 1] & 0xFFFF0000u) : (o[i >> 1] << 16));
                }
                const u32x2 o = {pack2<bf16_t>(x[0], x[1]), pack2<bf16_t>(x[2], x[3])};
                *reinterpret_cast<u32x2*>(p) = o;
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (c + i < dim) p[i] = Elem<O>::to(add ? Elem<O>::get(p[i]) + x[i] : x[i]);
        }
    }
};

// Rows of dW for few tokens, where a product of matrix tiles would be all
// first loads and epilogue: a thread keeps its columns of every token's h in
// registers and walks rows, whose dz the workgroup has read into LDS.  Sixteen
// tokens' products are made whatever n is: 2 tokens of 83873 x 896 take 54 us in
// bf16 (2.8 TB/s) and, with twice the bytes to write, in f32 (5.5).
constexpr int kFewGradRows = 64, kFewGradCols = 4;
template <class O>
__global__ __launch_bounds__(256) void few_weight_grad_kernel(const bf16_t* __restrict__ hidden, int64_t hidden_ld, int64_t dim,
                                                              const bf16_t* __restrict__ dz, const bf16_t* __restrict__ rest, int64_t width,
                                                              int64_t n, int64_t rows, const void* targets, int32_t targets64, WeightGradEpilogue<O> out) {
    __shared__ float d[kFewGradRows][kFewTokens];
    const int64_t v0 = (int64_t)blockIdx.x * kFewGradRows, c = ((int64_t)blockIdx.y * 256 + threadIdx.x) * kFewGradCols;
    const int count = (int)(rows - v0 < kFewGradRows ? rows - v0 : kFewGradRows);
    const float most = *out.unit;
    for (int i = threadIdx.x; i < kFewGradRows * kFewTokens; i += 256) {
        const int t = i / kFewGradRows, r = i % kFewGradRows;
        const int64_t at = t * width + v0 + r;
        d[r][t] = t < n && r < count ? (Elem<bf16_t>::get(dz[at]) + (rest ? Elem<bf16_t>::get(rest[at]) : 0.0f)) * most : 0.0f;
    }
    float h[kFewTokens][kFewGradCols];
#pragma unroll
    for (int t = 0; t < kFewTokens; ++t) {
        const bool counts = t < n && target_of(targets, targets64, t, out.vocab) >= 0;
#pragma unroll
        for (int l = 0; l < kFewGradCols; ++l)
            h[t][l] = counts && c + l < dim ? Elem<bf16_t>::get(hidden[t * hidden_ld + c + l]) : 0.0f;
    }
    __syncthreads();
    if (c >= dim) return;
    for (int r = 0; r < count; ++r) {
        f32x4 x = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int t = 0; t < kFewTokens; ++t)
#pragma unroll
            for (int l = 0; l < kFewGradCols; ++l) x[l] = __builtin_fmaf(d[r][t], h[t][l], x[l]);
        out.put(out.dw + (out.first + v0 + r) * out.ld + c, c, x);
    }
}

// lse and loss of a token from its partial statistics: 16 tokens a
// workgroup, 64 threads to a token, 8 slots a thread at a time.
constexpr int kJoinTokens = 16, kJoinSlots = 64;
__global__ __launch_bounds__(kJoinTokens* kJoinSlots) void join_stats_kernel(const float2* __restrict__ partial, int64_t slots,
                                                                            const float* __restrict__ target_logit,
                                                                            const void* targets, int32_t targets64, int64_t vocab,
                                                                            int64_t n, float* loss, float* lse) {
    __shared__ float tops[kJoinSlots][kJoinTokens], sums[kJoinSlots][kJoinTokens];
    const int x = threadIdx.x % kJoinTokens, y = threadIdx.x / kJoinTokens;
    const int64_t token = (int64_t)blockIdx.x * kJoinTokens + x;
    float top = -INFINITY, sum = 0.0f;
    if (token < n)
        for (int64_t s0 = y; s0 < slots; s0 += 8 * kJoinSlots) {
            float2 p[8];  // loaded together: with one token the loads' latency is the time
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                const int64_t s = s0 + u * kJoinSlots;
                p[u] = s < slots ? partial[s * n + token] : make_float2(-INFINITY, 0.0f);
            }
            float t = top;
#pragma unroll
            for (int u = 0; u < 8; ++u) t = fmaxf(t, p[u].x);
            // a slot beyond the vocabulary has maximum -inf and sum 0 (one of
            // NaN logits has sum NaN, which stays)
            const float base = base_of(t);
            sum = sum == 0.0f ? 0.0f : sum * __builtin_amdgcn_exp2f((base_of(top) - base) * kLog2e);
#pragma unroll
            for (int u = 0; u < 8; ++u) sum += p[u].y == 0.0f ? 0.0f : p[u].y * __builtin_amdgcn_exp2f((base_of(p[u].x) - base) * kLog2e);
            top = t;
        }
    tops[y][x] = top;
    sums[y][x] = sum;
    __syncthreads();
#pragma unroll
    for (int half = kJoinSlots / 2; half > 0; half >>= 1) {
        if (y < half) {
            const float a = tops[y][x], b = tops[y + half][x], t = fmaxf(a, b);
            const float sa = sums[y][x], sb = sums[y + half][x];
            tops[y][x] = t;
            sums[y][x] = (sa == 0.0f ? 0.0f : sa * __builtin_amdgcn_exp2f((base_of(a) - base_of(t)) * kLog2e)) +
                         (sb == 0.0f ? 0.0f : sb * __builtin_amdgcn_exp2f((base_of(b) - base_of(t)) * kLog2e));
        }
        __syncthreads();
    }
    if (y != 0 || token >= n) return;
    const float l = base_of(tops[0][x]) + logf(sums[0][x]);
    lse[token] = l;
    loss[token] = target_of(targets, targets64, token, vocab) < 0 ? 0.0f : l - target_logit[token];
}

// Rows with a width or alignment that 16-byte loads cannot take, copied into
// rows of `width` elements with zeros at the end.
// T: the widest unit that rows start on and are a multiple of.
template <class T>
__global__ __launch_bounds__(256) void pad_rows_kernel(const T* __restrict__ src, int64_t ld, int64_t rows, int64_t dim,
                                                       T* __restrict__ dst, int64_t width) {
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < rows * width; i += (int64_t)gridDim.x * 256) {
        const int64_t r = i / width, c = i - r * width;
        dst[i] = c < dim ? src[r * ld + c] : (T)0;
    }
}

// What the gradient starts from.  The first workgroup finds the largest |dloss|
// of the tokens that count (1 where there is none).  The others copy the hidden
// rows into rows of `width` units with zeros at the end, and zeros for a token
// without a target: in dW = dz^T h its dz of 0 would not keep a NaN or infinity
// out.  They stand there `parts` times, once for each part of dz.  T: the widest
// unit that rows start on and are a multiple of.
constexpr int kPrepareThreads = 1024, kPrepareRows = kPrepareThreads / 64;
template <class T>
__global__ __launch_bounds__(kPrepareThreads) void prepare_grad_kernel(const float* __restrict__ dloss, const void* targets,
                                                                       int32_t targets64, int64_t vocab, int64_t n, float* unit,
                                                                       const T* __restrict__ src, int64_t ld, int64_t dim,
                                                                       T* __restrict__ dst, int64_t width, int32_t parts) {
    if (blockIdx.x > 0) {
        const int lane = threadIdx.x & 63;
        for (int64_t token = (int64_t)(blockIdx.x - 1) * kPrepareRows + (threadIdx.x >> 6); token < n;
             token += (int64_t)(gridDim.x - 1) * kPrepareRows) {
            const bool counts = target_of(targets, targets64, token, vocab) >= 0;
            for (int64_t c = lane; c < width; c += 64) {
                const T x = counts && c < dim ? src[token * ld + c] : T{};
                for (int32_t k = 0; k < parts; ++k) dst[(k * n + token) * width + c] = x;
            }
        }
        return;
    }
    __shared__ float tops[16];
    float top = 0.0f;
    for (int64_t i = threadIdx.x; i < n; i += kPrepareThreads)
        if (target_of(targets, targets64, i, vocab) >= 0) top = fmaxf(top, fabsf(dloss[i]));
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor(top, off, 64));
    if ((threadIdx.x & 63) == 0) tops[threadIdx.x >> 6] = top;
    __syncthreads();
    if (threadIdx.x != 0) return;
    for (int k = 1; k < 16; ++k) top = fmaxf(top, tops[k]);
    *unit = top > 0.0f && top < INFINITY ? top : 1.0f;
}

// dh = unit * sum of the slabs, rounded to bf16.
__global__ __launch_bounds__(256) void finish_hidden_kernel(const float* __restrict__ sums, int64_t slab, int32_t slabs, int64_t ld,
                                                            int64_t dim, int64_t n, const float* __restrict__ unit,
                                                            bf16_t* __restrict__ out, int64_t out_ld, int32_t vec) {
    const float whole = *unit;
    const int64_t quads = (dim + 3) / 4;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n * quads; i += (int64_t)gridDim.x * 256) {
        const int64_t token = i / quads, c = 4 * (i - token * quads);
        f32x4 x = {0.0f, 0.0f, 0.0f, 0.0f};
        for (int32_t s = 0; s < slabs; ++s) x += *reinterpret_cast<const f32x4*>(sums + s * slab + token * ld + c);
        x *= whole;
        bf16_t* p = out + token * out_ld + c;
        if (vec) {
            const u32x2 y = {pack2<bf16_t>(x[0], x[1]), pack2<bf16_t>(x[2], x[3])};
            *reinterpret_cast<u32x2*>(p) = y;
        } else {
            for (int l = 0; l < 4 && c + l < dim; ++l) p[l] = Elem<bf16_t>::to(x[l]);
        }
    }
}

// ---- host -------------------------------------------------------------------

int64_t up(int64_t x, int64_t a) { return (x + a - 1) / a * a; }

constexpr int waves_m_of(int bn) { return bn == 64 ? 8 : 4; }

// Time of a product of `tiles` 256 x bn tiles and `steps` steps of k, in
// microseconds, fitted to what the kernels take (8 shapes from 100 x 100000 x
// 512 to 8192 x 32768 x 4096): a step of a 256-wide tile takes 1.2 us on an idle
// device and 1.6 on a full one, of a 128-wide one 0.8 to 1.06, of a 64-wide one
// 0.72 to 0.82, and 1.06 where two such workgroups share a CU.  A tile's first
// loads and its epilogue take about four steps' time.
double product_us(int64_t tiles, int bn, int64_t steps) {
    const double load = double(std::min<int64_t>(tiles, 256)) / 256;
    if (bn == 64 && tiles > 256) return double((tiles + 511) / 512) * 1.06 * double(steps + 4);
    const double step = bn == 256 ? 1.2 + 0.4 * load : bn == 128 ? 0.8 + 0.26 * load : 0.72 + 0.1 * load;
    return double((tiles + 255) / 256) * step * double(steps + 4);
}

constexpr int kWidths[] = {256, 128, 64};

// Rows of a product's long side that fill whole rounds of the device with
// 256-wide tiles, and the width for the rest, where that beats one width for
// all (1013 x 50001 x 1000 has 3.06 rounds of tiles).
struct Rows {
    int64_t full;  // rows of the first launch, 0: none
    int bn;        // width of the only, or second, launch
};

// Width in tokens of the logits' tiles: wide ones reuse more, narrow ones
// fill the device and its last round (512 x 16384 x 2048: 607, 907 and 861
// TFLOP/s at 256, 128 and 64; 1013 x 50001 x 1000: 644, 531 and 499).
// `kFewTokens` tokens and less are read without LDS.
int best_width(int64_t n, int64_t rows, int64_t dim, double* least) {
    int best = 0;
    for (int bn : kWidths) {
        const double us = product_us(up(rows, kBM) / kBM * (up(n, bn) / bn), bn, up(dim, kBK) / kBK);
        if (!best || us < *least) best = bn, *least = us;
    }
    return best;
}
Rows logits_rows(int64_t n, int64_t rows, int64_t dim, double* us = nullptr) {
    double whole = 0.0, rest;
    if (n <= kFewTokens) return Rows{0, kFewTokens};
    const int bn = best_width(n, rows, dim, &whole);
    if (us) *us = whole;
    const int64_t across = up(n, 256) / 256, tiles = up(rows, kBM) / kBM * across;
    const int64_t full = tiles / 256 * 256 / across * kBM;
    if (full == 0 || full >= rows) return Rows{0, bn};
    const int rest_bn = best_width(n, rows - full, dim, &rest);
    const double both = product_us(full / kBM * across, 256, up(dim, kBK) / kBK) + rest;
    if (both >= whole) return Rows{0, bn};
    if (us) *us = both;
    return Rows{full, rest_bn};
}
double logits_us(int64_t n, int64_t rows, int64_t dim) {
    double us = double(rows) * double(dim) * 5e-7;  // few tokens: bound by the weights
    logits_rows(n, rows, dim, &us);
    return us;
}

// Of dh: few tiles and a long k (the piece's rows), so k is split too; each
// split's binary32 sums are written and read again at the end, at some 5 TB/s.
// Chosen against measured (microseconds, both kernels): 1013 x 50001 x 1000
// 256 wide in 16 (101; in 4: 263, 64 wide in 8: 114), 512 x 16384 x 2048 128
// wide in 8 (44; 256 wide in 16: 49), 2048 x 32768 x 4096 256 wide in 2 (437;
// in 1: 715, in 4: 459).
struct HiddenShape {
    int bn, splits;
};
constexpr int64_t kSplitTokens = 16384;  // splits times tokens, unless there are more tokens
int64_t most_splits(int64_t n) { return std::max<int64_t>(1, std::min<int64_t>(64, kSplitTokens / std::max<int64_t>(n, 1))); }
HiddenShape hidden_shape(int64_t n, int64_t dim, int64_t piece, double* product = nullptr) {
    HiddenShape best{0, 1};
    double least = 0.0;
    for (int bn : kWidths)
        for (int s = 1; s <= most_splits(n) && (s == 1 || piece / s >= 256); s += s < 16 ? 1 : 8) {
            const int64_t tiles = up(dim, kBM) / kBM * (up(n, bn) / bn);
            const double one = product_us(tiles * s, bn, up(piece, kBK) / kBK / s);
            const double us = one + 1.6e-6 * double(n) * double(dim) * s;
            if (!best.bn || us < least) {
                best = HiddenShape{bn, s}, least = us;
                if (product) *product = one;
            }
        }
    return best;
}

// Vocabulary rows of a piece.  Longer pieces have fewer half-filled rounds and
// add to dh's sums less often; a dz of 128 MiB stays in the last-level cache,
// where its products read it (8192 x 131072 x 4096: dz 7.34 ms in pieces of 8192
// rows, 8.05 in pieces of 32768, the three products 20.6 and 21.2 ms; but 4000 x
// 100000 x 2048: 4.96 ms in seven pieces, 4.26 in one of 128 MiB or 1 GiB of dz).
// Chosen by the modelled time; a piece's dz and a padded bf16 copy of its
// weights take 512 MiB each, or those of 1024 rows
// (dz in two parts: half the rows).
constexpr int64_t kPieceBytes = int64_t(1) << 29, kLeastRows = 1024;
double piece_us(int64_t n, int64_t rows, int64_t dim, int parts) {
    double hidden;
    hidden_shape(n, dim, rows, &hidden);
    const double z = logits_us(n, rows, dim) * (2 * parts * n * rows > (int64_t(128) << 20) ? 1.08 : 1.0);
    const double weight = product_us(up(dim, kBM) / kBM * (up(rows, 256) / 256), 256, up(parts * n, kBK) / kBK);
    return z + hidden + weight + 15.0;
}
int64_t piece_rows(int64_t n, int64_t vocab, int64_t dim, int parts) {
    int64_t best = 0;
    double least = 0.0;
    for (int64_t most = kPieceBytes / 4; most <= kPieceBytes; most *= 2) {
        const int64_t by_dz = most / (2 * parts * std::max<int64_t>(n, 1)), by_copy = kPieceBytes / (2 * up(dim, 64));
        const int64_t rows = std::min(std::max(kLeastRows / parts, std::min(by_dz, by_copy) / 256 * 256), up(vocab, 256));
        const int64_t full = vocab / rows, rest = vocab - full * rows;
        const double us = double(full) * piece_us(n, rows, dim, parts) + (rest ? piece_us(n, rest, dim, parts) : 0.0) +
                          3e-7 * double(full + (rest > 0) - 1) * double(n) * double(dim);
        if (!best || us < least) best = rows, least = us;
        if (rows >= vocab) break;
    }
    return best;
}

// Partial statistics of a token: one for each wave's rows, 8 of a tile at most
// (a tile of few tokens has one for 32 rows).
int64_t stat_slots(int64_t rows, int width) {
    return width == kFewTokens ? up(rows, kFewRows) / kFewRows : up(rows, kBM) / kBM * waves_m_of(width);
}
int64_t most_slots(int64_t vocab) { return up(vocab, kBM) / kBM * 8; }

struct Work {
    float2* partial;
    float* target_logit;
    void *hidden, *weight;  // padded copies
    bf16_t* dz;
    float* sums;
    float* unit;
    int64_t bytes;
};

// Each part is as large as any count of tokens up to n needs it (pieces and
// splits change with n), so that a workspace serves the last, shorter batch too.
Work work_of(void* work, int64_t n, int64_t vocab, int64_t dim, int fp8, int grad) {
    Work w{};
    char* p = static_cast<char*>(work);
    int64_t at = 0;
    const auto take = [&](int64_t bytes) {
        char* q = p + at;
        at += up(bytes, 256);
        return q;
    };
    const int64_t width = up(dim, 64), rows = up(vocab, 256), esize = fp8 ? 1 : 2;
    w.hidden = take(n * width * 2 * (grad ? 2 : 1));
    w.weight = take(std::min(std::max(kPieceBytes / 2, kLeastRows * width), rows * width) * esize);
    const int64_t mark = at;
    // the loss and its gradient run one after the other: one space for both
    w.partial = reinterpret_cast<float2*>(take(most_slots(vocab) * n * 8));
    w.target_logit = reinterpret_cast<float*>(take(n * 4));
    w.bytes = at;
    if (grad) {
        at = mark;
        w.unit = reinterpret_cast<float*>(take(4));
        w.dz = reinterpret_cast<bf16_t*>(take(std::min(std::max(kPieceBytes, n * kLeastRows * 2), n * rows * 4)));
        w.sums = reinterpret_cast<float*>(take(std::min(64 * n, std::max(kSplitTokens, n)) * width * 4));
        w.bytes = std::max(w.bytes, at);
    }
    return w;
}

hipError_t allow_lds(const void* kernel, int bytes, std::atomic<uint64_t>& ready) {
    int dev = 0;
    hipError_t err = hipGetDevice(&dev);
    if (err != hipSuccess) return err;
    const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
    if (!bit || !(ready.load(std::memory_order_acquire) & bit)) {
        err = hipFuncSetAttribute(kernel, hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (err != hipSuccess) return err;
        ready.fetch_or(bit, std::memory_order_release);
    }
    return hipSuccess;
}

template <class A, class B, int kBN, int kWavesM, class Epilogue>
int launch_gemm(GemmArgs g, const Epilogue& e, void* stream) {
    static std::atomic<uint64_t> ready{0};
    constexpr int kLds = 2 * (A::kBytes + B::kBytes);
    const auto kernel = gemm_kernel<A, B, kBN, kWavesM, Epilogue>;
    hipError_t err = allow_lds(reinterpret_cast<const void*>(kernel), kLds, ready);
    if (err != hipSuccess) return err;
    g.tiles_m = (int32_t)(up(g.a.extent, kBM) / kBM);
    g.tiles_n = (int32_t)(up(g.b.extent, kBN) / kBN);
    if (g.splits < 1) g.splits = 1;
    g.k_per_split = up((g.k + g.splits - 1) / g.splits, 128);
    // Tiles of m in a group, 2/4/8/16: logits of 8192 x 131072 x 4096 at 1328/
    // 1350/1344/1290 TFLOP/s in BF16 and 1252/1280/1282/1228 in FP8, of 2048 x
    // 32768 x 4096 at 1150/1174/1173/1125 and 1076/1069/1111/1096.
    g.group_m = 8;
    hipLaunchKernelGGL(kernel, dim3((uint32_t)(g.tiles_m * g.tiles_n * g.splits)), dim3(kGemmThreads), kLds, (hipStream_t)stream, g, e);
    return hipGetLastError();
}

// A product whose A is a piece of the weights with k (or m) in its rows and
// whose B has tokens in its rows.
template <template <int> class A, int kBN, class Epilogue>
int launch_kc(const GemmArgs& g, const Epilogue& e, void* stream) {
    return launch_gemm<A<kBM>, BF16KC<kBN>, kBN, waves_m_of(kBN), Epilogue>(g, e, stream);
}
template <template <int, int> class A, int kBN, class Epilogue>
int launch_kr(const GemmArgs& g, const Epilogue& e, void* stream) {
    constexpr int kWavesM = waves_m_of(kBN);
    return launch_gemm<A<kBM, kBM / kWavesM / 16>, BF16KC<kBN>, kBN, kWavesM, Epilogue>(g, e, stream);
}

template <bool kFp8, class Epilogue>
int launch_few(const GemmArgs& g, const Epilogue& e, void* stream) {
    const uint32_t blocks = (uint32_t)(up(g.a.extent, kFewRows) / kFewRows);
    hipLaunchKernelGGL((few_tokens_kernel<kFp8, Epilogue>), dim3(blocks), dim3(64 * kFewWaves), 0, (hipStream_t)stream, g, e);
    return hipGetLastError();
}

template <class Epilogue>
int logits_launch(int fp8, int width, const GemmArgs& g, const Epilogue& e, void* stream) {
    switch (width) {
        case kFewTokens: return fp8 ? launch_few<true>(g, e, stream) : launch_few<false>(g, e, stream);
        case 64: return fp8 ? launch_kc<FP8KC, 64>(g, e, stream) : launch_kc<BF16KC, 64>(g, e, stream);
        case 128: return fp8 ? launch_kc<FP8KC, 128>(g, e, stream) : launch_kc<BF16KC, 128>(g, e, stream);
        default: return fp8 ? launch_kc<FP8KC, 256>(g, e, stream) : launch_kc<BF16KC, 256>(g, e, stream);
    }
}

int hidden_grad(int fp8, int bn, const GemmArgs& g, const SumEpilogue& e, void* stream) {
    switch (bn) {
        case 64: return fp8 ? launch_kr<FP8KR, 64>(g, e, stream) : launch_kr<BF16KR, 64>(g, e, stream);
        case 128: return fp8 ? launch_kr<FP8KR, 128>(g, e, stream) : launch_kr<BF16KR, 128>(g, e, stream);
        default: return fp8 ? launch_kr<FP8KR, 256>(g, e, stream) : launch_kr<BF16KR, 256>(g, e, stream);
    }
}

// All sizes in bytes.
int pad_rows(const void* src, int64_t ld, int64_t rows, int64_t dim, void* dst, int64_t width, void* stream) {
    const uint64_t marks = reinterpret_cast<uintptr_t>(src) | (uint64_t)ld | (uint64_t)dim;
    const auto launch = [&](auto unit) {
        typedef decltype(unit) T;
        const int64_t n = rows * width / (int64_t)sizeof(T);
        hipLaunchKernelGGL(pad_rows_kernel<T>, dim3((uint32_t)std::min<int64_t>((n + 255) / 256, 1 << 20)), dim3(256), 0,
                           (hipStream_t)stream, static_cast<const T*>(src), ld / (int64_t)sizeof(T), rows, dim / (int64_t)sizeof(T),
                           static_cast<T*>(dst), width / (int64_t)sizeof(T));
        return (int)hipGetLastError();
    };
    if (marks % 8 == 0) return launch(uint64_t{});
    if (marks % 4 == 0) return launch(uint32_t{});
    if (marks % 2 == 0) return launch(uint16_t{});
    return launch(uint8_t{});
}

bool loadable(const void* p, int64_t ld, int64_t dim, int size) {
    return dim * size % 16 == 0 && ld * size % 16 == 0 && reinterpret_cast<uintptr_t>(p) % 16 == 0;
}

// The operands as the products read them: in place where rows suit 16-byte
// loads, else padded copies (the weights' by pieces).  dW reads a copy of h
// always, in which tokens without a target are zero (8192 x 4096: 25 us with the
// largest dloss, 8 without the copy, of a gradient of 20 ms).
struct Source {
    Operand hidden;      // rows of tokens
    bool copy_weight;
    int64_t width, esize;
};

Source source_of(const VocabLossArgs& a, const Work& w, bool copy_hidden) {
    Source s;
    s.width = up(a.dim, 64);
    s.esize = a.fp8 ? 1 : 2;
    s.copy_weight = !loadable(a.weight, a.weight_ld, a.dim, (int)s.esize);
    s.hidden = copy_hidden ? Operand{w.hidden, s.width * 2, a.n, s.width} : Operand{a.hidden, a.hidden_ld * 2, a.n, a.dim};
    return s;
}

int prepare_grad(const VocabLossArgs& a, const Work& w, int64_t width, bool copy_hidden, void* stream) {
    const uint64_t marks = reinterpret_cast<uintptr_t>(a.hidden) | (uint64_t)(a.hidden_ld * 2) | (uint64_t)(a.dim * 2);
    const auto launch = [&](auto unit) {
        typedef decltype(unit) T;
        constexpr int kPer = (int)sizeof(T) / 2;
        const int64_t copies = copy_hidden ? std::min<int64_t>((a.n + kPrepareRows - 1) / kPrepareRows, 4096) : 0;
        hipLaunchKernelGGL(prepare_grad_kernel<T>, dim3((uint32_t)(1 + copies)), dim3(kPrepareThreads), 0, (hipStream_t)stream,
                           a.dloss, a.targets, a.targets64, a.vocab, a.n, w.unit, static_cast<const T*>(a.hidden),
                           a.hidden_ld / kPer, a.dim / kPer, static_cast<T*>(w.hidden), width / kPer, a.dz_parts);
        return (int)hipGetLastError();
    };
    if (marks % 16 == 0) return launch(u32x4{});
    if (marks % 4 == 0) return launch(uint32_t{});
    return launch(uint16_t{});
}

// Rows [first, first + rows) of the weights, rows in extent and dim in k.
int weight_piece(const VocabLossArgs& a, const Work& w, const Source& s, int64_t first, int64_t rows, Operand* o, void* stream) {
    const char* p = static_cast<const char*>(a.weight) + first * a.weight_ld * s.esize;
    if (!s.copy_weight) {
        *o = Operand{p, a.weight_ld * s.esize, rows, a.dim};
        return hipSuccess;
    }
    *o = Operand{w.weight, s.width * s.esize, rows, s.width};
    return pad_rows(p, a.weight_ld * s.esize, rows, a.dim * s.esize, w.weight, s.width * s.esize, stream);
}

// The tile scales of the piece that starts at vocabulary row `first`.
void set_grid(const VocabLossArgs& a, int64_t first, bool vocab_is_m, GemmArgs* g) {
    if (!a.fp8) return;
    const int64_t hb = up(a.vocab, kTileDim) / kTileDim, wb = up(a.dim, kTileDim) / kTileDim;
    g->grid = a.grid + first / kTileDim * wb;
    const int64_t rows = hb - first / kTileDim;
    g->grid_m = vocab_is_m ? wb : 1;
    g->grid_k = vocab_is_m ? 1 : wb;
    g->blocks_m = vocab_is_m ? rows : wb;
    g->blocks_k = vocab_is_m ? wb : rows;
}

// The logits of `rows` vocabulary rows from `first`, read from `weight`, in one
// launch or two; epilogue(at, count, width) gives that of rows [at, at + count)
// of them.
template <class F>
int logits(const VocabLossArgs& a, const Source& s, const Operand& weight, int64_t first, int64_t rows, F&& epilogue, void* stream) {
    const Rows r = logits_rows(a.n, rows, a.dim);
    for (int64_t at = 0; at < rows;) {
        const int64_t count = at < r.full ? r.full : rows - at;
        const int width = at < r.full ? 256 : r.bn;
        GemmArgs g{};
        g.a = Operand{static_cast<const char*>(weight.p) + at * weight.ld, weight.ld, count, weight.k};
        g.b = s.hidden;
        g.k = a.dim;
        set_grid(a, first + at, true, &g);
        const auto e = epilogue(at, count, width);
        const int err = logits_launch(a.fp8, width, g, e, stream);
        if (err) return err;
        at += count;
    }
    return hipSuccess;
}

template <class O>
int weight_grad_launch(const VocabLossArgs& a, const Work& w, const GemmArgs& d, int64_t rows, int64_t width, const WeightGradEpilogue<O>& e,
                       void* stream) {
    if (a.n > kFewTokens) return launch_gemm<BF16KR<kBM, 8>, BF16KR<256, 4>, 256, 2, WeightGradEpilogue<O>>(d, e, stream);
    const dim3 grid((uint32_t)((rows + kFewGradRows - 1) / kFewGradRows), (uint32_t)((a.dim + 256 * kFewGradCols - 1) / (256 * kFewGradCols)));
    hipLaunchKernelGGL(few_weight_grad_kernel<O>, grid, dim3(256), 0, (hipStream_t)stream, static_cast<const bf16_t*>(a.hidden),
                       a.hidden_ld, a.dim, w.dz, a.dz_parts > 1 ? w.dz + a.n * width : nullptr, width, a.n, rows, a.targets, a.targets64, e);
    return hipGetLastError();
}

// Rows [first, first + rows) of dW = dz^T h: m is the hidden width, n the
// vocabulary rows.
int weight_grad(const VocabLossArgs& a, const Work& w, const Source& s, int64_t first, int64_t rows, int64_t width, void* stream) {
    GemmArgs d{};
    d.k = a.dz_parts * a.n;
    d.a = Operand{s.hidden.p, s.hidden.ld, s.hidden.k, d.k};
    d.b = Operand{w.dz, width * 2, rows, d.k};
    const bool f32 = a.dweight_type == kF32;
    const int32_t vec = a.dweight_ld % 4 == 0 && reinterpret_cast<uintptr_t>(a.dweight) % (f32 ? 16 : 8) == 0;
    if (f32) {
        const WeightGradEpilogue<float> e{static_cast<float*>(a.dweight), a.dweight_ld, a.dim, first, a.vocab, w.unit, a.accumulate, vec};
        return weight_grad_launch<float>(a, w, d, rows, width, e, stream);
    }
    const WeightGradEpilogue<bf16_t> e{static_cast<bf16_t*>(a.dweight), a.dweight_ld, a.dim, first, a.vocab, w.unit, a.accumulate, vec};
    return weight_grad_launch<bf16_t>(a, w, d, rows, width, e, stream);
}

}  // namespace

int64_t vocab_loss_work_bytes(int64_t n, int64_t vocab, int64_t dim, int fp8, int grad) {
    return work_of(nullptr, n, vocab, dim, fp8, grad).bytes;
}

int launch_vocab_loss(const VocabLossArgs& a, void* work, void* stream) {
    if (a.n == 0) return hipSuccess;
    const Work w = work_of(work, a.n, a.vocab, a.dim, a.fp8, 0);
    const bool copy_hidden = !loadable(a.hidden, a.hidden_ld, a.dim, 2);
    const Source s = source_of(a, w, copy_hidden);
    int err = copy_hidden ? pad_rows(a.hidden, a.hidden_ld * 2, a.n, a.dim * 2, w.hidden, s.width * 2, stream) : hipSuccess;
    if (err) return err;
    const int64_t piece = s.copy_weight ? piece_rows(a.n, a.vocab, a.dim, 1) : a.vocab;
    int64_t slots = 0;
    for (int64_t first = 0; first < a.vocab; first += piece) {
        const int64_t rows = std::min(piece, a.vocab - first);
        Operand weight;
        err = weight_piece(a, w, s, first, rows, &weight, stream);
        if (err) return err;
        err = logits(a, s, weight, first, rows, [&](int64_t at, int64_t count, int width) {
            const StatsEpilogue e{w.partial, w.target_logit, a.targets, a.targets64, first + at, a.vocab, a.n, slots,
                                  width == kFewTokens ? 1 : waves_m_of(width)};
            slots += stat_slots(count, width);
            return e;
        }, stream);
        if (err) return err;
    }
    hipLaunchKernelGGL(join_stats_kernel, dim3((uint32_t)(up(a.n, kJoinTokens) / kJoinTokens)), dim3(kJoinTokens * kJoinSlots), 0,
                       (hipStream_t)stream, w.partial, slots, w.target_logit, a.targets, a.targets64, a.vocab, a.n, a.loss, a.lse);
    return hipGetLastError();
}

int launch_vocab_loss_grad(const VocabLossArgs& a, void* work, void* stream) {
    const Work w = work_of(work, a.n, a.vocab, a.dim, a.fp8, 1);
    // dW of few tokens reads h itself
    const bool copy_hidden = a.n > 0 && ((a.dweight && a.n > kFewTokens) || !loadable(a.hidden, a.hidden_ld, a.dim, 2));
    const Source s = source_of(a, w, copy_hidden);
    int err = prepare_grad(a, w, s.width, copy_hidden, stream);
    if (err) return err;
    const int64_t piece = piece_rows(a.n, a.vocab, a.dim, a.dz_parts);
    const HiddenShape shape = hidden_shape(a.n, a.dim, piece);
    for (int64_t first = 0; first < a.vocab; first += piece) {
        const int64_t rows = std::min(piece, a.vocab - first);
        const int64_t width = up(rows, kBM);
        Operand weight{};
        if (a.n > 0) {
            err = weight_piece(a, w, s, first, rows, &weight, stream);
            if (err) return err;
            err = logits(a, s, weight, first, rows, [&](int64_t at, int64_t, int) {
                return LogitGradEpilogue{w.dz + at, a.dz_parts > 1 ? w.dz + a.n * width + at : nullptr, width, first + at, a.vocab, a.n, a.lse, a.dloss, w.unit, a.targets, a.targets64};
            }, stream);
            if (err) return err;
        }
        if (a.dhidden && a.n > 0) {
            GemmArgs h{};
            h.a = Operand{weight.p, weight.ld, weight.k, rows};
            h.b = Operand{w.dz, width * 2, a.n, up(rows, kFewRows)};  // written that far, zeros at the end
            h.k = rows;
            h.splits = shape.splits;
            set_grid(a, first, false, &h);
            const SumEpilogue e{w.sums, s.width, a.n * s.width, s.width, a.n, first > 0};
            err = hidden_grad(a.fp8, shape.bn, h, e, stream);
            if (err) return err;
        }
        if (a.dweight) {
            err = weight_grad(a, w, s, first, rows, width, stream);
            if (err) return err;
        }
    }
    if (!a.dhidden || a.n == 0) return hipSuccess;
    const int32_t vec = a.dim % 4 == 0 && a.dhidden_ld % 4 == 0 && reinterpret_cast<uintptr_t>(a.dhidden) % 8 == 0;
    const int64_t quads = a.n * ((a.dim + 3) / 4);
    hipLaunchKernelGGL(finish_hidden_kernel, dim3((uint32_t)std::min<int64_t>((quads + 255) / 256, 16384)), dim3(256), 0,
                       (hipStream_t)stream, w.sums, a.n * s.width, shape.splits, s.width, a.dim, a.n, w.unit,
                       static_cast<bf16_t*>(a.dhidden), a.dhidden_ld, vec);
    return hipGetLastError();
}

}  // namespace bfz

extern "C" int bfz_vocab_loss_shape(int64_t n, int64_t vocab, int64_t dim, int32_t dweight_dtype, int64_t* shape) {
    using namespace bfz;
    if (!shape || n < 1 || vocab < 1 || dim < 1 || n > (int64_t(1) << 24) || vocab > (int64_t(1) << 27) || dim > (int64_t(1) << 20))
        return fail(BFZ_EINVAL, "bfz_vocab_loss_shape: null pointer or bad sizes");
    const Rows loss = logits_rows(n, vocab, dim);
    const int64_t piece = piece_rows(n, vocab, dim, dweight_dtype == kF32 ? 2 : 1);
    const Rows grad = logits_rows(n, std::min(piece, vocab), dim);
    const HiddenShape hidden = hidden_shape(n, dim, piece);
    const int64_t out[7] = {loss.full, loss.bn, piece, grad.full, grad.bn, hidden.bn, hidden.splits};
    std::copy(out, out + 7, shape);
    return BFZ_OK;
}
