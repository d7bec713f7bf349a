// Global gradient norm over many tensors, and clipping.
//
//   s = sum g^2,  norm = sqrt(s),  coef = min(1, max_norm / (norm + 1e-6)),
//   g' = g * coef
//
// Squares and sums are binary64: a binary32 square neither overflows nor
// underflows there, and a sum over 10^9 terms keeps 2^-53 * sqrt(10^9) of
// relative error.  The sum's order is fixed by the sizes alone: each
// workgroup takes a fixed share, adds its threads in a tree, and the last workgroup to finish adds the G partial sums in index order, so
// two runs give the same bits.
//
// Bound by reading the gradients, at few of them by the launch: 40 ragged
// tensors of 70.5M elements, half of them bf16, 46 us (4.6 TB/s), clipped into
// f32 buffers in another 104 us (4.7 TB/s); the tiles of a 202M-element shard
// 131 us (6.2 TB/s); one 256 x 384 tensor 5.2 us of a 7 us call.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "ops_internal.h"
#include "ops_device.h"

#pragma clang fp contract(off)

namespace bfz {
namespace {

constexpr int kThreads = 256;

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ double square_add(double acc, float x) {
    const double d = (double)x;
    return __builtin_fma(d, d, acc);  // the product of two binary32 is exact in binary64
}

// Elements [lo, hi) of a 16-byte block of 16 / sizeof(T) elements.
template <class T>
__device__ __forceinline__ double add_block(double acc, const u32x4& raw, int lo, int hi) {
    constexpr int kPer = 16 / sizeof(T);
#pragma unroll
    for (int l = 0; l < kPer; ++l) {
        const float x = Elem<T>::from_block(raw, l);
        acc = square_add(acc, l >= lo && l < hi ? x : 0.0f);
    }
    return acc;
}

// Squares of elements [e0, e1) of a tensor at any element alignment: whole
// 16-byte blocks from the boundary below, the ends masked.  A block is read
// only if it holds an element of the range, and an aligned 16-byte block
// never crosses a page.
template <class T>
__device__ __forceinline__ double sum_range(const T* p, int64_t e0, int64_t e1, double acc) {
    constexpr int kPer = 16 / sizeof(T);
    constexpr int kUnroll = 4;
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(p + e0);
    const int skew = (int)((a0 & 15u) / sizeof(T));
    const u32x4* blk = reinterpret_cast<const u32x4*>(a0 & ~uintptr_t(15));
    const int64_t n = e1 - e0 + skew;  // elements from the first block's start
    const int64_t blocks = (n + kPer - 1) / kPer;
    const int64_t whole = n / kPer;    // blocks with no masked end
    double acc2 = 0.0;
    for (int64_t b0 = threadIdx.x; b0 < blocks; b0 += kUnroll * kThreads) {
        if (b0 + (kUnroll - 1) * kThreads < whole && (skew == 0 || b0 > 0)) {
            u32x4 x[kUnroll];
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) x[u] = __builtin_nontemporal_load(blk + b0 + u * kThreads);
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                if (u & 1) acc2 = add_block<T>(acc2, x[u], 0, kPer);
                else acc = add_block<T>(acc, x[u], 0, kPer);
            }
        } else {
            for (int u = 0; u < kUnroll; ++u) {
                const int64_t b = b0 + u * kThreads;
                if (b >= blocks) break;
                const int hi = (int)(n - b * kPer < kPer ? n - b * kPer : kPer);
                acc = add_block<T>(acc, __builtin_nontemporal_load(blk + b), b == 0 ? skew : 0, hi);
            }
        }
    }
    return acc + acc2;
}

// Sum of acc over the workgroup, in a fixed order; valid in thread 0.
__device__ __forceinline__ double block_sum(double acc, double* lds) {
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) acc += __shfl_xor(acc, off, 64);
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = acc;
    __syncthreads();
    double s = lds[0];
#pragma unroll
    for (int w = 1; w < kThreads / 64; ++w) s += lds[w];
    __syncthreads();
    return s;
}

__device__ __forceinline__ void write_coef(double sumsq, double max_norm, float* norm, float* coef) {
    const double n = sqrt(sumsq);
    if (norm) *norm = (float)n;
    if (coef) {
        const double c = max_norm / (n + 1e-6);
        *coef = c >= 1.0 ? 1.0f : (float)c;  // NaN stays NaN
    }
}

// The end of a sum kernel: publish this workgroup's partial; the last one to
// arrive adds them all (thread t takes t, t + 256, ...), adds the earlier
// launches' sum and, in the last launch, writes the results.  The partials
// cross XCDs, whose L2s are separate: they are written, counted and read with
// agent-scope atomics, which act beyond the L2s, and the wait puts a
// workgroup's partial there before it is counted.  That is this hardware's
// promise, of device-scope stores and vmcnt, not the language's, whose release
// would also write the XCD's L2 back once per workgroup: 215 us instead of 152
// for the 40 ragged tensors and their clipping.
__device__ __forceinline__ void finish_sum(double acc, const NormOut& out, void* work) {
    __shared__ double lds[kThreads / 64];
    __shared__ uint32_t arrived;
    NormWork* w = static_cast<NormWork*>(work);
    double* partial = reinterpret_cast<double*>(static_cast<char*>(work) + 64);
    const double s = block_sum(acc, lds);
    if (threadIdx.x == 0) {
        __hip_atomic_store(&partial[blockIdx.x], s, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        __asm__ volatile("s_waitcnt vmcnt(0)" ::: "memory");
        arrived = __hip_atomic_fetch_add(&w->ticket, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    __syncthreads();
    if (arrived != gridDim.x - 1) return;
    double t = 0.0;
    for (uint32_t b = threadIdx.x; b < gridDim.x; b += kThreads)
        t += __hip_atomic_load(&partial[b], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    t = block_sum(t, lds);
    if (threadIdx.x != 0) return;
    if (!out.first) t += w->carry;
    w->carry = t;
    w->ticket = 0;
    if (!out.last) return;
    if (out.sumsq) *out.sumsq = t;
    write_coef(t, out.max_norm, out.norm, out.coef);
}

// Tensor of chunk c: the last one whose first chunk is <= c.
__device__ __forceinline__ int find_tensor(const TensorList& list, uint32_t c) {
    int lo = 0, hi = list.count - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (list.chunk0[mid] <= c) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// Workgroup b takes the consecutive chunks [b C / G, (b + 1) C / G): equal
// shares, and the tensor is searched for once and then walked.
__global__ __launch_bounds__(kThreads) void list_sumsq_kernel(TensorList list, NormOut out, void* work) {
    double acc = 0.0;
    uint32_t c = (uint32_t)((uint64_t)blockIdx.x * list.chunks / gridDim.x);
    const uint32_t end = (uint32_t)((uint64_t)(blockIdx.x + 1) * list.chunks / gridDim.x);
    int k = c < end ? find_tensor(list, c) : 0;
    while (c < end) {
        const uint32_t next = k + 1 < list.count ? list.chunk0[k + 1] : list.chunks;
        const uint32_t stop = next < end ? next : end;
        const int64_t e0 = (int64_t)(c - list.chunk0[k]) * list.chunk_elems;
        const int64_t e1 = (int64_t)(stop - list.chunk0[k]) * list.chunk_elems;
        const int64_t e = e1 < list.n[k] ? e1 : list.n[k];
        switch (list.in_type[k]) {
            case kF32: acc = sum_range((const float*)list.in[k], e0, e, acc); break;
            case kBF16: acc = sum_range((const bf16_t*)list.in[k], e0, e, acc); break;
            default: acc = sum_range((const f16_t*)list.in[k], e0, e, acc); break;
        }
        c = stop;
        ++k;
    }
    finish_sum(acc, out, work);
}

// The same over the tiles one rank owns, read from the row-major weights
// through the plan's table; padding slots add nothing.  Rows are 16-byte
// blocks from the boundary below, ends masked.
__global__ __launch_bounds__(kThreads) void shard_sumsq_kernel(const TileEntry* __restrict__ entries,
                                                               PackArgs grads, int64_t n_slots,
                                                               NormOut out, void* work) {
    double acc = 0.0, acc2 = 0.0;
    for (int64_t slot = blockIdx.x; slot < n_slots; slot += gridDim.x) {
        const TileEntry t = entries[slot];
        if (t.local < 0) continue;
        const float* origin = grads.src[t.local] + t.base;
        const int rows = t.valid_rows, cols = t.valid_cols;
        if ((t.ld & 3) == 0 && (reinterpret_cast<uintptr_t>(origin) & 15u) == 0) {
            // a multiple of 4 columns: each block lies wholly inside or outside
            const int c = 4 * (threadIdx.x & 31), r0 = threadIdx.x >> 5;
            const f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                f32x4 x[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const int r = r0 + 8 * (8 * h + k);
                    x[k] = zero;
                    if (r < rows && c < cols)
                        x[k] = __builtin_nontemporal_load(
                            reinterpret_cast<const f32x4*>(origin + (int64_t)r * t.ld + c));
                }
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    acc = square_add(acc, x[k][0]);
                    acc2 = square_add(acc2, x[k][1]);
                    acc = square_add(acc, x[k][2]);
                    acc2 = square_add(acc2, x[k][3]);
                }
            }
        } else {
            for (int i = threadIdx.x; i < rows * 33; i += kThreads) {
                const int r = i / 33, b = i - 33 * r;
                const uintptr_t a = reinterpret_cast<uintptr_t>(origin + (int64_t)r * t.ld);
                const int skew = (int)((a >> 2) & 3u);
                const int lo = b == 0 ? skew : 0, hi = cols + skew - 4 * b;
                if (hi <= 0) continue;
                const u32x4 x = *(reinterpret_cast<const u32x4*>(a & ~uintptr_t(15)) + b);
                acc = add_block<float>(acc, x, lo, hi < 4 ? hi : 4);
            }
        }
    }
    finish_sum(acc + acc2, out, work);
}

__global__ void clip_coef_kernel(const double* sumsq, double max_norm, float* norm, float* coef) {
    write_coef(*sumsq, max_norm, norm, coef);
}

// out = in * coef over elements [e0, e1): 8 elements per thread and step
// where both ends are 16-byte aligned, one otherwise (64M elements, f32 99 and
// 118 us, bf16 into f32 85 and 124).
template <class I, class O>
__device__ __forceinline__ void clip_range(const I* in, O* out, int64_t e0, int64_t e1, float coef) {
    const bool vec = ((reinterpret_cast<uintptr_t>(in + e0) | reinterpret_cast<uintptr_t>(out + e0)) & 15u) == 0;
    int64_t done = e0;
    if (vec) {
        const int64_t n8 = (e1 - e0) / 8;
        for (int64_t b = threadIdx.x; b < n8; b += kThreads) {
            float x[8];
            load8(in + e0 + 8 * b, x);
#pragma unroll
            for (int l = 0; l < 8; ++l) x[l] *= coef;
            store8(out + e0 + 8 * b, x);
        }
        done = e0 + 8 * n8;
    }
    for (int64_t e = done + threadIdx.x; e < e1; e += kThreads) out[e] = Elem<O>::to(Elem<I>::get(in[e]) * coef);
}

template <class I>
__device__ __forceinline__ void clip_to(const I* in, void* out, int type, int64_t e0, int64_t e1, float coef) {
    switch (type) {
        case kF32: clip_range(in, (float*)out, e0, e1, coef); break;
        case kBF16: clip_range(in, (bf16_t*)out, e0, e1, coef); break;
        default: clip_range(in, (f16_t*)out, e0, e1, coef); break;
    }
}

__global__ __launch_bounds__(kThreads) void clip_kernel(TensorList list, const float* __restrict__ coef_p) {
    const float coef = *coef_p;
    uint32_t c = (uint32_t)((uint64_t)blockIdx.x * list.chunks / gridDim.x);
    const uint32_t end = (uint32_t)((uint64_t)(blockIdx.x + 1) * list.chunks / gridDim.x);
    for (int k = c < end ? find_tensor(list, c) : 0; c < end; ++k) {
        const uint32_t next = k + 1 < list.count ? list.chunk0[k + 1] : list.chunks;
        const uint32_t stop = next < end ? next : end;
        const int64_t e0 = (int64_t)(c - list.chunk0[k]) * list.chunk_elems;
        const int64_t e1 = (int64_t)(stop - list.chunk0[k]) * list.chunk_elems;
        const int64_t e = e1 < list.n[k] ? e1 : list.n[k];
        c = stop;
        // nothing to clip and nowhere else to write it: g * 1 = g
        if (coef == 1.0f && list.in[k] == list.out[k]) continue;
        switch (list.in_type[k]) {
            case kF32: clip_to((const float*)list.in[k], list.out[k], list.out_type[k], e0, e, coef); break;
            case kBF16: clip_to((const bf16_t*)list.in[k], list.out[k], list.out_type[k], e0, e, coef); break;
            default: clip_to((const f16_t*)list.in[k], list.out[k], list.out_type[k], e0, e, coef); break;
        }
    }
}

}  // namespace

int launch_list_sumsq(const TensorList& list, const NormOut& out, void* work, void* stream) {
    const uint32_t blocks = std::max(1u, std::min(list.chunks, (uint32_t)kNormBlocks));
    hipLaunchKernelGGL(list_sumsq_kernel, dim3(blocks), dim3(kThreads), 0, (hipStream_t)stream, list, out, work);
    return hipGetLastError();
}

int launch_shard_sumsq(const TileEntry* d_entries, int64_t n_slots, const PackArgs& grads, const NormOut& out,
                       void* work, void* stream) {
    const uint32_t blocks = (uint32_t)std::max<int64_t>(1, std::min<int64_t>(n_slots, kNormBlocks));
    hipLaunchKernelGGL(shard_sumsq_kernel, dim3(blocks), dim3(kThreads), 0, (hipStream_t)stream, d_entries, grads,
                       n_slots, out, work);
    return hipGetLastError();
}

int launch_clip_coef(const double* sumsq, double max_norm, float* norm, float* coef, void* stream) {
    hipLaunchKernelGGL(clip_coef_kernel, dim3(1), dim3(1), 0, (hipStream_t)stream, sumsq, max_norm, norm, coef);
    return hipGetLastError();
}

int launch_clip(const TensorList& list, const float* coef, void* stream) {
    if (list.chunks == 0) return hipSuccess;
    const uint32_t blocks = std::min(list.chunks, 8192u);
    hipLaunchKernelGGL(clip_kernel, dim3(blocks), dim3(kThreads), 0, (hipStream_t)stream, list, coef);
    return hipGetLastError();
}

}  // namespace bfz
