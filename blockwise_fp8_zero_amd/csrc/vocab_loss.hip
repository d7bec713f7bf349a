// Softmax cross entropy over a large vocabulary, and its gradient, without
// the logits in memory.
//
//   z = h W^T,  lse[n] = log sum_v exp z[n][v],  loss[n] = lse[n] - z[n][t[n]]
//   dz[n][v] = dloss[n] (exp(z[n][v] - lse[n]) - [v = t[n]])
//   dh = dz W,  dW = dz^T h
//
// Forward: one product whose epilogue reduces every 256 logits of a token to
// their maximum and sum of exponentials; a small kernel joins those.  The
// work is 2 N V d operations, bound by the matrix cores once N is a few
// hundred, by reading W below that.
//
// Gradient: 6 N V d operations in three products over pieces of the
// vocabulary.  A piece's logits are computed again and leave the product as
// dz, rounded to bf16 (the matrix cores' input type: each dz is off by at
// most 2^-8 of itself, which the sums over v and n average out); then
// dz W adds onto dh's binary32 sums and dz^T h gives the piece's rows of dW.
// A piece is as large as its dz may be, so that the products stay long.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <atomic>

#include "vocab_gemm.h"

namespace bfz {
namespace {

constexpr float kLog2e = 1.44269504088896340736f;

// 2^x with subnormal results, which the instruction alone gives as zero.
__device__ __forceinline__ float exp2_full(float x) {
    const bool low = x < -126.0f;
    return __builtin_amdgcn_exp2f(low ? x + 64.0f : x) * (low ? 0x1p-64f : 1.0f);
}

__device__ __forceinline__ int64_t target_of(const void* targets, int wide, int64_t n, int64_t vocab) {
    return row_of(targets, wide, n, vocab);
}

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
#pragma unroll
        for (int u = 0; u < kTN; ++u) {
            const int64_t token = w.n0 + 16 * u + (w.lane & 15);
            const bool there = token < n;
            const int64_t t = there ? target_of(targets, targets64, token, vocab) : -1;
            const int64_t at = t - v0;
            float top = -INFINITY, mine = 0.0f;
            bool hit = false;
#pragma unroll
            for (int r = 0; r < kTM; ++r)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float z = acc[r][u][i];
                    if (v0 + 16 * r + i < vocab) top = fmaxf(top, z);
                    if (at == 16 * r + i) {
                        mine = z;
                        hit = true;
                    }
                }
            top = fmaxf(top, __shfl_xor(top, 16, 64));
            top = fmaxf(top, __shfl_xor(top, 32, 64));
            float sum = 0.0f;
#pragma unroll
            for (int r = 0; r < kTM; ++r)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (v0 + 16 * r + i < vocab) sum += __builtin_amdgcn_exp2f((acc[r][u][i] - top) * kLog2e);
            sum += __shfl_xor(sum, 16, 64);
            sum += __shfl_xor(sum, 32, 64);
            if (there && w.lane < 16) partial[slot * n + token] = make_float2(top, sum);
            if (there && hit) target_logit[token] = mine;
        }
    }
};

// dz of the piece, bf16 [token][width]; zero beyond the vocabulary.
struct LogitGradEpilogue {
    bf16_t* dz;
    int64_t width, first, vocab, n;
    const float* lse;
    const float* dloss;
    const void* targets;
    int32_t targets64;
    template <int kTM, int kTN>
    __device__ __forceinline__ void run(const f32x4 (&acc)[kTM][kTN], const WaveTile& w) const {
        const int64_t m0 = w.m0 + 4 * (w.lane >> 4);
#pragma unroll
        for (int u = 0; u < kTN; ++u) {
            const int64_t token = w.n0 + 16 * u + (w.lane & 15);
            if (token >= n) continue;
            const int64_t t = target_of(targets, targets64, token, vocab);
            const float up = t < 0 ? 0.0f : dloss[token], l = t < 0 ? 0.0f : lse[token];
            const int64_t at = t - first - m0;
            bf16_t* row = dz + token * width + m0;
#pragma unroll
            for (int r = 0; r < kTM; ++r) {
                float x[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float p = exp2_full((acc[r][u][i] - l) * kLog2e);
                    x[i] = at == 16 * r + i ? (p - 1.0f) * up : p * up;
                    if (t < 0 || first + m0 + 16 * r + i >= vocab) x[i] = 0.0f;
                }
                const u32x2 y = {pack2<bf16_t>(x[0], x[1]), pack2<bf16_t>(x[2], x[3])};
                *reinterpret_cast<u32x2*>(row + 16 * r) = y;
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
    int32_t add, vec;  // vec: 4 elements at a time are aligned
    template <int kTM, int kTN>
    __device__ __forceinline__ void run(const f32x4 (&acc)[kTM][kTN], const WaveTile& w) const {
        const int64_t m0 = w.m0 + 4 * (w.lane >> 4);
#pragma unroll
        for (int u = 0; u < kTN; ++u) {
            const int64_t v = first + w.n0 + 16 * u + (w.lane & 15);
            if (v >= vocab) continue;
            O* row = dw + v * ld + m0;
#pragma unroll
            for (int r = 0; r < kTM; ++r) {
                const f32x4 x = acc[r][u];
                O* p = row + 16 * r;
                if (vec && m0 + 16 * r + 4 <= dim) {
                    if constexpr (sizeof(O) == 4) {
                        f32x4 y = x;
                        if (add) y += *reinterpret_cast<const f32x4*>(p);
                        *reinterpret_cast<f32x4*>(p) = y;
                    } else {
                        f32x4 y = x;
                        if (add) {
                            const u32x2 o = *reinterpret_cast<const u32x2*>(p);
#pragma unroll
                            for (int i = 0; i < 4; ++i) y[i] += __uint_as_float((i & 1) ? (o[i >> 1] & 0xFFFF0000u) : (o[i >> 1] << 16));
                        }
                        const u32x2 o = {pack2<bf16_t>(y[0], y[1]), pack2<bf16_t>(y[2], y[3])};
                        *reinterpret_cast<u32x2*>(p) = o;
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (m0 + 16 * r + i < dim) p[i] = Elem<O>::to(add ? Elem<O>::get(p[i]) + x[i] : x[i]);
                }
            }
        }
    }
};

// lse and loss of a token from its partial statistics: 16 tokens a
// workgroup, 16 slots at a time.
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
        for (int64_t s = y; s < slots; s += kJoinSlots) {
            const float2 p = partial[s * n + token];
            // a slot beyond the vocabulary has maximum -inf and sum 0 (one of
            // NaN logits has sum NaN, which stays)
            const float t = fmaxf(top, p.x);
            if (p.y != 0.0f) {
                sum = (sum == 0.0f ? 0.0f : sum * __builtin_amdgcn_exp2f((top - t) * kLog2e)) + p.y * __builtin_amdgcn_exp2f((p.x - t) * kLog2e);
                top = t;
            }
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
            sums[y][x] = (sa == 0.0f ? 0.0f : sa * __builtin_amdgcn_exp2f((a - t) * kLog2e)) +
                         (sb == 0.0f ? 0.0f : sb * __builtin_amdgcn_exp2f((b - t) * kLog2e));
        }
        __syncthreads();
    }
    if (y != 0 || token >= n) return;
    const float l = tops[0][x] + logf(sums[0][x]);
    lse[token] = l;
    loss[token] = target_of(targets, targets64, token, vocab) < 0 ? 0.0f : l - target_logit[token];
}

// Rows with a width or alignment that 16-byte loads cannot take, copied into
// rows of `width` elements with zeros at the end.
template <class T>
__global__ void pad_rows_kernel(const T* __restrict__ src, int64_t ld, int64_t rows, int64_t dim, T* __restrict__ dst, int64_t width) {
    for (int64_t r = blockIdx.x; r < rows; r += gridDim.x)
        for (int64_t c = threadIdx.x; c < width; c += blockDim.x) dst[r * width + c] = c < dim ? src[r * ld + c] : (T)0;
}

// dh = sum of the slabs, rounded to bf16.
__global__ __launch_bounds__(256) void finish_hidden_kernel(const float* __restrict__ sums, int64_t slab, int32_t slabs, int64_t ld,
                                                            int64_t dim, int64_t n, bf16_t* __restrict__ out, int64_t out_ld, int32_t vec) {
    const int64_t quads = (dim + 3) / 4;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n * quads; i += (int64_t)gridDim.x * 256) {
        const int64_t token = i / quads, c = 4 * (i - token * quads);
        f32x4 x = {0.0f, 0.0f, 0.0f, 0.0f};
        for (int32_t s = 0; s < slabs; ++s) x += *reinterpret_cast<const f32x4*>(sums + s * slab + token * ld + c);
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

// Vocabulary rows of a piece: dz and a padded copy of the piece's weights
// take at most 512 MiB each.
int64_t piece_rows(int64_t n, int64_t vocab, int64_t dim) {
    const int64_t most = int64_t(512) << 20;
    const int64_t by_dz = most / (2 * std::max<int64_t>(n, 1)), by_copy = most / (2 * up(dim, 64));
    const int64_t rows = std::max<int64_t>(1024, std::min(by_dz, by_copy) / 256 * 256);
    return std::min(rows, up(vocab, 256));
}

// Splits of k that give a product of few tiles enough workgroups.
int splits_of(int64_t tiles, int64_t k) {
    int64_t s = 1;
    while (tiles * s < 384 && k / (s * 2) >= 512) s *= 2;
    return (int)s;
}

struct Work {
    float2* partial;
    float* target_logit;
    void *hidden, *weight;  // padded copies
    bf16_t* dz;
    float* sums;
    int64_t bytes;
};

int bn_of(int64_t n) { return n <= 64 ? 64 : n <= 128 ? 128 : 256; }
int waves_m_of(int bn) { return bn == 64 ? 8 : bn == 128 ? 4 : 2; }

int hidden_splits(int64_t n, int64_t dim, int64_t piece) {
    return splits_of((up(dim, kBM) / kBM) * (up(n, bn_of(n)) / bn_of(n)), piece);
}

Work work_of(void* work, int64_t n, int64_t vocab, int64_t dim, int fp8, int grad) {
    Work w{};
    char* p = static_cast<char*>(work);
    int64_t at = 0;
    const auto take = [&](int64_t bytes) {
        char* q = p + at;
        at += up(bytes, 256);
        return q;
    };
    const int64_t piece = piece_rows(n, vocab, dim), width = up(dim, 64);
    w.hidden = take(n * width * 2);
    w.weight = take(piece * width * (fp8 ? 1 : 2));
    const int64_t mark = at;
    // the loss and its gradient run one after the other: one space for both
    w.partial = reinterpret_cast<float2*>(take((up(vocab, kBM) / kBM + 1) * waves_m_of(bn_of(n)) * n * 8));
    w.target_logit = reinterpret_cast<float*>(take(n * 4));
    w.bytes = at;
    if (grad) {
        at = mark;
        w.dz = reinterpret_cast<bf16_t*>(take(n * piece * 2));
        w.sums = reinterpret_cast<float*>(take(hidden_splits(n, dim, piece) * n * width * 4));
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
    g.group_m = 8;
    hipLaunchKernelGGL(kernel, dim3((uint32_t)(g.tiles_m * g.tiles_n * g.splits)), dim3(kGemmThreads), kLds, (hipStream_t)stream, g, e);
    return hipGetLastError();
}

// A product whose A is a piece of the weights with k (or m) in its rows and
// whose B has tokens in its rows.
template <template <int> class A, int kBN, class Epilogue>
int launch_kc(const GemmArgs& g, const Epilogue& e, void* stream) {
    return launch_gemm<A<kBM>, BF16KC<kBN>, kBN, kBN == 64 ? 8 : kBN == 128 ? 4 : 2, Epilogue>(g, e, stream);
}
template <template <int, int> class A, int kBN, class Epilogue>
int launch_kr(const GemmArgs& g, const Epilogue& e, void* stream) {
    constexpr int kWavesM = kBN == 64 ? 8 : kBN == 128 ? 4 : 2;
    return launch_gemm<A<kBM, kBM / kWavesM / 16>, BF16KC<kBN>, kBN, kWavesM, Epilogue>(g, e, stream);
}

template <class Epilogue>
int logits(int fp8, int64_t n, const GemmArgs& g, const Epilogue& e, void* stream) {
    switch (bn_of(n)) {
        case 64: return fp8 ? launch_kc<FP8KC, 64>(g, e, stream) : launch_kc<BF16KC, 64>(g, e, stream);
        case 128: return fp8 ? launch_kc<FP8KC, 128>(g, e, stream) : launch_kc<BF16KC, 128>(g, e, stream);
        default: return fp8 ? launch_kc<FP8KC, 256>(g, e, stream) : launch_kc<BF16KC, 256>(g, e, stream);
    }
}

int hidden_grad(int fp8, int64_t n, const GemmArgs& g, const SumEpilogue& e, void* stream) {
    switch (bn_of(n)) {
        case 64: return fp8 ? launch_kr<FP8KR, 64>(g, e, stream) : launch_kr<BF16KR, 64>(g, e, stream);
        case 128: return fp8 ? launch_kr<FP8KR, 128>(g, e, stream) : launch_kr<BF16KR, 128>(g, e, stream);
        default: return fp8 ? launch_kr<FP8KR, 256>(g, e, stream) : launch_kr<BF16KR, 256>(g, e, stream);
    }
}

template <class T>
int pad_rows(const void* src, int64_t ld, int64_t rows, int64_t dim, void* dst, int64_t width, void* stream) {
    const uint32_t wgs = (uint32_t)std::min<int64_t>(rows, 65536);
    hipLaunchKernelGGL(pad_rows_kernel<T>, dim3(wgs), dim3(256), 0, (hipStream_t)stream, static_cast<const T*>(src), ld, rows, dim,
                       static_cast<T*>(dst), width);
    return hipGetLastError();
}

bool loadable(const void* p, int64_t ld, int64_t dim, int size) {
    return dim * size % 16 == 0 && ld * size % 16 == 0 && reinterpret_cast<uintptr_t>(p) % 16 == 0;
}

// The operands as the products read them: in place where rows suit 16-byte
// loads, else padded copies (the weights' by pieces).
struct Source {
    Operand hidden;      // rows of tokens
    bool copy_weight;
    int64_t width, esize;
};

int source_of(const VocabLossArgs& a, const Work& w, Source* s, void* stream) {
    s->width = up(a.dim, 64);
    s->esize = a.fp8 ? 1 : 2;
    s->copy_weight = !loadable(a.weight, a.weight_ld, a.dim, (int)s->esize);
    if (loadable(a.hidden, a.hidden_ld, a.dim, 2)) {
        s->hidden = Operand{a.hidden, a.hidden_ld * 2, a.n, a.dim};
        return hipSuccess;
    }
    s->hidden = Operand{w.hidden, s->width * 2, a.n, s->width};
    return pad_rows<uint16_t>(a.hidden, a.hidden_ld, a.n, a.dim, w.hidden, s->width, stream);
}

// Rows [first, first + rows) of the weights, rows in extent and dim in k.
int weight_piece(const VocabLossArgs& a, const Work& w, const Source& s, int64_t first, int64_t rows, Operand* o, void* stream) {
    const char* p = static_cast<const char*>(a.weight) + first * a.weight_ld * s.esize;
    if (!s.copy_weight) {
        *o = Operand{p, a.weight_ld * s.esize, rows, a.dim};
        return hipSuccess;
    }
    *o = Operand{w.weight, s.width * s.esize, rows, s.width};
    return a.fp8 ? pad_rows<uint8_t>(p, a.weight_ld, rows, a.dim, w.weight, s.width, stream)
                 : pad_rows<uint16_t>(p, a.weight_ld, rows, a.dim, w.weight, s.width, stream);
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

}  // namespace

int64_t vocab_loss_work_bytes(int64_t n, int64_t vocab, int64_t dim, int fp8, int grad) {
    return work_of(nullptr, n, vocab, dim, fp8, grad).bytes;
}

int launch_vocab_loss(const VocabLossArgs& a, void* work, void* stream) {
    if (a.n == 0) return hipSuccess;
    const Work w = work_of(work, a.n, a.vocab, a.dim, a.fp8, 0);
    Source s;
    int err = source_of(a, w, &s, stream);
    if (err) return err;
    const int waves_m = waves_m_of(bn_of(a.n));
    const int64_t piece = s.copy_weight ? piece_rows(a.n, a.vocab, a.dim) : a.vocab;
    int64_t slots = 0;
    for (int64_t first = 0; first < a.vocab; first += piece) {
        const int64_t rows = std::min(piece, a.vocab - first);
        GemmArgs g{};
        err = weight_piece(a, w, s, first, rows, &g.a, stream);
        if (err) return err;
        g.b = s.hidden;
        g.k = a.dim;
        set_grid(a, first, true, &g);
        const StatsEpilogue e{w.partial, w.target_logit, a.targets, a.targets64, first, a.vocab, a.n, slots, waves_m};
        err = logits(a.fp8, a.n, g, e, stream);
        if (err) return err;
        slots += up(rows, kBM) / kBM * waves_m;
    }
    hipLaunchKernelGGL(join_stats_kernel, dim3((uint32_t)(up(a.n, kJoinTokens) / kJoinTokens)), dim3(kJoinTokens * kJoinSlots), 0,
                       (hipStream_t)stream, w.partial, slots, w.target_logit, a.targets, a.targets64, a.vocab, a.n, a.loss, a.lse);
    return hipGetLastError();
}

int launch_vocab_loss_grad(const VocabLossArgs& a, void* work, void* stream) {
    const Work w = work_of(work, a.n, a.vocab, a.dim, a.fp8, 1);
    Source s{};
    int err = hipSuccess;
    if (a.n > 0) err = source_of(a, w, &s, stream);
    if (err) return err;
    const int64_t piece = piece_rows(a.n, a.vocab, a.dim);
    const int splits = hidden_splits(a.n, a.dim, piece);
    for (int64_t first = 0; first < a.vocab; first += piece) {
        const int64_t rows = std::min(piece, a.vocab - first);
        const int64_t width = up(rows, kBM);
        GemmArgs g{};
        Operand weight{};
        if (a.n > 0) {
            err = weight_piece(a, w, s, first, rows, &weight, stream);
            if (err) return err;
            g.a = weight;
            g.b = s.hidden;
            g.k = a.dim;
            set_grid(a, first, true, &g);
            const LogitGradEpilogue e{w.dz, width, first, a.vocab, a.n, a.lse, a.dloss, a.targets, a.targets64};
            err = logits(a.fp8, a.n, g, e, stream);
            if (err) return err;
        }
        if (a.dhidden && a.n > 0) {
            GemmArgs h{};
            h.a = Operand{weight.p, weight.ld, weight.k, rows};
            h.b = Operand{w.dz, width * 2, a.n, width};
            h.k = rows;
            h.splits = splits;
            set_grid(a, first, false, &h);
            const SumEpilogue e{w.sums, s.width, a.n * s.width, s.width, a.n, first > 0};
            err = hidden_grad(a.fp8, a.n, h, e, stream);
            if (err) return err;
        }
        if (a.dweight) {
            GemmArgs d{};
            d.a = Operand{s.hidden.p, s.hidden.ld, s.hidden.k, a.n};
            d.b = Operand{w.dz, width * 2, width, a.n};
            d.k = a.n;
            if (a.n == 0) d.a.extent = a.dim, d.b.extent = rows;
            const bool f32 = a.dweight_type == kF32;
            const int64_t unit = f32 ? 16 : 8;
            const int32_t vec = a.dweight_ld % 4 == 0 && reinterpret_cast<uintptr_t>(a.dweight) % unit == 0;
            if (f32) {
                const WeightGradEpilogue<float> e{static_cast<float*>(a.dweight), a.dweight_ld, a.dim, first, a.vocab, a.accumulate, vec};
                err = launch_gemm<BF16KR<kBM, 8>, BF16KR<256, 4>, 256, 2, WeightGradEpilogue<float>>(d, e, stream);
            } else {
                const WeightGradEpilogue<bf16_t> e{static_cast<bf16_t*>(a.dweight), a.dweight_ld, a.dim, first, a.vocab, a.accumulate, vec};
                err = launch_gemm<BF16KR<kBM, 8>, BF16KR<256, 4>, 256, 2, WeightGradEpilogue<bf16_t>>(d, e, stream);
            }
            if (err) return err;
        }
    }
    if (!a.dhidden || a.n == 0) return hipSuccess;
    const int32_t vec = a.dim % 4 == 0 && a.dhidden_ld % 4 == 0 && reinterpret_cast<uintptr_t>(a.dhidden) % 8 == 0;
    const int64_t quads = a.n * ((a.dim + 3) / 4);
    hipLaunchKernelGGL(finish_hidden_kernel, dim3((uint32_t)std::min<int64_t>((quads + 255) / 256, 16384)), dim3(256), 0,
                       (hipStream_t)stream, w.sums, a.n * s.width, splits, s.width, a.dim, a.n, static_cast<bf16_t*>(a.dhidden),
                       a.dhidden_ld, vec);
    return hipGetLastError();
}

}  // namespace bfz
