// The linear layer in E4M3: quantizer of activations, and the three products.
//
//   code = E4M3(x / s), s = amax / 448 of 128 columns of a row or of a 128x128 tile
//   y = X W^T,  dx = dY W,  dW = dY^T X, each value a code times its scale
//
// Quantizer: bound by memory, a group in registers between its largest value and its
// codes; 8192 x 4096 bf16 by rows 18 us (5.6 TB/s), by tiles 19 us (5.2).
//
// Products, bound by the matrix cores (codes_gemm.h): forward and dx read the weight
// and the codes as they lie, k along rows or across them; dW contracts over tokens
// and reads both operands across.  8192 x 11008 x 4096: forward 325 us (2.27
// PFLOP/s), dx 298 (2.48), dW in bf16 315 (2.34), in f32, by bf16 instructions, 641
// (1.15); the library's products of two E4M3 matrices with one scale each run at 2.4
// there (3.2 at 8192 in each direction), those of bf16 ones at 1.1 (1.6).  Up to 64
// tokens, bound by reading the weight: 4096 x 4096, 1 token 5.1 us (3.3 TB/s; 3.6 of
// it the bytes), 11008 x 4096, 64 tokens 17 us.  (Back-to-back calls, the first 30
// ms of them: under longer load the card's clock falls.)
#include <hip/hip_runtime.h>

#include <algorithm>
#include <atomic>

#include "codes_gemm.h"
#include "layer_internal.h"
#include "quant_device.h"

namespace bfz {
namespace {

constexpr int kThreads = 256;
constexpr int kCus = 256;
// Floats that the splits of a product may take: splits and tiles of 128 by 128 at
// most are one a CU.
constexpr int64_t kMostSums = int64_t(kCus) * kTileDim * kTileDim;

// ---- quantizer ------------------------------------------------------------------

// Row groups: 16 lanes hold a group, 8 columns each; a wave 4 groups of a row.
constexpr int kRowsOfWave = 2, kRowsOfWg = kRowsOfWave * kThreads / 64, kGroupsOfWave = 4;
static_assert(kThreads == kQuantizeRowsThreads && kRowsOfWg == kQuantizeRows && kGroupsOfWave * kTileDim == kQuantizeCols, "what the size checks count");

template <class T>
__global__ __launch_bounds__(kThreads) void quantize_rows_kernel(QuantizeArgs a, int32_t col_wgs) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t block = blockIdx.x;
    const int64_t c = (block % col_wgs) * (kGroupsOfWave * kTileDim) + 8 * lane;
    const int64_t r0 = block / col_wgs * kRowsOfWg + wave * kRowsOfWave;
    const int64_t left = a.dim - c;
    const int count = left <= 0 ? 0 : left >= 8 ? 8 : (int)left;
    const int64_t width = (a.dim + 15) / 16 * 16;
    float x[kRowsOfWave][8];
#pragma unroll
    for (int k = 0; k < kRowsOfWave; ++k)
        load8_any(static_cast<const T*>(a.x) + (r0 + k) * a.x_ld + c, r0 + k < a.n ? count : 0, x[k]);
#pragma unroll
    for (int k = 0; k < kRowsOfWave; ++k) {
        const float scale = scale_of(row_max(abs_max8(x[k])), a.pow2);
        uint32_t w[2];
        quantize8(x[k], Quotient(scale), w);
        if (r0 + k >= a.n) continue;
        if (c < width) *reinterpret_cast<u32x2*>(a.codes + (r0 + k) * a.codes_ld + c) = u32x2{w[0], w[1]};
        if ((lane & 15) == 0 && c < a.dim) a.scales[c / kTileDim * a.scales_ld + r0 + k] = scale;
    }
}

// Tiles: 16 lanes a row, the whole tile in registers, 4 rows a thread.
constexpr int kTileThreads = kQuantizeTilesThreads, kTileRows = kTileDim * 16 / kTileThreads, kTileStep = kTileThreads / 16;
template <class T>
__global__ __launch_bounds__(kTileThreads) void quantize_tiles_kernel(QuantizeArgs a, int32_t col_tiles) {
    __shared__ float tops[kTileThreads / 64];
    const int64_t i = blockIdx.x / col_tiles, j = blockIdx.x % col_tiles;
    const int64_t c = j * kTileDim + 8 * (threadIdx.x & 15);
    const int64_t left = a.dim - c;
    const int count = left <= 0 ? 0 : left >= 8 ? 8 : (int)left;
    const int64_t r0 = i * kTileDim + (threadIdx.x >> 4);
    const int64_t width = (a.dim + 15) / 16 * 16;
    float x[kTileRows][8];
    float top = 0.0f;
#pragma unroll
    for (int k = 0; k < kTileRows; ++k) {
        const int64_t r = r0 + kTileStep * k;
        load8_any(static_cast<const T*>(a.x) + r * a.x_ld + c, r < a.n ? count : 0, x[k]);
    }
#pragma unroll
    for (int k = 0; k < kTileRows; ++k) top = fmaxf(top, abs_max8(x[k]));
    top = wave_max(top);
    if ((threadIdx.x & 63) == 0) tops[threadIdx.x >> 6] = top;
    __syncthreads();
    top = tops[0];
#pragma unroll
    for (int w = 1; w < kTileThreads / 64; ++w) top = fmaxf(top, tops[w]);
    const float scale = scale_of(top, a.pow2);
    const Quotient q(scale);
#pragma unroll
    for (int k = 0; k < kTileRows; ++k) {
        const int64_t r = r0 + kTileStep * k;
        uint32_t w[2];
        quantize8(x[k], q, w);
        if (r < a.n && c < width) *reinterpret_cast<u32x2*>(a.codes + r * a.codes_ld + c) = u32x2{w[0], w[1]};
    }
    if (threadIdx.x == 0) a.scales[i * a.scales_ld + j] = scale;
}

template <class T>
int quantize(const QuantizeArgs& a, hipStream_t stream) {
    const dim3 wgs((uint32_t)quantize_wgs(a.n, a.dim, a.tiles));
    if (a.tiles) {
        hipLaunchKernelGGL((quantize_tiles_kernel<T>), wgs, dim3(kTileThreads), 0, stream, a, (int32_t)((a.dim + kTileDim - 1) / kTileDim));
    } else {
        hipLaunchKernelGGL((quantize_rows_kernel<T>), wgs, dim3(kThreads), 0, stream, a, (int32_t)((a.dim + kQuantizeCols - 1) / kQuantizeCols));
    }
    return hipGetLastError();
}

// ---- products -------------------------------------------------------------------

// Results of a product, rounded to their type, or a split's binary32 sums.  Two
// tiles of 16 rows are exchanged between the halves of lane pairs, so that a lane
// holds 8 consecutive m of a token.
struct StoreEpilogue {
    void* out;
    int64_t ld, slab;  // slab: from split to split
    int64_t m, n;      // extents
    int32_t type, add, vec;
    template <int kTM, int kTN>
    __device__ __forceinline__ void run(const f32x4 (&acc)[kTM][kTN], const WaveTile& w) const {
        const int g = w.lane >> 4;
#pragma unroll
        for (int u = 0; u < kTN; ++u) {
            const int64_t token = w.n0 + 16 * u + (w.lane & 15);
#pragma unroll
            for (int t = 0; t < kTM; t += 2) {
                __builtin_amdgcn_sched_barrier(0);  // one store's registers at a time
                float x[8];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(acc[t][u][i]), __float_as_uint(acc[t + 1][u][i]), false, false);
                    x[i] = __uint_as_float(r[0]);
                    x[4 + i] = __uint_as_float(r[1]);
                }
                const int64_t c = w.m0 + 16 * (t + (g & 1)) + 8 * (g >> 1);
                if (token >= n || c >= m) continue;
                const int64_t at = w.split * slab + token * ld + c;
                if (type == kF32) put(static_cast<float*>(out) + at, c, x);
                else if (type == kBF16) put(static_cast<bf16_t*>(out) + at, c, x);
                else put(static_cast<f16_t*>(out) + at, c, x);
            }
        }
    }
    // 4 results of a token from m on
    __device__ __forceinline__ void put4(int64_t token, int64_t c, const f32x4& x) const {
        if (token >= n) return;
        const int64_t at = token * ld + c;
        if (type == kF32) put4(static_cast<float*>(out) + at, c, x);
        else if (type == kBF16) put4(static_cast<bf16_t*>(out) + at, c, x);
        else put4(static_cast<f16_t*>(out) + at, c, x);
    }
    template <class O>
    __device__ __forceinline__ void put4(O* p, int64_t c, const f32x4& x) const {
        if (vec && c + 4 <= m) {
            if constexpr (sizeof(O) == 4) *reinterpret_cast<f32x4*>(p) = x;
            else *reinterpret_cast<u32x2*>(p) = u32x2{pack2<O>(x[0], x[1]), pack2<O>(x[2], x[3])};
        } else {
#pragma unroll
            for (int l = 0; l < 4; ++l)
                if (c + l < m) p[l] = Elem<O>::to(x[l]);
        }
    }
    template <class O>
    __device__ __forceinline__ void put(O* p, int64_t c, float (&x)[8]) const {
        if (vec && c + 8 <= m) {
            if (add) {
                float y[8];
                load8(p, y);
#pragma unroll
                for (int l = 0; l < 8; ++l) x[l] += y[l];
            }
            store8(p, x);
        } else {
#pragma unroll
            for (int l = 0; l < 8; ++l)
                if (c + l < m) p[l] = Elem<O>::to(add ? Elem<O>::get(p[l]) + x[l] : x[l]);
        }
    }
};

// Inputs of a product of few tokens that the product itself quantizes by rows: in
// LDS the codes, rows of `width` bytes with zeros at the end, then the scales
// [token][block].
struct RowInputs {
    const void* x;
    int32_t type;
    int64_t ld;
    int32_t n, dim, width, blocks;
    template <class T>
    __device__ __forceinline__ void quantize_type(char* lds) const {
        float* scales = reinterpret_cast<float*>(lds + n * width);
        const int pieces = blocks * 16;  // of 8 columns, whole groups
        for (int i = threadIdx.x; i < n * pieces; i += 64 * kFewKWaves) {
            const int token = i / pieces, c = 8 * (i - token * pieces);
            float y[8];
            load8_any(static_cast<const T*>(x) + token * ld + c, min(8, max(0, dim - c)), y);
            const float scale = scale_of(row_max(abs_max8(y)), false);
            uint32_t w[2];
            quantize8(y, Quotient(scale), w);
            *reinterpret_cast<u32x2*>(lds + token * width + c) = u32x2{w[0], w[1]};
            if ((threadIdx.x & 15) == 0) scales[token * blocks + c / kTileDim] = scale;
        }
    }
    __device__ __forceinline__ void quantize(char* lds) const {
        if (type == kF32) quantize_type<float>(lds);
        else if (type == kBF16) quantize_type<bf16_t>(lds);
        else quantize_type<f16_t>(lds);
    }
    __device__ __forceinline__ i32x8 fragment(const char* lds, int token, int kb, int q) const {
        if (token >= n || kb >= blocks) return i32x8{0, 0, 0, 0, 0, 0, 0, 0};
        const char* p = lds + token * width + kb * kTileDim + 16 * q;
        const i32x4 lo = *reinterpret_cast<const i32x4*>(p), hi = *reinterpret_cast<const i32x4*>(p + 64);
        return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    }
    __device__ __forceinline__ float scale(const char* lds, int token, int kb) const {
        return reinterpret_cast<const float*>(lds + n * width)[token * blocks + kb];
    }
};

// The sums of a split product, out = slabs added in their order; zeros where there
// is none.
template <class O>
__global__ __launch_bounds__(kThreads) void join_splits_kernel(const float* __restrict__ sums, int32_t splits, StoreEpilogue s) {
    const int64_t pieces = (s.m + 7) / 8;
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < s.n * pieces; i += (int64_t)gridDim.x * kThreads) {
        const int64_t token = i / pieces, c = 8 * (i - token * pieces);
        float x[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
        for (int32_t k = 0; k < splits; ++k) {
            float y[8];
            load8(sums + k * s.slab + token * (pieces * 8) + c, y);
#pragma unroll
            for (int l = 0; l < 8; ++l) x[l] += y[l];
        }
        s.put(static_cast<O*>(s.out) + token * s.ld + c, c, x);
    }
}

// A weight whose rows the products cannot read in place, copied into rows of
// `width` bytes with zeros at the end.
__global__ __launch_bounds__(kThreads) void copy_weight_kernel(const uint8_t* __restrict__ src, int64_t ld, int64_t rows, int64_t cols,
                                                               uint8_t* __restrict__ dst, int64_t width) {
    const int64_t words = width / 4;
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < rows * words; i += (int64_t)gridDim.x * kThreads) {
        const int64_t r = i / words, c = 4 * (i - r * words);
        uint32_t w = 0;
#pragma unroll
        for (int l = 0; l < 4; ++l)
            if (c + l < cols) w |= (uint32_t)src[r * ld + c + l] << (8 * l);
        reinterpret_cast<uint32_t*>(dst)[i] = w;
    }
}

// ---- host -------------------------------------------------------------------------

// More than 64 KiB of LDS is allowed for a kernel once on each device.
int allow_lds(const void* kernel, int bytes, std::atomic<uint64_t>& ready) {
    int dev = 0;
    hipError_t err = hipGetDevice(&dev);
    if (err != hipSuccess) return err;
    const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
    if (bit && (ready.load(std::memory_order_acquire) & bit)) return hipSuccess;
    err = hipFuncSetAttribute(kernel, hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (err == hipSuccess) ready.fetch_or(bit, std::memory_order_release);
    return err;
}

// Columns of n that go into whole tiles; the others go into tiles half as wide, so
// that the last round of workgroups is a short one.  A half tile takes some 0.55 of
// a whole one's time, and the CUs that the last whole tiles leave take it first.
int64_t whole_columns(int64_t tiles_m, int64_t n, int64_t width) {
    const int64_t tiles_n = (n + width - 1) / width;
    constexpr double kHalf = 0.55;
    int64_t best = tiles_n;
    double least = (double)((tiles_m * tiles_n + kCus - 1) / kCus);
    for (int64_t c = tiles_n - 1; c >= 0 && c >= tiles_n - 8; --c) {
        const int64_t whole = tiles_m * c, busy = whole % kCus;
        const int64_t halves = tiles_m * ((n - c * width + width / 2 - 1) / (width / 2));
        // by the end of a last round of length t, the CUs that are free at its start
        // take t / kHalf of them, the busy ones (t - 1) / kHalf
        for (double t : {kHalf, 1.0, 2 * kHalf, 1.0 + kHalf, 3 * kHalf, 1.0 + 2 * kHalf}) {
            const int64_t room = (kCus - busy) * (int64_t)(t / kHalf + 1e-6) + busy * (int64_t)(std::max(0.0, t - 1.0) / kHalf + 1e-6);
            if (room < halves || (busy > 0 && t < 1.0)) continue;
            const double time = (double)(whole / kCus) + t;
            if (time < least - 0.05) {
                least = time;
                best = c;
            }
            break;
        }
    }
    return best;
}

// Tiles of a product that is too small for 256-wide ones, and splits of k, by modelled
// time in us: a round of workgroups takes `start` and `step` a block of k, as measured
// at 2 to 86 blocks; splits cost a launch to join them and their sums' way out and
// back.  (On 45 sizes of 3e7 to 8e10 products the choice was the fastest, but for
// four by 4 to 16%.)  Modelled and measured, with bf16 instructions: 1013 x 1544 x 1008 11.8 and
// 11.3 in tiles 64 wide, 16.8 and 14.7 in 128; 3000 x 1700 x 3600 56 and 57 in pairs
// of workgroups, 81 and 76 in 64.  With E4M3 ones, 100 x 4096 x 11008 40.6 and 38.9 in
// one, 19.9 and 19.5 in four splits; 1300 x 4096 x 4096 36 and 37 in pairs, 54 and 49
// in 64.
struct Form {
    int32_t width, waves, of_cu;
    double start[2], step[2];  // with E4M3 instructions, with bf16 ones
};
constexpr Form kForms[] = {
    {128, 8, 1, {6.0, 8.0}, {0.6, 1.1}},
    {128, 4, 2, {6.0, 10.0}, {0.95, 1.6}},
    {64, 8, 1, {4.5, 6.0}, {0.42, 0.72}},
};
struct Small {
    int32_t width, waves, splits;
};
Small small_tiles(int64_t k, int64_t m, int64_t n, bool exact) {
    const int64_t blocks = (k + kTileDim - 1) / kTileDim;
    Small best{128, 8, 1};
    double least = 1e30;
    for (const Form& f : kForms) {
        const int64_t tiles = ((m + 127) / 128) * ((n + f.width - 1) / f.width);
        // splits where one workgroup a CU holds them all
        for (int64_t s = 1; s <= 16 && s <= std::max<int64_t>(1, blocks) && (s == 1 || (f.of_cu == 1 && s * tiles <= kCus)); ++s) {
            const double rounds = (double)((s * tiles + f.of_cu * kCus - 1) / (f.of_cu * kCus));
            const double join = s > 1 ? 3.5 + 0.3 * (double)s + (double)(s * m * n) * 8 / 6e6 : 0.0;
            const double time = rounds * (f.start[exact] + (double)((blocks + s - 1) / s) * f.step[exact]) + join;
            if (time < least) {
                least = time;
                best = Small{f.width, f.waves, (int32_t)s};
            }
        }
    }
    return best;
}

// Results that would show what the E4M3 instructions cut off (codes_gemm.h), or whose
// caller asks for exact products.
bool exact_products(int type, int asked) { return type != kBF16 || asked; }

// How a product is cut: tiles of m x n with so many waves each, splits of k, columns
// of whole tiles (the others are half as wide).
struct Shape {
    int32_t tile_m, tile_n, waves, splits;
    int64_t k_per_split, whole;
};

// 256 x 256 or, with bf16 instructions, 256 x 128 where tiles of 256 x 256 occupy the
// CUs; 256 x 128 where those do; else 128 x 64 or 128 x 128, one workgroup a CU with
// eight waves and four blocks in flight, or two of four waves a CU.
Shape shape_of(int64_t k, int64_t m, int64_t n, bool exact) {
    const auto tiles = [&](int64_t high, int64_t wide) { return ((m + high - 1) / high) * ((n + wide - 1) / wide); };
    const int64_t blocks = std::max<int64_t>(1, (k + kTileDim - 1) / kTileDim);
    if (tiles(256, 256) >= 192 || (!exact && tiles(256, 128) >= 192)) {
        const int32_t wide = tiles(256, 256) >= 192 && !exact ? 256 : 128;
        return Shape{256, wide, 8, 1, blocks * kTileDim, whole_columns((m + 255) / 256, n, wide)};
    }
    const Small small = small_tiles(k, m, n, exact);
    Shape s{128, small.width, small.waves, small.splits, (blocks + small.splits - 1) / small.splits * kTileDim, (n + small.width - 1) / small.width};
    s.splits = (int32_t)((blocks * kTileDim + s.k_per_split - 1) / s.k_per_split);
    return s;
}

template <bool kAKR, bool kBKR, int kTileM, int kTileN, int kWavesM, int kWavesN, int kStages, bool kExact, bool kHalves>
int launch_tiles(ProductArgs& g, const StoreEpilogue& e, const Shape& shape, hipStream_t stream) {
    constexpr int kLds = kStages * TileOf<kAKR, kBKR, kTileM, kTileN, kWavesM * kWavesN>::kStage;
    const auto kernel = codes_gemm_kernel<kAKR, kBKR, kTileM, kTileN, kWavesM, kWavesN, kStages, kExact, kHalves, StoreEpilogue>;
    static std::atomic<uint64_t> ready{0};  // a bit for each device
    const int rc = allow_lds(reinterpret_cast<const void*>(kernel), kLds, ready);
    if (rc) return rc;
    g.tiles_m = (int32_t)((g.a.extent + kTileM - 1) / kTileM);
    g.tiles_n = (int32_t)shape.whole;
    g.group_m = std::min(g.tiles_m, 4);
    g.half_tiles_n = (int32_t)(std::max<int64_t>(0, g.b.extent - shape.whole * kTileN + kTileN / 2 - 1) / (kTileN / 2));
    const int64_t wgs = (int64_t)g.tiles_m * ((int64_t)g.tiles_n * g.splits + g.half_tiles_n);
    hipLaunchKernelGGL(kernel, dim3((uint32_t)wgs), dim3(64 * kWavesM * kWavesN), kLds, stream, g, e);
    return hipGetLastError();
}

template <bool kAKR, bool kBKR, bool kExact>
int launch_product(ProductArgs& g, const StoreEpilogue& e, const Shape& shape, hipStream_t stream) {
    if constexpr (!kExact) {
        if (shape.tile_n == 256) return launch_tiles<kAKR, kBKR, 256, 256, 2, 4, 2, false, true>(g, e, shape, stream);
    }
    if (shape.tile_m == 256) return launch_tiles<kAKR, kBKR, 256, 128, 4, 2, 3, kExact, true>(g, e, shape, stream);
    if (shape.tile_n == 64) return launch_tiles<kAKR, kBKR, 128, 64, 4, 2, 4, kExact, false>(g, e, shape, stream);
    if (shape.waves == 8) return launch_tiles<kAKR, kBKR, 128, 128, 4, 2, 4, kExact, false>(g, e, shape, stream);
    return launch_tiles<kAKR, kBKR, 128, 128, 2, 2, 2, kExact, false>(g, e, shape, stream);
}

template <bool kAKR, bool kBKR>
int product(ProductArgs& g, const LinearArgs& a, int64_t m, int64_t n, float* sums, hipStream_t stream) {
    const bool exact = exact_products(a.out_type, a.exact);
    const int size = dtype_size(a.out_type);
    StoreEpilogue e{a.out, a.out_ld, 0, m, n, a.out_type, a.accumulate, 0};
    e.vec = ((reinterpret_cast<uintptr_t>(a.out) | (uint64_t)(a.out_ld * size)) & 15u) == 0;
    const Shape shape = shape_of(g.k, m, n, exact);
    g.splits = g.k == 0 ? 0 : shape.splits;
    g.k_per_split = shape.k_per_split;
    if (g.splits == 1) return exact ? launch_product<kAKR, kBKR, true>(g, e, shape, stream) : launch_product<kAKR, kBKR, false>(g, e, shape, stream);
    const int64_t pieces = (m + 7) / 8;
    e.slab = pieces * 8 * n;
    const StoreEpilogue part{sums, pieces * 8, e.slab, pieces * 8, n, kF32, 0, 1};
    const int rc = g.splits == 0 ? hipSuccess : exact ? launch_product<kAKR, kBKR, true>(g, part, shape, stream) : launch_product<kAKR, kBKR, false>(g, part, shape, stream);
    if (rc) return rc;
    const dim3 wgs((uint32_t)std::min<int64_t>((n * pieces + kThreads - 1) / kThreads, 1 << 20));
    if (a.out_type == kF32) hipLaunchKernelGGL((join_splits_kernel<float>), wgs, dim3(kThreads), 0, stream, sums, g.splits, e);
    else if (a.out_type == kBF16) hipLaunchKernelGGL((join_splits_kernel<bf16_t>), wgs, dim3(kThreads), 0, stream, sums, g.splits, e);
    else hipLaunchKernelGGL((join_splits_kernel<f16_t>), wgs, dim3(kThreads), 0, stream, sums, g.splits, e);
    return hipGetLastError();
}

constexpr int64_t kFewTokensMost = 64;

template <int kTM, int kTN, bool kExact, bool kQuantize>
int launch_few(const ProductArgs& g, const RowInputs& x, const StoreEpilogue& e, hipStream_t stream) {
    const int lds = kQuantize ? x.n * x.width + 4 * x.n * x.blocks : 0;
    const auto kernel = few_codes_kernel<kTM, kTN, kExact, kQuantize, RowInputs, StoreEpilogue>;
    hipLaunchKernelGGL(kernel, dim3((uint32_t)((e.m + 16 * kTM - 1) / (16 * kTM))),
                       dim3(64 * kFewKWaves), (size_t)lds, stream, g, x, e);
    return hipGetLastError();
}

// Tiles of 16 rows that a workgroup of few tokens takes, 16 tn of them at most: as
// few, up to three, as still fit the device in one round.  A CU holds one workgroup
// with 33 tokens and more, whose registers and LDS leave no room for a second, else
// two.  More than 12288 rows, or 16384 with up to 32 tokens, take further rounds: a
// fourth tile, or a third there, is not tried.
int32_t few_tiles(int64_t m, int32_t tn) {
    if (m <= 16 * kCus) return 1;
    return tn < 4 || m <= 2 * 16 * kCus ? 2 : 3;
}

template <int kTN, bool kExact, bool kQuantize>
int few_rows(const ProductArgs& g, const RowInputs& x, const StoreEpilogue& e, hipStream_t stream) {
    const int32_t tiles = few_tiles(e.m, kTN);
    if (tiles == 1) return launch_few<1, kTN, kExact, kQuantize>(g, x, e, stream);
    if constexpr (kTN == 4) {
        if (tiles == 3) return launch_few<3, kTN, kExact, kQuantize>(g, x, e, stream);
    }
    return launch_few<2, kTN, kExact, kQuantize>(g, x, e, stream);
}

// Up to 16 tokens the weight's bytes decide, and exact products cost a bfloat16
// result 2 to 5% (1 token on 4096 x 4096: 5.1 us instead of 4.9, 16 on 28672 x 8192:
// 48.4 instead of 48.0).  Beyond them they would cost it 10 to 40% (64 on 11008 x
// 4096: 21 us instead of 17, 33 on 28672 x 8192: 102 instead of 67).
bool exact_few(int type, int asked, int64_t n) { return n <= 16 || exact_products(type, asked); }

int few_tokens(const ProductArgs& g, const RowInputs* x, const StoreEpilogue& e, int asked, hipStream_t stream) {
    if (x) return few_rows<1, true, true>(g, *x, e, stream);
    const RowInputs none{};
    const bool exact = exact_few(e.type, asked, e.n);
    if (e.n <= 16) return few_rows<1, true, false>(g, none, e, stream);
    if (e.n <= 32) return exact ? few_rows<2, true, false>(g, none, e, stream) : few_rows<2, false, false>(g, none, e, stream);
    return exact ? few_rows<4, true, false>(g, none, e, stream) : few_rows<4, false, false>(g, none, e, stream);
}

void token_scales(ProductArgs& g, const Codes& c) {
    g.scales = c.scales;
    g.scales_ld = c.scales_ld;
    g.tiles = c.tiles ? kTilesOfN : kEachOfN;
}

int64_t round_up(int64_t n, int64_t to) { return (n + to - 1) / to * to; }

}  // namespace

int launch_quantize(const QuantizeArgs& a, void* stream) {
    const hipStream_t s = (hipStream_t)stream;
    return a.x_type == kF32 ? quantize<float>(a, s) : a.x_type == kBF16 ? quantize<bf16_t>(a, s) : quantize<f16_t>(a, s);
}

// The workspace: codes and scales of inputs, the copy of a weight, the sums of
// splits.
namespace {
int64_t codes_bytes(int64_t n, int64_t cols) { return round_up(n * round_up(cols, 16), 256) + round_up((cols + 127) / 128 * n * 4, 256); }
int64_t copy_bytes(int64_t rows, int64_t cols) { return round_up(rows * round_up(cols, 16), 256); }
}  // namespace

int64_t linear_work_bytes(int64_t n, int64_t rows, int64_t cols, int copy, int quantize) {
    return 4 * kMostSums + (copy ? copy_bytes(rows, cols) : 0) + (quantize ? codes_bytes(n, cols) : 0);
}

namespace {

// The weight as an operand, copied where its rows cannot be read in place.
int weight_operand(const LinearArgs& a, void* work, bool quantized, hipStream_t stream, Operand* o) {
    o->p = a.weight;
    o->ld = a.weight_ld;
    if (in_place(a.weight, a.weight_ld, a.cols)) return hipSuccess;
    uint8_t* copy = static_cast<uint8_t*>(work) + 4 * kMostSums + (quantized ? codes_bytes(a.n, a.cols) : 0);
    o->p = copy;
    o->ld = round_up(a.cols, 16);
    const int64_t wgs = std::min<int64_t>((a.rows * (o->ld / 4) + kThreads - 1) / kThreads, 16384);
    hipLaunchKernelGGL(copy_weight_kernel, dim3((uint32_t)wgs), dim3(kThreads), 0, stream, a.weight, a.weight_ld, a.rows, a.cols, copy, o->ld);
    return hipGetLastError();
}

}  // namespace

int launch_linear(const LinearArgs& given, void* work, void* stream) {
    ProductArgs g{};
    LinearArgs a = given;
    const hipStream_t s = (hipStream_t)stream;
    const int64_t wide = (a.cols + kTileDim - 1) / kTileDim, width = round_up(a.cols, 16);
    int rc = weight_operand(a, work, a.values != nullptr, s, &g.a);
    if (rc) return rc;
    const bool vec = ((reinterpret_cast<uintptr_t>(a.out) | (uint64_t)(a.out_ld * dtype_size(a.out_type))) & 15u) == 0;
    const StoreEpilogue e{a.out, a.out_ld, 0, a.rows, a.n, a.out_type, 0, vec};
    // Few values are quantized by the product itself: up to four pieces of 8 a
    // thread, in every workgroup anew, for a launch less (one token on 4096 x 4096:
    // 7 us instead of 10 in all).
    const bool inside = a.values && a.n <= 16 && a.n * wide * kTileDim <= 4 * 8 * 64 * kFewKWaves;
    if (a.values && !inside) {
        uint8_t* codes = static_cast<uint8_t*>(work) + 4 * kMostSums;
        float* scales = reinterpret_cast<float*>(codes + round_up(a.n * width, 256));
        rc = launch_quantize(QuantizeArgs{a.values, a.values_type, 0, 0, a.values_ld, a.n, a.cols, codes, width, scales, a.n}, stream);
        if (rc) return rc;
        a.x = Codes{codes, width, scales, a.n, 0};
    }
    g.a.extent = a.rows;
    g.a.k = width;
    g.b = Operand{a.x.p, a.x.ld, a.n, width};
    g.k = a.cols;
    g.grid = a.grid;
    g.grid_m = wide;
    g.grid_k = 1;
    g.blocks_m = (a.rows + kTileDim - 1) / kTileDim;
    g.blocks_k = wide;
    token_scales(g, a.x);
    if (a.n > kFewTokensMost) return product<false, false>(g, a, a.rows, a.n, static_cast<float*>(work), s);
    const RowInputs x{a.values, a.values_type, a.values_ld, (int32_t)a.n, (int32_t)a.cols, (int32_t)(wide * kTileDim), (int32_t)wide};
    return few_tokens(g, inside ? &x : nullptr, e, a.exact, s);
}

int launch_linear_grad_input(const LinearArgs& a, void* work, void* stream) {
    ProductArgs g{};
    const int rc = weight_operand(a, work, false, (hipStream_t)stream, &g.a);
    if (rc) return rc;
    const int64_t wide = (a.cols + kTileDim - 1) / kTileDim;
    g.a.extent = a.cols;
    g.a.k = a.rows;
    g.b = Operand{a.x.p, a.x.ld, a.n, round_up(a.rows, 16)};
    g.k = a.rows;
    g.grid = a.grid;
    g.grid_m = 1;
    g.grid_k = wide;
    g.blocks_m = wide;
    g.blocks_k = (a.rows + kTileDim - 1) / kTileDim;
    token_scales(g, a.x);
    return product<true, false>(g, a, a.cols, a.n, static_cast<float*>(work), (hipStream_t)stream);
}

int launch_linear_grad_weight(const LinearArgs& a, void* work, void* stream) {
    ProductArgs g{};
    g.a = Operand{a.other.p, a.other.ld, a.cols, a.n};
    g.b = Operand{a.x.p, a.x.ld, a.rows, a.n};
    g.k = a.n;
    g.grid = a.other.scales;
    g.grid_m = 1;
    g.grid_k = a.other.scales_ld;
    g.blocks_m = (a.cols + kTileDim - 1) / kTileDim;
    g.blocks_k = (a.n + kTileDim - 1) / kTileDim;
    // tokens of D are rows of dweight here, whose tiles' scales lie side by side
    g.scales = a.x.scales;
    g.scales_ld = a.x.scales_ld;
    g.tiles = kTilesOfK;
    return product<true, true>(g, a, a.cols, a.rows, static_cast<float*>(work), (hipStream_t)stream);
}

}  // namespace bfz

extern "C" int bfz_linear_shape(int32_t product, int64_t n, int64_t rows, int64_t cols, int32_t out_dtype, int64_t* shape) {
    using namespace bfz;
    if (!shape || product < 0 || product > 2 || n < 1 || rows < 1 || cols < 1 || n > (int64_t(1) << 24) || rows > (int64_t(1) << 20) ||
        cols > (int64_t(1) << 20) || (out_dtype != kF32 && out_dtype != kBF16 && out_dtype != kF16 && out_dtype != BFZ_BF16_EXACT))
        return fail(BFZ_EINVAL, "bfz_linear_shape: null pointer, bad sizes or types");
    const int64_t m = product == 0 ? rows : cols, across = product == 2 ? rows : n, k = product == 0 ? cols : product == 1 ? rows : n;
    const int asked = out_dtype == BFZ_BF16_EXACT, type = asked ? kBF16 : out_dtype;
    int64_t out[6];
    if (product == 0 && n <= kFewTokensMost) {
        const int32_t tn = n <= 16 ? 1 : n <= 32 ? 2 : 4;
        const int64_t few[6] = {16 * few_tiles(m, tn), 16 * tn, kFewKWaves, 1, n, exact_few(type, asked, n)};
        std::copy(few, few + 6, out);
    } else {
        const bool exact = exact_products(type, asked);
        const Shape s = shape_of(k, m, across, exact);
        const int64_t cut[6] = {s.tile_m, s.tile_n, s.waves, s.splits, std::min<int64_t>(across, s.whole * s.tile_n), exact};
        std::copy(cut, cut + 6, out);
    }
    std::copy(out, out + 6, shape);
    return BFZ_OK;
}
