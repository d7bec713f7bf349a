// The matrix product under the vocabulary loss and its gradient:
//
//   D[m][n] = sum over k of A[m][k] B[n][k]
//
// in binary32 on the matrix cores, from bf16 or E4M3 A and bf16 B, with the
// result handed in registers to an epilogue (softmax statistics, gradient of
// the logits, or a plain store).
//
// A workgroup of 8 waves owns a 256 x kBN tile and walks k in steps of 64.
// Each step's operands go from memory straight into LDS (16 bytes a lane),
// one step ahead of their use: while a step is multiplied, the next one is in
// flight.  Every step has two halves of 32 k, and a half's fragments are read
// from LDS while the other half is multiplied, so that one barrier a step is
// enough and it falls where all reads of the step are done.
//
// Operands come in two layouts.  KC: k is contiguous (rows of m or n).  KR: m
// or n is contiguous (rows of k); its fragments are read with the LDS
// transpose instructions, so that no operand is ever transposed in memory.
// LDS rows have no padding (the direct loads write lanes back to back);
// instead a row's 16- or 32-byte pieces are permuted by an XOR with its row
// number, chosen so that the lanes that read together touch all banks.
//
// 8192 x 32768 x 4096 runs at 1.13 to 1.39 PFLOP/s (epilogues included; boxes
// differ by 8%), the library's product of two bf16 matrices at 1.31 to 1.49
// there.  The matrix cores are busy 65 to 71% of the cycles with bf16 and 54 to
// 58% with E4M3, at a clock that their load lowers to 1.9 GHz; LDS 17 to 27%.
// What is left is the barrier, where all eight waves meet, and with E4M3 the
// conversions and rescaling (2 vector instructions for each matrix one; 0.7
// with bf16).  Letting two groups of four waves take turns at reading and
// multiplying measured 5-12% slower, rescaling between the matrix instructions
// no faster.
//
// E4M3 codes become bf16 exactly; their tile scales are applied to the
// binary32 sums.  A wave's rows lie in one 128-row tile, so its scale
// changes only with k: the sums are kept in units that follow the current
// tile's scale and multiplied by old / new unit every 128 k.  (A second set of
// sums in unscaled units would not fit the registers.)  The unit's exponent
// never falls, so however the scales fall the sums grow by less than a factor
// of two: a tile whose scale lies 2^e below the unit gives the unit its
// mantissa, and its codes are converted to code * 2^-e, exact in bf16.  What
// lies lower thus keeps its bits also where the sums are still zero, an all-zero
// tile's scale of 1 among them.  Past e = 100 the unit does fall, to 2^100
// times the scale: such sums overflow only past 2^79.
#pragma once

#include <utility>

#include "ops_device.h"
#include "ops_internal.h"

namespace bfz {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef int32_t i32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int kGemmThreads = 512, kGemmWaves = 8;
constexpr int kBM = 256;
constexpr int kBK = 64;
constexpr int kMostFall = 100;  // of a tile's scale below the unit of the sums

struct Operand {
    const void* p;
    int64_t ld;      // bytes from row to row
    int64_t extent;  // valid m (or n)
    int64_t k;       // valid k; beyond both, zero
};

struct GemmArgs {
    Operand a, b;
    int64_t k;             // k to walk
    int64_t k_per_split;   // multiple of 128
    const float* grid;     // scale of A's tile (m / 128, k / 128), or null
    int64_t grid_m, grid_k;      // its strides
    int64_t blocks_m, blocks_k;  // its sizes
    int32_t tiles_m, tiles_n, splits, group_m;
};

// f(0), f(1), ..., f(n - 1) with constant arguments.
template <int... I, class F>
__device__ __forceinline__ void each_of(std::integer_sequence<int, I...>, F&& f) {
    (f(std::integral_constant<int, I>{}), ...);
}
template <int kCount, class F>
__device__ __forceinline__ void each(F&& f) {
    each_of(std::make_integer_sequence<int, kCount>{}, f);
}

constexpr uint32_t kNowhere = 0xFFFFFFF0u;  // beyond every buffer: loads give zero
constexpr uint32_t kBufferBytes = 0x80000000u;

__device__ __forceinline__ i32x4 buffer_of(const char* base) {
    const uint64_t a = reinterpret_cast<uint64_t>(base);
    i32x4 r;
    r[0] = __builtin_amdgcn_readfirstlane((int)(uint32_t)a);
    r[1] = __builtin_amdgcn_readfirstlane((int)((uint32_t)(a >> 32) & 0xFFFFu));
    r[2] = (int)kBufferBytes;
    r[3] = 0x00020000;
    return r;
}

// 16 bytes a lane from memory to LDS at lds + 16 * lane.  In assembly, so
// that the compiler does not wait for it at the next LDS read: it has no
// result register, and wait_loads() stands before the barrier that publishes
// what it wrote.  m0, the LDS address, is a reserved register that the compiler
// sets right before each use of its own (named as clobbered it draws a warning
// and leaves the code as it is).
__device__ __forceinline__ void load_to_lds(const i32x4& buf, uint32_t offset, uint32_t lds) {
    __asm__ volatile(
        "s_mov_b32 m0, %0\n\t"
        "s_nop 0\n\t"
        "buffer_load_dwordx4 %1, %2, 0 offen lds"
        :
        : "s"(lds), "v"(offset), "s"(buf)
        : "memory");
}

__device__ __forceinline__ void wait_loads() { __asm__ volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory"); }

typedef __attribute__((address_space(3))) char lds_char;

__device__ __forceinline__ uint32_t lds_address(const char* p) {
    return (uint32_t)reinterpret_cast<uintptr_t>((lds_char*)p);
}

template <class T>
__device__ __forceinline__ T lds_read(uint32_t at) {
    return *(__attribute__((address_space(3))) const T*)(uintptr_t)at;
}

// ---- operand layouts ----------------------------------------------------------
// kRows: the tile's extent in m or n.  Each gives: bytes of a stage; the loads a
// wave issues for it (offset of load j; which k, or row of k, a lane's load
// covers, for the tail); the registers of a fragment and how it is read.

template <int kRows>
struct BF16KC {
    static constexpr int kBytes = kRows * kBK * 2;
    static constexpr int kLoads = kBytes / 1024 / kGemmWaves;
    static_assert(kLoads >= 1, "a stage has a load for each wave");
    static constexpr int kReads = 1;  // LDS instructions a fragment
    static constexpr bool kScaled = false;
    typedef bf16x8 Frag;
    uint32_t at[2];  // LDS offset of tile 0's fragment, by half
    __device__ __forceinline__ static const char* base(const Operand& o, int64_t row0, int64_t k0) {
        return static_cast<const char*>(o.p) + row0 * o.ld + k0 * 2;
    }
    __device__ __forceinline__ static int64_t advance(const Operand&) { return kBK * 2; }
    __device__ __forceinline__ static int k_of(int, int, int lane) { return 8 * ((lane & 7) ^ (lane >> 3)); }
    __device__ __forceinline__ static uint32_t offset(const Operand& o, int64_t row0, int j, int wave, int lane) {
        const int row = (j * kGemmWaves + wave) * 8 + (lane >> 3);
        return row0 + row < o.extent ? (uint32_t)(row * o.ld) + 16u * ((lane & 7) ^ (lane >> 3)) : kNowhere;
    }
    __device__ __forceinline__ BF16KC(uint32_t lds, int row0, int lane) {
#pragma unroll
        for (int h = 0; h < 2; ++h) at[h] = lds + (row0 + (lane & 15)) * 128 + (((4 * h + (lane >> 4)) ^ (lane & 7)) << 4);
    }
    __device__ __forceinline__ Frag read(uint32_t stage, int h, int t) const {
        return lds_read<bf16x8>(at[h] + stage + t * 2048);
    }
    __device__ __forceinline__ static bf16x8 value(const Frag& f, float) { return f; }
};

__device__ __forceinline__ bf16x8 codes_to_bf16(const u32x2& c, float keep) {
    bf16x8 r;
#pragma unroll
    for (int w = 0; w < 2; ++w) {
        const bf16x2 lo = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c[w], keep, false);
        const bf16x2 hi = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c[w], keep, true);
        r[4 * w] = lo[0];
        r[4 * w + 1] = lo[1];
        r[4 * w + 2] = hi[0];
        r[4 * w + 3] = hi[1];
    }
    return r;
}

template <int kRows>
struct FP8KC {
    static constexpr int kBytes = kRows * kBK;
    static constexpr int kLoads = kBytes / 1024 / kGemmWaves;
    static constexpr int kReads = 1;  // LDS instructions a fragment
    static constexpr bool kScaled = true;
    typedef u32x2 Frag;
    uint32_t at[2];
    __device__ __forceinline__ static const char* base(const Operand& o, int64_t row0, int64_t k0) {
        return static_cast<const char*>(o.p) + row0 * o.ld + k0;
    }
    __device__ __forceinline__ static int64_t advance(const Operand&) { return kBK; }
    __device__ __forceinline__ static int k_of(int, int, int lane) { return 16 * ((lane & 3) ^ ((lane >> 4) & 3)); }
    __device__ __forceinline__ static uint32_t offset(const Operand& o, int64_t row0, int j, int wave, int lane) {
        const int row = (j * kGemmWaves + wave) * 16 + (lane >> 2);
        return row0 + row < o.extent ? (uint32_t)(row * o.ld) + 16u * ((lane & 3) ^ ((lane >> 4) & 3)) : kNowhere;
    }
    __device__ __forceinline__ FP8KC(uint32_t lds, int row0, int lane) {
        const int g = lane >> 4;
#pragma unroll
        for (int h = 0; h < 2; ++h)
            at[h] = lds + (row0 + (lane & 15)) * 64 + (((2 * h + (g >> 1)) ^ ((lane >> 2) & 3)) << 4) + 8 * (g & 1);
    }
    __device__ __forceinline__ Frag read(uint32_t stage, int h, int t) const {
        return lds_read<u32x2>(at[h] + stage + t * 1024);
    }
    __device__ __forceinline__ static bf16x8 value(const Frag& f, float keep) { return codes_to_bf16(f, keep); }
};

// kTiles: the 16-wide tiles a wave reads.
template <int kRows, int kTiles>
struct BF16KR {
    static constexpr int kBytes = kRows * kBK * 2;
    static constexpr int kLoads = kBytes / 1024 / kGemmWaves;
    static constexpr int kPieces = kRows * 2 / 16;  // 16-byte pieces of a row
    static_assert(kRows == 256, "the permutation spans a 512-byte row");
    static constexpr int kReads = 2;  // LDS instructions a fragment
    static constexpr bool kScaled = false;
    typedef bf16x8 Frag;
    uint32_t at[kTiles];
    __device__ __forceinline__ static const char* base(const Operand& o, int64_t row0, int64_t k0) {
        return static_cast<const char*>(o.p) + k0 * o.ld + row0 * 2;
    }
    __device__ __forceinline__ static int64_t advance(const Operand& o) { return kBK * o.ld; }
    __device__ __forceinline__ static int k_of(int j, int wave, int lane) { return (j * kGemmWaves + wave) * 2 + (lane >> 5); }
    __device__ __forceinline__ static uint32_t offset(const Operand& o, int64_t row0, int j, int wave, int lane) {
        const int k = k_of(j, wave, lane);
        const int x = (k & 3) | (((k >> 3) & 3) << 2);
        const int piece = (lane & 31) ^ (x << 1);
        return row0 + 8 * piece < o.extent ? (uint32_t)(k * o.ld) + 16u * piece : kNowhere;
    }
    __device__ __forceinline__ BF16KR(uint32_t lds, int row0, int lane) {
        const int k = 8 * (lane >> 4) + ((lane & 15) >> 2);
#pragma unroll
        for (int t = 0; t < kTiles; ++t)
            at[t] = lds + k * 512 + (((row0 / 16 + t) ^ (lane >> 2)) << 5) + 8 * (lane & 3);
    }
    __device__ __forceinline__ Frag read(uint32_t stage, int h, int t) const {
        typedef short s16x4 __attribute__((ext_vector_type(4)));
        typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
        typedef short s16x8 __attribute__((ext_vector_type(8)));
        const uint32_t p = at[t] + stage + h * 32 * 512;
        const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(uintptr_t)p);
        const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(uintptr_t)(p + 4 * 512));
        const s16x8 r = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
        return __builtin_bit_cast(bf16x8, r);
    }
    __device__ __forceinline__ static bf16x8 value(const Frag& f, float) { return f; }
};

template <int kRows, int kTiles>
struct FP8KR {
    static constexpr int kBytes = kRows * kBK;
    static constexpr int kLoads = kBytes / 1024 / kGemmWaves;
    static_assert(kRows == 256, "the permutation spans a 256-byte row");
    static constexpr int kReads = 1;  // LDS instructions a fragment
    static constexpr bool kScaled = true;
    typedef u32x2 Frag;
    uint32_t at[kTiles];
    __device__ __forceinline__ static const char* base(const Operand& o, int64_t row0, int64_t k0) {
        return static_cast<const char*>(o.p) + k0 * o.ld + row0;
    }
    __device__ __forceinline__ static int64_t advance(const Operand& o) { return kBK * o.ld; }
    __device__ __forceinline__ static int k_of(int j, int wave, int lane) { return (j * kGemmWaves + wave) * 4 + (lane >> 4); }
    __device__ __forceinline__ static uint32_t offset(const Operand& o, int64_t row0, int j, int wave, int lane) {
        const int k = k_of(j, wave, lane);
        const int piece = (lane & 15) ^ (k & 15);
        return row0 + 16 * piece < o.extent ? (uint32_t)(k * o.ld) + 16u * piece : kNowhere;
    }
    __device__ __forceinline__ FP8KR(uint32_t lds, int row0, int lane) {
        const int k = 8 * (lane >> 4) + ((lane & 15) >> 1);
#pragma unroll
        for (int t = 0; t < kTiles; ++t)
            at[t] = lds + k * 256 + (((row0 / 16 + t) ^ (k & 15)) << 4) + 8 * (lane & 1);
    }
    __device__ __forceinline__ Frag read(uint32_t stage, int h, int t) const {
        typedef int i32x2 __attribute__((ext_vector_type(2)));
        typedef __attribute__((address_space(3))) i32x2 lds_i32x2;
        const i32x2 r = __builtin_amdgcn_ds_read_tr8_b64_v2i32((lds_i32x2*)(uintptr_t)(at[t] + stage + h * 32 * 256));
        return __builtin_bit_cast(u32x2, r);
    }
    __device__ __forceinline__ static bf16x8 value(const Frag& f, float keep) { return codes_to_bf16(f, keep); }
};

// ---- tile order -----------------------------------------------------------------
// Workgroups are dealt to the 8 XCDs in turn; each XCD takes one contiguous
// eighth of the tiles, in groups of group_m tiles of m by all n, so the
// workgroups that run on it together share operands in its L2.
__device__ __forceinline__ void tile_of(const GemmArgs& g, int& tm, int& tn, int& split) {
    const int total = g.tiles_m * g.tiles_n * g.splits;
    const int b = blockIdx.x, x = b & 7, each = total >> 3, more = total & 7;
    int l = x * each + min(x, more) + (b >> 3);
    split = l / (g.tiles_m * g.tiles_n);
    l -= split * g.tiles_m * g.tiles_n;
    const int group = l / (g.group_m * g.tiles_n);
    const int m0 = group * g.group_m;
    const int width = min(g.group_m, g.tiles_m - m0);
    const int in = l - group * g.group_m * g.tiles_n;
    tm = m0 + in % width;
    tn = in / width;
}

// Where a wave's results lie: its rows m0 + 16 t + 4 (lane / 16) + i, i < 4, of
// columns n0 + 16 u + lane % 16.
struct WaveTile {
    int64_t m0, n0;
    int tile_m, wave_m, split, lane;
};

template <class A, class B, int kBN, int kWavesM, class Epilogue>
__global__ __launch_bounds__(kGemmThreads, 2) void gemm_kernel(GemmArgs g, Epilogue epilogue) {
    constexpr int kWavesN = kGemmWaves / kWavesM;
    constexpr int kTM = kBM / kWavesM / 16, kTN = kBN / kWavesN / 16;
    static_assert(kTileDim % (kTM * 16) == 0, "a wave's rows share their tile scales");
    constexpr int kStage = A::kBytes + B::kBytes;
    constexpr uint32_t kOther = kStage;  // the second buffer; XOR with it toggles 0 and kStage
    extern __shared__ __attribute__((aligned(16))) char smem[];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave / kWavesN, wn = wave % kWavesN;
    int tm, tn, split;
    tile_of(g, tm, tn, split);
    const int64_t m0 = (int64_t)tm * kBM, n0 = (int64_t)tn * kBN;
    const int64_t k0 = split * g.k_per_split;
    const int64_t k1 = min(g.k, k0 + g.k_per_split);
    const int steps = (int)((max(k1 - k0, (int64_t)0) + kBK - 1) / kBK);

    const uint32_t lds = lds_address(smem);
    const A fa(lds, wm * kTM * 16, lane);
    const B fb(lds + A::kBytes, wn * kTN * 16, lane);
    uint32_t off_a[A::kLoads], off_b[B::kLoads];
#pragma unroll
    for (int j = 0; j < A::kLoads; ++j) off_a[j] = A::offset(g.a, m0, j, wave, lane);
#pragma unroll
    for (int j = 0; j < B::kLoads; ++j) off_b[j] = B::offset(g.b, n0, j, wave, lane);
    const char* base_a = A::base(g.a, m0, k0);
    const char* base_b = B::base(g.b, n0, k0);
    const int64_t adv_a = A::advance(g.a), adv_b = B::advance(g.b);
    const uint32_t lds_a = lds + wave * 1024, lds_b = lds_a + A::kBytes;

    // Loads of the next step into buffer `stage`, `parts` calls of which part
    // p issues its share; past the end of k they give zero (no branch: the
    // lanes' offsets are selected).
    int64_t left_a = g.a.k - k0, left_b = g.b.k - k0;
    constexpr int kLoads = A::kLoads + B::kLoads;
    auto issue = [&](uint32_t stage, auto part, auto of) {
        constexpr int p = decltype(part)::value, parts = decltype(of)::value;
        constexpr int from = p * kLoads / parts, to = (p + 1) * kLoads / parts;
        const i32x4 ra = buffer_of(base_a), rb = buffer_of(base_b);
        const int la = (int)max((int64_t)0, min(left_a, (int64_t)kBK)), lb = (int)max((int64_t)0, min(left_b, (int64_t)kBK));
        each<to - from>([&](auto i) {
            constexpr int j = from + decltype(i)::value;
            if constexpr (j < A::kLoads)
                load_to_lds(ra, A::k_of(j, wave, lane) < la ? off_a[j] : kNowhere, lds_a + stage + j * (kGemmWaves * 1024));
            else
                load_to_lds(rb, B::k_of(j - A::kLoads, wave, lane) < lb ? off_b[j - A::kLoads] : kNowhere,
                            lds_b + stage + (j - A::kLoads) * (kGemmWaves * 1024));
        });
        if constexpr (p + 1 < parts) return;
        base_a += adv_a;
        base_b += adv_b;
        left_a -= kBK;
        left_b -= kBK;
    };

    f32x4 acc[kTM][kTN];
#pragma unroll
    for (int t = 0; t < kTM; ++t)
#pragma unroll
        for (int u = 0; u < kTN; ++u) acc[t][u] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    typename A::Frag a[2][kTM];
    typename B::Frag b[2][kTN];
    auto read_half = [&](uint32_t stage, int h) {
#pragma unroll
        for (int u = 0; u < kTN; ++u) b[h][u] = fb.read(stage, h, u);
#pragma unroll
        for (int t = 0; t < kTM; ++t) a[h][t] = fa.read(stage, h, t);
    };

    // scale of this wave's A tiles in 128-k block kb
    float unit = 1.0f, keep = 1.0f;
    const float* grid_row = nullptr;
    if constexpr (A::kScaled) grid_row = g.grid + min((m0 + wm * kTM * 16) / kTileDim, g.blocks_m - 1) * g.grid_m;
    auto scale_at = [&](int64_t kb) { return grid_row[min(kb, g.blocks_k - 1) * g.grid_k]; };
    float next_scale = 1.0f;
    if constexpr (A::kScaled) unit = next_scale = scale_at(k0 / kTileDim);

    // Half h of a step: its multiplications in kTM parts, with the reads of the
    // other half (from buffer `from`) and, in the second half, the loads of the
    // step after next (into buffer `into`) spread over them.  The order is fixed
    // here: left to itself the compiler issues the reads, or the loads, in a row
    // while the matrix cores wait (8192 x 32768 x 4096, bf16: 1254 TFLOP/s with
    // its order, 1316 with this one; all reads in the first part 1298).
    auto half = [&](auto which, uint32_t from, uint32_t into) {
        constexpr int h = decltype(which)::value;
        bf16x8 av = A::value(a[h][0], keep);
        each<kTM>([&](auto part) {
            constexpr int t = decltype(part)::value;
            each<(t + 1) * kTN / kTM - t * kTN / kTM>([&](auto i) {
                constexpr int u = t * kTN / kTM + decltype(i)::value;
                b[1 - h][u] = fb.read(from, 1 - h, u);
            });
            a[1 - h][t] = fa.read(from, 1 - h, t);
            if constexpr (h == 1) issue(into, part, std::integral_constant<int, kTM>{});
#pragma unroll
            for (int u = 0; u < kTN; ++u)
                acc[t][u] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(av, b[h][u], acc[t][u], 0, 0, 0);
            if constexpr (t + 1 < kTM) av = A::value(a[h][t + 1], keep);
            __builtin_amdgcn_sched_barrier(0);
        });
    };
    constexpr std::integral_constant<int, 0> kNone{};
    constexpr std::integral_constant<int, 1> kOnce{};
    auto step = [&](uint32_t stage) {
        half(kNone, stage, 0);
        wait_loads();
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_sched_barrier(0);
        half(kOnce, stage ^ kOther, stage);
        __builtin_amdgcn_sched_barrier(0);
    };
    if (steps > 0) {
        issue(0, kNone, kOnce);
        issue(kOther, kNone, kOnce);
        wait_loads();
        __builtin_amdgcn_s_barrier();
        read_half(0, 0);
        for (int s = 0;;) {
            if constexpr (A::kScaled) {
                const float scale = next_scale;
                next_scale = scale_at(k0 / kTileDim + s / 2 + 1);
                // a NaN scale has exponent 0 here and leaves the sums NaN; a
                // zero one, which adds nothing, keeps the unit, and the
                // conversion takes 0 as 2^-127 (computing all this between the
                // previous step's multiplications measured 4% slower)
                const int fall = min(max(__builtin_amdgcn_frexp_expf(unit) - __builtin_amdgcn_frexp_expf(scale), 0), kMostFall);
                const bool none = scale == 0.0f;
                const float next = none ? unit : __builtin_amdgcn_ldexpf(scale, fall);
                const float by = none ? 1.0f : unit / next;
                unit = next;
                keep = none ? 0.0f : __uint_as_float((uint32_t)(127 - fall) << 23);
#pragma unroll
                for (int t = 0; t < kTM; ++t)
#pragma unroll
                    for (int u = 0; u < kTN; ++u)
#pragma unroll
                        for (int i = 0; i < 4; ++i) acc[t][u][i] *= by;
            }
            step(0);
            if (++s >= steps) break;
            step(kOther);
            if (++s >= steps) break;
        }
        wait_loads();  // the loads issued past the end
    }
    if constexpr (A::kScaled) {
#pragma unroll
        for (int t = 0; t < kTM; ++t)
#pragma unroll
            for (int u = 0; u < kTN; ++u)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[t][u][i] *= unit;
    }
    const WaveTile w{m0 + wm * kTM * 16, n0 + wn * kTN * 16, tm, wm, split, lane};
    epilogue.template run<kTM, kTN>(acc, w);
}

// ---- few tokens -------------------------------------------------------------------
// The same product for up to 16 tokens in all, bound by reading A once.
// Nothing is staged: four waves of a workgroup take 32 rows of A and share out
// its k in blocks of 128; a lane loads 32 k of one row of A and of one token
// straight into registers, the four lanes of a row 64 bytes side by side, two
// blocks ahead.  Which k a matrix instruction takes is free as long as A and B
// agree.  The waves' sums meet in LDS.  Here a block's sums fit beside the
// total, so tile scales are applied block by block.  One token on 32768 x 4096
// codes: 30 us, 4.5 TB/s (64-wide tiles through LDS: 57 us).  17 tokens and more
// do go through 64-wide tiles, which on a head of under 65536 rows leave CUs
// idle: 17 to 64 tokens 62 to 64 us there, on 131072 rows 143 to 148.
constexpr int kFewRows = 32, kFewTokens = 16, kFewWaves = 4;

template <bool kFp8, class Epilogue>
__global__ __launch_bounds__(64 * kFewWaves) void few_tokens_kernel(GemmArgs g, Epilogue epilogue) {
    constexpr int kSize = kFp8 ? 1 : 2;
    constexpr int kALoads = 2 * kSize, kBLoads = 4;  // 16-byte loads of 32 k
    constexpr int kAhead = 2;
    __shared__ f32x4 part[kFewWaves][2][64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int q = lane >> 4, r = lane & 15;
    const int64_t m0 = (int64_t)blockIdx.x * kFewRows;
    const __amdgpu_buffer_rsrc_t ra = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<char*>(static_cast<const char*>(g.a.p) + m0 * g.a.ld), (short)0, (int)kBufferBytes, 0x00020000);
    const __amdgpu_buffer_rsrc_t rb = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<char*>(static_cast<const char*>(g.b.p)), (short)0, (int)kBufferBytes, 0x00020000);
    uint32_t row_a[2];
#pragma unroll
    for (int t = 0; t < 2; ++t) row_a[t] = m0 + 16 * t + r < g.a.extent ? (uint32_t)((16 * t + r) * g.a.ld) : kNowhere;
    const uint32_t row_b = r < g.b.extent ? (uint32_t)(r * g.b.ld) : kNowhere;
    const float* scales = kFp8 ? g.grid + m0 / kTileDim * g.grid_m : nullptr;
    const int blocks = (int)((g.k + 127) / 128);

    f32x4 acc[2] = {f32x4{0.0f, 0.0f, 0.0f, 0.0f}, f32x4{0.0f, 0.0f, 0.0f, 0.0f}};
    for (int b0 = wave; b0 < blocks; b0 += kFewWaves * kAhead) {
        u32x4 a[kAhead][2][kALoads], b[kAhead][kBLoads];
        float scale[kAhead];
#pragma unroll
        for (int x = 0; x < kAhead; ++x) {
            const int block = b0 + x * kFewWaves;
            const int64_t k0 = (int64_t)block * 128;
            if constexpr (kFp8) scale[x] = scales[min((int64_t)block, g.blocks_k - 1) * g.grid_k];
#pragma unroll
            for (int l = 0; l < kALoads; ++l) {
                const int64_t k = k0 + (4 * l + q) * (16 / kSize);
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    const bool in = k < g.a.k && row_a[t] != kNowhere;
                    a[x][t][l] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(ra, in ? (int)(row_a[t] + (uint32_t)(k * kSize)) : (int)kNowhere, 0, 2));
                }
            }
#pragma unroll
            for (int l = 0; l < kBLoads; ++l) {
                // the k of instruction l: of E4M3, half l % 2 of A's 16 codes
                const int64_t k = kFp8 ? k0 + 64 * (l >> 1) + 16 * q + 8 * (l & 1) : k0 + 32 * l + 8 * q;
                const bool in = k < g.b.k && row_b != kNowhere;
                b[x][l] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rb, in ? (int)(row_b + (uint32_t)(k * 2)) : (int)kNowhere, 0, 0));
            }
        }
        __builtin_amdgcn_sched_barrier(0);  // all of them before the first use
#pragma unroll
        for (int x = 0; x < kAhead; ++x)
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                f32x4 sum = kFp8 ? f32x4{0.0f, 0.0f, 0.0f, 0.0f} : acc[t];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    bf16x8 av;
                    if constexpr (kFp8) av = codes_to_bf16(u32x2{a[x][t][j >> 1][2 * (j & 1)], a[x][t][j >> 1][2 * (j & 1) + 1]}, 1.0f);
                    else av = __builtin_bit_cast(bf16x8, a[x][t][j]);
                    sum = __builtin_amdgcn_mfma_f32_16x16x32_bf16(av, __builtin_bit_cast(bf16x8, b[x][j]), sum, 0, 0, 0);
                }
                acc[t] = kFp8 ? acc[t] + sum * scale[x] : sum;
            }
    }
#pragma unroll
    for (int t = 0; t < 2; ++t) part[wave][t][lane] = acc[t];
    __syncthreads();
    if (wave != 0) return;
    f32x4 sums[2][1];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        sums[t][0] = part[0][t][lane];
#pragma unroll
        for (int w = 1; w < kFewWaves; ++w) sums[t][0] += part[w][t][lane];
    }
    const WaveTile w{m0, 0, (int)blockIdx.x, 0, 0, lane};
    epilogue.template run<2, 1>(sums, w);
}

}  // namespace bfz
