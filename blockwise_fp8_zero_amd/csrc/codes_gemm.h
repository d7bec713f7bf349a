// The matrix product of E4M3 codes with a scale for each block of 128 k:
//
//   D[n][m] = sum over blocks kb of scale_b(n, kb) scale_a(m / 128, kb) P(n, m, kb)
//   P(n, m, kb) = sum over the block's k of A[m][k] B[n][k]
//
// A block's sum P is one matrix instruction of 128 k (or four of 32, below), its
// scaling one fused operation for each result: while a row of tiles is
// multiplied, the sums of the row before are scaled and added.
//
// A workgroup owns a tile of D and walks k a block at a time.  A block's operands go
// from memory straight into LDS (16 bytes a lane), into one of two to four buffers.
// When a wave has read the last of a block it meets the others; the loads of the
// block that many ahead then go into the buffer just read, and the last row of tiles
// is multiplied while the next block's first fragments are read.
//
// Operands come in two layouts, so that no operand is ever transposed in memory:
// KC, k contiguous, and KR, m or n contiguous (rows of k), read with the LDS
// transpose instruction.  Which k of a block a lane holds is free as long as both
// operands agree: lane group g = lane / 16 holds k 16 g to 16 g + 15 and 64 + 16 g
// on.  LDS rows have no padding (the direct loads write lanes back to back);
// their 16-byte pieces are permuted by an XOR with the row, chosen so that the
// lanes that read together touch all banks.
//
// 8192 x 11008 x 4096 runs at 2.27 to 2.48 PFLOP/s, the matrix cores busy 50 to 58% of
// the cycles (46% with bf16 instructions) at a clock that their load lowers to 1.8 to
// 1.9 GHz.  Without the scaling's
// vector instructions it would be 8% faster, without the loads from memory 20%.  What
// is left is the wait where all eight waves meet.  Fixing the order of reads and
// loads gave 7%, spreading the loads over half of a block's rows of tiles 3%, half
// as wide tiles in the last round 4 to 5%.  A walk over tiles that loads the next one
// ahead of its results did not fit the registers.
//
// kExact: the E4M3 matrix instructions align 8 products to the largest and keep
// 13 bits below its exponent, cut off towards zero.  That is some 5e-5 of a result:
// a bfloat16 one does not show it beside the 1.7e-3 of its own rounding (both come
// to the same 1.7e-3 from 64-bit results), a float16 one, whose rounding is 2e-4,
// and a float32 one do, and so would sums that cancel.  Those take bf16
// instructions on the codes' values, whose products are exact and whose sums are
// binary32, at half the rate.
#pragma once

#include <type_traits>

#include "vocab_gemm.h"

namespace bfz {

typedef int i32x8 __attribute__((ext_vector_type(8)));

// Where B's scales lie: [k / 128][n], or by 128x128 tile [n / 128][k / 128] or
// [k / 128][n / 128], rows scales_ld apart.
constexpr int kEachOfN = 0, kTilesOfN = 1, kTilesOfK = 2;

typedef __attribute__((address_space(3))) const char* lds_pointer;

template <class T>
__device__ __forceinline__ T lds_at(lds_pointer p) {
    return *(__attribute__((address_space(3))) const T*)p;
}

struct ProductArgs : GemmArgs {  // grid: scale of (m / 128, k / 128) at grid_m, grid_k; k_per_split a multiple of 128
    const float* scales;
    int64_t scales_ld;
    int32_t tiles;
    int32_t half_tiles_n;  // columns of tiles half as wide, after the tiles_n others
};

// ---- operand layouts ----------------------------------------------------------

template <int kRows, int kWaves>
struct CodesKC {
    static constexpr int kBytes = kRows * 128;
    static constexpr int kLoads = kBytes / 1024 / kWaves;
    static_assert(kLoads >= 1 && kBytes % (1024 * kWaves) == 0, "whole loads for each wave");
    uint32_t at[2];  // LDS offset of tile 0's fragment, by half
    __device__ __forceinline__ static const char* base(const Operand& o, int64_t row0, int64_t k0) {
        return static_cast<const char*>(o.p) + row0 * o.ld + k0;
    }
    __device__ __forceinline__ static int64_t advance(const Operand&) { return 128; }
    // k that lane `lane` of load j covers from; the same for every load
    __device__ __forceinline__ static int k_of(int, int, int lane) { return 16 * ((lane & 7) ^ (lane >> 3)); }
    __device__ __forceinline__ static uint32_t offset(const Operand& o, int64_t row0, int j, int wave, int lane) {
        const int row = (j * kWaves + wave) * 8 + (lane >> 3);
        return row0 + row < o.extent ? (uint32_t)(row * o.ld) + 16u * ((lane & 7) ^ (lane >> 3)) : kNowhere;
    }
    __device__ __forceinline__ CodesKC(uint32_t lds, int row0, int lane) {
#pragma unroll
        for (int h = 0; h < 2; ++h) at[h] = lds + (row0 + (lane & 15)) * 128 + (((4 * h + (lane >> 4)) ^ (lane & 7)) << 4);
    }
    __device__ __forceinline__ i32x8 read(uint32_t stage, int t) const {
        const i32x4 lo = lds_read<i32x4>(at[0] + stage + t * 2048), hi = lds_read<i32x4>(at[1] + stage + t * 2048);
        return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    }
};

// kTiles: the 16-wide tiles a wave reads.
template <int kRows, int kWaves, int kTiles>
struct CodesKR {
    static constexpr int kBytes = kRows * 128;
    static constexpr int kLoads = kBytes / 1024 / kWaves;
    static_assert(kLoads >= 1 && kBytes % (1024 * kWaves) == 0, "whole loads for each wave");
    static_assert(kRows == 256 || kRows == 128 || kRows == 64, "the permutation spans 256 bytes");
    static constexpr int kPieces = kRows / 16, kRowsOfLoad = 64 / kPieces;
    uint32_t at[kTiles];
    // by which a row's pieces are permuted: 8 rows that one transpose reads, of
    // two lane groups, fall on 16 different pieces of 256 bytes
    __device__ __forceinline__ static int mix(int k) {
        return kRows == 256 ? (k & 7) | ((k >> 1) & 8) : kRows == 128 ? ((k >> 1) & 3) | ((k >> 2) & 4) : ((k >> 2) & 1) | ((k >> 3) & 2);
    }
    __device__ __forceinline__ static const char* base(const Operand& o, int64_t row0, int64_t k0) {
        return static_cast<const char*>(o.p) + k0 * o.ld + row0;
    }
    __device__ __forceinline__ static int64_t advance(const Operand& o) { return 128 * o.ld; }
    __device__ __forceinline__ static int k_of(int j, int wave, int lane) { return (j * kWaves + wave) * kRowsOfLoad + lane / kPieces; }
    __device__ __forceinline__ static uint32_t offset(const Operand& o, int64_t row0, int j, int wave, int lane) {
        const int k = k_of(j, wave, lane);
        const int piece = (lane & (kPieces - 1)) ^ mix(k);
        return row0 + 16 * piece < o.extent ? (uint32_t)(k * o.ld) + 16u * piece : kNowhere;
    }
    __device__ __forceinline__ CodesKR(uint32_t lds, int row0, int lane) {
        const int k = 16 * (lane >> 4) + ((lane & 15) >> 1);
#pragma unroll
        for (int t = 0; t < kTiles; ++t) at[t] = lds + k * kRows + (((row0 / 16 + t) ^ mix(k)) << 4) + 8 * (lane & 1);
    }
    __device__ __forceinline__ i32x8 read(uint32_t stage, int t) const {
        typedef int i32x2 __attribute__((ext_vector_type(2)));
        typedef __attribute__((address_space(3))) i32x2 lds_i32x2;
        const uint32_t p = at[t] + stage;
        i32x8 r;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            // bits 3 and 6 of k do not enter mix
            const i32x2 x = __builtin_amdgcn_ds_read_tr8_b64_v2i32((lds_i32x2*)(uintptr_t)(p + (64 * (j >> 1) + 8 * (j & 1)) * kRows));
            r[2 * j] = x[0];
            r[2 * j + 1] = x[1];
        }
        return r;
    }
};

// ---- the kernel -----------------------------------------------------------------

// A fragment's values in kParts parts, whose products add up to the block's.
template <bool kExact>
struct Multiply;

template <>
struct Multiply<false> {
    static constexpr int kParts = 1;
    typedef i32x8 Value;
    __device__ __forceinline__ static Value value(const i32x8& f, int) { return f; }
    __device__ __forceinline__ static f32x4 run(const Value& a, const Value& b, const f32x4& c) {
        return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 0, 0, 0, 0, 0, 0);
    }
};

template <>
struct Multiply<true> {
    static constexpr int kParts = 4;
    typedef bf16x8 Value;
    __device__ __forceinline__ static Value value(const i32x8& f, int j) {
        return codes_to_bf16(u32x2{(uint32_t)f[2 * j], (uint32_t)f[2 * j + 1]}, 1.0f);
    }
    __device__ __forceinline__ static f32x4 run(const Value& a, const Value& b, const f32x4& c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
    }
};

// Tile l of a grid of them: workgroups are dealt to the 8 XCDs in turn; each XCD
// takes one contiguous eighth, in groups of group_m tiles of m by all n, so the
// workgroups that run on it together share operands in its L2.
__device__ __forceinline__ void place_of(int b, int tiles_m, int tiles_n, int splits, int group_m, int& tm, int& tn, int& split) {
    const int total = tiles_m * tiles_n * splits;
    const int x = b & 7, each = total >> 3, more = total & 7;
    int l = x * each + min(x, more) + (b >> 3);
    split = l / (tiles_m * tiles_n);
    l -= split * tiles_m * tiles_n;
    const int group = l / (group_m * tiles_n);
    const int m0 = group * group_m;
    const int width = min(group_m, tiles_m - m0);
    const int in = l - group * group_m * tiles_n;
    tm = m0 + in % width;
    tn = in / width;
}

// 4 bytes a lane from memory to LDS at lds + 4 * lane.
__device__ __forceinline__ void load_word_to_lds(const i32x4& buf, uint32_t offset, uint32_t lds) {
    __asm__ volatile(
        "s_mov_b32 m0, %0\n\t"
        "s_nop 0\n\t"
        "buffer_load_dword %1, %2, 0 offen lds"
        :
        : "s"(lds), "v"(offset), "s"(buf)
        : "memory");
}

template <int kCount>
__device__ __forceinline__ void wait_all_but() {
    __asm__ volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(kCount) : "memory");
}

// One tile.  Everything that the loop loads goes through LDS, scales included, in
// kStages buffers, by loads that the compiler does not count: a wave waits for the
// block it needs next and leaves those behind it in flight.
template <class A, class B, int kTileM, int kTileN, int kWavesM, int kWavesN, int kStages, bool kExact, class Epilogue>
__device__ __forceinline__ void run_tile(const ProductArgs& g, const Epilogue& epilogue, uint32_t lds, int tm, int split, int64_t n0) {
    constexpr int kTM = kTileM / kWavesM / 16, kTN = kTileN / kWavesN / 16;
    static_assert(kTileDim % (kTM * 16) == 0, "a wave's rows lie in one tile");
    constexpr uint32_t kScales = A::kBytes + B::kBytes;  // of the tile's tokens, behind the operands
    constexpr uint32_t kStage = kScales + 4 * kTileN;
    constexpr int kWaves = kWavesM * kWavesN;
    typedef Multiply<kExact> Mul;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave / kWavesN, wn = wave % kWavesN;
    const int64_t m0 = (int64_t)tm * kTileM;
    const int64_t k0 = split * g.k_per_split;
    const int64_t k1 = min(g.k, k0 + g.k_per_split);
    const int steps = (int)((k1 - k0 + kTileDim - 1) / kTileDim);
    const int64_t mw = m0 + wm * kTM * 16, nw = n0 + wn * kTN * 16;

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

    // Scales: each wave loads those of 64 tokens, in turn over the tile's (which
    // several waves load where it has fewer than 64 a wave: the same values).
    // Tokens beyond the last have its tile's, or zero.
    const int first = 64 * (wave % (kTileN / 64)) + lane;
    const int64_t tile0 = n0 / kTileDim, tile = min(n0 + first, g.b.extent - 1) / kTileDim;
    const bool each_n = g.tiles == kEachOfN;
    const uint32_t off_s = each_n ? (n0 + first < g.b.extent ? 4u * first : kNowhere)
                                  : (uint32_t)(4 * (tile - tile0) * (g.tiles == kTilesOfN ? g.scales_ld : 1));
    const char* base_s = reinterpret_cast<const char*>(g.tiles == kTilesOfN ? g.scales + tile0 * g.scales_ld + k0 / kTileDim
                                                                            : g.scales + k0 / kTileDim * g.scales_ld + (each_n ? n0 : tile0));
    const int64_t adv_s = 4 * (g.tiles == kTilesOfN ? 1 : g.scales_ld);
    const uint32_t lds_s = lds + kScales + 256 * (wave % (kTileN / 64));
    const uint32_t at_s = lds + kScales + 4 * (wn * kTN * 16 + (lane & 15));

    // Loads of the next block into buffer `stage`, `parts` calls of which part p
    // issues its share; past the end of k they give zero (no branch: the lanes'
    // offsets are selected).
    int left_a = (int)(g.a.k - k0), left_b = (int)(g.b.k - k0);
    constexpr int kLoads = A::kLoads + B::kLoads;
    auto issue = [&](uint32_t stage, auto part, auto of) {
        constexpr int p = decltype(part)::value, parts = decltype(of)::value;
        constexpr int from = p * kLoads / parts, to = (p + 1) * kLoads / parts;
        const i32x4 ra = buffer_of(base_a), rb = buffer_of(base_b);
        if constexpr (p == 0) {
            load_word_to_lds(buffer_of(base_s), left_b > 0 ? off_s : kNowhere, lds_s + stage);
            base_s += adv_s;
        }
        each<to - from>([&](auto i) {
            constexpr int j = from + decltype(i)::value;
            if constexpr (j < A::kLoads)
                load_to_lds(ra, A::k_of(j, wave, lane) < left_a ? off_a[j] : kNowhere, lds_a + stage + j * (kWaves * 1024));
            else
                load_to_lds(rb, B::k_of(j - A::kLoads, wave, lane) < left_b ? off_b[j - A::kLoads] : kNowhere,
                            lds_b + stage + (j - A::kLoads) * (kWaves * 1024));
        });
        if constexpr (p + 1 < parts) return;
        base_a += adv_a;
        base_b += adv_b;
        left_a -= kTileDim;
        left_b -= kTileDim;
    };
    constexpr std::integral_constant<int, 0> kNone{};
    constexpr std::integral_constant<int, 1> kOnce{};

    // the rows' scale of a block, by a scalar load
    typedef __attribute__((address_space(4))) const float constant_float;
    const float* scale_a = g.grid + min(mw / kTileDim, g.blocks_m - 1) * g.grid_m + k0 / kTileDim * g.grid_k;
    float next_a, now[kTN], by[kTN];
    auto load_scale = [&]() {
        next_a = *(constant_float*)(uintptr_t)scale_a;
        scale_a += g.grid_k;
    };
    auto take_scales = [&](uint32_t stage) {
#pragma unroll
        for (int u = 0; u < kTN; ++u) now[u] = lds_at<float>((lds_pointer)(uintptr_t)(at_s + stage) + 64 * u) * next_a;
    };

    f32x4 acc[kTM][kTN];
#pragma unroll
    for (int t = 0; t < kTM; ++t)
#pragma unroll
        for (int u = 0; u < kTN; ++u) acc[t][u] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

    // A block's loads go out over kSpread rows of tiles, from the last row of the
    // block before on: all at once they fill the queue, and a wave that waits
    // there cannot multiply.
    constexpr int kSpread = kTM / 2;
    constexpr std::integral_constant<int, kSpread> kParted{};
    load_scale();
    each<kStages - 1>([&](auto i) { issue(decltype(i)::value * kStage, kNone, kOnce); });
    uint32_t cur = 0, into = (kStages - 1) * kStage;
    issue(into, kNone, kParted);
    wait_all_but<(kStages - 2) * (kLoads + 1) + kLoads / kSpread + 1>();
    __builtin_amdgcn_s_barrier();
    take_scales(0);
    constexpr int kParts = Mul::kParts;
    // Rows of A are read kAhead rows before their use: two where they are converted
    // during the row before.
    constexpr int kAhead = kExact ? 2 : 1;
    i32x8 a[2], raw[kTN];
    typename Mul::Value av[kParts], b[kTN][kParts];
    f32x4 part[kTN];
    a[0] = fa.read(0, 0);
    if constexpr (kAhead == 2) a[1] = fa.read(0, 1);
#pragma unroll
    for (int u = 0; u < kTN; ++u) raw[u] = fb.read(0, u);
#pragma unroll
    for (int j = 0; j < kParts; ++j) av[j] = Mul::value(a[0], j);
    auto scale_row = [&](auto row, auto col) {
        constexpr int t = decltype(row)::value, u = decltype(col)::value;
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[t][u][i] = __builtin_fmaf(part[u][i], by[u], acc[t][u][i]);
    };
#pragma unroll
    for (int u = 0; u < kTN; ++u) {
        part[u] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        by[u] = 0.0f;
    }
    for (int s = 0; s < steps; ++s) {
        if (s + 1 < steps) load_scale();
        each<kTM>([&](auto row) {
            constexpr int t = decltype(row)::value;
            constexpr bool kLast = t == kTM - 1;
            if constexpr (kLast) {
                // every fragment of this block is read; the next block has arrived
                wait_all_but<(kStages - 2) * (kLoads + 1)>();
                __builtin_amdgcn_s_barrier();
                __builtin_amdgcn_sched_barrier(0);
                into = cur;
                cur = cur + kStage == kStages * kStage ? 0 : cur + kStage;
                take_scales(cur);
            }
            if constexpr (kAhead == 1) {
                a[(t + 1) & 1] = fa.read(cur, kLast ? 0 : t + 1);
            } else if constexpr (kLast) {
                a[(t + 1) & 1] = fa.read(cur, 0);
                a[t & 1] = fa.read(cur, 1);
            } else if constexpr (t + 2 < kTM) {
                a[t & 1] = fa.read(cur, t + 2);
            }
            __builtin_amdgcn_sched_barrier(0);
            f32x4 p[kTN];
            each<kParts * kTN>([&](auto both) {
                constexpr int j = decltype(both)::value / kTN, u = decltype(both)::value % kTN;
                constexpr std::integral_constant<int, u> col{};
                if constexpr (t == 0) b[u][j] = Mul::value(raw[u], j);
                p[u] = Mul::run(av[j], b[u][j], j == 0 ? f32x4{0.0f, 0.0f, 0.0f, 0.0f} : p[u]);
                if constexpr (kLast && j == kParts - 1) raw[u] = fb.read(cur, u);
                if constexpr (j == 0 && u == 1 && kLast) issue(into, kNone, kParted);
                if constexpr (j == 0 && u == 1 && t + 1 < kSpread) issue(into, std::integral_constant<int, (t + 1) % kSpread>{}, kParted);
                if constexpr (j == 0) {
                    scale_row(std::integral_constant<int, (t + kTM - 1) % kTM>{}, col);
                    if constexpr (t == 0) by[u] = now[u];
                }
                // the next row's values, a part at a time, once this row's are used
                if constexpr (u == kTN - 1 && !(kLast && kAhead == 2)) av[j] = Mul::value(a[(t + 1) & 1], j);
                __builtin_amdgcn_sched_barrier(0);
            });
            if constexpr (kLast && kAhead == 2) {
#pragma unroll
                for (int j = 0; j < kParts; ++j) av[j] = Mul::value(a[(t + 1) & 1], j);
            }
#pragma unroll
            for (int u = 0; u < kTN; ++u) part[u] = p[u];
        });
    }
    each<kTN>([&](auto col) { scale_row(std::integral_constant<int, kTM - 1>{}, col); });
    wait_loads();  // the loads issued past the end
    const WaveTile w{mw, nw, tm, wm, split, lane};
    epilogue.template run<kTM, kTN>(acc, w);
}

// Operands and LDS of a tile of this shape.
template <bool kAKR, bool kBKR, int kTileM, int kTileN, int kWaves>
struct TileOf {
    template <bool kKR, int kRows, int kTiles>
    using Layout = std::conditional_t<kKR, CodesKR<kRows, kWaves, kTiles>, CodesKC<kRows, kWaves>>;
    static constexpr int kStage = 128 * (kTileM + kTileN) + 4 * kTileN;
};

// Whole tiles, then, where a last round of them would leave CUs idle, tiles half as
// wide for the last columns.
template <bool kAKR, bool kBKR, int kTileM, int kTileN, int kWavesM, int kWavesN, int kStages, bool kExact, bool kHalves, class Epilogue>
__global__ __launch_bounds__(64 * kWavesM * kWavesN, 2) void codes_gemm_kernel(ProductArgs g, Epilogue epilogue) {
    typedef TileOf<kAKR, kBKR, kTileM, kTileN, kWavesM * kWavesN> Tile;
    typedef typename Tile::template Layout<kAKR, kTileM, kTileM / kWavesM / 16> A;
    extern __shared__ __attribute__((aligned(16))) char smem[];
    const uint32_t lds = lds_address(smem);
    const int whole = g.tiles_m * g.tiles_n * g.splits;
    int tm, tn, split;
    if (!kHalves || (int)blockIdx.x < whole) {
        typedef typename Tile::template Layout<kBKR, kTileN, kTileN / kWavesN / 16> B;
        place_of(blockIdx.x, g.tiles_m, g.tiles_n, g.splits, g.group_m, tm, tn, split);
        run_tile<A, B, kTileM, kTileN, kWavesM, kWavesN, kStages, kExact>(g, epilogue, lds, tm, split, (int64_t)tn * kTileN);
    } else if constexpr (kHalves) {
        typedef typename Tile::template Layout<kBKR, kTileN / 2, kTileN / 2 / kWavesN / 16> Half;
        place_of(blockIdx.x - whole, g.tiles_m, g.half_tiles_n, 1, g.group_m, tm, tn, split);
        run_tile<A, Half, kTileM, kTileN / 2, kWavesM, kWavesN, kStages, kExact>(g, epilogue, lds, tm, split, (int64_t)g.tiles_n * kTileN + (int64_t)tn * (kTileN / 2));
    }
}

// ---- few tokens -------------------------------------------------------------------
// The same product, both operands with k contiguous, for up to 16 kTN tokens in
// all, bound by reading A once.  Nothing is staged: eight waves of a workgroup take
// 16 kTM rows of A and share out the blocks of k; a lane loads its fragments of
// rows and tokens straight into registers, two or
// four rounds ahead.  The waves' sums meet
// in LDS.  kQuantize: B is a matrix of values, which each workgroup quantizes by
// rows into LDS while its first loads of A are under way.
constexpr int kFewKWaves = 8;

template <int kTM, int kTN, bool kExact, bool kQuantize, class Inputs, class Epilogue>
__global__ __launch_bounds__(64 * kFewKWaves) void few_codes_kernel(ProductArgs g, Inputs inputs, Epilogue epilogue) {
    constexpr int kAhead = kTM == 1 ? 4 : 2;  // rounds in registers
    typedef Multiply<kExact> Mul;
    __shared__ f32x4 sums[kFewKWaves][kTM][kTN][64];
    extern __shared__ __attribute__((aligned(16))) char smem[];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int q = lane >> 4, r = lane & 15;
    const int64_t m0 = (int64_t)blockIdx.x * (16 * kTM);
    const __amdgpu_buffer_rsrc_t ra = __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(static_cast<const char*>(g.a.p) + m0 * g.a.ld), (short)0,
                                                                        (int)kBufferBytes, 0x00020000);
    const __amdgpu_buffer_rsrc_t rb = __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(static_cast<const char*>(g.b.p)), (short)0, (int)kBufferBytes,
                                                                        0x00020000);
    const int blocks = (int)((g.k + kTileDim - 1) / kTileDim);
    const int last = (int)g.b.extent - 1;

    struct Round {
        i32x8 a[kTM], b[kTN];
        float scale[kTN], rows[kTM];
    };
    auto fragment = [&](const __amdgpu_buffer_rsrc_t& buf, uint32_t row, bool there, int kb, int64_t k) {
        i32x4 half[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int at = kb * kTileDim + 64 * h + 16 * q;
            half[h] = __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(buf, there && at < k ? (int)(row + (uint32_t)at) : (int)kNowhere, 0, 0));
        }
        return __builtin_shufflevector(half[0], half[1], 0, 1, 2, 3, 4, 5, 6, 7);
    };
    auto load_a = [&](Round& x, int kb) {
#pragma unroll
        for (int t = 0; t < kTM; ++t) {
            x.a[t] = fragment(ra, (uint32_t)((16 * t + r) * g.a.ld), m0 + 16 * t + r < g.a.extent, kb, g.a.k);
            // 16 rows lie in one tile, 48 may not
            x.rows[t] = g.grid[min((m0 + 16 * t) / kTileDim, g.blocks_m - 1) * g.grid_m + min(kb, blocks - 1) * g.grid_k];
        }
    };
    auto load_b = [&](Round& x, int kb) {
        const int at = min(kb, blocks - 1);
#pragma unroll
        for (int u = 0; u < kTN; ++u) {
            const int token = min(16 * u + r, last);
            if constexpr (kQuantize) {
                x.b[u] = inputs.fragment(smem, 16 * u + r, kb, q);
                x.scale[u] = inputs.scale(smem, token, at);
            } else {
                x.b[u] = fragment(rb, (uint32_t)(token * g.b.ld), 16 * u + r <= last, kb, g.b.k);
                x.scale[u] = g.scales[g.tiles == kTilesOfN ? token / kTileDim * g.scales_ld + at : at * g.scales_ld + token];
            }
        }
    };
    Round x[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) load_a(x[i], wave + i * kFewKWaves);
    if constexpr (kQuantize) {
        inputs.quantize(smem);
        __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) load_b(x[i], wave + i * kFewKWaves);

    f32x4 acc[kTM][kTN];
#pragma unroll
    for (int t = 0; t < kTM; ++t)
#pragma unroll
        for (int u = 0; u < kTN; ++u) acc[t][u] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    for (int b0 = wave; b0 < blocks; b0 += kAhead * kFewKWaves) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int kb = b0 + i * kFewKWaves;
            if (kb >= blocks) break;
            Round& y = x[i];
            // a row of tiles at a time, whose tokens' codes are converted anew:
            // their values for all rows would not fit the registers
#pragma unroll
            for (int t = 0; t < kTM; ++t) {
                typename Mul::Value av[Mul::kParts];
#pragma unroll
                for (int j = 0; j < Mul::kParts; ++j) av[j] = Mul::value(y.a[t], j);
#pragma unroll
                for (int u = 0; u < kTN; ++u) {
                    __asm__("" : "+v"(y.b[u]));  // not the values of the row before
                    f32x4 part = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int j = 0; j < Mul::kParts; ++j) part = Mul::run(av[j], Mul::value(y.b[u], j), part);
                    const float by = y.scale[u] * y.rows[t];
#pragma unroll
                    for (int l = 0; l < 4; ++l) acc[t][u][l] = __builtin_fmaf(part[l], by, acc[t][u][l]);
                }
            }
            const int next = kb + kAhead * kFewKWaves;
            if (next < blocks) {
                load_a(y, next);
                load_b(y, next);
            }
        }
    }
#pragma unroll
    for (int t = 0; t < kTM; ++t)
#pragma unroll
        for (int u = 0; u < kTN; ++u) sums[wave][t][u][lane] = acc[t][u];
    __syncthreads();
    for (int i = wave; i < kTM * kTN; i += kFewKWaves) {
        const int t = i / kTN, u = i % kTN;
        f32x4 sum = sums[0][t][u][lane];
#pragma unroll
        for (int w = 1; w < kFewKWaves; ++w) sum += sums[w][t][u][lane];
        epilogue.put4(16 * u + r, m0 + 16 * t + 4 * q, sum);
    }
}

}  // namespace bfz
