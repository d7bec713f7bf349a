// Token embedding from a row-major table (f32, bf16, fp16, or E4M3 codes
// with their 128x128 tile scales), and the table's gradient by sorted tokens.
//
//   out[n]    = scale * table[id[n]]           (zero for an id outside the table)
//   dtable[v] = (dtable[v] +) scale * sum over n with id[n] = v of dout[n]
//
// Both move bytes and compute next to nothing: the bound is HBM, or at few
// tokens the launches.  32768 tokens of 131072 x 4096: the lookup of E4M3 rows
// to bf16 80 us (4.0 TB/s of the bytes it cannot do without; bf16 rows 98, f32
// 148 us, 5.5 TB/s), the gradient from bf16 into f32 492 us: sort of the runs 24,
// merge and zero rows 328 (5.9 TB/s), sums 130, joins 15; into bf16 310 us.  A
// token that fills half the batch or all of it costs no more (522, 517 us).  3001
// tokens onto a tied 50001 x 1000 gradient: 19 us in three dependent launches of
// 5.5, 7.4 and 5.6.  One token of E4M3 rows: 2 us of a 7 us call.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "ops_device.h"
#include "ops_internal.h"

#pragma clang fp contract(off)

namespace bfz {
namespace {

constexpr int kThreads = 256;

// ---------------------------------------------------------------------
// Lookup.  A thread moves one piece of kVec elements; a workgroup takes one
// token (rows of 256 pieces or more) or 256 / pieces tokens.  Rows of odd width
// or alignment go element by element: 32768 tokens of 1001 E4M3 columns 41 us,
// of 1000 19 us.
// ---------------------------------------------------------------------

// kVec consecutive table elements as floats.
template <class T, int kVec>
struct Piece {
    static __device__ __forceinline__ void load(const T* p, float (&x)[kVec]) {
        if constexpr (kVec == 8) {
            load8(p, x);
        } else {
#pragma unroll
            for (int l = 0; l < kVec; ++l) x[l] = Elem<T>::get(p[l]);
        }
    }
};

template <int kVec>
struct Piece<uint8_t, kVec> {
    static __device__ __forceinline__ void load(const uint8_t* p, float (&x)[kVec]) {
        typedef uint32_t words __attribute__((ext_vector_type(kVec / 4 > 0 ? kVec / 4 : 1)));
        words w;
        if constexpr (kVec == 1) w = *p;
        else w = *reinterpret_cast<const words*>(p);
#pragma unroll
        for (int l = 0; l < kVec; ++l) {
            uint32_t v;
            if constexpr (kVec <= 4) v = (uint32_t)w[0];
            else v = w[l >> 2];
            switch (l & 3) {
                case 0: x[l] = __builtin_amdgcn_cvt_f32_fp8((int)v, 0); break;
                case 1: x[l] = __builtin_amdgcn_cvt_f32_fp8((int)v, 1); break;
                case 2: x[l] = __builtin_amdgcn_cvt_f32_fp8((int)v, 2); break;
                default: x[l] = __builtin_amdgcn_cvt_f32_fp8((int)v, 3); break;
            }
        }
    }
};

template <class T, int kVec>
__device__ __forceinline__ void store_piece(T* p, const float (&x)[kVec]) {
    if constexpr (kVec >= 8) {
#pragma unroll
        for (int h = 0; h < kVec / 8; ++h) {
            float y[8];
#pragma unroll
            for (int l = 0; l < 8; ++l) y[l] = x[8 * h + l];
            store8(p + 8 * h, y);
        }
    } else if constexpr (kVec == 4) {
        typedef uint32_t words __attribute__((ext_vector_type(sizeof(T))));  // 4 elements
        words w;
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int l = 0; l < 4; ++l) w[l] = __float_as_uint(x[l]);
        } else {
            w[0] = pack2<T>(x[0], x[1]);
            w[1] = pack2<T>(x[2], x[3]);
        }
        *reinterpret_cast<words*>(p) = w;
    } else {
#pragma unroll
        for (int l = 0; l < kVec; ++l) p[l] = Elem<T>::to(x[l]);
    }
}

template <class T, class O, int kVec>
__global__ __launch_bounds__(kThreads) void embed_kernel(EmbedArgs a, int32_t pieces, int32_t tokens_per_wg) {
    const T* table = static_cast<const T*>(a.table);
    O* out = static_cast<O*>(a.out);
    const int64_t wb = (a.dim + kTileDim - 1) / kTileDim;
    const int local = tokens_per_wg > 1 ? (int)threadIdx.x / pieces : 0;
    const int first = (int)threadIdx.x - local * pieces;
    if (local >= tokens_per_wg) return;
    for (int64_t n = (int64_t)blockIdx.x * tokens_per_wg + local; n < a.n; n += (int64_t)gridDim.x * tokens_per_wg) {
        const int64_t row = row_of(a.ids, a.ids64, n, a.vocab);
        O* dst = out + n * a.out_ld;
        for (int p = first; p < pieces; p += kThreads) {
            const int64_t c = (int64_t)p * kVec;
            float x[kVec];
#pragma unroll
            for (int l = 0; l < kVec; ++l) x[l] = 0.0f;
            if (row >= 0) {
                Piece<T, kVec>::load(table + row * a.table_ld + c, x);
                // the value first: a code of 0 stays 0 where the two scales'
                // product would overflow
                if constexpr (sizeof(T) == 1) {
                    const float g = a.grid[(row / kTileDim) * wb + c / kTileDim];
#pragma unroll
                    for (int l = 0; l < kVec; ++l) x[l] *= g;
                }
#pragma unroll
                for (int l = 0; l < kVec; ++l) x[l] *= a.scale;
            }
            store_piece<O, kVec>(dst + c, x);
        }
    }
}

// ---------------------------------------------------------------------
// Stable sort of the tokens by id.  Runs of kRun tokens are ranked by
// counting: every token is compared with every token of its run, two VALU
// operations a pair, the ids read from LDS by all lanes at once (32768 tokens
// 24 us; merges of 2048-token runs by sixteen searches, live or not, took 23 us
// for 3001 tokens, where one run of 4096 needs none).  Then up to
// sixteen runs at a time are merged by binary search: a token's place is its
// place in its own run plus, for each other run, how many of that run's come
// before it.  Ids outside the table get the key `vocab` and sort last.  One
// launch up to 4096 tokens, two up to 65536, one more for each factor of 16.
// ---------------------------------------------------------------------
constexpr int kRun = 4096;
constexpr int kRankWaves = 16, kRankThreads = 64 * kRankWaves;
constexpr int kMergeRuns = 16;

// How many keys of run[j0, j1) come before token i, whose key is `key`;
// kTies: 1 when all of them stand before token i, -1 after, 0 mixed.
template <int kTies>
__device__ __forceinline__ int32_t count_before(const int32_t* run, int j0, int j1, int i, int32_t key) {
    typedef int32_t i32x4 __attribute__((ext_vector_type(4)));
    int32_t before = 0;
#pragma unroll 2
    for (int j = j0; j < j1; j += 16) {
        i32x4 k[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) k[q] = *reinterpret_cast<const i32x4*>(&run[j + 4 * q]);
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int l = 0; l < 4; ++l) {
                if (kTies > 0) before += k[q][l] <= key;
                else if (kTies < 0) before += k[q][l] < key;
                else before += k[q][l] < key || (k[q][l] == key && j + 4 * q + l < i);
            }
    }
    return before;
}

// A workgroup ranks kGroup tokens of a run: its waves, and the 64 / kGroup
// lanes of each that hold the same token, share out the run's ids.
template <int kGroup>
__global__ __launch_bounds__(kRankThreads) void rank_runs_kernel(const void* ids, int ids64, int64_t n, int64_t vocab,
                                                                 int32_t* keys, int32_t* pos) {
    constexpr int kLanes = 64 / kGroup;
    __shared__ alignas(16) int32_t run[kRun];
    __shared__ int32_t count[kRankWaves][64];
    const int64_t base = (int64_t)(blockIdx.x / (kRun / kGroup)) * kRun;
    const int group = (int)(blockIdx.x % (kRun / kGroup)) * kGroup;
    const int len = (int)(n - base < kRun ? n - base : kRun);
    if (group >= len) return;
    constexpr int kUnit = kRankWaves * kLanes * 16;
    const int share = (len + kUnit - 1) / kUnit * kLanes * 16;  // ids per wave
#pragma unroll
    for (int u = 0; u < kRun / kRankThreads; ++u) {
        const int j = u * kRankThreads + threadIdx.x;
        int32_t k = 0x7FFFFFFF;  // past the end: after every key
        if (j < len) {
            const int64_t r = row_of(ids, ids64, base + j, vocab);
            k = r < 0 ? (int32_t)vocab : (int32_t)r;
        }
        run[j] = k;
    }
    __syncthreads();
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int i = group + lane % kGroup;
    const int32_t key = i < len ? run[i] : 0;
    const int w0 = w * share, w1 = w0 + share;
    const int j0 = w0 + lane / kGroup * (share / kLanes), j1 = j0 + share / kLanes;
    int32_t before;
    if (w1 <= group) before = count_before<1>(run, j0, j1, i, key);
    else if (w0 >= group + kGroup) before = count_before<-1>(run, j0, j1, i, key);
    else before = count_before<0>(run, j0, j1, i, key);
    count[w][lane] = before;
    __syncthreads();
    if (w != 0 || lane >= kGroup || i >= len) return;
    before = 0;
#pragma unroll
    for (int x = 0; x < kRankWaves; ++x)
#pragma unroll
        for (int y = 0; y < kLanes; ++y) before += count[x][y * kGroup + lane];
    keys[base + before] = key;
    pos[base + before] = (int32_t)(base + i);
}

// First index in [lo, n) whose key is >= v (or > v).
template <bool kUpper>
__device__ __forceinline__ int64_t bound_of(const int32_t* keys, int64_t lo, int64_t n, int64_t v) {
    int64_t left = n - lo;
    while (left > 0) {
        const int64_t half = left >> 1;
        const int64_t k = keys[lo + half];
        const bool before = kUpper ? k <= v : k < v;
        lo = before ? lo + half + 1 : lo;
        left = before ? left - half - 1 : half;
    }
    return lo;
}

// The zero rows of ids that do not occur, `rows` of them a workgroup: looked up
// together in the sorted runs of `len` tokens, then written.
constexpr int kFillRows = 64;  // most a workgroup takes
struct FillArgs {
    void* dtable;
    int64_t vocab, dim, ld;
    int32_t rows, wgs;
};

template <class O>
__device__ __forceinline__ void fill_absent(const FillArgs& f, int64_t wg, const int32_t* keys, int64_t n, int64_t len) {
    __shared__ int32_t present[kFillRows];
    const int64_t v0 = wg * f.rows;
    if (threadIdx.x < kFillRows) present[threadIdx.x] = v0 + threadIdx.x >= f.vocab || (int)threadIdx.x >= f.rows;
    __syncthreads();
    // a row to each of 64 lanes, the runs shared out over the four waves
    const int64_t v = v0 + (threadIdx.x & 63);
    for (int64_t r0 = (threadIdx.x >> 6) * len; r0 < n; r0 += (kThreads / 64) * len) {
        const int64_t end = r0 + len < n ? r0 + len : n;
        const int64_t at = bound_of<false>(keys, r0, end, v);
        if (at < end && keys[at] == v) present[threadIdx.x & 63] = 1;
    }
    __syncthreads();
    for (int r = 0; r < f.rows;) {
        if (present[r]) {
            ++r;
            continue;
        }
        // absent rows that lie back to back are one range
        int end = r + 1;
        if (f.ld == f.dim)
            while (end < f.rows && !present[end]) ++end;
        const int64_t n_elems = (end - r) * f.dim;
        // whole 16-byte blocks between the range's ends, whatever its alignment
        typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
        constexpr int kPer = 16 / sizeof(O);
        O* row = static_cast<O*>(f.dtable) + (v0 + r) * f.ld;
        const int64_t skew = (16 - (reinterpret_cast<uintptr_t>(row) & 15u)) % 16 / sizeof(O);
        const int64_t head = skew < n_elems ? skew : n_elems;
        const int64_t blocks = (n_elems - head) / kPer, tail = head + blocks * kPer;
        u32x4* block = reinterpret_cast<u32x4*>(row + head);
#pragma unroll 4
        for (int64_t c = threadIdx.x; c < blocks; c += kThreads) block[c] = u32x4{0u, 0u, 0u, 0u};
        if ((int64_t)threadIdx.x < head) row[threadIdx.x] = (O)0.0f;
        else if (tail + threadIdx.x - head < n_elems) row[tail + threadIdx.x - head] = (O)0.0f;
        r = end;
    }
}

// Merge of groups of kRuns sorted runs of `len` tokens each.  The searches of
// a token advance together, so their loads overlap.  Workgroups past the tokens
// fill the absent rows meanwhile: the merge waits for its searches, the fill
// for memory.
template <int kRuns, class O>
__global__ __launch_bounds__(kThreads) void merge_runs_kernel(const int32_t* __restrict__ keys, const int32_t* __restrict__ pos,
                                                              int32_t* __restrict__ out_keys, int32_t* __restrict__ out_pos,
                                                              int64_t n, int64_t len, int steps, FillArgs fill) {
    const int64_t merges = (n + kThreads - 1) / kThreads;
    if (blockIdx.x >= merges) {
        fill_absent<O>(fill, blockIdx.x - merges, keys, n, len);
        return;
    }
    const int64_t t = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (t >= n) return;
    const int64_t group = t / (len * kRuns) * (len * kRuns);
    const int mine = (int)((t - group) / len);
    const int32_t key = keys[t];
    // of run r: how many come before this token; searched in [lo, lo + left)
    int32_t lo[kRuns], left[kRuns];
#pragma unroll
    for (int r = 0; r < kRuns; ++r) {
        const int64_t have = n - (group + r * len);
        lo[r] = 0;
        left[r] = (int32_t)(r == mine || have <= 0 ? 0 : have < len ? have : len);
    }
    for (int s = 0; s < steps; ++s) {
#pragma unroll
        for (int r = 0; r < kRuns; ++r) {
            // an ended search reads its last place again and keeps its answer
            const int32_t half = left[r] >> 1;
            const int64_t at = group + r * len + lo[r] + half;
            const int32_t k = keys[at < n ? at : n - 1];
            const bool open = left[r] > 0, before = k < key || (k == key && r < mine);
            lo[r] = open && before ? lo[r] + half + 1 : lo[r];
            left[r] = !open ? 0 : before ? left[r] - half - 1 : half;
        }
    }
    int64_t at = t - mine * len;
#pragma unroll
    for (int r = 0; r < kRuns; ++r) at += lo[r];
    out_keys[at] = key;
    out_pos[at] = pos[t];
}

template <int kRuns, class O>
void merge_runs(const int32_t* keys, const int32_t* pos, int32_t* out_keys, int32_t* out_pos, int64_t n, int64_t len, int steps,
                const FillArgs& fill, void* stream) {
    hipLaunchKernelGGL((merge_runs_kernel<kRuns, O>), dim3((uint32_t)((n + kThreads - 1) / kThreads + fill.wgs)), dim3(kThreads),
                       0, (hipStream_t)stream, keys, pos, out_keys, out_pos, n, len, steps, fill);
}

// ---------------------------------------------------------------------
// Sums by segment.  A workgroup takes `per` consecutive sorted tokens and
// 256 * kVec columns, adds rows in ascending position, and writes a row of
// the gradient whose tokens all lie in its range; a row that continues over
// a border goes to two float partials per range (the part that began before
// it, the part that goes on after it), which join_kernel adds in order.
// The order of every sum is fixed by the sorted tokens and `per`, so two
// runs give the same bits.  Workgroups past the ranges write the zero rows
// of tokens that do not occur (kFillRows rows each), so the whole gradient
// is written once.
// ---------------------------------------------------------------------
constexpr int kMaxPer = 32;

struct SegmentArgs {
    const int32_t* keys;
    const int32_t* pos;
    float* head;  // [ranges][dim4]: the part of a range that continues a row begun before it
    float* tail;  // [ranges][dim4]: the part that goes on in the next range
    int64_t n, vocab, dim, dim4, dout_ld, dtable_ld, ranges;
    int32_t slabs, per;
    float scale;
    int32_t accumulate;
};

template <class O, int kVec>
__device__ __forceinline__ void write_row(O* dst, const float (&sum)[kVec], const SegmentArgs& a) {
    float y[kVec];
#pragma unroll
    for (int l = 0; l < kVec; ++l) y[l] = sum[l] * a.scale;
    if (a.accumulate) {
        float old[kVec];
        if constexpr (kVec >= 4 && sizeof(O) == 4) {
            typedef float f4 __attribute__((ext_vector_type(4)));
#pragma unroll
            for (int q = 0; q < kVec / 4; ++q) {
                const f4 o = *(reinterpret_cast<const f4*>(dst) + q);
#pragma unroll
                for (int l = 0; l < 4; ++l) old[4 * q + l] = o[l];
            }
        } else {
#pragma unroll
            for (int l = 0; l < kVec; ++l) old[l] = Elem<O>::get(dst[l]);
        }
#pragma unroll
        for (int l = 0; l < kVec; ++l) y[l] = old[l] + y[l];
    }
    store_piece<O, kVec>(dst, y);
}

template <int kVec>
__device__ __forceinline__ void store_partial(float* p, const float (&x)[kVec]) {
#pragma unroll
    for (int l = 0; l < kVec; ++l) p[l] = x[l];
}

template <class I, class O, int kVec>
__global__ __launch_bounds__(kThreads) void segment_kernel(const void* dout_p, void* dtable_p, SegmentArgs a, FillArgs fill) {
    const I* dout = static_cast<const I*>(dout_p);
    O* dtable = static_cast<O*>(dtable_p);
    __shared__ int32_t key[kMaxPer + 2], row[kMaxPer];
    const int64_t sums = a.ranges * a.slabs;
    if (blockIdx.x >= sums) {
        fill_absent<O>(fill, blockIdx.x - sums, a.keys, a.n, a.n > 0 ? a.n : 1);
        return;
    }
    const int64_t range = blockIdx.x / a.slabs;
    const int64_t c = ((int64_t)(blockIdx.x % a.slabs) * kThreads + threadIdx.x) * kVec;
    const int64_t e0 = range * a.per;
    const int count = (int)(a.n - e0 < a.per ? a.n - e0 : a.per);
    if (threadIdx.x < count + 2) {  // the neighbours' keys too; -1 outside
        const int64_t e = e0 + (int64_t)threadIdx.x - 1;
        key[threadIdx.x] = e >= 0 && e < a.n ? a.keys[e] : -1;
    }
    if (threadIdx.x < count) row[threadIdx.x] = a.pos[e0 + threadIdx.x];
    __syncthreads();
    if (c >= a.dim) return;
    float acc[kVec];
#pragma unroll
    for (int l = 0; l < kVec; ++l) acc[l] = 0.0f;
    bool began = key[1] != key[0];
    for (int b = 0; b < count; b += 8) {
        float x[8][kVec];
#pragma unroll
        for (int u = 0; u < 8; ++u)  // past the end the last row again: loaded, not used
            Piece<I, kVec>::load(dout + (int64_t)row[min(b + u, count - 1)] * a.dout_ld + c, x[u]);
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            if (b + u >= count) break;
#pragma unroll
            for (int l = 0; l < kVec; ++l) acc[l] += x[u][l];
            const int32_t k = key[b + u + 1];
            if (b + u + 1 < count && key[b + u + 2] == k) continue;
            const bool ends = key[b + u + 2] != k;
            if (k < a.vocab) {
                if (began && ends) write_row<O, kVec>(dtable + (int64_t)k * a.dtable_ld + c, acc, a);
                else store_partial<kVec>((began ? a.tail : a.head) + range * a.dim4 + c, acc);
            }
            began = true;
#pragma unroll
            for (int l = 0; l < kVec; ++l) acc[l] = 0.0f;
        }
    }
}

// Rows that cross ranges: the range a row begins in adds its tail and the
// heads of the ranges the row goes on through.
template <class O, int kVec>
__global__ __launch_bounds__(kThreads) void join_kernel(void* dtable_p, SegmentArgs a) {
    O* dtable = static_cast<O*>(dtable_p);
    const int64_t range = blockIdx.x / a.slabs;
    const int64_t c = ((int64_t)(blockIdx.x % a.slabs) * kThreads + threadIdx.x) * kVec;
    const int64_t e0 = range * a.per, e1 = e0 + a.per;
    if (e1 >= a.n) return;
    const int32_t k = a.keys[e1 - 1];
    if (k >= a.vocab || a.keys[e1] != k) return;                              // does not go on
    if (a.keys[e0] == k && e0 > 0 && a.keys[e0 - 1] == k) return;            // began earlier
    if (c >= a.dim) return;
    const int64_t last = (bound_of<true>(a.keys, e1, a.n, k) - 1) / a.per;
    float acc[kVec];
#pragma unroll
    for (int l = 0; l < kVec; ++l) acc[l] = a.tail[range * a.dim4 + c + l];
#pragma unroll 8
    for (int64_t r = range + 1; r <= last; ++r) {
#pragma unroll
        for (int l = 0; l < kVec; ++l) acc[l] += a.head[r * a.dim4 + c + l];
    }
    write_row<O, kVec>(dtable + (int64_t)k * a.dtable_ld + c, acc, a);
}

// Tokens per range: long ranges write fewer partials, short ones give a
// small batch more workgroups.
constexpr int64_t kLongTokens = 16384;
int32_t range_tokens(int64_t n) { return n >= kLongTokens ? 32 : 8; }

int64_t align_up(int64_t x, int64_t a) { return (x + a - 1) / a * a; }

bool aligned_rows(const void* p, int64_t ld, int64_t dim, int size, int vec) {
    const int64_t bytes = std::min<int64_t>(16, (int64_t)vec * size);
    return dim % vec == 0 && (reinterpret_cast<uintptr_t>(p) % bytes) == 0 && (ld * size) % bytes == 0;
}

template <class T, class O, int kVec>
int embed_vec(const EmbedArgs& a, void* stream) {
    const int64_t pieces = a.dim / kVec;
    const int32_t per_wg = pieces >= kThreads ? 1 : (int32_t)(kThreads / pieces);
    const int64_t wgs = std::min<int64_t>((a.n + per_wg - 1) / per_wg, 1 << 22);
    hipLaunchKernelGGL((embed_kernel<T, O, kVec>), dim3((uint32_t)wgs), dim3(kThreads), 0, (hipStream_t)stream, a,
                       (int32_t)pieces, per_wg);
    return hipGetLastError();
}

template <class T, class O>
int embed_types(const EmbedArgs& a, void* stream) {
    const auto fits = [&](int vec) {
        return aligned_rows(a.table, a.table_ld, a.dim, sizeof(T), vec) && aligned_rows(a.out, a.out_ld, a.dim, sizeof(O), vec);
    };
    if constexpr (sizeof(T) == 1)
        if (fits(16)) return embed_vec<T, O, 16>(a, stream);
    if (fits(8)) return embed_vec<T, O, 8>(a, stream);
    if (fits(4)) return embed_vec<T, O, 4>(a, stream);
    return embed_vec<T, O, 1>(a, stream);
}

template <class T>
int embed_out(const EmbedArgs& a, void* stream) {
    switch (a.out_type) {
        case kF32: return embed_types<T, float>(a, stream);
        case kBF16: return embed_types<T, bf16_t>(a, stream);
        default: return embed_types<T, f16_t>(a, stream);
    }
}

struct GradWork {
    int32_t *keys[2], *pos[2];
    float *head, *tail;
    int64_t bytes;
};

GradWork grad_work(void* work, int64_t n, int64_t dim) {
    GradWork g;
    char* p = static_cast<char*>(work);
    int64_t at = 0;
    const auto take = [&](int64_t bytes) {
        char* q = p + at;
        at += align_up(bytes, 256);
        return q;
    };
    for (int k = 0; k < 2; ++k) {
        g.keys[k] = reinterpret_cast<int32_t*>(take(4 * n));
        g.pos[k] = reinterpret_cast<int32_t*>(take(4 * n));
    }
    const int64_t ranges = (n + range_tokens(n) - 1) / range_tokens(n);
    g.head = reinterpret_cast<float*>(take(ranges * align_up(dim, 4) * 4));
    g.tail = reinterpret_cast<float*>(take(ranges * align_up(dim, 4) * 4));
    g.bytes = at;
    return g;
}

template <class I, class O, int kVec>
int segments(const EmbedGradArgs& a, const GradWork& g, void* stream) {
    FillArgs fill{a.dtable, a.vocab, a.dim, a.dtable_ld, 0, 0};
    if (!a.accumulate) {
        // 128 KiB a workgroup (131072 x 4096: 492 us; 64 KiB 503, 512 KiB 499)
        fill.rows = (int32_t)std::min<int64_t>(kFillRows, std::max<int64_t>(1, 128 * 1024 / (a.dim * (int64_t)sizeof(O))));
        fill.wgs = (int32_t)((a.vocab + fill.rows - 1) / fill.rows);
    }
    int at = 0;
    if (a.n > 0) {
        const int64_t runs = (a.n + kRun - 1) / kRun;
        // few tokens: 16 a workgroup, so that they reach the device's width
        const bool few = a.n <= 8192;
        const auto rank = few ? rank_runs_kernel<16> : rank_runs_kernel<64>;
        hipLaunchKernelGGL(rank, dim3((uint32_t)(runs * (kRun / (few ? 16 : 64)))), dim3(kRankThreads), 0, (hipStream_t)stream, a.ids,
                           a.ids64, a.n, a.vocab, g.keys[0], g.pos[0]);
        const hipError_t err = hipGetLastError();
        if (err != hipSuccess) return err;
    }
    for (int64_t len = kRun; len < a.n; len *= kMergeRuns) {
        int steps = 1;  // a search over m entries takes at most bits(m) steps
        while ((int64_t(1) << steps) <= len) ++steps;
        const auto merge = a.n <= 2 * len   ? merge_runs<2, O>
                           : a.n <= 4 * len ? merge_runs<4, O>
                           : a.n <= 8 * len ? merge_runs<8, O>
                                            : merge_runs<kMergeRuns, O>;
        const FillArgs none{};
        const bool last = len * kMergeRuns >= a.n;
        merge(g.keys[at], g.pos[at], g.keys[at ^ 1], g.pos[at ^ 1], a.n, len, steps, last ? fill : none, stream);
        const hipError_t err = hipGetLastError();
        if (err != hipSuccess) return err;
        if (last) fill = none;
        at ^= 1;
    }
    SegmentArgs s{};
    s.keys = g.keys[at];
    s.pos = g.pos[at];
    s.head = g.head;
    s.tail = g.tail;
    s.n = a.n;
    s.vocab = a.vocab;
    s.dim = a.dim;
    s.dim4 = align_up(a.dim, 4);
    s.dout_ld = a.dout_ld;
    s.dtable_ld = a.dtable_ld;
    s.per = range_tokens(a.n);
    s.ranges = (a.n + s.per - 1) / s.per;
    s.slabs = (int32_t)((a.dim + kThreads * kVec - 1) / (kThreads * kVec));
    s.scale = a.scale;
    s.accumulate = a.accumulate;
    const int64_t sums = s.ranges * s.slabs;
    if (sums + fill.wgs == 0) return hipSuccess;
    hipLaunchKernelGGL((segment_kernel<I, O, kVec>), dim3((uint32_t)(sums + fill.wgs)), dim3(kThreads), 0, (hipStream_t)stream,
                       a.dout, a.dtable, s, fill);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess || s.ranges <= 1) return err;
    hipLaunchKernelGGL((join_kernel<O, kVec>), dim3((uint32_t)sums), dim3(kThreads), 0, (hipStream_t)stream, a.dtable, s);
    return hipGetLastError();
}

template <class I, class O>
int segments_vec(const EmbedGradArgs& a, const GradWork& g, void* stream) {
    // (8 elements a thread of 16-bit rows measured 2-3% slower)
    if (aligned_rows(a.dout, a.dout_ld, a.dim, sizeof(I), 4) && aligned_rows(a.dtable, a.dtable_ld, a.dim, sizeof(O), 4))
        return segments<I, O, 4>(a, g, stream);
    return segments<I, O, 1>(a, g, stream);
}

template <class I>
int segments_out(const EmbedGradArgs& a, const GradWork& g, void* stream) {
    switch (a.dtable_type) {
        case kF32: return segments_vec<I, float>(a, g, stream);
        case kBF16: return segments_vec<I, bf16_t>(a, g, stream);
        default: return segments_vec<I, f16_t>(a, g, stream);
    }
}

}  // namespace

int launch_embed(const EmbedArgs& a, void* stream) {
    if (a.n == 0 || a.dim == 0) return hipSuccess;
    switch (a.table_type) {
        case kF32: return embed_out<float>(a, stream);
        case kBF16: return embed_out<bf16_t>(a, stream);
        case kF16: return embed_out<f16_t>(a, stream);
        default: return embed_out<uint8_t>(a, stream);
    }
}

// Enough for every count of tokens up to n (just below kLongTokens, the
// shorter ranges have more partials than somewhat above it).
int64_t embed_grad_work_bytes(int64_t n, int64_t dim) {
    return std::max(grad_work(nullptr, n, dim).bytes, grad_work(nullptr, std::min(n, kLongTokens - 1), dim).bytes);
}

int launch_embed_grad(const EmbedGradArgs& a, void* work, void* stream) {
    const GradWork g = grad_work(work, a.n, a.dim);
    switch (a.dout_type) {
        case kF32: return segments_out<float>(a, g, stream);
        case kBF16: return segments_out<bf16_t>(a, g, stream);
        default: return segments_out<f16_t>(a, g, stream);
    }
}

}  // namespace bfz
