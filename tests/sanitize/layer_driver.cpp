// CPU build of the C ABI of a layer's operators and of AdamW over many tensors
// (layer_abi.cpp, with plan.cpp and abi.cpp) for AddressSanitizer /
// UndefinedBehaviorSanitizer runs -- no GPU involved.  Launches are recorded: the
// lists of one AdamW call must cover every element of every tensor exactly once,
// in order, states and scales beside their elements; refused calls must launch
// nothing.  Exit status 0 when every check passes.
#include <hip/hip_runtime.h>

#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <vector>

#include "bfz.h"
#include "layer_internal.h"

extern "C" {
hipError_t hipGetDeviceCount(int* n) { return *n = 1, hipSuccess; }
hipError_t hipGetDevice(int* d) { return *d = 0, hipSuccess; }
hipError_t hipSetDevice(int) { return hipSuccess; }
hipError_t hipMalloc(void** p, size_t n) { return (*p = std::malloc(n)) ? hipSuccess : hipErrorOutOfMemory; }
hipError_t hipFree(void* p) { return std::free(p), hipSuccess; }
hipError_t hipMemcpy(void* d, const void* s, size_t n, hipMemcpyKind) { return std::memcpy(d, s, n), hipSuccess; }
const char* hipGetErrorString(hipError_t) { return "host stand-in error"; }
}

static int g_failures = 0;
#define CHECK(cond, ...)                                                 \
    do {                                                                 \
        if (!(cond)) {                                                   \
            std::fprintf(stderr, "CHECK failed at line %d: ", __LINE__); \
            std::fprintf(stderr, __VA_ARGS__);                           \
            std::fprintf(stderr, "\n");                                  \
            ++g_failures;                                                \
        }                                                                \
    } while (0)

namespace {
std::vector<bfz::AdamwList> g_lists;
std::vector<bfz::LinearArgs> g_products;
int g_launches = 0, g_fail = 0;
int done() {
    ++g_launches;
    const int e = g_fail;
    g_fail = 0;
    return e;
}
}  // namespace

namespace bfz {
int launch_pack(const TileEntry*, int64_t, float*, int64_t, const PackArgs&, void*) { return done(); }
int launch_unpack(const TileEntry*, int64_t, const uint8_t*, const float*, const UnpackArgs&, void*) { return done(); }
int launch_step(float*, const float*, float*, float*, uint8_t*, float*, int64_t, const StepScalars&, void*) { return done(); }
int launch_fold_step(const TileEntry*, int64_t, const PackArgs&, float*, float*, float*, uint8_t*, float*, const StepScalars&, void*) { return done(); }
int launch_fold_step_unfold(const TileEntry*, int64_t, const PackArgs&, const UnpackArgs&, float*, float*, float*, uint8_t*, float*,
                            const StepScalars&, void*) {
    return done();
}
int launch_fold_step_unfold_t(const TileEntry*, int64_t, const PackArgs&, const UnpackArgs&, const TransposeArgs&, float*, float*, float*,
                              uint8_t*, float*, const StepScalars&, void*) {
    return done();
}
int launch_transpose_pow2(const TileEntry*, const int32_t*, int64_t, const uint8_t*, const float*, const TransposeArgs&, void*) { return done(); }
int launch_encode(const float*, uint8_t*, int64_t, void*) { return done(); }
const char* hip_error_string(int) { return "host stand-in error"; }
int launch_quantize(const QuantizeArgs&, void*) { return done(); }
int64_t linear_work_bytes(int64_t n, int64_t rows, int64_t cols, int copy, int quantize) { return 256 + n * quantize + rows * cols * copy; }
int launch_linear(const LinearArgs& a, void*, void*) { return g_products.push_back(a), done(); }
int launch_linear_grad_input(const LinearArgs& a, void*, void*) { return g_products.push_back(a), done(); }
int launch_linear_grad_weight(const LinearArgs& a, void*, void*) { return g_products.push_back(a), done(); }
int launch_layer_norm(const LayerNormArgs&, void*) { return done(); }
int64_t layer_norm_work_bytes(int64_t n, int64_t dim) { return n + dim; }
int launch_layer_norm_grad(const LayerNormGradArgs&, void*, void*) { return done(); }
int launch_adamw_list(const AdamwList& l, const StepScalars& s, void*) {
    CHECK(s.b1 == 0.9f && s.has_decay == 1, "the step's scalars");
    g_lists.push_back(l);
    return done();
}
}  // namespace bfz

namespace {
template <class T>
T* at(uintptr_t a) { return reinterpret_cast<T*>(a); }

const bfz_adamw kHp{1e-3, 0.9, 0.95, 1e-8, 0.1, 5};

std::vector<bfz_adamw_tensor> tensors_of(const std::vector<int64_t>& sizes) {
    std::vector<bfz_adamw_tensor> t;
    uintptr_t a = uintptr_t(1) << 40;
    for (size_t k = 0; k < sizes.size(); ++k) {
        const bool codes = k & 1;
        const uintptr_t far = uintptr_t(1) << 50;
        t.push_back({at<void>(a), at<void>(a + far), at<void>(a + 2 * far), at<void>(a + 3 * far), codes ? at<float>(a + 4 * far) : nullptr,
                     codes ? at<float>(a + 5 * far) : nullptr, sizes[k], (int32_t)(k % 3), (int32_t)((k + 1) % 3), codes ? BFZ_E4M3 : BFZ_F32, 0});
        a += (uintptr_t)sizes[k] * 4 + 64;
    }
    return t;
}

void adamw_of(const std::vector<int64_t>& sizes) {
    const std::vector<bfz_adamw_tensor> t = tensors_of(sizes);
    bfz_adamw_tensor* heap = static_cast<bfz_adamw_tensor*>(std::malloc(t.size() * sizeof(bfz_adamw_tensor) + !t.size()));
    if (!t.empty()) std::memcpy(heap, t.data(), t.size() * sizeof(bfz_adamw_tensor));
    bfz_adamw* hp = static_cast<bfz_adamw*>(std::malloc(sizeof(bfz_adamw)));  // exactly its six fields
    *hp = kHp;
    g_lists.clear();
    CHECK(bfz_adamw_list(t.empty() ? nullptr : heap, (int32_t)t.size(), hp, nullptr, nullptr) == BFZ_OK, "%s", bfz_last_error());
    std::free(hp);
    std::free(heap);
    size_t k = 0;
    int64_t seen = 0;
    for (const bfz::AdamwList& l : g_lists) {
        CHECK(l.count > 0 && l.count <= bfz::kAdamwTensors, "%d tensors in a launch", l.count);
        uint64_t chunks = 0;
        for (int i = 0; i < l.count; ++i) {
            while (k < t.size() && seen == t[k].n) ++k, seen = 0;
            CHECK(k < t.size(), "more pieces than tensors");
            if (k >= t.size()) return;
            const bfz_adamw_tensor& x = t[k];
            const int se = bfz::dtype_size(x.state_dtype);
            CHECK(l.chunk0[i] == chunks, "chunk %u after %llu", l.chunk0[i], (unsigned long long)chunks);
            CHECK(seen % bfz::kStateBlock == 0, "a piece starts on a state block");
            CHECK(l.param[i] == static_cast<char*>(x.param) + seen * bfz::dtype_size(x.param_dtype) && l.param_type[i] == x.param_dtype, "param %zu", k);
            CHECK(l.grad[i] == static_cast<const char*>(x.grad) + seen * bfz::dtype_size(x.grad_dtype) && l.grad_type[i] == x.grad_dtype, "grad %zu", k);
            CHECK(l.m[i] == static_cast<char*>(x.m) + seen * se && l.v[i] == static_cast<char*>(x.v) + seen * se && l.state_type[i] == x.state_dtype, "states %zu", k);
            CHECK(l.m_scale[i] == (x.m_scale ? x.m_scale + seen / bfz::kStateBlock : nullptr), "m_scale %zu", k);
            CHECK(l.v_scale[i] == (x.v_scale ? x.v_scale + seen / bfz::kStateBlock : nullptr), "v_scale %zu", k);
            CHECK(l.n[i] > 0 && seen + l.n[i] <= x.n, "tensor %zu: %lld elements", k, (long long)l.n[i]);
            chunks += (uint64_t)((l.n[i] + bfz::kAdamwChunk - 1) / bfz::kAdamwChunk);
            seen += l.n[i];
        }
        CHECK(l.chunks == chunks && chunks <= (uint64_t(1) << 23), "%u chunks, %llu counted", l.chunks, (unsigned long long)chunks);
    }
    while (k < t.size() && seen == t[k].n) ++k, seen = 0;
    CHECK(k == t.size() && seen == 0, "tensors left over from %zu of %zu", k, t.size());
}
}  // namespace

int main() {
    adamw_of({});
    adamw_of({0});
    adamw_of({1, 255, 256, 257, 0, 4096, 4097});
    for (int n : {55, 56, 57, 112, 113, 300}) {
        std::vector<int64_t> sizes;
        for (int k = 0; k < n; ++k) sizes.push_back((k * 7919) % 20000);
        adamw_of(sizes);
    }
    // more chunks than a launch counts: 2^23 of 4096 elements
    adamw_of({int64_t(1) << 36, (int64_t(1) << 35) + 5, 7, int64_t(1) << 35});

    // a launch that fails is reported, and nothing follows it
    const std::vector<bfz_adamw_tensor> many = tensors_of(std::vector<int64_t>(200, 5));
    g_launches = 0;
    g_fail = 1;
    CHECK(bfz_adamw_list(many.data(), 200, &kHp, nullptr, nullptr) == BFZ_EHIP && g_launches == 1, "%d launches", g_launches);
    // a refused tensor, the last one, launches nothing
    std::vector<bfz_adamw_tensor> bad = many;
    bad[199].m = nullptr;
    g_launches = 0;
    CHECK(bfz_adamw_list(bad.data(), 200, &kHp, nullptr, nullptr) == BFZ_EINVAL && g_launches == 0, "%d launches", g_launches);

    // products: what reaches the launcher, and no launch without tokens
    g_products.clear();
    CHECK(bfz_linear(at<void>(0x1000), BFZ_BF16, 48, nullptr, 0, 0, 5, at<uint8_t>(0x2000), 48, at<float>(0x3000), 300, 33, at<void>(0x4000), BFZ_F32, 300,
                     at<void>(0x10000), nullptr) == BFZ_OK, "%s", bfz_last_error());
    CHECK(g_products.size() == 1 && g_products[0].values == at<void>(0x1000) && g_products[0].values_ld == 48 && g_products[0].n == 5, "values");
    CHECK(bfz_linear(at<void>(0x1000), BFZ_E4M3, 48, at<float>(0x5000), 7, 0, 5, at<uint8_t>(0x2001), 33, at<float>(0x3000), 300, 33, at<void>(0x4000), BFZ_F32,
                     300, at<void>(0x10000), nullptr) == BFZ_OK, "%s", bfz_last_error());
    CHECK(g_products.size() == 2 && g_products[1].values == nullptr && g_products[1].x.scales_ld == 7 && !g_products[1].x.tiles, "codes");
    g_launches = 0;
    CHECK(bfz_linear(nullptr, BFZ_E4M3, 48, nullptr, 1, 1, 0, at<uint8_t>(0x2000), 48, at<float>(0x3000), 300, 33, nullptr, BFZ_F32, 300, at<void>(0x10000),
                     nullptr) == BFZ_OK && g_launches == 0, "no tokens");
    CHECK(bfz_linear_grad_weight(nullptr, 304, nullptr, 3, nullptr, 48, nullptr, 1, 0, 300, 33, at<void>(0x4000), BFZ_F32, 33, 1, at<void>(0x10000), nullptr) ==
              BFZ_OK && g_launches == 0, "nothing to add");
    CHECK(bfz_linear_grad_weight(nullptr, 304, nullptr, 3, nullptr, 48, nullptr, 1, 0, 300, 33, at<void>(0x4000), BFZ_F32, 33, 0, at<void>(0x10000), nullptr) ==
              BFZ_OK && g_launches == 1, "zeros to write");
    if (g_failures) return std::fprintf(stderr, "%d checks failed\n", g_failures), 1;
    std::puts("all checks passed");
    return 0;
}
