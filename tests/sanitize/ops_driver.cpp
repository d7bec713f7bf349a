// CPU build of the operators' C ABI (ops_abi.cpp, with plan.cpp and abi.cpp)
// for AddressSanitizer / UndefinedBehaviorSanitizer runs -- no GPU involved.
// Launches are recorded: the tensor lists of one call must cover every
// element of every tensor exactly once, in order, with one first and one last
// launch; plan launches must cover the shard's slots; refused calls must
// launch nothing.  Exit status 0 when every check passes.
#include <hip/hip_runtime.h>

#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <vector>

#include "bfz.h"
#include "ops_internal.h"

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
std::vector<bfz::TensorList> g_lists;
std::vector<bfz::NormOut> g_outs;
int64_t g_slots = 0;
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
int launch_step(float*, const float*, float*, float*, uint8_t*, float*, int64_t, const StepScalars& s, void*) {
    CHECK(s.grad_scale != nullptr, "the clipped step passes its scale on");
    return done();
}
int launch_fold_step(const TileEntry*, int64_t, const PackArgs&, float*, float*, float*, uint8_t*, float*, const StepScalars& s, void*) {
    CHECK(s.grad_scale != nullptr, "the clipped step passes its scale on");
    return done();
}
int launch_fold_step_unfold(const TileEntry*, int64_t, const PackArgs&, const UnpackArgs&, float*, float*, float*, uint8_t*, float*,
                            const StepScalars& s, void*) {
    CHECK(s.grad_scale != nullptr, "the clipped step passes its scale on");
    return done();
}
int launch_fold_step_unfold_t(const TileEntry*, int64_t, const PackArgs&, const UnpackArgs&, const TransposeArgs&, float*, float*, float*,
                              uint8_t*, float*, const StepScalars& s, void*) {
    CHECK(s.grad_scale != nullptr, "the clipped step passes its scale on");
    return done();
}
int launch_transpose_pow2(const TileEntry*, const int32_t*, int64_t, const uint8_t*, const float*, const TransposeArgs&, void*) { return done(); }
int launch_encode(const float*, uint8_t*, int64_t, void*) { return done(); }
const char* hip_error_string(int) { return "host stand-in error"; }
int launch_list_sumsq(const TensorList& l, const NormOut& o, void*, void*) {
    g_lists.push_back(l);
    g_outs.push_back(o);
    return done();
}
int launch_shard_sumsq(const TileEntry*, int64_t n, const PackArgs&, const NormOut& o, void*, void*) {
    g_slots += n;
    g_outs.push_back(o);
    return done();
}
int launch_clip_coef(const double*, double, float*, float*, void*) { return done(); }
int launch_clip(const TensorList& l, const float*, void*) {
    g_lists.push_back(l);
    return done();
}
int launch_embed(const EmbedArgs&, void*) { return done(); }
int64_t embed_grad_work_bytes(int64_t n, int64_t dim) { return 16 * n + dim; }
int launch_embed_grad(const EmbedGradArgs&, void*, void*) { return done(); }
int64_t vocab_loss_work_bytes(int64_t n, int64_t, int64_t, int, int) { return 256 + n; }
int launch_vocab_loss(const VocabLossArgs&, void*, void*) { return done(); }
int launch_vocab_loss_grad(const VocabLossArgs&, void*, void*) { return done(); }
}  // namespace bfz

namespace {
template <class T>
T* at(uintptr_t a) { return reinterpret_cast<T*>(a); }

void reset() {
    g_lists.clear();
    g_outs.clear();
    g_slots = 0;
    g_launches = 0;
}

// The launched lists walk the tensors' elements exactly once, in order.
void check_lists(const std::vector<bfz_tensor>& in, const std::vector<bfz_tensor>* out) {
    size_t k = 0;
    int64_t done_elems = 0;
    for (const bfz::TensorList& l : g_lists) {
        CHECK(l.count >= 0 && l.count <= bfz::kListTensors, "%d tensors in a launch", l.count);
        uint64_t chunks = 0;
        for (int i = 0; i < l.count; ++i) {
            while (k < in.size() && done_elems == in[k].n) ++k, done_elems = 0;
            CHECK(k < in.size(), "more pieces than tensors");
            if (k >= in.size()) return;
            const int size = bfz::dtype_size(in[k].dtype);
            CHECK(l.chunk0[i] == chunks, "chunk %u after %llu", l.chunk0[i], (unsigned long long)chunks);
            CHECK(l.in[i] == static_cast<char*>(in[k].data) + done_elems * size && l.in_type[i] == in[k].dtype, "tensor %zu", k);
            if (out)
                CHECK(l.out[i] == static_cast<char*>((*out)[k].data) + done_elems * bfz::dtype_size((*out)[k].dtype) &&
                          l.out_type[i] == (*out)[k].dtype, "output %zu", k);
            CHECK(l.n[i] > 0 && done_elems + l.n[i] <= in[k].n, "tensor %zu: %lld elements", k, (long long)l.n[i]);
            chunks += (uint64_t)((l.n[i] + l.chunk_elems - 1) / l.chunk_elems);
            done_elems += l.n[i];
        }
        CHECK(l.chunks == chunks && chunks <= (uint64_t(1) << 31), "%u chunks, %llu counted", l.chunks, (unsigned long long)chunks);
    }
    while (k < in.size() && done_elems == in[k].n) ++k, done_elems = 0;
    CHECK(k == in.size() && done_elems == 0, "tensors left over from %zu of %zu", k, in.size());
    for (size_t i = 0; i < g_outs.size(); ++i)
        CHECK(g_outs[i].first == (i == 0) && g_outs[i].last == (i + 1 == g_outs.size()), "first and last of launch %zu", i);
}

void norm_of(const std::vector<int64_t>& sizes) {
    std::vector<bfz_tensor> in, out;
    uintptr_t a = uintptr_t(1) << 40;
    for (size_t k = 0; k < sizes.size(); ++k) {
        in.push_back({at<void>(a), sizes[k], (int32_t)(k % 3), 0});
        out.push_back({at<void>(a + (uintptr_t(1) << 56)), sizes[k], (int32_t)((k + 1) % 3), 0});
        a += (uintptr_t)sizes[k] * 4 + 64;
    }
    // exactly as many as are named, on the heap
    bfz_tensor* heap = static_cast<bfz_tensor*>(std::malloc(in.size() * sizeof(bfz_tensor) + !in.size()));
    if (!in.empty()) std::memcpy(heap, in.data(), in.size() * sizeof(bfz_tensor));
    reset();
    CHECK(bfz_grad_norm(in.empty() ? nullptr : heap, (int32_t)in.size(), 1.0, nullptr, at<float>(0x1000), at<float>(0x1004), at<void>(0x2000), nullptr) == BFZ_OK, "%s", bfz_last_error());
    CHECK(!g_outs.empty(), "a norm always writes its results");
    check_lists(in, nullptr);
    reset();
    CHECK(bfz_clip_grads(in.empty() ? nullptr : heap, out.data(), (int32_t)in.size(), at<float>(0x1000), nullptr) == BFZ_OK, "%s", bfz_last_error());
    check_lists(in, &out);
    std::free(heap);
}
}  // namespace

int main() {
    norm_of({});
    norm_of({0});
    norm_of({1});
    norm_of({4096, 4097, 0, 1, 0});
    for (int n : {95, 96, 97, 192, 193, 400}) {
        std::vector<int64_t> sizes;
        for (int k = 0; k < n; ++k) sizes.push_back((k * 7919) % 20000);
        norm_of(sizes);
    }
    // more chunks than a launch counts: 9 * 2^28
    norm_of(std::vector<int64_t>(9, int64_t(1) << 40));
    norm_of({int64_t(1) << 40, 3, int64_t(1) << 40});

    // a launch that fails is reported, and nothing follows it
    std::vector<bfz_tensor> many(200, bfz_tensor{at<void>(0x1000), 5, 0, 0});
    reset();
    g_fail = 1;
    CHECK(bfz_grad_norm(many.data(), 200, 1.0, nullptr, nullptr, nullptr, at<void>(0x2000), nullptr) == BFZ_EHIP && g_launches == 1, "failed launch");

    // plan launches cover the shard, segments of more weights than a launch takes too
    std::vector<int64_t> dims;
    std::vector<const float*> grads;
    for (int k = 0; k < 150; ++k) {
        for (int64_t d : {int64_t(1), int64_t(100 + k), int64_t(300)}) dims.push_back(d);
        grads.push_back(at<const float>(0x100000 * (k + 1)));
    }
    bfz_plan* plan = nullptr;
    CHECK(bfz_plan_create(dims.data(), 150, 1, 0, &plan) == BFZ_OK, "%s", bfz_last_error());
    reset();
    CHECK(bfz_shard_grad_norm(plan, grads.data(), 1.0, nullptr, at<float>(0x1000), nullptr, at<void>(0x2000), nullptr) == BFZ_OK, "%s", bfz_last_error());
    CHECK(g_slots == bfz_plan_shard_tiles(plan) && g_launches >= 3, "%lld slots in %d launches", (long long)g_slots, g_launches);
    for (size_t i = 0; i < g_outs.size(); ++i)
        CHECK(g_outs[i].first == (i == 0) && g_outs[i].last == (i + 1 == g_outs.size()), "first and last of launch %zu", i);
    // clipped steps
    bfz_adamw* hp = static_cast<bfz_adamw*>(std::malloc(sizeof(bfz_adamw)));
    *hp = bfz_adamw{1e-3, 0.9, 0.95, 1e-8, 0.1, 1};
    bfz_step_options pow2{1, 0, 0};
    std::vector<uint8_t*> bytes(150, at<uint8_t>(0x10000000));
    std::vector<float*> floats(150, at<float>(0x20000000));
    float *a = at<float>(0x1000), *b = at<float>(0x2000), *c = at<float>(0x3000), *scale = at<float>(0x4000), *coef = at<float>(0x5004);
    uint8_t* codes = at<uint8_t>(0x6000);
    CHECK(bfz_adamw_fp8_step_clip(a, b, b, c, codes, scale, 3, hp, nullptr, coef, nullptr) == BFZ_OK, "%s", bfz_last_error());
    CHECK(bfz_fold_adamw_fp8_step_clip(plan, grads.data(), a, b, c, codes, scale, hp, nullptr, coef, nullptr) == BFZ_OK, "%s", bfz_last_error());
    CHECK(bfz_fold_adamw_fp8_step_unpack_clip(plan, grads.data(), a, b, c, codes, scale, bytes.data(), floats.data(), hp, nullptr, coef, nullptr) == BFZ_OK, "%s", bfz_last_error());
    CHECK(bfz_fold_adamw_fp8_step_unpack_t_clip(plan, grads.data(), a, b, c, codes, scale, bytes.data(), floats.data(), bytes.data(), floats.data(), hp, &pow2, coef, nullptr) == BFZ_OK, "%s", bfz_last_error());
    reset();
    CHECK(bfz_fold_adamw_fp8_step_clip(plan, grads.data(), a, b, c, codes, scale, hp, nullptr, nullptr, nullptr) == BFZ_EINVAL && g_launches == 0, "null scale");
    std::free(hp);
    bfz_plan_destroy(plan);

    // refused calls launch nothing
    reset();
    CHECK(bfz_embed(at<void>(8), 1, 4, a, 0, nullptr, 10, 8, 7, 1.0f, b, 0, 8, nullptr) == BFZ_EINVAL, "overlapping rows");
    CHECK(bfz_embed_grad(at<void>(8), 1, 4, a, 0, 8, 10, 8, 1.0f, 0, b, 0, 8, nullptr, nullptr) == BFZ_EINVAL, "no workspace");
    CHECK(bfz_vocab_loss(a, 8, 4, b, 3, 8, nullptr, 10, 8, at<void>(8), 1, a, b, at<void>(0x100), nullptr) == BFZ_EINVAL, "codes without a grid");
    CHECK(g_launches == 0, "%d launches of refused calls", g_launches);
    // empty ones pass
    CHECK(bfz_embed(nullptr, 1, 0, a, 0, nullptr, 10, 8, 8, 1.0f, nullptr, 0, 8, nullptr) == BFZ_OK, "%s", bfz_last_error());
    CHECK(bfz_embed_grad(nullptr, 1, 0, nullptr, 0, 8, 10, 8, 1.0f, 0, b, 0, 8, nullptr, nullptr) == BFZ_OK, "%s", bfz_last_error());
    CHECK(bfz_vocab_loss(nullptr, 8, 0, b, 1, 8, nullptr, 10, 8, nullptr, 1, nullptr, nullptr, at<void>(0x100), nullptr) == BFZ_OK, "%s", bfz_last_error());
    if (g_failures) return 1;
    std::puts("all checks passed");
    return 0;
}
