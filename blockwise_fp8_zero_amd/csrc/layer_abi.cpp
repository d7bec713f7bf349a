// The C ABI of a layer's operators (quantizer, linear products, layer norm) and
// of AdamW over many tensors: argument checks and launches.
#include <hip/hip_runtime.h>

#include <cmath>

#include "layer_internal.h"

using namespace bfz;

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

int launched(const char* where, int err) {
    return err == hipSuccess ? BFZ_OK : fail(BFZ_EHIP, "%s: %s", where, hip_error_string(err));
}

bool float_type(int t) { return t == kF32 || t == kBF16 || t == kF16; }

int64_t blocks_of(int64_t n) { return (n + kTileDim - 1) / kTileDim; }

constexpr int64_t kMostTokens = int64_t(1) << 24, kMostDim = int64_t(1) << 20, kMostStride = int64_t(1) << 21;

// A matrix of rows ld elements apart.
int check_matrix(const void* p, int dtype, int64_t rows, int64_t dim, int64_t ld, int64_t most, const char* what, const char* where) {
    if (rows > 0 && !p) return fail(BFZ_EINVAL, "%s: %s: null pointer", where, what);
    if (ld < dim || ld > most) return fail(BFZ_EINVAL, "%s: %s: rows %lld elements apart, %lld wide", where, what, (long long)ld, (long long)dim);
    if (!aligned(p, dtype_size(dtype))) return fail(BFZ_EALIGN, "%s: %s must be aligned to its elements", where, what);
    return BFZ_OK;
}

int check_quantize(int64_t n, int64_t dim, int32_t tiles, const char* where) {
    if (!quantize_fits(n, dim, tiles != 0))
        return fail(BFZ_EINVAL, "%s: %lld rows of width %lld are too many for one call", where, (long long)n, (long long)dim);
    return BFZ_OK;
}

// Codes that products read: rows on 16-byte boundaries, read to the next
// multiple of 16 columns.
int check_codes(const uint8_t* p, int64_t rows, int64_t dim, int64_t ld, const char* what, const char* where) {
    const int rc = check_matrix(p, kE4M3, rows, dim, ld, kMostStride, what, where);
    if (rc) return rc;
    if (rows > 0 && (!aligned(p, 16) || ld % 16 != 0))
        return fail(BFZ_EALIGN, "%s: %s: rows must start on 16-byte boundaries", where, what);
    return BFZ_OK;
}

// Scales of [n, dim] codes, in the quantizer's forms.
int check_scales(const float* p, int64_t ld, int32_t tiles, int64_t n, int64_t dim, const char* what, const char* where) {
    if (n > 0 && !p) return fail(BFZ_EINVAL, "%s: %s: null pointer", where, what);
    const int64_t width = tiles ? blocks_of(dim) : n;
    if (ld < width || ld > kMostTokens)
        return fail(BFZ_EINVAL, "%s: %s: rows %lld scales apart, %lld wide", where, what, (long long)ld, (long long)width);
    if (!aligned(p, 4)) return fail(BFZ_EALIGN, "%s: %s must be 4-byte aligned", where, what);
    return BFZ_OK;
}

int check_sizes(int64_t n, int64_t rows, int64_t cols, const char* where) {
    if (n < 0 || rows < 1 || cols < 1 || n > kMostTokens || rows > kMostDim || cols > kMostDim)
        return fail(BFZ_EINVAL, "%s: need 0 <= n <= 2^24, 1 <= rows, cols <= 2^20", where);
    return BFZ_OK;
}

// A launch counts its work-items in 32 bits: under 2^23 tiles of 64 by 64 with
// 512 threads at most.
int check_tiles(int64_t m, int64_t n, const char* where) {
    if (((m + 63) / 64) * ((n + 63) / 64) >= (int64_t(1) << 23))
        return fail(BFZ_EINVAL, "%s: a result of %lld by %lld is too large for one call", where, (long long)n, (long long)m);
    return BFZ_OK;
}

int check_weight(const uint8_t* weight, int64_t weight_ld, const float* grid, int64_t rows, int64_t cols, const char* where) {
    const int rc = check_matrix(weight, kE4M3, rows, cols, weight_ld, kMostStride, "weight", where);
    if (rc) return rc;
    if (!grid) return fail(BFZ_EINVAL, "%s: grid: null pointer", where);
    if (!aligned(grid, 4)) return fail(BFZ_EALIGN, "%s: grid must be 4-byte aligned", where);
    return BFZ_OK;
}

int check_work(const void* work, const char* where) {
    if (!work) return fail(BFZ_EINVAL, "%s: null workspace", where);
    if (!aligned(work, 256)) return fail(BFZ_EALIGN, "%s: the workspace must be 256-byte aligned", where);
    return BFZ_OK;
}

int check_out(const void* out, int32_t dtype, int64_t rows, int64_t dim, int64_t ld, const char* what, const char* where) {
    if (!float_type(dtype)) return fail(BFZ_EINVAL, "%s: %s: unsupported dtype", where, what);
    return check_matrix(out, dtype, rows, dim, ld, int64_t(1) << 32, what, where);
}

// The type of a product's result, and whether exact products are asked for.
int32_t result_type(int32_t dtype, int32_t* exact) {
    *exact = dtype == BFZ_BF16_EXACT;
    return *exact ? kBF16 : dtype;
}

}  // namespace

extern "C" int bfz_quantize(const void* x, int32_t x_dtype, int64_t x_ld, int64_t n, int64_t dim, int32_t tiles, int32_t pow2,
                            uint8_t* codes, int64_t codes_ld, float* scales, int64_t scales_ld, void* stream) {
    const char* where = "bfz_quantize";
    if (n < 0 || dim < 1 || n > kMostTokens || dim > kMostDim)
        return fail(BFZ_EINVAL, "%s: need 0 <= n <= 2^24, 1 <= dim <= 2^20", where);
    int rc = check_quantize(n, dim, tiles, where);
    if (!rc) rc = check_out(x, x_dtype, n, dim, x_ld, "x", where);
    if (!rc) rc = check_codes(codes, n, dim, codes_ld, "codes", where);
    if (!rc) rc = check_scales(scales, scales_ld, tiles, n, dim, "scales", where);
    if (rc) return rc;
    const QuantizeArgs a{x, x_dtype, tiles != 0, pow2 != 0, x_ld, n, dim, codes, codes_ld, scales, scales_ld};
    return n == 0 ? BFZ_OK : launched(where, launch_quantize(a, stream));
}

extern "C" int64_t bfz_linear_work_bytes(int64_t n, int64_t rows, int64_t cols, int32_t x_dtype, int32_t copy) {
    if (n < 0 || rows < 1 || cols < 1 || n > kMostTokens || rows > kMostDim || cols > kMostDim ||
        !(float_type(x_dtype) || x_dtype == kE4M3))
        return 0;
    return linear_work_bytes(n, rows, cols, copy != 0 || cols % 16 != 0, x_dtype != kE4M3);
}

extern "C" int bfz_linear(const void* x, int32_t x_dtype, int64_t x_ld, const float* scales, int64_t scales_ld, int32_t tiles, int64_t n,
                          const uint8_t* weight, int64_t weight_ld, const float* grid, int64_t rows, int64_t cols, void* out,
                          int32_t out_dtype, int64_t out_ld, void* work, void* stream) {
    const char* where = "bfz_linear";
    int32_t exact;
    out_dtype = result_type(out_dtype, &exact);
    int rc = check_sizes(n, rows, cols, where);
    if (!rc) rc = check_tiles(rows, n, where);
    if (!rc) rc = check_weight(weight, weight_ld, grid, rows, cols, where);
    if (!rc) rc = check_out(out, out_dtype, n, rows, out_ld, "out", where);
    if (!rc) rc = check_work(work, where);
    if (rc) return rc;
    LinearArgs a{};
    if (x_dtype == kE4M3) {
        rc = check_codes(static_cast<const uint8_t*>(x), n, cols, x_ld, "x", where);
        if (!rc) rc = check_scales(scales, scales_ld, tiles, n, cols, "scales", where);
        if (rc) return rc;
        a.x = Codes{static_cast<const uint8_t*>(x), x_ld, scales, scales_ld, tiles != 0};
    } else {
        if (scales || tiles) return fail(BFZ_EINVAL, "%s: only E4M3 codes come with scales", where);
        rc = check_out(x, x_dtype, n, cols, x_ld, "x", where);
        if (!rc) rc = check_quantize(n, cols, 0, where);
        if (rc) return rc;
        a.values = x;
        a.values_type = x_dtype;
        a.values_ld = x_ld;
    }
    a.weight = weight;
    a.grid = grid;
    a.weight_ld = weight_ld;
    a.n = n;
    a.rows = rows;
    a.cols = cols;
    a.out = out;
    a.exact = exact;
    a.out_type = out_dtype;
    a.out_ld = out_ld;
    return n == 0 ? BFZ_OK : launched(where, launch_linear(a, work, stream));
}

extern "C" int bfz_linear_grad_input(const uint8_t* dout, int64_t dout_ld, const float* scales, int64_t scales_ld, int32_t tiles, int64_t n,
                                     const uint8_t* weight, int64_t weight_ld, const float* grid, int64_t rows, int64_t cols, void* dx,
                                     int32_t dx_dtype, int64_t dx_ld, int32_t accumulate, void* work, void* stream) {
    const char* where = "bfz_linear_grad_input";
    int32_t exact;
    dx_dtype = result_type(dx_dtype, &exact);
    int rc = check_sizes(n, rows, cols, where);
    if (!rc) rc = check_tiles(cols, n, where);
    if (!rc) rc = check_weight(weight, weight_ld, grid, rows, cols, where);
    if (!rc) rc = check_codes(dout, n, rows, dout_ld, "dout", where);
    if (!rc) rc = check_scales(scales, scales_ld, tiles, n, rows, "scales", where);
    if (!rc) rc = check_out(dx, dx_dtype, n, cols, dx_ld, "dx", where);
    if (!rc) rc = check_work(work, where);
    if (rc) return rc;
    LinearArgs a{};
    a.x = Codes{dout, dout_ld, scales, scales_ld, tiles != 0};
    a.weight = weight;
    a.grid = grid;
    a.weight_ld = weight_ld;
    a.n = n;
    a.rows = rows;
    a.cols = cols;
    a.out = dx;
    a.exact = exact;
    a.out_type = dx_dtype;
    a.out_ld = dx_ld;
    a.accumulate = accumulate != 0;
    return n == 0 ? BFZ_OK : launched(where, launch_linear_grad_input(a, work, stream));
}

extern "C" int bfz_linear_grad_weight(const uint8_t* dout, int64_t dout_ld, const float* dout_grid, int64_t dout_grid_ld, const uint8_t* x,
                                      int64_t x_ld, const float* x_grid, int64_t x_grid_ld, int64_t n, int64_t rows, int64_t cols,
                                      void* dweight, int32_t dweight_dtype, int64_t dweight_ld, int32_t accumulate, void* work,
                                      void* stream) {
    const char* where = "bfz_linear_grad_weight";
    int32_t exact;
    dweight_dtype = result_type(dweight_dtype, &exact);
    int rc = check_sizes(n, rows, cols, where);
    if (!rc) rc = check_tiles(cols, rows, where);
    if (!rc) rc = check_codes(dout, n, rows, dout_ld, "dout", where);
    if (!rc) rc = check_scales(dout_grid, dout_grid_ld, 1, n, rows, "dout_grid", where);
    if (!rc) rc = check_codes(x, n, cols, x_ld, "x", where);
    if (!rc) rc = check_scales(x_grid, x_grid_ld, 1, n, cols, "x_grid", where);
    if (!rc) rc = check_out(dweight, dweight_dtype, rows, cols, dweight_ld, "dweight", where);
    if (!rc) rc = check_work(work, where);
    if (rc) return rc;
    if (n == 0 && accumulate) return BFZ_OK;
    LinearArgs a{};
    a.x = Codes{dout, dout_ld, dout_grid, dout_grid_ld, 1};
    a.other = Codes{x, x_ld, x_grid, x_grid_ld, 1};
    a.n = n;
    a.rows = rows;
    a.cols = cols;
    a.out = dweight;
    a.exact = exact;
    a.out_type = dweight_dtype;
    a.out_ld = dweight_ld;
    a.accumulate = accumulate != 0;
    return launched(where, launch_linear_grad_weight(a, work, stream));
}

// ---- layer norm -----------------------------------------------------------------

namespace {

int check_norm_sizes(int64_t n, int64_t dim, const char* where) {
    if (n < 0 || n > kMostTokens || dim < 1 || dim > kNormMostDim)
        return fail(BFZ_EINVAL, "%s: need 0 <= n <= 2^24, 1 <= dim <= %lld", where, (long long)kNormMostDim);
    return BFZ_OK;
}

int check_vector(const void* p, int dtype, const char* what, const char* where) {
    if (!aligned(p, dtype_size(dtype))) return fail(BFZ_EALIGN, "%s: %s must be aligned to its elements", where, what);
    return BFZ_OK;
}

}  // namespace

extern "C" int bfz_layer_norm(const void* x, int32_t x_dtype, int64_t x_ld, int64_t n, int64_t dim, const void* weight, const void* bias,
                              int32_t param_dtype, float eps, void* out, int32_t out_dtype, int64_t out_ld, float* mean, float* rstd,
                              void* stream) {
    const char* where = "bfz_layer_norm";
    int rc = check_norm_sizes(n, dim, where);
    if (rc) return rc;
    if (!(eps > 0.0f) || !std::isfinite(eps)) return fail(BFZ_EINVAL, "%s: eps must be positive and finite", where);
    if (!float_type(param_dtype)) return fail(BFZ_EINVAL, "%s: weight and bias: unsupported dtype", where);
    rc = check_out(x, x_dtype, n, dim, x_ld, "x", where);
    if (!rc) rc = check_out(out, out_dtype, n, dim, out_ld, "out", where);
    if (!rc) rc = check_vector(weight, param_dtype, "weight", where);
    if (!rc) rc = check_vector(bias, param_dtype, "bias", where);
    if (!rc) rc = check_vector(mean, kF32, "mean", where);
    if (!rc) rc = check_vector(rstd, kF32, "rstd", where);
    if (rc || n == 0) return rc;
    const LayerNormArgs a{x, weight, bias, out, mean, rstd, x_dtype, param_dtype, out_dtype, x_ld, out_ld, n, dim, eps};
    return launched(where, launch_layer_norm(a, stream));
}

extern "C" int64_t bfz_layer_norm_work_bytes(int64_t n, int64_t dim) {
    return n < 0 || n > kMostTokens || dim < 1 || dim > kNormMostDim ? 0 : layer_norm_work_bytes(n, dim);
}

extern "C" int bfz_layer_norm_grad(const void* dout, int32_t dout_dtype, int64_t dout_ld, const void* x, int32_t x_dtype, int64_t x_ld,
                                   int64_t n, int64_t dim, const void* weight, int32_t param_dtype, const float* mean, const float* rstd,
                                   void* dx, int32_t dx_dtype, int64_t dx_ld, void* dweight, void* dbias, int32_t dparam_dtype,
                                   int32_t accumulate, void* work, void* stream) {
    const char* where = "bfz_layer_norm_grad";
    int rc = check_norm_sizes(n, dim, where);
    if (rc) return rc;
    if (!float_type(param_dtype) || !float_type(dparam_dtype))
        return fail(BFZ_EINVAL, "%s: weight, dweight and dbias: unsupported dtype", where);
    rc = check_out(dout, dout_dtype, n, dim, dout_ld, "dout", where);
    if (!rc) rc = check_out(x, x_dtype, n, dim, x_ld, "x", where);
    if (!rc && dx) rc = check_out(dx, dx_dtype, n, dim, dx_ld, "dx", where);
    if (!rc) rc = check_vector(weight, param_dtype, "weight", where);
    if (!rc) rc = check_vector(dweight, dparam_dtype, "dweight", where);
    if (!rc) rc = check_vector(dbias, dparam_dtype, "dbias", where);
    if (!rc && n > 0 && (!mean || !rstd)) rc = fail(BFZ_EINVAL, "%s: null pointer", where);
    if (!rc) rc = check_vector(mean, kF32, "mean", where);
    if (!rc) rc = check_vector(rstd, kF32, "rstd", where);
    if (!rc && (dweight || dbias)) rc = check_work(work, where);
    if (rc) return rc;
    if (n == 0 && (accumulate || (!dweight && !dbias))) return BFZ_OK;
    const LayerNormGradArgs a{dout, x, weight, mean, rstd, dx, dweight, dbias, dout_dtype, x_dtype, param_dtype, dx_dtype, dparam_dtype,
                              accumulate != 0, dout_ld, x_ld, dx_ld, n, dim};
    return launched(where, launch_layer_norm_grad(a, work, stream));
}

// ---- AdamW over many tensors ------------------------------------------------------

namespace {

int check_adamw_tensor(const bfz_adamw_tensor& t, int32_t k, const char* where) {
    if (!float_type(t.param_dtype) || !float_type(t.grad_dtype) || !(t.state_dtype == kF32 || t.state_dtype == kE4M3) || t.reserved != 0)
        return fail(BFZ_EINVAL, "%s: tensor %d: param and grad must be BFZ_F32, BFZ_BF16 or BFZ_F16, the states BFZ_F32 or BFZ_E4M3, reserved 0",
                    where, k);
    if (t.n < 0 || t.n > (int64_t(1) << 40)) return fail(BFZ_EINVAL, "%s: tensor %d: %lld elements", where, k, (long long)t.n);
    if (t.n == 0) return BFZ_OK;
    const bool codes = t.state_dtype == kE4M3;
    if (!t.param || !t.grad || !t.m || !t.v || (codes && (!t.m_scale || !t.v_scale)))
        return fail(BFZ_EINVAL, "%s: tensor %d: null pointer", where, k);
    if (!codes && (t.m_scale || t.v_scale)) return fail(BFZ_EINVAL, "%s: tensor %d: only E4M3 states have scales", where, k);
    if (!aligned(t.param, dtype_size(t.param_dtype)) || !aligned(t.grad, dtype_size(t.grad_dtype)) ||
        !aligned(t.m, dtype_size(t.state_dtype)) || !aligned(t.v, dtype_size(t.state_dtype)) || !aligned(t.m_scale, 4) ||
        !aligned(t.v_scale, 4))
        return fail(BFZ_EALIGN, "%s: tensor %d must be aligned to its elements", where, k);
    return BFZ_OK;
}

}  // namespace

extern "C" int bfz_adamw_list(const bfz_adamw_tensor* tensors, int32_t n_tensors, const bfz_adamw* hp, const float* grad_scale,
                              void* stream) {
    const char* where = "bfz_adamw_list";
    if (n_tensors < 0 || (n_tensors > 0 && !tensors) || !hp) return fail(BFZ_EINVAL, "%s: null pointer or negative count", where);
    if (!aligned(grad_scale, 4)) return fail(BFZ_EALIGN, "%s: grad_scale must be 4-byte aligned", where);
    StepScalars s;
    int rc = make_scalars(hp, nullptr, &s, where);
    for (int32_t k = 0; !rc && k < n_tensors; ++k) rc = check_adamw_tensor(tensors[k], k, where);
    if (rc) return rc;
    s.grad_scale = grad_scale;
    AdamwList list{};
    int64_t chunks = 0;
    // a launch's chunks are counted in 23 bits: 256 threads each
    constexpr int64_t kMostChunks = int64_t(1) << 23;
    auto flush = [&]() {
        if (list.count == 0) return BFZ_OK;
        list.chunks = (uint32_t)chunks;
        const int e = launched(where, launch_adamw_list(list, s, stream));
        list.count = 0;
        chunks = 0;
        return e;
    };
    for (int32_t k = 0; k < n_tensors; ++k) {
        const bfz_adamw_tensor& t = tensors[k];
        for (int64_t at = 0; at < t.n;) {
            const int64_t room = (kMostChunks - chunks) * kAdamwChunk;
            const int64_t take = t.n - at < room ? t.n - at : room;
            const int32_t i = list.count++;
            const int se = dtype_size(t.state_dtype);
            list.param[i] = static_cast<char*>(t.param) + at * dtype_size(t.param_dtype);
            list.grad[i] = static_cast<const char*>(t.grad) + at * dtype_size(t.grad_dtype);
            list.m[i] = static_cast<char*>(t.m) + at * se;
            list.v[i] = static_cast<char*>(t.v) + at * se;
            list.m_scale[i] = t.m_scale ? t.m_scale + at / kStateBlock : nullptr;
            list.v_scale[i] = t.v_scale ? t.v_scale + at / kStateBlock : nullptr;
            list.n[i] = take;
            list.chunk0[i] = (uint32_t)chunks;
            list.param_type[i] = (uint8_t)t.param_dtype;
            list.grad_type[i] = (uint8_t)t.grad_dtype;
            list.state_type[i] = (uint8_t)t.state_dtype;
            chunks += (take + kAdamwChunk - 1) / kAdamwChunk;
            at += take;
            if (list.count == kAdamwTensors || chunks == kMostChunks) {
                rc = flush();
                if (rc) return rc;
            }
        }
    }
    return flush();
}
