// The C ABI of the operators around the step: argument checks and launches.
#include <hip/hip_runtime.h>

#include <cmath>

#include "ops_internal.h"

using namespace bfz;

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

int hip_fail(const char* where, int err) {
    return fail(BFZ_EHIP, "%s: %s", where, hip_error_string(err));
}

int launched(const char* where, int err) { return err == hipSuccess ? BFZ_OK : hip_fail(where, err); }

bool float_type(int t) { return t == kF32 || t == kBF16 || t == kF16; }

int check_norm(double max_norm, const double* sumsq, const float* norm, const float* coef, const char* where) {
    if (!(max_norm > 0.0)) return fail(BFZ_EINVAL, "%s: max_norm must be positive", where);
    if (!aligned(sumsq, 8)) return fail(BFZ_EALIGN, "%s: sumsq must be 8-byte aligned", where);
    if (!aligned(norm, 4) || !aligned(coef, 4))
        return fail(BFZ_EALIGN, "%s: norm and coef must be 4-byte aligned", where);
    return BFZ_OK;
}

int check_work(const void* work, const char* where) {
    if (!work) return fail(BFZ_EINVAL, "%s: null workspace", where);
    if (!aligned(work, 16)) return fail(BFZ_EALIGN, "%s: the workspace must be 16-byte aligned", where);
    return BFZ_OK;
}

int check_tensor(const bfz_tensor& t, int32_t k, const char* what, const char* where) {
    if (!float_type(t.dtype) || t.reserved != 0)
        return fail(BFZ_EINVAL, "%s: %s %d: dtype must be BFZ_F32, BFZ_BF16 or BFZ_F16 and reserved 0", where, what, k);
    if (t.n < 0 || t.n > (int64_t(1) << 40))
        return fail(BFZ_EINVAL, "%s: %s %d: %lld elements", where, what, k, (long long)t.n);
    if (t.n > 0 && !t.data) return fail(BFZ_EINVAL, "%s: %s %d: null pointer", where, what, k);
    if (!aligned(t.data, dtype_size(t.dtype)))
        return fail(BFZ_EALIGN, "%s: %s %d must be aligned to its elements", where, what, k);
    return BFZ_OK;
}

// Elements of a chunk, the unit that tensors are shared out by: four 16-byte
// float loads a thread of a workgroup, so that one small weight spreads over
// the device.
constexpr int64_t kChunkElems = 4096;

// Calls launch(list, first, last) for runs of kListTensors tensors; empty
// tensors are left out.  outs may be null.
template <class F>
int for_lists(const bfz_tensor* grads, const bfz_tensor* outs, int32_t n, F&& launch) {
    int32_t left = 0;
    for (int32_t k = 0; k < n; ++k) left += grads[k].n > 0;
    TensorList list{};
    list.chunk_elems = kChunkElems;
    bool first = true;
    if (left == 0) return launch(list, true, true);
    int64_t chunks = 0;
    for (int32_t k = 0; k < n; ++k) {
        if (grads[k].n == 0) continue;
        // a tensor of more chunks than a launch counts goes in several pieces
        for (int64_t at = 0; at < grads[k].n;) {
            const int64_t room = ((int64_t(1) << 31) - chunks) * list.chunk_elems;
            const int64_t take = grads[k].n - at < room ? grads[k].n - at : room;
            const int32_t i = list.count++;
            list.in[i] = static_cast<const char*>(grads[k].data) + at * dtype_size(grads[k].dtype);
            list.out[i] = outs ? static_cast<char*>(outs[k].data) + at * dtype_size(outs[k].dtype) : nullptr;
            list.in_type[i] = (uint8_t)grads[k].dtype;
            list.out_type[i] = outs ? (uint8_t)outs[k].dtype : 0;
            list.n[i] = take;
            list.chunk0[i] = (uint32_t)chunks;
            chunks += (take + list.chunk_elems - 1) / list.chunk_elems;
            at += take;
            const bool done = at == grads[k].n && left == 1;
            if (done || list.count == kListTensors || chunks >= (int64_t(1) << 31)) {
                list.chunks = (uint32_t)chunks;
                const int rc = launch(list, first, done);
                if (rc) return rc;
                first = false;
                list.count = 0;
                chunks = 0;
            }
        }
        --left;
    }
    return BFZ_OK;
}

}  // namespace

extern "C" int64_t bfz_norm_work_bytes(void) { return kNormWorkBytes; }

extern "C" int bfz_grad_norm(const bfz_tensor* grads, int32_t n_tensors, double max_norm, double* sumsq, float* norm,
                             float* coef, void* work, void* stream) {
    const char* where = "bfz_grad_norm";
    if (n_tensors < 0 || (n_tensors > 0 && !grads)) return fail(BFZ_EINVAL, "%s: null pointer or negative count", where);
    int rc = check_norm(max_norm, sumsq, norm, coef, where);
    if (!rc) rc = check_work(work, where);
    for (int32_t k = 0; !rc && k < n_tensors; ++k) rc = check_tensor(grads[k], k, "gradient", where);
    if (rc) return rc;
    return for_lists(grads, nullptr, n_tensors, [&](const TensorList& list, bool first, bool last) {
        const NormOut out{sumsq, norm, coef, max_norm, first, last};
        return launched(where, launch_list_sumsq(list, out, work, stream));
    });
}

extern "C" int bfz_shard_grad_norm(const bfz_plan* plan, const float* const* grad, double max_norm, double* sumsq,
                                   float* norm, float* coef, void* work, void* stream) {
    const char* where = "bfz_shard_grad_norm";
    if (!plan || !grad) return fail(BFZ_EINVAL, "%s: null pointer", where);
    int rc = check_norm(max_norm, sumsq, norm, coef, where);
    if (!rc) rc = check_work(work, where);
    if (!rc) rc = check_plan(plan, where);
    if (!rc) rc = check_weights(plan, reinterpret_cast<const void* const*>(grad), where);
    if (rc) return rc;
    for (int32_t w = 0; w < plan->n_weights; ++w)
        if (grad[w] && !aligned(grad[w], 4))
            return fail(BFZ_EALIGN, "%s: gradient %d must be 4-byte aligned", where, w);
    const size_t n = plan->segments.size();
    if (n == 0) {
        const NormOut out{sumsq, norm, coef, max_norm, 1, 1};
        return launched(where, launch_shard_sumsq(plan->d_entries, 0, PackArgs{}, out, work, stream));
    }
    for (size_t i = 0; i < n; ++i) {
        const Segment& seg = plan->segments[i];
        PackArgs args{};
        for (int32_t k = 0; k < seg.n_weights; ++k) args.src[k] = grad[seg.weight0 + k];
        const NormOut out{sumsq, norm, coef, max_norm, i == 0, i + 1 == n};
        rc = launched(where, launch_shard_sumsq(plan->d_entries + seg.slot0, seg.n_slots, args, out, work, stream));
        if (rc) return rc;
    }
    return BFZ_OK;
}

extern "C" int bfz_clip_coef(const double* sumsq, double max_norm, float* norm, float* coef, void* stream) {
    const char* where = "bfz_clip_coef";
    if (!sumsq) return fail(BFZ_EINVAL, "%s: null pointer", where);
    const int rc = check_norm(max_norm, sumsq, norm, coef, where);
    return rc ? rc : launched(where, launch_clip_coef(sumsq, max_norm, norm, coef, stream));
}

extern "C" int bfz_clip_grads(const bfz_tensor* grads, const bfz_tensor* outs, int32_t n_tensors, const float* coef,
                              void* stream) {
    const char* where = "bfz_clip_grads";
    if (n_tensors < 0 || (n_tensors > 0 && (!grads || !outs)) || !coef)
        return fail(BFZ_EINVAL, "%s: null pointer or negative count", where);
    if (!aligned(coef, 4)) return fail(BFZ_EALIGN, "%s: coef must be 4-byte aligned", where);
    for (int32_t k = 0; k < n_tensors; ++k) {
        int rc = check_tensor(grads[k], k, "gradient", where);
        if (!rc) rc = check_tensor(outs[k], k, "output", where);
        if (rc) return rc;
        if (outs[k].n != grads[k].n)
            return fail(BFZ_EINVAL, "%s: output %d has %lld elements, its gradient %lld", where, k, (long long)outs[k].n,
                        (long long)grads[k].n);
        if (outs[k].n > 0 && outs[k].data == grads[k].data && outs[k].dtype != grads[k].dtype)
            return fail(BFZ_EINVAL, "%s: output %d is its gradient's memory with another dtype", where, k);
    }
    return for_lists(grads, outs, n_tensors, [&](const TensorList& list, bool, bool) {
        return launched(where, launch_clip(list, coef, stream));
    });
}

namespace {

int check_ids(const void* ids, int32_t ids64, int64_t n, int64_t vocab, int64_t dim, const char* where) {
    if (n < 0 || vocab < 1 || dim < 1 || vocab > (int64_t(1) << 27) || n > (int64_t(1) << 27) || dim > (int64_t(1) << 24))
        return fail(BFZ_EINVAL, "%s: need 0 <= n <= 2^27, 1 <= vocab <= 2^27, 1 <= dim <= 2^24", where);
    if (n > 0 && !ids) return fail(BFZ_EINVAL, "%s: null pointer", where);
    if (!aligned(ids, ids64 ? 8 : 4)) return fail(BFZ_EALIGN, "%s: ids must be aligned to their elements", where);
    return BFZ_OK;
}

// A matrix of rows ld elements apart.
int check_matrix(const void* p, int dtype, int64_t rows, int64_t dim, int64_t ld, const char* what, const char* where) {
    if (rows > 0 && !p) return fail(BFZ_EINVAL, "%s: %s: null pointer", where, what);
    if (ld < dim || ld > (int64_t(1) << 32)) return fail(BFZ_EINVAL, "%s: %s: rows %lld elements apart, %lld wide", where, what, (long long)ld, (long long)dim);
    if (!aligned(p, dtype_size(dtype))) return fail(BFZ_EALIGN, "%s: %s must be aligned to its elements", where, what);
    return BFZ_OK;
}

}  // namespace

extern "C" int bfz_embed(const void* ids, int32_t ids64, int64_t n, const void* table, int32_t table_dtype,
                         const float* grid, int64_t vocab, int64_t dim, int64_t table_ld, float scale, void* out,
                         int32_t out_dtype, int64_t out_ld, void* stream) {
    const char* where = "bfz_embed";
    int rc = check_ids(ids, ids64, n, vocab, dim, where);
    if (rc) return rc;
    if (!(float_type(table_dtype) || table_dtype == kE4M3) || !float_type(out_dtype))
        return fail(BFZ_EINVAL, "%s: unsupported dtype", where);
    if ((table_dtype == kE4M3) != (grid != nullptr))
        return fail(BFZ_EINVAL, "%s: E4M3 codes need their scale grid, other tables none", where);
    if (!aligned(grid, 4)) return fail(BFZ_EALIGN, "%s: grid must be 4-byte aligned", where);
    rc = check_matrix(table, table_dtype, vocab, dim, table_ld, "table", where);
    if (!rc) rc = check_matrix(out, out_dtype, n, dim, out_ld, "out", where);
    if (rc) return rc;
    const EmbedArgs a{ids, ids64, table_dtype, out_dtype, table, grid, out, n, vocab, dim, table_ld, out_ld, scale};
    return launched(where, launch_embed(a, stream));
}

extern "C" int64_t bfz_embed_grad_work_bytes(int64_t n, int64_t dim) {
    return n < 0 || dim < 1 || n > (int64_t(1) << 27) || dim > (int64_t(1) << 24) ? 0 : embed_grad_work_bytes(n, dim);
}

extern "C" int bfz_embed_grad(const void* ids, int32_t ids64, int64_t n, const void* dout, int32_t dout_dtype,
                              int64_t dout_ld, int64_t vocab, int64_t dim, float scale, int32_t accumulate, void* dtable,
                              int32_t dtable_dtype, int64_t dtable_ld, void* work, void* stream) {
    const char* where = "bfz_embed_grad";
    int rc = check_ids(ids, ids64, n, vocab, dim, where);
    if (rc) return rc;
    if (!float_type(dout_dtype) || !float_type(dtable_dtype)) return fail(BFZ_EINVAL, "%s: unsupported dtype", where);
    rc = check_matrix(dout, dout_dtype, n, dim, dout_ld, "dout", where);
    if (!rc) rc = check_matrix(dtable, dtable_dtype, vocab, dim, dtable_ld, "dtable", where);
    if (!rc && n > 0) rc = check_work(work, where);
    if (rc) return rc;
    // a launch counts its work-items in 32 bits: 2^24 workgroups of 256.  A
    // workgroup fills 64 rows or 128 KiB of them, one row at least.
    const int64_t fill = dim * dtype_size(dtable_dtype) > 2048 ? vocab / (1 + (128 * 1024) / (dim * dtype_size(dtable_dtype))) * 2 : vocab / 64;
    if (((n + 7) / 8) * ((dim + 255) / 256) + fill >= (int64_t(1) << 24) - 1)
        return fail(BFZ_EINVAL, "%s: %lld tokens and %lld rows of width %lld are too many for one call", where, (long long)n,
                    (long long)vocab, (long long)dim);
    const EmbedGradArgs a{ids, ids64, dout_dtype, dtable_dtype, dout, dtable, n, vocab, dim, dout_ld, dtable_ld, scale, accumulate};
    return launched(where, launch_embed_grad(a, work, stream));
}

namespace {

int check_loss(const void* hidden, int64_t hidden_ld, int64_t n, const void* weight, int32_t weight_dtype, int64_t weight_ld,
               const float* grid, int64_t vocab, int64_t dim, const void* targets, int32_t targets64, const void* work,
               const char* where) {
    if (n < 0 || vocab < 1 || dim < 1 || n > (int64_t(1) << 24) || vocab > (int64_t(1) << 27) || dim > (int64_t(1) << 20))
        return fail(BFZ_EINVAL, "%s: need 0 <= n <= 2^24, 1 <= vocab <= 2^27, 1 <= dim <= 2^20", where);
    // a launch counts its work-items in 32 bits: under 2^23 tiles of 512
    if (((vocab + 255) / 256) * ((n + 63) / 64) >= (int64_t(1) << 23) ||
        ((dim + 255) / 256) * ((n + 63) / 64) >= (int64_t(1) << 23))
        return fail(BFZ_EINVAL, "%s: %lld tokens by %lld rows of width %lld are too many for one call", where, (long long)n,
                    (long long)vocab, (long long)dim);
    if (weight_dtype != kBF16 && weight_dtype != kE4M3)
        return fail(BFZ_EINVAL, "%s: the weight must be BFZ_BF16 or BFZ_E4M3", where);
    if ((weight_dtype == kE4M3) != (grid != nullptr))
        return fail(BFZ_EINVAL, "%s: E4M3 codes need their scale grid, bf16 weights none", where);
    if (!aligned(grid, 4)) return fail(BFZ_EALIGN, "%s: grid must be 4-byte aligned", where);
    if (hidden_ld > (int64_t(1) << 21) || weight_ld > (int64_t(1) << 21))
        return fail(BFZ_EINVAL, "%s: strides are at most 2^21", where);
    int rc = check_matrix(hidden, kBF16, n, dim, hidden_ld, "hidden", where);
    if (!rc) rc = check_matrix(weight, weight_dtype, vocab, dim, weight_ld, "weight", where);
    if (rc) return rc;
    if (n > 0 && !targets) return fail(BFZ_EINVAL, "%s: null pointer", where);
    if (!aligned(targets, targets64 ? 8 : 4)) return fail(BFZ_EALIGN, "%s: targets must be aligned to their elements", where);
    if (!work) return fail(BFZ_EINVAL, "%s: null workspace", where);
    if (!aligned(work, 256)) return fail(BFZ_EALIGN, "%s: the workspace must be 256-byte aligned", where);
    return BFZ_OK;
}

}  // namespace

extern "C" int64_t bfz_vocab_loss_work_bytes(int64_t n, int64_t vocab, int64_t dim, int32_t weight_dtype, int32_t grad) {
    if (n < 0 || vocab < 1 || dim < 1 || n > (int64_t(1) << 24) || vocab > (int64_t(1) << 27) || dim > (int64_t(1) << 20) ||
        (weight_dtype != kBF16 && weight_dtype != kE4M3))
        return 0;
    return vocab_loss_work_bytes(n, vocab, dim, weight_dtype == kE4M3, grad != 0);
}

extern "C" int bfz_vocab_loss(const void* hidden, int64_t hidden_ld, int64_t n, const void* weight, int32_t weight_dtype,
                              int64_t weight_ld, const float* grid, int64_t vocab, int64_t dim, const void* targets,
                              int32_t targets64, float* loss, float* lse, void* work, void* stream) {
    const char* where = "bfz_vocab_loss";
    const int rc = check_loss(hidden, hidden_ld, n, weight, weight_dtype, weight_ld, grid, vocab, dim, targets, targets64, work, where);
    if (rc) return rc;
    if (n > 0 && (!loss || !lse)) return fail(BFZ_EINVAL, "%s: null pointer", where);
    if (!aligned(loss, 4) || !aligned(lse, 4)) return fail(BFZ_EALIGN, "%s: loss and lse must be 4-byte aligned", where);
    VocabLossArgs a{};
    a.hidden = hidden;
    a.weight = weight;
    a.grid = grid;
    a.targets = targets;
    a.targets64 = targets64;
    a.fp8 = weight_dtype == kE4M3;
    a.n = n;
    a.vocab = vocab;
    a.dim = dim;
    a.hidden_ld = hidden_ld;
    a.weight_ld = weight_ld;
    a.loss = loss;
    a.lse = lse;
    return launched(where, launch_vocab_loss(a, work, stream));
}

extern "C" int bfz_vocab_loss_grad(const void* hidden, int64_t hidden_ld, int64_t n, const void* weight, int32_t weight_dtype,
                                   int64_t weight_ld, const float* grid, int64_t vocab, int64_t dim, const void* targets,
                                   int32_t targets64, const float* lse, const float* dloss, void* dhidden, int64_t dhidden_ld,
                                   void* dweight, int32_t dweight_dtype, int64_t dweight_ld, int32_t accumulate, void* work,
                                   void* stream) {
    const char* where = "bfz_vocab_loss_grad";
    int rc = check_loss(hidden, hidden_ld, n, weight, weight_dtype, weight_ld, grid, vocab, dim, targets, targets64, work, where);
    if (rc) return rc;
    if (n > 0 && (!lse || !dloss)) return fail(BFZ_EINVAL, "%s: null pointer", where);
    if (!aligned(lse, 4) || !aligned(dloss, 4)) return fail(BFZ_EALIGN, "%s: lse and dloss must be 4-byte aligned", where);
    if (dhidden) rc = check_matrix(dhidden, kBF16, n, dim, dhidden_ld, "dhidden", where);
    if (rc) return rc;
    const bool two_parts = dweight && dweight_dtype == kF32;
    if (dweight) {
        if (dweight_dtype == BFZ_F32_ROUNDED) dweight_dtype = kF32;
        if (dweight_dtype != kBF16 && dweight_dtype != kF32)
            return fail(BFZ_EINVAL, "%s: dweight must be BFZ_BF16, BFZ_F32 or BFZ_F32_ROUNDED", where);
        rc = check_matrix(dweight, dweight_dtype, vocab, dim, dweight_ld, "dweight", where);
        if (rc) return rc;
    }
    VocabLossArgs a{};
    a.hidden = hidden;
    a.weight = weight;
    a.grid = grid;
    a.targets = targets;
    a.targets64 = targets64;
    a.fp8 = weight_dtype == kE4M3;
    a.n = n;
    a.vocab = vocab;
    a.dim = dim;
    a.hidden_ld = hidden_ld;
    a.weight_ld = weight_ld;
    a.lse = const_cast<float*>(lse);
    a.dloss = dloss;
    a.dhidden = dhidden;
    a.dhidden_ld = dhidden_ld;
    a.dweight = dweight;
    a.dweight_type = dweight_dtype;
    a.dz_parts = two_parts ? 2 : 1;
    a.dweight_ld = dweight_ld;
    a.accumulate = accumulate;
    return launched(where, launch_vocab_loss_grad(a, work, stream));
}
