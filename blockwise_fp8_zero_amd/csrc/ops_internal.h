// Declarations shared by the operators around the step (gradient norm and
// clipping, token embedding, vocabulary cross entropy): launch arguments
// and launchers.  Launchers return a hipError_t value as int.
#pragma once

#include "bfz_internal.h"

namespace bfz {

constexpr int kF32 = BFZ_F32, kBF16 = BFZ_BF16, kF16 = BFZ_F16, kE4M3 = BFZ_E4M3;

inline int dtype_size(int t) { return t == kF32 ? 4 : t == kE4M3 ? 1 : 2; }

// ---- gradient norm ----------------------------------------------------------

// Workspace: header, then one partial sum per workgroup of a launch.
struct NormWork {
    uint32_t ticket;  // workgroups done in this launch; zero between launches
    uint32_t pad;
    double carry;     // sum of the launches before this one
};
constexpr int kNormBlocks = 2048;  // most workgroups of a launch
constexpr int64_t kNormWorkBytes = 64 + int64_t(kNormBlocks) * 8;

// Tensors one launch covers: their table travels as a kernel argument.
constexpr int kListTensors = 96;
struct TensorList {
    const void* in[kListTensors];
    void* out[kListTensors];       // clip only
    int64_t n[kListTensors];
    uint32_t chunk0[kListTensors]; // first chunk of each tensor in the launch
    uint8_t in_type[kListTensors], out_type[kListTensors];
    int32_t count;
    uint32_t chunks;
    int64_t chunk_elems;
};
static_assert(sizeof(TensorList) <= 3400, "kernel arguments are at most 4 KiB");

// What the last workgroup of the last launch writes (each may be null).
struct NormOut {
    double* sumsq;
    float* norm;
    float* coef;
    double max_norm;
    int32_t first, last;  // this launch starts / ends the sum
};

int launch_list_sumsq(const TensorList& list, const NormOut& out, void* work, void* stream);
int launch_shard_sumsq(const TileEntry* d_entries, int64_t n_slots, const PackArgs& grads,
                       const NormOut& out, void* work, void* stream);
int launch_clip_coef(const double* sumsq, double max_norm, float* norm, float* coef, void* stream);
int launch_clip(const TensorList& list, const float* coef, void* stream);

// ---- token embedding --------------------------------------------------------

struct EmbedArgs {
    const void* ids;  // int64 when ids64, else int32
    int32_t ids64;
    int32_t table_type, out_type;
    const void* table;
    const float* grid;  // tile scales of an E4M3 table, else null
    void* out;
    int64_t n, vocab, dim, table_ld, out_ld;  // strides in elements
    float scale;
};
int launch_embed(const EmbedArgs& a, void* stream);

struct EmbedGradArgs {
    const void* ids;
    int32_t ids64;
    int32_t dout_type, dtable_type;
    const void* dout;
    void* dtable;
    int64_t n, vocab, dim, dout_ld, dtable_ld;
    float scale;
    int32_t accumulate;
};
int64_t embed_grad_work_bytes(int64_t n, int64_t dim);
int launch_embed_grad(const EmbedGradArgs& a, void* work, void* stream);

// ---- vocabulary cross entropy -----------------------------------------------

struct VocabLossArgs {
    const void* hidden;   // bf16 [n, dim]
    const void* weight;   // bf16 or E4M3 codes [vocab, dim]
    const float* grid;    // tile scales of E4M3 codes, else null
    const void* targets;  // int64 when targets64, else int32
    int32_t targets64, fp8;
    int64_t n, vocab, dim, hidden_ld, weight_ld;
    float* loss;          // forward
    float* lse;           // forward: written; gradient: read
    const float* dloss;   // gradient
    void* dhidden;        // bf16, or null
    void* dweight;        // bf16 or f32, or null
    int32_t dweight_type, accumulate;
    int32_t dz_parts;     // bf16 parts of dz that dweight is made of: 1 or 2
    int64_t dhidden_ld, dweight_ld;
};
int64_t vocab_loss_work_bytes(int64_t n, int64_t vocab, int64_t dim, int fp8, int grad);
int launch_vocab_loss(const VocabLossArgs& a, void* work, void* stream);
int launch_vocab_loss_grad(const VocabLossArgs& a, void* work, void* stream);

}  // namespace bfz
