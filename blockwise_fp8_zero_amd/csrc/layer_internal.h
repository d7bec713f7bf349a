// Declarations shared by the operators of a layer (E4M3 linear products with
// their quantizer, layer norm) and by AdamW over many tensors: launch
// arguments and launchers.  Launchers return a hipError_t value as int.
#pragma once

#include "ops_internal.h"

namespace bfz {

// ---- quantizer --------------------------------------------------------------

struct QuantizeArgs {
    const void* x;
    int32_t x_type;
    int32_t tiles, pow2;
    int64_t x_ld, n, dim;
    uint8_t* codes;
    int64_t codes_ld;
    float* scales;  // rows: [ceil(dim/128)][scales_ld >= n]; tiles: [ceil(n/128)][scales_ld >= ceil(dim/128)]
    int64_t scales_ld;
};
int launch_quantize(const QuantizeArgs& a, void* stream);

// The quantizer's workgroups: 8 rows by 512 columns with 256 threads, or a tile with
// 512.  A launch counts its work-items in 32 bits.
constexpr int kQuantizeRowsThreads = 256, kQuantizeTilesThreads = 512;
constexpr int64_t kQuantizeRows = 8, kQuantizeCols = 512;
inline int64_t quantize_wgs(int64_t n, int64_t dim, int tiles) {
    const int64_t high = tiles ? kTileDim : kQuantizeRows, wide = tiles ? kTileDim : kQuantizeCols;
    return ((n + high - 1) / high) * ((dim + wide - 1) / wide);
}
inline bool quantize_fits(int64_t n, int64_t dim, int tiles) {
    return quantize_wgs(n, dim, tiles) < (int64_t(1) << 32) / (tiles ? kQuantizeTilesThreads : kQuantizeRowsThreads);
}

// ---- products ---------------------------------------------------------------

// Codes of activations or of their gradients, [n, dim], with their scales in
// either of the quantizer's forms.
struct Codes {
    const uint8_t* p;
    int64_t ld;
    const float* scales;
    int64_t scales_ld;
    int32_t tiles;
};

struct LinearArgs {
    Codes x;                // forward: the input; gradients: of the output
    Codes other;            // gradient of the weight: the input
    const void* values;     // forward: the input where x is yet to be made of it, else null
    int32_t values_type;
    int64_t values_ld;
    const uint8_t* weight;  // [rows, cols]
    const float* grid;
    int64_t weight_ld;
    int64_t n, rows, cols;
    void* out;
    int32_t out_type, accumulate, exact;
    int64_t out_ld;
};
// Of the products' workspace; copy: the weight's rows have to be copied;
// quantize: so have the inputs' codes and scales to be made.
int64_t linear_work_bytes(int64_t n, int64_t rows, int64_t cols, int copy, int quantize);
int launch_linear(const LinearArgs& a, void* work, void* stream);
int launch_linear_grad_input(const LinearArgs& a, void* work, void* stream);
int launch_linear_grad_weight(const LinearArgs& a, void* work, void* stream);

// Rows that the products read in place: on 16-byte boundaries, a multiple of
// 16 wide.
inline bool in_place(const void* p, int64_t ld, int64_t cols) {
    return ((reinterpret_cast<uintptr_t>(p) | (uint64_t)ld | (uint64_t)cols) & 15u) == 0;
}

// ---- layer norm -------------------------------------------------------------

constexpr int64_t kNormMostDim = 32768;

struct LayerNormArgs {
    const void* x;
    const void* weight;  // or null: ones
    const void* bias;    // or null: zeros
    void* out;
    float* mean;  // or null
    float* rstd;
    int32_t x_type, param_type, out_type;
    int64_t x_ld, out_ld, n, dim;
    float eps;
};
int launch_layer_norm(const LayerNormArgs& a, void* stream);

struct LayerNormGradArgs {
    const void* dout;
    const void* x;
    const void* weight;
    const float* mean;
    const float* rstd;
    void* dx;       // or null
    void* dweight;  // or null
    void* dbias;    // or null
    int32_t dout_type, x_type, param_type, dx_type, dparam_type, accumulate;
    int64_t dout_ld, x_ld, dx_ld, n, dim;
};
int64_t layer_norm_work_bytes(int64_t n, int64_t dim);
int launch_layer_norm_grad(const LayerNormGradArgs& a, void* work, void* stream);

// ---- AdamW over many tensors ------------------------------------------------

constexpr int kStateBlock = 256;   // elements that share the scales of 8-bit states
constexpr int kAdamwTensors = 56;  // of one launch: their table travels as a kernel argument
struct AdamwList {
    void* param[kAdamwTensors];
    const void* grad[kAdamwTensors];
    void* m[kAdamwTensors];
    void* v[kAdamwTensors];
    float* m_scale[kAdamwTensors];
    float* v_scale[kAdamwTensors];
    int64_t n[kAdamwTensors];
    uint32_t chunk0[kAdamwTensors];  // first chunk of each tensor in the launch
    uint8_t param_type[kAdamwTensors], grad_type[kAdamwTensors], state_type[kAdamwTensors];
    int32_t count;
    uint32_t chunks;
};
constexpr int64_t kAdamwChunk = 4096;  // elements, a multiple of kStateBlock
static_assert(sizeof(AdamwList) + sizeof(StepScalars) <= 3800, "kernel arguments are at most 4 KiB");
int launch_adamw_list(const AdamwList& list, const StepScalars& s, void* stream);

}  // namespace bfz
