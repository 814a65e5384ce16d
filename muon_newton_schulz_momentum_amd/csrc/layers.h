// Launch wrappers of the expert layers' kernels (internal): gated blocks, 8-bit integer products, gathered and combined rows.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "muon.h"

namespace muon {

// One launch of products.  What it computes goes by its form:
//   FORM_GATED   out[0] = act(a[0] b[0]^T) * (a[0] b[1]^T), the two sums into out[1] and out[2] where those are there
//   FORM_SCALED  out[0] = a[0] b[0]^T by their rows' scales (8-bit integers)
//   FORM_GRAD_X  out[0] = a[0] b[0] + a[1] b[1]; a's rows are padded to multiples of 64 with zeros
//   FORM_GRAD_W  out[w] = a[w]^T b[0] for w = 0, 1, over each group's rows
enum LayerForm { FORM_GATED, FORM_SCALED, FORM_GRAD_X, FORM_GRAD_W };

struct LayerArgs {
    const uint8_t *a[2], *b[2];
    const float *sa, *sb[2];           // scales of 8-bit integers' rows
    int64_t lda, ldb, stride_b;        // in bytes
    int64_t stride_sb;                 // in scales
    const int32_t* offsets;            // nullable: no groups
    void* out[3];
    int64_t ld_out[2], out_stride;     // in elements; ld_out[1]: of out[1] and out[2] (FORM_GATED)
    int64_t m, n, k;                   // rows and columns of out, depth (of each product that is added up)
    int32_t groups, mode, accumulate, activation;
    int32_t tiles_m, tiles_n, tiles;   // set by the launch
    int32_t vec;                       // rows of out are 16-byte aligned
};

// dg = d u act'(g), du = d act(g) for rows [offsets[0], offsets[groups]) of m, or all; zeros from column n on to a multiple of 64
struct GatedGradArgs {
    const uint16_t *grad, *pre_gate, *pre_up;
    uint16_t *grad_pre_gate, *grad_pre_up;
    int64_t m, n, ld_grad, ld_pre, ld_out;
    const int32_t* offsets;
    int32_t groups, activation;
};

struct Int8QuantizeArgs {
    const void* src;
    const int32_t* gather;
    const int32_t* limit;
    int8_t* codes;
    float* scales;
    int64_t rows, cols, ld, batch_stride, src_rows, total;  // total: rows of all matrices
    int64_t kp;                                             // row stride of codes
    int32_t per;
};

struct GatherRowsArgs {
    const void* src;
    const int32_t* rows;
    const int32_t* limit;
    void* out;
    const float* weights;
    const void* y;
    const int32_t* position;
    float* grad_weights;
    int64_t cols, ld, ld_out, ld_y, n_rows, choices;
    int32_t per;
};

struct CombineRowsArgs {
    const void* src;
    const int32_t* position;
    const float* weights;
    const void* residual;
    void* out;
    int64_t n_rows, cols, ld, ld_out, ld_residual, tokens;
    int32_t top_k;
};

// Whether a launch's output tiles can be counted; launch_layer takes no others.
bool layer_fits(LayerArgs a, LayerForm form);
hipError_t launch_layer(LayerArgs a, LayerForm form, int32_t operands, int32_t out_dtype, hipStream_t s);
hipError_t launch_gated_grad(const GatedGradArgs& a, hipStream_t s);
hipError_t launch_int8_quantize(const Int8QuantizeArgs& a, int32_t src_dtype, hipStream_t s);
hipError_t launch_gather_rows(const GatherRowsArgs& a, int32_t dtype, hipStream_t s);
hipError_t launch_combine_rows(const CombineRowsArgs& a, int32_t dtype, int32_t out_dtype, hipStream_t s);

}  // namespace muon
