// Launch wrappers of the routed-expert kernels (internal).
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "muon.h"

namespace muon {

struct RouteArgs {
    const void* logits;
    const float* bias;         // nullable
    int32_t* experts;          // tokens x top_k
    float* weights;            // tokens x top_k
    int64_t tokens, ld;
    int32_t n_experts, top_k, n_groups, top_groups, score, renormalize;
    float scale;
};

struct RouteBackwardArgs {
    const void* logits;
    const int32_t* experts;
    const float* grad_weights;
    void* grad_logits;
    int64_t tokens, ld, ld_grad;
    int32_t n_experts, top_k, score, renormalize;
    float scale;
};

// Choices that one workgroup groups in a single launch, and that a workgroup takes of more.
constexpr int64_t GROUP_SINGLE_MAX = 8192;
constexpr int64_t GROUP_CHUNK = 2048;

struct GroupRowsArgs {
    const int32_t* experts;
    int32_t* counts;
    int32_t* offsets;
    int32_t* rows;
    int32_t* position;
    int32_t* partial;          // workspace: chunks x n_experts
    int64_t n, capacity, chunks;
    int32_t n_experts, align;
};

struct QuantizeArgs {
    const void* src;
    const int32_t* gather;
    const int32_t* limit;
    uint8_t *codes, *scales, *codes_t, *scales_t;
    int64_t rows, cols, ld, batch_stride, src_rows;
    int64_t kp, sp;            // row strides of codes and scales
    int64_t kp_t, sp_t;        // and of the transposed copy
    int32_t per;
    int32_t tiles_r, tiles_c;  // 128 x 128 tiles of a matrix
    int64_t tiles;             // of all matrices
};

struct ProductArgs {
    const uint8_t *a, *as, *b, *bs;
    int64_t lda, ldas, ldb, ldbs, stride_b, stride_bs;
    int32_t shift_a, shift_b;  // scale row of matrix row r: r >> shift (0 or 7)
    const int32_t* offsets;
    void* out;
    int64_t ld_out, out_stride;
    int64_t m, n, k;
    int32_t groups, mode, accumulate;
    int32_t tiles_m, tiles_n, tiles;
    int32_t vec;               // out rows are 16-byte aligned
};

hipError_t launch_route(const RouteArgs& a, int32_t dtype, hipStream_t s);
hipError_t launch_route_backward(const RouteBackwardArgs& a, int32_t dtype, hipStream_t s);
hipError_t launch_group_rows(const GroupRowsArgs& a, hipStream_t s);
hipError_t launch_balance(const float* bias, const int32_t* counts, int32_t n, float rate, float* out, hipStream_t s);
hipError_t launch_quantize(const QuantizeArgs& a, int32_t src_dtype, int32_t format, int32_t square, hipStream_t s);
// Whether the output tiles can be counted; launch_product takes no others.
bool product_fits(ProductArgs a);
hipError_t launch_product(ProductArgs a, int32_t a_format, int32_t out_dtype, bool full_sums, hipStream_t s);

}  // namespace muon
