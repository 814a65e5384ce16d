// Entry points of the expert layers: gated blocks, 8-bit integer quantisation and products, gathered and combined rows.
// Arguments are checked here, on the host; a kernel is only launched with sizes and strides that keep it inside the
// buffers they describe.
#include <hip/hip_runtime.h>

#include "api_checks.h"
#include "layers.h"

using namespace muon;
using namespace muon::checks;

namespace {

constexpr int64_t MAX_LD_BYTES = 1 << 23;  // row stride of an operand: a tile's 256 rows lie within 2^31 bytes
constexpr int64_t MAX_INT8_DEPTH = 131071; // 2^31 / (128 * 128), less one: no sum leaves 32 bits

int64_t size_of(int32_t dtype) { return dtype == MUON_DTYPE_F32 ? 4 : 2; }

// rows x cols bfloat16 or float32 values with a row stride
muon_status check_rows(const void* p, int64_t ld, int64_t cols, const char* who, const char* name) {
    if (ld < cols || ld > MAX_I32) return fail(MUON_ERR_SHAPE, who, (std::string("row stride of ") + name + " must be at least its columns and below 2^31").c_str());
    if (!p) return fail(MUON_ERR_INVALID_ARG, who, (std::string(name) + " is NULL").c_str());
    if (misaligned(p)) return fail(MUON_ERR_ALIGNMENT, who, (std::string(name) + " must be 16-byte aligned").c_str());
    return MUON_OK;
}

// An operand of `rows` rows of k values per group.  Without depth only its scales are read.
muon_status check_operand(const muon_operand& o, int32_t operands, int64_t rows, int64_t k, int64_t groups, const char* who, const char* name) {
    const bool i8 = operands == MUON_OPERANDS_INT8;
    auto wrong = [&](muon_status s, const char* what) { return fail(s, who, (std::string(name) + what).c_str()); };
    if ((k > 0 && !o.data) || (i8 && !o.scales)) return wrong(MUON_ERR_INVALID_ARG, ": data and, of 8-bit integers, scales must be non-NULL");
    if (!i8 && o.scales) return wrong(MUON_ERR_INVALID_ARG, ": bfloat16 has no scales");
    if ((k > 0 && misaligned(o.data)) || ((uintptr_t)o.scales & 3u) != 0) return wrong(MUON_ERR_ALIGNMENT, ": data must be 16-byte aligned (scales 4-byte)");
    if (i8 && groups > 1 && o.stride_scales < rows) return wrong(MUON_ERR_SHAPE, ": stride_scales must hold one matrix's scales");
    if (k == 0) return MUON_OK;
    if (i8 ? o.ld % 16 != 0 || o.ld < round_up(k, 128) || o.ld >= MAX_LD_BYTES : o.ld < k || o.ld >= MAX_LD_BYTES / 2)
        return wrong(MUON_ERR_SHAPE, i8 ? ": row stride must be a multiple of 16, at least round_up(k, 128) and below 2^23"
                                        : ": row stride must be at least k and below 2^22");
    if (groups > 1) {
        const double need = (double)(rows - 1) * (double)o.ld + (double)(i8 ? round_up(k, 128) : k);
        if ((double)o.stride < need || (i8 && o.stride % 16 != 0))
            return wrong(MUON_ERR_SHAPE, ": stride must hold one matrix (and, of codes, be a multiple of 16)");
    }
    return MUON_OK;
}
muon_status check_alike(const muon_operand& gate, const muon_operand& up, int32_t operands, int64_t k, int64_t groups, const char* who) {
    if ((k > 0 && (gate.ld != up.ld || (groups > 1 && gate.stride != up.stride))) ||
        (operands == MUON_OPERANDS_INT8 && groups > 1 && gate.stride_scales != up.stride_scales))
        return fail(MUON_ERR_SHAPE, who, "gate and up must have the same strides");
    return MUON_OK;
}
Extent values_of(const muon_operand& o, int32_t operands, int64_t rows, int64_t k, int64_t groups) {
    const bool i8 = operands == MUON_OPERANDS_INT8;
    if (k == 0) return extent(nullptr, 0.0);
    return extent(o.data, groups, o.stride, rows, o.ld, i8 ? round_up(k, 128) : k, i8 ? 1 : 2);
}
Extent scales_of(const muon_operand& o, int64_t rows, int64_t groups) { return extent(o.scales, groups, o.stride_scales, 1, rows, rows, 4); }

// mode, groups and sizes that the products have in common
muon_status check_product(int32_t mode, int32_t groups, int64_t m, int64_t n, int64_t k, int64_t max_k, const int32_t* offsets, const char* who) {
    if (mode != MUON_PRODUCT_DENSE && mode != MUON_PRODUCT_ROWS) return fail(MUON_ERR_INVALID_ARG, who, "mode must be MUON_PRODUCT_DENSE or MUON_PRODUCT_ROWS");
    if (groups < 1 || groups > MUON_MAX_EXPERTS || (mode == MUON_PRODUCT_DENSE && groups != 1))
        return fail(MUON_ERR_INVALID_ARG, who, "groups must be in [1, 1024], and 1 without groups");
    if (m < 0 || n < 0 || k < 0 || m > MAX_I32 - 127 || n > MAX_I32 - 127 || k > max_k)
        return fail(MUON_ERR_SHAPE, who, max_k == MAX_INT8_DEPTH ? "m, n and k must be at least 0, m and n below 2^31 - 127, k below 2^17"
                                                                : "m, n and k must be at least 0 and below 2^31 - 127");
    if (mode == MUON_PRODUCT_ROWS && m > 0 && n > 0 && !offsets) return fail(MUON_ERR_INVALID_ARG, who, "offsets is NULL");
    if (((uintptr_t)offsets & 3u) != 0) return fail(MUON_ERR_ALIGNMENT, who, "offsets must be 4-byte aligned");
    return MUON_OK;
}

// The same for the launch; operands are set by the caller.
LayerArgs layer_args(int32_t mode, int32_t groups, const int32_t* offsets, int64_t m, int64_t n, int64_t k) {
    LayerArgs a{};
    a.mode = mode;
    a.groups = groups;
    a.offsets = mode == MUON_PRODUCT_DENSE ? nullptr : offsets;
    a.m = m;
    a.n = n;
    a.k = k;
    return a;
}
// (without depth values and their strides were not checked and are not read)
void set_a(LayerArgs& a, int i, const void* p, const float* scales, int64_t ld, int64_t size) {
    a.sa = scales;
    if (a.k == 0) return;
    a.a[i] = static_cast<const uint8_t*>(p);
    a.lda = ld * size;
}
void set_b(LayerArgs& a, int i, const muon_operand& o, int64_t size) {
    if (a.k > 0) {
        a.b[i] = static_cast<const uint8_t*>(o.data);
        a.ldb = o.ld * size;
        a.stride_b = a.groups > 1 ? o.stride * size : 0;
    }
    a.sb[i] = o.scales;
    a.stride_sb = a.groups > 1 ? o.stride_scales : 0;
}

#define MUON_RETURN_IF(e)                \
    do {                                 \
        const muon_status st_ = (e);     \
        if (st_ != MUON_OK) return st_;  \
    } while (0)

}  // namespace

extern "C" {

muon_status muon_int8_quantize(const muon_int8_quantize_config* c, void* stream) try {
    clear_error();
    const char* who = "muon_int8_quantize";
    if (!c) return fail(MUON_ERR_INVALID_ARG, who, "config is NULL");
    if (!is_dtype(c->src_dtype)) return fail(MUON_ERR_INVALID_ARG, who, "src_dtype must be F32 or BF16");
    if (c->batch < 0 || c->rows < 0 || c->cols < 1 || c->batch > MAX_I32 || c->rows > MAX_I32 || c->cols > MAX_I32 - 127 ||
        c->batch * c->rows > MAX_I32)
        return fail(MUON_ERR_SHAPE, who, "batch and rows must be at least 0, cols at least 1, batch * rows and cols + 127 below 2^31");
    if (c->ld < c->cols || c->ld > MAX_I32) return fail(MUON_ERR_SHAPE, who, "ld must be in [cols, 2^31)");
    if ((c->gather || c->limit) && c->batch > 1) return fail(MUON_ERR_INVALID_ARG, who, "gather and limit go with one matrix");
    if (c->gather && (c->per < 1 || c->src_rows < 0))
        return fail(MUON_ERR_INVALID_ARG, who, "per must be at least 1 and src_rows at least 0");
    if (c->batch > 1 && (double)c->batch_stride < (double)(c->rows - 1) * (double)c->ld + (double)c->cols)
        return fail(MUON_ERR_SHAPE, who, "batch_stride must hold one matrix");
    if (c->batch == 0 || c->rows == 0) return MUON_OK;
    const int64_t src_rows = c->gather ? c->src_rows : c->rows;
    if ((!c->src && src_rows > 0) || !c->codes || !c->scales) return fail(MUON_ERR_INVALID_ARG, who, "src, codes and scales must be non-NULL");
    if (misaligned(c->src) || misaligned(c->gather) || misaligned(c->codes) || misaligned(c->scales) || ((uintptr_t)c->limit & 3u) != 0)
        return fail(MUON_ERR_ALIGNMENT, who, "buffers must be 16-byte aligned (limit 4-byte)");
    Int8QuantizeArgs a{};
    a.kp = round_up(c->cols, 128);
    const double n = (double)c->batch * (double)c->rows;
    const Extent in[] = {extent(c->src, c->batch, c->batch_stride, src_rows, c->ld, c->cols, size_of(c->src_dtype)),
                         extent(c->gather, 4.0 * (double)c->rows), extent(c->limit, 4.0)};
    const Extent out[] = {extent(c->codes, n * (double)a.kp), extent(c->scales, 4.0 * n)};
    if (collide(out, in)) return fail(MUON_ERR_INVALID_ARG, who, "an output overlaps an input or another output");
    a.src = c->src;
    a.gather = c->gather;
    a.limit = c->limit;
    a.codes = c->codes;
    a.scales = c->scales;
    a.rows = c->rows;
    a.cols = c->cols;
    a.ld = c->ld;
    a.batch_stride = c->batch > 1 ? c->batch_stride : 0;
    a.src_rows = src_rows;
    a.total = c->batch * c->rows;
    a.per = c->gather ? c->per : 1;
    return launched(launch_int8_quantize(a, c->src_dtype, static_cast<hipStream_t>(stream)), who);
} catch (...) {
    return MUON_ERR_INVALID_ARG;
}

muon_status muon_int8_product(const muon_int8_product_config* c, void* stream) try {
    clear_error();
    const char* who = "muon_int8_product";
    if (!c) return fail(MUON_ERR_INVALID_ARG, who, "config is NULL");
    if (!is_dtype(c->out_dtype)) return fail(MUON_ERR_INVALID_ARG, who, "out_dtype must be F32 or BF16");
    MUON_RETURN_IF(check_product(c->mode, c->groups, c->m, c->n, c->k, MAX_INT8_DEPTH, c->offsets, who));
    if (c->ld_out < c->n || c->ld_out > MAX_I32) return fail(MUON_ERR_SHAPE, who, "ld_out must be at least n and below 2^31");
    if (c->m == 0 || c->n == 0) return MUON_OK;
    MUON_RETURN_IF(check_rows(c->out, c->ld_out, c->n, who, "out"));
    MUON_RETURN_IF(check_operand(c->a, MUON_OPERANDS_INT8, c->m, c->k, 1, who, "a"));
    MUON_RETURN_IF(check_operand(c->b, MUON_OPERANDS_INT8, c->n, c->k, c->groups, who, "b"));
    LayerArgs a = layer_args(c->mode, c->groups, c->offsets, c->m, c->n, c->k);
    set_a(a, 0, c->a.data, c->a.scales, c->a.ld, 1);
    set_b(a, 0, c->b, 1);
    a.out[0] = c->out;
    a.ld_out[0] = c->ld_out;
    a.vec = c->ld_out * size_of(c->out_dtype) % 16 == 0;
    if (!layer_fits(a, FORM_SCALED)) return fail(MUON_ERR_SHAPE, who, "2^31 or more output tiles");
    const Extent out[] = {extent(c->out, 1, 0, c->m, c->ld_out, c->n, size_of(c->out_dtype))};
    const Extent in[] = {values_of(c->a, MUON_OPERANDS_INT8, c->m, c->k, 1), scales_of(c->a, c->m, 1),
                         values_of(c->b, MUON_OPERANDS_INT8, c->n, c->k, c->groups), scales_of(c->b, c->n, c->groups),
                         extent(a.offsets, 4.0 * (double)(c->groups + 1))};
    if (collide(out, in)) return fail(MUON_ERR_INVALID_ARG, who, "out overlaps an operand or offsets");
    return launched(launch_layer(a, FORM_SCALED, MUON_OPERANDS_INT8, c->out_dtype, static_cast<hipStream_t>(stream)), who);
} catch (...) {
    return MUON_ERR_INVALID_ARG;
}

muon_status muon_gated(const muon_gated_config* c, void* stream) try {
    clear_error();
    const char* who = "muon_gated";
    if (!c) return fail(MUON_ERR_INVALID_ARG, who, "config is NULL");
    if (c->operands != MUON_OPERANDS_BF16 && c->operands != MUON_OPERANDS_INT8) return fail(MUON_ERR_INVALID_ARG, who, "unknown operands");
    if (c->activation < MUON_ACT_SILU || c->activation > MUON_ACT_RELU) return fail(MUON_ERR_INVALID_ARG, who, "unknown activation");
    const bool i8 = c->operands == MUON_OPERANDS_INT8;
    MUON_RETURN_IF(check_product(c->mode, c->groups, c->m, c->n, c->k, i8 ? MAX_INT8_DEPTH : MAX_I32 - 127, c->offsets, who));
    if (!c->pre_gate != !c->pre_up) return fail(MUON_ERR_INVALID_ARG, who, "pre_gate and pre_up go together");
    if (c->m == 0 || c->n == 0) return MUON_OK;
    MUON_RETURN_IF(check_rows(c->out, c->ld_out, c->n, who, "out"));
    if (c->pre_gate) {
        MUON_RETURN_IF(check_rows(c->pre_gate, c->ld_pre, c->n, who, "pre_gate"));
        MUON_RETURN_IF(check_rows(c->pre_up, c->ld_pre, c->n, who, "pre_up"));
    }
    MUON_RETURN_IF(check_operand(c->x, c->operands, c->m, c->k, 1, who, "x"));
    MUON_RETURN_IF(check_operand(c->gate, c->operands, c->n, c->k, c->groups, who, "gate"));
    MUON_RETURN_IF(check_operand(c->up, c->operands, c->n, c->k, c->groups, who, "up"));
    MUON_RETURN_IF(check_alike(c->gate, c->up, c->operands, c->k, c->groups, who));
    const int64_t size = i8 ? 1 : 2;
    LayerArgs a = layer_args(c->mode, c->groups, c->offsets, c->m, c->n, c->k);
    set_a(a, 0, c->x.data, c->x.scales, c->x.ld, size);
    set_b(a, 0, c->gate, size);
    set_b(a, 1, c->up, size);
    a.out[0] = c->out;
    a.out[1] = c->pre_gate;
    a.out[2] = c->pre_up;
    a.ld_out[0] = c->ld_out;
    a.ld_out[1] = c->ld_pre;
    a.vec = c->ld_out % 8 == 0 && (!c->pre_gate || c->ld_pre % 8 == 0);
    a.activation = c->activation;
    if (!layer_fits(a, FORM_GATED)) return fail(MUON_ERR_SHAPE, who, "2^31 or more output tiles");
    const Extent out[] = {extent(c->out, 1, 0, c->m, c->ld_out, c->n, 2), extent(c->pre_gate, 1, 0, c->m, c->ld_pre, c->n, 2),
                          extent(c->pre_up, 1, 0, c->m, c->ld_pre, c->n, 2)};
    const Extent in[] = {values_of(c->x, c->operands, c->m, c->k, 1), scales_of(c->x, c->m, 1),
                         values_of(c->gate, c->operands, c->n, c->k, c->groups), scales_of(c->gate, c->n, c->groups),
                         values_of(c->up, c->operands, c->n, c->k, c->groups), scales_of(c->up, c->n, c->groups),
                         extent(a.offsets, 4.0 * (double)(c->groups + 1))};
    if (collide(out, in)) return fail(MUON_ERR_INVALID_ARG, who, "an output overlaps an input or another output");
    return launched(launch_layer(a, FORM_GATED, c->operands, MUON_DTYPE_BF16, static_cast<hipStream_t>(stream)), who);
} catch (...) {
    return MUON_ERR_INVALID_ARG;
}

muon_status muon_gated_backward(const muon_gated_backward_config* c, void* stream) try {
    clear_error();
    const char* who = "muon_gated_backward";
    const int32_t bf16 = MUON_OPERANDS_BF16;
    if (!c) return fail(MUON_ERR_INVALID_ARG, who, "config is NULL");
    if (c->activation < MUON_ACT_SILU || c->activation > MUON_ACT_RELU) return fail(MUON_ERR_INVALID_ARG, who, "unknown activation");
    MUON_RETURN_IF(check_product(c->mode, c->groups, c->m, c->n, c->k, MAX_I32 - 127, c->offsets, who));
    if (!c->grad_gate != !c->grad_up) return fail(MUON_ERR_INVALID_ARG, who, "grad_gate and grad_up go together");
    if (!is_dtype(c->grad_dtype)) return fail(MUON_ERR_INVALID_ARG, who, "grad_dtype must be F32 or BF16");
    if (c->accumulate != 0 && (c->accumulate != 1 || c->grad_dtype != MUON_DTYPE_F32))
        return fail(MUON_ERR_INVALID_ARG, who, "accumulate must be 0 or, for float32 gradients, 1");
    if (c->n == 0) {
        if (c->grad_x && c->m > 0 && c->k > 0) return fail(MUON_ERR_SHAPE, who, "n must be at least 1 for grad_x, which would be zeros");
        return MUON_OK;
    }
    const bool weights = c->grad_gate && c->k > 0, to_x = c->grad_x && c->m > 0 && c->k > 0, rows = c->mode == MUON_PRODUCT_ROWS;
    if (weights) {
        MUON_RETURN_IF(check_rows(c->grad_gate, c->ld_grad_w, c->k, who, "grad_gate"));
        MUON_RETURN_IF(check_rows(c->grad_up, c->ld_grad_w, c->k, who, "grad_up"));
        if (c->groups > 1 && (double)c->stride_grad_w < (double)(c->n - 1) * (double)c->ld_grad_w + (double)c->k)
            return fail(MUON_ERR_SHAPE, who, "stride_grad_w must hold one group");
        // without rows the gradients are still written (zeros)
        if (rows && !c->offsets) return fail(MUON_ERR_INVALID_ARG, who, "offsets is NULL");
    }
    if (c->m > 0) {
        MUON_RETURN_IF(check_rows(c->grad, c->ld_grad, c->n, who, "grad"));
        MUON_RETURN_IF(check_rows(c->pre_gate, c->ld_pre, c->n, who, "pre_gate"));
        MUON_RETURN_IF(check_rows(c->pre_up, c->ld_pre, c->n, who, "pre_up"));
        MUON_RETURN_IF(check_rows(c->grad_pre_gate, c->ld_grad_pre, c->n, who, "grad_pre_gate"));
        MUON_RETURN_IF(check_rows(c->grad_pre_up, c->ld_grad_pre, c->n, who, "grad_pre_up"));
        if (c->ld_grad_pre % 64 != 0 || c->ld_grad_pre >= MAX_LD_BYTES / 2)
            return fail(MUON_ERR_SHAPE, who, "ld_grad_pre must be a multiple of 64 and below 2^22");
        if (weights) MUON_RETURN_IF(check_operand(c->x, bf16, c->m, c->k, 1, who, "x"));
    }
    if (to_x) {
        MUON_RETURN_IF(check_rows(c->grad_x, c->ld_grad_x, c->k, who, "grad_x"));
        MUON_RETURN_IF(check_operand(c->gate, bf16, c->n, c->k, c->groups, who, "gate"));
        MUON_RETURN_IF(check_operand(c->up, bf16, c->n, c->k, c->groups, who, "up"));
        MUON_RETURN_IF(check_alike(c->gate, c->up, bf16, c->k, c->groups, who));
    }
    LayerArgs x = layer_args(c->mode, c->groups, c->offsets, c->m, c->k, c->n);
    set_a(x, 0, c->grad_pre_gate, nullptr, c->ld_grad_pre, 2);
    set_a(x, 1, c->grad_pre_up, nullptr, c->ld_grad_pre, 2);
    set_b(x, 0, c->gate, 2);
    set_b(x, 1, c->up, 2);
    x.out[0] = c->grad_x;
    x.ld_out[0] = c->ld_grad_x;
    x.vec = c->ld_grad_x % 8 == 0;
    LayerArgs w = layer_args(rows ? MUON_PRODUCT_DEPTH : MUON_PRODUCT_DENSE, c->groups, c->offsets, c->n, c->k, c->m);
    set_a(w, 0, c->grad_pre_gate, nullptr, c->ld_grad_pre, 2);
    set_a(w, 1, c->grad_pre_up, nullptr, c->ld_grad_pre, 2);
    set_b(w, 0, c->x, 2);
    w.stride_b = 0;
    w.out[0] = c->grad_gate;
    w.out[1] = c->grad_up;
    w.ld_out[0] = c->ld_grad_w;
    w.out_stride = c->groups > 1 ? c->stride_grad_w : 0;
    w.vec = c->ld_grad_w * size_of(c->grad_dtype) % 16 == 0 && w.out_stride * size_of(c->grad_dtype) % 16 == 0;
    w.accumulate = c->accumulate;
    if ((to_x && !layer_fits(x, FORM_GRAD_X)) || (weights && !layer_fits(w, FORM_GRAD_W)))
        return fail(MUON_ERR_SHAPE, who, "2^31 or more output tiles");
    const bool in_place = c->grad_pre_gate == c->pre_gate && c->grad_pre_up == c->pre_up && c->ld_grad_pre == c->ld_pre;
    const int64_t size = size_of(c->grad_dtype);
    const Extent out[] = {extent(c->m > 0 ? c->grad_pre_gate : nullptr, 1, 0, c->m, c->ld_grad_pre, round_up(c->n, 64), 2),
                          extent(c->m > 0 ? c->grad_pre_up : nullptr, 1, 0, c->m, c->ld_grad_pre, round_up(c->n, 64), 2),
                          extent(to_x ? c->grad_x : nullptr, 1, 0, c->m, c->ld_grad_x, c->k, 2),
                          extent(weights ? c->grad_gate : nullptr, c->groups, c->stride_grad_w, c->n, c->ld_grad_w, c->k, size),
                          extent(weights ? c->grad_up : nullptr, c->groups, c->stride_grad_w, c->n, c->ld_grad_w, c->k, size)};
    const Extent in[] = {extent(c->grad, 1, 0, c->m, c->ld_grad, c->n, 2),
                         extent(in_place ? nullptr : c->pre_gate, 1, 0, c->m, c->ld_pre, c->n, 2),
                         extent(in_place ? nullptr : c->pre_up, 1, 0, c->m, c->ld_pre, c->n, 2),
                         values_of(weights ? c->x : muon_operand{}, bf16, c->m, c->k, 1),
                         values_of(to_x ? c->gate : muon_operand{}, bf16, c->n, c->k, c->groups),
                         values_of(to_x ? c->up : muon_operand{}, bf16, c->n, c->k, c->groups),
                         extent(x.offsets, 4.0 * (double)(c->groups + 1))};
    if (collide(out, in)) return fail(MUON_ERR_INVALID_ARG, who, "an output overlaps an input or another output");
    GatedGradArgs g{};
    g.grad = c->grad;
    g.pre_gate = c->pre_gate;
    g.pre_up = c->pre_up;
    g.grad_pre_gate = c->grad_pre_gate;
    g.grad_pre_up = c->grad_pre_up;
    g.m = c->m;
    g.n = c->n;
    g.ld_grad = c->ld_grad;
    g.ld_pre = c->ld_pre;
    g.ld_out = c->ld_grad_pre;
    g.offsets = x.offsets;
    g.groups = c->groups;
    g.activation = c->activation;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    MUON_RETURN_IF(launched(launch_gated_grad(g, s), who));
    if (to_x) MUON_RETURN_IF(launched(launch_layer(x, FORM_GRAD_X, bf16, MUON_DTYPE_BF16, s), who));
    if (weights) MUON_RETURN_IF(launched(launch_layer(w, FORM_GRAD_W, bf16, c->grad_dtype, s), who));
    return MUON_OK;
} catch (...) {
    return MUON_ERR_INVALID_ARG;
}

muon_status muon_gather_rows(const muon_gather_rows_config* c, void* stream) try {
    clear_error();
    const char* who = "muon_gather_rows";
    if (!c) return fail(MUON_ERR_INVALID_ARG, who, "config is NULL");
    if (!is_dtype(c->dtype)) return fail(MUON_ERR_INVALID_ARG, who, "dtype must be F32 or BF16");
    if (c->per < 1) return fail(MUON_ERR_INVALID_ARG, who, "per must be at least 1");
    if (c->src_rows < 0 || c->src_rows > MAX_I32 || c->src_rows * c->per > MAX_I32 || c->n_rows < 0 || c->n_rows > (1 << 30) || c->cols < 1 || c->cols > MAX_I32)
        return fail(MUON_ERR_SHAPE, who, "src_rows * per must be below 2^31, n_rows at most 2^30, cols in [1, 2^31)");
    // buffers of 0 elements may be NULL: out and y without rows, position and grad_weights without choices
    const int64_t choices = c->src_rows * c->per, size = size_of(c->dtype);
    if (choices > 0 && (!c->position != !c->grad_weights || (c->n_rows > 0 && !c->y != !c->grad_weights)))
        return fail(MUON_ERR_INVALID_ARG, who, "y, position and grad_weights go together");
    if (c->n_rows > 0 && !c->out && !c->y) return fail(MUON_ERR_INVALID_ARG, who, "no output");
    const bool gathers = c->n_rows > 0 && c->out, grads = choices > 0 && c->grad_weights;
    if (!gathers && !grads) return MUON_OK;
    if (c->src_rows > 0) MUON_RETURN_IF(check_rows(c->src, c->ld, c->cols, who, "src"));
    if (c->n_rows > 0) {
        if (!c->rows) return fail(MUON_ERR_INVALID_ARG, who, "rows is NULL");
        if (c->out) MUON_RETURN_IF(check_rows(c->out, c->ld_out, c->cols, who, "out"));
        if (grads) MUON_RETURN_IF(check_rows(c->y, c->ld_y, c->cols, who, "y"));
    }
    if (misaligned(c->rows) || misaligned(c->weights) || misaligned(c->position) || misaligned(c->grad_weights) || ((uintptr_t)c->limit & 3u) != 0)
        return fail(MUON_ERR_ALIGNMENT, who, "buffers must be 16-byte aligned (limit 4-byte)");
    const Extent out[] = {extent(c->out, 1, 0, c->n_rows, c->ld_out, c->cols, size), extent(c->grad_weights, 4.0 * (double)choices)};
    const Extent in[] = {extent(c->src, 1, 0, c->src_rows, c->ld, c->cols, size), extent(c->rows, 4.0 * (double)c->n_rows),
                         extent(c->limit, 4.0), extent(c->weights, 4.0 * (double)choices), extent(c->position, 4.0 * (double)choices),
                         extent(c->y, 1, 0, c->n_rows, c->ld_y, c->cols, size)};
    if (collide(out, in)) return fail(MUON_ERR_INVALID_ARG, who, "an output overlaps an input or another output");
    GatherRowsArgs a{};
    a.src = c->src;
    a.rows = c->rows;
    a.limit = c->limit;
    a.out = gathers ? c->out : nullptr;
    a.weights = c->weights;
    a.y = grads ? c->y : nullptr;
    a.position = grads ? c->position : nullptr;
    a.grad_weights = grads ? c->grad_weights : nullptr;
    a.cols = c->cols;
    a.ld = c->ld;
    a.ld_out = c->ld_out;
    a.ld_y = c->ld_y;
    a.n_rows = c->n_rows;
    a.choices = choices;
    a.per = c->per;
    return launched(launch_gather_rows(a, c->dtype, static_cast<hipStream_t>(stream)), who);
} catch (...) {
    return MUON_ERR_INVALID_ARG;
}

muon_status muon_combine_rows(const muon_combine_rows_config* c, void* stream) try {
    clear_error();
    const char* who = "muon_combine_rows";
    if (!c) return fail(MUON_ERR_INVALID_ARG, who, "config is NULL");
    if (!is_dtype(c->dtype) || !is_dtype(c->out_dtype)) return fail(MUON_ERR_INVALID_ARG, who, "dtype and out_dtype must be F32 or BF16");
    if (c->top_k < 1 || c->top_k > MUON_MAX_TOP_K) return fail(MUON_ERR_SHAPE, who, "top_k must be in [1, 64]");
    if (c->tokens < 0 || c->tokens > MAX_I32 || c->tokens * c->top_k > MAX_I32 || c->n_rows < 0 || c->n_rows > MAX_I32 || c->cols < 1 || c->cols > MAX_I32)
        return fail(MUON_ERR_SHAPE, who, "tokens * top_k and n_rows must be below 2^31, cols in [1, 2^31)");
    if (c->tokens == 0) return MUON_OK;
    MUON_RETURN_IF(check_rows(c->out, c->ld_out, c->cols, who, "out"));
    if (c->n_rows > 0) MUON_RETURN_IF(check_rows(c->src, c->ld, c->cols, who, "src"));
    if (c->residual) MUON_RETURN_IF(check_rows(c->residual, c->ld_residual, c->cols, who, "residual"));
    if (!c->position) return fail(MUON_ERR_INVALID_ARG, who, "position is NULL");
    if (misaligned(c->position) || misaligned(c->weights)) return fail(MUON_ERR_ALIGNMENT, who, "buffers must be 16-byte aligned");
    const int64_t choices = c->tokens * c->top_k, size = size_of(c->out_dtype);
    const bool in_place = c->residual == c->out && c->ld_residual == c->ld_out;
    const Extent out[] = {extent(c->out, 1, 0, c->tokens, c->ld_out, c->cols, size)};
    const Extent in[] = {extent(c->src, 1, 0, c->n_rows, c->ld, c->cols, size_of(c->dtype)), extent(c->position, 4.0 * (double)choices),
                         extent(c->weights, 4.0 * (double)choices),
                         extent(in_place ? nullptr : c->residual, 1, 0, c->tokens, c->ld_residual, c->cols, size)};
    if (collide(out, in)) return fail(MUON_ERR_INVALID_ARG, who, "out overlaps an input (it may be residual)");
    CombineRowsArgs a{};
    a.src = c->src;
    a.position = c->position;
    a.weights = c->weights;
    a.residual = c->residual;
    a.out = c->out;
    a.n_rows = c->n_rows;
    a.cols = c->cols;
    a.ld = c->ld;
    a.ld_out = c->ld_out;
    a.ld_residual = c->ld_residual;
    a.tokens = c->tokens;
    a.top_k = c->top_k;
    return launched(launch_combine_rows(a, c->dtype, c->out_dtype, static_cast<hipStream_t>(stream)), who);
} catch (...) {
    return MUON_ERR_INVALID_ARG;
}

}  // extern "C"
