// Entry points of the routed-expert operators.  Arguments are checked here, on the host; a kernel
// is only launched with sizes and strides that keep it inside the buffers they describe.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <string>

#include "experts.h"
#include "plan_internal.h"

using namespace muon;

namespace {

constexpr int64_t MAX_I32 = 0x7fffffff;
constexpr int64_t MAX_LD = 1 << 23;       // of an operand of a product
// a launch holds fewer than 2^32 threads: up to 64 a token in workgroups of 256, 256 a tile
constexpr int64_t MAX_TOKENS = (1 << 26) - 4, MAX_QUANTIZE_TILES = 1 << 24;

muon_status fail(muon_status s, const char* who, const char* what) {
    return set_error(s, std::string(who) + ": " + what);
}

muon_status launched(hipError_t e, const char* who) {
    return e == hipSuccess ? MUON_OK : set_error(MUON_ERR_HIP, std::string(who) + ": " + hipGetErrorString(e));
}

bool misaligned(const void* p) { return ((uintptr_t)p & 15u) != 0; }

int64_t round_up(int64_t a, int64_t b) { return ceil_div(a, b) * b; }

// The bytes of a buffer from the first that a call may touch to the last.  Rows and matrices lie a stride apart and the last
// of them ends with its own columns: what follows belongs to someone else.
struct Extent {
    const void* p;
    double bytes;                         // (sizes are products that may pass 64 bits)
    uint64_t step = 0, width = 0;         // rows of `width` bytes, `step` bytes apart; 0: no gaps
};
Extent extent(const void* p, double bytes) { return {p, bytes}; }
// `count` matrices of `rows` x `cols` elements
Extent extent(const void* p, int64_t count, int64_t stride, int64_t rows, int64_t ld, int64_t cols, int64_t size = 1) {
    if (count < 1 || rows < 1) return {p, 0};
    Extent e{p, ((double)(count - 1) * (double)stride + (double)(rows - 1) * (double)ld + (double)cols) * (double)size};
    if (ld > cols && (count == 1 || stride % ld == 0)) {
        e.step = (uint64_t)(ld * size);
        e.width = (uint64_t)(cols * size);
    }
    return e;
}
bool overlap(const Extent& a, const Extent& b) {
    const double x = (double)(uintptr_t)a.p, y = (double)(uintptr_t)b.p;
    if (!(a.p && b.p && a.bytes > 0 && b.bytes > 0 && x < y + b.bytes && y < x + a.bytes)) return false;
    if (a.step == 0 || a.step != b.step) return true;
    // b's rows in the gaps between a's: two column ranges of one matrix
    const uint64_t d = ((uintptr_t)b.p % a.step + a.step - (uintptr_t)a.p % a.step) % a.step;
    return d < a.width || d + b.width > a.step;
}

// Whether an output overlaps an input or another output.
template <int N, int M>
bool collide(const Extent (&out)[N], const Extent (&in)[M]) {
    for (int i = 0; i < N; ++i) {
        for (const Extent& e : in)
            if (overlap(out[i], e)) return true;
        for (int j = 0; j < i; ++j)
            if (overlap(out[i], out[j])) return true;
    }
    return false;
}

bool is_dtype(int32_t d) { return d == MUON_DTYPE_F32 || d == MUON_DTYPE_BF16; }

muon_status check_route(const muon_route_config* c, const char* who) {
    if (!c) return fail(MUON_ERR_INVALID_ARG, who, "config is NULL");
    if (c->n_experts < 1 || c->n_experts > MUON_MAX_EXPERTS)
        return fail(MUON_ERR_SHAPE, who, "n_experts must be in [1, 1024]");
    if (c->top_k < 1 || c->top_k > c->n_experts || c->top_k > MUON_MAX_TOP_K)
        return fail(MUON_ERR_SHAPE, who, "top_k must be in [1, min(n_experts, 64)]");
    if (c->tokens < 0 || c->tokens > MAX_TOKENS || c->tokens * c->top_k > MAX_I32)
        return fail(MUON_ERR_SHAPE, who, "tokens must be in [0, 2^26 - 4] and tokens * top_k below 2^31");
    if (c->ld < c->n_experts || c->ld > MAX_I32) return fail(MUON_ERR_SHAPE, who, "ld must be in [n_experts, 2^31)");
    if (!is_dtype(c->dtype)) return fail(MUON_ERR_INVALID_ARG, who, "dtype must be F32 or BF16");
    if (c->score != MUON_SCORE_SOFTMAX && c->score != MUON_SCORE_SIGMOID)
        return fail(MUON_ERR_INVALID_ARG, who, "unknown score");
    if (c->n_groups < 1 || c->n_groups > 64 || c->n_experts % c->n_groups != 0)
        return fail(MUON_ERR_INVALID_ARG, who, "n_groups must divide n_experts and be at most 64");
    if (c->top_groups < 1 || c->top_groups > c->n_groups)
        return fail(MUON_ERR_INVALID_ARG, who, "top_groups must be in [1, n_groups]");
    if (c->renormalize != 0 && c->renormalize != 1)
        return fail(MUON_ERR_INVALID_ARG, who, "renormalize must be 0 or 1");
    if (!std::isfinite(c->scale)) return fail(MUON_ERR_INVALID_ARG, who, "scale must be finite");
    return MUON_OK;
}

Extent logits_of(const muon_route_config& c, const void* p, int64_t ld) {
    return extent(p, 1, 0, c.tokens, ld, c.n_experts, c.dtype == MUON_DTYPE_F32 ? 4 : 2);
}
Extent choices_of(const muon_route_config& c, const void* p) { return extent(p, 4.0 * (double)c.tokens * (double)c.top_k); }

muon_status check_group(int64_t n, int32_t n_experts, int32_t align, const char* who) {
    if (n_experts < 1 || n_experts > MUON_MAX_EXPERTS)
        return fail(MUON_ERR_SHAPE, who, "n_experts must be in [1, 1024]");
    if (align < 1 || align > 128 || (align & (align - 1)) != 0)
        return fail(MUON_ERR_INVALID_ARG, who, "align must be 1, 2, 4, ..., 128");
    // the capacity, n + n_experts * 127 rounded up to 128 at most, is an int32 (as a difference: no sum that could overflow)
    if (n < 0 || n > MAX_I32 - 127 - (int64_t)n_experts * 128)
        return fail(MUON_ERR_SHAPE, who, "n must be at least 0 and the padded rows below 2^31");
    return MUON_OK;
}

int64_t group_capacity(int64_t n, int32_t n_experts, int32_t align) {
    return round_up(n + std::min<int64_t>(n, n_experts) * (align - 1), align);
}

int64_t group_chunks(int64_t n) { return n <= GROUP_SINGLE_MAX ? 0 : ceil_div(n, GROUP_CHUNK); }

// One operand of a product: `rows` matrix rows (per group) of k codes.
muon_status check_operand(const muon_fp8_operand& o, int64_t rows, int64_t k, int64_t groups, const char* who) {
    if (!o.codes || !o.scales) return fail(MUON_ERR_INVALID_ARG, who, "codes and scales must be non-NULL");
    if (o.square != 0 && o.square != 1) return fail(MUON_ERR_INVALID_ARG, who, "square must be 0 or 1");
    if (misaligned(o.codes) || misaligned(o.scales))
        return fail(MUON_ERR_ALIGNMENT, who, "codes and scales must be 16-byte aligned");
    // a tile's 256 rows lie within 2^31 bytes of its first
    if (o.ld % 16 != 0 || o.ld < round_up(k, 128) || o.ld >= MAX_LD)
        return fail(MUON_ERR_SHAPE, who, "ld must be a multiple of 16, at least round_up(k, 128) and below 2^23");
    if (o.ld_scales % 4 != 0 || o.ld_scales < round_up(ceil_div(k, 128), 4) || o.ld_scales >= MAX_LD)
        return fail(MUON_ERR_SHAPE, who,
                    "ld_scales must be a multiple of 4, at least round_up(ceil(k / 128), 4) and below 2^23");
    if (groups > 1) {
        const int64_t srows = o.square ? ceil_div(rows, 128) : rows;
        if (o.stride % 16 != 0 || o.stride_scales % 4 != 0 || o.stride < 0 || o.stride_scales < 0 ||
            (double)o.stride < (double)(rows - 1) * (double)o.ld + (double)round_up(k, 128) ||
            (double)o.stride_scales < (double)(srows - 1) * (double)o.ld_scales + (double)ceil_div(k, 128))
            return fail(MUON_ERR_SHAPE, who, "b's group strides must be multiples of 16 and 4 and hold one group");
    }
    return MUON_OK;
}

Extent codes_of(const muon_fp8_operand& o, int64_t rows, int64_t k, int64_t groups) {
    return extent(o.codes, groups, o.stride, rows, o.ld, round_up(k, 128));
}
Extent scales_of(const muon_fp8_operand& o, int64_t rows, int64_t k, int64_t groups) {
    return extent(o.scales, groups, o.stride_scales, o.square ? ceil_div(rows, 128) : rows, o.ld_scales,
                  round_up(ceil_div(k, 128), 4));
}

}  // namespace

extern "C" {

muon_status muon_route(const muon_route_config* c, const void* logits, const float* bias, int32_t* experts,
                       float* weights, void* stream) try {
    clear_error();
    const char* who = "muon_route";
    const muon_status st = check_route(c, who);
    if (st != MUON_OK) return st;
    if (c->tokens == 0) return MUON_OK;
    if (!logits || !experts || !weights) return fail(MUON_ERR_INVALID_ARG, who, "NULL buffer");
    if (misaligned(logits) || misaligned(bias) || misaligned(experts) || misaligned(weights))
        return fail(MUON_ERR_ALIGNMENT, who, "buffers must be 16-byte aligned");
    const Extent out[] = {choices_of(*c, experts), choices_of(*c, weights)};
    const Extent in[] = {logits_of(*c, logits, c->ld), extent(bias, 4.0 * (double)c->n_experts)};
    if (collide(out, in)) return fail(MUON_ERR_INVALID_ARG, who, "an output overlaps an input or another output");
    RouteArgs a{};
    a.logits = logits;
    a.bias = bias;
    a.experts = experts;
    a.weights = weights;
    a.tokens = c->tokens;
    a.ld = c->ld;
    a.n_experts = c->n_experts;
    a.top_k = c->top_k;
    a.n_groups = c->n_groups;
    a.top_groups = c->top_groups;
    a.score = c->score;
    a.renormalize = c->renormalize;
    a.scale = c->scale;
    return launched(launch_route(a, c->dtype, static_cast<hipStream_t>(stream)), who);
} catch (...) {
    return MUON_ERR_INVALID_ARG;
}

muon_status muon_route_backward(const muon_route_config* c, const void* logits, const int32_t* experts,
                                const float* grad_weights, void* grad_logits, int64_t ld_grad, void* stream) try {
    clear_error();
    const char* who = "muon_route_backward";
    const muon_status st = check_route(c, who);
    if (st != MUON_OK) return st;
    if (ld_grad < c->n_experts || ld_grad > MAX_I32)
        return fail(MUON_ERR_SHAPE, who, "ld_grad must be in [n_experts, 2^31)");
    if (c->tokens == 0) return MUON_OK;
    if (!logits || !experts || !grad_weights || !grad_logits) return fail(MUON_ERR_INVALID_ARG, who, "NULL buffer");
    if (misaligned(logits) || misaligned(experts) || misaligned(grad_weights) || misaligned(grad_logits))
        return fail(MUON_ERR_ALIGNMENT, who, "buffers must be 16-byte aligned");
    const bool in_place = grad_logits == logits && ld_grad == c->ld;
    const Extent out[] = {logits_of(*c, grad_logits, ld_grad)};
    const Extent in[] = {choices_of(*c, experts), choices_of(*c, grad_weights), logits_of(*c, in_place ? nullptr : logits, c->ld)};
    if (collide(out, in))
        return fail(MUON_ERR_INVALID_ARG, who, "grad_logits overlaps an input (it may be logits, with the same ld)");
    RouteBackwardArgs a{};
    a.logits = logits;
    a.experts = experts;
    a.grad_weights = grad_weights;
    a.grad_logits = grad_logits;
    a.tokens = c->tokens;
    a.ld = c->ld;
    a.ld_grad = ld_grad;
    a.n_experts = c->n_experts;
    a.top_k = c->top_k;
    a.score = c->score;
    a.renormalize = c->renormalize;
    a.scale = c->scale;
    return launched(launch_route_backward(a, c->dtype, static_cast<hipStream_t>(stream)), who);
} catch (...) {
    return MUON_ERR_INVALID_ARG;
}

muon_status muon_group_rows_workspace(int64_t n, int32_t n_experts, uint64_t* bytes) try {
    clear_error();
    const char* who = "muon_group_rows_workspace";
    const muon_status st = check_group(n, n_experts, 1, who);
    if (st != MUON_OK) return st;
    if (!bytes) return fail(MUON_ERR_INVALID_ARG, who, "NULL bytes");
    *bytes = (uint64_t)group_chunks(n) * (uint64_t)n_experts * sizeof(int32_t);
    return MUON_OK;
} catch (...) {
    return MUON_ERR_INVALID_ARG;
}

muon_status muon_group_rows_capacity(int64_t n, int32_t n_experts, int32_t align, int64_t* rows) try {
    clear_error();
    const char* who = "muon_group_rows_capacity";
    const muon_status st = check_group(n, n_experts, align, who);
    if (st != MUON_OK) return st;
    if (!rows) return fail(MUON_ERR_INVALID_ARG, who, "NULL rows");
    *rows = group_capacity(n, n_experts, align);
    return MUON_OK;
} catch (...) {
    return MUON_ERR_INVALID_ARG;
}

muon_status muon_group_rows(const int32_t* experts, int64_t n, int32_t n_experts, int32_t align, int32_t* counts,
                            int32_t* offsets, int32_t* rows, int32_t* position, void* workspace,
                            uint64_t workspace_bytes, void* stream) try {
    clear_error();
    const char* who = "muon_group_rows";
    const muon_status st = check_group(n, n_experts, align, who);
    if (st != MUON_OK) return st;
    GroupRowsArgs a{};
    a.n = n;
    a.capacity = group_capacity(n, n_experts, align);
    a.chunks = group_chunks(n);
    // without choices counts and offsets are still written (zeros)
    if (!counts || !offsets || (n > 0 && (!experts || !rows || !position)))
        return fail(MUON_ERR_INVALID_ARG, who, "NULL buffer");
    if (misaligned(experts) || misaligned(counts) || misaligned(offsets) || misaligned(rows) || misaligned(position) ||
        misaligned(workspace))
        return fail(MUON_ERR_ALIGNMENT, who, "buffers must be 16-byte aligned");
    const uint64_t need = (uint64_t)a.chunks * (uint64_t)n_experts * sizeof(int32_t);
    if (need > 0 && !workspace) return fail(MUON_ERR_INVALID_ARG, who, "workspace is NULL");
    if (workspace_bytes < need)
        return fail(MUON_ERR_WORKSPACE_TOO_SMALL, who, "workspace below muon_group_rows_workspace()");
    const Extent out[] = {extent(counts, 4.0 * n_experts), extent(offsets, 4.0 * (n_experts + 1)),
                          extent(rows, 4.0 * (double)a.capacity), extent(position, 4.0 * (double)n),
                          extent(workspace, (double)need)};
    const Extent in[] = {extent(experts, 4.0 * (double)n)};
    if (collide(out, in)) return fail(MUON_ERR_INVALID_ARG, who, "an output overlaps an input or another output");
    a.experts = experts;
    a.counts = counts;
    a.offsets = offsets;
    a.rows = rows;
    a.position = position;
    a.partial = static_cast<int32_t*>(workspace);
    a.n_experts = n_experts;
    a.align = align;
    return launched(launch_group_rows(a, static_cast<hipStream_t>(stream)), who);
} catch (...) {
    return MUON_ERR_INVALID_ARG;
}

muon_status muon_balance_step(const float* bias, const int32_t* counts, int32_t n_experts, float rate,
                              float* bias_out, void* stream) try {
    clear_error();
    const char* who = "muon_balance_step";
    if (n_experts < 1 || n_experts > MUON_MAX_EXPERTS)
        return fail(MUON_ERR_SHAPE, who, "n_experts must be in [1, 1024]");
    if (!bias || !counts || !bias_out) return fail(MUON_ERR_INVALID_ARG, who, "NULL buffer");
    if (!std::isfinite(rate)) return fail(MUON_ERR_INVALID_ARG, who, "rate must be finite");
    if (misaligned(bias) || misaligned(counts) || misaligned(bias_out))
        return fail(MUON_ERR_ALIGNMENT, who, "buffers must be 16-byte aligned");
    const Extent out[] = {extent(bias_out, 4.0 * n_experts)};
    const Extent in[] = {extent(counts, 4.0 * n_experts), extent(bias_out == bias ? nullptr : bias, 4.0 * n_experts)};
    if (collide(out, in)) return fail(MUON_ERR_INVALID_ARG, who, "bias_out overlaps an input (it may be bias)");
    return launched(launch_balance(bias, counts, n_experts, rate, bias_out, static_cast<hipStream_t>(stream)), who);
} catch (...) {
    return MUON_ERR_INVALID_ARG;
}

muon_status muon_fp8_quantize(const muon_fp8_quantize_config* c, void* stream) try {
    clear_error();
    const char* who = "muon_fp8_quantize";
    if (!c) return fail(MUON_ERR_INVALID_ARG, who, "config is NULL");
    if (!is_dtype(c->src_dtype)) return fail(MUON_ERR_INVALID_ARG, who, "src_dtype must be F32 or BF16");
    if (c->format != MUON_FP8_E4M3 && c->format != MUON_FP8_E5M2)
        return fail(MUON_ERR_INVALID_ARG, who, "unknown format");
    if (c->square != 0 && c->square != 1) return fail(MUON_ERR_INVALID_ARG, who, "square must be 0 or 1");
    if (c->batch < 0 || c->rows < 0 || c->cols < 1 || c->rows > MAX_I32 - 127 || c->cols > MAX_I32 - 127 || c->batch > MAX_I32)
        return fail(MUON_ERR_SHAPE, who, "batch and rows must be at least 0, cols at least 1, all below 2^31 - 127");
    if (c->ld < c->cols || c->ld > MAX_I32) return fail(MUON_ERR_SHAPE, who, "ld must be in [cols, 2^31)");
    if ((c->gather || c->limit) && c->batch > 1)
        return fail(MUON_ERR_INVALID_ARG, who, "gather and limit go with one matrix");
    if (c->limit && c->square) return fail(MUON_ERR_INVALID_ARG, who, "limit goes with row blocks");
    if (c->gather && (c->per < 1 || c->src_rows < 0))
        return fail(MUON_ERR_INVALID_ARG, who, "per must be at least 1 and src_rows at least 0");
    const int64_t src_rows = c->gather ? c->src_rows : c->rows;
    if (c->batch > 1 && (double)c->batch_stride < (double)(c->rows - 1) * (double)c->ld + (double)c->cols)
        return fail(MUON_ERR_SHAPE, who, "batch_stride must hold one matrix");
    QuantizeArgs a{};
    a.tiles_r = (int32_t)ceil_div(c->rows, 128);
    a.tiles_c = (int32_t)ceil_div(c->cols, 128);
    const double tiles = (double)c->batch * (double)a.tiles_r * (double)a.tiles_c;
    if (tiles >= (double)MAX_QUANTIZE_TILES) return fail(MUON_ERR_SHAPE, who, "2^24 or more tiles of 128 x 128");
    if (!c->codes && !c->codes_t) return fail(MUON_ERR_INVALID_ARG, who, "no output");
    if (!c->codes != !c->scales || !c->codes_t != !c->scales_t)
        return fail(MUON_ERR_INVALID_ARG, who, "codes and scales go together");
    if (tiles == 0) return MUON_OK;
    if (!c->src && src_rows > 0) return fail(MUON_ERR_INVALID_ARG, who, "src is NULL");
    if (misaligned(c->src) || misaligned(c->gather) || misaligned(c->codes) || misaligned(c->scales) ||
        misaligned(c->codes_t) || misaligned(c->scales_t) || ((uintptr_t)c->limit & 3u) != 0)
        return fail(MUON_ERR_ALIGNMENT, who, "buffers must be 16-byte aligned (limit 4-byte)");
    a.kp = round_up(c->cols, 128);
    a.sp = round_up(a.tiles_c, 4);
    a.kp_t = round_up(c->rows, 128);
    a.sp_t = round_up(a.tiles_r, 4);
    const Extent in[] = {extent(c->src, c->batch, c->batch_stride, src_rows, c->ld, c->cols,
                                c->src_dtype == MUON_DTYPE_F32 ? 4 : 2),
                         extent(c->gather, 4.0 * (double)c->rows), extent(c->limit, 4.0)};
    const double n = (double)c->batch;
    const Extent out[] = {extent(c->codes, n * (double)c->rows * (double)a.kp),
                          extent(c->scales, n * (double)(c->square ? a.tiles_r : c->rows) * (double)a.sp),
                          extent(c->codes_t, n * (double)c->cols * (double)a.kp_t),
                          extent(c->scales_t, n * (double)(c->square ? a.tiles_c : c->cols) * (double)a.sp_t)};
    if (collide(out, in)) return fail(MUON_ERR_INVALID_ARG, who, "an output overlaps an input or another output");
    a.src = c->src;
    a.gather = c->gather;
    a.limit = c->limit;
    a.codes = c->codes;
    a.scales = c->scales;
    a.codes_t = c->codes_t;
    a.scales_t = c->scales_t;
    a.rows = c->rows;
    a.cols = c->cols;
    a.ld = c->ld;
    a.batch_stride = c->batch > 1 ? c->batch_stride : 0;
    a.src_rows = src_rows;
    a.per = c->gather ? c->per : 1;
    a.tiles = c->batch * a.tiles_r * a.tiles_c;
    return launched(launch_quantize(a, c->src_dtype, c->format, c->square, static_cast<hipStream_t>(stream)), who);
} catch (...) {
    return MUON_ERR_INVALID_ARG;
}

muon_status muon_fp8_product(const muon_fp8_product_config* c, void* stream) try {
    clear_error();
    const char* who = "muon_fp8_product";
    if (!c) return fail(MUON_ERR_INVALID_ARG, who, "config is NULL");
    const bool full_sums = (c->mode & MUON_PRODUCT_FULL_SUMS) != 0;
    const int32_t mode = c->mode & ~MUON_PRODUCT_FULL_SUMS;
    if (mode != MUON_PRODUCT_DENSE && mode != MUON_PRODUCT_ROWS && mode != MUON_PRODUCT_DEPTH)
        return fail(MUON_ERR_INVALID_ARG, who, "unknown mode");
    const bool rows = mode == MUON_PRODUCT_ROWS, depth = mode == MUON_PRODUCT_DEPTH;
    if (c->groups < 1 || c->groups > MUON_MAX_EXPERTS || (mode == MUON_PRODUCT_DENSE && c->groups != 1))
        return fail(MUON_ERR_INVALID_ARG, who, "groups must be in [1, 1024], and 1 without groups");
    if (c->m < 0 || c->n < 0 || c->k < 0 || c->m > MAX_I32 || c->n > MAX_I32 || c->k > MAX_I32 - 127)
        return fail(MUON_ERR_SHAPE, who, "m, n and k must be at least 0 and below 2^31 - 127");
    if (c->a.format != MUON_FP8_E4M3 && c->a.format != MUON_FP8_E5M2)
        return fail(MUON_ERR_INVALID_ARG, who, "unknown format of a");
    if (c->b.format != MUON_FP8_E4M3) return fail(MUON_ERR_INVALID_ARG, who, "b must be e4m3");
    if (!is_dtype(c->out_dtype)) return fail(MUON_ERR_INVALID_ARG, who, "out_dtype must be F32 or BF16");
    if (c->accumulate != 0 && (c->accumulate != 1 || c->out_dtype != MUON_DTYPE_F32))
        return fail(MUON_ERR_INVALID_ARG, who, "accumulate must be 0 or, for a float32 out, 1");
    if (c->ld_out < c->n) return fail(MUON_ERR_SHAPE, who, "ld_out must be at least n");
    if (c->ld_out > MAX_I32) return fail(MUON_ERR_SHAPE, who, "ld_out must be below 2^31");
    if (depth && c->groups > 1 && (double)c->out_stride < (double)(c->m - 1) * (double)c->ld_out + (double)c->n)
        return fail(MUON_ERR_SHAPE, who, "out_stride must hold one group");
    if (c->m == 0 || c->n == 0) return MUON_OK;
    if (!c->out || (mode != MUON_PRODUCT_DENSE && !c->offsets))
        return fail(MUON_ERR_INVALID_ARG, who, "out and, with groups, offsets must be non-NULL");
    if (misaligned(c->out) || ((uintptr_t)c->offsets & 3u) != 0)
        return fail(MUON_ERR_ALIGNMENT, who, "out must be 16-byte aligned (offsets 4-byte)");
    if (c->k > 0) {
        muon_status st = check_operand(c->a, c->m, c->k, 1, who);
        if (st == MUON_OK) st = check_operand(c->b, c->n, c->k, rows ? c->groups : 1, who);
        if (st != MUON_OK) return st;
    }
    const int64_t size = c->out_dtype == MUON_DTYPE_F32 ? 4 : 2;
    ProductArgs a{};
    a.a = static_cast<const uint8_t*>(c->a.codes);
    a.as = static_cast<const uint8_t*>(c->a.scales);
    a.b = static_cast<const uint8_t*>(c->b.codes);
    a.bs = static_cast<const uint8_t*>(c->b.scales);
    a.lda = c->a.ld;
    a.ldas = c->a.ld_scales;
    a.ldb = c->b.ld;
    a.ldbs = c->b.ld_scales;
    a.stride_b = c->groups > 1 ? c->b.stride : 0;
    a.stride_bs = c->groups > 1 ? c->b.stride_scales : 0;
    a.shift_a = c->a.square ? 7 : 0;
    a.shift_b = c->b.square ? 7 : 0;
    a.offsets = c->offsets;
    a.out = c->out;
    a.ld_out = c->ld_out;
    a.out_stride = depth ? c->out_stride : 0;
    a.m = c->m;
    a.n = c->n;
    a.k = c->k;
    a.groups = c->groups;
    a.mode = mode;
    a.accumulate = c->accumulate;
    a.vec = c->ld_out * size % 16 == 0 && a.out_stride * size % 16 == 0;
    if (!product_fits(a)) return fail(MUON_ERR_SHAPE, who, "2^31 or more output tiles");
    const Extent out = extent(c->out, depth ? c->groups : 1, c->out_stride, c->m, c->ld_out, c->n, size);
    const int64_t b_groups = rows ? c->groups : 1;
    if (overlap(out, extent(c->offsets, 4.0 * (double)(c->groups + 1))) ||
        (c->k > 0 && (overlap(out, codes_of(c->a, c->m, c->k, 1)) || overlap(out, scales_of(c->a, c->m, c->k, 1)) ||
                      overlap(out, codes_of(c->b, c->n, c->k, b_groups)) || overlap(out, scales_of(c->b, c->n, c->k, b_groups)))))
        return fail(MUON_ERR_INVALID_ARG, who, "out overlaps an operand or offsets");
    return launched(launch_product(a, c->a.format, c->out_dtype, full_sums, static_cast<hipStream_t>(stream)), who);
} catch (...) {
    return MUON_ERR_INVALID_ARG;
}

}  // extern "C"
