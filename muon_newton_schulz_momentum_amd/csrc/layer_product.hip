// Products of the expert layers (gfx950 matrix cores): the gated block, 8-bit integer products, and the gated block's
// gradients (the forms of layers.h).
//
// An operand is a panel of rows with the depth along them (x and weights forwards, the pre-activations' gradients in
// FORM_GRAD_X) or, "across", of depth rows (weights in FORM_GRAD_X, both operands of FORM_GRAD_W, whose depth is the tokens).
// b's rows are the matrix instruction's first operand: a lane then holds runs of 4 consecutive columns of one row of out.
#include <type_traits>

#include "activation.h"
#include "device_common.h"
#include "layers.h"
#include "tile_walk.h"

namespace muon {
namespace {

using namespace tiles;

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x16 __attribute__((ext_vector_type(16)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef i32x4 i32x4_any __attribute__((aligned(1)));       // 16 bytes that may begin anywhere

// bfloat16 or 8-bit integer values: 16 bytes of a row are a lane's part of one instruction of either kind.
template <class E>
struct Cores;
template <>
struct Cores<uint16_t> {
    typedef f32x16 sums;
    static __device__ __forceinline__ sums mul(i32x4 b, i32x4 a, sums c) {
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, b), __builtin_bit_cast(bf16x8, a), c, 0, 0, 0);
    }
};
template <>
struct Cores<int8_t> {
    typedef i32x16 sums;
    static __device__ __forceinline__ sums mul(i32x4 b, i32x4 a, sums c) { return __builtin_amdgcn_mfma_i32_32x32x32_i8(b, a, c, 0, 0, 0); }
};

template <int FORM>
constexpr bool a_across = FORM == FORM_GRAD_W;
template <int FORM>
constexpr bool b_across = FORM == FORM_GRAD_X || FORM == FORM_GRAD_W;
template <int FORM>
constexpr int parts = FORM == FORM_GRAD_X ? 2 : 1;         // products that are added up
template <int FORM>
constexpr int pair = FORM == FORM_GRAD_W ? 2 : 1;          // products of a launch

__device__ __forceinline__ float gated_value(int activation, float g, float u) {
    return (activation == MUON_ACT_SILU   ? dev::activate<MUON_ACT_SILU>(g)
            : activation == MUON_ACT_GELU ? dev::activate<MUON_ACT_GELU>(g)
                                          : dev::activate<MUON_ACT_RELU>(g)) * u;
}

// ---- 128 x 128 tiles for any alignment ------------------------------------------------------
//
// 4 waves of 64 x 64; every 16 bytes of an operand are checked against its end, so rows may begin anywhere.
constexpr int ANY = 128, ANY_THREADS = 256;

// 16 bytes at byte `at` of a row of `end` bytes; zeros behind its end.
template <class E>
__device__ __forceinline__ i32x4 load_checked(const uint8_t* row, int64_t at, int64_t end) {
    if (at + 16 <= end) return *reinterpret_cast<const i32x4_any*>(row + at);
    i32x4 v = {0, 0, 0, 0};
#pragma unroll
    for (int e = 0; e < 16 / (int)sizeof(E); ++e) {
        const int64_t b = at + e * (int)sizeof(E);
        if (b < end) v[e * sizeof(E) / 4] |= (int)((uint32_t)(std::make_unsigned_t<E>)*reinterpret_cast<const E*>(row + b) << (8 * (e * sizeof(E) % 4)));
    }
    return v;
}

template <class E, int FORM, class OUT>
__global__ __launch_bounds__(ANY_THREADS) void layer_any_kernel(LayerArgs p) {
    constexpr bool GATED = FORM == FORM_GATED, I8 = sizeof(E) == 1;
    constexpr int STEP = 64, ROW = STEP + 16;              // bytes of a row in a step, and apart in LDS
    constexpr int COLS = GATED ? ANY / 2 : ANY;            // columns of out in a tile
    __shared__ __attribute__((aligned(16))) uint8_t smem[2][ANY * ROW];
    __shared__ int bounds[MUON_MAX_EXPERTS + 1], ends[MUON_MAX_EXPERTS + 1];
    __shared__ int64_t wave_tot[ANY_THREADS / 64];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave >> 1, wn = wave & 1, fr = lane & 31, fk = lane >> 5;
    if (p.mode != MUON_PRODUCT_DENSE) read_segments<1, ANY_THREADS>(p, ANY, bounds, ends, wave_tot);
    Walk my = walk<pair<FORM>>(p, ends);
    for (int t = next_tile(p, my); t >= 0; t = next_tile(p, my)) {
        const Tile x = decode<1, pair<FORM>>(p, t, ANY, COLS, bounds, ends);
        const int64_t group_b = p.mode == MUON_PRODUCT_ROWS ? x.group : 0;
        typename Cores<E>::sums acc[2][2] = {};
        for (int part = 0; part < parts<FORM>; ++part)
            for (int64_t k0 = x.kb0; k0 < x.kb1; k0 += STEP / (int)sizeof(E)) {
                // operand `op`: 128 rows of its panel
                auto stage = [&](int op, bool across) {
                    if (!across) {
                        const int r = tid >> 1;
                        const uint8_t* row = nullptr;
                        if (op == 0) {
                            if (r < x.rows_a) row = p.a[part] + (x.m0 + r) * p.lda;
                        } else {
                            const int w = GATED ? r / COLS : part, c = GATED ? r % COLS : r;
                            if (c < x.rows_b) row = p.b[w] + group_b * p.stride_b[w] + (x.n0 + c) * p.ldb[w];
                        }
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            const int at = 32 * (tid & 1) + 16 * c;
                            i32x4 v = {0, 0, 0, 0};
                            if (row) v = load_checked<E>(row, k0 * (int)sizeof(E) + at, (int64_t)x.kb1 * (int)sizeof(E));
                            *reinterpret_cast<i32x4*>(smem[op] + r * ROW + at) = v;
                        }
                    } else {
                        const int kk = tid >> 3, c0 = 16 * (tid & 7);
                        const int w = op == 0 ? x.which : part;
                        const uint8_t* row = op == 0 ? p.a[w] + (k0 + kk) * p.lda : p.b[w] + group_b * p.stride_b[w] + (k0 + kk) * p.ldb[w];
                        const int64_t first = (op == 0 ? x.m0 : x.n0) + c0, end = op == 0 ? p.m : p.n;
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            i32x4 v = {0, 0, 0, 0};
                            if (k0 + kk < x.kb1) v = load_checked<E>(row, 2 * (first + 8 * c), 2 * end);
#pragma unroll
                            for (int e = 0; e < 8; ++e)
                                *reinterpret_cast<uint16_t*>(smem[op] + (c0 + 8 * c + e) * ROW + 2 * kk) = (uint16_t)((uint32_t)v[e / 2] >> (16 * (e & 1)));
                        }
                    }
                };
                stage(0, a_across<FORM>);
                stage(1, b_across<FORM>);
                __syncthreads();
#pragma unroll
                for (int kk = 0; kk < 2; ++kk) {
                    i32x4 fa[2], fb[2];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        fa[i] = *reinterpret_cast<const i32x4*>(smem[0] + (64 * wm + 32 * i + fr) * ROW + 32 * kk + 16 * fk);
                        fb[i] = *reinterpret_cast<const i32x4*>(smem[1] + ((GATED ? 64 * i + 32 * wn : 64 * wn + 32 * i) + fr) * ROW + 32 * kk + 16 * fk);
                    }
#pragma unroll
                    for (int i = 0; i < 2; ++i)
#pragma unroll
                        for (int j = 0; j < 2; ++j) acc[i][j] = Cores<E>::mul(fb[j], fa[i], acc[i][j]);
                }
                __syncthreads();
            }
        // a lane's sums: row fr of a block, columns 8 q + 4 fk + (0 .. 3)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int r = 64 * wm + 32 * i + fr;
            if (r >= x.rows_a) continue;
            const float sa = I8 ? p.sa[x.m0 + r] : 1.f;
            auto column = [&](int w, int64_t c, float v) { return I8 ? v * sa * p.sb[w][group_b * p.stride_sb[w] + c] : v; };
#pragma unroll
            for (int v = 0; v < 16; ++v) {
                const int c = 8 * (v >> 2) + 4 * fk + (v & 3);
                if constexpr (GATED) {
                    if (32 * wn + c >= x.rows_b) continue;
                    const int64_t col = x.n0 + 32 * wn + c;
                    const float g = column(0, col, (float)acc[i][0][v]), u = column(1, col, (float)acc[i][1][v]);
                    static_cast<uint16_t*>(p.out[0])[(x.m0 + r) * p.ld_out[0] + col] = dev::f32_to_bf16(gated_value(p.activation, g, u));
                    if (p.out[1]) {
                        static_cast<uint16_t*>(p.out[1])[(x.m0 + r) * p.ld_out[1] + col] = dev::f32_to_bf16(g);
                        static_cast<uint16_t*>(p.out[2])[(x.m0 + r) * p.ld_out[2] + col] = dev::f32_to_bf16(u);
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        if (64 * wn + 32 * j + c >= x.rows_b) continue;
                        const int64_t col = x.n0 + 64 * wn + 32 * j + c;
                        const float s = column(0, col, (float)acc[i][j][v]);
                        OUT* o = static_cast<OUT*>(p.out[x.which]) + (p.mode == MUON_PRODUCT_DEPTH ? x.group * p.out_stride : 0) +
                                 (x.m0 + r) * p.ld_out[x.which] + col;
                        if constexpr (sizeof(OUT) == 4) *o = p.accumulate ? *o + s : s;
                        else *o = dev::f32_to_bf16(s);
                    }
                }
            }
        }
    }
}

template <class E, int FORM, class OUT>
hipError_t layer_as(LayerArgs a, hipStream_t s) {
    const int64_t total = count_tiles<pair<FORM>>(a, ANY, FORM == FORM_GATED ? ANY / 2 : ANY);
    if (total == 0) return hipSuccess;
    const dim3 grid((unsigned)std::min<int64_t>((total + NUM_XCD - 1) / NUM_XCD * NUM_XCD, 2 * CUS)), block(ANY_THREADS);
    hipLaunchKernelGGL((layer_any_kernel<E, FORM, OUT>), grid, block, 0, s, a);
    return hipGetLastError();
}

}  // namespace

bool layer_fits(LayerArgs a, LayerForm form) {
    return (form == FORM_GRAD_W ? count_tiles<2>(a, ANY, ANY) : count_tiles<1>(a, ANY, ANY / 2)) >= 0;
}

hipError_t launch_layer(LayerArgs a, LayerForm form, int32_t operands, int32_t out_dtype, hipStream_t s) {
    const bool f32 = out_dtype == MUON_DTYPE_F32;
    switch (form) {
        case FORM_GATED:
            return operands == MUON_OPERANDS_INT8 ? layer_as<int8_t, FORM_GATED, uint16_t>(a, s) : layer_as<uint16_t, FORM_GATED, uint16_t>(a, s);
        case FORM_SCALED: return f32 ? layer_as<int8_t, FORM_SCALED, float>(a, s) : layer_as<int8_t, FORM_SCALED, uint16_t>(a, s);
        case FORM_GRAD_X: return layer_as<uint16_t, FORM_GRAD_X, uint16_t>(a, s);
        default: return f32 ? layer_as<uint16_t, FORM_GRAD_W, float>(a, s) : layer_as<uint16_t, FORM_GRAD_W, uint16_t>(a, s);
    }
}

}  // namespace muon
