// Products of the expert layers (gfx950 matrix cores): the gated block, 8-bit integer products, and the gated block's
// gradients (the forms of layers.h).
//
// An operand is a panel of rows with the depth along them (x and weights forwards, the pre-activations' gradients in
// FORM_GRAD_X) or, "across", of depth rows (weights in FORM_GRAD_X, both operands of FORM_GRAD_W, whose depth is the tokens).
// b's rows are the matrix instruction's first operand: a lane then holds runs of 4 consecutive columns of one row of out.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "activation.h"
#include "device_common.h"
#include "layers.h"
#include "tile_walk.h"

namespace muon {
namespace {

using namespace tiles;

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
// 16 bytes that may begin anywhere
typedef i32x4 i32x4_any __attribute__((aligned(1)));
typedef f32x4 f32x4_any __attribute__((aligned(4)));
typedef uint32_t u32x2_any __attribute__((ext_vector_type(2), aligned(2)));

// bfloat16 or 8-bit integer values: 16 bytes of a row are a lane's part of one instruction of either kind, which multiplies 16
// rows by 16 over 64 bytes of depth.  The 32 x 32 forms are the slower ones here: with all CUs busy the card's power sets the clock,
// and on normal values those alone reach 1.72 PFLOP/s in bfloat16 and 3.32 in 8-bit integers, these 1.95 and 3.94.
template <class E>
struct Cores;
template <>
struct Cores<uint16_t> {
    typedef f32x4 sums;
    static __device__ __forceinline__ sums mul(i32x4 b, i32x4 a, sums c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, b), __builtin_bit_cast(bf16x8, a), c, 0, 0, 0);
    }
};
template <>
struct Cores<int8_t> {
    typedef i32x4 sums;
    static __device__ __forceinline__ sums mul(i32x4 b, i32x4 a, sums c) { return __builtin_amdgcn_mfma_i32_16x16x64_i8(b, a, c, 0, 0, 0); }
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

// ---- gradients with fewer than 8 features or columns ----------------------------------------------
//
// 128 x 128 tiles, 4 waves of 64 x 64, one step at a time; every 16 bytes of an operand are checked against its end.
constexpr int ANY = 128, ANY_THREADS = 256;

template <int FORM, class OUT>
__global__ __launch_bounds__(ANY_THREADS) void layer_any_kernel(LayerArgs p) {
    constexpr int STEP = 64, ROW = STEP + 16;              // bytes of a row in a step, and apart in LDS
    __shared__ __attribute__((aligned(16))) uint8_t smem[2][ANY * ROW];
    __shared__ int bounds[MUON_MAX_EXPERTS + 1], ends[MUON_MAX_EXPERTS + 1];
    __shared__ int64_t wave_tot[ANY_THREADS / 64];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave >> 1, wn = wave & 1, fr = lane & 31, fk = lane >> 5;
    if (p.mode != MUON_PRODUCT_DENSE) read_segments<1, ANY_THREADS>(p, ANY, bounds, ends, wave_tot);
    Walk my = walk<pair<FORM>>(p, ends);
    for (int t = next_tile(p, my); t >= 0; t = next_tile(p, my)) {
        const Tile x = decode<1, pair<FORM>>(p, t, ANY, ANY, bounds, ends);
        const int64_t to_group = p.mode == MUON_PRODUCT_ROWS ? x.group * p.stride_b : 0;
        f32x16 acc[2][2] = {};
        for (int part = 0; part < parts<FORM>; ++part)
            for (int64_t k0 = x.kb0; k0 < x.kb1; k0 += STEP / 2) {
                // 128 rows of a panel along: two chunks of one a thread
                auto along = [&](uint8_t* to, const uint8_t* row) {
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const int at = 32 * (tid & 1) + 16 * c;
                        i32x4 v = {0, 0, 0, 0};
                        if (row) v = load_checked<uint16_t>(row, 2 * k0 + at, 2 * (int64_t)x.kb1);
                        *reinterpret_cast<i32x4*>(to + (tid >> 1) * ROW + at) = v;
                    }
                };
                // or 32 depth rows across, transposed: 16 columns from `first` a thread
                auto across = [&](uint8_t* to, const uint8_t* base, int64_t ld, int64_t first, int64_t end) {
                    const int kk = tid >> 3, c0 = 16 * (tid & 7);
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        i32x4 v = {0, 0, 0, 0};
                        if (k0 + kk < x.kb1) v = load_checked<uint16_t>(base + (k0 + kk) * ld, 2 * (first + c0 + 8 * c), 2 * end);
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            *reinterpret_cast<uint16_t*>(to + (c0 + 8 * c + e) * ROW + 2 * kk) = (uint16_t)((uint32_t)v[e / 2] >> (16 * (e & 1)));
                    }
                };
                if constexpr (a_across<FORM>) across(smem[0], p.a[x.which], p.lda, x.m0, p.m);
                else along(smem[0], (tid >> 1) < x.rows_a ? p.a[part] + (x.m0 + (tid >> 1)) * p.lda : nullptr);
                across(smem[1], p.b[part] + to_group, p.ldb, x.n0, p.n);
                __syncthreads();
#pragma unroll
                for (int kk = 0; kk < 2; ++kk) {
                    i32x4 fa[2], fb[2];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        fa[i] = *reinterpret_cast<const i32x4*>(smem[0] + (64 * wm + 32 * i + fr) * ROW + 32 * kk + 16 * fk);
                        fb[i] = *reinterpret_cast<const i32x4*>(smem[1] + (64 * wn + 32 * i + fr) * ROW + 32 * kk + 16 * fk);
                    }
#pragma unroll
                    for (int i = 0; i < 2; ++i)
#pragma unroll
                        for (int j = 0; j < 2; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, fb[j]), __builtin_bit_cast(bf16x8, fa[i]), acc[i][j], 0, 0, 0);
                }
                __syncthreads();
            }
        // a lane's sums: row fr of a block, columns 8 q + 4 fk + (0 .. 3)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int r = 64 * wm + 32 * i + fr;
            if (r >= x.rows_a) continue;
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int v = 0; v < 16; ++v) {
                    const int c = 64 * wn + 32 * j + 8 * (v >> 2) + 4 * fk + (v & 3);
                    if (c >= x.rows_b) continue;
                    OUT* o = static_cast<OUT*>(p.out[x.which]) + (p.mode == MUON_PRODUCT_DEPTH ? x.group * p.out_stride : 0) +
                             (x.m0 + r) * p.ld_out[0] + x.n0 + c;
                    if constexpr (sizeof(OUT) == 4) *o = p.accumulate ? *o + acc[i][j][v] : acc[i][j][v];
                    else *o = dev::f32_to_bf16(acc[i][j][v]);
                }
        }
    }
}

// ---- big tiles ------------------------------------------------------------------------------
//
// 256, 128 or 64 rows of a by 256 of b (ROWS; see big_cost), one workgroup of 8 waves per CU that goes through its share of the tiles.
// Wave (h, c) of 2 x 4 takes the 16-row blocks 2 i + h of a and 64 rows of b, so that a tile with fewer rows (a segment's end) leaves
// both wave rows half of what there is.  Of a gated block a tile has 128 columns: b's panel holds 128 rows of gate and the
// same 128 of up, a wave 32 of each, so a lane has both sums of a value of out.
//
// Bound by the matrix cores, whose clock falls to what the card's power allows (1.4 to 2.0 GHz): 8192 x 4096 x 4096 gate and up
// in bfloat16 takes 423 to 440 us (1.25 to 1.30 PFLOP/s), its gradients 895 (1.23), its product in 8-bit integers 115 (2.39 POP/s).  Tried
// and left out: two workgroups of 128 x 256 per CU (20 to 25 % more time), 32 x 32 instructions (4 to 7 % more), every second
// workgroup begun half a tile later, so that not all store at once (nothing).
constexpr int TILE = 256, WAVES = 8, THREADS = 64 * WAVES;
constexpr int FN = 4;                                      // 16 x 16 blocks of a wave along b; along a: FM
constexpr int STEP = 128;                                  // bytes of a row in a step: 64 bfloat16 values, 128 codes

template <int N>
using ic = std::integral_constant<int, N>;

// Keeps the matrix instructions that have written acc so far in front of what follows.
template <class S, int FM>
__device__ __forceinline__ void pin(S (&acc)[FM][FN]) {
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) asm volatile("" : "+v"(acc[i][j]));
}

// A fragment of a panel that lies across: 4 x 4 blocks of 16-bit values are transposed among 16 lanes.
__device__ __forceinline__ uint64_t read_transposed(const uint8_t* at) {
    typedef short i16x4 __attribute__((ext_vector_type(4)));
    return __builtin_bit_cast(uint64_t, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                                            (__attribute__((address_space(3))) i16x4*)(const __attribute__((address_space(3))) uint8_t*)at));
}

// Operands go global -> VGPR -> LDS, a step (128 bytes of depth) ahead of the stage that is multiplied, of which there are
// two; the step's one barrier comes in the middle of its last sub-step, whose fragments are then in registers.
//
// LDS serves a 16-byte read 16 lanes at a time, which have all 16 rows of a block but not one depth (lanes 0 to 3, 12 to 15, 20 to 23
// and 24 to 27 for one), and a 16-byte write 8 lanes at a time, here a row's 8 chunks.  So of a panel along its rows, chunk c of
// row r lies in the r ^ c-th of the 16 slots of its block's c-th 256 bytes: reads fall on different rows' slots, writes on
// different chunks'.  (Rows of 144 bytes had conflicts in 38 % of LDS's cycles.)  A panel across lies in 64 depth rows of all its columns, whose 32-byte
// pieces (16 columns) are permuted by the row, so that the 8 rows that half a wave's transposing read touches fall on 8 different ones.
//
// Nothing in the main loop deals with ends:
//   * a depth that is no multiple of the step is taken with its remainder first, whose loads are masked where they are stored
//     before the loop; of GRAD_X the rows of a are padded to whole steps with zeros;
//   * rows of a panel along, and depth rows of one across, that are behind the end lie behind the end of the buffer that the
//     loads go through (the row is in the vector part of the offset: see fp8_panel.h) and arrive as zeros;
//   * of a panel across the last 8 columns are loaded again where fewer than 8 are left: in those 8 places of the tile
//     the last columns come last, and out is stored accordingly.
// So a 16-byte load never crosses the end of a row, and rows may begin anywhere.
template <class E, int FORM, class OUT, int ROWS>
__global__ __launch_bounds__(THREADS) __attribute__((amdgpu_waves_per_eu(2, 2))) void layer_kernel(LayerArgs p) {
    constexpr bool GATED = FORM == FORM_GATED, I8 = sizeof(E) == 1, F32 = sizeof(OUT) == 4;
    constexpr bool ACROSS_A = a_across<FORM>, ACROSS_B = b_across<FORM>, TWO = parts<FORM> == 2;
    constexpr int ES = (int)sizeof(E), UNIT = STEP / ES;   // values of a step
    constexpr int COLS = GATED ? TILE / 2 : TILE;
    constexpr int FM = ROWS / 32;                          // row blocks of a wave
    constexpr int LA = ROWS / 64, NLOAD = LA + 4;          // load instructions of a step
    constexpr int BLOCK = 16 * STEP, KROW_A = 2 * ROWS, KROW_B = 2 * TILE;  // LDS bytes of 16 rows of a panel along, of a depth row across
    constexpr int PANEL_A = ROWS * STEP, STAGE = PANEL_A + TILE * STEP;
    constexpr int CPA = ROWS / 8, CPB = TILE / 8, KA = THREADS / CPA, KB = THREADS / CPB;  // 16-byte chunks of a depth row, depth rows of a load
    static_assert(ROWS >= 64 && KA * LA == UNIT * ES / 2, "loads make up a step");
    constexpr int EPL = 16 / (int)sizeof(OUT);             // values of out in 16 bytes
    constexpr int OCOLS = GATED ? 96 : 64;                 // columns that a wave stages: out, gate and up; or out
    constexpr int OROW = OCOLS * (int)sizeof(OUT) + (F32 ? 0 : 16);  // (a float32 row's 16 pieces are permuted by the row instead)
    constexpr int WB = WAVES * 32 * OROW <= STAGE ? 2 : 1; // row blocks of out that go through a stage at a time
    static_assert(WAVES * 16 * WB * OROW <= STAGE && FM % WB == 0, "out goes through one stage");
    // The next tile's first two steps are loaded in this one's last two: weight gradients have few steps a tile and much to store (64 of
    // 2 x 1024 x 4096 over 448 rows each: 651 us against 710), and it costs little where there is one loop.  Of an expert's rows, 256
    // at a time, the last ones are too often few to be multiplied as if they were all there: those tiles have a loop of their own,
    // and there it takes registers and gains nothing.
    constexpr bool AHEAD = ACROSS_A || ROWS < 256;
    __shared__ __attribute__((aligned(1024))) uint8_t smem[2 * STAGE];
    __shared__ int bounds[MUON_MAX_EXPERTS + 1], ends[MUON_MAX_EXPERTS + 1];
    __shared__ int64_t wave_tot[WAVES];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wh = wave >> 2, wc = wave & 3;               // wave row and column
    // opaque, so that what is worked out of it per tile is not kept through the main loop, which has registers for a few values only
    auto thread = []() {
        int t = threadIdx.x;
        asm volatile("" : "+v"(t));
        return t;
    };

    if (p.mode != MUON_PRODUCT_DENSE) read_segments<1, THREADS>(p, ROWS, bounds, ends, wave_tot);
    Walk my = walk<pair<FORM>>(p, ends);
    int t = next_tile(p, my);
    if (t < 0) return;

    // Staging: along, load i brings rows 64 i + t / 8, chunk t % 8; across, depth rows KA i + t / CPA, chunk t % CPA (KB, CPB).
    // The permutation of 32-byte pieces does not change from load to load; rows of 128 bytes are two to 256.
    auto swizzle = [](int k, int row_bytes) { return row_bytes == 128 ? ((k >> 1) & 1) | ((k >> 2) & 2) : ((k & 3) << 1) | ((k >> 3) & 1); };
    // (worked out where it is needed, as are the fragments' places)
    struct Place {
        int along, across_a, across_b;
    };
    auto stores_at = [&]() {
        const int t = thread();
        auto place = [&](int row, int chunk, int row_bytes) { return row * row_bytes + (((chunk >> 1) ^ swizzle(row, row_bytes)) << 5) + ((chunk & 1) << 4); };
        return Place{(t >> 7) * BLOCK + (t & 7) * 256 + ((((t >> 3) & 15) ^ (t & 7)) << 4), place(t / CPA, t % CPA, KROW_A), place(t / CPB, t % CPB, KROW_B)};
    };

    // A tile's operands: their first rows (along) or depth row 0 (across), sizes of the buffers along; the depth's begin, its
    // values before the whole steps, those of each part, and all steps.
    struct Span {
        const uint8_t *a, *b;
        int bytes_a, bytes_b, first, rest, whole, steps;
    };
    Span cur{}, nxt{};                                     // of the tile that is multiplied, and (AHEAD) of the next one
    int va = 0, vb = 0, va_next = 0, vb_next = 0;          // the lane's offset from there in load 0
    int ahead_ok = 0;                                      // -1 where the next tile's first two steps are loaded in this one's last two
    const int lda = (int)p.lda, ldb = (int)p.ldb;
    i32x4 staged[NLOAD];
    // Where a step's loads go: operands' buffers, and their scalar offset along (pieces of this are the same for all of a step).
    struct Aim {
        const uint8_t *a, *b;
        int bytes_a, bytes_b, along, va, vb;
    };
    auto mask = [](bool valid) {
        int keep = __builtin_amdgcn_readfirstlane(valid ? -1 : 0);
        asm volatile("" : "+s"(keep));
        return keep;
    };
    // Step `step` of a tile, or nowhere where keep is 0 and not -1 (from an empty buffer, which fetches nothing).  No branch, which
    // in the main loop would let the compiler move the matrix instructions behind it.
    auto aim = [&](const Span& x, int step, int keep) {
        const int lead = min(x.rest, 1), w = step - lead;
        const int partial = w >> 31;                       // -1 for the remainder
        const int part = TWO ? (x.whole - 1 - w) >> 31 : 0;  // 0, or -1 for the second
        int at = UNIT * (w - (x.whole & part)), valid;
        if (TWO) {
            valid = min(UNIT, (int)p.k - at);
        } else {
            at = x.first + ((x.rest + at) & ~partial);
            valid = UNIT + ((x.rest - UNIT) & partial);
        }
        at &= keep;
        Aim r;
        r.a = x.a + (TWO ? (p.a[1] - p.a[0]) & (int64_t)part : 0) + (ACROSS_A ? (int64_t)at * lda : 0);
        r.b = x.b + (TWO ? (p.b[1] - p.b[0]) & (int64_t)part : 0) + (ACROSS_B ? (int64_t)at * ldb : 0);
        r.bytes_a = (ACROSS_A ? (valid - 1) * lda + 2 * (int)p.m : x.bytes_a) & keep;
        r.bytes_b = (ACROSS_B ? (valid - 1) * ldb + 2 * (int)p.n : x.bytes_b) & keep;
        r.along = at * ES;
        r.va = va;
        r.vb = vb;
        return r;
    };
    // Step `step` of the tile that is multiplied, or behind its last the next tile's first two, or nowhere.
    auto aim_on = [&](int step) {
        const int over = mask(step >= cur.steps);          // -1 or 0
        if constexpr (!AHEAD) {
            return aim(cur, step, ~over);
        } else {
            auto pick = [&](int x, int y) { return x ^ ((x ^ y) & over); };
            auto pick_ptr = [&](const uint8_t* x, const uint8_t* y) {
                return (const uint8_t*)((uint64_t)x ^ (((uint64_t)x ^ (uint64_t)y) & (uint64_t)(int64_t)over));
            };
            const Span x = {pick_ptr(cur.a, nxt.a), pick_ptr(cur.b, nxt.b), pick(cur.bytes_a, nxt.bytes_a), pick(cur.bytes_b, nxt.bytes_b),
                            pick(cur.first, nxt.first), pick(cur.rest, nxt.rest), pick(cur.whole, nxt.whole), 0};
            Aim r = aim(x, step - (cur.steps & over), ~over | ahead_ok);
            if (ACROSS_A) r.va = pick(va, va_next);
            if (ACROSS_B) r.vb = pick(vb, vb_next);
            return r;
        }
    };
    // Chunk d of a step into its register.
    auto load = [&](int d, const Aim& r) {
        const bool is_a = d < LA;
        const int i = is_a ? d : d - LA;
        const bool across = is_a ? ACROSS_A : ACROSS_B;
        // (opaque, or the sums of all d stay in registers)
        int32_t rows_on = (across ? (is_a ? KA : KB) * i : 64 * (GATED && !is_a ? i & 1 : i)) * (is_a ? lda : ldb);
        asm volatile("" : "+s"(rows_on));
        // (of a gated block b's loads 0 and 1 bring gate, 2 and 3 up)
        const uint8_t* base = (is_a ? r.a : r.b) + (GATED && !is_a && i >= 2 ? p.b[1] - p.b[0] : 0);
        const __amdgpu_buffer_rsrc_t buf = __builtin_amdgcn_make_buffer_rsrc((void*)base, 0, is_a ? r.bytes_a : r.bytes_b, 0x00020000);
        staged[d] = __builtin_amdgcn_raw_buffer_load_b128(buf, (is_a ? r.va : r.vb) + rows_on, across ? 0 : r.along, 0);
    };
    auto store = [&](int d, int st, const Place& p) {
        const bool is_a = d < LA;
        const int i = is_a ? d : d - LA;
        const int at = !(is_a ? ACROSS_A : ACROSS_B) ? p.along + 4 * BLOCK * i : is_a ? p.across_a + KA * KROW_A * i : p.across_b + KB * KROW_B * i;
        *reinterpret_cast<i32x4*>(smem + st * STAGE + (is_a ? 0 : PANEL_A) + at) = staged[d];
    };
    auto span = [&](const Tile& x, bool there, int& va, int& vb) {
        const int t = thread(), lrow = t >> 3, lchunk = t & 7;
        auto all = [](int v) { return __builtin_amdgcn_readfirstlane(v); };
        Span r;
        r.a = uniform(p.a[ACROSS_A ? x.which : 0] + (ACROSS_A ? 0 : x.m0 * p.lda));
        r.b = uniform(p.b[0] + (p.mode == MUON_PRODUCT_ROWS ? x.group * p.stride_b : 0) + (ACROSS_B ? 0 : x.n0 * p.ldb));
        const int depth = x.kb1 - x.kb0;
        r.first = all(x.kb0);
        r.rest = all(I8 || TWO ? 0 : depth % UNIT);
        r.whole = all(I8 || TWO ? (depth + UNIT - 1) / UNIT : depth / UNIT);
        r.steps = all(there ? (r.rest > 0) + parts<FORM> * r.whole : 0);
        const int row_bytes = I8 || TWO ? r.whole * STEP : x.kb1 * ES;
        r.bytes_a = all((x.rows_a - 1) * lda + row_bytes);
        r.bytes_b = all((x.rows_b - 1) * ldb + row_bytes);
        auto column = [](int64_t c, int64_t n) { return 2 * (int)min(c, n - 8); };
        va = ACROSS_A ? t / CPA * lda + column(x.m0 + 8 * (t % CPA), p.m) : lrow * lda + 16 * lchunk;
        vb = ACROSS_B ? t / CPB * ldb + column(x.n0 + 8 * (t % CPB), p.n) : lrow * ldb + 16 * lchunk;
        return r;
    };
    // The first loads of a tile, or, where they were loaded ahead, none.
    auto begin = [&](int keep) {
        const Aim r = aim(cur, 0, mask(cur.steps > 0) & keep);
#pragma unroll
        for (int d = 0; d < NLOAD; ++d) load(d, r);
    };
    // Its first step into LDS, the second into the registers.
    auto fill = [&](int st) {
        // values of a lane's chunk that are in the partial step; the others follow in the next one
        const int have = cur.rest > 0 ? min(max(cur.rest * ES - 16 * (thread() & 7), 0), 16) : 16;
        i32x4 inside;
#pragma unroll
        for (int e = 0; e < 4; ++e) inside[e] = have >= 4 * e + 4 ? -1 : have == 4 * e + 2 ? 0xffff : 0;
        const Aim r = aim_on(1);
        const Place at = stores_at();
#pragma unroll
        for (int d = 0; d < NLOAD; ++d) {
            if (!I8 && !TWO && !(d < LA ? ACROSS_A : ACROSS_B)) staged[d] &= inside;
            store(d, st, at);
            load(d, r);
        }
    };

    // A fragment, 16 bytes of a row's depth, in sub-step kk: along in one read; across in two, whose lanes take depth rows tk and
    // columns tc.  (Blocks i of a and j of b lie apart by bits of the address that nothing else of it has: 2 i + wh is
    // i << 1 | wh, 4 wc + j is wc << 2 | j.)
    struct Fragments {
        int a, b;
    };
    auto fragments_at = [&]() {
        const int t = thread(), fr = t & 15, fk = (t >> 4) & 3;
        const int tk = 8 * fk + (fr >> 2), tc = 4 * (t & 3);
        Fragments r;
        r.a = ACROSS_A ? tk * KROW_A + ((wh ^ swizzle(tk, KROW_A)) << 5) + 2 * tc : wh * BLOCK + fk * 256 + ((fr ^ fk) << 4);
        r.b = PANEL_A + (ACROSS_B ? tk * KROW_B + (((4 * wc) ^ swizzle(tk, KROW_B)) << 5) + 2 * tc : (GATED ? 2 : 4) * wc * BLOCK + fk * 256 + ((fr ^ fk) << 4));
        return r;
    };
    static_assert(PANEL_A % 512 == 0 && STAGE % 512 == 0, "stages and panels begin on multiples of all rows");
    auto read_across = [&](int at, int row_bytes) {
        typedef uint64_t u64x2 __attribute__((ext_vector_type(2)));
        return __builtin_bit_cast(i32x4, u64x2{read_transposed(smem + at), read_transposed(smem + at + 4 * row_bytes)});
    };
    auto read_a = [&](int ra, int i, int st, int kk) {
        if constexpr (ACROSS_A) return read_across(((ra + st * STAGE) ^ (i << 6)) + 32 * KROW_A * kk, KROW_A);
        else return *reinterpret_cast<const i32x4*>(smem + ((ra + st * STAGE) ^ (kk << 6)) + 2 * BLOCK * i + 1024 * kk);
    };
    auto read_b = [&](int rb, int j, int st, int kk) {
        if constexpr (ACROSS_B) return read_across(((rb + st * STAGE) ^ (j << 5)) + 32 * KROW_B * kk, KROW_B);
        else return *reinterpret_cast<const i32x4*>(smem + ((rb + st * STAGE) ^ (kk << 6)) + (GATED ? (j >> 1) * (TILE / 32) + (j & 1) : j) * BLOCK + 1024 * kk);
    };

    // Waits for the loads in flight, where they are the last steps' empty ones: what comes may have other uses for their registers, and
    // would wait in the main loop.
    auto settle = [&]() {
#pragma unroll
        for (int d = 0; d < NLOAD; ++d) asm volatile("" : : "v"(staged[d]));
    };

    typename Cores<E>::sums acc[FM][FN];
    // The steps of a tile for a wave whose first PAIRS pairs of row blocks have rows.
    //
    // A step is two sub-steps; in each a pair's 8 matrix instructions stand together.  Behind them go staging, over the slots before the
    // step's barrier (half way through the second sub-step), and the next sub-step's reads: a's in place, b's to the other
    // registers.
    int begins = 0;                                        // stage of the tile's first step
    auto multiply = [&](auto pairs_) {
        constexpr int PAIRS = decltype(pairs_)::value, TURN = PAIRS / 2;   // pairs of a sub-step; of the second one before the barrier
        i32x4 fa[2 * PAIRS], fb[2][FN];
        const Fragments fragments = fragments_at();
        const Place stores = stores_at();
        // (in the order of the loop's reads, as a wait there covers both)
#pragma unroll
        for (int j = 0; j < FN; ++j) {
            fb[0][j] = read_b(fragments.b, j, begins, 0);
            __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll
        for (int i = 0; i < 2 * PAIRS; ++i) {
            fa[i] = read_a(fragments.a, i, begins, 0);
            __builtin_amdgcn_sched_barrier(0);
        }
        for (int step = 0; step < cur.steps; ++step) {
            const Aim ahead = aim_on(step + 2);
            const int st = (begins + step) & 1, st_next = st ^ 1;
            auto stage = [&](int d) {
                store(d, st_next, stores);
                load(d, ahead);
            };
            // Pair q in sub-step kk, read(f) behind its instruction f.  Columns go to and fro, so that an instruction has an operand in common
            // with the one before it: 1 to 2 % less time where power sets the clock (b's held longer than a's instead: 1 % more).
            auto pair_of = [&](int q, int kk, auto read) {
                constexpr int ALL = (PAIRS + TURN) * 2 * FN;   // slots of staging
#pragma unroll
                for (int f = 0; f < 2 * FN; ++f) {
                    const int i = 2 * q + f / FN, j = f < FN ? f : 2 * FN - 1 - f, g = (PAIRS * kk + q) * 2 * FN + f;
                    __builtin_amdgcn_sched_barrier(0);
                    acc[i][j] = Cores<E>::mul(fb[kk][j], fa[i], acc[i][j]);
                    __builtin_amdgcn_sched_barrier(0);
                    if (g < ALL && (g + 1) * NLOAD / ALL > g * NLOAD / ALL) stage(g * NLOAD / ALL);
                    read(f);
                }
            };
            // a's of pair q are read for the next sub-step behind their last use
            auto renew = [&](int q, int f, int rst, int kk) {
                if (f == FN - 1) fa[2 * q] = read_a(fragments.a, 2 * q, rst, kk);
                if (f == 2 * FN - 1) fa[2 * q + 1] = read_a(fragments.a, 2 * q + 1, rst, kk);
            };
            // the next step's first fragments: b's, and the a's that were used before the barrier
            auto first = [&](int f) {
                if (f < FN) fb[0][f] = read_b(fragments.b, f, st_next, 0);
                else if (f - FN < 2 * TURN) fa[f - FN] = read_a(fragments.a, f - FN, st_next, 0);
            };
#pragma unroll
            for (int q = 0; q < PAIRS; ++q)
                pair_of(q, 0, [&](int f) {
                    if (q == 0 && f < FN) fb[1][f] = read_b(fragments.b, f, st, 1);
                    renew(q, f, st, 1);
                });
#pragma unroll
            for (int q = 0; q < TURN; ++q) pair_of(q, 1, [](int) {});
            pin(acc);
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
            __builtin_amdgcn_s_barrier();
            asm volatile("" ::: "memory");
#pragma unroll
            for (int q = TURN; q < PAIRS; ++q)
                pair_of(q, 1, [&](int f) {
                    if (q == TURN) first(f);
                    renew(q, f, st_next, 0);
                });
        }
        if (!AHEAD) settle();
    };

    // Scales of the lane's rows and columns (8-bit integers), asked for before the next tile's loads.
    float sa[I8 ? FM : 1];
    f32x4 sb[I8 ? FN : 1];
    Tile done;
    auto read_scales = [&](const Tile& x) {
        if constexpr (I8) {
            const int64_t group = p.mode == MUON_PRODUCT_ROWS ? x.group * p.stride_sb : 0;
            const int t = thread(), fr = t & 15, fk = (t >> 4) & 3;
#pragma unroll
            for (int i = 0; i < FM; ++i) sa[i] = p.sa[x.m0 + min(32 * i + 16 * wh + fr, x.rows_a - 1)];
#pragma unroll
            for (int j = 0; j < FN; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    sb[j][e] = p.sb[GATED ? j >> 1 : 0][group + x.n0 + min(GATED ? 32 * wc + 16 * (j & 1) + 4 * fk + e : 64 * wc + 16 * j + 4 * fk + e, x.rows_b - 1)];
        }
    };
    // Row blocks WB w on of out: 16 or 32 rows of the wave through its part of the stage of the tile's last step (which is not read any
    // more after that step's barrier, nor written before the next tile's first step), then in 16-byte stores along the rows, which leave the caches to the operands.
    auto write = [&](int w2, int st) {  // w2 < FM / WB
        const int ln = thread() & 63;
        uint8_t* mine = smem + st * STAGE + wave * 16 * WB * OROW;
        // byte of column col of row r there
        auto at = [&](int r, int col) { return r * OROW + (F32 ? ((col >> 2) ^ (r & 15)) << 4 : col * (int)sizeof(OUT)); };
        const int r0 = 32 * WB * w2 + 16 * wh;             // (the second block's are 32 rows on)
        if (r0 >= done.rows_a) return;
        auto put = [&](int row, int col, const f32x4& v) {
            uint8_t* o = mine + at(row, col);
            if constexpr (F32) *reinterpret_cast<f32x4*>(o) = v;
            else *reinterpret_cast<uint2*>(o) = make_uint2(dev::f32x2_to_bf16x2(v[0], v[1]), dev::f32x2_to_bf16x2(v[2], v[3]));
        };
#pragma unroll
        for (int b = 0; b < WB; ++b) {
            const int i = WB * w2 + b, row = 16 * b + (ln & 15), c = 4 * (ln >> 4);
            auto scaled = [&](int j) {
                f32x4 v;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if constexpr (I8) v[e] = (float)acc[i][j][e] * sa[i] * sb[j][e];
                    else v[e] = acc[i][j][e];
                }
                return v;
            };
            if constexpr (GATED) {
#pragma unroll
                for (int j = 0; j < FN / 2; ++j) {
                    const f32x4 g = scaled(j), u = scaled(j + FN / 2);
                    f32x4 h;
#pragma unroll
                    for (int e = 0; e < 4; ++e) h[e] = gated_value(p.activation, g[e], u[e]);
                    put(row, 16 * j + c, h);
                    if (p.out[1]) {
                        put(row, 32 + 16 * j + c, g);
                        put(row, 64 + 16 * j + c, u);
                    }
                }
            } else {
#pragma unroll
                for (int j = 0; j < FN; ++j) put(row, 16 * j + c, scaled(j));
            }
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        constexpr int WIDTH = GATED ? 32 : 64;             // columns of out of the wave
        constexpr int LPR = WIDTH / EPL, RPS = 64 / LPR;   // lanes per row, rows per store
        const int col = ln % LPR * EPL, row = ln / LPR;
        const int64_t c0 = done.n0 + WIDTH * wc + col;     // the lane's first column
        const int64_t left = p.n - c0;
        // places of 8 columns (across: of rows too) with fewer left hold the last 8
        const int64_t back = ACROSS_B && (c0 & ~7) + 8 > p.n ? (c0 & ~7) + 8 - p.n : 0;
#pragma unroll
        for (int w = 0; w < (GATED ? 3 : 1); ++w) {
            OUT* out = static_cast<OUT*>(p.out[GATED ? w : done.which]);
            if (GATED && !out) continue;
            const int64_t ld = p.ld_out[GATED && w ? 1 : 0];
            if (p.mode == MUON_PRODUCT_DEPTH) out += done.group * p.out_stride;
#pragma unroll
            for (int q = 0; q < 16 * WB / RPS; ++q) {
                const uint4 u = *reinterpret_cast<const uint4*>(mine + at(q * RPS + row, 32 * w + col));
                const int in_tile = r0 + (q * RPS + row) % 16 + (q * RPS + row) / 16 * 32;
                int64_t r = done.m0 + in_tile;
                if (ACROSS_A && (r & ~7) + 8 > p.m) {
                    const int64_t place = r & ~7;
                    r += p.m - 8 - place;
                    if (r < place) continue;
                } else if (in_tile >= done.rows_a) {
                    continue;
                }
                OUT* o = out + r * ld + c0;
                if (EPL <= left && back == 0) {
                    if constexpr (F32) {
                        f32x4 v = __builtin_bit_cast(f32x4, u);
                        if (p.accumulate) v += *reinterpret_cast<const f32x4_any*>(o);
                        if (p.vec) __builtin_nontemporal_store(v, reinterpret_cast<f32x4*>(o));
                        else *reinterpret_cast<f32x4_any*>(o) = v;
                    } else {
                        if (p.vec) __builtin_nontemporal_store(__builtin_bit_cast(i32x4, u), reinterpret_cast<i32x4*>(o));
                        else *reinterpret_cast<i32x4_any*>(o) = __builtin_bit_cast(i32x4, u);
                    }
                } else {
                    const uint32_t word[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                    for (int e = 0; e < EPL; ++e) {
                        const int64_t c = e - back;        // from c0; the place begins (c0 & 7) before it
                        if (c >= left || c < -(c0 & 7)) continue;
                        if constexpr (F32) o[c] = p.accumulate ? o[c] + __uint_as_float(word[e]) : __uint_as_float(word[e]);
                        else o[c] = (uint16_t)(word[e / 2] >> (16 * (e & 1)));
                    }
                }
            }
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
    };

    // The tiles.  The next tile's first loads come before this one's stores, behind which loads would wait (a wave's loads and stores
    // end in order).  Where there is no next tile or no depth they fetch nothing, but are there: past a branch around them the
    // compiler would hold their registers for loads in flight, and wait in the main loop for all that are.
    Tile x = decode<1, pair<FORM>>(p, t, ROWS, COLS, bounds, ends), x_next = x;
    cur = span(x, true, va, vb);
    begin(-1);
    auto look = [&]() {
        t = next_tile(p, my);
        x_next = decode<1, pair<FORM>>(p, max(t, 0), ROWS, COLS, bounds, ends);
        nxt = span(x_next, t >= 0, va_next, vb_next);
        ahead_ok = mask(nxt.steps >= 2 && (I8 || TWO || ACROSS_A || nxt.rest == 0));   // (along, a remainder has to be masked)
    };
    if (AHEAD) look();
    fill(0);
    for (;;) {
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
            for (int j = 0; j < FN; ++j) acc[i][j] = typename Cores<E>::sums{};
        if (cur.steps > 0) {
            asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
            const int pairs = (x.rows_a - 16 * wh + 63) / 64;   // (row block i has rows 16 (2 i + wh) .. + 15)
            if constexpr (AHEAD) multiply(ic<FM / 2>{});
            else if (pairs >= 3) multiply(ic<4>{});
            else multiply(ic<2>{});
        }
        done = x;
        read_scales(done);
        const int free = cur.steps > 0 ? (begins + cur.steps - 1) & 1 : begins ^ 1;   // the stage that out may go through
        const bool loaded = AHEAD && cur.steps > 0 && ahead_ok != 0;                  // the next tile's first steps are under way
        begins = free ^ 1;
        if (AHEAD) {
            x = x_next;
            cur = nxt;
            va = va_next;
            vb = vb_next;
            if (t < 0) cur.steps = -1;                     // the end
            else if (!loaded) begin(-1);
            if (t >= 0) look();
        } else {
            t = next_tile(p, my);
            x = decode<1, pair<FORM>>(p, max(t, 0), ROWS, COLS, bounds, ends);
            cur = span(x, t >= 0, va, vb);
            if (t < 0) cur.steps = -1;
            begin(-1);
        }
        if constexpr (I8) {                                // (as well: past a row block that is left out)
#pragma unroll
            for (int i = 0; i < FM; ++i) asm volatile("" : "+v"(sa[i]));
#pragma unroll
            for (int j = 0; j < FN; ++j) asm volatile("" : "+v"(sb[j]));
        }
#pragma unroll
        for (int w = 0; w < FM / WB; ++w) {
            if (w == FM / WB / 2 && (!AHEAD || (!loaded && cur.steps >= 0))) fill(begins);
            write(w, free);
        }
        if (cur.steps < 0) break;
    }
}

// ---- few rows or few tiles: 16 or 32 rows by 16 or more columns, depth split over the waves -----------------
//
// For serving, where 256 x 256 tiles would leave most of the chip idle.  Each of 8 waves takes every eighth step (128 bytes) of the
// depth of a tile of 16 RB rows of a by 16 NB rows of b (of a gated block NB / 2 blocks of gate and as many of up), its fragments
// straight from memory into registers, AHEAD steps at a time, so that a tile's loads are under way together; the
// waves' sums are added up through LDS in the order of the waves.  Bound by memory, and for a single call by its latency
// (1 row by 5632 x 2048 gate and up in bfloat16: 13.1 us for 46 MB that the last-level cache keeps from call to call, 16.2 from memory; 1 row
// by 2048 x 5632 in 8-bit integers: 7.0 us, 11.5 MB).
template <class E, int FORM, class OUT, int RB, int NB, int AHEAD>
__global__ __launch_bounds__(THREADS) void layer_few_kernel(LayerArgs p) {
    constexpr bool GATED = FORM == FORM_GATED, I8 = sizeof(E) == 1, F32 = sizeof(OUT) == 4;
    constexpr int ES = (int)sizeof(E), UNIT = STEP / ES;
    constexpr int ROWS = 16 * RB, COLS = 16 * NB, SUMS = COLS + 4;  // of sums; a row of them in LDS
    constexpr int OUT_COLS = GATED ? COLS / 2 : COLS;
    typedef typename Cores<E>::sums sums_t;
    __shared__ __attribute__((aligned(16))) int sums[WAVES][ROWS * SUMS];
    __shared__ int bounds[MUON_MAX_EXPERTS + 1], ends[MUON_MAX_EXPERTS + 1];
    __shared__ int64_t wave_tot[WAVES];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int fr = lane & 15, fk = lane >> 4;
    if (p.mode != MUON_PRODUCT_DENSE) read_segments<1, THREADS>(p, ROWS, bounds, ends, wave_tot);
    Walk my = walk<1>(p, ends);
    for (int t = next_tile(p, my); t >= 0; t = next_tile(p, my)) {
        const Tile x = decode<1, 1>(p, t, ROWS, OUT_COLS, bounds, ends);
        const int64_t group = p.mode == MUON_PRODUCT_ROWS ? x.group : 0;
        // the lane's rows; those past the end repeat the last: their sums are not stored
        const uint8_t *ra[RB], *rb[NB];
#pragma unroll
        for (int i = 0; i < RB; ++i) ra[i] = p.a[0] + (x.m0 + min(16 * i + fr, x.rows_a - 1)) * p.lda;
#pragma unroll
        for (int j = 0; j < NB; ++j) {
            const int w = GATED ? j / (NB / 2) : 0, c = 16 * (GATED ? j % (NB / 2) : j) + fr;
            rb[j] = p.b[w] + group * p.stride_b + (x.n0 + min(c, x.rows_b - 1)) * p.ldb;
        }
        sums_t acc[RB][NB] = {};
        // U steps from `step` on, every eighth; a lane's 32 bytes of each are two instructions' parts
        auto steps = [&](auto u_, auto load, int step) {
            constexpr int U = decltype(u_)::value;
            i32x4 fa[U][RB][2], fb[U][NB][2];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int64_t at = (int64_t)(step + u * WAVES) * STEP + 32 * fk;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
#pragma unroll
                    for (int j = 0; j < NB; ++j) fb[u][j][h] = load(rb[j], at + 16 * h);
#pragma unroll
                    for (int i = 0; i < RB; ++i) fa[u][i][h] = load(ra[i], at + 16 * h);
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int i = 0; i < RB; ++i)
#pragma unroll
                        for (int j = 0; j < NB; ++j) acc[i][j] = Cores<E>::mul(fb[u][j][h], fa[u][i][h], acc[i][j]);
        };
        auto whole = [](const uint8_t* row, int64_t at) -> i32x4 { return *reinterpret_cast<const i32x4_any*>(row + at); };
        const int depth = x.kb1;
        const int n_steps = I8 ? (depth + UNIT - 1) / UNIT : depth / UNIT;   // rows of codes are whole steps
        int step = wave;
        for (; step + (AHEAD - 1) * WAVES < n_steps; step += AHEAD * WAVES) steps(ic<AHEAD>{}, whole, step);
        for (; step < n_steps; step += WAVES) steps(ic<1>{}, whole, step);
        if (!I8 && step == n_steps && depth % UNIT != 0)   // the remainder is the next wave's
            steps(ic<1>{}, [&](const uint8_t* row, int64_t at) { return load_checked<E>(row, at, (int64_t)depth * ES); }, step);
        // a lane's sums are rows 16 i + fr, columns 16 j + 4 fk + (0 .. 3)
#pragma unroll
        for (int i = 0; i < RB; ++i)
#pragma unroll
            for (int j = 0; j < NB; ++j) *reinterpret_cast<sums_t*>(&sums[wave][(16 * i + fr) * SUMS + 16 * j + 4 * fk]) = acc[i][j];
        __syncthreads();
        for (int id = tid; id < ROWS * OUT_COLS / 4; id += THREADS) {
            const int row = id / (OUT_COLS / 4), col = 4 * (id % (OUT_COLS / 4));
            if (row >= x.rows_a) continue;
            const int64_t left = p.n - x.n0 - col;
            f32x4 v[GATED ? 2 : 1];
#pragma unroll
            for (int w = 0; w < (GATED ? 2 : 1); ++w) {
                const int at = row * SUMS + w * OUT_COLS + col;
                sums_t s = *reinterpret_cast<const sums_t*>(&sums[0][at]);
#pragma unroll
                for (int u = 1; u < WAVES; ++u) s += *reinterpret_cast<const sums_t*>(&sums[u][at]);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    v[w][e] = (float)s[e];
                    if constexpr (I8)
                        if (e < left) v[w][e] = v[w][e] * p.sa[x.m0 + row] * p.sb[w][group * p.stride_sb + x.n0 + col + e];
                }
            }
            auto put = [&](OUT* o, const f32x4& u) {
                if (left >= 4) {
                    if constexpr (F32) *reinterpret_cast<f32x4_any*>(o) = u;
                    else *reinterpret_cast<u32x2_any*>(o) = u32x2_any{dev::f32x2_to_bf16x2(u[0], u[1]), dev::f32x2_to_bf16x2(u[2], u[3])};
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        if (e >= left) continue;
                        if constexpr (F32) o[e] = u[e];
                        else o[e] = dev::f32_to_bf16(u[e]);
                    }
                }
            };
            const int64_t r = x.m0 + row, c = x.n0 + col;
            OUT* o = static_cast<OUT*>(p.out[0]) + r * p.ld_out[0] + c;
            if constexpr (GATED) {
                f32x4 h;
#pragma unroll
                for (int e = 0; e < 4; ++e) h[e] = gated_value(p.activation, v[0][e], v[1][e]);
                put(o, h);
                if (p.out[1]) {
                    put(static_cast<OUT*>(p.out[1]) + r * p.ld_out[1] + c, v[0]);
                    put(static_cast<OUT*>(p.out[2]) + r * p.ld_out[1] + c, v[1]);
                }
            } else {
                put(o, v[0]);
            }
        }
        __syncthreads();                                   // the sums are read
    }
}

// Whether the 256 x 256 tiles' loads fit: at least one of 16 bytes in a row (and a whole step where the depth's remainder
// comes first and its loads reach beyond it).
template <class E, int FORM>
bool tile_loads_fit(const LayerArgs& a) {
    if (a_across<FORM>) return a.m >= 8 && a.n >= 8;
    return b_across<FORM> ? a.n >= 8 : sizeof(E) == 1 || a.k >= STEP / 2;
}

// What a launch of the big tiles' kernel would take, in us, from what it measured: rounds of tiles, each a constant and so much a
// step, less where few CUs work (clock and caches).  A step of 256 x 256 takes 1.11 us alone on the chip and 1.43 with all CUs
// busy, with 128 rows 0.77 and 1.04, with 64 0.57 and 0.69; of 256 rows of which 192, 128 or 64 are there, 1.11, 0.79, 0.80 alone.  (The
// constants are from before the loops of 4 and 2 pairs and lie within 17 % of that.)
// Gate and up in bfloat16, 4096 x 4096 by 1024: 103 us in 512 tiles of 64 rows, 74 in 256 of 128, 96 in 128 of 256;
// 1024 x 4096: 46, 60, 87.  112 rows of 8-bit integers by as many experts, 4096 x 1024: 88, 94, 99.  57344 rows by 128
// experts, bfloat16: 1656, 1230, 1063.
struct Cost {
    int64_t tiles;
    double us;
};
template <int FORM>
Cost big_cost(LayerArgs a, int rows, double steps) {
    constexpr bool GATED = FORM == FORM_GATED;
    const int64_t most = count_tiles<pair<FORM>>(a, rows, GATED ? TILE / 2 : TILE);
    double n = (double)most, used = rows;
    if (a.mode == MUON_PRODUCT_ROWS) {
        // segments end inside tiles, on average in the middle
        const double segments = (double)std::min<int64_t>(a.m, a.groups);
        n = std::max((double)a.m / rows + 0.5 * segments, segments) * a.tiles_n;
        if (rows == 256) used = std::min(used, (double)a.m / segments);
    } else if (!a_across<FORM> && rows == 256) {
        used = std::min(used, (double)a.m);
    }
    static const double small[2][4] = {{0.57, 0.72, 5.7, 2.0}, {0.77, 1.0, 6.8, 3.5}};
    static const double full[4][4] = {{0.73, 0.85, 7.0, 2.0}, {0.92, 1.15, 8.0, 3.0}, {1.05, 1.35, 9.0, 4.0}, {1.14, 1.47, 9.5, 5.0}};
    const double(&c)[4] = rows < 256 ? small[rows / 128] : full[std::max((int)std::ceil(used / 64.0), 1) - 1];
    auto round = [&](double share) { return c[2] + (GATED ? c[3] : 0.0) + steps * (c[0] + (c[1] - c[0]) * share); };
    const double whole = std::floor(n / CUS), left = n / CUS - whole;
    return {most, whole * round(1.0) + (left > 0 ? round(left) : 0.0)};
}

// A launch: the kernel (rows of the big tiles; 0 to 2 for few rows; -1 for any size) and its arguments.
struct Plan {
    int pick;
    Cost cost;
    LayerArgs args;
};
template <class E, int FORM>
Plan plan(const LayerArgs& a) {
    constexpr bool GATED = FORM == FORM_GATED;
    const double depth = (double)a.k * (double)sizeof(E) / STEP / (a.mode == MUON_PRODUCT_DEPTH ? a.groups : 1);
    const double steps = std::ceil(depth) * parts<FORM>;
    Plan best{-1, {0, 1e30}, a};
    auto offer = [&](int pick, const Cost& cost, const LayerArgs& args) {
        if (cost.tiles >= 0 && cost.us < best.cost.us) best = {pick, cost, args};
    };
    if (tile_loads_fit<E, FORM>(a))
        for (int rows : {256, 128, 64}) {
            LayerArgs big = a;
            count_tiles<pair<FORM>>(big, rows, GATED ? TILE / 2 : TILE);
            offer(rows, big_cost<FORM>(a, rows, steps), big);
        }
    if constexpr (GATED || FORM == FORM_SCALED) {
        // 16 rows, 32 rows, 32 rows by 64 columns: bound by a wave's share of the depth where there are few tiles, by the steps of
        // all tiles where there are many (1 row by 5632 x 2048 gate and up in bfloat16, weights from memory: 16, 18, 16 us and 28 in
        // tiles of 64 rows; 64 rows: 40, 32, 30, 32; 256 rows: 130, 94, 76, 31; 1 row by 2048 x 5632 in 8-bit integers: 7, 8, 15, 30)
        static const double wait[2][3] = {{0.65, 0.75, 2.4}, {1.2, 1.55, 2.4}}, rate[2][3] = {{1900, 1290, 625}, {1500, 1024, 740}};
        for (int i = 0; i < 3; ++i) {
            LayerArgs few = a;
            const int64_t n = count_tiles<1>(few, i == 0 ? 16 : 32, i == 2 ? (GATED ? 32 : 64) : 16);
            offer(i, {n, 3.0 + std::max(steps / WAVES * wait[GATED][i], (double)n * (steps + 2.0) / rate[GATED][i])}, few);
        }
    }
    return best;
}

template <class E, int FORM, class OUT>
hipError_t launch(const Plan& p, hipStream_t s) {
    auto grid = [&](int64_t most) { return dim3((unsigned)std::min<int64_t>((p.cost.tiles + NUM_XCD - 1) / NUM_XCD * NUM_XCD, most)); };
    if constexpr (FORM == FORM_GATED || FORM == FORM_SCALED) {
        constexpr int THIN = FORM == FORM_GATED ? 2 : 1;
        if (p.pick == 0) hipLaunchKernelGGL((layer_few_kernel<E, FORM, OUT, 1, THIN, 4>), grid(4 * CUS), dim3(THREADS), 0, s, p.args);
        else if (p.pick == 1) hipLaunchKernelGGL((layer_few_kernel<E, FORM, OUT, 2, THIN, 4>), grid(2 * CUS), dim3(THREADS), 0, s, p.args);
        else if (p.pick == 2) hipLaunchKernelGGL((layer_few_kernel<E, FORM, OUT, 2, 4, 2>), grid(2 * CUS), dim3(THREADS), 0, s, p.args);
    }
    if (p.pick == 64) hipLaunchKernelGGL((layer_kernel<E, FORM, OUT, 64>), grid(CUS), dim3(THREADS), 0, s, p.args);
    else if (p.pick == 128) hipLaunchKernelGGL((layer_kernel<E, FORM, OUT, 128>), grid(CUS), dim3(THREADS), 0, s, p.args);
    else if (p.pick == 256) hipLaunchKernelGGL((layer_kernel<E, FORM, OUT, 256>), grid(CUS), dim3(THREADS), 0, s, p.args);
    return hipGetLastError();
}

template <class E, int FORM, class OUT>
hipError_t layer_as(const LayerArgs& a, hipStream_t s) {
    if (a.m == 0 || a.n == 0) return hipSuccess;
    const Plan all = plan<E, FORM>(a);
    if constexpr (b_across<FORM>)
        if (all.pick < 0) {
            LayerArgs any = a;
            const int64_t n = count_tiles<pair<FORM>>(any, ANY, ANY);
            hipLaunchKernelGGL((layer_any_kernel<FORM, OUT>), dim3((unsigned)std::min<int64_t>((n + NUM_XCD - 1) / NUM_XCD * NUM_XCD, 2 * CUS)), dim3(ANY_THREADS), 0, s, any);
            return hipGetLastError();
        }
    // Without segments the tiles' last round may leave most CUs idle: then the rows of the whole rounds go first, and the others in a
    // launch of their own, in what suits them (two products of 5632 x 2048 over 8191 in 352 tiles: 417 us in one launch, 379 in 256
    // tiles and 192 of 128 rows).
    if (a.mode == MUON_PRODUCT_DENSE && all.cost.tiles > CUS) {
        LayerArgs first = a, rest = a;
        const int64_t n = count_tiles<pair<FORM>>(first, TILE, FORM == FORM_GATED ? TILE / 2 : TILE);
        const int64_t rows = n / CUS * CUS / (pair<FORM> * first.tiles_n) * TILE;
        if (rows > 0 && rows < a.m) {
            first.m = rows;
            rest.m = a.m - rows;
            for (int i = 0; i < 2; ++i)
                if (rest.a[i]) rest.a[i] += a_across<FORM> ? rows * 2 : rows * rest.lda;
            for (int i = 0; i < 3; ++i)
                if (rest.out[i]) rest.out[i] = static_cast<OUT*>(rest.out[i]) + rows * rest.ld_out[FORM == FORM_GATED && i ? 1 : 0];
            if (sizeof(E) == 1) rest.sa += rows;
            const Plan one = plan<E, FORM>(first), two = plan<E, FORM>(rest);
            if (one.cost.us + two.cost.us + 2.0 < all.cost.us) {
                const hipError_t error = launch<E, FORM, OUT>(one, s);
                return error != hipSuccess ? error : launch<E, FORM, OUT>(two, s);
            }
        }
    }
    return launch<E, FORM, OUT>(all, s);
}

}  // namespace

// (the kernel that takes any size of a form)
bool layer_fits(LayerArgs a, LayerForm form) {
    return (form == FORM_GRAD_W ? count_tiles<2>(a, ANY, ANY) : form == FORM_GRAD_X ? count_tiles<1>(a, ANY, ANY) : count_tiles<1>(a, 32, 32)) >= 0;
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
