// 8-bit products with a power-of-two scale for each block of 128 (gfx950 matrix cores).
//
//     out[i][j] = sum over blocks kb of 2^(ea[i][kb] + eb[j][kb]) * sum over k in kb of a[i][k] b[j][k].
//
// v_mfma_scale_f32_32x32x64_f8f6f4 multiplies 32 rows by 32 rows over 64 values of k, half a
// block, and takes both scale exponents as bytes, so scaling costs no instruction and the
// sum over blocks stays in the float32 accumulators.  A lane supplies 32 values of one row and that
// row's scale; which 32 of the 64 is free as long as both operands agree, as all of them share the scale.
// b's rows are the instruction's first operand: a lane then holds runs of 4 consecutive columns
// of one row of out.
//
// That instruction adds 8 products at a time after shifting them to the largest one's exponent, and drops
// what falls below 2^-13 of it (measured: 256 * 256 - 256 * 256 + 1 is 0 within such a group and 1 across
// groups).  It is the choice for a bfloat16 out: codes of 4 bits leave a product uncertain by 2^-4 of itself, 70 times
// the 7 * 2^-13 that its 7 neighbours may lose, and of sums of normal values 1.4e-5 is lost, where bfloat16's half step
// is 3.9e-3.  But where a group's largest products cancel, its small ones are gone.  So full float32 sums can be asked for
// (full_sums), and a float32 out, which is there to go on being added up, always has them: the codes become
// bfloat16 values (exact, the scale included) and v_mfma_f32_32x32x16_bf16 adds them up, at half the rate (16381 x 5632 x 2048
// to bfloat16: 178 us and 351; 57344 rows of 128 experts: 296 and 589; 112 rows of 512, bound by memory: 96 and 92).
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "device_common.h"
#include "experts.h"
#include "fp8_panel.h"

namespace muon {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
// in rows of out that need not begin on a 16-byte boundary
typedef f32x4 f32x4_any __attribute__((aligned(4)));
typedef i32x4 i32x4_any __attribute__((aligned(2)));
typedef uint2 uint2_any __attribute__((aligned(2)));

constexpr int NUM_XCD = 8, CUS = 256;
constexpr int KB = 128;                   // values that share a scale

// Bands of BAND tile rows, each walked column by column: the tiles an XCD runs at once share panels.
constexpr int BAND = 8;
__device__ __forceinline__ void band_decode(int t, int tm, int tn, int& ti, int& tj) {
    const int band = t / (BAND * tn);
    const int r0 = band * BAND;
    const int rows = min(BAND, tm - r0);
    const int w = t - band * BAND * tn;
    tj = w / rows;
    ti = r0 + (w - tj * rows);
}

__device__ __forceinline__ const uint8_t* uniform(const uint8_t* p) {
    const uint64_t v = (uint64_t)p;
    const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v), hi = __builtin_amdgcn_readfirstlane((uint32_t)(v >> 32));
    return (const uint8_t*)(((uint64_t)hi << 32) | lo);
}

// 4 bytes a lane from the buffer at offset + soffset to lds_base + 4 * lane; past the buffer's end zeros arrive.
// The compiler does not track the load; loads end in order, so waiting for a later one covers it.
__device__ __forceinline__ void load_dword_to_lds(__amdgpu_buffer_rsrc_t buf, int offset, int soffset, const uint32_t* lds_base) {
    const uint32_t base = __builtin_amdgcn_readfirstlane(
        (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) uint32_t*)lds_base);
    asm volatile("s_mov_b32 m0, %3\n\ts_nop 0\n\tbuffer_load_dword %0, %1, %2 offen lds"
                 : : "v"(offset), "s"(buf), "s"(soffset), "s"(base) : "memory", "m0");
}

// 8 codes (two dwords) times the scale as bfloat16.
template <int FMT>
__device__ __forceinline__ bf16x8 widen(int lo, int hi, float scale) {
    if constexpr (FMT == MUON_FP8_E4M3) {
        const auto a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, false);
        const auto b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, true);
        const auto c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, false);
        const auto d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, true);
        return bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
    } else {
        const auto a = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(lo, scale, false);
        const auto b = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(lo, scale, true);
        const auto c = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(hi, scale, false);
        const auto d = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(hi, scale, true);
        return bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
    }
}

// Keeps the matrix instructions that have written acc so far in front of what follows: the compiler would
// move them past a branch to where their results are used.
template <int FM, int FN>
__device__ __forceinline__ void pin(f32x16 (&acc)[FM][FN]) {
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) asm volatile("" : "+v"(acc[i][j]));
}

constexpr int WAVES = 8, THREADS = 64 * WAVES;

struct Tile {
    int64_t m0, n0;            // first row of a, of b
    int rows_a, rows_b;        // rows of either inside the tile
    int group, kb0, kb1;       // blocks of k [kb0, kb1)
};

// Whether a depth-grouped launch deals every group's tiles to all XCDs (see Walk): where that leaves an XCD 8 of them,
// which share operand panels, and workgroups have several tiles.
__device__ __forceinline__ bool in_parts(const ProductArgs& p) {
    return p.mode == MUON_PRODUCT_DEPTH && p.tiles_m * p.tiles_n >= 8 * NUM_XCD && p.tiles > (int)gridDim.x;
}

// The segments' bounds, clamped to the operand, and in ends how many tile rows lie before each segment (rows-grouped),
// or the groups in the order of falling depth (depth-grouped), into LDS, by the whole workgroup.
constexpr int SORT_MAX_GROUPS = 256;      // each thread compares with every group; many groups even out by themselves
__device__ __forceinline__ void read_segments(const ProductArgs& p, int tile_rows, int* bounds, int* ends, int64_t* wave_tot) {
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int64_t limit = p.mode == MUON_PRODUCT_ROWS ? p.m : (p.k + KB - 1) / KB * KB;
    for (int g = tid; g <= p.groups; g += THREADS) bounds[g] = (int)min(max((int64_t)p.offsets[g], (int64_t)0), limit);
    if (tid == 0 && p.mode == MUON_PRODUCT_ROWS) ends[0] = 0;
    __syncthreads();
    if (p.mode != MUON_PRODUCT_ROWS) {
        auto depth = [&](int g) { return bounds[g + 1] / KB - bounds[g] / KB; };
        for (int g = tid; g < p.groups; g += THREADS) {
            int before = g;
            if (in_parts(p) && p.groups <= SORT_MAX_GROUPS) {
                before = 0;
                const int mine = depth(g);
                for (int h = 0; h < p.groups; ++h) {
                    const int other = depth(h);
                    before += other > mine || (other == mine && h < g);
                }
            }
            ends[before] = g;
        }
        __syncthreads();
        return;
    }
    // sums in 64 bits and capped: falling offsets, which are not allowed, must not lead outside the operand either
    int64_t before = 0;
    for (int g0 = 0; g0 < p.groups; g0 += THREADS) {
        const int g = g0 + tid;
        int64_t inc = g < p.groups ? ((int64_t)max(bounds[g + 1] - bounds[g], 0) + tile_rows - 1) / tile_rows : 0;
#pragma unroll
        for (int off = 1; off < 64; off <<= 1) {
            const int64_t o = __shfl_up(inc, off, 64);
            if (lane >= off) inc += o;
        }
        if (lane == 63) wave_tot[wave] = inc;
        __syncthreads();
        int64_t total = 0;
        for (int w = 0; w < WAVES; ++w) {
            if (w < wave) inc += wave_tot[w];
            total += wave_tot[w];
        }
        if (g < p.groups) ends[g + 1] = (int)min(before + inc, (int64_t)1 << 30);
        before += total;
        __syncthreads();
    }
}

// Tile t of the launch, of up to tile_rows x tile_cols.
__device__ __forceinline__ Tile decode(const ProductArgs& p, int t, int tile_rows, int tile_cols, const int* bounds,
                                       const int* ends) {
    auto at = [](const int* v) { return __builtin_amdgcn_readfirstlane(*v); };
    Tile r;
    r.group = 0;
    r.kb0 = 0;
    r.kb1 = (int)((p.k + KB - 1) / KB);
    int64_t m1 = p.m;
    int tm, tn;
    if (p.mode == MUON_PRODUCT_ROWS) {
        tm = t / p.tiles_n;
        tn = t - tm * p.tiles_n;
        int lo = 0, hi = p.groups;                         // the last g with ends[g] <= tm
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (at(ends + mid) <= tm) lo = mid;
            else hi = mid;
        }
        r.group = lo;
        r.m0 = at(bounds + lo) + (int64_t)(tm - at(ends + lo)) * tile_rows;
        m1 = at(bounds + lo + 1);
    } else {
        if (p.mode == MUON_PRODUCT_DEPTH) {
            const int per = p.tiles_m * p.tiles_n, nth = t / per;
            t -= nth * per;
            r.group = at(ends + nth);
            r.kb0 = at(bounds + r.group) / KB;
            r.kb1 = max(at(bounds + r.group + 1) / KB, r.kb0);
        }
        band_decode(t, p.tiles_m, p.tiles_n, tm, tn);
        r.m0 = (int64_t)tm * tile_rows;
    }
    r.n0 = (int64_t)tn * tile_cols;
    r.rows_a = (int)min(m1 - r.m0, (int64_t)tile_rows);
    r.rows_b = (int)min(p.n - r.n0, (int64_t)tile_cols);
    return r;
}

// A workgroup's tiles.  Workgroups are dealt to the XCDs in turn.  Each XCD takes a contiguous share of the tiles and its
// workgroups walk it together, so that the tiles that run at once share operand panels in its L2.
//
// Depth-grouped, tiles of different groups take different times.  In parts, each XCD takes an eighth of every group's
// tiles, the deepest group first, and its workgroups walk them to and fro: 8 groups of 1024 x 4096 over 9000 in
// float32 82 us against 104, 64 groups 390 against 406; with one tile in a part the shared panels are lost (128 groups of
// 512 x 1024: 57 us against 42).
struct Walk {
    int pos, last, step, turn; // tile or place in the XCD's share, its end, step; to and fro: a step's other length
    int chunk, chunks;         // tiles of a group in a part, parts of a group; 0 without parts
};
__device__ __forceinline__ Walk walk(const ProductArgs& p, const int* ends) {
    const int xcd = blockIdx.x % NUM_XCD, nth = blockIdx.x / NUM_XCD, all = gridDim.x / NUM_XCD;
    if (in_parts(p)) {
        const int per = p.tiles_m * p.tiles_n;
        const int chunk = (per + NUM_XCD - 1) / NUM_XCD, chunks = (per + chunk - 1) / chunk;
        const int mine = (p.groups * chunks - xcd + NUM_XCD - 1) / NUM_XCD;
        return {nth, mine * chunk, 2 * (all - nth) - 1, 2 * nth + 1, chunk, chunks};
    }
    int total = p.tiles;
    if (p.mode == MUON_PRODUCT_ROWS)
        total = (int)min((int64_t)__builtin_amdgcn_readfirstlane(ends[p.groups]) * p.tiles_n, (int64_t)p.tiles);
    const int share = total / NUM_XCD, rest = total % NUM_XCD;
    const int first = xcd * share + min(xcd, rest);
    return {first + nth, first + share + (xcd < rest ? 1 : 0), all, all, 0, 0};
}
// The tile at the walk's place or the next one that has one, which the walk is put past; -1 at the end.
__device__ __forceinline__ int next_tile(const ProductArgs& p, Walk& w) {
    while (w.pos < w.last) {
        const int at = w.pos, step = w.step;
        w.pos += step;
        w.step = w.turn;
        w.turn = step;
        if (w.chunk == 0) return at;
        // part q of all groups' parts is the XCD's q / 8-th; the last part of a group may be short
        const int q = at / w.chunk * NUM_XCD + blockIdx.x % NUM_XCD, group = q / w.chunks;
        const int t = (q - group * w.chunks) * w.chunk + at % w.chunk, per = p.tiles_m * p.tiles_n;
        if (t < per) return group * per + t;
    }
    return -1;
}

// ---- 256 x 256 tiles ----------------------------------------------------------------------
//
// One workgroup of 8 waves per CU that goes through its share of the tiles.  Wave (h, c) of 2 x 4 takes the 32-row
// blocks 2 i + h and columns 64 c .. 64 c + 63, so that a tile with fewer rows (a segment's end) leaves both
// wave rows half of what there is: a wave runs its first NB of 4 row blocks.
constexpr int TILE = 256;
constexpr int FM = 4, FN = 2;                             // 32 x 32 blocks of a wave

template <int N>
using ic = std::integral_constant<int, N>;

// A step is one block of k.  Operands go global -> VGPR -> LDS: while a step is multiplied from one of two LDS
// stages, the next one's registers are stored to the other stage and at once loaded again for the
// step after it.  (A lone 256 x 256 tile of depth 16384 takes 133 us this way and 152
// with loads straight to LDS; the matrix instructions alone would take 121.)
// Rows are 144 bytes apart in LDS: the 16 rows that a fragment read touches fall on 16 different 16-byte slots of the
// 256 bytes that LDS serves at once, and every read is one address plus a constant.
//
// A step has two sub-steps of 64 values.  Its one barrier comes in the middle of the second, whose fragments are then in
// registers: past it the next stage is complete and this one may be overwritten.  The matrix instructions
// before it cover the fragment reads that it waits for, those behind it the next stage's first reads.
//
// 16381 x 5632 x 2048 in bfloat16: 170 us, 2.2 PFLOP/s; 8192 x 8192 x 8320: 2.5.  57344 rows of 128 experts, 1024 x 4096:
// 274-282 us.  Weight gradients of 64 experts, 1024 x 4096 in float32 over 28672 rows: 398 us, about 140 of products and
// 200 of stores (1.07 GB), one after the other: a wave's loads and stores retire in order.
// All 256 registers of a lane are taken: accumulators 128, staged operands 32, fragments 48 or 64, scales 6, addresses.  14 values
// (20 for PRECISE) that a tile's beginning and end use spill to scratch, before and behind the main loops: inside there is
// no scratch access, which would wait for the staged loads.
//
// PRECISE: full float32 sums, by the bfloat16 instruction.
template <int AFMT, class OUT, bool PRECISE>
__global__ __launch_bounds__(THREADS) __attribute__((amdgpu_waves_per_eu(2, 2))) void product_kernel(ProductArgs p) {
    constexpr bool F32 = sizeof(OUT) == 4;
    constexpr int LA = TILE / 64, NLOAD = 2 * LA;          // load instructions of a step: 64 rows each
    constexpr int ROW = 144, PANEL = TILE * ROW, STAGE = 2 * PANEL;
    constexpr int EPL = 16 / sizeof(OUT);                  // values of out in 16 bytes
    constexpr int OROW = 64 * sizeof(OUT) + 16;            // a row of out in LDS
    static_assert(WAVES * 32 * OROW <= STAGE, "out goes through one stage");
    __shared__ __attribute__((aligned(1024))) uint8_t smem[2 * STAGE];
    __shared__ __attribute__((aligned(1024))) uint32_t scale_words[2][2 * TILE];
    __shared__ int bounds[MUON_MAX_EXPERTS + 1], ends[MUON_MAX_EXPERTS + 1];
    __shared__ int64_t wave_tot[WAVES];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wh = wave >> 2, wn = (wave & 3) * 64;        // wave row; first column
    const int fr = lane & 31, fk = lane >> 5;
    const int kp = (int)((p.k + KB - 1) / KB) * KB, sp = (kp / KB + 3) / 4 * 4;

    if (p.mode != MUON_PRODUCT_DENSE) read_segments(p, TILE, bounds, ends, wave_tot);
    Walk my = walk(p, ends);
    int t = next_tile(p, my);
    if (t < 0) return;

    // staging: load d of wave w brings rows 8 w + 64 i + lane / 8 of an operand
    const int lrow = 8 * wave + (lane >> 3), lchunk = lane & 7;
    const int32_t va = Panel::lane(lrow, lchunk, (int)p.lda), vb = Panel::lane(lrow, lchunk, (int)p.ldb);
    const int wst = lrow * ROW + 16 * lchunk;

    const uint8_t *abase, *bbase, *scale_base;
    int bytes_a, bytes_b, scale_bytes, vs, s0, s1;
    i32x4 staged[NLOAD];
    // Chunk d of a step into its register.  keep is -1, or 0 past the last step: then from an empty buffer, which
    // fetches nothing (a branch in the main loop would let the compiler move the matrix instructions behind it).
    auto load = [&](int d, int step, int keep) {
        const int i = d < LA ? d : d - LA;
        int32_t rows_on = Panel::rows(64 * i, (int)(d < LA ? p.lda : p.ldb));
        asm volatile("" : "+s"(rows_on));                  // added here, or the sums of all d stay in registers
        const int32_t of_row = (d < LA ? va : vb) + rows_on;
        const int32_t of_block = Panel::block(step) & keep;
        const __amdgpu_buffer_rsrc_t buf = __builtin_amdgcn_make_buffer_rsrc(
            (void*)(d < LA ? abase : bbase), 0, (d < LA ? bytes_a : bytes_b) & keep, 0x00020000);
        staged[d] = __builtin_amdgcn_raw_buffer_load_b128(buf, of_row, of_block, 0);
    };
    auto mask = [](bool valid) {
        int keep = __builtin_amdgcn_readfirstlane(valid ? -1 : 0);
        asm volatile("" : "+s"(keep));
        return keep;
    };
    auto store = [&](int d, int st) {
        const int i = d < LA ? d : d - LA;
        *reinterpret_cast<i32x4*>(smem + st * STAGE + (d < LA ? 0 : PANEL) + 64 * ROW * i + wst) = staged[d];
    };
    // Scales, a word of 4 blocks' bytes per row of the tile (a's rows, then b's; wave w brings 64 of them), go through
    // LDS, two groups of 4 blocks in turn.
    auto load_scales = [&](int g, bool valid) {
        load_dword_to_lds(__builtin_amdgcn_make_buffer_rsrc((void*)scale_base, 0, valid ? scale_bytes : 0, 0x00020000), vs,
                          valid ? 4 * g : 0, &scale_words[g & 1][64 * wave]);
    };
    uint32_t ea[FM], eb[FN];
    auto read_scales = [&](int g) {
#pragma unroll
        for (int i = 0; i < FM; ++i) ea[i] = scale_words[g & 1][64 * i + 32 * wh + fr];
#pragma unroll
        for (int j = 0; j < FN; ++j) eb[j] = scale_words[g & 1][TILE + wn + 32 * j + fr];
    };
    // The tile's operands, and the first loads of them.
    auto begin = [&](const Tile& x) {
        int ln = lane;
        asm volatile("" : "+v"(ln));                       // as in write
        const bool per_group = p.mode == MUON_PRODUCT_ROWS;
        abase = p.a + x.m0 * p.lda;
        bbase = p.b + (per_group ? x.group * p.stride_b : 0) + x.n0 * p.ldb;
        bytes_a = Panel::bytes(x.rows_a, (int)p.lda, kp);
        bytes_b = Panel::bytes(x.rows_b, (int)p.ldb, kp);
        const bool is_a = wave < WAVES / 2;
        const int64_t r0 = is_a ? x.m0 : x.n0, sh = is_a ? p.shift_a : p.shift_b;
        const int ld = (int)(is_a ? p.ldas : p.ldbs), last = (is_a ? x.rows_a : x.rows_b) - 1;
        const int64_t base = r0 >> sh;
        vs = (int)(((r0 + min((64 * wave) % TILE + ln, last)) >> sh) - base) * ld;
        scale_bytes = __builtin_amdgcn_readfirstlane((int)(((r0 + last) >> sh) - base) * ld + sp);
        scale_base = uniform((is_a ? p.as : p.bs + (per_group ? x.group * p.stride_bs : 0)) + base * ld);
        s0 = __builtin_amdgcn_readfirstlane(x.kb0);
        s1 = __builtin_amdgcn_readfirstlane(x.kb1);
        load_scales(x.kb0 >> 2, s0 < s1);
        load_scales((x.kb0 >> 2) + 1, ((x.kb0 >> 2) + 1) * 4 < x.kb1);
#pragma unroll
        for (int d = 0; d < NLOAD; ++d) load(d, s0, mask(s0 < s1));
    };

    // fragments of sub-step kk: 32 codes of a row
    auto fragment = [&](const uint8_t* row, int kk) {
        const i32x4 lo = *reinterpret_cast<const i32x4*>(row + 64 * kk);
        const i32x4 hi = *reinterpret_cast<const i32x4*>(row + 64 * kk + 16);
        return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    };
    const int ra = (32 * wh + fr) * ROW + 32 * fk, rb = PANEL + (wn + fr) * ROW + 32 * fk;
    auto read_a = [&](int i, int st, int kk) { return fragment(smem + st * STAGE + ra + 64 * i * ROW, kk); };
    auto read_b = [&](int j, int st, int kk) { return fragment(smem + st * STAGE + rb + 32 * j * ROW, kk); };

    f32x16 acc[FM][FN];
    // The steps of a tile for a wave with NB row blocks.
    auto multiply = [&](auto nb_) {
        constexpr int NB = decltype(nb_)::value;
        // slots of a sub-step: groups of matrix instructions that staging and reads go behind; the barrier comes
        // before slot BAR of the second
        constexpr int SLOTS = PRECISE ? 4 * NB : NB * FN, BAR = PRECISE ? 2 * NB : NB / 2 * FN, HALF = NB / 2;
        read_scales(s0 >> 2);
        i32x8 fa[NB], fb[2][FN];                           // a's are refilled in place, b's alternate
#pragma unroll
        for (int i = 0; i < NB; ++i) fa[i] = read_a(i, 0, 0);
#pragma unroll
        for (int j = 0; j < FN; ++j) fb[0][j] = read_b(j, 0, 0);
        for (int step = s0; step < s1; ++step) {
            const int ahead = mask(step + 2 < s1);
            const int st = (step - s0) & 1, st_next = st ^ 1;
            const int sh = 8 * (step & 3);
#pragma unroll
            for (int kk = 0; kk < 2; ++kk) {
                const int cur = kk, nxt = kk ^ 1;
                const bool last = kk == 1;
                const int rst = last ? st_next : st;
                auto turn = [&]() {                          // the barrier of a step, and the scales of the next
                    pin(acc);
                    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
                    __builtin_amdgcn_s_barrier();
                    asm volatile("" ::: "memory");
                    if (((step + 1) & 3) == 0) {
                        // this sub-step has its exponents, and the words of the group before last are free
                        const int g = (step + 1) >> 2;
                        read_scales(g);
                        load_scales(g + 1, (g + 1) * 4 < s1);
                    }
                };
                auto stage = [&](int f) {                    // this slot's share of the staging, before the barrier
                    constexpr int ALL = SLOTS + BAR;
                    if (last && f >= BAR) return;
                    const int g = kk * SLOTS + f;
#pragma unroll
                    for (int d = g * NLOAD / ALL; d < (g + 1) * NLOAD / ALL; ++d) {
                        store(d, st_next);
                        load(d, step + 2, ahead);
                    }
                };
                if constexpr (PRECISE) {
                    float xa[NB], xb[FN];
#pragma unroll
                    for (int i = 0; i < NB; ++i) xa[i] = __uint_as_float(((ea[i] >> sh) & 255u) << 23);
#pragma unroll
                    for (int j = 0; j < FN; ++j) xb[j] = __uint_as_float(((eb[j] >> sh) & 255u) << 23);
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        if (last && q == 2) turn();
                        bf16x8 wb[FN];
#pragma unroll
                        for (int j = 0; j < FN; ++j)
                            wb[j] = widen<MUON_FP8_E4M3>(fb[cur][j][2 * q], fb[cur][j][2 * q + 1], xb[j]);
#pragma unroll
                        for (int i = 0; i < NB; ++i) {
                            const bf16x8 wa = widen<AFMT>(fa[i][2 * q], fa[i][2 * q + 1], xa[i]);
                            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                            for (int j = 0; j < FN; ++j)
                                acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(wb[j], wa, acc[i][j], 0, 0, 0);
                            __builtin_amdgcn_sched_barrier(0);
                            stage(q * NB + i);
                            if (q == 2 && i == 0)
#pragma unroll
                                for (int j = 0; j < FN; ++j) fb[nxt][j] = read_b(j, rst, nxt);
                            if (q == 3) fa[i] = read_a(i, rst, nxt);
                        }
                    }
                } else {
                    int xa[NB], xb[FN];
#pragma unroll
                    for (int i = 0; i < NB; ++i) xa[i] = (int)(ea[i] >> sh);
#pragma unroll
                    for (int j = 0; j < FN; ++j) xb[j] = (int)(eb[j] >> sh);
#pragma unroll
                    for (int i = 0; i < NB; ++i) {
                        if (last && i == HALF) turn();
#pragma unroll
                        for (int j = 0; j < FN; ++j) {
                            __builtin_amdgcn_sched_barrier(0);
                            acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(fb[cur][j], fa[i], acc[i][j], 0, AFMT, 0,
                                                                                        xb[j], 0, xa[i]);
                            __builtin_amdgcn_sched_barrier(0);
                            stage(i * FN + j);
                            if (i == (last ? HALF : 0)) {
                                fb[nxt][j] = read_b(j, rst, nxt);
                                if (last && j < HALF) fa[j] = read_a(j, rst, nxt);
                            }
                            if (j == FN - 1 && (!last || i >= HALF)) fa[i] = read_a(i, rst, nxt);
                        }
                    }
                }
            }
        }
    };

    // The first step into LDS, the second into the registers.
    auto fill = [&]() {
        if (s0 >= s1) return;
#pragma unroll
        for (int d = 0; d < NLOAD; ++d) {
            store(d, 0);
            load(d, s0 + 1, mask(s0 + 1 < s1));
        }
    };
    // Row block i of out: 32 rows x 64 columns of the wave through its part of the second stage (which nobody reads
    // between a tile's last barrier and the next one's first step), then in 16-byte stores along the rows, which leave
    // the caches to the operands (64 weight gradients of 1024 x 4096 over 512 each: 193 us against 295).
    OUT* out;
    Tile done;
    auto write = [&](int i) {
        // opaque, so that the addresses are worked out per tile instead of being kept through the main loop
        int ln = lane;
        asm volatile("" : "+v"(ln));
        uint8_t* mine = smem + STAGE + wave * 32 * OROW;
        const int r0 = 64 * i + 32 * wh;
        if (r0 >= done.rows_a) return;
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                uint8_t* o = mine + (ln & 31) * OROW + (32 * j + 8 * q + 4 * (ln >> 5)) * sizeof(OUT);
                const f32x4 v = {acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
                if constexpr (F32) *reinterpret_cast<f32x4*>(o) = v;
                else *reinterpret_cast<uint2*>(o) = make_uint2(dev::f32x2_to_bf16x2(v[0], v[1]), dev::f32x2_to_bf16x2(v[2], v[3]));
            }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        constexpr int LPR = 64 / EPL, RPS = 64 / LPR;      // lanes per row, rows per store
        const int col = ln % LPR * EPL, row = ln / LPR;
        const int64_t left = p.n - done.n0 - wn - col;     // columns of out from the lane's first
        OUT* o = out + (done.m0 + r0 + row) * p.ld_out + done.n0 + wn + col;
#pragma unroll
        for (int q = 0; q < 32 / RPS; ++q, o += RPS * p.ld_out) {
            const uint4 w = *reinterpret_cast<const uint4*>(mine + (q * RPS + row) * OROW + col * sizeof(OUT));
            if (r0 + q * RPS + row >= done.rows_a) continue;
            if (EPL <= left) {
                if constexpr (F32) {
                    f32x4 v = __builtin_bit_cast(f32x4, w);
                    if (p.accumulate) v += *reinterpret_cast<const f32x4_any*>(o);
                    if (p.vec) __builtin_nontemporal_store(v, reinterpret_cast<f32x4*>(o));
                    else *reinterpret_cast<f32x4_any*>(o) = v;
                } else {
                    if (p.vec) __builtin_nontemporal_store(__builtin_bit_cast(i32x4, w), reinterpret_cast<i32x4*>(o));
                    else *reinterpret_cast<i32x4_any*>(o) = __builtin_bit_cast(i32x4, w);
                }
            } else {
                const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int e = 0; e < EPL; ++e) {
                    if (e >= left) continue;
                    if constexpr (F32) o[e] = p.accumulate ? o[e] + __uint_as_float(u[e]) : __uint_as_float(u[e]);
                    else o[e] = (uint16_t)(u[e / 2] >> (16 * (e & 1)));
                }
            }
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
    };

    Tile x = decode(p, t, TILE, TILE, bounds, ends);
    begin(x);
    fill();
    for (;;) {
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
            for (int j = 0; j < FN; ++j)
#pragma unroll
                for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.f;
        if (s0 < s1) {
            asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
            const int blocks = (x.rows_a - 32 * wh + 63) / 64;
            if (blocks >= 4) multiply(ic<4>{});
            else if (blocks == 3) multiply(ic<3>{});
            else if (blocks == 2) multiply(ic<2>{});
            else multiply(ic<1>{});
        }
        done = x;
        out = static_cast<OUT*>(p.out) + (p.mode == MUON_PRODUCT_DEPTH ? done.group * p.out_stride : 0);
        t = next_tile(p, my);
        const bool more = t >= 0;
        // the next tile's first loads run beside this one's stores
        if (more) {
            x = decode(p, t, TILE, TILE, bounds, ends);
            begin(x);
        }
        write(0);
        write(1);
        if (more) fill();
        write(2);
        write(3);
        if (!more) break;
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");      // the scale words' loads write LDS
}

// ---- few tiles: 32 x 64 or 32 x 16, depth split over the waves ---------------------------------
//
// Where 256 x 256 tiles would leave most of the chip idle.  Each of 8 waves takes every eighth block of k of a tile of
// 32 rows of a by 16 NB rows of b, its fragments (v_mfma_scale_f32_16x16x128_f8f6f4: a block at once) straight from
// memory into registers, AHEAD blocks at a time, so that a tile's loads are under way together; the waves' sums are
// added up through LDS in the order of the waves.  Bound by the loads' latency, then by L2 (16 rows by 4096 x 4096: 6 us
// of kernel; 256 rows: 30 us).
constexpr int FEW_ROWS = 32;

template <int AFMT, class OUT, bool PRECISE, int NB, int AHEAD>
__global__ __launch_bounds__(THREADS) void product_few_kernel(ProductArgs p) {
    constexpr bool F32 = sizeof(OUT) == 4;
    constexpr int COLS = 16 * NB, SUMS = COLS + 4;         // columns of a tile; a row of sums in LDS
    __shared__ __attribute__((aligned(16))) float sums[WAVES][FEW_ROWS * SUMS];
    __shared__ int bounds[MUON_MAX_EXPERTS + 1], ends[MUON_MAX_EXPERTS + 1];
    __shared__ int64_t wave_tot[WAVES];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int fr = lane & 15, fk = lane >> 4;
    if (p.mode != MUON_PRODUCT_DENSE) read_segments(p, FEW_ROWS, bounds, ends, wave_tot);
    Walk my = walk(p, ends);
    for (int t = next_tile(p, my); t >= 0; t = next_tile(p, my)) {
        const Tile x = decode(p, t, FEW_ROWS, COLS, bounds, ends);
        const bool per_group = p.mode == MUON_PRODUCT_ROWS;
        // offsets of the lane's rows from the tile's first; rows past the end repeat the last: their sums are not stored
        const uint8_t* abase = p.a + x.m0 * p.lda;
        const uint8_t* bbase = p.b + (per_group ? x.group * p.stride_b : 0) + x.n0 * p.ldb;
        const int64_t sa0 = x.m0 >> p.shift_a, sb0 = x.n0 >> p.shift_b;
        const uint8_t* as = p.as + sa0 * p.ldas;
        const uint8_t* bs = p.bs + (per_group ? x.group * p.stride_bs : 0) + sb0 * p.ldbs;
        uint32_t oa[2], sa[2], ob[NB], sb[NB];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int r = min(16 * i + fr, x.rows_a - 1);
            oa[i] = (uint32_t)r * (uint32_t)p.lda + 32 * fk;
            sa[i] = (uint32_t)(((x.m0 + r) >> p.shift_a) - sa0) * (uint32_t)p.ldas;
        }
#pragma unroll
        for (int j = 0; j < NB; ++j) {
            const int r = min(16 * j + fr, x.rows_b - 1);
            ob[j] = (uint32_t)r * (uint32_t)p.ldb + 32 * fk;
            sb[j] = (uint32_t)(((x.n0 + r) >> p.shift_b) - sb0) * (uint32_t)p.ldbs;
        }
        auto codes = [](const uint8_t* at) {
            const i32x4 lo = *reinterpret_cast<const i32x4*>(at), hi = *reinterpret_cast<const i32x4*>(at + 16);
            return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
        };
        f32x4 acc[2][NB];
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < NB; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
        // U blocks from kb0 on, all of them there
        auto blocks = [&](auto u_, int kb0) {
            constexpr int U = decltype(u_)::value;
            i32x8 fa[U][2], fb[U][NB];
            int ea[U][2], eb[U][NB];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int kb = kb0 + u * WAVES;
                const int64_t k = (int64_t)kb * KB;
#pragma unroll
                for (int j = 0; j < NB; ++j) {
                    fb[u][j] = codes(bbase + k + ob[j]);
                    eb[u][j] = bs[sb[j] + kb];
                }
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    fa[u][i] = codes(abase + k + oa[i]);
                    ea[u][i] = as[sa[i] + kb];
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if constexpr (PRECISE) {
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        bf16x8 wa[2];
#pragma unroll
                        for (int i = 0; i < 2; ++i)
                            wa[i] = widen<AFMT>(fa[u][i][2 * q], fa[u][i][2 * q + 1], __uint_as_float((uint32_t)ea[u][i] << 23));
#pragma unroll
                        for (int j = 0; j < NB; ++j) {
                            const bf16x8 wb = widen<MUON_FP8_E4M3>(fb[u][j][2 * q], fb[u][j][2 * q + 1], __uint_as_float((uint32_t)eb[u][j] << 23));
#pragma unroll
                            for (int i = 0; i < 2; ++i) acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wb, wa[i], acc[i][j], 0, 0, 0);
                        }
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 2; ++i)
#pragma unroll
                        for (int j = 0; j < NB; ++j)
                            acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fb[u][j], fa[u][i], acc[i][j], 0, AFMT, 0, eb[u][j], 0, ea[u][i]);
                }
            }
        };
        int kb = x.kb0 + wave;
        for (; kb + (AHEAD - 1) * WAVES < x.kb1; kb += AHEAD * WAVES) blocks(ic<AHEAD>{}, kb);
        for (; kb < x.kb1; kb += WAVES) blocks(ic<1>{}, kb);
        // a lane's sums are rows 16 i + fr, columns 16 j + 4 fk + (0 .. 3)
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < NB; ++j) *reinterpret_cast<f32x4*>(&sums[wave][(16 * i + fr) * SUMS + 16 * j + 4 * fk]) = acc[i][j];
        __syncthreads();
        if (tid < FEW_ROWS * COLS / 4) {
            const int row = tid / (COLS / 4), col = 4 * (tid % (COLS / 4));
            f32x4 v = *reinterpret_cast<const f32x4*>(&sums[0][row * SUMS + col]);
#pragma unroll
            for (int w = 1; w < WAVES; ++w) v += *reinterpret_cast<const f32x4*>(&sums[w][row * SUMS + col]);
            if (row < x.rows_a) {
                OUT* o = static_cast<OUT*>(p.out) + (p.mode == MUON_PRODUCT_DEPTH ? x.group * p.out_stride : 0) +
                         (x.m0 + row) * p.ld_out + x.n0 + col;
                const int64_t left = p.n - x.n0 - col;
                if (left >= 4) {
                    if constexpr (F32) {
                        f32x4_any* o4 = reinterpret_cast<f32x4_any*>(o);
                        if (p.accumulate) v += *o4;
                        *o4 = v;
                    } else {
                        *reinterpret_cast<uint2_any*>(o) = make_uint2(dev::f32x2_to_bf16x2(v[0], v[1]), dev::f32x2_to_bf16x2(v[2], v[3]));
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        if (e >= left) continue;
                        if constexpr (F32) o[e] = p.accumulate ? o[e] + v[e] : v[e];
                        else o[e] = dev::f32_to_bf16(v[e]);
                    }
                }
            }
        }
        __syncthreads();                                   // the sums are read
    }
}

// Tiles of a launch, at most; -1 for too many.
int64_t count_tiles(ProductArgs& a, int tile_rows, int tile_cols) {
    a.tiles_n = (int32_t)((a.n + tile_cols - 1) / tile_cols);
    a.tiles_m = (int32_t)((a.m + tile_rows - 1) / tile_rows);
    // every segment may end inside a tile, but not more of them than there are rows
    int64_t rows = a.tiles_m;
    if (a.mode == MUON_PRODUCT_ROWS) rows = a.m / tile_rows + (a.m < a.groups ? a.m : (int64_t)a.groups);
    if (a.mode == MUON_PRODUCT_DEPTH) rows *= a.groups;
    const int64_t total = rows * a.tiles_n;
    if (total >= ((int64_t)1 << 31) - 2 * CUS) return -1;   // a workgroup's step past its last tile stays an int
    a.tiles = (int32_t)total;
    return total;
}

template <int AFMT, class OUT, bool PRECISE>
hipError_t product_as(ProductArgs a, hipStream_t s) {
    ProductArgs few = a, thin = a;
    const int64_t n_big = count_tiles(a, TILE, TILE), n_few = count_tiles(few, FEW_ROWS, 64), n_thin = count_tiles(thin, FEW_ROWS, 16);
    if (n_big == 0) return hipSuccess;
    // What each would take, in us, from what they measured: big tiles by the round of 256 (256 x 4096 x 4096: 38 us in
    // bfloat16, 76 with full sums), the others by the depth of a wave where there are few tiles and by the blocks of all
    // tiles where there are many.  1 row by 4096 x 4096: 26 us in big tiles, 12 in 32 x 64, 6 in 32 x 16; 256 rows: 38,
    // 30, 61; 512 rows: 40, 55, 118; 256 x 256 x 16384: 128, 52, 31; 112 rows of 512 experts, 1024 x 4096: 94, 104, 115.
    const double kb = (double)((a.k + KB - 1) / KB) / (a.mode == MUON_PRODUCT_DEPTH ? a.groups : 1);
    // (a big tile runs as many of its 4 row blocks as it has rows for: of its 64 rows each)
    const int64_t rows = a.mode == MUON_PRODUCT_ROWS ? a.m / std::min<int64_t>(a.m, a.groups) : a.m;
    const double more = (double)std::min<int64_t>((std::min<int64_t>(rows, TILE) + 63) / 64 - 1, 3) / 3.0;
    const double step = PRECISE ? 1.0 + 1.2 * more : 0.66 + 0.39 * more;
    const double t_big = std::ceil((double)n_big / CUS) * (5.0 + kb * step);
    const double t_few = n_few < 0 ? 1e30 : 5.0 + std::max(kb / WAVES * 2.5, (double)n_few * (kb + 2.0) / 590.0);
    const double t_thin = n_thin < 0 ? 1e30 : 4.0 + std::max(kb / WAVES * 1.6, (double)n_thin * (kb + 1.5) / 1150.0);
    const int pick = t_big <= std::min(t_few, t_thin) ? 0 : t_few <= t_thin ? 1 : 2;
    const int64_t total = pick == 0 ? n_big : pick == 1 ? n_few : n_thin;
    // workgroups: as many as run at once, and of 32 x 64 tiles (153 registers and more: one a CU) as many again
    const int64_t most = pick == 0 ? CUS : 2 * CUS;
    const dim3 grid((unsigned)std::min<int64_t>((total + NUM_XCD - 1) / NUM_XCD * NUM_XCD, most)), block(THREADS);
    if (pick == 0) hipLaunchKernelGGL((product_kernel<AFMT, OUT, PRECISE>), grid, block, 0, s, a);
    else if (pick == 1) hipLaunchKernelGGL((product_few_kernel<AFMT, OUT, PRECISE, 4, 2>), grid, block, 0, s, few);
    else hipLaunchKernelGGL((product_few_kernel<AFMT, OUT, PRECISE, 1, 4>), grid, block, 0, s, thin);
    return hipGetLastError();
}

}  // namespace

bool product_fits(ProductArgs a) { return count_tiles(a, TILE, TILE) >= 0; }

hipError_t launch_product(ProductArgs a, int32_t a_format, int32_t out_dtype, bool full_sums, hipStream_t s) {
    const bool e4m3 = a_format == MUON_FP8_E4M3;
    if (out_dtype == MUON_DTYPE_F32) return e4m3 ? product_as<0, float, true>(a, s) : product_as<1, float, true>(a, s);
    if (full_sums) return e4m3 ? product_as<0, uint16_t, true>(a, s) : product_as<1, uint16_t, true>(a, s);
    return e4m3 ? product_as<0, uint16_t, false>(a, s) : product_as<1, uint16_t, false>(a, s);
}

}  // namespace muon
