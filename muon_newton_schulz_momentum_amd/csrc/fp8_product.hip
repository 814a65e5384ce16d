// 8-bit products with a power-of-two scale for each block of 128 (gfx950 matrix cores).
//
//     out[i][j] = sum over blocks kb of 2^(ea[i][kb] + eb[j][kb]) * sum over k in kb of a[i][k] b[j][k].
//
// v_mfma_scale_f32_16x16x128_f8f6f4 multiplies 16 rows by 16 rows over 128 values of k, one
// block, and takes both scale exponents as bytes, so scaling costs no instruction and the
// sum over blocks stays in the float32 accumulators.  A lane supplies 32 values of one row and that
// row's scale; which 32 of the 128 is free as long as both operands agree, as all of them share the scale.
// b's rows are the instruction's first operand: a lane then holds 4 consecutive columns
// of one row of out.
//
// That instruction adds 8 products at a time after shifting them to the largest one's exponent, and drops
// what falls below 2^-13 of it (measured: 256 * 256 - 256 * 256 + 1 is 0 within such a group and 1 across
// groups): 1.4e-5 of a sum of normal values.  A bfloat16 out (half step 3.9e-3) does not see it.  A float32
// out is asked for where sums go on being added up, so there the codes become bfloat16
// values (exact, the scale included) and v_mfma_f32_16x16x32_bf16 keeps full float32 sums, at half the rate.
//
// 128 x 128 output tiles, 4 waves of 64 x 64.  Operand tiles of 128 bytes a row go from global
// memory straight to LDS, the next step's while this one is multiplied.  Row r's 16-byte
// chunk c is at c ^ ((r >> 1) & 7): the 16 rows that a fragment read touches then fall on 16
// different 16-byte slots of the 256 bytes that LDS serves at once.
#include "device_common.h"
#include "experts.h"

namespace muon {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int NUM_XCD = 8;
constexpr int TILE = 128, KB = 128;

// Consecutive tiles on one XCD (workgroups are dealt to the XCDs in turn).
__device__ __forceinline__ int xcd_remap(int b, int g) {
    const int xcd = b % NUM_XCD, local = b / NUM_XCD;
    const int q = g / NUM_XCD, r = g % NUM_XCD;
    return xcd < r ? xcd * (q + 1) + local : r * (q + 1) + (xcd - r) * q + local;
}

// 16 bytes a lane from global memory to lds_base + 16 * lane.  The compiler does not track the load;
// it is waited for with vmcnt before the barrier that publishes the stage.
__device__ __forceinline__ void load_to_lds(const uint8_t* src, const uint8_t* lds_base) {
    const uint32_t base = __builtin_amdgcn_readfirstlane(
        (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) uint8_t*)lds_base);
    asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off" : : "v"(src), "s"(base) : "memory", "m0");
}

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

// 8 codes (two dwords) times 2^(byte - 127) as bfloat16.
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

// The segment of tile row `tile` of a rows-grouped launch: segments take ceil(length / TILE) tile
// rows each, in order.  False past the last one.  Run by the whole workgroup.
__device__ __forceinline__ bool find_segment(const ProductArgs& p, int tile, int& group, int64_t& lo, int64_t& hi) {
    __shared__ int wave_tot[4], found[2];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    for (int g0 = 0; g0 < p.groups; g0 += 256) {
        const int g = g0 + tid;
        int tiles = 0;
        if (g < p.groups) {
            const int64_t s = min(max((int64_t)p.offsets[g], (int64_t)0), p.m);
            const int64_t e = min(max((int64_t)p.offsets[g + 1], s), p.m);
            tiles = (int)((e - s + TILE - 1) / TILE);
        }
        int inc = tiles;
#pragma unroll
        for (int off = 1; off < 64; off <<= 1) {
            const int o = __shfl_up(inc, off, 64);
            if (lane >= off) inc += o;
        }
        if (lane == 63) wave_tot[wave] = inc;
        __syncthreads();
        int total = 0;
        for (int w = 0; w < 4; ++w) {
            if (w < wave) inc += wave_tot[w];
            total += wave_tot[w];
        }
        if (tile < total) {
            if (tile < inc && tile >= inc - tiles) { found[0] = g; found[1] = tile - (inc - tiles); }
            __syncthreads();
            group = found[0];
            const int64_t s = min(max((int64_t)p.offsets[group], (int64_t)0), p.m);
            hi = min(max((int64_t)p.offsets[group + 1], s), p.m);
            lo = s + (int64_t)found[1] * TILE;
            return true;
        }
        tile -= total;
        __syncthreads();
    }
    return false;
}

template <int AFMT, class OUT>
__global__ __launch_bounds__(256) void product_kernel(ProductArgs p) {
    __shared__ __attribute__((aligned(1024))) uint8_t smem[2][2][TILE * KB];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int wm = (wave >> 1) * 64, wn = (wave & 1) * 64;
    const int b = xcd_remap(blockIdx.x, gridDim.x);

    // the tile: rows [m0, m1) of a, from n0 of b, blocks [kb0, kb1)
    int group = 0;
    int64_t m0, m1 = p.m;
    int kb0 = 0, kb1 = (int)((p.k + KB - 1) / KB);
    const int tn = b % p.tiles_n;
    int tm = b / p.tiles_n;
    if (p.mode == MUON_PRODUCT_ROWS) {
        if (!find_segment(p, tm, group, m0, m1)) return;
    } else {
        if (p.mode == MUON_PRODUCT_DEPTH) {
            group = tm / p.tiles_m;
            tm -= group * p.tiles_m;
            const int64_t all = (int64_t)kb1 * KB;
            const int64_t s = min(max((int64_t)p.offsets[group], (int64_t)0), all);
            const int64_t e = min(max((int64_t)p.offsets[group + 1], s), all);
            kb0 = (int)(s / KB);
            kb1 = (int)(e / KB);
        }
        m0 = (int64_t)tm * TILE;
    }
    const int64_t n0 = (int64_t)tn * TILE;
    const bool per_group = p.mode == MUON_PRODUCT_ROWS;
    const uint8_t* bq = p.b + (per_group ? group * p.stride_b : 0);
    const uint8_t* bs = p.bs + (per_group ? group * p.stride_bs : 0);

    // staging: wave w loads 8 rows a time, rows 8 (w + 4 i) of either tile; rows past the end repeat the last
    const uint8_t *ga[4], *gb[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int row = 8 * (wave + 4 * i) + (lane >> 3);
        const int chunk = (lane & 7) ^ ((row >> 1) & 7);
        ga[i] = p.a + min(m0 + row, m1 - 1) * p.lda + 16 * chunk;
        gb[i] = bq + min(n0 + row, p.n - 1) * p.ldb + 16 * chunk;
    }
    auto stage = [&](int kb, int st) {
        const int64_t k = (int64_t)kb * KB;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            load_to_lds(ga[i] + k, &smem[st][0][1024 * (wave + 4 * i)]);
            load_to_lds(gb[i] + k, &smem[st][1][1024 * (wave + 4 * i)]);
        }
    };
    // scales of the fragments' rows
    const int fr = lane & 15, fk = lane >> 4;
    const uint8_t *sa[4], *sb[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        sa[i] = p.as + (min(m0 + wm + 16 * i + fr, m1 - 1) >> p.shift_a) * p.ldas;
        sb[i] = bs + (min(n0 + wn + 16 * i + fr, p.n - 1) >> p.shift_b) * p.ldbs;
    }
    // fragment: 32 of a row's 128 bytes, chunks 2 fk and 2 fk + 1
    auto fragment = [&](const uint8_t* tile, int row) {
        const int sw = (row >> 1) & 7;
        const i32x4 lo = *reinterpret_cast<const i32x4*>(tile + row * KB + 16 * ((2 * fk) ^ sw));
        const i32x4 hi = *reinterpret_cast<const i32x4*>(tile + row * KB + 16 * ((2 * fk + 1) ^ sw));
        return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    };

    f32x4 acc[4][4];                                       // [fragment of m][fragment of n]
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

    if (kb0 < kb1) stage(kb0, 0);
    for (int kb = kb0; kb < kb1; ++kb) {
        const int st = (kb - kb0) & 1;
        int ea[4], eb[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            ea[i] = sa[i][kb];
            eb[i] = sb[i][kb];
        }
        asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
        __syncthreads();                                   // this stage is in; the other is no longer read
        if (kb + 1 < kb1) stage(kb + 1, st ^ 1);
        i32x8 fa[4], fb[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            fa[i] = fragment(smem[st][0], wm + 16 * i + fr);
            fb[i] = fragment(smem[st][1], wn + 16 * i + fr);
        }
        if constexpr (sizeof(OUT) == 4) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                bf16x8 wa[4], wb[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    wa[i] = widen<AFMT>(fa[i][2 * q], fa[i][2 * q + 1], __uint_as_float((uint32_t)ea[i] << 23));
                    wb[i] = widen<MUON_FP8_E4M3>(fb[i][2 * q], fb[i][2 * q + 1], __uint_as_float((uint32_t)eb[i] << 23));
                }
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wb[j], wa[i], acc[i][j], 0, 0, 0);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                        fb[j], fa[i], acc[i][j], 0, AFMT, 0, eb[j], 0, ea[i]);
        }
    }

    OUT* out = static_cast<OUT*>(p.out) + (p.mode == MUON_PRODUCT_DEPTH ? group * p.out_stride : 0);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t r = m0 + wm + 16 * i + fr;
        if (r >= m1) continue;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int64_t c = n0 + wn + 16 * j + 4 * fk;
            OUT* o = out + r * p.ld_out + c;
            f32x4 v = acc[i][j];
            if (p.vec && c + 4 <= p.n) {
                if constexpr (sizeof(OUT) == 4) {
                    f32x4* o4 = reinterpret_cast<f32x4*>(o);
                    if (p.accumulate) v += *o4;
                    *o4 = v;
                } else {
                    *reinterpret_cast<uint2*>(o) = make_uint2(dev::f32x2_to_bf16x2(v[0], v[1]), dev::f32x2_to_bf16x2(v[2], v[3]));
                }
            } else {
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    if (c + q >= p.n) continue;
                    if constexpr (sizeof(OUT) == 4) o[q] = p.accumulate ? o[q] + v[q] : v[q];
                    else o[q] = dev::f32_to_bf16(v[q]);
                }
            }
        }
    }
}

}  // namespace

hipError_t launch_product(ProductArgs a, int32_t a_format, int32_t out_dtype, hipStream_t s) {
    a.tiles_n = (int32_t)((a.n + TILE - 1) / TILE);
    a.tiles_m = (int32_t)((a.m + TILE - 1) / TILE);
    // every segment may end inside a tile, but not more of them than there are rows
    int64_t rows = a.tiles_m;
    if (a.mode == MUON_PRODUCT_ROWS) rows = a.m / TILE + (a.m < a.groups ? a.m : (int64_t)a.groups);
    if (a.mode == MUON_PRODUCT_DEPTH) rows *= a.groups;
    const int64_t total = rows * a.tiles_n;
    if (total >= (int64_t)1 << 31) return hipErrorInvalidConfiguration;
    if (total == 0) return hipSuccess;
    const dim3 grid((unsigned)total), block(256);
    const bool f32 = out_dtype == MUON_DTYPE_F32;
    if (a_format == MUON_FP8_E4M3) {
        if (f32) hipLaunchKernelGGL((product_kernel<0, float>), grid, block, 0, s, a);
        else hipLaunchKernelGGL((product_kernel<0, uint16_t>), grid, block, 0, s, a);
    } else {
        if (f32) hipLaunchKernelGGL((product_kernel<1, float>), grid, block, 0, s, a);
        else hipLaunchKernelGGL((product_kernel<1, uint16_t>), grid, block, 0, s, a);
    }
    return hipGetLastError();
}

}  // namespace muon
