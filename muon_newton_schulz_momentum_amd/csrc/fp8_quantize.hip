// Block quantisation to 8 bits (gfx950).
//
// For a block of values with the largest finite magnitude amax, e is the least exponent with
// amax <= MAX * 2^e (MAX = 1.75 * 2^8 for e4m3, 1.75 * 2^15 for e5m2): with amax = f * 2^E, 1 <= f
// < 2, that is E - 8 (or E - 15), and one more where f > 1.75.  The code is v * 2^-e, which never exceeds MAX, rounded
// once by the scaling conversion instruction.
//
// One workgroup takes a 128 x 128 tile, 8 x 8 values a thread: src is read once whatever is
// written, a row's block and (in the transposed copy) a column's block lie inside the tile, and a thread's
// 8 values down a column are 8 consecutive bytes of the transposed copy.
//
// Bound by memory: 64 float32 matrices of 1024 x 4096 in squares, both orientations, 1.61 GB in 283 us (5.7 TB/s);
// 57344 rows of 4096 bfloat16 gathered from 8192, both orientations, 0.54 GB in 119 us (4.5 TB/s), where the
// vector instructions are as near their limit (about 8 a value, issued in 93 % of the busy cycles; 26 % in the first).
// Twice the tiles a workgroup held more registers and was slower.
#include "device_common.h"
#include "experts.h"

namespace muon {
namespace {

constexpr int QT = 128;            // tile edge = block length

// Scale exponent + 127 of a block whose largest magnitude has these float32 bits.
template <int FMT>
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax) {
    const int e = (int)(amax >> 23) - (FMT == MUON_FP8_E4M3 ? 8 : 15) + ((amax & 0x7fffffu) > 0x600000u ? 1 : 0);
    return (uint32_t)max(e, 0);
}
// The byte as the conversions take it.
__device__ __forceinline__ float scale_operand(uint32_t byte) { return __uint_as_float(byte << 23); }

constexpr uint32_t INF_BITS = 0x7f800000u;

typedef short s16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

// Over the 16 lanes of a row, to all of them.
__device__ __forceinline__ uint32_t max16(uint32_t v) {
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xb1, 0xf, 0xf, false));    // neighbours
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4e, 0xf, 0xf, false));    // pairs
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x141, 0xf, 0xf, false));   // halves of 8
    return max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x140, 0xf, 0xf, false));  // halves of 16
}
// Over the same lane of the wave's four rows, to all of them.
__device__ __forceinline__ uint32_t max_rows(uint32_t v) {
    const auto a = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    v = max((uint32_t)a[0], (uint32_t)a[1]);
    const auto b = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    return max((uint32_t)b[0], (uint32_t)b[1]);
}

// Two values over 2^(byte - 127) as codes in the low or high half of a word: one instruction each, rounding to nearest
// even; scale carries the byte in its exponent.
template <int FMT, bool HIGH>
__device__ __forceinline__ s16x2 convert2(s16x2 old, float a, float b, float scale) {
    if constexpr (FMT == MUON_FP8_E4M3) return __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(old, a, b, scale, HIGH);
    else return __builtin_amdgcn_cvt_scalef32_pk_bf8_f32(old, a, b, scale, HIGH);
}
template <int FMT, bool HIGH>
__device__ __forceinline__ s16x2 convert2(s16x2 old, uint32_t pair, float scale) {
    const bf16x2 v = __builtin_bit_cast(bf16x2, pair);
    if constexpr (FMT == MUON_FP8_E4M3) return __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(old, v, scale, HIGH);
    else return __builtin_amdgcn_cvt_scalef32_pk_bf8_bf16(old, v, scale, HIGH);
}

// Codes are not read again here, and a source row that is gathered several times is: stores that do not stay in the
// caches leave it there (8192 rows of 4096 gathered 7 times, with the transpose: 140 us against 185).
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
__device__ __forceinline__ void store_once(uint8_t* p, uint2 v) {
    __builtin_nontemporal_store(__builtin_bit_cast(uint64_t, v), reinterpret_cast<uint64_t*>(p));
}
__device__ __forceinline__ void store_once(uint8_t* p, uint4 v) {
    __builtin_nontemporal_store(__builtin_bit_cast(u32x4, v), reinterpret_cast<u32x4*>(p));
}

// Rows of src need not begin on a 16-byte boundary.
typedef float f32x4_any __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));

// A thread's 8 x 8 values as they are in memory.
template <class T>
struct Block;

template <>
struct Block<float> {
    float v[8][8];
    __device__ __forceinline__ void clear(int i) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] = 0.f;
    }
    __device__ __forceinline__ void load(int i, const float* p) {
        const f32x4_any a = *reinterpret_cast<const f32x4_any*>(p), b = *reinterpret_cast<const f32x4_any*>(p + 4);
        v[i][0] = a.x; v[i][1] = a.y; v[i][2] = a.z; v[i][3] = a.w;
        v[i][4] = b.x; v[i][5] = b.y; v[i][6] = b.z; v[i][7] = b.w;
    }
    __device__ __forceinline__ void set(int i, int j, float x) { v[i][j] = x; }
    // Largest magnitude bits of each row and column; with FINITE infinities and NaN count as zeros.
    template <bool FINITE>
    __device__ __forceinline__ void maxima(uint32_t (&row)[8], uint32_t (&col)[8]) const {
#pragma unroll
        for (int i = 0; i < 8; ++i) row[i] = col[i] = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                uint32_t u = __float_as_uint(v[i][j]) & 0x7fffffffu;
                if (FINITE && u >= INF_BITS) u = 0;
                row[i] = max(row[i], u);
                col[j] = max(col[j], u);
            }
    }
    __device__ __forceinline__ void infinities_to_nan() {
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if ((__float_as_uint(v[i][j]) & 0x7fffffffu) == INF_BITS) v[i][j] = __uint_as_float(0x7fc00000u);
    }
    template <int FMT>
    __device__ __forceinline__ uint2 row_codes(int i, float scale) const {
        s16x2 a = {0, 0}, b = {0, 0};
        a = convert2<FMT, false>(a, v[i][0], v[i][1], scale);
        a = convert2<FMT, true>(a, v[i][2], v[i][3], scale);
        b = convert2<FMT, false>(b, v[i][4], v[i][5], scale);
        b = convert2<FMT, true>(b, v[i][6], v[i][7], scale);
        return make_uint2(__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b));
    }
    template <int FMT>
    __device__ __forceinline__ uint2 col_codes(int j, float scale) const {
        s16x2 a = {0, 0}, b = {0, 0};
        a = convert2<FMT, false>(a, v[0][j], v[1][j], scale);
        a = convert2<FMT, true>(a, v[2][j], v[3][j], scale);
        b = convert2<FMT, false>(b, v[4][j], v[5][j], scale);
        b = convert2<FMT, true>(b, v[6][j], v[7][j], scale);
        return make_uint2(__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b));
    }
};

template <>
struct Block<uint16_t> {
    uint32_t w[8][4];          // two values a word
    __device__ __forceinline__ void clear(int i) { w[i][0] = w[i][1] = w[i][2] = w[i][3] = 0; }
    __device__ __forceinline__ void load(int i, const uint16_t* p) {
        const u32x4_any u = *reinterpret_cast<const u32x4_any*>(p);
        w[i][0] = u.x; w[i][1] = u.y; w[i][2] = u.z; w[i][3] = u.w;
    }
    __device__ __forceinline__ void set(int i, int j, uint16_t x) { w[i][j >> 1] |= (uint32_t)x << (16 * (j & 1)); }
    template <bool FINITE>
    __device__ __forceinline__ void maxima(uint32_t (&row)[8], uint32_t (&col)[8]) const {
        typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
        u16x2 c[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) c[k] = u16x2{0, 0};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            u16x2 r = {0, 0};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                uint32_t u = w[i][k] & 0x7fff7fffu;
                if (FINITE && (u & 0xffffu) >= 0x7f80u) u &= 0xffff0000u;
                if (FINITE && u >= INF_BITS) u &= 0xffffu;
                const u16x2 h = __builtin_bit_cast(u16x2, u);
                r = __builtin_elementwise_max(r, h);
                c[k] = __builtin_elementwise_max(c[k], h);
            }
            row[i] = (uint32_t)max(r[0], r[1]) << 16;
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            col[2 * k] = (uint32_t)c[k][0] << 16;
            col[2 * k + 1] = (uint32_t)c[k][1] << 16;
        }
    }
    __device__ __forceinline__ void infinities_to_nan() {
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if ((w[i][k] & 0x7fffu) == 0x7f80u) w[i][k] |= 0x40u;
                if ((w[i][k] & 0x7fff0000u) == INF_BITS) w[i][k] |= 0x400000u;
            }
    }
    template <int FMT>
    __device__ __forceinline__ uint2 row_codes(int i, float scale) const {
        s16x2 a = {0, 0}, b = {0, 0};
        a = convert2<FMT, false>(a, w[i][0], scale);
        a = convert2<FMT, true>(a, w[i][1], scale);
        b = convert2<FMT, false>(b, w[i][2], scale);
        b = convert2<FMT, true>(b, w[i][3], scale);
        return make_uint2(__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b));
    }
    // values (i, j) and (i + 1, j) in one word
    __device__ __forceinline__ uint32_t pair(int i, int j) const {
        return __builtin_amdgcn_perm(w[i + 1][j >> 1], w[i][j >> 1], j & 1 ? 0x07060302u : 0x05040100u);
    }
    template <int FMT>
    __device__ __forceinline__ uint2 col_codes(int j, float scale) const {
        s16x2 a = {0, 0}, b = {0, 0};
        a = convert2<FMT, false>(a, pair(0, j), scale);
        a = convert2<FMT, true>(a, pair(2, j), scale);
        b = convert2<FMT, false>(b, pair(4, j), scale);
        b = convert2<FMT, true>(b, pair(6, j), scale);
        return make_uint2(__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b));
    }
};

template <class T, int FMT, bool SQUARE>
__global__ __launch_bounds__(256) void quantize_kernel(QuantizeArgs p) {
    __shared__ __attribute__((aligned(16))) uint8_t lds_t[QT * QT];
    __shared__ __attribute__((aligned(16))) uint32_t col_amax[4][QT];
    __shared__ uint32_t tile_amax[4];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int cg = tid & 15, rg = tid >> 4;
    const int64_t per_mat = (int64_t)p.tiles_r * p.tiles_c;
    const int64_t mat = blockIdx.x / per_mat;
    const int t = (int)(blockIdx.x - mat * per_mat);
    const int tr = t / p.tiles_c, tc = t - tr * p.tiles_c;
    const int64_t r0 = (int64_t)tr * QT, c0 = (int64_t)tc * QT;
    const int64_t end = p.limit ? min(p.rows, max((int64_t)*p.limit, (int64_t)0)) : p.rows;
    if (r0 >= end) return;

    const T* src = static_cast<const T*>(p.src) + mat * p.batch_stride;
    const int64_t c = c0 + 8 * cg;
    Block<T> v;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        v.clear(i);
        const int64_t r = r0 + 8 * rg + i;
        if (r >= end) continue;
        int64_t sr = r;
        if (p.gather) {
            const int g = p.gather[r];
            if (g < 0) continue;
            sr = g / p.per;
            if (sr >= p.src_rows) continue;
        }
        const T* row = src + sr * p.ld;
        if (c + 8 <= p.cols) {
            v.load(i, row + c);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (c + j < p.cols) v.set(i, j, row[c + j]);
        }
    }

    uint32_t row_max[8], col_max[8], all = 0;
    v.template maxima<false>(row_max, col_max);
#pragma unroll
    for (int i = 0; i < 8; ++i) all = max(all, row_max[i]);
    if (__ballot(all >= INF_BITS)) {                       // an infinity or NaN among the wave's values
        v.infinities_to_nan();
        v.template maxima<true>(row_max, col_max);
        all = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) all = max(all, row_max[i]);
    }
    if (SQUARE) {
        all = max_rows(max16(all));
        if (lane == 0) tile_amax[wave] = all;
        __syncthreads();
        all = max(max(tile_amax[0], tile_amax[1]), max(tile_amax[2], tile_amax[3]));
    }
    const uint32_t tile_byte = scale_byte<FMT>(all);

    if (p.codes) {
        uint8_t* codes = p.codes + mat * p.rows * p.kp;
        uint8_t* scales = p.scales + mat * (SQUARE ? p.tiles_r : p.rows) * p.sp;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int64_t r = r0 + 8 * rg + i;
            const uint32_t byte = SQUARE ? tile_byte : scale_byte<FMT>(max16(row_max[i]));
            if (r < end) {
                store_once(codes + r * p.kp + c, v.template row_codes<FMT>(i, scale_operand(byte)));
                if (!SQUARE) {
                    if (cg == 0) scales[r * p.sp + tc] = (uint8_t)byte;
                    else if (tc + 1 == p.tiles_c && tc + cg < p.sp) scales[r * p.sp + tc + cg] = 0;
                }
            }
        }
        if (SQUARE && tid < 4 && (tid == 0 || (tc + 1 == p.tiles_c && tc + tid < p.sp)))
            scales[(int64_t)tr * p.sp + tc + tid] = tid == 0 ? (uint8_t)tile_byte : 0;
    }

    if (p.codes_t) {
        // columns 8 cg .. 8 cg + 7: over the wave's four row groups, then over the waves
        if (!SQUARE) {
#pragma unroll
            for (int j = 0; j < 8; ++j) col_max[j] = max_rows(col_max[j]);
            if (lane < 16) {
                uint4* to = reinterpret_cast<uint4*>(col_amax[wave] + 8 * cg);
                to[0] = make_uint4(col_max[0], col_max[1], col_max[2], col_max[3]);
                to[1] = make_uint4(col_max[4], col_max[5], col_max[6], col_max[7]);
            }
            __syncthreads();
#pragma unroll
            for (int w = 0; w < 4; ++w)
#pragma unroll
                for (int j = 0; j < 8; ++j) col_max[j] = max(col_max[j], col_amax[w][8 * cg + j]);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t byte = SQUARE ? tile_byte : scale_byte<FMT>(col_max[j]);
            // 8-byte granule rg of transposed row col, at granule rg ^ cg: the 16 lanes of a row group hit 16 granules
            *reinterpret_cast<uint2*>(lds_t + (8 * cg + j) * QT + 8 * (rg ^ cg)) = v.template col_codes<FMT>(j, scale_operand(byte));
        }
        __syncthreads();
        uint8_t* codes = p.codes_t + mat * p.cols * p.kp_t;
        uint8_t* scales = p.scales_t + mat * (SQUARE ? p.tiles_c : p.cols) * p.sp_t;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int col = 32 * i + (tid >> 3), q = tid & 7;
            if (c0 + col >= p.cols) continue;
            const int f = (col >> 3) & 15;
            uint4 w = *reinterpret_cast<const uint4*>(lds_t + col * QT + 16 * (q ^ (f >> 1)));
            if (f & 1) w = make_uint4(w.z, w.w, w.x, w.y);
            store_once(codes + (c0 + col) * p.kp_t + r0 + 16 * q, w);
        }
        const bool last = tr + 1 == p.tiles_r;
        if (SQUARE) {
            if (tid < 4 && (tid == 0 || (last && tr + tid < p.sp_t)))
                scales[(int64_t)tc * p.sp_t + tr + tid] = tid == 0 ? (uint8_t)tile_byte : 0;
        } else if (tid < QT && c0 + tid < p.cols) {
            const uint32_t m = max(max(col_amax[0][tid], col_amax[1][tid]), max(col_amax[2][tid], col_amax[3][tid]));
            uint8_t* s = scales + (c0 + tid) * p.sp_t + tr;
            s[0] = (uint8_t)scale_byte<FMT>(m);
            for (int q = 1; last && tr + q < p.sp_t; ++q) s[q] = 0;
        }
    }
}

template <class T, int FMT>
void quantize_as(const QuantizeArgs& a, int32_t square, hipStream_t s) {
    const dim3 grid((unsigned)a.tiles);
    if (square) hipLaunchKernelGGL((quantize_kernel<T, FMT, true>), grid, dim3(256), 0, s, a);
    else hipLaunchKernelGGL((quantize_kernel<T, FMT, false>), grid, dim3(256), 0, s, a);
}

}  // namespace

hipError_t launch_quantize(const QuantizeArgs& a, int32_t src_dtype, int32_t format, int32_t square, hipStream_t s) {
    if (src_dtype == MUON_DTYPE_F32) {
        if (format == MUON_FP8_E4M3) quantize_as<float, MUON_FP8_E4M3>(a, square, s);
        else quantize_as<float, MUON_FP8_E5M2>(a, square, s);
    } else {
        if (format == MUON_FP8_E4M3) quantize_as<uint16_t, MUON_FP8_E4M3>(a, square, s);
        else quantize_as<uint16_t, MUON_FP8_E5M2>(a, square, s);
    }
    return hipGetLastError();
}

}  // namespace muon
