// Block quantisation to 8 bits (gfx950).
//
// For a block of values with the largest finite magnitude amax, e is the least exponent with
// amax <= MAX * 2^e (MAX = 1.75 * 2^8 for e4m3, 1.75 * 2^15 for e5m2): with amax = f * 2^E, 1 <= f
// < 2, that is E - 8 (or E - 15), and one more where f > 1.75.  The code is v * 2^-e, an exact product
// of float32 values, rounded once by the conversion instruction; it never exceeds MAX.
//
// One workgroup takes a 128 x 128 tile, 8 x 8 values a thread: src is read once whatever is
// written, a row's block and (in the transposed copy) a column's block lie inside the tile, and a thread's
// 8 values down a column are 8 consecutive bytes of the transposed copy.
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
__device__ __forceinline__ float inverse_scale(uint32_t byte) { return __uint_as_float((254u - byte) << 23); }

// Magnitude bits of a finite value, 0 for an infinity or NaN.
__device__ __forceinline__ uint32_t finite_bits(float v) {
    const uint32_t u = __float_as_uint(v) & 0x7fffffffu;
    return u < 0x7f800000u ? u : 0u;
}

template <int FMT>
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d) {
    int w = 0;
    if (FMT == MUON_FP8_E4M3) {
        w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, w, false);
        w = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
    } else {
        w = __builtin_amdgcn_cvt_pk_bf8_f32(a, b, w, false);
        w = __builtin_amdgcn_cvt_pk_bf8_f32(c, d, w, true);
    }
    return (uint32_t)w;
}

// v * s, with a NaN for an infinity.
__device__ __forceinline__ float scaled(float v, float s) {
    return fabsf(v) < INFINITY ? v * s : __uint_as_float(0x7fc00000u);
}

__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
    const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
__device__ __forceinline__ void load8(const uint16_t* p, float (&v)[8]) {
    const uint4 a = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        v[2 * j] = __uint_as_float(w[j] << 16);
        v[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
    }
}
__device__ __forceinline__ float load1(const float* p) { return *p; }
__device__ __forceinline__ float load1(const uint16_t* p) { return dev::bf16_to_f32(*p); }

template <class T, int FMT, bool SQUARE>
__global__ __launch_bounds__(256) void quantize_kernel(QuantizeArgs p, int vec) {
    __shared__ __attribute__((aligned(16))) uint8_t lds_t[QT * QT];
    __shared__ uint32_t col_amax[4][QT];
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
    float v[8][8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] = 0.f;
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
        if (vec && c + 8 <= p.cols) {
            load8(row + c, v[i]);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (c + j < p.cols) v[i][j] = load1(row + c + j);
        }
    }

    uint32_t all = 0;
    if (SQUARE) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) all = max(all, finite_bits(v[i][j]));
#pragma unroll
        for (int off = 32; off > 0; off >>= 1) all = max(all, (uint32_t)__shfl_xor((int)all, off, 64));
        if (lane == 0) tile_amax[wave] = all;
        __syncthreads();
        all = max(max(tile_amax[0], tile_amax[1]), max(tile_amax[2], tile_amax[3]));
    }
    const uint32_t tile_byte = scale_byte<FMT>(all);
    const float tile_inv = inverse_scale(tile_byte);

    if (p.codes) {
        uint8_t* codes = p.codes + mat * p.rows * p.kp;
        uint8_t* scales = p.scales + mat * (SQUARE ? p.tiles_r : p.rows) * p.sp;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int64_t r = r0 + 8 * rg + i;
            uint32_t byte = tile_byte;
            float inv = tile_inv;
            if (!SQUARE) {
                uint32_t m = 0;
#pragma unroll
                for (int j = 0; j < 8; ++j) m = max(m, finite_bits(v[i][j]));
#pragma unroll
                for (int off = 8; off > 0; off >>= 1) m = max(m, (uint32_t)__shfl_xor((int)m, off, 64));
                byte = scale_byte<FMT>(m);
                inv = inverse_scale(byte);
            }
            if (r < end) {
                uint2 w;
                w.x = codes4<FMT>(scaled(v[i][0], inv), scaled(v[i][1], inv), scaled(v[i][2], inv), scaled(v[i][3], inv));
                w.y = codes4<FMT>(scaled(v[i][4], inv), scaled(v[i][5], inv), scaled(v[i][6], inv), scaled(v[i][7], inv));
                *reinterpret_cast<uint2*>(codes + r * p.kp + c) = w;
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
        // lane of columns 8 cg .. 8 cg + 7: column amax over the wave's four row groups, then over the waves
        float inv[8];
        if (!SQUARE) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                uint32_t m = 0;
#pragma unroll
                for (int i = 0; i < 8; ++i) m = max(m, finite_bits(v[i][j]));
                m = max(m, (uint32_t)__shfl_xor((int)m, 16, 64));
                m = max(m, (uint32_t)__shfl_xor((int)m, 32, 64));
                if (lane < 16) col_amax[wave][8 * cg + j] = m;
            }
            __syncthreads();
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int col = 8 * cg + j;
            inv[j] = tile_inv;
            if (!SQUARE) {
                const uint32_t m = max(max(col_amax[0][col], col_amax[1][col]), max(col_amax[2][col], col_amax[3][col]));
                inv[j] = inverse_scale(scale_byte<FMT>(m));
            }
            uint2 w;
            w.x = codes4<FMT>(scaled(v[0][j], inv[j]), scaled(v[1][j], inv[j]), scaled(v[2][j], inv[j]), scaled(v[3][j], inv[j]));
            w.y = codes4<FMT>(scaled(v[4][j], inv[j]), scaled(v[5][j], inv[j]), scaled(v[6][j], inv[j]), scaled(v[7][j], inv[j]));
            // 8-byte granule rg of transposed row col, at granule rg ^ cg: the 16 lanes of a row group hit 16 granules
            *reinterpret_cast<uint2*>(lds_t + col * QT + 8 * (rg ^ cg)) = w;
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
            *reinterpret_cast<uint4*>(codes + (c0 + col) * p.kp_t + r0 + 16 * q) = w;
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
    // 16-byte loads where every row of src begins on one
    const int64_t size = sizeof(T);
    const int vec = a.ld * size % 16 == 0 && a.batch_stride * size % 16 == 0;
    const dim3 grid((unsigned)a.tiles);
    if (square) hipLaunchKernelGGL((quantize_kernel<T, FMT, true>), grid, dim3(256), 0, s, a, vec);
    else hipLaunchKernelGGL((quantize_kernel<T, FMT, false>), grid, dim3(256), 0, s, a, vec);
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
