// Row operations of the expert layers (gfx950): 8-bit integer quantisation, rows gathered into expert order and combined
// back, and the gradients of the gated block's pre-activations.  All are bound by memory.
#include <algorithm>

#include "activation.h"
#include "device_common.h"
#include "layers.h"

namespace muon {
namespace {

typedef float f32x4_any __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));

constexpr int THREADS = 256, WAVE = 64;
constexpr int V = 8;                                       // values of a lane's load

// A launch's waves take its items in turn.
__device__ __forceinline__ int64_t first_wave() { return (int64_t)blockIdx.x * (THREADS / WAVE) + (threadIdx.x >> 6); }
__device__ __forceinline__ int64_t all_waves() { return (int64_t)gridDim.x * (THREADS / WAVE); }

// 8 values from column c of a row of `cols`, zeros behind its end; rows may begin anywhere.
__device__ __forceinline__ void load8(const float* row, int64_t c, int64_t cols, float (&v)[V]) {
    if (c + V <= cols) {
        const f32x4_any a = *reinterpret_cast<const f32x4_any*>(row + c), b = *reinterpret_cast<const f32x4_any*>(row + c + 4);
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    } else {
#pragma unroll
        for (int e = 0; e < V; ++e) v[e] = c + e < cols ? row[c + e] : 0.f;
    }
}
__device__ __forceinline__ void load8(const uint16_t* row, int64_t c, int64_t cols, float (&v)[V]) {
    if (c + V <= cols) {
        const u32x4_any a = *reinterpret_cast<const u32x4_any*>(row + c);
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int e = 0; e < V; ++e) v[e] = __uint_as_float(e & 1 ? w[e / 2] & 0xffff0000u : w[e / 2] << 16);
    } else {
#pragma unroll
        for (int e = 0; e < V; ++e) v[e] = c + e < cols ? dev::bf16_to_f32(row[c + e]) : 0.f;
    }
}
__device__ __forceinline__ void store8(float* row, int64_t c, int64_t cols, const float (&v)[V]) {
    if (c + V <= cols) {
        *reinterpret_cast<f32x4_any*>(row + c) = f32x4_any{v[0], v[1], v[2], v[3]};
        *reinterpret_cast<f32x4_any*>(row + c + 4) = f32x4_any{v[4], v[5], v[6], v[7]};
    } else {
#pragma unroll
        for (int e = 0; e < V; ++e)
            if (c + e < cols) row[c + e] = v[e];
    }
}
__device__ __forceinline__ void store8(uint16_t* row, int64_t c, int64_t cols, const float (&v)[V]) {
    if (c + V <= cols) {
        *reinterpret_cast<u32x4_any*>(row + c) = u32x4_any{dev::f32x2_to_bf16x2(v[0], v[1]), dev::f32x2_to_bf16x2(v[2], v[3]),
                                                           dev::f32x2_to_bf16x2(v[4], v[5]), dev::f32x2_to_bf16x2(v[6], v[7])};
    } else {
#pragma unroll
        for (int e = 0; e < V; ++e)
            if (c + e < cols) row[c + e] = dev::f32_to_bf16(v[e]);
    }
}

// ---- 8-bit integer quantisation ---------------------------------------------------------------

// The whole number nearest x / s, ties to even, kept in [-127, 127], whatever x / s: rint of the approximate quotient is off by one
// at most; what is left, x - c s, is exact in one fused multiply-add (its magnitude is near s / 2 or less and it is a
// multiple of the smaller of x's and s's last places), and its double against s decides.
__device__ __forceinline__ int exact_code(float x, float s, float inverse) {
    float c = fminf(fmaxf(rintf(x * inverse), -127.f), 127.f);
    const float left = fmaf(-c, s, x), twice = 2.f * fabsf(left);
    const bool odd = ((int)c & 1) != 0;
    if (twice > s || (twice == s && odd)) c += copysignf(1.f, left);
    return (int)fminf(fmaxf(c, -127.f), 127.f);
}

// 8 values' codes.  x times the rounded inverse is within 127.5 * 2^-23 < 2^-16 of the quotient (s above 2^-64, where |x| <= 127 s
// (1 + 2^-24)), so its nearest whole number is the code unless it lies within 2^-15 of a border: then the wave takes the exact
// way.  Adding 1.5 * 2^23 rounds to a whole number, ties to even, and leaves its two's complement in the low bits.
__device__ __forceinline__ uint2 codes8(const float (&v)[V], float s, float inverse) {
    uint32_t q[V];
    float worst = 0.f;
#pragma unroll
    for (int e = 0; e < V; ++e) {
        const float x = v[e] * inverse, f = x + 12582912.f;
        q[e] = __float_as_uint(f);
        worst = fmaxf(worst, fabsf(x - (f - 12582912.f)));
    }
    if (__builtin_amdgcn_ballot_w64(worst > 0.5f - 0x1p-15f) == 0) {
        const uint32_t a = __builtin_amdgcn_perm(q[1], q[0], 0x0c0c0400), b = __builtin_amdgcn_perm(q[3], q[2], 0x04000c0c);
        const uint32_t c = __builtin_amdgcn_perm(q[5], q[4], 0x0c0c0400), d = __builtin_amdgcn_perm(q[7], q[6], 0x04000c0c);
        return make_uint2(a | b, c | d);
    }
    uint32_t w[2] = {0, 0};
#pragma unroll
    for (int e = 0; e < V; ++e) w[e / 4] |= ((uint32_t)exact_code(v[e], s, inverse) & 255u) << (8 * (e & 3));
    return make_uint2(w[0], w[1]);
}

// 8 values as they are in memory.
template <class T>
struct Raw;
template <>
struct Raw<float> {
    float v[V];
    __device__ __forceinline__ void load(const float* at) {
        const f32x4_any a = *reinterpret_cast<const f32x4_any*>(at), b = *reinterpret_cast<const f32x4_any*>(at + 4);
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    }
    __device__ __forceinline__ void load_checked(const float* row, int64_t c, int64_t cols) { load8(row, c, cols, v); }
    __device__ __forceinline__ void get(float (&to)[V]) const {
#pragma unroll
        for (int e = 0; e < V; ++e) to[e] = v[e];
    }
};
template <>
struct Raw<uint16_t> {
    uint32_t w[V / 2];
    __device__ __forceinline__ void load(const uint16_t* at) {
        const u32x4_any a = *reinterpret_cast<const u32x4_any*>(at);
        w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
    }
    __device__ __forceinline__ void load_checked(const uint16_t* row, int64_t c, int64_t cols) {
        float v[V];
        load8(row, c, cols, v);
#pragma unroll
        for (int e = 0; e < V / 2; ++e) w[e] = dev::f32x2_to_bf16x2(v[2 * e], v[2 * e + 1]);
    }
    // (unpacked anew wherever they are used)
    __device__ __forceinline__ void get(float (&to)[V]) {
        asm volatile("" : "+v"(w[0]), "+v"(w[1]), "+v"(w[2]), "+v"(w[3]));
#pragma unroll
        for (int e = 0; e < V; ++e) to[e] = __uint_as_float(e & 1 ? w[e / 2] & 0xffff0000u : w[e / 2] << 16);
    }
};

// LANES (16, a wave or the workgroup) take a row, whose values stay in registers between its largest magnitude and its codes, CHUNKS of 8 a
// lane; CHUNKS 0: longer rows, read twice, or shorter ones than 8.  A chunk that would pass the end of its row is the row's last 8 values,
// whose codes are shifted to their place.  Bound by vector instructions and memory alike (16381 rows of 8704 bfloat16: 75 us, of which
// 64 in the kernel, 428 MB; read twice and checked at every load 127).
template <class T, int LANES, int CHUNKS>
__global__ __launch_bounds__(THREADS) void int8_quantize_kernel(Int8QuantizeArgs p) {
    __shared__ uint32_t tops[THREADS / WAVE];
    const int tid = threadIdx.x, lane = tid % LANES;
    const int64_t end = p.limit ? min((int64_t)*p.limit, p.total) : p.total;
    for (int64_t r = (int64_t)blockIdx.x * (THREADS / LANES) + tid / LANES; r < end; r += (int64_t)gridDim.x * (THREADS / LANES)) {
        const T* row = nullptr;
        if (p.gather) {
            const int c = p.gather[r];
            if (c >= 0 && c / p.per < p.src_rows) row = static_cast<const T*>(p.src) + (int64_t)(c / p.per) * p.ld;
        } else if (p.batch_stride == 0) {
            row = static_cast<const T*>(p.src) + r * p.ld;
        } else {
            row = static_cast<const T*>(p.src) + r / p.rows * p.batch_stride + r % p.rows * p.ld;
        }
        Raw<T> raw[CHUNKS > 0 ? CHUNKS : 1];
        uint32_t top = 0;                                  // bits of magnitudes are ordered as the magnitudes are
        auto largest = [&](Raw<T>& x) {
            float v[V];
            x.get(v);
#pragma unroll
            for (int e = 0; e < V; ++e) top = max(top, __float_as_uint(v[e]) & 0x7fffffffu);
        };
        const int cols = (int)p.cols;
        if (row) {
            if constexpr (CHUNKS > 0) {
#pragma unroll
                for (int i = 0; i < CHUNKS; ++i) raw[i].load(row + min((i * LANES + lane) * V, cols - V));
#pragma unroll
                for (int i = 0; i < CHUNKS; ++i) largest(raw[i]);
            } else {
                for (int64_t c = lane * V; c < cols; c += LANES * V) {
                    raw[0].load_checked(row, c, cols);
                    largest(raw[0]);
                }
            }
        }
#pragma unroll
        for (int off = (LANES < WAVE ? LANES : WAVE) / 2; off > 0; off >>= 1) top = max(top, (uint32_t)__shfl_xor((int)top, off, 64));
        if (LANES > WAVE) {
            if (tid % WAVE == 0) tops[tid / WAVE] = top;
            __syncthreads();
#pragma unroll
            for (int w = 0; w < THREADS / WAVE; ++w) top = max(top, tops[w]);
            __syncthreads();                               // before the next row's
        }
        const bool finite = top < 0x7f800000u;
        const float s = finite ? __uint_as_float(top) / 127.f : __uint_as_float(0x7fc00000u);
        if (lane == 0) p.scales[r] = s;
        // small scales are brought to where their inverse and all steps are exact; there s may have been rounded far
        const bool tiny = s < 0x1p-64f, any = row && finite && s > 0.f;
        const float lift = tiny ? 0x1p64f : 1.f, lifted = s * lift, inverse = 1.f / lifted;
        auto codes = [&](Raw<T>& x) {
            float v[V];
            x.get(v);
            if (!tiny) return codes8(v, s, inverse);
#pragma unroll
            for (int e = 0; e < V; ++e) v[e] = (float)exact_code(v[e] * lift, lifted, inverse);
            return codes8(v, 1.f, 1.f);
        };
        auto put = [&](int64_t c, uint64_t w) { __builtin_nontemporal_store(w, reinterpret_cast<uint64_t*>(p.codes + r * p.kp + c)); };
        if constexpr (CHUNKS > 0) {
#pragma unroll
            for (int i = 0; i < CHUNKS; ++i) {
                const int c = (i * LANES + lane) * V, before = c - max(cols - V, 0);
                uint64_t w = 0;
                if (any) w = __builtin_bit_cast(uint64_t, codes(raw[i]));
                if (before > 0) w = before < V ? w >> (8 * before) : 0;
                if (c < p.kp) put(c, w);
            }
        } else {
            for (int64_t c = lane * V; c < p.kp; c += LANES * V) {
                uint64_t w = 0;
                if (any && c < cols) {
                    raw[0].load_checked(row, c, cols);
                    w = __builtin_bit_cast(uint64_t, codes(raw[0]));
                }
                put(c, w);
            }
        }
    }
}

// ---- rows to experts and back -----------------------------------------------------------------

// The sum over a row's columns of from * y, and from times w into out where that is there; a whole wave.
template <class T>
__device__ __forceinline__ float row_of(const GatherRowsArgs& p, const T* from, float w, const T* y, T* out, int lane) {
    float dot = 0.f;
    for (int64_t i = lane * V; i < p.cols; i += WAVE * V) {
        float v[V] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        if (from) load8(from, i, p.cols, v);
        if (y) {
            float u[V];
            load8(y, i, p.cols, u);
#pragma unroll
            for (int e = 0; e < V; ++e) dot = fmaf(v[e], u[e], dot);
        }
        if (out) {
#pragma unroll
            for (int e = 0; e < V; ++e) v[e] *= w;
            store8(out, i, p.cols, v);
        }
    }
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) dot += __shfl_xor(dot, off, 64);
    return dot;
}

// One wave per row of out, which also forms the gradient of its choice's weight; behind those, one wave per 64 choices for
// the weights of choices that no row has (0), or whose row is not their own or is behind the limit.  So a row of y is read once, beside
// the row that it is the gradient of, and no sum needs an atomic.  Bound by memory (57344 rows of 4096 bfloat16, with the weights'
// gradients: 208 us, 1.01 GB, 4.8 TB/s).
template <class T>
__global__ __launch_bounds__(THREADS) void gather_rows_kernel(GatherRowsArgs p) {
    const int lane = threadIdx.x & 63;
    const int64_t limit = p.limit ? min((int64_t)*p.limit, p.n_rows) : p.n_rows;
    const int64_t waves = p.n_rows + (p.grad_weights ? (p.choices + WAVE - 1) / WAVE : 0);
    const T* src = static_cast<const T*>(p.src);
    const T* y = static_cast<const T*>(p.y);
    for (int64_t r = first_wave(); r < waves; r += all_waves()) {
        if (r < p.n_rows) {
            if (r >= limit) continue;
            const int c = p.rows[r];
            const bool there = c >= 0 && c < p.choices;
            const bool dots = there && p.grad_weights && p.position[c] == r;
            const float dot = row_of<T>(p, there ? src + (int64_t)(c / p.per) * p.ld : nullptr, there && p.weights ? p.weights[c] : 1.f,
                                        dots ? y + r * p.ld_y : nullptr, p.out ? static_cast<T*>(p.out) + r * p.ld_out : nullptr, lane);
            if (dots && lane == 0) p.grad_weights[c] = dot;
        } else {
            const int64_t c = (r - p.n_rows) * WAVE + lane;
            int at = -1;
            bool left = false;
            if (c < p.choices) {
                at = p.position[c];
                if (at < 0 || at >= p.n_rows) p.grad_weights[c] = 0.f;
                else left = at >= limit || p.rows[at] != c;
            }
            for (uint64_t todo = __builtin_amdgcn_ballot_w64(left); todo; todo &= todo - 1) {
                const int which = __builtin_ctzll(todo);
                const int64_t cc = (r - p.n_rows) * WAVE + which;
                const int64_t rr = __shfl(at, which, 64);
                const float dot = row_of<T>(p, src + cc / p.per * p.ld, 1.f, y + rr * p.ld_y, nullptr, lane);
                if (lane == 0) p.grad_weights[cc] = dot;
            }
        }
    }
}

// One wave per token and 512 columns, whose rows are added up in the order of the token's choices.  Bound by memory (8192 tokens of
// 7 rows of 4096 bfloat16: 120 us, 537 MB, 4.5 TB/s).
template <class T, class OUT>
__global__ __launch_bounds__(THREADS) void combine_rows_kernel(CombineRowsArgs p, int32_t parts) {
    const int lane = threadIdx.x & 63;
    for (int64_t id = first_wave(); id < p.tokens * parts; id += all_waves()) {
        const int64_t t = id / parts, i = id % parts * (WAVE * V) + lane * V;
        if (i >= p.cols) continue;
        float sum[V] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        if (p.residual) load8(static_cast<const OUT*>(p.residual) + t * p.ld_residual, i, p.cols, sum);
        for (int j = 0; j < p.top_k; ++j) {
            const int64_t r = p.position[t * p.top_k + j];
            if (r < 0 || r >= p.n_rows) continue;
            const float w = p.weights ? p.weights[t * p.top_k + j] : 1.f;
            float v[V];
            load8(static_cast<const T*>(p.src) + r * p.ld, i, p.cols, v);
#pragma unroll
            for (int e = 0; e < V; ++e) sum[e] = fmaf(w, v[e], sum[e]);
        }
        store8(static_cast<OUT*>(p.out) + t * p.ld_out, i, p.cols, sum);
    }
}

// ---- gradients of the pre-activations ----------------------------------------------------------

// dg = d u act'(g), du = d act(g), each rounded once to bfloat16: as operands of the matrix instructions, which multiply no
// wider type at this rate, and so that they are read at half the bytes by the products that follow.  So every term of those
// products is off by up to 2^-8 of itself, whatever their length and the type of their result: relative to the gradients of unrounded
// terms, bfloat16 results are off by 2.35e-3 (2-norm; their own rounding alone is 1.66e-3) and float32 ones by 1.66e-3
// (2.5e-8), from 16 rows to 8191 alike.  Terms of twice the bits would be twice the products.  Bound by memory (8191 x 5632, gelu: 75 us for 461 MB).
template <int ACT>
__global__ __launch_bounds__(THREADS) void gated_grad_kernel(GatedGradArgs p, int32_t parts) {
    int64_t first = 0, end = p.m;
    if (p.offsets) {
        first = min(max((int64_t)p.offsets[0], first), p.m);
        end = min(max((int64_t)p.offsets[p.groups], first), p.m);
    }
    const int64_t padded = (int64_t)parts * V;             // zeros from n on
    for (int64_t id = first * parts + (int64_t)blockIdx.x * THREADS + threadIdx.x; id < end * parts; id += (int64_t)gridDim.x * THREADS) {
        const int64_t r = id / parts, i = id % parts * V;
        float d[V], g[V], u[V], dg[V], du[V];
        load8(p.grad + r * p.ld_grad, i, p.n, d);
        load8(p.pre_gate + r * p.ld_pre, i, p.n, g);
        load8(p.pre_up + r * p.ld_pre, i, p.n, u);
#pragma unroll
        for (int e = 0; e < V; ++e) {
            float value, slope;
            dev::activate<ACT>(g[e], value, slope);
            dg[e] = d[e] * u[e] * slope;
            du[e] = d[e] * value;
        }
        store8(p.grad_pre_gate + r * p.ld_out, i, padded, dg);
        store8(p.grad_pre_up + r * p.ld_out, i, padded, du);
    }
}

// Workgroups for so many items; those beyond the most that a launch takes are looped over.
unsigned blocks_of(int64_t items, int64_t per) { return (unsigned)std::min<int64_t>((items + per - 1) / per, 1 << 22); }

}  // namespace

hipError_t launch_gated_grad(const GatedGradArgs& a, hipStream_t s) {
    if (a.m == 0 || a.n == 0) return hipSuccess;
    const int32_t parts = (int32_t)((a.n + 63) / 64 * (64 / V));
    const dim3 grid(blocks_of(a.m * parts, THREADS)), block(THREADS);
    if (a.activation == MUON_ACT_SILU) hipLaunchKernelGGL((gated_grad_kernel<MUON_ACT_SILU>), grid, block, 0, s, a, parts);
    else if (a.activation == MUON_ACT_GELU) hipLaunchKernelGGL((gated_grad_kernel<MUON_ACT_GELU>), grid, block, 0, s, a, parts);
    else hipLaunchKernelGGL((gated_grad_kernel<MUON_ACT_RELU>), grid, block, 0, s, a, parts);
    return hipGetLastError();
}

namespace {

template <class T>
hipError_t quantize_as(const Int8QuantizeArgs& a, hipStream_t s) {
    // Where there are rows for all CUs: 16 lanes a row of up to 256 values (200000 rows of 128 bfloat16: 27 us, with a wave 77), a
    // wave up to 4096; else, and for longer ones, the workgroup.  A row takes the least number of chunks that holds it, as those behind
    // its end cost what others do: 2, 4 or 8 of a wave; of the workgroup 1, 2, 5 (4097 to 10240 columns, between 2 and 8) or
    // 8, from 16385 columns on none (157 million bfloat16 values in rows of 4096: 86 us, of 4104 in 5 chunks 139, of 8704 in 5 90, of 10240
    // in 5 83, of 10248 in 8 109, of 16384 in 8 90, of 16392 read twice 121).
    const int64_t chunks = (a.kp + V - 1) / V;
    const int lanes = a.cols < V || a.total < 4096 || chunks > 8 * WAVE ? THREADS : chunks > 32 ? WAVE : 16;
    const int64_t each = a.cols < V ? 9 : (chunks + lanes - 1) / lanes;
    const dim3 grid(blocks_of(a.total, THREADS / lanes)), block(THREADS);
#define MUON_QUANTIZE(L, C) hipLaunchKernelGGL((int8_quantize_kernel<T, L, C>), grid, block, 0, s, a)
    if (lanes == 16) MUON_QUANTIZE(16, 2);
    else if (lanes == WAVE && each <= 2) MUON_QUANTIZE(WAVE, 2);
    else if (lanes == WAVE && each <= 4) MUON_QUANTIZE(WAVE, 4);
    else if (lanes == WAVE) MUON_QUANTIZE(WAVE, 8);
    else if (each <= 1) MUON_QUANTIZE(THREADS, 1);
    else if (each <= 2) MUON_QUANTIZE(THREADS, 2);
    else if (each <= 5) MUON_QUANTIZE(THREADS, 5);
    else if (each <= 8) MUON_QUANTIZE(THREADS, 8);
    else MUON_QUANTIZE(THREADS, 0);
#undef MUON_QUANTIZE
    return hipGetLastError();
}

}  // namespace

hipError_t launch_int8_quantize(const Int8QuantizeArgs& a, int32_t src_dtype, hipStream_t s) {
    if (a.total == 0) return hipSuccess;
    return src_dtype == MUON_DTYPE_F32 ? quantize_as<float>(a, s) : quantize_as<uint16_t>(a, s);
}

hipError_t launch_gather_rows(const GatherRowsArgs& a, int32_t dtype, hipStream_t s) {
    const int64_t waves = a.n_rows + (a.grad_weights ? (a.choices + WAVE - 1) / WAVE : 0);
    if (waves == 0) return hipSuccess;
    const dim3 grid(blocks_of(waves, THREADS / WAVE)), block(THREADS);
    if (dtype == MUON_DTYPE_F32) hipLaunchKernelGGL((gather_rows_kernel<float>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((gather_rows_kernel<uint16_t>), grid, block, 0, s, a);
    return hipGetLastError();
}

hipError_t launch_combine_rows(const CombineRowsArgs& a, int32_t dtype, int32_t out_dtype, hipStream_t s) {
    if (a.tokens == 0 || a.cols == 0) return hipSuccess;
    const int32_t parts = (int32_t)((a.cols + WAVE * V - 1) / (WAVE * V));
    const dim3 grid(blocks_of(a.tokens * parts, THREADS / WAVE)), block(THREADS);
    const bool f = dtype == MUON_DTYPE_F32, of = out_dtype == MUON_DTYPE_F32;
    if (f && of) hipLaunchKernelGGL((combine_rows_kernel<float, float>), grid, block, 0, s, a, parts);
    else if (f) hipLaunchKernelGGL((combine_rows_kernel<float, uint16_t>), grid, block, 0, s, a, parts);
    else if (of) hipLaunchKernelGGL((combine_rows_kernel<uint16_t, float>), grid, block, 0, s, a, parts);
    else hipLaunchKernelGGL((combine_rows_kernel<uint16_t, uint16_t>), grid, block, 0, s, a, parts);
    return hipGetLastError();
}

}  // namespace muon
