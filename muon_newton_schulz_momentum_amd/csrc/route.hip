// Routing to experts, its backward pass, and the grouping of the routed rows (gfx950).
//
// Routing, per token with logits x over E experts:
//     s_e = exp(x_e - max x) / sum_i exp(x_i - max x)   or   1 / (1 + exp(-x_e)),
//     key_e = s_e + b_e   (x_e itself without a bias),
//     the top_k largest keys (of the best groups), w_j = scale * s_j / (sum of the chosen s).
// One wave takes one token and keeps its E values in registers (expert lane + 64 i in
// register i).  The scores and keys are float64: two experts' keys that differ in float64 but not in
// float32 would otherwise be taken in the order of their rounding errors.
//
// Backward, with g_j the weights' gradients times scale and w'_j the weights before scale:
//     renormalised: ds_j = (g_j - sum_i g_i w'_i) / sum s;   otherwise ds_j = g_j;
//     sigmoid: dx_j = ds_j s_j (1 - s_j);   softmax: dx_e = s_e (ds_e - sum_i ds_i s_i),
// where the renormalised softmax's inner sum is zero, so only chosen experts get a gradient.
#include <algorithm>

#include "device_common.h"
#include "experts.h"

namespace muon {
namespace {

constexpr float F32_MAX = 3.4028234663852886e38f;
constexpr int ROUTE_WAVES = 4;

__device__ __forceinline__ float load_logit(const float* p) { return *p; }
__device__ __forceinline__ float load_logit(const uint16_t* p) { return dev::bf16_to_f32(*p); }
__device__ __forceinline__ void store_logit(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_logit(uint16_t* p, float v) { *p = dev::f32_to_bf16(v); }

// -inf for an expert that is out (-inf, NaN), the largest finite value for +inf.
__device__ __forceinline__ float clean_logit(float x) { return x > -INFINITY ? fminf(x, F32_MAX) : -INFINITY; }

__device__ __forceinline__ double sigmoid64(double x) { return 1.0 / (1.0 + exp(-x)); }

__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) v = fmaxf(v, __shfl_xor(v, off, 64));
    return v;
}
__device__ __forceinline__ float wave_sum32(float v) {
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off, 64);
    return v;
}

// The largest key of a wave and its index, the lowest index among equal keys; every lane gets it.
__device__ __forceinline__ void wave_best(double& key, int& idx) {
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) {
        const double k = __shfl_xor(key, off, 64);
        const int i = __shfl_xor(idx, off, 64);
        if (k > key || (k == key && i < idx)) { key = k; idx = i; }
    }
}

template <class T, int V>
__global__ __launch_bounds__(64 * ROUTE_WAVES) void route_kernel(RouteArgs p) {
    const int lane = threadIdx.x & 63;
    const int64_t t = (int64_t)blockIdx.x * ROUTE_WAVES + (threadIdx.x >> 6);
    if (t >= p.tokens) return;
    const T* row = static_cast<const T*>(p.logits) + t * p.ld;
    float x[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int e = lane + 64 * i;
        x[i] = e < p.n_experts ? clean_logit(load_logit(row + e)) : -INFINITY;
    }
    double s[V], key[V];
    if (p.score == MUON_SCORE_SOFTMAX) {
        float top = -INFINITY;
#pragma unroll
        for (int i = 0; i < V; ++i) top = fmaxf(top, x[i]);
        top = wave_max(top);
        double z = 0.0;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            s[i] = x[i] > -INFINITY ? exp((double)x[i] - (double)top) : 0.0;
            z += s[i];
        }
        z = dev::wave_sum(z);
#pragma unroll
        for (int i = 0; i < V; ++i) s[i] = z > 0.0 ? s[i] / z : 0.0;
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) s[i] = x[i] > -INFINITY ? sigmoid64((double)x[i]) : 0.0;
    }
    // keys; -inf marks an expert that is out (a NaN key puts it out too)
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int e = lane + 64 * i;
        double k = (double)x[i];
        if ((p.bias || p.n_groups > 1) && x[i] > -INFINITY) {
            k = s[i] + (p.bias ? (double)p.bias[e] : 0.0);
            if (!(k > -INFINITY)) k = -INFINITY;
        }
        key[i] = k;
    }
    if (p.n_groups > 1) {
        // each group's two largest keys, then the groups by rank: a group stays when fewer than
        // top_groups others come before it (a larger sum, or the same and a lower index)
        const int per = p.n_experts / p.n_groups;
        double worth = -INFINITY;                          // lane g: group g's
        for (int g = 0; g < p.n_groups; ++g) {
            double k1 = -INFINITY, k2 = -INFINITY;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int e = lane + 64 * i;
                const double k = e >= g * per && e < (g + 1) * per ? key[i] : -INFINITY;
                if (k > k1) { k2 = k1; k1 = k; }
                else if (k > k2) k2 = k;
            }
#pragma unroll
            for (int off = 32; off > 0; off >>= 1) {
                const double o1 = __shfl_xor(k1, off, 64), o2 = __shfl_xor(k2, off, 64);
                const double lo = fmin(k1, o1);
                k1 = fmax(k1, o1);
                k2 = fmax(lo, fmax(k2, o2));
            }
            if (lane == g) worth = k1 == -INFINITY ? -INFINITY : k1 + (k2 == -INFINITY ? 0.0 : k2);
        }
        int before = 0;
        for (int g = 0; g < p.n_groups; ++g) {
            const double w = __shfl(worth, g, 64);
            if (w > worth || (w == worth && g < lane)) ++before;
        }
        const uint64_t kept = __ballot(lane < p.n_groups && before < p.top_groups);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int e = lane + 64 * i;
            if (e < p.n_experts && !((kept >> (e / per)) & 1)) key[i] = -INFINITY;
            else if (!p.bias) key[i] = (double)x[i];
        }
    }
    int my_expert = -1;
    double my_score = 0.0;
    for (int j = 0; j < p.top_k; ++j) {
        double best = -INFINITY;
        int at = 1 << 20;
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (key[i] > best) { best = key[i]; at = lane + 64 * i; }
        wave_best(best, at);
        if (best == -INFINITY) break;
        double sc = 0.0;
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (at == lane + 64 * i) { sc = s[i]; key[i] = -INFINITY; }
        sc = __shfl(sc, at & 63, 64);
        if (lane == j) { my_expert = at; my_score = sc; }
    }
    double w = my_score;
    if (p.renormalize) {
        const double total = dev::wave_sum(my_score);
        w = total > 0.0 ? my_score / total : 0.0;
    }
    if (lane < p.top_k) {
        p.experts[t * p.top_k + lane] = my_expert;
        p.weights[t * p.top_k + lane] = (float)(w * (double)p.scale);
    }
}

template <class T, int V>
__global__ __launch_bounds__(64 * ROUTE_WAVES) void route_backward_kernel(RouteBackwardArgs p) {
    const int lane = threadIdx.x & 63;
    const int64_t t = (int64_t)blockIdx.x * ROUTE_WAVES + (threadIdx.x >> 6);
    if (t >= p.tokens) return;
    const T* row = static_cast<const T*>(p.logits) + t * p.ld;
    T* grad = static_cast<T*>(p.grad_logits) + t * p.ld_grad;
    // lane j: slot j's expert, logit and gradient
    int e = -1;
    float xj = -INFINITY, g = 0.f;
    if (lane < p.top_k) {
        e = p.experts[t * p.top_k + lane];
        if (e < 0 || e >= p.n_experts) e = -1;
        if (e >= 0) xj = clean_logit(load_logit(row + e));
        if (!(xj > -INFINITY)) e = -1;
        if (e >= 0) g = p.grad_weights[t * p.top_k + lane] * p.scale;
    }
    float out[V];
#pragma unroll
    for (int i = 0; i < V; ++i) out[i] = 0.f;
    float dx = 0.f;                                        // lane j: what slot j adds to its expert
    if (p.score == MUON_SCORE_SIGMOID) {
        const double s = e >= 0 ? sigmoid64((double)xj) : 0.0;
        const double rest = e >= 0 ? 1.0 / (1.0 + exp((double)xj)) : 0.0;   // 1 - s
        if (p.renormalize) {
            const double total = dev::wave_sum(s);
            const double w = total > 0.0 ? s / total : 0.0;
            const double mean = dev::wave_sum((double)g * w);
            dx = e >= 0 ? (float)(w * rest * ((double)g - mean)) : 0.f;
        } else {
            dx = (float)((double)g * s * rest);
        }
    } else if (p.renormalize) {
        const float top = wave_max(xj);
        const double ex = e >= 0 ? exp((double)xj - (double)top) : 0.0;
        const double total = dev::wave_sum(ex);
        const double w = total > 0.0 ? ex / total : 0.0;
        const double mean = dev::wave_sum((double)g * w);
        dx = e >= 0 ? (float)(w * ((double)g - mean)) : 0.f;
    } else {
        float x[V], top = -INFINITY;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int ei = lane + 64 * i;
            x[i] = ei < p.n_experts ? clean_logit(load_logit(row + ei)) : -INFINITY;
            top = fmaxf(top, x[i]);
        }
        top = wave_max(top);
        float z = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            x[i] = x[i] > -INFINITY ? expf(x[i] - top) : 0.f;
            z += x[i];
        }
        z = wave_sum32(z);
        const float inv = z > 0.f ? 1.f / z : 0.f;
        const float pj = e >= 0 ? expf(xj - top) * inv : 0.f;
        const float mean = wave_sum32(g * pj);
        dx = g * pj;
#pragma unroll
        for (int i = 0; i < V; ++i) out[i] = -x[i] * inv * mean;
    }
    for (int j = 0; j < p.top_k; ++j) {
        const int ej = __shfl(e, j, 64);
        const float dj = __shfl(dx, j, 64);
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (ej == lane + 64 * i) out[i] += dj;
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int ei = lane + 64 * i;
        if (ei < p.n_experts) store_logit(grad + ei, out[i]);
    }
}

// ---- grouping ---------------------------------------------------------------------------
//
// A stable counting sort.  A workgroup takes a run of consecutive choices and each of its waves
// a run of those, so that positions follow from counts: choices of an expert in earlier
// runs, then in the earlier waves of this one, then in the earlier lanes of the wave, found
// by matching the bits of the expert across the wave with ballots.

constexpr int GROUP_WAVES = 16;
constexpr int GROUP_THREADS = 64 * GROUP_WAVES;

// Lanes whose value equals this lane's (10 bits are enough for MUON_MAX_EXPERTS; out of range: -1).
__device__ __forceinline__ uint64_t match_lanes(int v) {
    uint64_t m = __ballot(v >= 0);
    if (v < 0) return 0;
#pragma unroll
    for (int b = 0; b < 10; ++b) {
        const bool bit = (v >> b) & 1;
        const uint64_t with = __ballot(bit);
        m &= bit ? with : ~with;
    }
    return m;
}

__device__ __forceinline__ int load_choice(const GroupRowsArgs& p, int64_t i, int64_t end) {
    if (i >= end) return -1;
    const int e = p.experts[i];
    return e >= 0 && e < p.n_experts ? e : -1;
}

// Exclusive prefix over the workgroup of one value per thread (and the total).
__device__ __forceinline__ int block_prefix(int v, int* wave_tot, int& total) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int inc = v;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
        const int o = __shfl_up(inc, off, 64);
        if (lane >= off) inc += o;
    }
    if (lane == 63) wave_tot[wave] = inc;
    __syncthreads();
    int before = 0;
    total = 0;
    for (int w = 0; w < GROUP_WAVES; ++w) {
        if (w < wave) before += wave_tot[w];
        total += wave_tot[w];
    }
    __syncthreads();
    return before + inc - v;
}

// Places the choices [lo, hi): cursor[w][e] is where wave w's first choice of expert e goes.
__device__ __forceinline__ void place(const GroupRowsArgs& p, int64_t lo, int64_t hi, int64_t per_wave, int* cursor) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t w0 = lo + wave * per_wave, w1 = min(hi, w0 + per_wave);
    int* mine = cursor + wave * p.n_experts;
    for (int64_t i0 = w0; i0 < w1; i0 += 64) {
        const int64_t i = i0 + lane;
        const int e = load_choice(p, i, w1);
        const uint64_t same = match_lanes(e);
        int at = -1;
        if (e >= 0) at = mine[e] + __popcll(same & ((1ull << lane) - 1));
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");   // the reads come before the write
        __builtin_amdgcn_wave_barrier();
        if (e >= 0 && (same >> lane) == 1) mine[e] = at + 1;   // the last lane of the expert
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        if (i < w1) p.position[i] = at;
        if (e >= 0) p.rows[at] = (int32_t)i;
    }
}

// hist[w][e]: choices of expert e in wave w's run of [lo, hi).
__device__ __forceinline__ void count(const GroupRowsArgs& p, int64_t lo, int64_t hi, int64_t per_wave, int* hist) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    for (int i = threadIdx.x; i < GROUP_WAVES * p.n_experts; i += GROUP_THREADS) hist[i] = 0;
    __syncthreads();
    const int64_t w0 = lo + wave * per_wave, w1 = min(hi, w0 + per_wave);
    for (int64_t i = w0 + lane; i < w1; i += 64) {
        const int e = load_choice(p, i, w1);
        if (e >= 0) atomicAdd(&hist[wave * p.n_experts + e], 1);   // a count: the order does not matter
    }
    __syncthreads();
}

// All of a small call in one workgroup.
__global__ __launch_bounds__(GROUP_THREADS) void group_single_kernel(GroupRowsArgs p) {
    extern __shared__ int lds[];
    __shared__ int wave_tot[GROUP_WAVES];
    const int64_t per_wave = ((p.n + GROUP_WAVES - 1) / GROUP_WAVES + 63) / 64 * 64;
    count(p, 0, p.n, per_wave, lds);
    const int e = threadIdx.x;
    int c = 0;
    if (e < p.n_experts)
        for (int w = 0; w < GROUP_WAVES; ++w) c += lds[w * p.n_experts + e];
    const int padded = (c + p.align - 1) / p.align * p.align;
    int total;
    const int start = block_prefix(padded, wave_tot, total);
    if (e < p.n_experts) {
        int at = start;
        for (int w = 0; w < GROUP_WAVES; ++w) {
            const int h = lds[w * p.n_experts + e];
            lds[w * p.n_experts + e] = at;
            at += h;
        }
        p.counts[e] = c;
        p.offsets[e] = start;
        for (int r = start + c; r < start + padded; ++r) p.rows[r] = -1;
    }
    if (threadIdx.x == 0) p.offsets[p.n_experts] = total;
    for (int64_t r = total + threadIdx.x; r < p.capacity; r += GROUP_THREADS) p.rows[r] = -1;
    __syncthreads();
    place(p, 0, p.n, per_wave, lds);
}

__global__ __launch_bounds__(GROUP_THREADS) void group_count_kernel(GroupRowsArgs p) {
    extern __shared__ int lds[];
    const int64_t lo = blockIdx.x * GROUP_CHUNK, hi = min(p.n, lo + GROUP_CHUNK);
    count(p, lo, hi, GROUP_CHUNK / GROUP_WAVES, lds);
    for (int e = threadIdx.x; e < p.n_experts; e += GROUP_THREADS) {
        int c = 0;
        for (int w = 0; w < GROUP_WAVES; ++w) c += lds[w * p.n_experts + e];
        p.partial[blockIdx.x * (int64_t)p.n_experts + e] = c;
    }
}

// partial[chunk][e] becomes the row where the chunk's first choice of expert e goes.
__global__ __launch_bounds__(GROUP_THREADS) void group_scan_kernel(GroupRowsArgs p) {
    __shared__ int wave_tot[GROUP_WAVES];
    const int e = threadIdx.x;
    int c = 0;
    if (e < p.n_experts)
        for (int64_t b = 0; b < p.chunks; ++b) c += p.partial[b * p.n_experts + e];
    const int padded = (c + p.align - 1) / p.align * p.align;
    int total;
    const int start = block_prefix(padded, wave_tot, total);
    if (e < p.n_experts) {
        int at = start;
        for (int64_t b = 0; b < p.chunks; ++b) {
            const int h = p.partial[b * p.n_experts + e];
            p.partial[b * p.n_experts + e] = at;
            at += h;
        }
        p.counts[e] = c;
        p.offsets[e] = start;
    }
    if (threadIdx.x == 0) p.offsets[p.n_experts] = total;
}

__global__ __launch_bounds__(GROUP_THREADS) void group_place_kernel(GroupRowsArgs p) {
    extern __shared__ int lds[];
    const int64_t lo = blockIdx.x * GROUP_CHUNK, hi = min(p.n, lo + GROUP_CHUNK);
    count(p, lo, hi, GROUP_CHUNK / GROUP_WAVES, lds);
    for (int e = threadIdx.x; e < p.n_experts; e += GROUP_THREADS) {
        int at = p.partial[blockIdx.x * (int64_t)p.n_experts + e];
        for (int w = 0; w < GROUP_WAVES; ++w) {
            const int h = lds[w * p.n_experts + e];
            lds[w * p.n_experts + e] = at;
            at += h;
        }
    }
    __syncthreads();
    place(p, lo, hi, GROUP_CHUNK / GROUP_WAVES, lds);
    // the padding of segments, and what lies behind the last one
    for (int64_t e = blockIdx.x; e < p.n_experts; e += gridDim.x)
        for (int64_t r = (int64_t)p.offsets[e] + p.counts[e] + threadIdx.x; r < p.offsets[e + 1]; r += GROUP_THREADS)
            p.rows[r] = -1;
    const int64_t step = (int64_t)gridDim.x * GROUP_THREADS;
    for (int64_t r = p.offsets[p.n_experts] + blockIdx.x * (int64_t)GROUP_THREADS + threadIdx.x; r < p.capacity; r += step)
        p.rows[r] = -1;
}

__global__ __launch_bounds__(GROUP_THREADS) void balance_kernel(const float* bias, const int32_t* counts, int32_t n,
                                                                 float rate, float* out) {
    __shared__ long long part[GROUP_WAVES];
    const int e = threadIdx.x;
    const long long c = e < n ? counts[e] : 0;
    long long sum = c;
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) sum += __shfl_xor(sum, off, 64);
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = sum;
    __syncthreads();
    long long total = 0;
    for (int w = 0; w < GROUP_WAVES; ++w) total += part[w];
    if (e >= n) return;
    const long long d = total - c * n;
    out[e] = d > 0 ? bias[e] + rate : d < 0 ? bias[e] - rate : bias[e];
}

template <class T>
hipError_t route_by_width(const RouteArgs& a, hipStream_t s) {
    const dim3 grid((unsigned)((a.tokens + ROUTE_WAVES - 1) / ROUTE_WAVES)), block(64 * ROUTE_WAVES);
    if (a.n_experts <= 128) hipLaunchKernelGGL((route_kernel<T, 2>), grid, block, 0, s, a);
    else if (a.n_experts <= 512) hipLaunchKernelGGL((route_kernel<T, 8>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((route_kernel<T, 16>), grid, block, 0, s, a);
    return hipGetLastError();
}

template <class T>
hipError_t backward_by_width(const RouteBackwardArgs& a, hipStream_t s) {
    const dim3 grid((unsigned)((a.tokens + ROUTE_WAVES - 1) / ROUTE_WAVES)), block(64 * ROUTE_WAVES);
    if (a.n_experts <= 128) hipLaunchKernelGGL((route_backward_kernel<T, 2>), grid, block, 0, s, a);
    else if (a.n_experts <= 512) hipLaunchKernelGGL((route_backward_kernel<T, 8>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((route_backward_kernel<T, 16>), grid, block, 0, s, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_route(const RouteArgs& a, int32_t dtype, hipStream_t s) {
    return dtype == MUON_DTYPE_F32 ? route_by_width<float>(a, s) : route_by_width<uint16_t>(a, s);
}

hipError_t launch_route_backward(const RouteBackwardArgs& a, int32_t dtype, hipStream_t s) {
    return dtype == MUON_DTYPE_F32 ? backward_by_width<float>(a, s) : backward_by_width<uint16_t>(a, s);
}

hipError_t launch_group_rows(const GroupRowsArgs& a, hipStream_t s) {
    const unsigned lds = (unsigned)(GROUP_WAVES * a.n_experts * sizeof(int));   // at most 64 KiB
    const dim3 block(GROUP_THREADS);
    if (a.n <= GROUP_SINGLE_MAX) {
        hipLaunchKernelGGL(group_single_kernel, dim3(1), block, lds, s, a);
        return hipGetLastError();
    }
    const dim3 grid((unsigned)a.chunks);
    hipLaunchKernelGGL(group_count_kernel, grid, block, lds, s, a);
    hipLaunchKernelGGL(group_scan_kernel, dim3(1), block, 0, s, a);
    hipLaunchKernelGGL(group_place_kernel, grid, block, lds, s, a);
    return hipGetLastError();
}

hipError_t launch_balance(const float* bias, const int32_t* counts, int32_t n, float rate, float* out, hipStream_t s) {
    hipLaunchKernelGGL(balance_kernel, dim3(1), dim3(GROUP_THREADS), 0, s, bias, counts, n, rate, out);
    return hipGetLastError();
}

}  // namespace muon
