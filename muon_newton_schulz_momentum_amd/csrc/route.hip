// Routing to experts, its backward pass, and the grouping of the routed rows (gfx950).
//
// Routing, per token with logits x over E experts:
//     s_e = exp(x_e - max x) / sum_i exp(x_i - max x)   or   1 / (1 + exp(-x_e)),
//     key_e = s_e + b_e   (x_e itself without a bias),
//     the top_k largest keys (of the best groups), w_j = scale * s_j / (sum of the chosen s).
// The choice is that of float64 scores and keys: two experts' keys that differ in float64 but not in
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

// Renormalised weights are ratios, which exist where the scores underflow: the softmax's are formed from the largest chosen
// logit on, and so are the sigmoid's where all chosen logits are below this (there 1 / (1 + exp(-x)) is exp(x) in float64).
constexpr float TINY_SIGMOID = -700.f;

__device__ __forceinline__ double sigmoid64(double x) { return 1.0 / (1.0 + exp(-x)); }

__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) v = fmaxf(v, __shfl_xor(v, off, 64));
    return v;
}

template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xf, 0xf, false);
}
template <int CTRL>
__device__ __forceinline__ float dppf(float v) { return __uint_as_float(dpp<CTRL>(__float_as_uint(v))); }

// Exchanges that, one after another, spread over 2, 4, 8 and 16 lanes: neighbours, pairs, halves of 8, halves of 16.
constexpr int XCHG_1 = 0xb1, XCHG_2 = 0x4e, XCHG_4 = 0x141, XCHG_8 = 0x140;

__device__ __forceinline__ uint32_t row_value(uint32_t v, int row) { return (uint32_t)__builtin_amdgcn_readlane((int)v, 16 * row); }

template <int CTRL>
__device__ __forceinline__ double dppd(double v) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    return __builtin_bit_cast(double, (uint64_t)dpp<CTRL>((uint32_t)u) | ((uint64_t)dpp<CTRL>((uint32_t)(u >> 32)) << 32));
}
__device__ __forceinline__ double row_valued(double v, int row) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    return __builtin_bit_cast(double, (uint64_t)row_value((uint32_t)u, row) | ((uint64_t)row_value((uint32_t)(u >> 32), row) << 32));
}

// The largest key of a wave and its index, the lowest index among equal keys; every lane gets it.
__device__ __forceinline__ void wave_best(double& key, int& idx) {
    auto better = [&](double k, int i) {
        if (k > key || (k == key && i < idx)) { key = k; idx = i; }
    };
    better(dppd<XCHG_1>(key), (int)dpp<XCHG_1>((uint32_t)idx));
    better(dppd<XCHG_2>(key), (int)dpp<XCHG_2>((uint32_t)idx));
    better(dppd<XCHG_4>(key), (int)dpp<XCHG_4>((uint32_t)idx));
    better(dppd<XCHG_8>(key), (int)dpp<XCHG_8>((uint32_t)idx));
    const double k = key;
    const int i = idx;
#pragma unroll
    for (int r = 0; r < 4; ++r) better(row_valued(k, r), (int)row_value((uint32_t)i, r));
}

// The two largest keys of 16 lanes, and of a wave.
__device__ __forceinline__ void merge2(double& k1, double& k2, double o1, double o2) {
    k2 = fmax(fmin(k1, o1), fmax(k2, o2));
    k1 = fmax(k1, o1);
}
__device__ __forceinline__ void row_best2(double& k1, double& k2) {
    merge2(k1, k2, dppd<XCHG_1>(k1), dppd<XCHG_1>(k2));
    merge2(k1, k2, dppd<XCHG_2>(k1), dppd<XCHG_2>(k2));
    merge2(k1, k2, dppd<XCHG_4>(k1), dppd<XCHG_4>(k2));
    merge2(k1, k2, dppd<XCHG_8>(k1), dppd<XCHG_8>(k2));
}
__device__ __forceinline__ void wave_best2(double& k1, double& k2) {
    row_best2(k1, k2);
    const double r1 = k1, r2 = k2;
    k1 = row_valued(r1, 0);
    k2 = row_valued(r2, 0);
#pragma unroll
    for (int r = 1; r < 4; ++r) merge2(k1, k2, row_valued(r1, r), row_valued(r2, r));
}
// A group's worth by its two largest keys (-inf: none).
__device__ __forceinline__ double worth_of(double k1, double k2) {
    return k1 == -INFINITY ? -INFINITY : k1 + (k2 == -INFINITY ? 0.0 : k2);
}

// One token by one wave in float64, expert lane + 64 i in the lane's i-th place of x and key (LDS).  route_kernel comes
// here for the odd token, with the code not in the instruction cache: so the loops with exponentials are not
// unrolled (16 KiB of unrolled code for 512 experts took 13 us for one token).
template <class T, int V>
__device__ __forceinline__ void route_exact(const RouteArgs& p, int64_t t, float* x, double* key) {
    const int lane = threadIdx.x & 63;
    const T* row = static_cast<const T*>(p.logits) + t * p.ld;
    const bool softmax = p.score == MUON_SCORE_SOFTMAX;
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int e = lane + 64 * i;
        const float v = e < p.n_experts ? clean_logit(load_logit(row + e)) : -INFINITY;
        x[e] = v;
        top = fmaxf(top, v);
    }
    top = wave_max(top);
    // the sigmoid, or the softmax before its division by z
    auto raw = [&](float v) {
        const double ex = exp(softmax ? (double)v - (double)top : -(double)v);
        return softmax ? ex : 1.0 / (1.0 + ex);
    };
    const bool scored = p.bias || p.n_groups > 1;
    double z = 1.0;
    if (scored || (softmax && !p.renormalize)) {           // otherwise z cancels
        z = 0.0;
#pragma unroll 1
        for (int i = 0; i < V; ++i) {
            const float v = x[lane + 64 * i];
            const double s = v > -INFINITY ? raw(v) : 0.0;
            key[lane + 64 * i] = s;
            z += s;
        }
        z = softmax ? dev::wave_sum(z) : 1.0;
    }
    // keys; -inf marks an expert that is out (a NaN key puts it out too)
#pragma unroll 1
    for (int i = 0; i < V; ++i) {
        const int e = lane + 64 * i;
        double k = (double)x[e];
        if (scored && x[e] > -INFINITY) {
            k = key[e] / z + (p.bias ? (double)p.bias[e] : 0.0);
            if (!(k > -INFINITY)) k = -INFINITY;
        }
        key[e] = k;
    }
    if (p.n_groups > 1) {
        // each group's two largest keys, then the groups by rank: a group stays when fewer than
        // top_groups others come before it (a larger sum, or the same and a lower index)
        const int per = p.n_experts / p.n_groups;
        double worth = -INFINITY;                          // lane g: group g's
        for (int g = 0; g < p.n_groups; ++g) {
            double k1 = -INFINITY, k2 = -INFINITY;
            for (int i = g * per / 64; i <= ((g + 1) * per - 1) / 64; ++i) {
                const int e = lane + 64 * i;
                const double k = e >= g * per && e < (g + 1) * per ? key[e] : -INFINITY;
                if (k > k1) { k2 = k1; k1 = k; }
                else if (k > k2) k2 = k;
            }
            wave_best2(k1, k2);
            if (lane == g) worth = worth_of(k1, k2);
        }
        int before = 0;
        for (int g = 0; g < p.n_groups; ++g) {
            const double w = __shfl(worth, g, 64);
            if (w > worth || (w == worth && g < lane)) ++before;
        }
        const uint64_t kept = __ballot(lane < p.n_groups && before < p.top_groups);
#pragma unroll 1
        for (int i = 0; i < V; ++i) {
            const int e = lane + 64 * i;
            if (e < p.n_experts && !((kept >> (e / per)) & 1)) key[e] = -INFINITY;
            else if (!p.bias) key[e] = (double)x[e];
        }
    }
    int my_expert = -1;
    for (int j = 0; j < p.top_k; ++j) {
        double best = -INFINITY;
        int at = 1 << 20;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const double k = key[lane + 64 * i];
            if (k > best) { best = k; at = lane + 64 * i; }
        }
        wave_best(best, at);
        if (best == -INFINITY) break;
        if ((at & 63) == lane) key[at] = -INFINITY;
        if (lane == j) my_expert = at;
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");   // other lanes' places of x
    __builtin_amdgcn_wave_barrier();
    const float my_x = my_expert >= 0 ? x[my_expert] : -INFINITY;
    double w;
    if (p.renormalize) {
        const float high = wave_max(my_x);
        const double s = my_expert < 0 ? 0.0 : softmax || high < TINY_SIGMOID ? exp((double)my_x - (double)high) : raw(my_x);
        const double total = dev::wave_sum(s);
        w = total > 0.0 ? s / total : 0.0;
    } else {
        w = my_expert >= 0 ? raw(my_x) / z : 0.0;
    }
    if (lane < p.top_k) {
        p.experts[t * p.top_k + lane] = my_expert;
        p.weights[t * p.top_k + lane] = (float)(w * (double)p.scale);
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");   // the next token's come after
    __builtin_amdgcn_wave_barrier();
}

template <class T, int V>
__global__ __launch_bounds__(64 * ROUTE_WAVES) void route_exact_kernel(RouteArgs p) {
    __shared__ double key[ROUTE_WAVES][64 * V];
    __shared__ float x[ROUTE_WAVES][64 * V];
    const int wave = threadIdx.x >> 6;
    const int64_t t = (int64_t)blockIdx.x * ROUTE_WAVES + wave;
    if (t < p.tokens) route_exact<T, V>(p, t, x[wave], key[wave]);
}

// ---- 16 or 64 lanes a token -----------------------------------------------------------------
//
// Lane l of LT takes experts 4 LT c + 4 l + v (c < C, v < 4).  Scores and keys are float32, as ordered integers
// whose last 6 bits give way to the expert's place in its lane.  Each lane sorts out its 4 largest (a maximum
// and three medians per value; again when they are used up), and top_k + 1 rounds take the largest of all lanes.
// What float32 cannot decide is found by looking at what was taken: two neighbours nearer than the keys' error.
// They (with a bias, in one token of forty at 512 experts) are settled by
// taking on to 16 experts and ranking those by their float64 keys, and two groups at the border by their float64 sums;
// whatever is left is done again by the whole wave in float64.  So the choice is always the float64 one.
// 65537 tokens of 512 float32 logits, 7 by softmax: 40 us, 3.4 TB/s, bound by the sorting's vector instructions (1140 a wave:
// issued in all of its busy cycles); 8192 in 8 groups by sigmoid and bias, bfloat16: 21 us, two waves a SIMD, each a
// chain of reductions (vector instructions in half of the busy cycles).
constexpr int FAST_MAX_K = 15;
constexpr int64_t WIDE_MAX_TOKENS = 4096;

// Over the LT lanes of a token, to all of them.
template <int LT>
__device__ __forceinline__ uint32_t token_max(uint32_t v) {
    v = max(v, dpp<XCHG_1>(v));
    v = max(v, dpp<XCHG_2>(v));
    v = max(v, dpp<XCHG_4>(v));
    v = max(v, dpp<XCHG_8>(v));
    if (LT == 64) v = max(max(row_value(v, 0), row_value(v, 1)), max(row_value(v, 2), row_value(v, 3)));
    return v;
}
template <int LT>
__device__ __forceinline__ float token_maxf(float v) {
    v = fmaxf(v, dppf<XCHG_1>(v));
    v = fmaxf(v, dppf<XCHG_2>(v));
    v = fmaxf(v, dppf<XCHG_4>(v));
    v = fmaxf(v, dppf<XCHG_8>(v));
    if (LT == 64) {
        const uint32_t u = __float_as_uint(v);
        v = fmaxf(fmaxf(__uint_as_float(row_value(u, 0)), __uint_as_float(row_value(u, 1))),
                  fmaxf(__uint_as_float(row_value(u, 2)), __uint_as_float(row_value(u, 3))));
    }
    return v;
}
template <int LT>
__device__ __forceinline__ float token_sum(float v) {
    v += dppf<XCHG_1>(v);
    v += dppf<XCHG_2>(v);
    v += dppf<XCHG_4>(v);
    v += dppf<XCHG_8>(v);
    if (LT == 64) {
        const uint32_t u = __float_as_uint(v);
        v = (__uint_as_float(row_value(u, 0)) + __uint_as_float(row_value(u, 1))) +
            (__uint_as_float(row_value(u, 2)) + __uint_as_float(row_value(u, 3)));
    }
    return v;
}

// Order-preserving bits of a float32 and back; the zeros are equal (-0 + 0 is 0).
__device__ __forceinline__ uint32_t ordered(float f) {
    const uint32_t u = __float_as_uint(f + 0.f);
    return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t u) {
    return __uint_as_float(u ^ (((u >> 31) - 1u) | 0x80000000u));
}

__device__ __forceinline__ uint32_t med3(uint32_t a, uint32_t b, uint32_t c) {
    return max(min(a, b), min(max(a, b), c));
}

// Two largest of two pairs, each in falling order.
__device__ __forceinline__ void merge2(float& a1, float& a2, float b1, float b2) {
    a2 = fmaxf(fminf(a1, b1), fmaxf(a2, b2));
    a1 = fmaxf(a1, b1);
}

__device__ __forceinline__ void load4(const float* p, float (&v)[4]) {
    const float4 a = *reinterpret_cast<const float4*>(p);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
}
__device__ __forceinline__ void load4(const uint16_t* p, float (&v)[4]) {
    const uint2 a = *reinterpret_cast<const uint2*>(p);
    v[0] = __uint_as_float(a.x << 16); v[1] = __uint_as_float(a.x & 0xffff0000u);
    v[2] = __uint_as_float(a.y << 16); v[3] = __uint_as_float(a.y & 0xffff0000u);
}

// Two keys (a above b) that float32 tells apart: scores are off by less than 2^-21, and the place has taken 2^-17 of
// the size away.
__device__ __forceinline__ bool apart(float a, float b) { return a - b > 0x1p-16f * fmaxf(1.f, fabsf(a)); }

// GROUPS: n_groups > 1 (16 lanes only).  Four waves a SIMD at least: at three, which the widest form would have, 65536 tokens
// in 8 groups take 93 us instead of 78.
template <class T, int LT, int C, bool GROUPS>
__global__ __launch_bounds__(64 * ROUTE_WAVES) __attribute__((amdgpu_waves_per_eu(4))) void route_kernel(RouteArgs p, int vec) {
    constexpr int PT = 64 / LT;                            // tokens a wave
    static_assert(!GROUPS || LT == 16, "groups lie in 16 lanes");
    constexpr int V = LT * C / 16;
    // of a wave: its four tokens' keys while their groups are chosen, later the token done again (keys, logits)
    constexpr int KEYS = 66 * C + 1, DOUBLES = std::max(64 * V + 32 * V, GROUPS ? 2 * KEYS : 0);
    __shared__ double room[ROUTE_WAVES][DOUBLES];
    const int lane = threadIdx.x & 63, l = lane & (LT - 1);
    const int64_t t0 = ((int64_t)blockIdx.x * ROUTE_WAVES + (threadIdx.x >> 6)) * PT;
    if (t0 >= p.tokens) return;
    const int64_t t = t0 + lane / LT;
    const bool live = t < p.tokens;
    const T* row = static_cast<const T*>(p.logits) + (live ? t : t0) * p.ld;
    auto expert = [&](int c, int v) { return 4 * LT * c + 4 * l + v; };
    float x[C][4];
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int e = expert(c, 0);
        if (vec) {
            if (e < p.n_experts) load4(row + e, x[c]);
            else x[c][0] = x[c][1] = x[c][2] = x[c][3] = -INFINITY;
        } else {
#pragma unroll
            for (int v = 0; v < 4; ++v) x[c][v] = e + v < p.n_experts ? load_logit(row + e + v) : -INFINITY;
        }
    }
    float top = -INFINITY;
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            x[c][v] = clean_logit(x[c][v]);
            top = fmaxf(top, x[c][v]);
        }
    top = token_maxf<LT>(top);
    const bool any = top > -INFINITY;
    const bool softmax = p.score == MUON_SCORE_SOFTMAX;
    const bool scored = p.bias || GROUPS;                  // the choice goes by scores
    // key[c][v]: the score plus bias; and the softmax's sum
    float z = 0.f, key[C][4];
    if (softmax && (scored || !p.renormalize)) {
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                key[c][v] = any ? __expf(x[c][v] - top) : 0.f;
                z += key[c][v];
            }
        z = token_sum<LT>(z);
        const float inv = any ? 1.f / z : 0.f;
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int v = 0; v < 4; ++v) key[c][v] *= inv;
    } else if (scored) {
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int v = 0; v < 4; ++v) key[c][v] = __builtin_amdgcn_rcpf(1.f + __expf(-x[c][v]));
    }
    if (p.bias) {
#pragma unroll
        for (int c = 0; c < C; ++c) {
            float b[4] = {0.f, 0.f, 0.f, 0.f};
            if (p.n_experts % 4 == 0) {
                if (expert(c, 0) < p.n_experts) load4(p.bias + expert(c, 0), b);
            } else {
#pragma unroll
                for (int v = 0; v < 4; ++v)
                    if (expert(c, v) < p.n_experts) b[v] = p.bias[expert(c, v)];
            }
#pragma unroll
            for (int v = 0; v < 4; ++v) key[c][v] += b[v];
        }
    }
    bool again = false;                                    // for the whole wave in float64
    uint64_t kept = ~0ull;                                 // groups that stay
    float* keys = reinterpret_cast<float*>(room[threadIdx.x >> 6]) + (GROUPS ? (lane >> 4) * KEYS : 0);
    const int per = GROUPS ? p.n_experts / p.n_groups : 1;
    if constexpr (GROUPS) {
        // Through LDS, expert e at e + e / 32 (and tokens 66 C + 1 apart), so that groups begin on different banks.  Up to
        // 16 groups: 2^share lanes each; more: a lane takes every 16th.
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int v = 0; v < 4; ++v)                    // a NaN key is out
                keys[66 * c + 4 * l + (l >> 3) + v] = x[c][v] > -INFINITY && key[c][v] > -INFINITY ? key[c][v] : -INFINITY;
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        const int share = p.n_groups <= 2 ? 3 : p.n_groups <= 4 ? 2 : p.n_groups <= 8 ? 1 : 0, step = 1 << share;
        // lane l: groups l + 16 i, their two largest added up, and what float32 may be off by
        float worth[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY}, off[4] = {0.f, 0.f, 0.f, 0.f};
        // A sigmoid is off by less than 2^-21, a softmax (but for its row's sum) by less than that part of the largest one, 1 / z; a
        // key and the sum by their rounding, 2^-24 of a size that is at most the larger of the two keys (which may cancel) or
        // twice that.  With a bias the error of z counts, too (without one it is a factor of all groups): 2^-18 of the scores.
        const float largest = !softmax ? 1.f : any ? 1.f / z : 0.f;
        const float of_scores = 0x1p-20f * largest + (softmax && p.bias ? 0x1p-18f * fminf(2.f * largest, 1.f) : 0.f);
#pragma unroll 1
        for (int i = 0; 16 * i < p.n_groups; ++i) {
            const int g = (l >> share) + 16 * i, first = g * per, end = g < p.n_groups ? first + per : first;
            float m1 = -INFINITY, m2 = -INFINITY;
            for (int e0 = first + (l & (step - 1)); e0 < end; e0 += 8 * step)
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int e = e0 + j * step;
                    const float k = e < end ? keys[e + (e >> 5)] : -INFINITY;
                    m2 = fmaxf(fminf(m1, k), m2);
                    m1 = fmaxf(m1, k);
                }
            if (share >= 1) merge2(m1, m2, dppf<XCHG_1>(m1), dppf<XCHG_1>(m2));
            if (share >= 2) merge2(m1, m2, dppf<XCHG_2>(m1), dppf<XCHG_2>(m2));
            if (share >= 3) merge2(m1, m2, dppf<XCHG_4>(m1), dppf<XCHG_4>(m2));
            m2 = m2 == -INFINITY ? 0.f : m2;
            // an infinite key is exact; finite sums stay finite (and so above a group without an expert)
            const bool sum = fabsf(m1) != INFINITY;
            const float w = sum ? fminf(fmaxf(m1 + m2, -F32_MAX), F32_MAX) : m1;
            const float d = sum ? of_scores + 0x1p-21f * fmaxf(fabsf(m1), fabsf(m2)) : 0.f;
            const int from = (lane & 48) + ((l << share) & 15);
            const float my_w = __shfl(w, from, 64), my_d = __shfl(d, from, 64);
#pragma unroll
            for (int q = 0; q < 4; ++q)
                if (q == i && l + 16 * i < p.n_groups) {
                    worth[q] = my_w;
                    off[q] = my_d;
                }
        }
        float best[4] = {worth[0], worth[1], worth[2], worth[3]};
        kept = 0;
        for (int r = 0; r < p.top_groups; ++r) {           // the largest; of equal sums the lowest group
            const float w = token_maxf<LT>(fmaxf(fmaxf(best[0], best[1]), fmaxf(best[2], best[3])));
            uint32_t at = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (best[i] == w && l + 16 * i < p.n_groups && !((kept >> (l + 16 * i)) & 1)) at = max(at, (uint32_t)(64 - (l + 16 * i)));
            at = token_max<LT>(at);
            if (at != 0) kept |= 1ull << (64 - (int)at);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (l + 16 * i == 64 - (int)at) best[i] = -INFINITY;
        }
        // what those that stay are worth at least, the others at most
        float low = INFINITY, high = -INFINITY;
        auto stays_in = [&](int i) { return (kept >> (l + 16 * i)) & 1; };
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (l + 16 * i >= p.n_groups) continue;
            if (stays_in(i)) low = fminf(low, worth[i] - off[i]);
            else if (worth[i] > -INFINITY) high = fmaxf(high, worth[i] + off[i]);
        }
        low = -token_maxf<LT>(-low);
        high = token_maxf<LT>(high);
        const bool near = high > -INFINITY && !(low > high);
        if (__ballot(near)) {
            // which of either side could belong to the other
            float both = 0.f;
            uint32_t in = 0, out = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (l + 16 * i >= p.n_groups || worth[i] == -INFINITY) continue;
                if (stays_in(i)) {
                    if (!(worth[i] - off[i] > high)) { both += 1.f; in = (uint32_t)(l + 16 * i); }
                } else if (!(worth[i] + off[i] < low)) {
                    both += 64.f;
                    out = (uint32_t)(l + 16 * i);
                }
            }
            both = token_sum<LT>(both);
            const int last_in = (int)token_max<LT>(in), first_out = (int)token_max<LT>(out);
            // one of each: those two groups alone in float64, unless their scores need the whole row's sum
            again |= near && (both != 65.f || (softmax && p.bias));
            double sums[2];
#pragma unroll 1
            for (int side = 0; side < 2; ++side) {
                double k1 = -INFINITY, k2 = -INFINITY;
                const int g0 = (side == 0 ? last_in : first_out) * per;
#pragma unroll 1
                for (int e0 = 4 * l; e0 < per; e0 += 64)
#pragma unroll
                    for (int v = 0; v < 4; ++v) {
                        if (!near || e0 + v >= per) continue;
                        const float xv = clean_logit(load_logit(row + g0 + e0 + v));
                        const double ex = exp(softmax ? (double)xv - (double)top : -(double)xv);
                        double k = (softmax ? ex : 1.0 / (1.0 + ex)) + (p.bias ? (double)p.bias[g0 + e0 + v] : 0.0);
                        if (!(xv > -INFINITY && k > -INFINITY)) k = -INFINITY;
                        merge2(k1, k2, k, -INFINITY);
                    }
                row_best2(k1, k2);
                sums[side] = worth_of(k1, k2);
            }
            if (near && both == 65.f && (sums[1] > sums[0] || (sums[1] == sums[0] && first_out < last_in)))
                kept ^= 1ull << last_in | 1ull << first_out;
        }
    }
    // Each lane's 4 largest keys, ordered, the place in the lane in the last 6 bits (larger: lower expert).  bfloat16
    // logits are decided by 16 bits: there the expert itself fits behind them, and equal logits need no second look.  (One
    // up: +inf, as float32's largest value, is above bfloat16's largest; the others' lower bits are all zeros or, negative, ones.)
    const bool whole = sizeof(T) == 2 && !p.bias;
    uint32_t bits[C][4];
    const uint32_t inv = GROUPS ? (1u << 20) / (uint32_t)per + 1 : 0;   // e / per is e * inv >> 20 for e * per < 2^20
#pragma unroll
    for (int c = 0; c < C; ++c) {
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            const bool stays = !GROUPS || (kept >> (((uint32_t)expert(c, v) * inv >> 20) & 63u)) & 1;
            // (from LDS where it is there: fewer registers while the groups are chosen)
            const float k = !p.bias ? x[c][v] : GROUPS ? keys[66 * c + 4 * l + (l >> 3) + v] : key[c][v];
            const bool in = stays && x[c][v] > -INFINITY && k > -INFINITY;
            const uint32_t o = ordered(k);
            const uint32_t kv = whole ? ((o + 1u) & 0xffff0000u) | (uint32_t)(1023 - expert(c, v)) : (o & ~63u) | (uint32_t)(63 - (4 * c + v));
            bits[c][v] = in ? kv : 0u;
        }
    }
    uint32_t k0, k1, k2, k3;                               // the 4 largest below `below`
    int had = 0;                                           // of them taken
    auto sort_out = [&](uint32_t below, bool me) {
        uint32_t a0 = 0, a1 = 0, a2 = 0, a3 = 0;
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                const uint32_t u = bits[c][v] < below ? bits[c][v] : 0u;
                a3 = med3(a2, a3, u);
                a2 = med3(a1, a2, u);
                a1 = med3(a0, a1, u);
                a0 = max(a0, u);
            }
        if (me) { k0 = a0; k1 = a1; k2 = a2; k3 = a3; had = 0; }
    };
    sort_out(0xffffffffu, true);
    int mine = -1;                                         // lane j: the j-th expert taken
    auto take = [&](uint32_t w, int j) {
        // the winner's expert to every lane of the token; the lowest of equal bits
        const int place = 63 - (int)(w & 63u);
        const int here = whole ? 1023 - (int)(w & 1023u) : 4 * LT * (place >> 2) + 4 * l + (place & 3);
        const int e = 1024 - (int)token_max<LT>(w != 0 && k0 == w ? (uint32_t)(1024 - here) : 0u);
        const bool won = w != 0 && k0 == w && here == e;
        if (l == j && w != 0) mine = e;
        if (won) {
            k0 = k1;
            k1 = k2;
            k2 = k3;
            k3 = 0;
            ++had;
        }
        if (__ballot(had == 4)) sort_out(w, had == 4);
    };
    // whether float32 decides that a (larger bits) comes before b
    auto tell = [&](uint32_t a, uint32_t b) {
        return p.bias ? apart(unordered(a), unordered(b)) : whole || a >> 6 != b >> 6;
    };
    bool close = false;                                    // two neighbours, or the border, that it does not
    uint32_t before = 0, w = token_max<LT>(k0);
    for (int j = 0; j < p.top_k; ++j) {
        take(w, j);
        before = w;
        w = token_max<LT>(k0);
        if (w != 0) close |= !tell(before, w);
    }

    int slot = l;                                          // where this lane's expert goes
    if (__ballot(close && !again)) {
        // The keys of the 16 first, one a lane, ranked in float64.  Whoever was not taken is below the 16th; so the
        // ranking holds if the 16th is apart from the last chosen.
        const uint32_t last = before;
        for (int j = p.top_k; j < 16; ++j) {
            take(w, j);
            before = w;
            w = token_max<LT>(k0);
        }
        if (close) again |= before != 0 && !tell(last, before);
        double k64 = -INFINITY, s64 = 0.0;
        if (mine >= 0) {
            const float xj = clean_logit(load_logit(row + mine));
            k64 = (double)xj;
            if (p.bias) {
                const double ex = exp(softmax ? (double)xj - (double)top : -(double)xj);
                s64 = softmax ? ex / (double)z : 1.0 / (1.0 + ex);
                k64 = s64 + (double)p.bias[mine];
            }
        }
        // The softmax's sum is float32's, off by less than 2^-18 of itself: which moves the difference of two keys
        // by no more than that part of the difference of their scores.
        const bool rough = p.bias && softmax;
        int rank = 0;
        bool open = false;
        for (int j = 0; j < 16; ++j) {
            const double other = __shfl(k64, (lane & ~(LT - 1)) + j, 64);
            const int e = __shfl(mine, (lane & ~(LT - 1)) + j, 64);
            if (other > k64 || (other == k64 && e >= 0 && e < mine)) ++rank;
            if (rough) {
                const double d = fabs(__shfl(s64, (lane & ~(LT - 1)) + j, 64) - s64);
                open |= mine >= 0 && e >= 0 && d > 0.0 && !(fabs(other - k64) > 0x1p-18 * d);
            }
        }
        if (close) {
            if (rough) again |= token_max<LT>(open ? 1u : 0u) != 0;
            slot = mine >= 0 ? rank : l;
            if (slot >= p.top_k) mine = -1;
        } else if (l >= p.top_k) {
            mine = -1;
        }
    }

    float s = 0.f;
    if (mine >= 0) {
        const float xj = clean_logit(load_logit(row + mine));
        const float ex = expf(softmax ? xj - top : -fabsf(xj));   // (exp(-x) overflows before the score is lost)
        s = softmax ? ex : (xj >= 0.f ? 1.f : ex) / (1.f + ex);
    }
    float weight = s;
    if (p.renormalize) {
        const float total = token_sum<LT>(s);
        again |= token_max<LT>(mine >= 0 ? 1u : 0u) != 0 && !(total > 1e-12f);   // its terms may have lost digits
        weight = total > 0.f ? s / total : 0.f;
    } else if (softmax) {
        weight = any ? s / z : 0.f;
    }
    if (live && !again && slot < p.top_k && (mine >= 0 || slot == l)) {
        p.experts[t * p.top_k + slot] = mine;
        p.weights[t * p.top_k + slot] = weight * p.scale;
    }
    uint64_t left = __ballot(live && again && l == 0);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");   // the groups' keys have been read
    __builtin_amdgcn_wave_barrier();
    while (left) {
        const int g = __builtin_ctzll(left);
        left &= left - 1;
        double* mine = room[threadIdx.x >> 6];
        route_exact<T, V>(p, t0 + g / LT, reinterpret_cast<float*>(mine + 64 * V), mine);
    }
}

// Stores that do not stay in the caches (65536 rows of 512 float32: 27 us against 33).
typedef float f32x4 __attribute__((ext_vector_type(4)));
__device__ __forceinline__ void store4(float* p, const float (&v)[4]) {
    __builtin_nontemporal_store(f32x4{v[0], v[1], v[2], v[3]}, reinterpret_cast<f32x4*>(p));
}
__device__ __forceinline__ void store4(uint16_t* p, const float (&v)[4]) {
    const uint2 w = make_uint2(dev::f32x2_to_bf16x2(v[0], v[1]), dev::f32x2_to_bf16x2(v[2], v[3]));
    __builtin_nontemporal_store(__builtin_bit_cast(uint64_t, w), reinterpret_cast<uint64_t*>(p));
}

__device__ __forceinline__ double token_sum16(double v) {
    v += dppd<XCHG_1>(v);
    v += dppd<XCHG_2>(v);
    v += dppd<XCHG_4>(v);
    return v + dppd<XCHG_8>(v);
}

// The exponentials of a row: by the instruction where 16 lanes have all of it (what is below 2^-126 is lost).
template <int LT>
__device__ __forceinline__ float row_exp(float v) { return LT == 16 ? __expf(v) : expf(v); }

// The sum of v over the slots that have this lane's expert, in their order, and whether this is the first of them.
template <int LT, class S>
__device__ __forceinline__ S of_expert(int e, float v, int top_k, bool& first) {
    const int lane = threadIdx.x & 63, l = lane & (LT - 1);
    S all = 0;
    first = true;
    for (int j = 0; j < top_k; ++j) {
        const int ej = __shfl(e, (lane & ~(LT - 1)) + j, 64);
        const float vj = __shfl(v, (lane & ~(LT - 1)) + j, 64);
        if (ej == e) {
            all += (S)vj;
            first &= j >= l;
        }
    }
    return all;
}

// The plain softmax's gradient from its row's exponentials: dx_e = s_e (sum of e's g - sum_i g_i s_i) of a chosen expert, and
// what the others' exponentials are multiplied by, -(sum_i g_i s_i) / z.
// Near s = 1 that difference is g (1 - s), all of whose digits come from the sum z without the largest term.  So z is
// summed in float64, with the chosen experts' terms (float32 in z as it comes) in float64 as in the numerators; what is left of
// float32 is the exponentials of the others, good to some 2^-18 of themselves.
struct ChosenSoftmax {
    float dx;
    float other;
};
template <int LT, class SUM>
__device__ __forceinline__ ChosenSoftmax chosen_softmax(int e, float xj, float top, float gw, double scale, double z, int top_k, SUM sum) {
    bool first;
    const double all = of_expert<LT, double>(e, gw, top_k, first) * scale;
    const double ex = e >= 0 ? exp((double)xj - (double)top) : 0.0;
    z += sum(e >= 0 && first ? ex - (double)row_exp<LT>(xj - top) : 0.0);
    const double inv = z > 0.0 ? 1.0 / z : 0.0, s = ex * inv;
    const double mean = sum((double)gw * scale * s);       // (scaled here: float32's rounding would be a part of the difference)
    return {e >= 0 ? (float)(s * (all - mean)) : 0.f, (float)(-mean * inv)};
}

// Backward for up to 16 slots: 16 lanes a token as in route_kernel, lane j also slot j.  Renormalised weights and sigmoids
// need the chosen logits only; the plain softmax reads the row.  65537 x 512 float32: renormalised 27 us (5.0 TB/s written,
// bound by memory), by plain softmax 47 us (5.7 TB/s; the vector instructions are as near their limit).
template <class T, int C>
__global__ __launch_bounds__(64 * ROUTE_WAVES) void route_backward_kernel(RouteBackwardArgs p, int vec) {
    const int lane = threadIdx.x & 63, l = lane & 15;
    const int64_t t0 = ((int64_t)blockIdx.x * ROUTE_WAVES + (threadIdx.x >> 6)) * 4;
    if (t0 >= p.tokens) return;
    const bool live = t0 + (lane >> 4) < p.tokens;
    const int64_t t = live ? t0 + (lane >> 4) : t0;
    const T* row = static_cast<const T*>(p.logits) + t * p.ld;
    T* grad = static_cast<T*>(p.grad_logits) + t * p.ld_grad;
    int e = -1;
    float xj = -INFINITY, gw = 0.f;
    if (l < p.top_k) {
        e = p.experts[t * p.top_k + l];
        if (e < 0 || e >= p.n_experts) e = -1;
        if (e >= 0) xj = clean_logit(load_logit(row + e));
        if (!(xj > -INFINITY)) e = -1;
        if (e >= 0) gw = p.grad_weights[t * p.top_k + l];
    }
    const double g = (double)gw * (double)p.scale;         // (exact: where gradients are nearly alike, their differences count)
    float out[C][4];
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
        for (int v = 0; v < 4; ++v) out[c][v] = 0.f;
    float dx;                                              // what slot l's expert gets from it
    if (p.score == MUON_SCORE_SIGMOID) {
        const float high = token_maxf<16>(xj);
        const bool tiny = p.renormalize && high < TINY_SIGMOID;
        const double ex = exp(tiny ? (double)xj - (double)high : -fabs((double)xj));   // s and 1 - s without cancellation
        const double big = tiny ? 1.0 : 1.0 / (1.0 + ex), small = ex * big;
        const double s = e < 0 ? 0.0 : xj >= 0.f ? big : small, rest = xj >= 0.f ? small : big;
        if (p.renormalize) {
            const double total = token_sum16(s);
            const double w = total > 0.0 ? s / total : 0.0;
            const double mean = token_sum16(g * w);
            dx = e >= 0 ? (float)(w * rest * (g - mean)) : 0.f;
        } else {
            dx = e >= 0 ? (float)(g * s * rest) : 0.f;
        }
    } else if (p.renormalize) {
        const float top = token_maxf<16>(xj);
        const double ex = e >= 0 ? exp((double)xj - (double)top) : 0.0;
        const double total = token_sum16(ex);
        const double w = total > 0.0 ? ex / total : 0.0;
        const double mean = token_sum16(g * w);
        dx = e >= 0 ? (float)(w * (g - mean)) : 0.f;
    } else {
        float top = -INFINITY;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int ei = 64 * c + 4 * l;
            if (vec) {
                if (ei < p.n_experts) load4(row + ei, out[c]);
                else out[c][0] = out[c][1] = out[c][2] = out[c][3] = -INFINITY;
            } else {
#pragma unroll
                for (int v = 0; v < 4; ++v) out[c][v] = ei + v < p.n_experts ? load_logit(row + ei + v) : -INFINITY;
            }
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                out[c][v] = clean_logit(out[c][v]);
                top = fmaxf(top, out[c][v]);
            }
        }
        top = token_maxf<16>(top);
        double z = 0.0;
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                out[c][v] = out[c][v] > -INFINITY ? row_exp<16>(out[c][v] - top) : 0.f;
                z += (double)out[c][v];
            }
        z = token_sum16(z);
        const ChosenSoftmax r = chosen_softmax<16>(e, xj, top, gw, (double)p.scale, z, p.top_k, [](double v) { return token_sum16(v); });
        dx = r.dx;
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int v = 0; v < 4; ++v) out[c][v] *= r.other;
    }
    // from here on dx is all that the slot's expert gets
    bool first;
    if (p.score == MUON_SCORE_SIGMOID || p.renormalize) dx = of_expert<16, float>(e, dx, p.top_k, first);
    for (int j = 0; j < p.top_k; ++j) {
        const int place = __shfl(e, (lane & 48) + j, 64) - 4 * l;
        const float dj = __shfl(dx, (lane & 48) + j, 64);
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int v = 0; v < 4; ++v)
                out[c][v] = place == 64 * c + v ? dj : out[c][v];
    }
    if (!live) return;
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int ei = 64 * c + 4 * l;
        if (vec) {
            if (ei < p.n_experts) store4(grad + ei, out[c]);
        } else {
#pragma unroll
            for (int v = 0; v < 4; ++v)
                if (ei + v < p.n_experts) store_logit(grad + ei + v, out[c][v]);
        }
    }
}

// Backward for any number of slots: a wave a token.
template <class T, int V>
__global__ __launch_bounds__(64 * ROUTE_WAVES) void route_backward_wave_kernel(RouteBackwardArgs p) {
    const int lane = threadIdx.x & 63;
    const int64_t t = (int64_t)blockIdx.x * ROUTE_WAVES + (threadIdx.x >> 6);
    if (t >= p.tokens) return;
    const T* row = static_cast<const T*>(p.logits) + t * p.ld;
    T* grad = static_cast<T*>(p.grad_logits) + t * p.ld_grad;
    // lane j: slot j's expert, logit and gradient
    int e = -1;
    float xj = -INFINITY, gw = 0.f;
    if (lane < p.top_k) {
        e = p.experts[t * p.top_k + lane];
        if (e < 0 || e >= p.n_experts) e = -1;
        if (e >= 0) xj = clean_logit(load_logit(row + e));
        if (!(xj > -INFINITY)) e = -1;
        if (e >= 0) gw = p.grad_weights[t * p.top_k + lane];
    }
    const double g = (double)gw * (double)p.scale;         // (exact: where gradients are nearly alike, their differences count)
    float out[V];
#pragma unroll
    for (int i = 0; i < V; ++i) out[i] = 0.f;
    float dx = 0.f;                                        // lane j: what slot j's expert gets from it
    if (p.score == MUON_SCORE_SIGMOID) {
        const float high = wave_max(xj);
        const bool tiny = p.renormalize && high < TINY_SIGMOID;
        const double s = e < 0 ? 0.0 : tiny ? exp((double)xj - (double)high) : sigmoid64((double)xj);
        const double rest = e >= 0 ? 1.0 / (1.0 + exp((double)xj)) : 0.0;   // 1 - s
        if (p.renormalize) {
            const double total = dev::wave_sum(s);
            const double w = total > 0.0 ? s / total : 0.0;
            const double mean = dev::wave_sum(g * w);
            dx = e >= 0 ? (float)(w * rest * (g - mean)) : 0.f;
        } else {
            dx = (float)(g * s * rest);
        }
    } else if (p.renormalize) {
        const float top = wave_max(xj);
        const double ex = e >= 0 ? exp((double)xj - (double)top) : 0.0;
        const double total = dev::wave_sum(ex);
        const double w = total > 0.0 ? ex / total : 0.0;
        const double mean = dev::wave_sum(g * w);
        dx = e >= 0 ? (float)(w * (g - mean)) : 0.f;
    } else {
        float x[V], top = -INFINITY;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int ei = lane + 64 * i;
            x[i] = ei < p.n_experts ? clean_logit(load_logit(row + ei)) : -INFINITY;
            top = fmaxf(top, x[i]);
        }
        top = wave_max(top);
        double z = 0.0;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            x[i] = x[i] > -INFINITY ? row_exp<64>(x[i] - top) : 0.f;
            z += (double)x[i];
        }
        z = dev::wave_sum(z);
        const ChosenSoftmax r = chosen_softmax<64>(e, xj, top, gw, (double)p.scale, z, p.top_k, [](double v) { return dev::wave_sum(v); });
        dx = r.dx;
#pragma unroll
        for (int i = 0; i < V; ++i) out[i] = x[i] * r.other;
    }
    bool first;
    if (p.score == MUON_SCORE_SIGMOID || p.renormalize) dx = of_expert<64, float>(e, dx, p.top_k, first);   // all that the slot's expert gets
    for (int j = 0; j < p.top_k; ++j) {
        const int ej = __shfl(e, j, 64);
        const float dj = __shfl(dx, j, 64);
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (ej == lane + 64 * i) out[i] = dj;
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
// by matching the bits of the expert across the wave with ballots.  458759 choices of 512 experts: counts 3.2 us, prefix
// 4.6, placement 10.4 (4-byte stores to all segments; the bytes alone would take 1.2); 112 in one workgroup: 3.8 us.

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

// A workgroup's choices from lo on: wave w has 64 per consecutive ones (per <= PER), lane l every 64th of them.
template <int PER>
struct Run {
    int64_t first;             // the lane's first choice
    int per;
    int e[PER];                // experts, -1 for none
    __device__ __forceinline__ Run(const GroupRowsArgs& p, int64_t lo, int per_) : per(per_) {
        first = lo + (int64_t)(threadIdx.x >> 6) * 64 * per + (threadIdx.x & 63);
#pragma unroll
        for (int k = 0; k < PER; ++k) e[k] = load_choice(p, first + 64 * k, k < per ? p.n : 0);
    }
    // hist[w][e]: choices of expert e in wave w's run.
    __device__ __forceinline__ void count(int n_experts, int* hist) const {
        for (int i = threadIdx.x; i < GROUP_WAVES * n_experts; i += GROUP_THREADS) hist[i] = 0;
        __syncthreads();
        int* mine = hist + (threadIdx.x >> 6) * n_experts;
#pragma unroll
        for (int k = 0; k < PER; ++k)
            if (e[k] >= 0) atomicAdd(&mine[e[k]], 1);      // a count: the order does not matter
        __syncthreads();
    }
    // cursor[w][e] is where wave w's first choice of expert e goes.
    __device__ __forceinline__ void place(const GroupRowsArgs& p, int* cursor) const {
        const int lane = threadIdx.x & 63;
        int* mine = cursor + (threadIdx.x >> 6) * p.n_experts;
#pragma unroll
        for (int k = 0; k < PER; ++k) {
            const int64_t i = first + 64 * k;
            if (k >= per || i - lane >= p.n) break;
            const uint64_t same = match_lanes(e[k]);
            int at = -1;
            if (e[k] >= 0) at = mine[e[k]] + __popcll(same & ((1ull << lane) - 1));
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");   // the reads come before the write
            __builtin_amdgcn_wave_barrier();
            if (e[k] >= 0 && (same >> lane) == 1) mine[e[k]] = at + 1;   // the last lane of the expert
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
            if (i < p.n) p.position[i] = at;
            if (e[k] >= 0) p.rows[at] = (int32_t)i;
        }
    }
};
constexpr int SINGLE_PER = GROUP_SINGLE_MAX / GROUP_THREADS, CHUNK_PER = GROUP_CHUNK / GROUP_THREADS;

// All of a small call in one workgroup.
__global__ __launch_bounds__(GROUP_THREADS) void group_single_kernel(GroupRowsArgs p) {
    extern __shared__ int lds[];
    __shared__ int wave_tot[GROUP_WAVES];
    const Run<SINGLE_PER> run(p, 0, (int)((p.n + GROUP_THREADS - 1) / GROUP_THREADS));
    run.count(p.n_experts, lds);
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
    run.place(p, lds);
}

__global__ __launch_bounds__(GROUP_THREADS) void group_count_kernel(GroupRowsArgs p) {
    extern __shared__ int lds[];
    const Run<CHUNK_PER> run(p, blockIdx.x * (int64_t)GROUP_CHUNK, CHUNK_PER);
    run.count(p.n_experts, lds);
    for (int e = threadIdx.x; e < p.n_experts; e += GROUP_THREADS) {
        int c = 0;
        for (int w = 0; w < GROUP_WAVES; ++w) c += lds[w * p.n_experts + e];
        p.partial[blockIdx.x * (int64_t)p.n_experts + e] = c;
    }
}

// partial[chunk][e] becomes the number of the expert's choices in earlier chunks, and counts[e] all of them: a wave
// for each expert, a lane for each of 64 chunks at a time, the loads of 256 chunks together.
constexpr int PREFIX_AHEAD = 4;
__global__ __launch_bounds__(256) void group_prefix_kernel(GroupRowsArgs p) {
    const int lane = threadIdx.x & 63, e = blockIdx.x * 4 + (threadIdx.x >> 6);
    if (e >= p.n_experts) return;
    int before = 0;
    for (int64_t b0 = 0; b0 < p.chunks; b0 += 64 * PREFIX_AHEAD) {
        int h[PREFIX_AHEAD];
#pragma unroll
        for (int k = 0; k < PREFIX_AHEAD; ++k) {
            const int64_t b = b0 + 64 * k + lane;
            h[k] = b < p.chunks ? p.partial[b * p.n_experts + e] : 0;
        }
#pragma unroll
        for (int k = 0; k < PREFIX_AHEAD; ++k) {
            const int64_t b = b0 + 64 * k + lane;
            int inc = h[k];
#pragma unroll
            for (int off = 1; off < 64; off <<= 1) {
                const int o = __shfl_up(inc, off, 64);
                if (lane >= off) inc += o;
            }
            if (b < p.chunks) p.partial[b * p.n_experts + e] = before + inc - h[k];
            before += __shfl(inc, 63, 64);
        }
    }
    if (lane == 0) p.counts[e] = before;
}

// Every workgroup works the offsets out from the counts; the first writes them down.
__global__ __launch_bounds__(GROUP_THREADS) void group_place_kernel(GroupRowsArgs p) {
    extern __shared__ int lds[];
    __shared__ int wave_tot[GROUP_WAVES];
    const Run<CHUNK_PER> run(p, blockIdx.x * (int64_t)GROUP_CHUNK, CHUNK_PER);
    const int e = threadIdx.x;
    const int c = e < p.n_experts ? p.counts[e] : 0;
    const int earlier = e < p.n_experts ? p.partial[blockIdx.x * (int64_t)p.n_experts + e] : 0;
    run.count(p.n_experts, lds);
    const int padded = (c + p.align - 1) / p.align * p.align;
    int total;
    const int start = block_prefix(padded, wave_tot, total);
    if (e < p.n_experts) {
        int at = start + earlier;
        for (int w = 0; w < GROUP_WAVES; ++w) {
            const int h = lds[w * p.n_experts + e];
            lds[w * p.n_experts + e] = at;
            at += h;
        }
        if (blockIdx.x == 0) p.offsets[e] = start;
        // a segment's padding
        if (e % gridDim.x == blockIdx.x)
            for (int r = start + c; r < start + padded; ++r) p.rows[r] = -1;
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) p.offsets[p.n_experts] = total;
    __syncthreads();
    run.place(p, lds);
    // what lies behind the last segment
    const int64_t step = (int64_t)gridDim.x * GROUP_THREADS;
    for (int64_t r = total + blockIdx.x * (int64_t)GROUP_THREADS + threadIdx.x; r < p.capacity; r += step) p.rows[r] = -1;
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

// Variants, by what the sizes allow and what they measured (of 512 experts, times of whole calls back to back, which
// take 9.5 us at least):
//   * 16 lanes a token from 4096 tokens on (65536 tokens, 7 by softmax: 38 us, by sigmoid and bias 55; 64 lanes: 57 and
//     78), and for groups of up to 512 experts;
//   * 64 lanes below (2048 tokens by sigmoid and bias: 11.1 us against 14.2), where a wave's own time counts, and above
//     512 experts, whose values 16 lanes cannot hold;
//   * the float64 wave for what neither covers: more than 15 choices (65536 tokens, 20 choices: 284 us), groups of more
//     than 512 experts.
template <class T>
hipError_t route_by_width(const RouteArgs& a, hipStream_t s) {
    const bool few = a.top_k <= FAST_MAX_K, flat = a.n_groups == 1;
    const bool wide = few && flat && (a.tokens < WIDE_MAX_TOKENS || a.n_experts > 512);
    const bool narrow = few && !wide && a.n_experts <= 512;
    const int64_t per_block = ROUTE_WAVES * (narrow ? 4 : 1);
    const dim3 grid((unsigned)((a.tokens + per_block - 1) / per_block)), block(64 * ROUTE_WAVES);
    const int vec = a.ld % 4 == 0 && a.n_experts % 4 == 0;
    if (wide) {
        if (a.n_experts <= 256) hipLaunchKernelGGL((route_kernel<T, 64, 1, false>), grid, block, 0, s, a, vec);
        else if (a.n_experts <= 512) hipLaunchKernelGGL((route_kernel<T, 64, 2, false>), grid, block, 0, s, a, vec);
        else hipLaunchKernelGGL((route_kernel<T, 64, 4, false>), grid, block, 0, s, a, vec);
    } else if (narrow && flat) {
        if (a.n_experts <= 128) hipLaunchKernelGGL((route_kernel<T, 16, 2, false>), grid, block, 0, s, a, vec);
        else hipLaunchKernelGGL((route_kernel<T, 16, 8, false>), grid, block, 0, s, a, vec);
    } else if (narrow) {
        if (a.n_experts <= 128) hipLaunchKernelGGL((route_kernel<T, 16, 2, true>), grid, block, 0, s, a, vec);
        else hipLaunchKernelGGL((route_kernel<T, 16, 8, true>), grid, block, 0, s, a, vec);
    } else {
        if (a.n_experts <= 128) hipLaunchKernelGGL((route_exact_kernel<T, 2>), grid, block, 0, s, a);
        else if (a.n_experts <= 512) hipLaunchKernelGGL((route_exact_kernel<T, 8>), grid, block, 0, s, a);
        else hipLaunchKernelGGL((route_exact_kernel<T, 16>), grid, block, 0, s, a);
    }
    return hipGetLastError();
}

template <class T>
hipError_t backward_by_width(const RouteBackwardArgs& a, hipStream_t s) {
    const bool fast = a.top_k <= 16;
    const int64_t per_block = ROUTE_WAVES * (fast ? 4 : 1);
    const dim3 grid((unsigned)((a.tokens + per_block - 1) / per_block)), block(64 * ROUTE_WAVES);
    const int vec = a.ld % 4 == 0 && a.ld_grad % 4 == 0 && a.n_experts % 4 == 0;
    if (fast) {
        if (a.n_experts <= 128) hipLaunchKernelGGL((route_backward_kernel<T, 2>), grid, block, 0, s, a, vec);
        else if (a.n_experts <= 512) hipLaunchKernelGGL((route_backward_kernel<T, 8>), grid, block, 0, s, a, vec);
        else hipLaunchKernelGGL((route_backward_kernel<T, 16>), grid, block, 0, s, a, vec);
    } else {
        if (a.n_experts <= 128) hipLaunchKernelGGL((route_backward_wave_kernel<T, 2>), grid, block, 0, s, a);
        else if (a.n_experts <= 512) hipLaunchKernelGGL((route_backward_wave_kernel<T, 8>), grid, block, 0, s, a);
        else hipLaunchKernelGGL((route_backward_wave_kernel<T, 16>), grid, block, 0, s, a);
    }
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
    hipLaunchKernelGGL(group_prefix_kernel, dim3((unsigned)((a.n_experts + 3) / 4)), dim3(256), 0, s, a);
    hipLaunchKernelGGL(group_place_kernel, grid, block, lds, s, a);
    return hipGetLastError();
}

hipError_t launch_balance(const float* bias, const int32_t* counts, int32_t n, float rate, float* out, hipStream_t s) {
    hipLaunchKernelGGL(balance_kernel, dim3(1), dim3(GROUP_THREADS), 0, s, bias, counts, n, rate, out);
    return hipGetLastError();
}

}  // namespace muon
