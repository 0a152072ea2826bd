// layer_gate.hpp -- gfx950 kernels of the gate (top-k of the router's logits with
// per-expert counts, balance and z losses), its gradient, and combine's
// gradient.
//
// Sixteen lanes own one token, four tokens to a wave: lane j of the group
// holds elements 64 c + 4 j ... +3 of the row (16-byte loads), and every
// reduction over a row is four DPP steps inside the 16 lanes, which cost no
// LDS and serve four tokens at once.  The steps pair lanes symmetrically, so
// that all 16 lanes end with the same bits.
#pragma once

#include <hip/hip_runtime.h>
#include <limits.h>
#include <stdint.h>

namespace epdc_layer {

constexpr int kGateThreads = 512;
constexpr int kGateTokens = kGateThreads / 16;  // of a block's pass
constexpr int kGateMaxBlocks = 256;
constexpr int kMaxTopk = 16;

enum { kScoreSoftmax = 0, kScoreSigmoid = 1 };

struct GateArgs {
    int32_t tokens, experts, topk;
    int32_t score, renorm, bf16;
    float scale;
    const void *logits;
    const float *bias;
    const uint8_t *mask;
    float *weights;
    int32_t *indices;
    // balance: counts [E+1], losses [2] and scratch (ticket, then one row of
    // partials per block: E + 1 counts, E probability sums, the z sum)
    int32_t *counts;
    float *losses;
    uint32_t *ticket;
    float *partial;
    // backward
    const int32_t *in_indices;
    const float *grad_weights;
    const int32_t *in_counts;
    const float *grad_losses;
    void *grad_logits;
};

__host__ __device__ inline int gate_partial_words(int experts) { return 2 * experts + 2; }

template <int kCtrl>
__device__ inline float dpp_f(float v)
{
    return __int_as_float(
        __builtin_amdgcn_update_dpp(0, __float_as_int(v), kCtrl, 0xf, 0xf, false));
}
template <int kCtrl>
__device__ inline int dpp_i(int v)
{
    return __builtin_amdgcn_update_dpp(0, v, kCtrl, 0xf, 0xf, false);
}
template <int kCtrl>
__device__ inline double dpp_d(double v)
{
    const uint64_t u = (uint64_t)__double_as_longlong(v);
    const uint32_t lo = (uint32_t)dpp_i<kCtrl>((int)(uint32_t)u);
    const uint32_t hi = (uint32_t)dpp_i<kCtrl>((int)(uint32_t)(u >> 32));
    return __longlong_as_double((long long)(((uint64_t)hi << 32) | lo));
}

// lane ^ 1, lane ^ 2, then the mirrors inside 8 and inside 16 lanes
constexpr int kXor1 = 0xB1, kXor2 = 0x4E, kMirror8 = 0x141, kMirror16 = 0x140;

#define EPDC_GROUP_REDUCE(name, T, dpp, expr)      \
    __device__ inline T name(T a)                  \
    {                                              \
        T b = dpp<kXor1>(a);                       \
        a = expr;                                  \
        b = dpp<kXor2>(a);                         \
        a = expr;                                  \
        b = dpp<kMirror8>(a);                      \
        a = expr;                                  \
        b = dpp<kMirror16>(a);                     \
        return expr;                               \
    }
EPDC_GROUP_REDUCE(group_max, float, dpp_f, (a > b ? a : b))
EPDC_GROUP_REDUCE(group_sum, float, dpp_f, (a + b))
EPDC_GROUP_REDUCE(group_min, int, dpp_i, (a < b ? a : b))
EPDC_GROUP_REDUCE(group_or, int, dpp_i, (a | b))
EPDC_GROUP_REDUCE(group_max, double, dpp_d, (a > b ? a : b))
EPDC_GROUP_REDUCE(group_sum, double, dpp_d, (a + b))
#undef EPDC_GROUP_REDUCE

template <typename T>
__device__ inline T lowest();
template <>
__device__ inline float lowest<float>() { return -__builtin_inff(); }
template <>
__device__ inline double lowest<double>() { return -__builtin_inf(); }

// Element of this lane's slot v: 64 (v / 4) + 4 j + v % 4.
__device__ inline int slot_expert(int v, int j) { return (v >> 2) * 64 + j * 4 + (v & 3); }

template <int kV>
__device__ inline void load_logits(const GateArgs &a, int64_t token, int j, float (&l)[kV])
{
    const float none = lowest<float>();
    const int E = a.experts;
    const bool wide = (E & 3) == 0;  // rows of whole 4-element vectors stay aligned
    const size_t row = (size_t)token * E;
#pragma unroll
    for (int c = 0; c < kV / 4; ++c) {
        const int e = c * 64 + j * 4;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            l[c * 4 + i] = none;
        if (a.bf16) {
            const uint16_t *p = static_cast<const uint16_t *>(a.logits) + row + e;
            if (wide && e < E) {
                const uint2 w = *reinterpret_cast<const uint2 *>(p);
                l[c * 4 + 0] = __uint_as_float(w.x << 16);
                l[c * 4 + 1] = __uint_as_float(w.x & 0xFFFF0000u);
                l[c * 4 + 2] = __uint_as_float(w.y << 16);
                l[c * 4 + 3] = __uint_as_float(w.y & 0xFFFF0000u);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (e + i < E)
                        l[c * 4 + i] = __uint_as_float((uint32_t)p[i] << 16);
            }
        } else {
            const float *p = static_cast<const float *>(a.logits) + row + e;
            if (wide && e < E) {
                const float4 w = *reinterpret_cast<const float4 *>(p);
                l[c * 4 + 0] = w.x;
                l[c * 4 + 1] = w.y;
                l[c * 4 + 2] = w.z;
                l[c * 4 + 3] = w.w;
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (e + i < E)
                        l[c * 4 + i] = p[i];
            }
        }
    }
}

// What a token's logits make of it.
enum { kTokenOut = 0, kTokenIn = 1, kTokenBad = 2 };

template <int kV>
__device__ inline int classify(const GateArgs &a, int64_t token, const float (&l)[kV], float &m)
{
    float top = lowest<float>();
    int bad = 0;
#pragma unroll
    for (int v = 0; v < kV; ++v) {
        bad |= !(l[v] < __builtin_inff());  // NaN or +inf
        top = l[v] > top ? l[v] : top;
    }
    m = group_max(top);
    bad = group_or(bad);
    if (a.mask && a.mask[token] == 0)
        return kTokenOut;
    if (bad)
        return kTokenBad;
    return m == lowest<float>() ? kTokenOut : kTokenIn;
}

// The largest key of the group and its expert (lowest index among equals);
// expert -1 when nothing is left.
template <int kV, typename T>
__device__ inline void group_top(const T (&key)[kV], int j, T &best, int &expert)
{
    T top = lowest<T>();
    int at = INT_MAX;
#pragma unroll
    for (int v = 0; v < kV; ++v)
        if (key[v] > top) {  // slots ascend in expert order
            top = key[v];
            at = slot_expert(v, j);
        }
    best = group_max(top);
    expert = group_min(top == best ? at : INT_MAX);
    if (expert == INT_MAX)
        expert = -1;
}

template <int kV, typename T>
__device__ inline void drop(T (&key)[kV], int j, int expert)
{
#pragma unroll
    for (int v = 0; v < kV; ++v)
        if (slot_expert(v, j) == expert)
            key[v] = lowest<T>();
}

// log of a chosen score up to a constant of the row, without underflow:
// softmax: the logit; sigmoid: log sigma(l) = min(l, 0) - log(1 + exp(-|l|))
__device__ inline float log_score(int score, float l)
{
    if (score == kScoreSoftmax)
        return l;
    return fminf(l, 0.0f) - log1pf(expf(-fabsf(l)));
}

__device__ inline float sigmoid(float l) { return 1.0f / (1.0f + expf(-l)); }

// Keys with a bias, s + b, are rounded sums of rounded scores.  In fp32 s is
// off by a few ulp of at most 1 and the sum by half an ulp of the key, so two
// neighbours of the order further apart than this are certainly in order.
__device__ inline float key_slack(float k) { return 1.5e-6f + 2.5e-7f * fabsf(k); }

__device__ inline void store_agent(float *p, float v)
{
    __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ inline float load_agent(const float *p)
{
    return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// Reads the logits once; a token's choice is kept by its group's lanes (lane k
// has choice k).  With a balance, each lane sums its experts' probabilities
// over its tokens; waves, then blocks, are added in a fixed order, the blocks
// by the last one to finish.
template <int kV, bool kBalance>
__global__ __launch_bounds__(kGateThreads) void k_gate(const GateArgs a)
{
    constexpr int kWaves = kGateThreads / 64;
    extern __shared__ __align__(16) uint8_t dyn[];
    int *cnt = reinterpret_cast<int *>(dyn);                       // [E + 1]
    float *sum = reinterpret_cast<float *>(dyn) + a.experts + 1;   // [waves][E]
    float *zsum = sum + kWaves * a.experts;                        // [kGateTokens]
    __shared__ int last;

    const int tid = threadIdx.x, lane = tid & 63, wave = tid / 64, j = tid & 15;
    const int E = a.experts, K = a.topk;
    if (kBalance) {
        for (int e = tid; e <= E; e += kGateThreads)
            cnt[e] = 0;
        __syncthreads();
    }
    float bias[kV], prob[kV], z = 0.0f;
#pragma unroll
    for (int v = 0; v < kV; ++v) {
        const int e = slot_expert(v, j);
        bias[v] = a.bias && e < E ? a.bias[e] : 0.0f;
        prob[v] = 0.0f;
    }
    const bool softmax = a.score == kScoreSoftmax;
    const bool scores = kBalance || a.bias != nullptr || (softmax && !a.renorm);

    for (int64_t t0 = (int64_t)blockIdx.x * kGateTokens; t0 < a.tokens;
         t0 += (int64_t)gridDim.x * kGateTokens) {
        const int64_t t = t0 + tid / 16;
        if (t >= a.tokens)
            continue;
        float l[kV], s[kV], m;
        load_logits<kV>(a, t, j, l);
        const int kind = classify<kV>(a, t, l, m);
        int chosen = -1;      // lane k: choice k
        float total = 1.0f, lse = 0.0f;
        if (kind == kTokenIn) {
            if (scores) {
                float part = 0.0f, esum = 0.0f;
#pragma unroll
                for (int v = 0; v < kV; ++v) {
                    const float x = expf(l[v] - m);
                    s[v] = softmax ? x : sigmoid(l[v]);
                    part += s[v];
                    esum += x;
                }
                total = group_sum(part);
                if (kBalance)
                    lse = m + logf(group_sum(esum));
                const float r = 1.0f / total;
#pragma unroll
                for (int v = 0; v < kV; ++v) {
                    if (kBalance)
                        prob[v] += s[v] * r;
                    if (softmax)
                        s[v] *= r;
                }
            }
            float key[kV];
#pragma unroll
            for (int v = 0; v < kV; ++v)
                key[v] = a.bias && l[v] > lowest<float>() ? s[v] + bias[v] : l[v];
            float before = __builtin_inff();
            bool close = false;
            for (int k = 0; k <= K; ++k) {  // with a bias one more, to see the border
                if (k == K && !a.bias)
                    break;
                float best;
                int e;
                group_top<kV>(key, j, best, e);
                if (a.bias && e >= 0)
                    close |= before - best <= key_slack(best);
                before = best;
                if (k < K && j == k)
                    chosen = e;
                drop<kV>(key, j, e);
            }
            if (close) {  // the same in 64 bits
                double key64[kV], part = 0.0, sum64 = 1.0;
#pragma unroll
                for (int v = 0; v < kV; ++v) {
                    const double x = (double)l[v];
                    key64[v] = softmax ? exp(x - (double)m) : 1.0 / (1.0 + exp(-x));
                    part += key64[v];
                }
                if (softmax)
                    sum64 = group_sum(part);
#pragma unroll
                for (int v = 0; v < kV; ++v)
                    key64[v] = l[v] > lowest<float>() ? key64[v] / sum64 + (double)bias[v]
                                                      : lowest<double>();
                for (int k = 0; k < K; ++k) {
                    double best;
                    int e;
                    group_top<kV>(key64, j, best, e);
                    if (j == k)
                        chosen = e;
                    drop<kV>(key64, j, e);
                }
            }
        }
        const bool have = chosen >= 0;
        float x = lowest<float>(), w = 0.0f;
        if (have) {
            const size_t at = (size_t)t * E + chosen;
            x = a.bf16 ? __uint_as_float((uint32_t)static_cast<const uint16_t *>(a.logits)[at] << 16)
                       : static_cast<const float *>(a.logits)[at];
        }
        if (a.renorm) {
            const float ls = have ? log_score(a.score, x) : lowest<float>();
            const float top = group_max(ls);
            const float p = have ? expf(ls - top) : 0.0f;
            w = a.scale * (p / group_sum(p));
        } else if (have) {
            w = a.scale * (softmax ? expf(x - m) / total : sigmoid(x));
        }
        if (!have)
            w = kind == kTokenBad ? __builtin_nanf("") : 0.0f;
        if (j < K) {
            a.weights[t * K + j] = w;
            a.indices[t * K + j] = chosen;
        }
        if (kBalance) {
            if (have && j < K)
                atomicAdd(&cnt[chosen], 1);
            if (kind != kTokenOut && j == 0) {
                atomicAdd(&cnt[E], 1);
                z += kind == kTokenBad ? __builtin_nanf("") : lse * lse;
            }
            if (kind == kTokenBad)
                prob[0] = __builtin_nanf("");
        }
    }
    if (!kBalance)
        return;

    // the wave's four groups, then the block's waves
#pragma unroll
    for (int v = 0; v < kV; ++v) {
        float p = prob[v];
        p += __shfl_xor(p, 16, 64);
        p += __shfl_xor(p, 32, 64);
        const int e = slot_expert(v, j);
        if (lane < 16 && e < E)
            sum[wave * E + e] = p;
    }
    if (j == 0)
        zsum[tid / 16] = z;
    __syncthreads();
    const int words = gate_partial_words(E);
    float *mine = a.partial + (size_t)blockIdx.x * words;
    for (int e = tid; e < E; e += kGateThreads) {
        float p = 0.0f;
#pragma unroll
        for (int w = 0; w < kWaves; ++w)
            p += sum[w * E + e];
        store_agent(mine + e, __int_as_float(cnt[e]));
        store_agent(mine + E + 1 + e, p);
    }
    if (tid == 0) {
        float zz = 0.0f;
        for (int i = 0; i < kGateTokens; ++i)
            zz += zsum[i];
        store_agent(mine + E, __int_as_float(cnt[E]));
        store_agent(mine + 2 * E + 1, zz);
    }
    // every store of the block is at the device's point of coherence before
    // the ticket is taken
    __builtin_amdgcn_s_waitcnt(0);
    __syncthreads();
    if (tid == 0)
        last = __hip_atomic_fetch_add(a.ticket, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) ==
               gridDim.x - 1;
    __syncthreads();
    if (!last)
        return;
    const int nb = gridDim.x;
    for (int i = tid; i <= E; i += kGateThreads) {  // counts, and the token count
        int c = 0;
#pragma unroll 16
        for (int b = 0; b < nb; ++b)
            c += __float_as_int(load_agent(a.partial + (size_t)b * words + i));
        cnt[i] = c;
        a.counts[i] = c;
    }
    for (int i = tid; i <= E; i += kGateThreads) {  // probabilities, and the z sum
        float p = 0.0f;
#pragma unroll 16
        for (int b = 0; b < nb; ++b)
            p += load_agent(a.partial + (size_t)b * words + E + 1 + i);
        sum[i] = p;
    }
    __syncthreads();
    if (wave == 0) {
        const float n = (float)(cnt[E] > 1 ? cnt[E] : 1);
        float d = 0.0f;
        for (int e = lane; e < E; e += 64)
            d += (float)cnt[e] * sum[e];
#pragma unroll
        for (int x = 1; x < 64; x <<= 1)
            d += __shfl_xor(d, x, 64);
        if (lane == 0) {
            a.losses[0] = (float)E * (d / n / (n * (float)K));
            a.losses[1] = sum[E] / n;
            *a.ticket = 0;  // ready for the next call, which the stream orders after this one
        }
    }
}

// One pass over the logits: with p the scores' softmax (sigmoid: s / sum s),
//   d/dl_j of scale * r(chosen)  and of  E/n sum_e f_e p_e  and of  lse^2 / n.
template <int kV>
__global__ __launch_bounds__(kGateThreads) void k_gate_backward(const GateArgs a)
{
    extern __shared__ __align__(16) float f[];  // [E]: an expert's share of the choices
    const int tid = threadIdx.x, j = tid & 15;
    const int E = a.experts, K = a.topk;
    const bool softmax = a.score == kScoreSoftmax, balance = a.in_counts != nullptr;
    float gb = 0.0f, gz = 0.0f;
    float share[kV];
#pragma unroll
    for (int v = 0; v < kV; ++v)
        share[v] = 0.0f;
    if (balance) {
        const int n = a.in_counts[E] > 1 ? a.in_counts[E] : 1;
        for (int e = tid; e < E; e += kGateThreads)
            f[e] = (float)a.in_counts[e] / ((float)n * (float)K);
        gb = a.grad_losses[0] * (float)E / (float)n;
        gz = a.grad_losses[1] * 2.0f / (float)n;
        __syncthreads();
#pragma unroll
        for (int v = 0; v < kV; ++v) {
            const int e = slot_expert(v, j);
            share[v] = e < E ? f[e] : 0.0f;
        }
    }
    for (int64_t t0 = (int64_t)blockIdx.x * kGateTokens; t0 < a.tokens;
         t0 += (int64_t)gridDim.x * kGateTokens) {
        const int64_t t = t0 + tid / 16;
        if (t >= a.tokens)
            continue;
        float l[kV], m;
        load_logits<kV>(a, t, j, l);
        const int kind = classify<kV>(a, t, l, m);
        float d[kV];
#pragma unroll
        for (int v = 0; v < kV; ++v)
            d[v] = kind == kTokenBad ? __builtin_nanf("") : 0.0f;
        if (kind == kTokenIn) {
            // the rows' softmax x / xs and sigmoids s / ss
            float x[kV], s[kV], xs = 0.0f, ss = 0.0f, fp = 0.0f;
#pragma unroll
            for (int v = 0; v < kV; ++v) {
                x[v] = expf(l[v] - m);
                xs += x[v];
                s[v] = softmax ? x[v] : sigmoid(l[v]);
                ss += s[v];
                fp += share[v] * s[v];
            }
            xs = group_sum(xs);
            ss = group_sum(ss);
            fp = group_sum(fp) / ss;
            // the chosen: lane k holds choice k, its gradient and its share r
            int e = -1;
            float g = 0.0f, le = lowest<float>();
            if (j < K && a.grad_weights) {
                e = a.in_indices[t * K + j];
                e = e >= 0 && e < E ? e : -1;
                if (e >= 0) {
                    g = a.grad_weights[t * K + j] * a.scale;
                    const size_t at = (size_t)t * E + e;
                    le = a.bf16 ? __uint_as_float(
                                      (uint32_t)static_cast<const uint16_t *>(a.logits)[at] << 16)
                                : static_cast<const float *>(a.logits)[at];
                }
            }
            float r = 0.0f, dc = 0.0f, all = 0.0f;  // all: taken from every p of a softmax
            if (a.renorm) {
                const float ls = e >= 0 ? log_score(a.score, le) : lowest<float>();
                const float top = group_max(ls);
                r = e >= 0 ? expf(ls - top) : 0.0f;
                const float rs = group_sum(r);
                r = rs > 0.0f ? r / rs : 0.0f;
                dc = r * (g - group_sum(g * r));
                if (!softmax)
                    dc *= e >= 0 ? 1.0f - sigmoid(le) : 0.0f;
            } else if (softmax) {
                r = e >= 0 ? expf(le - m) / xs : 0.0f;
                dc = g * r;
                all = group_sum(dc);
            } else {
                r = e >= 0 ? sigmoid(le) : 0.0f;
                dc = g * r * (1.0f - r);
            }
            const float lse = m + logf(xs), rx = 1.0f / xs, rs = 1.0f / ss;
#pragma unroll
            for (int v = 0; v < kV; ++v) {
                const float q = x[v] * rx;
                float b = gb * (s[v] * rs) * (share[v] - fp);
                if (!softmax)
                    b *= 1.0f - s[v];
                d[v] = b + (gz * lse - all) * q;
            }
            for (int k = 0; k < K; ++k) {
                const int ek = __shfl(e, k, 16);
                const float dk = __shfl(dc, k, 16);
#pragma unroll
                for (int v = 0; v < kV; ++v)
                    d[v] += slot_expert(v, j) == ek ? dk : 0.0f;
            }
#pragma unroll
            for (int v = 0; v < kV; ++v)
                if (l[v] == lowest<float>())
                    d[v] = 0.0f;
        }
        const size_t row = (size_t)t * E;
        const bool wide = (E & 3) == 0;
#pragma unroll
        for (int c = 0; c < kV / 4; ++c) {
            const int e = c * 64 + j * 4;
            if (a.bf16) {
                __bf16 *p = static_cast<__bf16 *>(a.grad_logits) + row + e;
                if (wide && e < E) {
                    *reinterpret_cast<bf16x4 *>(p) =
                        to_bf16(f32x4{d[c * 4], d[c * 4 + 1], d[c * 4 + 2], d[c * 4 + 3]});
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (e + i < E)
                            p[i] = (__bf16)d[c * 4 + i];
                }
            } else {
                float *p = static_cast<float *>(a.grad_logits) + row + e;
                if (wide && e < E) {
                    *reinterpret_cast<f32x4 *>(p) =
                        f32x4{d[c * 4], d[c * 4 + 1], d[c * 4 + 2], d[c * 4 + 3]};
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (e + i < E)
                            p[i] = d[c * 4 + i];
                }
            }
        }
    }
}

// ---------------------------------------------------------------------------
// Combine's gradient
// ---------------------------------------------------------------------------

struct CombineGradArgs {
    int32_t tokens, topk, row_vecs;  // 16-byte vectors of a row
    const int32_t *slot_of;
    const uint8_t *grad_output, *input;
    const float *weights;
    uint8_t *grad_input;
    float *grad_weights;
};

constexpr int kCombineGradThreads = 256;

// A block per token: a thread reads a vector of the token's gradient once and
// serves the K rows with it -- the row's vector for the dot product in, the
// scaled gradient out.  Bytes are the bound (one row read and one written per
// pair).
template <int kTopk>
__global__ __launch_bounds__(kCombineGradThreads) void k_combine_grad(const CombineGradArgs a)
{
    constexpr int kMax = kTopk ? kTopk : kMaxTopk, kWaves = kCombineGradThreads / 64;
    __shared__ float part[kWaves][kMax];
    const int K = kTopk ? kTopk : a.topk;
    const int64_t t = blockIdx.x;
    const int lane = threadIdx.x & 63, wave = threadIdx.x / 64;
    int slot[kMax];
    float w[kMax], dot[kMax];
#pragma unroll
    for (int k = 0; k < kMax; ++k) {
        slot[k] = -1;
        w[k] = 1.0f;
        dot[k] = 0.0f;
        if (k < K) {
            const int s = uniform(a.slot_of[t * K + k]);
            slot[k] = s >= 0 && s < (int64_t)a.tokens * K ? s : -1;
            if (a.weights && slot[k] >= 0)
                w[k] = a.weights[(size_t)slot[k] * K + k];
        }
    }
    const size_t row_bytes = (size_t)a.row_vecs * 16;
    for (int v = threadIdx.x; v < a.row_vecs; v += kCombineGradThreads) {
        const bf16x8 g = *reinterpret_cast<const bf16x8 *>(a.grad_output + t * row_bytes +
                                                           (size_t)v * 16);
        float gf[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            gf[i] = (float)g[i];
#pragma unroll
        for (int k = 0; k < kMax; ++k) {
            if (k >= K || slot[k] < 0)
                continue;
            const size_t at = (size_t)slot[k] * row_bytes + (size_t)v * 16;
            if (a.grad_weights) {
                const bf16x8 x = __builtin_nontemporal_load(
                    reinterpret_cast<const bf16x8 *>(a.input + at));
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    dot[k] += gf[i] * (float)x[i];
            }
            if (a.grad_input) {
                bf16x8 o;
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    o[i] = (__bf16)(w[k] * gf[i]);
                __builtin_nontemporal_store(o, reinterpret_cast<bf16x8 *>(a.grad_input + at));
            }
        }
    }
    if (!a.grad_weights)
        return;
#pragma unroll
    for (int k = 0; k < kMax; ++k) {
#pragma unroll
        for (int x = 1; x < 64; x <<= 1)
            dot[k] += __shfl_xor(dot[k], x, 64);
        if (lane == 0)
            part[wave][k] = dot[k];
    }
    __syncthreads();
    if ((int)threadIdx.x < K) {
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < kWaves; ++i)
            s += part[i][threadIdx.x];
        a.grad_weights[t * K + threadIdx.x] = s;
    }
}

}  // namespace epdc_layer
