// layer_gate.hpp -- gfx950 kernels of the gate (top-k of the router's logits with
// per-expert counts, balance and z losses), its gradient, and combine's
// gradient.
//
// A group of kLanes lanes owns one token: 16, four tokens to a wave, when there
// are tokens enough to fill the chip, else the whole wave.  Every reduction over
// a row is four DPP steps inside 16 lanes (and two row swaps for 64), which cost
// no LDS; the steps pair lanes symmetrically, so that all lanes of the group end
// with the same bits.
#pragma once

#include <hip/hip_runtime.h>
#include <limits.h>
#include <stdint.h>

namespace epdc_layer {

constexpr int kGateThreads = 512;
constexpr int kGateMaxBlocks = 512;  // two of 8 waves per CU
constexpr int kGateMaxFan = 32;

// Rows of partial sums one block adds; two levels of them hold every block.
__host__ __device__ inline int gate_fan(int blocks) { return blocks <= 256 ? 16 : kGateMaxFan; }
static_assert(kGateMaxBlocks <= kGateMaxFan * kGateMaxFan, "two levels of sums");
// A whole wave per token up to 16 tokens per expert, then 16 lanes.  In 16 lanes
// a token's chain of top-k steps is longer and few tokens leave most SIMDs with
// one wave or none; with many the whole waves' steps are mostly idle lanes.
// Forward and backward with a balance, 64 lanes against 16: 256 experts, 2048
// tokens 23 and 30 us, 4096: 29 and 31, 8192: 38 and 33; 128 experts, 2048
// tokens: 20 and 22, 4093: 25 and 23.
__host__ __device__ inline int64_t gate_wave_tokens(int experts) { return 16 * (int64_t)experts; }

__host__ __device__ inline int gate_lanes(int64_t tokens, int experts)
{
    return tokens <= gate_wave_tokens(experts) ? 64 : 16;
}

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
    // balance: counts [E+1], losses [2] and scratch (tickets, then a row of
    // partials per block and per fan of blocks)
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

// The other operand of a reduction across rows of 16 lanes (kRows 1: lane ^ 16,
// 2: lane ^ 32): a swap of rows between two copies leaves in one of them the
// lane's own value and in the other its partner's.
template <int kRows>
__device__ inline void row_swap(uint32_t v, uint32_t &a, uint32_t &b)
{
    const auto r = kRows == 1 ? __builtin_amdgcn_permlane16_swap(v, v, false, false)
                              : __builtin_amdgcn_permlane32_swap(v, v, false, false);
    a = r[0];
    b = r[1];
}
template <int kRows>
__device__ inline void across(float v, float &a, float &b)
{
    uint32_t x, y;
    row_swap<kRows>(__float_as_uint(v), x, y);
    a = __uint_as_float(x);
    b = __uint_as_float(y);
}
template <int kRows>
__device__ inline void across(int v, int &a, int &b)
{
    uint32_t x, y;
    row_swap<kRows>((uint32_t)v, x, y);
    a = (int)x;
    b = (int)y;
}
template <int kRows>
__device__ inline void across(double v, double &a, double &b)
{
    const uint64_t u = (uint64_t)__double_as_longlong(v);
    uint32_t lx, ly, hx, hy;
    row_swap<kRows>((uint32_t)u, lx, ly);
    row_swap<kRows>((uint32_t)(u >> 32), hx, hy);
    a = __longlong_as_double((long long)(((uint64_t)hx << 32) | lx));
    b = __longlong_as_double((long long)(((uint64_t)hy << 32) | ly));
}

#define EPDC_GROUP_REDUCE(name, T, dpp, expr)      \
    template <int kLanes>                          \
    __device__ inline T name(T a)                  \
    {                                              \
        T b = dpp<kXor1>(a);                       \
        a = expr;                                  \
        b = dpp<kXor2>(a);                         \
        a = expr;                                  \
        b = dpp<kMirror8>(a);                      \
        a = expr;                                  \
        b = dpp<kMirror16>(a);                     \
        a = expr;                                  \
        if constexpr (kLanes == 64) {              \
            across<1>(a, a, b);                    \
            a = expr;                              \
            across<2>(a, a, b);                    \
            a = expr;                              \
        }                                          \
        return a;                                  \
    }
EPDC_GROUP_REDUCE(group_max, float, dpp_f, fmaxf(a, b))
EPDC_GROUP_REDUCE(group_sum, float, dpp_f, (a + b))
EPDC_GROUP_REDUCE(group_min, int, dpp_i, (a < b ? a : b))
EPDC_GROUP_REDUCE(group_or, int, dpp_i, (a | b))
EPDC_GROUP_REDUCE(group_max, double, dpp_d, fmax(a, b))
EPDC_GROUP_REDUCE(group_sum, double, dpp_d, (a + b))
#undef EPDC_GROUP_REDUCE

template <typename T>
__device__ inline T lowest();
template <>
__device__ inline float lowest<float>() { return -__builtin_inff(); }
template <>
__device__ inline double lowest<double>() { return -__builtin_inf(); }

// Element of lane j's slot v: a lane holds kW consecutive elements of every
// kLanes * kW (16-byte loads of fp32 where kW is 4).
template <int kLanes, int kV>
__device__ inline int slot_expert(int v, int j)
{
    constexpr int kW = kV < 4 ? kV : 4;
    return v / kW * (kLanes * kW) + j * kW + v % kW;
}

__device__ inline float logit_at(const GateArgs &a, size_t at)
{
    return a.bf16 ? __uint_as_float((uint32_t)static_cast<const uint16_t *>(a.logits)[at] << 16)
                  : static_cast<const float *>(a.logits)[at];
}

template <int kLanes, int kV>
__device__ inline void load_logits(const GateArgs &a, int64_t token, int j, float (&l)[kV])
{
    constexpr int kW = kV < 4 ? kV : 4;
    const int E = a.experts;
    const bool wide = kW == 4 && (E & 3) == 0;  // rows of whole vectors stay aligned
    const size_t row = (size_t)token * E;
#pragma unroll
    for (int c = 0; c < kV / kW; ++c) {
        const int e = slot_expert<kLanes, kV>(c * kW, j);
#pragma unroll
        for (int i = 0; i < kW; ++i)
            l[c * kW + i] = lowest<float>();
        if (wide) {
            if (e >= E)
                continue;
            if (a.bf16) {
                const uint2 w = *reinterpret_cast<const uint2 *>(
                    static_cast<const uint16_t *>(a.logits) + row + e);
                const uint32_t u[4] = {w.x << 16, w.x & 0xFFFF0000u, w.y << 16, w.y & 0xFFFF0000u};
#pragma unroll
                for (int i = 0; i < kW; ++i)
                    l[c * kW + i] = __uint_as_float(u[i]);
            } else {
                const f32x4 w = *reinterpret_cast<const f32x4 *>(
                    static_cast<const float *>(a.logits) + row + e);
#pragma unroll
                for (int i = 0; i < kW; ++i)
                    l[c * kW + i] = w[i];
            }
        } else {
#pragma unroll
            for (int i = 0; i < kW; ++i)
                if (e + i < E)
                    l[c * kW + i] = logit_at(a, row + e + i);
        }
    }
}

// What a token's logits make of it.
enum { kTokenOut = 0, kTokenIn = 1, kTokenBad = 2 };

template <int kLanes, int kV>
__device__ inline int classify(const GateArgs &a, bool masked, const float (&l)[kV], float &m)
{
    float top = lowest<float>();
    int bad = 0;
#pragma unroll
    for (int v = 0; v < kV; ++v) {
        bad |= !(l[v] < __builtin_inff());  // NaN or +inf
        top = fmaxf(top, l[v]);
    }
    m = group_max<kLanes>(top);
    bad = group_or<kLanes>(bad);
    if (masked)
        return kTokenOut;
    if (bad)
        return kTokenBad;
    return m == lowest<float>() ? kTokenOut : kTokenIn;
}

// Take the group's largest key and its expert (lowest index among equals) out
// of the keys; expert -1 when nothing is left.
template <int kLanes, int kV, typename T>
__device__ inline void take_top(T (&key)[kV], int j, T &best, int &expert)
{
    T top = lowest<T>();
#pragma unroll
    for (int v = 0; v < kV; ++v)
        top = key[v] > top ? key[v] : top;
    best = group_max<kLanes>(top);
    int at = INT_MAX;
#pragma unroll
    for (int v = kV - 1; v >= 0; --v)
        at = key[v] == best ? slot_expert<kLanes, kV>(v, j) : at;
    expert = group_min<kLanes>(at);
    // this lane's slot of that expert, if it has it
    const int mine = expert == at ? at : -1;
#pragma unroll
    for (int v = 0; v < kV; ++v)
        key[v] = mine == slot_expert<kLanes, kV>(v, j) ? lowest<T>() : key[v];
    if (best == lowest<T>())
        expert = -1;
}

// exp in fp32 to about an ulp in six instructions: the hardware's 2^x of
// x log2(e), and the part of that product that fp32 does not hold as a factor.
// Arguments below -150 give 0.
__device__ inline float exp_near(float x)
{
    x = fmaxf(x, -150.0f);
    const float h = x * 1.44269502f;
    const float r = __builtin_fmaf(x, 1.92596303e-8f, __builtin_fmaf(x, 1.44269502f, -h));
    const float p = __builtin_amdgcn_exp2f(h);
    return __builtin_fmaf(p, r * 0.693147181f, p);
}

// 1 / x to about an ulp: the hardware's reciprocal and one Newton step
__device__ inline float recip_near(float x)
{
    const float r = __builtin_amdgcn_rcpf(x);
    return __builtin_fmaf(__builtin_fmaf(-x, r, 1.0f), r, r);
}

// log of a chosen score up to a constant of the row, without underflow:
// softmax: the logit; sigmoid: log sigma(l) = min(l, 0) - log(1 + exp(-|l|))
__device__ inline float log_score(int score, float l)
{
    if (score == kScoreSoftmax)
        return l;
    return fminf(l, 0.0f) - log1pf(expf(-fabsf(l)));
}

// The smaller of a sigmoid s and 1 - s, by the exponential of -|l|, which cannot
// overflow; 0 for -inf.  The slope s (1 - s) comes from it: by way of s
// rounded, 1 - s would be lost near 1.
__device__ inline float sigmoid_low(float l)
{
    const float x = exp_near(-fabsf(l));
    return x * recip_near(1.0f + x);
}
__device__ inline float sigmoid_of_low(float l, float low) { return l >= 0.0f ? 1.0f - low : low; }
__device__ inline float sigmoid(float l) { return sigmoid_of_low(l, sigmoid_low(l)); }

// A sigmoid's shares s / sum s where the row's largest logit m is this low: all
// s are e^l to within e^-20 of themselves (far below an ulp), so the shares are
// the softmax's, whose terms e^(l - m) do not vanish together as the s do.
__device__ inline bool far_below(float m) { return m < -20.0f; }

// Keys with a bias, s + b, are rounded sums of rounded scores; two neighbours of
// the order further apart than this are certainly in order.  In units of 2^-24:
// a softmax's sum has at most kV + 5 additions (kV - 1 in the lane, 4 or 6 across)
// of terms off by 4, its inverse and the product by one each, its terms' own 4
// count once, since the two scores add up to at most 1: kV + 15.  A sigmoid
// is off by 5, two of them by 10.  The sum s + b is off by half an ulp of each key.
template <int kV>
__device__ inline float key_slack(float k)
{
    return (kV + 16) * 5.9604645e-8f + 2.5e-7f * fabsf(k);
}

__device__ inline void store_agent(float *p, float v)
{
    __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// exp in 64 bits for x <= 0 or so, rolled up: it is hardly ever called, and the
// library's, inlined, fills the scalar registers of the whole kernel with its
// constants.  x = n ln 2 + r, and the series of e^r to r^14 / 14! (|r| < 0.35).
__device__ inline double exp_rolled(double x)
{
    x = x < -800.0 ? -800.0 : (x > 700.0 ? 700.0 : x);
    const double n = rint(x * 1.4426950408889634);
    // ln 2 in two parts, the first with zeros enough that n times it is exact
    const double r = fma(n, -1.9082149292705877e-10, fma(n, -0.6931471803691238, x));
    double p = 1.0, k = 14.0;
#pragma unroll 1
    for (; k > 0.5; k -= 1.0)
        p = fma(p * r, 1.0 / k, 1.0);
    return ldexp(p, (int)n);
}

// The key of expert e in 64 bits; -inf if it is unavailable.
__device__ inline double key64(const GateArgs &a, int64_t t, int e, double m, double inv_sum)
{
    const double l = (double)logit_at(a, (size_t)t * a.experts + e);
    if (!(l > lowest<double>()))
        return lowest<double>();
    const double x = exp_rolled(a.score == kScoreSoftmax ? l - m : -l);
    return (a.score == kScoreSoftmax ? x * inv_sum : 1.0 / (1.0 + x)) + (double)a.bias[e];
}

// The choice in 64 bits, for a token whose keys fp32 cannot put in order.
// `cand`: its first fp32 candidates, one per lane, which hold the true choice
// unless `more` follow as closely (equal logits and biases, say); then every
// expert is compared, key by key, without any array of keys: this code must not
// cost the common path registers.
template <int kLanes>
__device__ inline int choose64(const GateArgs &a, int64_t t, int j, float m, int cand, bool more)
{
    double inv = 1.0;
    if (a.score == kScoreSoftmax) {
        double part = 0.0;
#pragma unroll 1
        for (int e = j; e < a.experts; e += kLanes)
            part += exp_rolled((double)logit_at(a, (size_t)t * a.experts + e) - (double)m);
        inv = 1.0 / group_sum<kLanes>(part);
    }
    int chosen = -1;
    if (!more) {
        const double key = cand >= 0 ? key64(a, t, cand, m, inv) : lowest<double>();
        int rank = cand >= 0 ? 0 : -1;
#pragma unroll 1
        for (int i = 0; i < kMaxTopk; ++i) {
            const double k2 = __shfl(key, i, kLanes);
            const int e2 = __shfl(cand, i, kLanes);
            if (cand >= 0 && e2 >= 0 && (k2 > key || (k2 == key && e2 < cand)))
                ++rank;
        }
#pragma unroll 1
        for (int i = 0; i < kMaxTopk; ++i) {
            const int e2 = __shfl(cand, i, kLanes);
            if (__shfl(rank, i, kLanes) == j)
                chosen = e2;
        }
        return j < a.topk ? chosen : -1;
    }
    double last = -lowest<double>();
    int last_e = -1;
#pragma unroll 1
    for (int k = 0; k < a.topk; ++k) {
        double best = lowest<double>();
        int at = INT_MAX;
#pragma unroll 1
        for (int e = j; e < a.experts; e += kLanes) {
            const double key = key64(a, t, e, m, inv);
            if (key > best && (key < last || (key == last && e > last_e))) {
                best = key;
                at = e;
            }
        }
        const double top = group_max<kLanes>(best);
        if (!(top > lowest<double>()))
            break;
        last_e = group_min<kLanes>(best == top ? at : INT_MAX);
        last = top;
        if (j == k)
            chosen = last_e;
    }
    return chosen;
}

// Reads the logits once; a token's choice is kept by its group's lanes (lane k
// has choice k).  With a balance, each lane sums its experts' probabilities
// over its tokens; waves, then blocks, are added in a fixed order, the blocks
// by the last one to finish.  (32768 x 256 fp32, sigmoid, top-8 with balance:
// 50 us, 0.7 TB/s; 4093 x 128 bf16: 16 us; one token of 256 experts: 6 us, a
// launch.  Large batches are bound by the choice's steps per token, not bytes.)
template <int kLanes, int kV, bool kBalance>
__global__ __launch_bounds__(kGateThreads, kV < 32 ? 4 : 2) void k_gate(const GateArgs a)
{
    constexpr int kWaves = kGateThreads / 64, kTokens = kGateThreads / kLanes;
    extern __shared__ __align__(16) uint8_t dyn[];
    int *cnt = reinterpret_cast<int *>(dyn);                       // [E + 1]
    float *sum = reinterpret_cast<float *>(dyn) + a.experts + 1;   // [waves][E]
    float *zsum = sum + kWaves * a.experts;                        // [kTokens]
    __shared__ int last;
    __shared__ __align__(16) float bias[kGateThreads];  // as many as experts at most

    const int tid = threadIdx.x, lane = tid & 63, wave = tid / 64, j = tid & (kLanes - 1);
    const int E = a.experts, K = a.topk;
    if (a.bias)
        bias[tid] = tid < E ? a.bias[tid] : 0.0f;
    if (kBalance)
        for (int e = tid; e <= E; e += kGateThreads)
            cnt[e] = 0;
    if (kBalance || a.bias)
        __syncthreads();
    float prob[kV], z = 0.0f;
#pragma unroll
    for (int v = 0; v < kV; ++v)
        prob[v] = 0.0f;
    const bool softmax = a.score == kScoreSoftmax;
    const bool scores = kBalance || a.bias != nullptr || (softmax && !a.renorm);

    for (int64_t t0 = (int64_t)blockIdx.x * kTokens; t0 < a.tokens;
         t0 += (int64_t)gridDim.x * kTokens) {
        const int64_t t = t0 + tid / kLanes;
        if (t >= a.tokens)
            continue;
        float l[kV], m;
        load_logits<kLanes, kV>(a, t, j, l);
        const int kind = classify<kLanes, kV>(a, a.mask && a.mask[t] == 0, l, m);
        int chosen = -1;      // lane k: choice k
        float inv = 1.0f, lse = 0.0f;
        if (kind == kTokenIn) {
            float key[kV];
#pragma unroll
            for (int v = 0; v < kV; ++v)
                key[v] = l[v];
            if (scores) {
                // s: what the shares are of; a key's score is one factor away
                const bool exps = softmax || (kBalance && far_below(m));
                float s[kV], part = 0.0f, esum = 0.0f;
#pragma unroll
                for (int v = 0; v < kV; ++v) {
                    const float x = softmax || kBalance ? exp_near(l[v] - m) : 0.0f;
                    s[v] = exps ? x : sigmoid(l[v]);
                    part += s[v];
                    esum += x;
                }
                if (softmax || kBalance)
                    inv = 1.0f / group_sum<kLanes>(part);
                if (kBalance)
                    lse = m + logf(softmax ? 1.0f / inv : group_sum<kLanes>(esum));
                const float of_key = softmax ? inv : (exps ? exp_near(m) : 1.0f);
#pragma unroll
                for (int v = 0; v < kV; ++v) {
                    if (kBalance)
                        prob[v] += s[v] * inv;
                    if (a.bias && l[v] > lowest<float>())
                        key[v] = s[v] * of_key + bias[slot_expert<kLanes, kV>(v, j)];
                }
            }
            // with a bias on to the first clear gap behind the choice, 16 at most
            float before = __builtin_inff();
            bool close = false, more = false;
            for (int k = 0; k < K || a.bias; ++k) {
                float best;
                int e;
                take_top<kLanes, kV>(key, j, best, e);
                if (e < 0)
                    break;
                const bool near = before - best <= key_slack<kV>(best);
                if (k >= K && !near)
                    break;
                close |= near;
                if (k == kMaxTopk) {
                    more = true;
                    break;
                }
                before = best;
                if (j == k)
                    chosen = e;
            }
            if (close && a.bias)
                chosen = choose64<kLanes>(a, t, j, m, chosen, more);
            else if (j >= K)
                chosen = -1;
        }
        const bool have = chosen >= 0;
        float x = lowest<float>(), w = 0.0f;
        if (have)
            x = logit_at(a, (size_t)t * E + chosen);
        if (a.renorm) {
            const float ls = have ? log_score(a.score, x) : lowest<float>();
            const float top = group_max<kLanes>(ls);
            const float p = have ? expf(ls - top) : 0.0f;
            w = a.scale * (p / group_sum<kLanes>(p));
        } else if (have) {
            w = a.scale * (softmax ? expf(x - m) * inv : 1.0f / (1.0f + expf(-x)));
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

    // the wave's groups, then the block's waves
#pragma unroll
    for (int v = 0; v < kV; ++v) {
        float p = prob[v];
        if (kLanes == 16) {
            p += __shfl_xor(p, 16, 64);
            p += __shfl_xor(p, 32, 64);
        }
        const int e = slot_expert<kLanes, kV>(v, j);
        if (lane < kLanes && e < E)
            sum[wave * E + e] = p;
    }
    if (j == 0)
        zsum[tid / kLanes] = z;
    __syncthreads();
    // a row of partials: E counts, E probability sums, the token count, the z sum
    const int words = gate_partial_words(E);
    float *mine = a.partial + (size_t)blockIdx.x * words;
    for (int e = tid; e < E; e += kGateThreads) {
        float p = 0.0f;
#pragma unroll
        for (int w = 0; w < kWaves; ++w)
            p += sum[w * E + e];
        store_agent(mine + e, __int_as_float(cnt[e]));
        store_agent(mine + E + e, p);
    }
    if (wave == 0) {
        float zz = lane < kTokens ? zsum[lane] : 0.0f;
#pragma unroll
        for (int x = 1; x < 64; x <<= 1)
            zz += __shfl_xor(zz, x, 64);
        if (lane == 0) {
            store_agent(mine + 2 * E, __int_as_float(cnt[E]));
            store_agent(mine + 2 * E + 1, zz);
        }
    }
    // Every block's stores are at the device's point of coherence before it takes
    // a ticket.  The last of each `fan` blocks adds their rows, the last of
    // those the sums: with one level its last block alone read 256 rows, 40 us more.
    // Stores, tickets and loads are relaxed atomics of the agent's scope.  That the
    // wait for a wave's own stores orders them is no promise of the language but
    // of gfx950: such accesses are made in the memory that all XCDs share, so a
    // release would only add the write-back of an L2 that holds none of them,
    // and an acquire the drop of lines that nothing reads.
    const auto done = [&](uint32_t *ticket, uint32_t count) {
        __builtin_amdgcn_s_waitcnt(0);
        __syncthreads();
        if (tid == 0) {
            last = __hip_atomic_fetch_add(ticket, 1u, __ATOMIC_RELAXED,
                                          __HIP_MEMORY_SCOPE_AGENT) == count - 1;
            if (last)  // ready for the next call, which the stream orders after this one
                __hip_atomic_store(ticket, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
        __syncthreads();
        return last != 0;
    };
    // words 2 i and 2 i + 1 added over rows; every load is in flight at once
    const auto add_rows = [&](const float *from, int rows, int i, float &x, float &y) {
        uint64_t w[kGateMaxFan];
#pragma unroll
        for (int b = 0; b < kGateMaxFan; ++b)
            w[b] = b < rows ? __hip_atomic_load(
                                  reinterpret_cast<const uint64_t *>(from + (size_t)b * words) + i,
                                  __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT)
                            : 0;
        const auto word = [&](int at, int shift) {
            int c = 0;
            float p = 0.0f;
#pragma unroll
            for (int b = 0; b < kGateMaxFan; ++b) {
                c += (int)(uint32_t)(w[b] >> shift);
                p += __uint_as_float((uint32_t)(w[b] >> shift));
            }
            return at < E || at == 2 * E ? __int_as_float(c) : p;
        };
        x = word(2 * i, 0);
        y = word(2 * i + 1, 32);
    };
    const int nb = gridDim.x, fan = gate_fan(nb), groups = (nb + fan - 1) / fan;
    const int group = blockIdx.x / fan, first = group * fan;
    const int in_group = nb - first < fan ? nb - first : fan;
    if (!done(a.ticket + 1 + group, in_group))
        return;
    float *tops = a.partial + (size_t)nb * words;
    if (groups > 1) {
        for (int i = tid; i < words / 2; i += kGateThreads) {
            float x, y;
            add_rows(a.partial + (size_t)first * words, in_group, i, x, y);
            store_agent(tops + (size_t)group * words + 2 * i, x);
            store_agent(tops + (size_t)group * words + 2 * i + 1, y);
        }
        if (!done(a.ticket, groups))
            return;
    }
    const auto take = [&](int at, float v) {
        if (at < E || at == 2 * E) {
            const int e = at < E ? at : E;
            cnt[e] = __float_as_int(v);
            a.counts[e] = __float_as_int(v);
        } else {
            sum[at < 2 * E ? at - E : E] = v;
        }
    };
    for (int i = tid; i < words / 2; i += kGateThreads) {
        float x, y;
        add_rows(groups > 1 ? tops : a.partial, groups > 1 ? groups : nb, i, x, y);
        take(2 * i, x);
        take(2 * i + 1, y);
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
        }
    }
}

// One pass over the logits: with p the scores' softmax (sigmoid: s / sum s),
//   d/dl_j of scale * r(chosen)  and of  E/n sum_e f_e p_e  and of  lse^2 / n.
// (32768 x 256 fp32: 33 us, 2.0 TB/s; 4093 x 128 bf16: 6 us.)
template <int kLanes, int kV>
__global__ __launch_bounds__(kGateThreads, kV < 32 ? 4 : 2) void k_gate_backward(const GateArgs a)
{
    constexpr int kTokens = kGateThreads / kLanes, kW = kV < 4 ? kV : 4;
    const int tid = threadIdx.x, j = tid & (kLanes - 1);
    const int E = a.experts, K = a.topk;
    const bool softmax = a.score == kScoreSoftmax, balance = a.in_counts != nullptr;
    float gb = 0.0f, gz = 0.0f;
    float share[kV];
#pragma unroll
    for (int v = 0; v < kV; ++v)
        share[v] = 0.0f;
    if (balance) {
        const int n = a.in_counts[E] > 1 ? a.in_counts[E] : 1;
        const float per = 1.0f / ((float)n * (float)K);
        gb = a.grad_losses[0] * (float)E / (float)n;
        gz = a.grad_losses[1] * 2.0f / (float)n;
#pragma unroll
        for (int v = 0; v < kV; ++v) {
            const int e = slot_expert<kLanes, kV>(v, j);
            share[v] = e < E ? (float)a.in_counts[e] * per : 0.0f;
        }
    }
    for (int64_t t0 = (int64_t)blockIdx.x * kTokens; t0 < a.tokens;
         t0 += (int64_t)gridDim.x * kTokens) {
        const int64_t t = t0 + tid / kLanes;
        if (t >= a.tokens)
            continue;
        float l[kV], m;
        load_logits<kLanes, kV>(a, t, j, l);
        // the chosen: lane k holds choice k
        int e = -1;
        float g = 0.0f;
        if (j < K && a.grad_weights) {
            e = a.in_indices[t * K + j];
            e = e >= 0 && e < E ? e : -1;
            if (e >= 0)
                g = a.grad_weights[t * K + j] * a.scale;
        }
        const int kind = classify<kLanes, kV>(a, a.mask && a.mask[t] == 0, l, m);
        float d[kV];
#pragma unroll
        for (int v = 0; v < kV; ++v)
            d[v] = kind == kTokenBad ? __builtin_nanf("") : 0.0f;
        if (kind == kTokenIn) {
            // the rows' softmax x / xs and shares s / ss; low: s, of a sigmoid's
            // that and 1 - s the smaller
            const bool exps = softmax || far_below(m);
            float x[kV], low[kV], xs = 0.0f, ss = 0.0f, fp = 0.0f;
#pragma unroll
            for (int v = 0; v < kV; ++v) {
                x[v] = exp_near(l[v] - m);
                xs += x[v];
                low[v] = exps ? x[v] : sigmoid_low(l[v]);
                const float s = exps ? x[v] : sigmoid_of_low(l[v], low[v]);
                ss += s;
                fp += share[v] * s;
            }
            xs = group_sum<kLanes>(xs);
            ss = softmax ? xs : group_sum<kLanes>(ss);
            fp = group_sum<kLanes>(fp) / ss;
            const float le = e >= 0 ? logit_at(a, (size_t)t * E + e) : lowest<float>();
            float r = 0.0f, dc = 0.0f, all = 0.0f;  // all: taken from every p of a softmax
            if (a.renorm) {
                const float ls = e >= 0 ? log_score(a.score, le) : lowest<float>();
                const float top = group_max<kLanes>(ls);
                r = e >= 0 ? expf(ls - top) : 0.0f;
                const float rs = group_sum<kLanes>(r);
                r = rs > 0.0f ? r / rs : 0.0f;
                dc = r * (g - group_sum<kLanes>(g * r));
                if (!softmax)
                    dc *= e >= 0 ? sigmoid(-le) : 0.0f;
            } else if (softmax) {
                r = e >= 0 ? expf(le - m) / xs : 0.0f;
                dc = g * r;
                all = group_sum<kLanes>(dc);
            } else {
                const float lo = sigmoid_low(le);   // 0 without a choice
                dc = g * lo * (1.0f - lo);
            }
            const float lse = m + logf(xs), rx = 1.0f / xs, rs = 1.0f / ss;
#pragma unroll
            for (int v = 0; v < kV; ++v) {
                const float q = x[v] * rx;
                float b = gb * (low[v] * rs) * (share[v] - fp);
                if (!exps)   // of far_below's, 1 to within e^-20
                    b *= 1.0f - low[v];
                d[v] = b + (gz * lse - all) * q;
            }
            if (a.grad_weights)
                for (int k = 0; k < K; ++k) {
                    const int ek = __shfl(e, k, kLanes);
                    const float dk = __shfl(dc, k, kLanes);
#pragma unroll
                    for (int v = 0; v < kV; ++v)
                        d[v] += slot_expert<kLanes, kV>(v, j) == ek ? dk : 0.0f;
                }
#pragma unroll
            for (int v = 0; v < kV; ++v)
                if (l[v] == lowest<float>())
                    d[v] = 0.0f;
        }
        const size_t row = (size_t)t * E;
        const bool wide = kW == 4 && (E & 3) == 0;
#pragma unroll
        for (int c = 0; c < kV / kW; ++c) {
            const int at = slot_expert<kLanes, kV>(c * kW, j);
            if (wide) {
                if (at >= E)
                    continue;
                const f32x4 o{d[c * kW], d[c * kW + 1 % kW], d[c * kW + 2 % kW],
                              d[c * kW + 3 % kW]};
                if (a.bf16)
                    *reinterpret_cast<bf16x4 *>(static_cast<__bf16 *>(a.grad_logits) + row + at) =
                        to_bf16(o);
                else
                    *reinterpret_cast<f32x4 *>(static_cast<float *>(a.grad_logits) + row + at) = o;
            } else {
#pragma unroll
                for (int i = 0; i < kW; ++i)
                    if (at + i < E) {
                        if (a.bf16)
                            static_cast<__bf16 *>(a.grad_logits)[row + at + i] =
                                (__bf16)d[c * kW + i];
                        else
                            static_cast<float *>(a.grad_logits)[row + at + i] = d[c * kW + i];
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
    int32_t first;                   // token of the launch's first block
    const int32_t *slot_of;
    const uint8_t *grad_output, *input;
    const float *weights;
    uint8_t *grad_input;
    float *grad_weights;
};

constexpr int kCombineGradThreads = 512;

// A block per token: a thread reads a vector of the token's gradient once and
// serves the K rows with it -- the row's vector for the dot product in, the
// scaled gradient out.  Bytes are the bound (one row read and one written per
// pair): 4096 x 7168 bf16, top-8, 998 MB in 193 to 196 us, 5.1 TB/s of the 5.7
// that copies reach; with 1024 threads 225 us where 512 took 195.
template <int kTopk>
__global__ __launch_bounds__(kCombineGradThreads) void k_combine_grad(const CombineGradArgs a)
{
    constexpr int kMax = kTopk ? kTopk : kMaxTopk, kWaves = kCombineGradThreads / 64;
    __shared__ float part[kWaves][kMax];
    const int K = kTopk ? kTopk : a.topk;
    const int64_t t = (int64_t)a.first + blockIdx.x;
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
