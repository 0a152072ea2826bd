// layer_few.hpp -- gfx950 kernels of a layer for few tokens: dispatch, the experts'
// two products and combine as two launches,
//   k_few_up:    h[t, k]  = act(x[t] W1[e]^T + b1[e]),      e = indices[t, k]
//   k_few_down:  y[t]     = sum_k w[t, k] (h[t, k] W2[e]^T + b2[e])
//
// The weights of the experts that are asked for are the traffic, read once as in
// k_product_stream (whole 128-byte lines past the caches, turned through LDS into
// fragments); nothing is routed in memory.  Every block finds the experts'
// tokens from the indices itself: at most 1024, a token set per expert in one
// 64-bit word.  8-bit weights are widened to bf16, which holds them exactly, so
// the activations stay bf16.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "layer_product.hpp"

namespace epdc_layer {

constexpr int kFewTokens = 64, kFewPairs = 1024;

struct FewArgs {
    int32_t tokens, topk, experts, first_expert;
    int32_t hidden, inner, act;
    const uint8_t *x;
    const float *weights;
    const int32_t *indices;
    const uint8_t *w1, *w2;
    const float *s1, *s2, *b1, *b2;
    uint8_t *h;    // [tokens * topk, inner] bf16
    uint8_t *out;  // [tokens, hidden] bf16
};

// Who asks for which expert, in LDS.
struct FewRouting {
    uint64_t tokens[kMaxExperts];   // of an expert of this call
    int16_t id[kFewPairs];          // expert of a pair, -1 for none of this call's
    int16_t active[kMaxExperts];    // experts with tokens, ascending
};

// Fills the routing and ends with a barrier; returns the number of active experts.
template <int kThreads>
__device__ inline int few_routing(const FewArgs &a, FewRouting &r)
{
    const int tid = threadIdx.x, lane = tid & 63;
    for (int e = tid; e < a.experts; e += kThreads)
        r.tokens[e] = 0;
    __syncthreads();
    const int pairs = a.tokens * a.topk;
    for (int p = tid; p < pairs; p += kThreads) {
        const uint32_t e = (uint32_t)a.indices[p] - (uint32_t)a.first_expert;
        const bool in = e < (uint32_t)a.experts;
        r.id[p] = (int16_t)(in ? e : -1);
        if (in)
            atomicOr(reinterpret_cast<unsigned long long *>(&r.tokens[e]),
                     1ull << (p / a.topk));
    }
    __syncthreads();
    int count = 0;
    for (int e0 = 0; e0 < a.experts; e0 += 64) {
        const int e = e0 + lane;
        const bool some = e < a.experts && r.tokens[e] != 0;
        const uint64_t set = __ballot(some);
        if (some && tid < 64)
            r.active[count + __popcll(set & ((1ull << lane) - 1))] = (int16_t)e;
        count += __popcll(set);
    }
    __syncthreads();
    return uniform(count);
}

// The tokens of a set in ascending order, one per lane of the wave, in `list`.
__device__ inline int few_rows(uint64_t set, int lane, uint8_t *list)
{
    if (set >> lane & 1)
        list[__popcll(set & ((1ull << lane) - 1))] = (uint8_t)lane;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    return __popcll(set);
}

// 16 bytes of weight as fragments of 8 bf16: as they are, or widened.
template <int kType>
struct FewWeight {
    static constexpr int kFrags = 2 / element_bytes(kType);
    __device__ static inline void widen(i32x4 w, i32x4 (&f)[kFrags])
    {
        if constexpr (kType == kTypeBf16) {
            f[0] = w;
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint32_t lo, hi;   // elements 0, 1 and 2, 3 of word i
                if constexpr (kType == kTypeE4m3) {
                    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
                    const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[i], 1.0f, false);
                    const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[i], 1.0f, true);
                    lo = __builtin_bit_cast(uint32_t, a);
                    hi = __builtin_bit_cast(uint32_t, b);
                } else {   // a code of 8 bits fits bf16's significand: the upper half of its fp32
                    uint32_t u[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        u[k] = __float_as_uint((float)(int8_t)((uint32_t)w[i] >> (8 * k)));
                    lo = __builtin_amdgcn_perm(u[1], u[0], 0x07060302u);
                    hi = __builtin_amdgcn_perm(u[3], u[2], 0x07060302u);
                }
                f[i / 2][i % 2 * 2] = (int)lo;
                f[i / 2][i % 2 * 2 + 1] = (int)hi;
            }
        }
    }
};

// A wave's part of rows x columns: kMI * 16 rows of bf16 (x or h) by 16 columns of kQ
// weights, over the steps [s0, s1) of 128 weight bytes, `stride` steps apart.
template <int kType, int kMI, int kQ>
struct FewProduct {
    typedef FewWeight<kType> Weight;
    static constexpr int kFrags = Weight::kFrags;
    static constexpr int kStep = kStepBytes / element_bytes(kType);  // elements
    static constexpr int kTurnBytes = 2 * kQ * 16 * kStepBytes;      // LDS of a wave
    // steps whose loads are in flight
    static constexpr int kBatch = kType == kTypeBf16 ? 4 / kMI : 2 / kMI;

    int contract, lane, rows;   // rows: that hold a token
    uint8_t *turn;
    const uint8_t *qp[kQ][2];
    const float *scale[kQ];     // e4m3: of the columns' block
    __amdgpu_buffer_rsrc_t p;
    uint32_t off[kMI];          // of this lane's row and contraction part in p, or kNowhere
    f32x4 acc[kMI][kQ];

    __device__ inline void clear()
    {
#pragma unroll
        for (int i = 0; i < kMI; ++i)
#pragma unroll
            for (int q = 0; q < kQ; ++q)
                acc[i][q] = f32x4{0, 0, 0, 0};
    }
    // from column c0 of each q of expert e's weight, cols columns each (rows in memory)
    __device__ inline void weights(const uint8_t *w, const float *s, int e, int c0, int cols)
    {
        const size_t bytes = (size_t)contract * element_bytes(kType);
        w += (size_t)e * kQ * cols * bytes;
#pragma unroll
        for (int q = 0; q < kQ; ++q) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                int c = c0 + h * 8 + (lane >> 3);
                c = (c < cols ? c : cols - 1) + q * cols;
                qp[q][h] = w + c * bytes + (lane & 7) * 16;
            }
            if constexpr (kType == kTypeE4m3) {
                const int of_expert = (kQ * cols + 127) / 128;
                scale[q] = s + ((size_t)e * of_expert + (q * cols + c0) / 128) * (contract / 128);
            }
        }
    }
    template <bool kTail>
    __device__ inline void load(int s, i32x4 (&w)[kQ][2], i32x4 (&x)[kMI][2][kFrags])
    {
        const bool in = !kTail || s * kStep + (lane & 7) * (16 / element_bytes(kType)) < contract;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int q = 0; q < kQ; ++q) {
                const i32x4 *at = reinterpret_cast<const i32x4 *>(qp[q][h] + (size_t)s * kStepBytes);
                w[q][h] = in ? __builtin_nontemporal_load(at) : i32x4{0, 0, 0, 0};
            }
#pragma unroll
            for (int i = 0; i < kMI; ++i) {
                if (i * 16 >= rows)
                    continue;
#pragma unroll
                for (int f = 0; f < kFrags; ++f) {
                    const int el = s * kStep + h * (kStep / 2) + (lane >> 4) * (8 * kFrags) + f * 8;
                    const uint32_t o = kTail && el >= contract
                                           ? kNowhere
                                           : off[i] + (s * kStep + h * (kStep / 2) + f * 8) * 2;
                    x[i][h][f] = __builtin_bit_cast(
                        i32x4, __builtin_amdgcn_raw_buffer_load_b128(p, o, 0, 0));
                }
            }
        }
    }
    // lines of 8 + 8 columns to fragments of 16; lanes read what others wrote, in
    // the order in which the wave's LDS accesses run
    __device__ inline void turned(i32x4 (&w)[kQ][2], int buf)
    {
        typedef StraightTile<16, 1, false> Turn;
        uint8_t *to = turn + buf * (kQ * 16 * kStepBytes);
#pragma unroll
        for (int q = 0; q < kQ; ++q)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int r = h * 8 + (lane >> 3);
                *reinterpret_cast<i32x4 *>(to + (q * 16 + r) * kStepBytes +
                                           ((lane & 7) ^ (r & 7)) * 16) = w[q][h];
            }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int q = 0; q < kQ; ++q)
#pragma unroll
            for (int h = 0; h < 2; ++h)
                w[q][h] = Turn::frag(to + q * 16 * kStepBytes, 0, h, lane);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
    }
    __device__ inline void multiply(int s, const i32x4 (&w)[kQ][2],
                                    const i32x4 (&x)[kMI][2][kFrags])
    {
#pragma unroll
        for (int q = 0; q < kQ; ++q) {
            i32x4 f[2][kFrags];
            Weight::widen(w[q][0], f[0]);
            Weight::widen(w[q][1], f[1]);
#pragma unroll
            for (int i = 0; i < kMI; ++i) {
                if (i * 16 >= rows)
                    continue;
                f32x4 d = kType == kTypeE4m3 ? f32x4{0, 0, 0, 0} : acc[i][q];
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int k = 0; k < kFrags; ++k)
                        d = mfma_bf16(f[h][k], x[i][h][k], d);
                if constexpr (kType == kTypeE4m3) {
                    const float by = scale[q][s];
#pragma unroll
                    for (int v = 0; v < 4; ++v)
                        acc[i][q][v] = __builtin_fmaf(d[v], by, acc[i][q][v]);
                } else {
                    acc[i][q] = d;
                }
            }
        }
    }
    __device__ inline void run(int s0, int s1, int stride)
    {
        const int whole = contract / kStep;
        int s = s0;
        for (; s + (kBatch - 1) * stride < (s1 < whole ? s1 : whole); s += kBatch * stride) {
            i32x4 w[kBatch][kQ][2], x[kBatch][kMI][2][kFrags];
#pragma unroll
            for (int b = 0; b < kBatch; ++b)
                load<false>(s + b * stride, w[b], x[b]);
#pragma unroll
            for (int b = 0; b < kBatch; ++b) {
                turned(w[b], b & 1);
                multiply(s + b * stride, w[b], x[b]);
            }
        }
        for (; s < s1; s += stride) {
            i32x4 w[kQ][2], x[kMI][2][kFrags];
            load<true>(s, w, x);
            turned(w, 0);
            multiply(s, w, x);
        }
    }
};

constexpr int kFewUpWaves = 4, kFewDownWaves = 8;

// A block: 16 columns of h (gated: 16 gate and 16 up) of one active expert; its waves
// take the contraction's steps in turn.
template <int kType, int kMI, bool kGated>
__global__ __launch_bounds__(kFewUpWaves *kWave) void k_few_up(const FewArgs a)
{
    constexpr int kQ = kGated ? 2 : 1;
    typedef FewProduct<kType, kMI, kQ> Product;
    __shared__ FewRouting routing;
    __shared__ __align__(16) f32x4 part[kFewUpWaves][kMI * kQ][kWave];
    __shared__ __align__(16) uint8_t turn[kFewUpWaves][Product::kTurnBytes];
    __shared__ uint8_t lists[kFewUpWaves][kFewTokens];
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x / kWave);
    const int count = few_routing<kFewUpWaves * kWave>(a, routing);
    const int col_tiles = (a.inner + 15) / 16, n = blockIdx.x / col_tiles;
    if (n >= count)
        return;
    const int e = uniform(routing.active[n]), c0 = (blockIdx.x - n * col_tiles) * 16;
    const int rows = uniform(few_rows(routing.tokens[e], lane, lists[wave]));
    Product m;
    m.contract = a.hidden;
    m.lane = lane;
    m.turn = turn[wave];
    m.p = buffer_at(a.x, (uint32_t)a.tokens * a.hidden * 2);
    const int cols = a.inner * kQ;
    m.weights(a.w1, a.s1, e, c0, a.inner);
    const int steps = (a.hidden + Product::kStep - 1) / Product::kStep;
    for (int r0 = 0; r0 < rows; r0 += kMI * 16) {
        m.rows = rows - r0;
#pragma unroll
        for (int i = 0; i < kMI; ++i) {
            const int r = r0 + i * 16 + (lane & 15);
            m.off[i] = r < rows ? (uint32_t)lists[wave][r] * a.hidden * 2 +
                                      (lane >> 4) * (Product::kFrags * 16)
                                : kNowhere;
        }
        m.clear();
        m.run(wave, steps, kFewUpWaves);
        if (r0 > 0)
            __syncthreads();   // the parts of the rows before have been read
#pragma unroll
        for (int i = 0; i < kMI; ++i)
#pragma unroll
            for (int q = 0; q < kQ; ++q)
                part[wave][i * kQ + q][lane] = m.acc[i][q];
        __syncthreads();
        // wave i finishes row block i, adding the waves' parts in order
        for (int i = wave; i < kMI; i += kFewUpWaves) {
            f32x4 z[2] = {f32x4{0, 0, 0, 0}, f32x4{0, 0, 0, 0}};
#pragma unroll
            for (int q = 0; q < kQ; ++q)
#pragma unroll
                for (int w = 0; w < kFewUpWaves; ++w)
                    z[q] += part[w][i * kQ + q][lane];
            const int r = r0 + i * 16 + (lane & 15), c = c0 + (lane >> 4) * 4;
            if (r >= rows || c >= a.inner)
                continue;
#pragma unroll
            for (int q = 0; q < kQ; ++q) {
                const size_t at = (size_t)e * cols + q * a.inner + c;
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    if constexpr (kType == kTypeInt8)
                        z[q][v] *= a.s1[at + v];
                    if (a.b1)
                        z[q][v] += a.b1[at + v];
                }
            }
            f32x4 y;
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                y[v] = act_one(a.act, z[0][v]);
                if (kGated)
                    y[v] *= z[1][v];
            }
            const int t = lists[wave][r];
            for (int k = 0; k < a.topk; ++k)
                if (routing.id[t * a.topk + k] == e)
                    *reinterpret_cast<bf16x4 *>(
                        a.h + ((size_t)(t * a.topk + k) * a.inner + c) * 2) = to_bf16(y);
        }
    }
}

// A block: 16 columns of y over every active expert.  The experts' contractions end to
// end are one list of steps, of which each wave takes an equal run; where a run
// leaves an expert, its sums go, weighted, to the wave's totals of the tokens in
// LDS, and the waves' totals are added in order.  (Rows of tokens that do not ask
// for an expert never meet its weights, whatever these hold.)
template <int kType, int kMI>
__global__ __launch_bounds__(kFewDownWaves *kWave) void k_few_down(const FewArgs a)
{
    typedef FewProduct<kType, kMI, 1> Product;
    __shared__ FewRouting routing;
    __shared__ __align__(16) f32x4 total[kFewDownWaves][kFewTokens][4];
    __shared__ __align__(16) uint8_t turn[kFewDownWaves][Product::kTurnBytes];
    __shared__ uint8_t lists[kFewDownWaves][kFewTokens];
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x / kWave);
    const int count = few_routing<kFewDownWaves * kWave>(a, routing);
    const int c0 = blockIdx.x * 16;
    for (int i = lane; i < a.tokens * 4; i += kWave)
        total[wave][i / 4][i % 4] = f32x4{0, 0, 0, 0};
    Product m;
    m.contract = a.inner;
    m.lane = lane;
    m.turn = turn[wave];
    m.p = buffer_at(a.h, (uint32_t)a.tokens * a.topk * a.inner * 2);
    const int steps = (a.inner + Product::kStep - 1) / Product::kStep;
    const int all = count * steps;
    int at = (int)((int64_t)all * wave / kFewDownWaves);
    const int end = (int)((int64_t)all * (wave + 1) / kFewDownWaves);
    while (at < end) {
        const int n = at / steps, s0 = at - n * steps;
        const int left = end - at, s1 = s0 + left < steps ? s0 + left : steps;
        at += s1 - s0;
        const int e = uniform(routing.active[n]);
        const int rows = uniform(few_rows(routing.tokens[e], lane, lists[wave]));
        m.weights(a.w2, a.s2, e, c0, a.hidden);
        for (int r0 = 0; r0 < rows; r0 += kMI * 16) {
            m.rows = rows - r0;
            int token[kMI];
            float by[kMI];   // the token's weight for this expert
#pragma unroll
            for (int i = 0; i < kMI; ++i) {
                const int r = r0 + i * 16 + (lane & 15);
                token[i] = -1;
                by[i] = 0.0f;
                m.off[i] = kNowhere;
                if (r < rows) {
                    token[i] = lists[wave][r];
                    for (int k = a.topk - 1; k >= 0; --k) {
                        const int p = token[i] * a.topk + k;
                        if (routing.id[p] == e) {
                            by[i] += a.weights ? a.weights[p] : 1.0f;
                            m.off[i] = (uint32_t)p * a.inner * 2 +
                                       (lane >> 4) * (Product::kFrags * 16);
                        }
                    }
                }
            }
            m.clear();
            m.run(s0, s1, 1);
            const int c = c0 + (lane >> 4) * 4;
#pragma unroll
            for (int i = 0; i < kMI; ++i) {
                if (token[i] < 0 || c >= a.hidden)
                    continue;
                f32x4 &sum = total[wave][token[i]][lane >> 4];
                f32x4 o = m.acc[i][0];
                const size_t col = (size_t)e * a.hidden + c;
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    if constexpr (kType == kTypeInt8)
                        o[v] *= a.s2[col + v];
                    if (a.b2 && s0 == 0)
                        o[v] += a.b2[col + v];
                    sum[v] = __builtin_fmaf(by[i], o[v], sum[v]);
                }
            }
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < a.tokens * 4; i += kFewDownWaves * kWave) {
        const int c = c0 + i % 4 * 4;
        if (c >= a.hidden)
            continue;
        f32x4 y = total[0][i / 4][i % 4];
#pragma unroll
        for (int w = 1; w < kFewDownWaves; ++w)
            y += total[w][i / 4][i % 4];
        *reinterpret_cast<bf16x4 *>(a.out + ((size_t)(i / 4) * a.hidden + c) * 2) = to_bf16(y);
    }
}

}  // namespace epdc_layer
