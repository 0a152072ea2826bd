// layer_rows.hpp -- gfx950 kernels over whole rows: the root-mean-square norm with
// the residual's addition and rows in 8 bits, its gradient, and bf16 rows into
// 8 bits.
//
// A team of 1, 4, 8 or 16 waves owns a row and keeps it in registers from its one
// read to its one write; the row's sums go through LDS once.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "layer_gate.hpp"
#include "layer_product.hpp"

namespace epdc_layer {

enum Codes { kCodesNone, kCodesE4m3, kCodesInt8 };

constexpr int kMaxNormFeatures = 1 << 15;   // what 16 waves hold
constexpr int kMaxQuantFeatures = 1 << 17;
constexpr int kCodeBlock = 128;             // e4m3: columns of a scale

// Threads of a block whose teams are of kWaves waves.
constexpr int team_threads(int waves) { return waves < 4 ? 256 : waves * 64; }

__device__ inline int abs_bits(float v) { return __float_as_int(v) & 0x7fffffff; }

// Largest of the absolute values' bit patterns over 16 or 64 lanes, in every lane of
// them.  As whole numbers, because NaN lies above infinity then: a row that holds
// one gets a scale of NaN instead of one of the other values'.
template <int kLanes>
__device__ inline int group_top(int a)
{
    const auto take = [&](int b) { a = a > b ? a : b; };
    take(dpp_i<kXor1>(a));
    take(dpp_i<kXor2>(a));
    take(dpp_i<kMirror8>(a));
    take(dpp_i<kMirror16>(a));
    if constexpr (kLanes == 64) {
        int x, y;
        across<1>(a, x, y);
        a = x > y ? x : y;
        across<2>(a, x, y);
        a = x > y ? x : y;
    }
    return a;
}

// What a row is reduced to: the sum of its squares, a sum of products, the largest
// pattern.
struct RowSums {
    float squares, cross;
    int top;
};

// Over a team, in every lane.  Between two calls with the same `parts` there is always one
// with others, whose barrier separates the readers of the first from the writers of the
// second.
template <int kWaves, bool kCross, bool kTop>
__device__ inline RowSums team_reduce(RowSums s, RowSums (&parts)[kWaves])
{
    s.squares = group_sum<64>(s.squares);
    if constexpr (kCross)
        s.cross = group_sum<64>(s.cross);
    if constexpr (kTop)
        s.top = group_top<64>(s.top);
    if constexpr (kWaves > 1) {
        if ((threadIdx.x & 63) == 0)
            parts[threadIdx.x / 64] = s;
        __syncthreads();
        s = parts[0];
#pragma unroll
        for (int w = 1; w < kWaves; ++w) {
            s.squares += parts[w].squares;
            s.cross += parts[w].cross;
            s.top = s.top > parts[w].top ? s.top : parts[w].top;
        }
    }
    return s;
}

// x / s to nearest, for the codes of a row or block: from the correctly rounded
// reciprocal r of s, two corrections of the quotient by its exact remainder, of
// which the second gives the rounding of the true quotient.  Five instructions
// where the division itself takes about fourteen slots.  `plain`: s is so small or
// large that a remainder might not be exact, or no number.
__device__ inline float quotient(float x, float s, float r, bool plain)
{
    if (plain)
        return x / s;
    float q = x * r;
    q = __builtin_fmaf(__builtin_fmaf(-q, s, x), r, q);
    return __builtin_fmaf(__builtin_fmaf(-q, s, x), r, q);
}
__device__ inline bool plain_scale(float s) { return !(s >= 0x1p-60f && s <= 0x1p60f); }

// Codes of values whose largest is `limit` scales: 4 per word.  The clamp is for
// scales below the normal numbers, which are off by more than the codes' range
// has room for.
template <int kCodes>
__device__ inline uint32_t four_codes(const float *v, float s, float r, bool plain)
{
    float q[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        q[i] = s == 0.0f ? 0.0f : quotient(v[i], s, r, plain);
        if (plain)
            q[i] = kCodes == kCodesE4m3 ? __builtin_amdgcn_fmed3f(q[i], -448.0f, 448.0f)
                                        : __builtin_amdgcn_fmed3f(q[i], -127.0f, 127.0f);
        else if (kCodes == kCodesE4m3)   // a zero's sign, which it lost to a remainder of +0
            q[i] = __builtin_copysignf(q[i], v[i]);
    }
    if constexpr (kCodes == kCodesE4m3) {
        const uint32_t lo = __builtin_amdgcn_cvt_pk_fp8_f32(q[0], q[1], 0u, false);
        return __builtin_amdgcn_cvt_pk_fp8_f32(q[2], q[3], lo, true);
    } else {
        // adding 1.5 * 2^23 rounds to a whole number, to even, and leaves it in the low bits
        uint32_t u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            u[i] = __float_as_uint(q[i] + 12582912.0f);
        const uint32_t lo = __builtin_amdgcn_perm(u[1], u[0], 0x0c0c0400u);
        const uint32_t hi = __builtin_amdgcn_perm(u[3], u[2], 0x0c0c0400u);
        return lo | hi << 16;
    }
}

// ---------------------------------------------------------------------------
// The norm
// ---------------------------------------------------------------------------

struct NormArgs {
    int32_t rows, vecs;      // vecs: 16-byte vectors of a row, 8 elements each
    int32_t weight_bf16;
    float features, eps;
    const uint8_t *input, *residual, *weight;  // residual: or NULL
    uint8_t *out, *sum, *codes;                // out, sum: or NULL
    float *scales;
    // backward
    const uint8_t *grad_out, *grad_sum;
    uint8_t *grad_input;
    float *partial;          // [blocks * teams][features], or NULL
};

__device__ inline void weight_at(const NormArgs &a, int v, float (&w)[8])
{
    if (a.weight_bf16) {
        const bf16x8 b = *reinterpret_cast<const bf16x8 *>(a.weight + (size_t)v * 16);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            w[i] = (float)b[i];
    } else {
        const f32x4 *p = reinterpret_cast<const f32x4 *>(a.weight + (size_t)v * 32);
        const f32x4 lo = p[0], hi = p[1];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            w[i] = lo[i];
            w[4 + i] = hi[i];
        }
    }
}

// 1 / sqrt(mean of squares + eps) from the team's sum of squares.  Where the sum, or the mean
// with eps, is beyond fp32, or the mean is so small that squares may have lost bits below
// the normal numbers, the team adds squares(c) instead, those of its elements times a
// power of two.  Elements are below 2^128, and below 2^-12 where the mean is below 2^-40.
template <int kWaves, typename F>
__device__ inline float inverse_rms(const NormArgs &a, float sum, RowSums (&parts)[kWaves],
                                    F &&squares)
{
    const float mean = sum / a.features + a.eps;
    if (mean >= 0x1p-40f && mean < __builtin_inff())
        return 1.0f / sqrtf(mean);
    const float c = mean < 1.0f ? 0x1p72f : 0x1p-80f;
    const RowSums s = team_reduce<kWaves, false, false>(RowSums{squares(c), 0.0f, 0}, parts);
    return c / sqrtf(s.squares / a.features + a.eps * c * c);
}

// Whether a product that should be a number of the usual size is one: not 0, beyond fp32
// or so small that it may have lost bits.
__device__ inline bool in_range(float v) { return v >= 0x1p-100f && v < __builtin_inff(); }

// s = x + r, y = s w / rms(s), each rounded once from fp32; codes from the unrounded y.
// Bytes are the bound.  The sum leaves past the caches, as nothing reads it before the
// layer's weights have gone through them, out does not: with the router's product behind it
// 4096 x 7168 took 68.8 us, sum past the caches 67.7, both 75.9.  (4096 x 7168 with the
// residual into bf16 and e4m3, 265 MB: 46.5 us, 5.7 TB/s; one row 2.7.)  The weight comes
// last, as s w can leave fp32 where y does not.  The largest |y| of an int8 row still
// comes with the first reduction, from the largest |s w|, unless that has left it.
template <int kWaves, int kV, int kCodes>
__global__ __launch_bounds__(team_threads(kWaves)) void k_rms_norm(const NormArgs a)
{
    constexpr int kTeams = team_threads(kWaves) / (kWaves * 64), kLanes = kWaves * 64;
    __shared__ RowSums parts[2][kWaves], again[kWaves], tops[kWaves];
    const int tid = threadIdx.x & (kLanes - 1), team = threadIdx.x / kLanes;
    int turn = 0;
    for (int64_t row = (int64_t)blockIdx.x * kTeams + team; row < a.rows;
         row += (int64_t)gridDim.x * kTeams, turn ^= 1) {
        const size_t at = (size_t)row * a.vecs;
        bf16x8 x[kV], res[kV];
        float t[kV][8], w[kV][8];
#pragma unroll
        for (int k = 0; k < kV; ++k) {
            const int v = k * kLanes + tid;
            x[k] = res[k] = bf16x8{};
            if (v < a.vecs) {
                x[k] = *reinterpret_cast<const bf16x8 *>(a.input + (at + v) * 16);
                if (a.residual)
                    res[k] = *reinterpret_cast<const bf16x8 *>(a.residual + (at + v) * 16);
                weight_at(a, v, w[k]);
            }
        }
        RowSums s = {0.0f, 0.0f, 0};
#pragma unroll
        for (int k = 0; k < kV; ++k) {
            const int v = k * kLanes + tid;
            bf16x8 o;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                t[k][i] = (float)x[k][i];
                if (a.residual)
                    t[k][i] += (float)res[k][i];
                o[i] = (__bf16)t[k][i];
                s.squares = __builtin_fmaf(t[k][i], t[k][i], s.squares);
            }
            if (v >= a.vecs)
                continue;
            if (a.sum)
                __builtin_nontemporal_store(o, reinterpret_cast<bf16x8 *>(a.sum + (at + v) * 16));
            if constexpr (kCodes == kCodesInt8) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int b = abs_bits(t[k][i] * w[k][i]);
                    s.top = s.top > b ? s.top : b;
                }
            }
        }
        s = team_reduce<kWaves, false, kCodes == kCodesInt8>(s, parts[turn]);
        const float inv = inverse_rms(a, s.squares, again, [&](float c) {
            float sum = 0.0f;
#pragma unroll
            for (int k = 0; k < kV; ++k)
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    sum = __builtin_fmaf(t[k][i] * c, t[k][i] * c, sum);
            return sum;
        });
        float scale = 0.0f, recip = 0.0f;
        bool plain = false;
        if constexpr (kCodes == kCodesInt8) {
            float top = __int_as_float(s.top) * inv;
            if (!in_range(__int_as_float(s.top))) {
                RowSums y = {0.0f, 0.0f, 0};
#pragma unroll
                for (int k = 0; k < kV; ++k)
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int b = k * kLanes + tid < a.vecs
                                          ? abs_bits(t[k][i] * inv * w[k][i])
                                          : 0;
                        y.top = y.top > b ? y.top : b;
                    }
                top = __int_as_float(team_reduce<kWaves, false, true>(y, tops).top);
            }
            scale = top / 127.0f;
            recip = 1.0f / scale;
            plain = plain_scale(scale);
            if (tid == 0)
                a.scales[row] = scale;
        }
#pragma unroll
        for (int k = 0; k < kV; ++k) {
            const int v = k * kLanes + tid;
            if (v >= a.vecs)
                continue;
            bf16x8 o;
            int top = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                t[k][i] = t[k][i] * inv * w[k][i];
                o[i] = (__bf16)t[k][i];
                if (kCodes == kCodesE4m3) {
                    const int b = abs_bits(t[k][i]);
                    top = top > b ? top : b;
                }
            }
            if (a.out)
                *reinterpret_cast<bf16x8 *>(a.out + (at + v) * 16) = o;
            if constexpr (kCodes == kCodesE4m3) {   // a block is 16 lanes' vectors
                scale = __int_as_float(group_top<16>(top)) / 448.0f;
                recip = 1.0f / scale;
                plain = plain_scale(scale);
                if ((tid & 15) == 0)
                    a.scales[(at + v) / 16] = scale;
            }
            if constexpr (kCodes != kCodesNone)
                *reinterpret_cast<uint2 *>(a.codes + (at + v) * 8) =
                    uint2{four_codes<kCodes>(t[k], scale, recip, plain),
                          four_codes<kCodes>(t[k] + 4, scale, recip, plain)};
        }
    }
}

// With q = 1 / rms(s), n = s q and g = dy w:  dx = q (g - n mean(g n)) + dsum, and the
// team's share of dw = sum dy n over its rows.  Rows are dealt to the teams in
// turn, and the teams' shares are added in order (k_norm_weight_grad), so nothing
// varies.  (8192 x 7168 with dsum, 470 MB: 94 us, 5.0 TB/s, and 5 for the shares; with the
// weight loaded for every row, and so every row's loads waited for, 14 us more.)  Rows of
// more than 16384 elements spill: 2048 x 32768 157 us, 153 without the second sum below.
template <int kWaves, int kV>
__global__ __launch_bounds__(team_threads(kWaves)) void k_rms_norm_grad(const NormArgs a)
{
    constexpr int kTeams = team_threads(kWaves) / (kWaves * 64), kLanes = kWaves * 64;
    __shared__ RowSums parts[2][kWaves], again[kWaves], crosses[kWaves];
    const int tid = threadIdx.x & (kLanes - 1), team = threadIdx.x / kLanes;
    // Where registers allow, a row's loads are in flight while the row before it is worked
    // on, and the weight stays in registers: its loads would wait for theirs.
    constexpr bool kAhead = kWaves < 16;
    float held[kAhead ? kV : 1][8] = {}, dw[kV][8] = {};
    if constexpr (kAhead) {
#pragma unroll
        for (int k = 0; k < kV; ++k)
            if (k * kLanes + tid < a.vecs)
                weight_at(a, k * kLanes + tid, held[k]);
    }
    const auto weight = [&](int k, float(&w)[8]) {
        if constexpr (kAhead) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                w[i] = held[k][i];
        } else {
            weight_at(a, k * kLanes + tid, w);
        }
    };
    bf16x8 s[kV], dy[kV], ds[kV], next_s[kV], next_dy[kV], next_ds[kV];
    const auto load = [&](int64_t row, bf16x8(&to_s)[kV], bf16x8(&to_dy)[kV], bf16x8(&to_ds)[kV]) {
        const size_t at = (size_t)row * a.vecs;
#pragma unroll
        for (int k = 0; k < kV; ++k) {
            const int v = k * kLanes + tid;
            to_s[k] = to_dy[k] = to_ds[k] = bf16x8{};
            if (row < a.rows && v < a.vecs) {
                to_s[k] = *reinterpret_cast<const bf16x8 *>(a.input + (at + v) * 16);
                to_dy[k] = *reinterpret_cast<const bf16x8 *>(a.grad_out + (at + v) * 16);
                if (a.grad_sum)
                    to_ds[k] = *reinterpret_cast<const bf16x8 *>(a.grad_sum + (at + v) * 16);
            }
        }
    };
    int turn = 0;
    const int64_t first = (int64_t)blockIdx.x * kTeams + team, stride = (int64_t)gridDim.x * kTeams;
    if (kAhead)
        load(first, next_s, next_dy, next_ds);
    for (int64_t row = first; row < a.rows; row += stride, turn ^= 1) {
        const size_t at = (size_t)row * a.vecs;
        if constexpr (kAhead) {
#pragma unroll
            for (int k = 0; k < kV; ++k) {
                s[k] = next_s[k];
                dy[k] = next_dy[k];
                ds[k] = next_ds[k];
            }
            load(row + stride, next_s, next_dy, next_ds);
        } else {
            load(row, s, dy, ds);
        }
        RowSums sums = {0.0f, 0.0f, 0};
#pragma unroll
        for (int k = 0; k < kV; ++k) {
            const int v = k * kLanes + tid;
            if (v >= a.vecs)
                continue;
            float w[8];
            weight(k, w);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float x = (float)s[k][i];
                sums.squares = __builtin_fmaf(x, x, sums.squares);
                sums.cross = __builtin_fmaf((float)dy[k][i] * w[i], x, sums.cross);
            }
        }
        sums = team_reduce<kWaves, true, false>(sums, parts[turn]);
        const float inv = inverse_rms(a, sums.squares, again, [&](float c) {
            float sum = 0.0f;
#pragma unroll
            for (int k = 0; k < kV; ++k)
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float x = (float)s[k][i] * c;
                    sum = __builtin_fmaf(x, x, sum);
                }
            return sum;
        });
        float mean = sums.cross * inv / a.features;   // of g n
        // Products dy w x beyond fp32, or of an x so small that they may be below it: from
        // n instead, which is of the usual size, before the sum.
        if (!(fabsf(mean) < __builtin_inff()) || inv > 0x1p20f) {
            RowSums c = {0.0f, 0.0f, 0};
            const float part = 1.0f / a.features;
#pragma unroll
            for (int k = 0; k < kV; ++k) {
                if (k * kLanes + tid >= a.vecs)
                    continue;
                float w[8];
                weight(k, w);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    c.cross = __builtin_fmaf((float)dy[k][i] * w[i],
                                             (float)s[k][i] * inv * part, c.cross);
            }
            mean = team_reduce<kWaves, true, false>(c, crosses).cross;
        }
#pragma unroll
        for (int k = 0; k < kV; ++k) {
            const int v = k * kLanes + tid;
            if (v >= a.vecs)
                continue;
            float w[8];
            weight(k, w);
            bf16x8 o;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float n = (float)s[k][i] * inv, d = (float)dy[k][i];
                dw[k][i] = __builtin_fmaf(d, n, dw[k][i]);
                float g = inv * __builtin_fmaf(-n, mean, d * w[i]);
                if (a.grad_sum)
                    g += (float)ds[k][i];
                o[i] = (__bf16)g;
            }
            *reinterpret_cast<bf16x8 *>(a.grad_input + (at + v) * 16) = o;
        }
    }
    if (!a.partial)
        return;
    f32x4 *mine = reinterpret_cast<f32x4 *>(a.partial) + (size_t)first * a.vecs * 2;
#pragma unroll
    for (int k = 0; k < kV; ++k) {
        const int v = k * kLanes + tid;
        if (v < a.vecs) {
            mine[v * 2] = f32x4{dw[k][0], dw[k][1], dw[k][2], dw[k][3]};
            mine[v * 2 + 1] = f32x4{dw[k][4], dw[k][5], dw[k][6], dw[k][7]};
        }
    }
}

struct NormWeightGradArgs {
    int32_t teams, quads;    // rows of partial; 16-byte vectors of a row
    const float *partial;
    float *grad_weight;
};

constexpr int kWeightGradQuads = 8, kWeightGradLanes = 64;

// dw: the teams' shares added column by column, 128 bytes of 64 shares at a time.
__global__ __launch_bounds__(kWeightGradQuads *kWeightGradLanes) void k_norm_weight_grad(
    const NormWeightGradArgs a)
{
    __shared__ f32x4 part[kWeightGradLanes][kWeightGradQuads];
    const int c = threadIdx.x % kWeightGradQuads, lane = threadIdx.x / kWeightGradQuads;
    const int quad = blockIdx.x * kWeightGradQuads + c;
    const f32x4 *p = reinterpret_cast<const f32x4 *>(a.partial) + quad;
    f32x4 s = {0, 0, 0, 0};
    if (quad < a.quads) {
#pragma unroll 4
        for (int r = lane; r < a.teams; r += kWeightGradLanes)
            s += p[(size_t)r * a.quads];
    }
    part[lane][c] = s;
    __syncthreads();
    if (lane != 0 || quad >= a.quads)
        return;
    for (int r = 1; r < kWeightGradLanes; ++r)
        s += part[r][c];
    reinterpret_cast<f32x4 *>(a.grad_weight)[quad] = s;
}

// ---------------------------------------------------------------------------
// Rows in 8 bits
// ---------------------------------------------------------------------------

struct QuantArgs {
    int32_t rows, experts, vecs;   // vecs: of 16 elements
    const int32_t *expert_off;     // or NULL: all rows
    const uint8_t *input;
    uint8_t *codes;
    float *scales;
};

__device__ inline void row_range(const QuantArgs &a, int64_t &r0, int64_t &r1)
{
    r0 = a.expert_off ? clamp_row(a.expert_off, 0, a.rows) : 0;
    r1 = a.expert_off ? clamp_row(a.expert_off, a.experts, a.rows) : a.rows;
}

// 16 elements of bf16 from 32 bytes; the largest pattern of their absolute values
// (a bf16's above 16 zero bits)
struct Sixteen {
    u32x4 w[2];
    __device__ inline void load(const uint8_t *p)
    {
        w[0] = reinterpret_cast<const u32x4 *>(p)[0];
        w[1] = reinterpret_cast<const u32x4 *>(p)[1];
    }
    __device__ inline int top() const
    {
        typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
        u16x2 m = {0, 0};
#pragma unroll
        for (int i = 0; i < 8; ++i)
            m = __builtin_elementwise_max(
                m, __builtin_bit_cast(u16x2, w[i / 4][i % 4] & 0x7fff7fffu));
        return (int)(m[0] > m[1] ? m[0] : m[1]) << 16;
    }
    template <int kCodes>
    __device__ inline u32x4 codes(float s, float r, bool plain) const
    {
        u32x4 c;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t lo = w[i / 2][i % 2 * 2], hi = w[i / 2][i % 2 * 2 + 1];
            const float v[4] = {__uint_as_float(lo << 16), __uint_as_float(lo & 0xffff0000u),
                                __uint_as_float(hi << 16), __uint_as_float(hi & 0xffff0000u)};
            c[i] = four_codes<kCodes>(v, s, r, plain);
        }
        return c;
    }
};

constexpr int kQuantThreads = 256;

// e4m3: eight lanes hold a block of 128 columns, whatever row it is of.  (32768 x 2048,
// 203 MB: 33 us, 6.2 TB/s.)
__global__ __launch_bounds__(kQuantThreads) void k_quantize_e4m3(const QuantArgs a)
{
    int64_t r0, r1;
    row_range(a, r0, r1);
    const int64_t end = r1 * a.vecs;
    for (int64_t v = r0 * a.vecs + (int64_t)blockIdx.x * kQuantThreads + threadIdx.x; v < end;
         v += (int64_t)gridDim.x * kQuantThreads) {
        Sixteen x;
        x.load(a.input + v * 32);
        int m = x.top();
        int b = dpp_i<kXor1>(m);
        m = m > b ? m : b;
        b = dpp_i<kXor2>(m);
        m = m > b ? m : b;
        b = dpp_i<kMirror8>(m);
        m = m > b ? m : b;
        const float s = __int_as_float(m) / 448.0f;
        *reinterpret_cast<u32x4 *>(a.codes + v * 16) =
            x.codes<kCodesE4m3>(s, 1.0f / s, plain_scale(s));
        if ((threadIdx.x & 7) == 0)
            a.scales[v / 8] = s;
    }
}

// int8: a team per row.  (1000 x 2048: 5.4 us, 4096 x 7168 17; 32768 x 2048, where half the
// lanes of a team have nothing to load, 81.)
template <int kWaves, int kV>
__global__ __launch_bounds__(team_threads(kWaves)) void k_quantize_int8(const QuantArgs a)
{
    constexpr int kTeams = team_threads(kWaves) / (kWaves * 64), kLanes = kWaves * 64;
    __shared__ int parts[2][kWaves];
    const int tid = threadIdx.x & (kLanes - 1), team = threadIdx.x / kLanes;
    int64_t r0, r1;
    row_range(a, r0, r1);
    int turn = 0;
    for (int64_t row = r0 + (int64_t)blockIdx.x * kTeams + team; row < r1;
         row += (int64_t)gridDim.x * kTeams, turn ^= 1) {
        const size_t at = (size_t)row * a.vecs;
        Sixteen x[kV];
        int top = 0;
#pragma unroll
        for (int k = 0; k < kV; ++k) {
            x[k].w[0] = x[k].w[1] = u32x4{0, 0, 0, 0};
            if (k * kLanes + tid < a.vecs)
                x[k].load(a.input + (at + k * kLanes + tid) * 32);
        }
#pragma unroll
        for (int k = 0; k < kV; ++k) {
            const int m = x[k].top();
            top = top > m ? top : m;
        }
        top = group_top<64>(top);
        if constexpr (kWaves > 1) {
            if ((threadIdx.x & 63) == 0)
                parts[turn][threadIdx.x / 64] = top;
            __syncthreads();
#pragma unroll
            for (int w = 0; w < kWaves; ++w)
                top = top > parts[turn][w] ? top : parts[turn][w];
        }
        const float s = __int_as_float(top) / 127.0f, r = 1.0f / s;
        const bool plain = plain_scale(s);
        if (tid == 0)
            a.scales[row] = s;
#pragma unroll
        for (int k = 0; k < kV; ++k)
            if (k * kLanes + tid < a.vecs)
                *reinterpret_cast<u32x4 *>(a.codes + (at + k * kLanes + tid) * 16) =
                    x[k].template codes<kCodesInt8>(s, r, plain);
    }
}

}  // namespace epdc_layer
