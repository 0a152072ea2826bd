// layer_few.hpp -- gfx950 kernels of a layer for few tokens: dispatch, the experts'
// two products and combine as two launches,
//   k_few_up:    h[t, k]  = act(x[t] W1[e]^T + b1[e]),      e = indices[t, k]
//   k_few_down:  y[t]     = sum_k w[t, k] (h[t, k] W2[e]^T + b2[e])
//
// The weights of the experts that are asked for are the traffic, read once for every
// unit of up to 4, 16 or 32 rows of an expert, in whole 128-byte lines, past the caches if
// rows of weight are whole lines and through them if not, and turned through LDS into
// fragments, as in k_product_stream; nothing is routed in memory.  Every block finds the experts' rows
// from the indices itself: at most 1024, a token set per expert in one 64-bit
// word.  8-bit weights are widened to bf16, which holds them exactly, so the
// activations stay bf16.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "layer_gate.hpp"
#include "layer_product.hpp"

namespace epdc_layer {

constexpr int kFewTokens = 64, kFewPairs = 1024;
// Registers for loads in flight, of the 128 that a wave has where a SIMD holds four.
constexpr int kFewSlotRegs = 62;

struct FewArgs {
    int32_t tokens, topk, experts, first_expert;
    int32_t hidden, inner, act;
    uint32_t per_token;   // 2^16 / topk, rounded up past it: p * per_token >> 16 = p / topk
    const uint8_t *x;
    const float *weights;
    const int32_t *indices;
    const uint8_t *w1, *w2;
    const float *s1, *s2, *b1, *b2;
    uint8_t *h;    // [tokens * topk, inner] bf16: written at the first of a token's pairs
                   // with an expert
    uint8_t *out;  // [tokens, hidden] bf16
    // blocks that share the steps of a column tile of y, the sums they leave
    // [tiles][splits][tokens][16] and their tickets [tiles] (more than one of them)
    int32_t splits;
    float *partial;
    uint32_t *ticket;
};

__host__ __device__ inline uint32_t few_per_token(int topk) { return 65536u / topk + 1; }
__device__ inline int few_token(const FewArgs &a, int pair)
{
    return (int)((uint32_t)pair * a.per_token >> 16);   // exact for pairs below 1024
}

// The rows of the experts (one per token and expert, experts and tokens ascending), in
// LDS, and the units of work they make: up to 4, 16 or 32 rows of an expert.
struct FewRouting {
    uint64_t tokens[kMaxExperts];   // that ask for an expert
    uint16_t start[kMaxExperts];    // first row of an expert
    uint16_t row[kFewPairs];        // the token, above the first of its pairs (10 bits)
    uint32_t unit[kMaxExperts + kFewPairs / 4];   // expert, first row, rows
    int units, rows, pairs;
};

struct FewUnit {
    int expert, first, rows;
};

__device__ inline FewUnit few_unit(const FewRouting &r, int n)
{
    const uint32_t u = (uint32_t)uniform((int)r.unit[n]);
    return {(int)(u & 0x3ff), (int)(u >> 10 & 0x7ff), (int)(u >> 21)};
}

// Sum over the lanes up to this one; eight adds without LDS.
__device__ inline int sum_upto(int v)
{
    v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, true);   // row_shr 1, 2, 4, 8
    v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, true);
    v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, true);
    v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, true);
    v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false);  // row 0 to 1, 2 to 3
    v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false);  // rows 0, 1 to 2, 3
    return v;
}

// Fills the routing, and `weight` of a row unless it is NULL, and ends with a barrier;
// returns the number of units.
template <int kThreads, int kUnitRows>
__device__ inline int few_routing(const FewArgs &a, FewRouting &r, float *weight)
{
    constexpr int kEach = kFewPairs / kThreads;
    const int tid = threadIdx.x, lane = tid & 63, pairs = a.tokens * a.topk;
    uint32_t expert[kEach];
    float w[kEach];
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        const int p = i * kThreads + tid;
        expert[i] = ~0u;
        w[i] = 1.0f;
        if (p < pairs) {
            expert[i] = (uint32_t)a.indices[p] - (uint32_t)a.first_expert;
            if (weight && a.weights)
                w[i] = a.weights[p];
        }
    }
    for (int e = tid; e < a.experts; e += kThreads)
        r.tokens[e] = 0;
    if (tid == 0)
        r.pairs = 0;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        if (i * kThreads >= pairs)
            break;
        const int p = i * kThreads + tid;
        const bool in = expert[i] < (uint32_t)a.experts;
        if (in)
            atomicOr(reinterpret_cast<unsigned long long *>(&r.tokens[expert[i]]),
                     1ull << few_token(a, p));
        const int have = __popcll(__ballot(in));
        if (lane == 0 && have)
            atomicAdd(&r.pairs, have);
    }
    __syncthreads();
    if (tid < 64) {
        int rows = 0, units = 0;
        for (int e0 = 0; e0 < a.experts; e0 += 64) {
            const int e = e0 + lane, n = e < a.experts ? __popcll(r.tokens[e]) : 0;
            const int u = (n + kUnitRows - 1) / kUnitRows;
            const int upto = sum_upto(n | u << 16);   // both at once: at most 1024 of each
            const int first = rows + (upto & 0xffff) - n, at = units + (upto >> 16) - u;
            if (e < a.experts)
                r.start[e] = (uint16_t)first;
            for (int i = 0; i < u; ++i) {
                const int left = n - i * kUnitRows;
                r.unit[at + i] = (uint32_t)e | (uint32_t)(first + i * kUnitRows) << 10 |
                                 (uint32_t)(left < kUnitRows ? left : kUnitRows) << 21;
            }
            const int all = __builtin_amdgcn_readlane(upto, 63);
            rows += all & 0xffff;
            units += all >> 16;
        }
        if (lane == 0) {
            r.units = units;
            r.rows = rows;
        }
    }
    __syncthreads();
    const bool repeats = r.rows != r.pairs;   // a token that lists an expert twice
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        const int p = i * kThreads + tid, e = (int)expert[i];
        if (expert[i] >= (uint32_t)a.experts)
            continue;
        const int t = few_token(a, p);
        bool first = true;
        if (repeats)
            for (int k = 0; k < a.topk; ++k) {
                const int q = t * a.topk + k;
                if (q == p || a.indices[q] != e + a.first_expert)
                    continue;
                first &= q > p;
                w[i] += a.weights ? a.weights[q] : 1.0f;
            }
        if (first) {
            const int row = r.start[e] + __popcll(r.tokens[e] & ((1ull << t) - 1));
            r.row[row] = (uint16_t)(t << 10 | p);
            if (weight)
                weight[row] = w[i];
        }
    }
    __syncthreads();
    return uniform(r.units);
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

// Rows of a unit beside 8-bit weights whose part of a step one load of a wave holds.
constexpr int kFewLineRows = 4;

// Registers of a step's loads, and the waves of a SIMD: four where two steps' loads fit
// into theirs, else two.
constexpr int few_slot_regs(int type, int rows, int q)
{
    return q * 8 + (rows < 16 ? 4 : (rows + 15) / 16 * 16 / element_bytes(type)) +
           (type != kTypeBf16 ? 1 : 0);
}
constexpr int few_waves(int type, int rows, int q)
{
    return 2 * few_slot_regs(type, rows, q) <= kFewSlotRegs + 4 ? 4 : 2;
}

// A wave's share of rows x columns: kRows rows of bf16 (x or h) by 16 columns of kQ
// weights, a step of 128 weight bytes at a time.  The loads of kDepth steps are in
// flight: a step's slot is loaded again as soon as it has been multiplied.  Loads past
// the end of a contraction, or of a wave's steps, give zeros without traffic, so that
// every step runs the same instructions and waits for its own loads only.
//
// Units of four rows take theirs as the weights, a step's part of all of them by one
// load, and turn them through LDS; 16 or 32 rows come as fragments.  A load instruction
// of 16 bytes a lane keeps a CU's address unit for 16 cycles whether its lanes are
// active or not: with fragments for 32 rows beside every 2 KiB of 8-bit weights (ten
// instructions) 32 tokens through 4 of 64 int8 experts of 2048 x 4096 streamed them at
// 4.2 TB/s, however many waves or loads in flight.  (Beside bf16, 64 features a step,
// eight rows in a load gained nothing on fragments of 16.)
//
// kWhole: every row of the weight begins with a line.  Rows that do not are read in whole
// lines all the same, each once, and a step's window of the contraction lags so far behind its
// line that every row has it: with a lag of 7, window s is the row's 16-byte chunks 8 s - 7
// ... 8 s, of which line s holds those that a wave's LDS did not have from line s - 1.  A row's
// place in its first line is the same eight rows on, as chunks are eight to a line.  The lines
// go through the caches, since two rows share one.  (us of both launches, loaded as 128
// bytes of every row that lie in two lines, and so: one token, 8 bf16 experts of 7176 x
// 2056 162, 135; 60 tokens, 64 of 4104 x 1416 686, 501; 37 tokens, 32 int8 of 2064 x 1040 60,
// 52.  Past the caches the last takes 59.)
template <int kType, int kRows, int kQ, bool kWhole>
struct FewProduct {
    typedef FewWeight<kType> Weight;
    static constexpr int kFrags = Weight::kFrags;
    static constexpr int kStep = kStepBytes / element_bytes(kType);  // elements
    static constexpr int kMI = (kRows + 15) / 16;
    static constexpr bool kLine = kRows < 16;
    static_assert(!kLine || (kRows == kFewLineRows && kType != kTypeBf16), "in one load");
    static constexpr int kXLoads = kLine ? 1 : kMI * 2 * kFrags;
    static constexpr int kChunk = 16 / element_bytes(kType);  // elements
    static constexpr int kTurns = kWhole ? 1 : kQ;
    static constexpr int kTurnBytes = kTurns * 16 * kStepBytes + (kLine ? 1024 : 0);  // of a wave
    static constexpr bool kBeside = kType != kTypeBf16;
    static constexpr int kSlotRegs = few_slot_regs(kType, kRows, kQ);
    static constexpr int kFit = 4 / few_waves(kType, kRows, kQ) * kFewSlotRegs / kSlotRegs;
    static constexpr int kDepth = kFit < 2 ? 2 : kFit < 4 ? kFit : 4;
    static_assert(kSlotRegs == kQ * 8 + kXLoads * 4 + (kBeside ? 1 : 0), "registers of a slot");

    struct Slot {
        i32x4 w[kQ][2], x[kXLoads];
        int beside;   // scales and biases (below)
    };

    int contract, steps, lane;
    int chunk;   // of the row that this lane loads in step 0
    int lag;     // of windows behind their lines, in chunks: the last place of a row in a line
    uint8_t *turn;
    __amdgpu_buffer_rsrc_t q, p;
    // 8-bit weights: what belongs to the 16 columns of each part comes with every step, a
    // word a lane, as a load at a unit's end would wait for all loads in flight.  Lanes 0
    // to 15 and 16 to 31: int8 the channels' scales of part 0 and 1, e4m3 the scale of
    // the step's block, 32 to 47 and 48 to 63: the biases.
    const float *beside_at;
    int beside;          // of the last step
    uint32_t qoff[kQ][2];
    uint32_t off[kMI];   // of this lane's row and contraction part in p, or kNowhere
    const float *nowhere;
    f32x4 acc[kMI][kQ];

    __device__ inline void init(const uint8_t *weight, int contraction, int l, uint8_t *t,
                                const uint8_t *rows, uint32_t bytes, const void *some_word)
    {
        nowhere = static_cast<const float *>(some_word);
        contract = contraction;
        lane = l;
        turn = t;
        chunk = lane & 7;
        lag = 0;
        if constexpr (!kWhole) {
            const int at = (uint32_t)(uintptr_t)weight / 16 & 7, row = contract / kChunk;
            chunk -= (at + (lane >> 3) * row) & 7;
            lag = at || row & 1 ? 7 : row & 2 ? 6 : 4;
            // chunks before a row's first meet rows of zeros, and so may not be just anything
#pragma unroll
            for (int i = 0; i < kTurns * 2; ++i)
                reinterpret_cast<i32x4 *>(turn)[i * kWave + lane] = i32x4{0, 0, 0, 0};
        }
        steps = (contraction + lag * kChunk + kStep - 1) / kStep;
        p = buffer_at(rows, bytes);
        clear();
    }
    __device__ inline void clear()
    {
#pragma unroll
        for (int i = 0; i < kMI; ++i)
#pragma unroll
            for (int j = 0; j < kQ; ++j)
                acc[i][j] = f32x4{0, 0, 0, 0};
    }
    // loads from here on are of columns c0 ... c0 + 15 of each of the kQ parts of expert e's
    // weight, `cols` columns (rows in memory) a part; row(i): the row of p that is row i of
    // the unit, or -1
    template <typename F>
    __device__ inline void expert(const uint8_t *w, const float *s, const float *bias, int e,
                                  int c0, int cols, F &&row)
    {
        const uint32_t bytes = (uint32_t)kQ * cols * contract * element_bytes(kType);
        q = buffer_at(w + (size_t)e * bytes, bytes);
#pragma unroll
        for (int j = 0; j < kQ; ++j)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                int c = c0 + h * 8 + (lane >> 3);
                c = (c < cols ? c : c - 8) + j * cols;
                qoff[j][h] = (uint32_t)c * contract * element_bytes(kType) + chunk * 16;
            }
#pragma unroll
        for (int i = 0; i < kMI; ++i) {
            const int r = row(kLine ? lane / (64 / kRows) : i * 16 + (lane & 15));
            const int part = kLine ? lane % (64 / kRows) * 16 : (lane >> 4) * (kFrags * 16);
            off[i] = r < 0 ? kNowhere : (uint32_t)r * contract * 2 + part;
        }
        if constexpr (!kBeside)
            return;
        // where there is nothing to load, a word of the indices stands in
        const int part = lane >> 4 & 1 & (kQ - 1), c = c0 + (lane & 15);
        const size_t col = (size_t)e * kQ * cols + part * cols + (c < cols ? c : cols - 1);
        beside_at = nowhere;
        if (lane >= 32) {
            if (bias)
                beside_at = bias + col;
        } else if constexpr (kType == kTypeInt8) {
            beside_at = s + col;
        } else if constexpr (kType == kTypeE4m3) {
            beside_at = s + ((size_t)e * ((kQ * cols + 127) / 128) + (part * cols + c0) / 128) *
                                (contract / 128);
        }
    }
    __device__ inline void load(Slot &to, int s)
    {
        const int begin = s * kStep - lag * kChunk, left = contract - begin;
        const uint32_t at = (uint32_t)s * kStepBytes, xat = (uint32_t)begin * 2;
        const bool in = (uint32_t)(s * 8 + chunk) < (uint32_t)contract / kChunk;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int j = 0; j < kQ; ++j)
                to.w[j][h] = __builtin_bit_cast(
                    i32x4, __builtin_amdgcn_raw_buffer_load_b128(
                               q, in ? qoff[j][h] + at : kNowhere, 0, kWhole ? 2 /* nt */ : 0));
#pragma unroll
        for (int n = 0; n < kXLoads; ++n) {
            // fragment f of half h of row tile i
            const int i = n / (2 * kFrags), h = n / kFrags % 2, f = n % kFrags;
            const int el = kLine ? 0 : h * (kStep / 2) + f * 8;
            const int lane_el = kLine ? lane % (64 / kRows) * 8 : (lane >> 4) * (8 * kFrags);
            to.x[n] = __builtin_bit_cast(
                i32x4, __builtin_amdgcn_raw_buffer_load_b128(
                           p,
                           el + lane_el < left && (kWhole || el + lane_el + begin >= 0)
                               ? off[i] + xat + el * 2
                               : kNowhere,
                           0, 0));
        }
        if constexpr (kBeside) {
            int word = 0;
            if constexpr (kType == kTypeE4m3)
                word = lane < 32 ? (s < steps ? s : steps - 1) : 0;
            to.beside = __float_as_int(beside_at[word]);
        }
    }
    // this lane's four columns of group g of the lanes
    __device__ inline f32x4 columns(int g) const
    {
        f32x4 v;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            v[i] = __int_as_float(__shfl(beside, g * 16 + (lane >> 4) * 4 + i, 64));
        return v;
    }
    // and of part j's biases, of expert e's columns from c0 on
    __device__ inline f32x4 biases(const float *bias, int e, int j, int c0, int cols) const
    {
        if constexpr (kBeside)
            return columns(2 + j);
        f32x4 v;
        const float *at = bias + (size_t)e * kQ * cols + j * cols;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int c = c0 + (lane >> 4) * 4 + i;
            v[i] = at[c < cols ? c : cols - 1];
        }
        return v;
    }
    // lines of 8 + 8 columns to fragments of 16; lanes read what others wrote, in
    // the order in which the wave's LDS accesses run
    __device__ inline void turned(i32x4 (&w)[2], int part)
    {
        typedef StraightTile<16, 1, false> Turn;
        uint8_t *const at = turn + (kWhole ? 0 : part) * 16 * kStepBytes;
        const i32x4 line[2] = {w[0], w[1]};
        const auto write = [&] {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int r = h * 8 + (lane >> 3);
                *reinterpret_cast<i32x4 *>(at + r * kStepBytes +
                                           (((chunk + lag) & 7) ^ (r & 7)) * 16) = line[h];
            }
        };
        const auto sync = [] {
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
        };
        if (kWhole || chunk <= 7 - lag)
            write();
        sync();
#pragma unroll
        for (int h = 0; h < 2; ++h)
            w[h] = Turn::frag(at, 0, h, lane);
        sync();
        if constexpr (!kWhole) {   // the next window's
            if (chunk > 7 - lag)
                write();
        }
    }
    // rows taken as a line to fragments of 16, of which kRows are its own
    __device__ inline void turned_rows(i32x4 line, i32x4 (&x)[2][kFrags])
    {
        constexpr int kChunks = 64 / kRows;   // of 16 bytes, in a row's part of a step
        uint8_t *at = turn + kTurns * 16 * kStepBytes;
        const int to = lane / kChunks, r = lane & (kRows - 1);
        *reinterpret_cast<i32x4 *>(at + to * (kChunks * 16) +
                                   ((lane % kChunks) ^ (to & 7)) * 16) = line;
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int f = 0; f < kFrags; ++f) {
                const int c = h * (kChunks / 2) + (lane >> 4) * kFrags + f;
                x[h][f] = *reinterpret_cast<const i32x4 *>(at + r * (kChunks * 16) +
                                                           (c ^ (r & 7)) * 16);
            }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
    }
    __device__ inline void multiply(Slot &of)
    {
        i32x4 x[kMI][2][kFrags];
        if constexpr (kLine) {
            turned_rows(of.x[0], x[0]);
        } else {
#pragma unroll
            for (int n = 0; n < kXLoads; ++n)
                x[n / (2 * kFrags)][n / kFrags % 2][n % kFrags] = of.x[n];
        }
#pragma unroll
        for (int j = 0; j < kQ; ++j)
            turned(of.w[j], j);
#pragma unroll
        for (int j = 0; j < kQ; ++j) {
            float scale = 1.0f;
            if constexpr (kType == kTypeE4m3)
                scale = __int_as_float(__builtin_amdgcn_readlane(of.beside, j * 16));
            i32x4 f[2][kFrags];
            Weight::widen(of.w[j][0], f[0]);
            Weight::widen(of.w[j][1], f[1]);
#pragma unroll
            for (int i = 0; i < kMI; ++i) {
                f32x4 d = kType == kTypeE4m3 ? f32x4{0, 0, 0, 0} : acc[i][j];
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int k = 0; k < kFrags; ++k)
                        d = mfma_bf16(f[h][k], x[i][h][k], d);
                if constexpr (kType == kTypeE4m3) {
#pragma unroll
                    for (int v = 0; v < 4; ++v)
                        acc[i][j][v] = __builtin_fmaf(d[v], scale, acc[i][j][v]);
                } else {
                    acc[i][j] = d;
                }
            }
        }
        // What the slot gives is taken before it is loaded again: else parts of it go to
        // other registers, whose copies at the end of the loop wait for every load.
        if constexpr (kBeside) {
            beside = of.beside;
            asm volatile("" : "+v"(beside));
        }
        if constexpr (kType == kTypeE4m3) {
#pragma unroll
            for (int i = 0; i < kMI; ++i)
#pragma unroll
                for (int j = 0; j < kQ; ++j)
                    asm volatile("" : "+v"(acc[i][j]));
        }
    }
};

constexpr int kFewUpWaves = 4, kFewDownWaves = 8;
constexpr int kFewShort = 4;        // steps of a wave
constexpr int kFewMostSplits = 8;
constexpr int kFewUpBlocks = 1024;  // four to a CU

// h is rounded to bf16, the type in which the matrix cores take it and in which
// expert_product leaves it; that costs the result as much again as its own rounding.
// A tile: 16 columns of h (gated: 16 gate and 16 up) for one unit of rows; a block's
// waves take the contraction's steps in turn (in runs, each behind the line before its
// first, where rows are not whole lines) and add up through LDS.  Blocks stay for
// tile after tile, the next one's loads in flight while a tile ends.  (One token through
// 8 of 64 bf16 experts of 7168 x 2 x 2048, 470 MB: 70 us, 6.7 TB/s; 16 tokens through 82 of
// 128 e4m3 experts of 4096 x 2 x 2048, 1.38 GB: 221 us, 6.2 TB/s; 8 pairs of 256 x 2 x 128:
// 5.0 us, of which the routing takes 1.2 and a launch without it 1.7.)
template <int kType, int kRows, bool kGated, bool kWhole>
__global__ __launch_bounds__(kFewUpWaves *kWave, few_waves(kType, kRows, kGated ? 2 : 1)) void
k_few_up(const FewArgs a)
{
    constexpr int kQ = kGated ? 2 : 1;
    typedef FewProduct<kType, kRows, kQ, kWhole> Product;
    constexpr int kMI = Product::kMI;
    __shared__ FewRouting routing;
    __shared__ __align__(16) f32x4 parts[kFewUpWaves][kMI * kQ][kWave];
    __shared__ __align__(16) uint8_t turn[kFewUpWaves][Product::kTurnBytes];
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x / kWave);
    const int units = few_routing<kFewUpWaves * kWave, kRows>(a, routing, nullptr);
    const int col_tiles = (a.inner + 15) / 16, tiles = units * col_tiles;
    int tile = blockIdx.x;
    if (tile == 0 && a.splits > 1)   // for the launch behind this one
        for (int i = threadIdx.x; i < (a.hidden + 15) / 16; i += kFewUpWaves * kWave)
            a.ticket[i] = 0;
    if (tile >= tiles)
        return;
    Product m;
    m.init(a.w1, a.hidden, lane, turn[wave], a.x, (uint32_t)a.tokens * a.hidden * 2, a.indices);
    // every wave runs as many steps of a tile; some of them may lie past the end
    const int share = (m.steps + kFewUpWaves - 1) / kFewUpWaves, per = share + !kWhole;
    const int count = (tiles - tile + (int)gridDim.x - 1) / (int)gridDim.x * per;
    int load_tile = tile, load_step = 0, loaded = 0;
    const auto enter = [&] {
        const int n = load_tile / col_tiles, c0 = (load_tile - n * col_tiles) * 16;
        const FewUnit u = few_unit(routing, n);
        m.expert(a.w1, a.s1, a.b1, u.expert, c0, a.inner, [&](int r) {
            return r < u.rows ? routing.row[u.first + r] >> 10 : -1;
        });
    };
    const auto next_load = [&](typename Product::Slot &to) {
        const int s = kWhole ? load_step * kFewUpWaves + wave : wave * share - 1 + load_step;
        m.load(to, loaded < count ? s : m.steps);
        ++loaded;
        if (++load_step == per && loaded < count) {
            load_step = 0;
            load_tile += gridDim.x;
            enter();
        }
    };
    const auto leave = [&] {
        const int n = tile / col_tiles, c0 = (tile - n * col_tiles) * 16;
        const FewUnit u = few_unit(routing, n);
        __syncthreads();   // the last tile's parts have been read
#pragma unroll
        for (int i = 0; i < kMI; ++i)
#pragma unroll
            for (int q = 0; q < kQ; ++q)
                parts[wave][i * kQ + q][lane] = m.acc[i][q];
        m.clear();
        __syncthreads();
        // wave i finishes row block i, adding the waves' parts in order
        if (wave < kMI) {
            f32x4 z[2] = {f32x4{0, 0, 0, 0}, f32x4{0, 0, 0, 0}};
#pragma unroll
            for (int q = 0; q < kQ; ++q) {
#pragma unroll
                for (int w = 0; w < kFewUpWaves; ++w)
                    z[q] += parts[w][wave * kQ + q][lane];
                if constexpr (kType == kTypeInt8)
                    z[q] *= m.columns(q);
                if (a.b1)
                    z[q] += m.biases(a.b1, u.expert, q, c0, a.inner);
            }
            f32x4 y;
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                y[v] = act_one(a.act, z[0][v]);
                if (kGated)
                    y[v] *= z[1][v];
            }
            const int r = wave * 16 + (lane & 15), c = c0 + (lane >> 4) * 4;
            if (r < u.rows && c < a.inner)
                *reinterpret_cast<bf16x4 *>(
                    a.h + ((size_t)(routing.row[u.first + r] & 0x3ff) * a.inner + c) * 2) =
                    to_bf16(y);
        }
        tile += gridDim.x;
    };
    // a short list with few loads in flight: those past its end are not for nothing
    // (8 pairs of 256 x 128: 6.9 us with eight steps, 6.0 with two)
    const auto pipeline = [&](auto depth) {
        constexpr int kDepth = decltype(depth)::value;
        typename Product::Slot slot[kDepth];
#pragma unroll
        for (int b = 0; b < kDepth; ++b)
            next_load(slot[b]);
        int step = 0;
        for (int i = 0; i < count; i += kDepth)
#pragma unroll
            for (int b = 0; b < kDepth; ++b) {
                m.multiply(slot[b]);
                if (!kWhole && step == 0)
                    m.clear();
                next_load(slot[b]);
                if (++step == per && i + b < count) {
                    leave();
                    step = 0;
                }
            }
    };
    enter();
    if (count <= kFewShort)
        pipeline(Count<2>());
    else
        pipeline(Count<Product::kDepth>());
}

// A block: 16 columns of y over every unit, or one of a.splits parts of that.  The units'
// contractions end to end are one list of steps, of which each wave takes an equal run;
// where a run leaves a unit, its sums go, weighted, to the wave's totals of the tokens in
// LDS, and the waves' totals are added in order.  (Rows of tokens that do not ask for an
// expert never meet its weights, whatever these hold.)  Where y has few columns the
// blocks of a tile share its list; the last to finish adds their sums in order.  (The same
// layers' second products, 235 MB: 43 us, 5.5 TB/s, and 0.69 GB: 108 us, 6.4 TB/s.  With
// four waves taking neighbouring steps in turn, longer runs of a row at a time, as fast.)
template <int kType, int kRows, bool kWhole>
__global__ __launch_bounds__(kFewDownWaves *kWave, few_waves(kType, kRows, 1)) void k_few_down(
    const FewArgs a)
{
    typedef FewProduct<kType, kRows, 1, kWhole> Product;
    constexpr int kMI = Product::kMI;
    __shared__ FewRouting routing;
    __shared__ float weight[kFewPairs];
    __shared__ __align__(16) f32x4 total[kFewDownWaves][kFewTokens][4];
    __shared__ __align__(16) uint8_t turn[kFewDownWaves][Product::kTurnBytes];
    __shared__ int last;
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x / kWave);
    const int units = few_routing<kFewDownWaves * kWave, kRows>(a, routing, weight);
    const int col_tiles = (a.hidden + 15) / 16, split = blockIdx.x / col_tiles;
    const int tile = blockIdx.x - split * col_tiles, c0 = tile * 16;
    for (int i = lane; i < a.tokens * 4; i += kWave)
        total[wave][i / 4][i % 4] = f32x4{0, 0, 0, 0};
    Product m;
    m.init(a.w2, a.inner, lane, turn[wave], a.h, (uint32_t)a.tokens * a.topk * a.inner * 2,
           a.indices);
    const int all = units * m.steps, runs = kFewDownWaves * a.splits;
    const int run = split * kFewDownWaves + wave;
    const int begin = (int)((int64_t)all * run / runs);
    int count = (int)((int64_t)all * (run + 1) / runs) - begin;
    // where loads and multiplications are in the list
    int load_unit = begin / m.steps, load_step = begin - load_unit * m.steps, loaded = 0;
    bool first = load_step == 0;
    const bool behind = !kWhole && !first && count > 0;   // the line before the run's first
    load_step -= behind;
    count += behind;
    int unit = load_unit, step = load_step;
    const auto enter = [&] {
        const FewUnit u = few_unit(routing, load_unit);
        m.expert(a.w2, a.s2, a.b2, u.expert, c0, a.hidden, [&](int r) {
            return r < u.rows ? routing.row[u.first + r] & 0x3ff : -1;
        });
    };
    const auto next_load = [&](typename Product::Slot &to) {
        m.load(to, loaded < count ? load_step : m.steps);
        ++loaded;
        if (++load_step == m.steps && loaded < count) {
            load_step = 0;
            ++load_unit;
            enter();
        }
    };
    // the unit's sums into the totals; its bias with its first step
    const auto leave = [&] {
        const FewUnit u = few_unit(routing, unit);
        const int quad = lane >> 4;
        f32x4 by = {1, 1, 1, 1}, plus = {0, 0, 0, 0};
        if constexpr (kType == kTypeInt8)
            by = m.columns(0);
        if (a.b2 && first)
            plus = m.biases(a.b2, u.expert, 0, c0, a.hidden);
#pragma unroll
        for (int i = 0; i < kMI; ++i) {
            const int r = i * 16 + (lane & 15);
            if (r >= u.rows)
                continue;
            const float w = weight[u.first + r];
            f32x4 &sum = total[wave][routing.row[u.first + r] >> 10][quad];
            f32x4 t = sum;
#pragma unroll
            for (int v = 0; v < 4; ++v)
                t[v] = __builtin_fmaf(w, m.acc[i][0][v] * by[v] + plus[v], t[v]);
            sum = t;
        }
        m.clear();
    };
    const auto pipeline = [&](auto depth) {
        constexpr int kDepth = decltype(depth)::value;
        typename Product::Slot slot[kDepth];
#pragma unroll
        for (int b = 0; b < kDepth; ++b)
            next_load(slot[b]);
        for (int i = 0; i < count; i += kDepth)
#pragma unroll
            for (int b = 0; b < kDepth; ++b) {
                m.multiply(slot[b]);
                if (behind && i + b == 0)
                    m.clear();
                next_load(slot[b]);
                if (i + b == count - 1 || (i + b < count && step == m.steps - 1))
                    leave();
                if (++step == m.steps) {
                    step = 0;
                    ++unit;
                    first = true;
                }
            }
    };
    if (count > 0) {
        enter();
        if (count <= kFewShort)
            pipeline(Count<2>());
        else
            pipeline(Count<Product::kDepth>());
    }
    __syncthreads();
    const auto sum_of = [&](int i) {
        f32x4 y = total[0][i / 4][i % 4];
#pragma unroll
        for (int w = 1; w < kFewDownWaves; ++w)
            y += total[w][i / 4][i % 4];
        return y;
    };
    const auto store = [&](int i, f32x4 y) {
        const int c = c0 + i % 4 * 4;
        if (c < a.hidden)
            *reinterpret_cast<bf16x4 *>(a.out + ((size_t)(i / 4) * a.hidden + c) * 2) = to_bf16(y);
    };
    if (a.splits == 1) {
        for (int i = threadIdx.x; i < a.tokens * 4; i += kFewDownWaves * kWave)
            store(i, sum_of(i));
        return;
    }
    // The blocks' sums go through the memory that all XCDs share, and so do the tickets:
    // relaxed accesses of the agent's scope, ordered by each wave's wait for its own stores
    // before the block takes a ticket (as in k_gate).
    const int words = a.tokens * 16;
    float *tops = a.partial + (size_t)tile * a.splits * words;
    for (int i = threadIdx.x; i < a.tokens * 4; i += kFewDownWaves * kWave) {
        const f32x4 y = sum_of(i);
#pragma unroll
        for (int v = 0; v < 4; ++v)
            store_agent(tops + (size_t)split * words + i * 4 + v, y[v]);
    }
    __builtin_amdgcn_s_waitcnt(0);
    __syncthreads();
    if (threadIdx.x == 0)
        last = __hip_atomic_fetch_add(a.ticket + tile, 1u, __ATOMIC_RELAXED,
                                      __HIP_MEMORY_SCOPE_AGENT) == (uint32_t)a.splits - 1;
    __syncthreads();
    if (!last)
        return;
    for (int i = threadIdx.x; i < a.tokens * 4; i += kFewDownWaves * kWave) {
        f32x4 y = {0, 0, 0, 0}, part[kFewMostSplits];
#pragma unroll
        for (int z = 0; z < kFewMostSplits; ++z)
#pragma unroll
            for (int v = 0; v < 4; ++v)
                part[z][v] = z < a.splits
                                 ? __hip_atomic_load(tops + (size_t)z * words + i * 4 + v,
                                                     __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT)
                                 : 0.0f;
#pragma unroll
        for (int z = 0; z < kFewMostSplits; ++z)
            y += part[z];
        store(i, y);
    }
}

}  // namespace epdc_layer
