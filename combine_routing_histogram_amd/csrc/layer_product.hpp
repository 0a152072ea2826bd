// layer_product.hpp -- gfx950 kernels of the experts' matrix products over the
// received rows: out = act(x W^T + b) + residual per expert, and the gradients
// dx = dz W, dW = dz^T x, db = sum dz.
//
// All three products run through one tile kernel.  A tile is 64 or 256 "P" rows
// by 256 "Q" columns; the MFMA's first operand is Q and its second P, so a lane
// ends with four consecutive output columns of one row.  Operands go from
// HBM to LDS by direct loads (16 bytes a lane, no registers between) and from
// LDS to the matrix cores as fragments whose contraction index lies along a
// lane's registers.  Where memory has the contraction along the rows (W of dx,
// both operands of dW) the fragment is read with the transposing LDS load.
#pragma once

#include <hip/hip_runtime.h>
#include <limits.h>
#include <stdint.h>

namespace epdc_layer {

typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kWave = 64;
constexpr int kMaxExperts = 512;
constexpr int kXcds = 8;
constexpr int kStepBytes = 128;  // contraction bytes of one LDS row (untransposed operand)

enum Product { kForward, kGradInput, kGradWeight };

// Types of a product's operands.
enum Type { kTypeBf16, kTypeE4m3, kTypeInt8 };

constexpr int element_bytes(int type) { return type == kTypeBf16 ? 2 : 1; }

enum Act { kActNone, kActRelu, kActGelu, kActSilu, kActSwiglu, kActGeglu };

struct ProductArgs {
    int32_t rows;        // rows of the received layout the call may touch
    int32_t experts;
    int32_t contract;    // contraction length (rows of the expert for kGradWeight)
    int32_t p_bytes;     // bytes of a row of p
    int32_t q_bytes;     // bytes of a row of q
    int32_t out_rows;    // kGradWeight: rows of one expert's gradient
    int32_t out_cols;    // columns of out
    int32_t weight_rows; // out_features
    int32_t col_tiles;   // column tiles of an expert
    int32_t row_tiles;   // kGradWeight: row tiles of an expert
    int32_t act;
    int32_t out_fp32;    // kGradWeight: out holds fp32
    const uint8_t *p, *q;
    const float *scales, *weight_scales;  // e4m3: per 128 columns; int8: per row
    const float *bias;
    const uint16_t *residual;
    const int32_t *expert_off;
    uint8_t *out;
    uint16_t *preact;
};

__device__ inline int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

__device__ inline float bf16_to_f32(uint16_t b) { return __uint_as_float((uint32_t)b << 16); }

__device__ inline bf16x4 to_bf16(f32x4 v)
{
    return bf16x4{(__bf16)v[0], (__bf16)v[1], (__bf16)v[2], (__bf16)v[3]};
}

// The activations, in fp32.  x / (1 + exp(-x)) tends to -0 for large negative
// x; exp and the reciprocal are the hardware's (about 1 ulp each, far below
// the rounding of the bf16 result).
__device__ inline float act_silu(float x)
{
    return x * __builtin_amdgcn_rcpf(1.0f + __expf(-x));
}
// The normal distribution function, and e^(-x^2 / 2), which it goes through.  By way
// of 1 + erf its tail would cancel: at -5 several percent of it are lost, below
// -5.5 all.  Its tail times e^(x^2 / 2) is smooth and falls like 1 / x: s P(s) with
// s = 1 / (1 + 0.305 |x|), P of degree 7 by least squares reweighted toward the
// largest relative error over [0, 14], which is 2^-23; with the exponential's
// argument rounded 2^-18 at 8.  (gelu over 32768 x 512 x 4096 and its gradients:
// 350 and 818 us with 1 + erff, 386 and 858 with erfcf, 284 and 756 so.)
__device__ inline float normal_cdf(float x, float &e)
{
    const float s = __builtin_amdgcn_rcpf(__builtin_fmaf(0.305f, fabsf(x), 1.0f));
    e = __builtin_amdgcn_exp2f(x * x * -0.72134752f);
    float p = 0.0366991945f;
    p = __builtin_fmaf(p, s, -0.15298833f);
    p = __builtin_fmaf(p, s, 0.185716927f);
    p = __builtin_fmaf(p, s, -0.0379768424f);
    p = __builtin_fmaf(p, s, 0.121021688f);
    p = __builtin_fmaf(p, s, 0.103420861f);
    p = __builtin_fmaf(p, s, 0.122466817f);
    p = __builtin_fmaf(p, s, 0.121639736f);
    const float tail = p * s * e;
    return x < 0.0f ? tail : 1.0f - tail;
}
__device__ inline float act_gelu(float x)
{
    float e;
    return x * normal_cdf(x, e);
}

__device__ inline float act_one(int act, float x)
{
    switch (act) {
    case kActRelu: return x > 0.0f ? x : (x != x ? x : 0.0f);
    case kActGelu:
    case kActGeglu: return act_gelu(x);
    case kActSilu:
    case kActSwiglu: return act_silu(x);
    default: return x;
    }
}

__device__ inline float act_one_grad(int act, float x)
{
    switch (act) {
    case kActRelu: return x > 0.0f ? 1.0f : (x != x ? x : 0.0f);
    case kActGelu:
    case kActGeglu: {
        float e;
        const float cdf = normal_cdf(x, e);
        return __builtin_fmaf(x * 0.39894228f, e, cdf);
    }
    case kActSilu:
    case kActSwiglu: {
        const float s = __builtin_amdgcn_rcpf(1.0f + __expf(-x));
        return s * (1.0f + x * (1.0f - s));
    }
    default: return 1.0f;
    }
}

__host__ __device__ inline bool act_gated(int act) { return act >= kActSwiglu; }

// ---------------------------------------------------------------------------
// Which tile a block computes
// ---------------------------------------------------------------------------
//
// Tiles are numbered expert by expert, inside an expert by bands of up to 8 row
// tiles, inside a band column by column.  Blocks go to the XCDs in turn (block b
// is number b / 8 of XCD b % 8); each XCD takes runs of 32 consecutive tiles,
// about a patch of 8 x 4, which its 32 CUs read through one L2 (12 operand
// tiles instead of 64), and the 8 XCDs take neighbouring runs, mostly of one
// expert, so that what one has read the others find in the last-level cache.
// (One expert per XCD instead read 4.1 GB from HBM for 0.94 GB of operands:
// 32768 x 7168 x 4096 over 8 experts 1944 us where this order took 1766.)  The counts per expert
// are on the device only: every block scans the offsets (at most 513 ints, in
// L2) into an index of its own.

struct Tile {
    int expert, row0, rows, row_tile, col_tile;
};

constexpr int kBandRows = 8, kRun = 32;

__device__ inline int tile_number(int block)
{
    const int slot = block / kXcds;
    return (slot / kRun * kXcds + block % kXcds) * kRun + slot % kRun;
}

// Tile `local` of an expert of mt x nt tiles.
__device__ inline void place(int local, int mt, int nt, Tile &t)
{
    const int band = local / (kBandRows * nt), in = local - band * (kBandRows * nt);
    const int first = band * kBandRows;
    const int rows = mt - first < kBandRows ? mt - first : kBandRows;
    t.col_tile = in / rows;
    t.row_tile = first + in - t.col_tile * rows;
}

__device__ inline int clamp_row(const int32_t *off, int i, int rows)
{
    const int v = off[i];
    return v < 0 ? 0 : (v > rows ? rows : v);
}

// The experts' first tiles and rows, in LDS.
struct TileIndex {
    int first[kMaxExperts];      // INT_MAX behind the last expert
    int start[kMaxExperts + 1];
    int wave_sum[16];
    int total;
};

// Fills the index, and ends with a barrier.
template <int kThreads>
__device__ inline void build_index(const ProductArgs &a, int bm, TileIndex &x)
{
    constexpr int kEach = kMaxExperts / kThreads, kWaves = kThreads / kWave;
    static_assert(kMaxExperts % kThreads == 0 && kWaves <= 16, "whole experts per thread");
    const int tid = threadIdx.x, lane = tid & 63, wave = tid / kWave;
    int n[kEach], cnt = 0;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        const int e = tid * kEach + i;
        n[i] = 0;
        if (e < a.experts) {
            const int r0 = clamp_row(a.expert_off, e, a.rows);
            const int r1 = clamp_row(a.expert_off, e + 1, a.rows);
            x.start[e] = r0;
            if (e == a.experts - 1)
                x.start[a.experts] = r1;
            n[i] = r1 > r0 ? (r1 - r0 + bm - 1) / bm * a.col_tiles : 0;
        }
        cnt += n[i];
    }
    int incl = cnt;
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) {
        const int u = __shfl_up(incl, d, kWave);
        if (lane >= d)
            incl += u;
    }
    if (lane == kWave - 1)
        x.wave_sum[wave] = incl;
    __syncthreads();
    int total = 0, first = incl - cnt;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
        const int v = x.wave_sum[w];
        first += w < wave ? v : 0;
        total += v;
    }
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        const int e = tid * kEach + i;
        x.first[e] = e < a.experts ? first : INT_MAX;
        first += n[i];
    }
    if (tid == 0)
        x.total = total;
    __syncthreads();
}

// Tile `id` of all; false past the total.  Every wave finds it for itself: the
// expert is the last whose first tile is not behind it.
__device__ inline bool find_tile(const ProductArgs &a, const TileIndex &x, int id, int bm, Tile &t)
{
    if (id >= uniform(x.total))
        return false;
    const int lane = threadIdx.x & 63;
    int upto = 0;
#pragma unroll
    for (int k = 0; k < kMaxExperts / kWave; ++k)
        upto += __popcll(__ballot(x.first[k * kWave + lane] <= id));
    t.expert = uniform(upto - 1);
    const int start = uniform(x.start[t.expert]);
    const int have = uniform(x.start[t.expert + 1]) - start;
    place(id - uniform(x.first[t.expert]), (have + bm - 1) / bm, a.col_tiles, t);
    t.row0 = start + t.row_tile * bm;
    const int left = have - t.row_tile * bm;
    t.rows = left < bm ? left : bm;
    return true;
}

// ---------------------------------------------------------------------------
// Operand tiles in LDS
// ---------------------------------------------------------------------------

typedef __attribute__((address_space(3))) uint8_t lds_byte;

// base and bytes are the same in every lane; saying so keeps the descriptor in
// scalar registers where the compiler took a vector division into them.
__device__ inline __amdgpu_buffer_rsrc_t buffer_at(const uint8_t *base, uint32_t bytes)
{
    const uint64_t p = (uint64_t)base;
    const uint64_t u = ((uint64_t)(uint32_t)uniform((int)(p >> 32)) << 32) |
                       (uint32_t)uniform((int)(uint32_t)p);
    return __builtin_amdgcn_make_buffer_rsrc((void *)u, 0, uniform((int)bytes), 0x00020000);
}

// 16 bytes per lane from `at + off` to LDS, lane order from `lds` on.  Written out
// because the compiler, which cannot tell the two buffers of a tile apart,
// else waits for every such load before a transposing LDS read; when they have
// landed is wait_and_meet's business.  Nothing returns to registers.  M0 holds
// the LDS address; it is reserved to the compiler, which takes no clobber of
// it, so the compiler's own code may not use it.  The descriptor can come from
// v_readfirstlane just before: a memory instruction may read a scalar register five
// wait states after a vector instruction wrote it, which the compiler sees to
// in its own code but not in asm; s_mov and s_nop 3 are five.  Without them a
// load can take the last step's bound.  tests/test_layer_asm.py reads the
// listing for both.
__device__ __forceinline__ void load_direct(__amdgpu_buffer_rsrc_t at, uint32_t off, uint8_t *lds)
{
    const int to = uniform((int)(uint32_t)(uintptr_t)(lds_byte *)lds);
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 3\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"(to),
                 "v"(off), "s"(at));
}

constexpr uint32_t kNowhere = 0x80000000u;  // past every buffer below: the load gives zeros
constexpr uint32_t kOpen = 0x7fffffffu;

// An operand whose contraction index runs along memory rows: LDS holds kRows
// rows of 128 bytes.  A direct load fills 1 KiB (8 rows) of LDS in lane order,
// so the bank swizzle -- 16-byte chunk c of row r sits at chunk c ^ (r & 7) --
// is applied to the address a lane loads from.  Fragment reads of 16 rows x 16
// bytes then touch every bank evenly.
// kWhole: the contraction is whole steps, so only steps past the end are cut.
template <int kRows, int kWaves, bool kWhole>
struct StraightTile {
    static constexpr int kBytes = kRows * kStepBytes;
    static constexpr int kReads = 1;  // LDS reads of a fragment
    static constexpr int kLoads = kRows / 8 / kWaves;
    static_assert(kRows % (8 * kWaves) == 0, "whole loads per wave");
    uint32_t off[kLoads];
    const uint8_t *base;
    int chunk;  // of this lane, in elements of 16 bytes

    // row(r): the source row of LDS row r, in bounds
    template <typename F>
    __device__ inline void init(const uint8_t *b, int row_bytes, int wave, int lane, F &&row)
    {
        base = b;
        chunk = (lane & 7) ^ (lane >> 3);
#pragma unroll
        for (int d = 0; d < kLoads; ++d)
            off[d] = (uint32_t)row((d * kWaves + wave) * 8 + (lane >> 3)) * (uint32_t)row_bytes +
                     (uint32_t)chunk * 16;
    }
    // step: which 128 bytes of the rows; left: contraction bytes from there on
    // (none left: zeros, and no traffic)
    template <int kCount = kLoads>
    __device__ inline void load(uint8_t *lds, int step, int left, int wave)
    {
        const __amdgpu_buffer_rsrc_t rs =
            buffer_at(base + (size_t)step * kStepBytes, kWhole && left <= 0 ? 0 : kOpen);
        const bool out = !kWhole && chunk * 16 >= left;
#pragma unroll
        for (int d = 0; d < kCount; ++d)
            load_direct(rs, out ? kNowhere : off[d], lds + (d * kWaves + wave) * 1024);
    }
    // 16 rows from row0; half 0 or 1 of the step.  Lane l: row l % 16, 16 bytes.
    __device__ static inline i32x4 frag(const uint8_t *lds, int row0, int half, int lane)
    {
        const int r = row0 + (lane & 15);
        const int c = (half * 4 + (lane >> 4)) ^ (lane & 7);
        return *reinterpret_cast<const i32x4 *>(lds + r * kStepBytes + c * 16);
    }
};

// An operand whose contraction index runs across memory rows (bf16): LDS holds
// 64 contraction rows of kCols elements.  The transposing read takes 8 bytes
// per lane, four rows by 32 bytes per 16 lanes; chunk pairs are swizzled by
// the row (r & 3, and bit 3) so that the rows of one read and its neighbour
// lie in different banks.
template <int kCols, int kWaves>
struct CrossTile {
    static constexpr int kRowBytes = kCols * 2;
    static constexpr int kBytes = 64 * kRowBytes;
    static constexpr int kReads = 2;
    static constexpr int kChunks = kRowBytes / 16;
    static constexpr int kRowsPerLoad = 64 / kChunks;
    static constexpr int kLoads = kBytes / 1024 / kWaves;
    static_assert(kChunks <= 64 && kChunks >= 16, "a load covers whole rows");
    static_assert(kBytes % (1024 * kWaves) == 0, "whole loads per wave");
    uint32_t off[kLoads];
    const uint8_t *base;
    int row_bytes;

    __device__ static inline int key(int r) { return ((r & 3) | ((r >> 1) & 4)) << 1; }

    // b: the first contraction row; col0_bytes: of the tile's first column
    __device__ inline void init(const uint8_t *b, int rb, uint32_t col0_bytes, int wave, int lane)
    {
        base = b;
        row_bytes = rb;
#pragma unroll
        for (int d = 0; d < kLoads; ++d) {
            const int r = (d * kWaves + wave) * kRowsPerLoad + lane / kChunks;
            off[d] = (uint32_t)r * (uint32_t)rb + col0_bytes +
                     (uint32_t)((lane % kChunks) ^ key(r)) * 16;
        }
    }
    // left: contraction rows from this step on; later rows read as zeros, and
    // so does whatever a ragged column tile takes behind the last of them
    template <int kCount = kLoads>
    __device__ inline void load(uint8_t *lds, int step, int left, int wave)
    {
        static_assert(kCount == kLoads, "all columns of the tile");
        const uint32_t rows = left < 64 ? (left > 0 ? left : 0) : 64;
        const __amdgpu_buffer_rsrc_t rs =
            buffer_at(base + (size_t)step * 64 * row_bytes, rows * (uint32_t)row_bytes);
#pragma unroll
        for (int d = 0; d < kLoads; ++d)
            load_direct(rs, off[d], lds + (d * kWaves + wave) * 1024);
    }
    // 16 columns from col0, contraction rows half*32 + (lane/16)*8 ... +7
    __device__ static inline i32x4 frag(const uint8_t *lds, int col0, int half, int lane)
    {
        const int g = lane >> 4, q = lane & 3, r = (lane >> 2) & 3;
        const int row = half * 32 + g * 8 + r;
        const int c = ((col0 >> 3) + (q >> 1)) ^ key(row);
        const uint8_t *p = lds + row * kRowBytes + c * 16 + (q & 1) * 8;
        typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
        const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)p);
        const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(p + 4 * kRowBytes));
        const s16x8 v = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
        return __builtin_bit_cast(i32x4, v);
    }
};

template <bool kCross, int kExtent, int kWaves, bool kWhole>
struct PickTile {
    typedef StraightTile<kExtent, kWaves, kWhole> type;
};
template <int kExtent, int kWaves, bool kWhole>
struct PickTile<true, kExtent, kWaves, kWhole> {
    typedef CrossTile<kExtent, kWaves> type;
};

__device__ inline f32x4 mfma_bf16(i32x4 a, i32x4 b, f32x4 c)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// e4m3 x e4m3 over 128 contraction elements; the block scales of the
// instruction are 1 (exponent byte 127).  The matrix cores cut the products of
// 8 consecutive elements off at 2^-13 of the largest exponent among them
// before they add them in fp32 (the instruction over 32 elements does the
// same); the only way round it is to widen the codes to bf16, at half the
// rate, for errors that lie 2^-15 or so of the result below its bf16 rounding.
__device__ inline f32x4 mfma_e4m3(i32x8 a, i32x8 b, f32x4 c)
{
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 0, 0, 0, 0x7f7f7f7f, 0,
                                                            0x7f7f7f7f);
}

// int8 x int8 over 64 contraction elements, exact in 32-bit integers
__device__ inline i32x4 mfma_int8(i32x4 a, i32x4 b, i32x4 c)
{
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(a, b, c, 0, 0, 0);
}

// 64 bytes of contraction: their products added to an accumulator of the type
__device__ inline void multiply_add(i32x4 a, i32x4 b, f32x4 &c) { c = mfma_bf16(a, b, c); }
__device__ inline void multiply_add(i32x4 a, i32x4 b, i32x4 &c) { c = mfma_int8(a, b, c); }

template <int kType>
struct AccumulatorOf {
    typedef f32x4 type;
};
template <>
struct AccumulatorOf<kTypeInt8> {
    typedef i32x4 type;
};

__device__ inline f32x4 to_f32(f32x4 v) { return v; }
__device__ inline f32x4 to_f32(i32x4 v)
{
    return f32x4{(float)v[0], (float)v[1], (float)v[2], (float)v[3]};
}

__device__ inline i32x8 join(i32x4 a, i32x4 b)
{
    return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
}

template <int kN>
struct Count {
    static constexpr int value = kN;
};

template <int kN, int kAt = 0, typename F>
__device__ __forceinline__ void unrolled(F &&f)
{
    if constexpr (kAt < kN) {
        f(Count<kAt>());
        unrolled<kN, kAt + 1>(f);
    }
}

// All but the kYoungest youngest direct loads and every LDS read of this wave
// are done, and so are the other waves' at the same point; the compiler may
// move no LDS access across it.
template <int kYoungest>
__device__ __forceinline__ void wait_and_meet()
{
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(kYoungest) : "memory");
}

// Spread LDS reads and direct loads between the multiplications of the code
// before it: left to itself the compiler gathers the reads and then waits.
template <int kReads, int kMuls, int kLoads, int kAt = 0>
__device__ __forceinline__ void weave()
{
    constexpr int kGroups = kReads < kMuls ? kReads : kMuls;
    if constexpr (kAt < kGroups) {
        constexpr int kR = (kAt + 1) * kReads / kGroups - kAt * kReads / kGroups;
        constexpr int kM = (kAt + 1) * kMuls / kGroups - kAt * kMuls / kGroups;
        constexpr int kL = (kAt + 1) * kLoads / kGroups - kAt * kLoads / kGroups;
        __builtin_amdgcn_sched_group_barrier(0x100, kR, 0);
        __builtin_amdgcn_sched_group_barrier(0x008, kM, 0);
        if constexpr (kL > 0)
            __builtin_amdgcn_sched_group_barrier(0x020, kL, 0);
        weave<kReads, kMuls, kLoads, kAt + 1>();
    } else {
        __builtin_amdgcn_sched_barrier(0);
    }
}

// Four consecutive output columns of one row: bias, activation and residual in
// fp32, one rounding.  z: the product; up: its second half (gated).
__device__ inline void finish_forward(const ProductArgs &a, int expert, int row, int col,
                                      f32x4 z, f32x4 up)
{
    const bool gated = act_gated(a.act);
    if (a.bias) {
        const float *b = a.bias + (size_t)expert * a.weight_rows + col;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            z[i] += b[i];
            if (gated)
                up[i] += b[a.out_cols + i];
        }
    }
    if (a.preact) {
        uint16_t *z0 = a.preact + (size_t)row * a.weight_rows + col;
        *reinterpret_cast<bf16x4 *>(z0) = to_bf16(z);
        if (gated)
            *reinterpret_cast<bf16x4 *>(z0 + a.out_cols) = to_bf16(up);
    }
    f32x4 y;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        y[i] = act_one(a.act, z[i]);
        if (gated)
            y[i] *= up[i];
    }
    const size_t at = (size_t)row * a.out_cols + col;
    if (a.residual) {
        const ushort4 r = *reinterpret_cast<const ushort4 *>(a.residual + at);
        y += f32x4{bf16_to_f32(r.x), bf16_to_f32(r.y), bf16_to_f32(r.z), bf16_to_f32(r.w)};
    }
    *reinterpret_cast<bf16x4 *>(a.out + at * 2) = to_bf16(y);
}

// Eight consecutive output columns of one row, as finish_forward; the biases (0
// for none) and the residual are loaded beforehand.
__device__ inline void finish_forward8(const ProductArgs &a, int row, int col, float (&z)[8],
                                       float (&up)[8], const float (&bz)[8], const float (&bu)[8],
                                       bf16x8 res)
{
    const bool gated = act_gated(a.act);
    if (a.bias) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            z[i] += bz[i];
            up[i] += bu[i];
        }
    }
    bf16x8 o;
    if (a.preact) {
        uint16_t *z0 = a.preact + (size_t)row * a.weight_rows + col;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            o[i] = (__bf16)z[i];
        *reinterpret_cast<bf16x8 *>(z0) = o;
        if (gated) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                o[i] = (__bf16)up[i];
            *reinterpret_cast<bf16x8 *>(z0 + a.out_cols) = o;
        }
    }
    switch (a.act) {
    case kActRelu:
#pragma unroll
        for (int i = 0; i < 8; ++i)
            z[i] = act_one(kActRelu, z[i]);
        break;
    case kActGelu:
    case kActGeglu:
#pragma unroll
        for (int i = 0; i < 8; ++i)
            z[i] = act_gelu(z[i]);
        break;
    case kActSilu:
    case kActSwiglu:
#pragma unroll
        for (int i = 0; i < 8; ++i)
            z[i] = act_silu(z[i]);
        break;
    }
    if (gated) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            z[i] *= up[i];
    }
    if (a.residual) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            z[i] += (float)res[i];
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        o[i] = (__bf16)z[i];
    *reinterpret_cast<bf16x8 *>(a.out + ((size_t)row * a.out_cols + col) * 2) = o;
}

// ---------------------------------------------------------------------------
// The tile kernel
// ---------------------------------------------------------------------------
//
// A tile is kGroups * 64 P rows by 256 Q columns, worked on by eight waves, two
// along P and four along Q; the two of a SIMD share its columns and take the
// 16-row blocks in turn, so a ragged tile of g groups costs each of them
// g / kGroups of the work.  A step is 128 bytes of contraction.  Its operands
// arrive as four units: P0 and P1, the first and second half of the rows, Q0
// and Q1, 128 columns each (gated: Q0 gate rows, Q1 the up rows of the same
// columns, so that a lane ends with both factors of its outputs).
//
// A step runs in two halves, one barrier each:
//   A: P0 x Q0, P0 x Q1, while Q1 and P1 are read from LDS
//   B: P1 x Q0, P1 x Q1, while P0 and Q0 of the next step are read
// Each unit is read once, into registers; by the barrier after that every wave
// has it, and its LDS takes the unit of two steps on.  So of the two steps that
// LDS holds all but the pair being read is in flight: the loads of a pair have
// one and a half steps to land.  (With whole steps as the unit, loads drain
// at every barrier: loads alone took 1483 us for 32768 x 7168 x 4096 where these
// take 1188, and the multiplications alone 1344.)
//
// Reached, 1420 to 1470 us for 32768 x 7168 x 4096 bf16 over 8 even experts: 1.31 to
// 1.35 PFLOP/s of the 1.43 of a library product; e4m3 950 to 980 us.  Skewed over
// 64 experts 1.80 to 1.91 ms, e4m3 1.17 to 1.21: the last tiles and row groups that
// are not full.
//
// int8 runs as bf16 does, a step's 128 bytes being 128 features instead of 64, with exact
// sums; a row's and a column's scales meet them as the accumulators leave: 800 to 820 us,
// 2.4 POP/s where a library product of 8192 x 8192 x 8192 reaches 2.0, skewed 0.97 to 1.02 ms.

constexpr int kTileWaves = 8, kTileWavesM = 2, kTileWavesN = 4, kTileCols = 256;

// LDS of a block: P0, P1, Q0 and Q1 of two steps; e4m3: also the scales of four
// steps, 16 bytes for every row and every four columns, twice.  The index before
// them and the results behind use the operands' part.  (Blocks that stayed for
// tile after tile, bringing in the next one's operands while results left,
// gained 1 to 3% on even rows and lost 4% on skewed ones.)
template <bool kE4m3, int kGroups>
struct TileLds {
    static constexpr int kP1 = (kGroups + 1) / 2 * 64 * kStepBytes;
    static constexpr int kQ0 = kGroups * 64 * kStepBytes, kQ1 = kQ0 + 128 * kStepBytes;
    static constexpr int kStage = kQ1 + 128 * kStepBytes;
    static constexpr int kScales = 2 * kStage, kScaleBytes = kGroups * 1024 + 1024;
    static constexpr int kBytes = kScales + (kE4m3 ? 2 * kScaleBytes : 0);
    static constexpr int kOutWave = 16 * 32 * 4;  // 16 rows of 32 columns, fp32
    static_assert(kTileWaves * kOutWave <= kBytes && sizeof(TileIndex) <= kBytes, "both fit");
    static_assert(kBytes <= 160 * 1024, "LDS of a CU");
};

#ifdef __HIP_DEVICE_COMPILE__  // the host pass needs the launch stubs only
// A tile of one product: which, and its contraction length in elements.
struct TileWork {
    Tile t;
    int contract, col0;
    bool gated;
};

// The operands of a tile with kA 64-row groups of rows, and their loads.
template <int kProduct, int kType, int kGroups, int kA>
struct TileOperands {
    static constexpr bool kE4m3 = kType == kTypeE4m3;
    typedef TileLds<kE4m3, kGroups> Lds;
    static constexpr int kG0 = (kGroups + 1) / 2, kG1 = kGroups / 2;  // groups of P0, P1
    static constexpr int kA0 = (kA + 1) / 2, kA1 = kA / 2;            // those with rows
    static constexpr bool kPCross = kProduct == kGradWeight, kQCross = kProduct != kForward;
    typedef typename PickTile<kPCross, kG0 * 64, kTileWaves, kE4m3>::type PTile0;
    typedef typename PickTile<kPCross, (kG1 ? kG1 : 1) * 64, kTileWaves, kE4m3>::type PTile1;
    typedef typename PickTile<kQCross, 128, kTileWaves, kE4m3>::type QTile;
    static constexpr int kL0 = kPCross ? PTile0::kLoads : kA0;
    static constexpr int kL1 = kPCross ? PTile1::kLoads : kA1;
    // loads of a pair of units; the few of scales are not counted, so now and
    // then a wave waits for one load more than it needs
    static constexpr int kAll0 = kL0 + QTile::kLoads, kAll1 = (kA1 ? kL1 : 0) + QTile::kLoads;
    static constexpr int kElem = element_bytes(kType);
    static constexpr int kStep = kStepBytes / kElem;  // contraction elements per step

    PTile0 p0;
    PTile1 p1;
    QTile q0, q1;
    uint8_t *lds;
    int contract, wave;
    bool scaler;
    const uint8_t *scale_base;
    uint32_t scale_off, scale_end;

    __device__ inline void init(const ProductArgs &a, const TileWork &w, uint8_t *l, int wv,
                                int lane)
    {
        const Tile &t = w.t;
        lds = l;
        contract = w.contract;
        wave = wv;
        // weight row of column c of unit h (forward)
        const auto weight_row = [&](int h, int c) {
            const int n = w.gated ? a.weight_rows / 2 : a.weight_rows;
            const int r = w.col0 + c + (w.gated ? 0 : h * 128);
            return (r < n ? r : n - 1) + (w.gated ? h * n : 0);
        };
        if constexpr (kProduct == kForward) {
            const uint8_t *q = a.q + (size_t)t.expert * a.weight_rows * a.q_bytes;
            q0.init(q, a.q_bytes, wave, lane, [&](int r) { return weight_row(0, r); });
            q1.init(q, a.q_bytes, wave, lane, [&](int r) { return weight_row(1, r); });
        } else {
            const uint8_t *q = a.q + (kProduct == kGradInput
                                          ? (size_t)t.expert * a.weight_rows * a.q_bytes
                                          : (size_t)t.row0 * a.q_bytes);
            q0.init(q, a.q_bytes, (uint32_t)w.col0 * 2, wave, lane);
            q1.init(q, a.q_bytes, (uint32_t)w.col0 * 2 + 256, wave, lane);
        }
        const uint8_t *p = a.p + (size_t)t.row0 * a.p_bytes;
        if constexpr (kPCross) {
            p0.init(p, a.p_bytes, (uint32_t)(t.row_tile * kGroups * 64) * 2, wave, lane);
            p1.init(p, a.p_bytes, (uint32_t)(t.row_tile * kGroups * 64) * 2 + 256, wave, lane);
        } else {
            const auto row = [&](int r) { return r < t.rows ? r : t.rows - 1; };
            p0.init(p, a.p_bytes, wave, lane, row);
            if constexpr (kA1 > 0)
                p1.init(p, a.p_bytes, wave, lane, [&](int r) { return row(kA0 * 64 + r); });
        }
        // e4m3: the first waves bring the rows' scales, 64 rows each, the fifth the
        // columns', once every four steps; 16 bytes at a time because a row's
        // scales lie in a line of their own
        scaler = kE4m3 && (wave < kA || wave == 4);
        if constexpr (kE4m3) {
            const int blocks = contract / 128;
            if (wave == 4) {
                const int nb = (a.weight_rows + 127) / 128;
                scale_base = reinterpret_cast<const uint8_t *>(a.weight_scales +
                                                               (size_t)t.expert * nb * blocks);
                scale_end = (uint32_t)nb * blocks * 4;
                scale_off = (uint32_t)(weight_row(lane / 32, lane % 32 * 4) / 128) * blocks * 4;
            } else {
                int r = wave * 64 + lane;
                r = r < t.rows ? r : t.rows - 1;
                scale_base = reinterpret_cast<const uint8_t *>(a.scales + (size_t)t.row0 * blocks);
                scale_end = (uint32_t)t.rows * blocks * 4;
                scale_off = (uint32_t)r * blocks * 4;
            }
        }
    }
    __device__ inline void load_scales(int group)
    {
        if (scaler)
            load_direct(buffer_at(scale_base, scale_end), scale_off + group * 16,
                        lds + Lds::kScales + (group & 1) * Lds::kScaleBytes +
                            (wave == 4 ? kGroups : wave) * 1024);
    }
    __device__ inline void load0(int s)
    {
        uint8_t *st = lds + (s & 1) * Lds::kStage;
        const int left = contract - s * kStep;
        p0.template load<kL0>(st, s, kPCross ? left : left * kElem, wave);
        q0.load(st + Lds::kQ0, s, kQCross ? left : left * kElem, wave);
    }
    __device__ inline void load1(int s)
    {
        uint8_t *st = lds + (s & 1) * Lds::kStage;
        const int left = contract - s * kStep;
        q1.load(st + Lds::kQ1, s, kQCross ? left : left * kElem, wave);
        if constexpr (kA1 > 0)
            p1.template load<kL1>(st + Lds::kP1, s, kPCross ? left : left * kElem, wave);
    }
    // the first two steps
    __device__ inline void start()
    {
        if constexpr (kE4m3)
            load_scales(0);
        load0(0);
        load1(0);
        load0(1);
        load1(1);
    }
};

template <int kProduct, int kType, int kGroups>
__device__ __forceinline__ void product_tile(const ProductArgs &a, int block, uint8_t *lds)
{
    constexpr bool kE4m3 = kType == kTypeE4m3, kInt8 = kType == kTypeInt8;
    typedef typename AccumulatorOf<kType>::type Acc;
    typedef TileLds<kE4m3, kGroups> Lds;
    constexpr int kBM = kGroups * 64;
    constexpr int kP1At = Lds::kP1, kQ0At = Lds::kQ0, kQ1At = Lds::kQ1, kStage = Lds::kStage;
    constexpr int kScaleAt = Lds::kScales, kScaleBytes = Lds::kScaleBytes;
    constexpr int kStep = kStepBytes / element_bytes(kType);

    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x / kWave);
    const int wm = wave / kTileWavesN, wn = wave % kTileWavesN;
    const bool gated = kProduct == kForward && act_gated(a.act);

    TileWork w;
    Tile &t = w.t;
    w.contract = a.contract;
    w.gated = gated;
    if constexpr (kProduct == kGradWeight) {
        const int per = a.row_tiles * a.col_tiles, id = tile_number(block);
        t.expert = id / per;
        if (t.expert >= a.experts)
            return;
        place(id - t.expert * per, a.row_tiles, a.col_tiles, t);
        t.row0 = uniform(clamp_row(a.expert_off, t.expert, a.rows));
        const int n = uniform(clamp_row(a.expert_off, t.expert + 1, a.rows)) - t.row0;
        w.contract = n < 0 ? 0 : n;
        t.rows = a.out_rows - t.row_tile * kBM;
        t.rows = t.rows < kBM ? t.rows : kBM;
    } else {
        TileIndex &index = *reinterpret_cast<TileIndex *>(lds);
        build_index<kTileWaves * kWave>(a, kBM, index);
        if (!find_tile(a, index, tile_number(block), kBM, t))
            return;
        __syncthreads();  // the index's LDS becomes the operands'
    }
    w.col0 = t.col_tile * (gated ? kTileCols / 2 : kTileCols);

    constexpr int kMI = kGroups * 2;
    Acc acc[kMI][4];
    auto sweep = [&](auto groups) {
        constexpr int kA = decltype(groups)::value;  // 64-row groups that hold rows
        typedef TileOperands<kProduct, kType, kGroups, kA> Operands;
        typedef typename Operands::PTile0 PTile0;
        typedef typename Operands::PTile1 PTile1;
        typedef typename Operands::QTile QTile;
        constexpr int kA0 = Operands::kA0, kA1 = Operands::kA1;
        constexpr int kI0 = 2 * kA0, kI1 = 2 * kA1;  // row blocks of a wave
        constexpr int kN0 = kI0, kN1 = kI1 ? kI1 : 1;
        constexpr int kAll0 = Operands::kAll0, kAll1 = Operands::kAll1;
        Operands o;
        o.init(a, w, lds, wave, lane);
        o.start();
        const int steps = (w.contract + kStep - 1) / kStep;
#pragma unroll
        for (int i = 0; i < kMI; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                acc[i][j] = Acc{0, 0, 0, 0};
        // scale of row r (column group: row kGroups * 64 + c / 4) in step s
        const auto scale = [&](int s, int r) {
            return reinterpret_cast<const float *>(lds + kScaleAt +
                                                   (s >> 2 & 1) * kScaleBytes)[r * 4 + (s & 3)];
        };

        i32x4 fp0[kN0][2], fp1[kN1][2], fq0[2][2], fq1[2][2];
        float sp0[kN0], sp1[kN1], sq0[2], sq1[2];
        const auto read_p0 = [&](int s) {
            const uint8_t *st = lds + (s & 1) * kStage;
#pragma unroll
            for (int i = 0; i < kI0; ++i) {
                const int r = (i * kTileWavesM + wm) * 16;
                fp0[i][0] = PTile0::frag(st, r, 0, lane);
                fp0[i][1] = PTile0::frag(st, r, 1, lane);
                if constexpr (kE4m3)
                    sp0[i] = scale(s, r + (lane & 15));
            }
        };
        const auto read_p1 = [&](int s) {
            const uint8_t *st = lds + (s & 1) * kStage;
#pragma unroll
            for (int i = 0; i < kI1; ++i) {
                const int r = (i * kTileWavesM + wm) * 16;
                fp1[i][0] = PTile1::frag(st + kP1At, r, 0, lane);
                fp1[i][1] = PTile1::frag(st + kP1At, r, 1, lane);
                if constexpr (kE4m3)
                    sp1[i] = scale(s, kA0 * 64 + r + (lane & 15));
            }
        };
        const auto read_q = [&](int s, int h, i32x4 (&f)[2][2], float (&sc)[2]) {
            const uint8_t *st = lds + (s & 1) * kStage;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int c = wn * 32 + j * 16;
                f[j][0] = QTile::frag(st + (h ? kQ1At : kQ0At), c, 0, lane);
                f[j][1] = QTile::frag(st + (h ? kQ1At : kQ0At), c, 1, lane);
                if constexpr (kE4m3)
                    sc[j] = scale(s, kGroups * 64 + h * 32 + c / 4 + (lane >> 4));
            }
        };
        // bf16 and int8: row blocks i0 ... of acc by columns j0, j0 + 1
        const auto multiply = [&](auto count, int i0, int j0, const auto &p, const auto &q) {
            constexpr int kI = decltype(count)::value;
#pragma unroll
            for (int half = 0; half < 2; ++half)
#pragma unroll
                for (int i = 0; i < kI; ++i)
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                        multiply_add(q[j][half], p[i][half], acc[i0 + i][j0 + j]);
        };
        // e4m3: the products of a step's 128 features are scaled as they are added
        // to acc, four multiply-adds per matrix instruction.  They follow kLag
        // instructions later, in its shadow: at once they would wait for it.
        constexpr int kLag = kGroups < 4 ? 3 : 1;  // as registers allow
        f32x4 late[kLag];
        float late_scale[kLag];
#pragma unroll
        for (int k = 0; k < kLag; ++k) {
            late[k] = f32x4{0, 0, 0, 0};
            late_scale[k] = 0.0f;
        }
        const auto add_late = [&](auto row, auto col) {
            Acc &to = acc[decltype(row)::value][decltype(col)::value];
#pragma unroll
            for (int v = 0; v < 4; ++v)
                to[v] = __builtin_fmaf(late[0][v], late_scale[0], to[v]);
#pragma unroll
            for (int k = 0; k + 1 < kLag; ++k) {
                late[k] = late[k + 1];
                late_scale[k] = late_scale[k + 1];
            }
        };
        // row blocks kAt ... kAt + kI - 1 by all four column blocks; before them
        // the last ones of the phase over kPrevI blocks from kPrevAt
        const auto multiply_scaled = [&](auto ci, auto cat, auto cprev, auto cprev_at,
                                         const auto &p, const auto &ps) {
            constexpr int kI = decltype(ci)::value, kAt = decltype(cat)::value;
            constexpr int kPrevI = decltype(cprev)::value, kPrevAt = decltype(cprev_at)::value;
            unrolled<4 * kI>([&](auto cn) {
                constexpr int n = decltype(cn)::value;
                constexpr int h = n / (2 * kI), i = n / 2 % kI, j = n % 2;
                const i32x4(&q)[2] = h ? fq1[j] : fq0[j];
                const f32x4 d = mfma_e4m3(join(q[0], q[1]), join(p[i][0], p[i][1]),
                                          f32x4{0, 0, 0, 0});
                const float scale = ps[i] * (h ? sq1[j] : sq0[j]);
                constexpr int m = n >= kLag ? n - kLag : 4 * kPrevI + n - kLag;
                constexpr int mi = n >= kLag ? kI : kPrevI, ma = n >= kLag ? kAt : kPrevAt;
                add_late(Count<ma + m / 2 % mi>(), Count<m / (2 * mi) * 2 + m % 2>());
                late[kLag - 1] = d;
                late_scale[kLag - 1] = scale;
                // vector arithmetic stays where it is; memory and scalar code may pass
                __builtin_amdgcn_sched_barrier(0x0004 | 0x0010 | 0x0080);
            });
        };
        constexpr int kEach = 4;  // bf16 multiplications of a row block by two columns
        constexpr int kScaleReads = kE4m3 ? 1 : 0;
        constexpr int kReadP0 = kI0 * (2 * PTile0::kReads + kScaleReads);
        constexpr int kReadP1 = kI1 * (2 * PTile1::kReads + kScaleReads);
        constexpr int kReadQ = 2 * (2 * QTile::kReads + kScaleReads);

        wait_and_meet<kAll0 + kAll1>();
        read_p0(0);
        read_q(0, 0, fq0, sq0);
        wait_and_meet<kAll0 + kAll1>();
        for (int s = 0; s < steps; ++s) {
            if constexpr (kE4m3) {
                // the group before has been read; this one is needed from step s + 4
                if ((s & 3) == 0)
                    o.load_scales((s >> 2) + 1);
            }
            o.load0(s + 2);
            read_q(s, 1, fq1, sq1);
            read_p1(s);
            if constexpr (kE4m3) {
                multiply_scaled(Count<kI0>(), Count<0>(), Count<kI1 ? kI1 : kI0>(),
                                Count<kI1 ? kI0 : 0>(), fp0, sp0);
            } else {
                multiply(Count<kI0>(), 0, 0, fp0, fq0);
                weave<kReadQ + kReadP1, kI0 * kEach, kAll0>();
                multiply(Count<kI0>(), 0, 2, fp0, fq1);
            }
            wait_and_meet<kAll0 + kAll1>();
            o.load1(s + 2);
            read_p0(s + 1);  // after the last step: zeros, never used
            if constexpr (kE4m3) {
                multiply_scaled(Count<kI1>(), Count<kI0>(), Count<kI0>(), Count<0>(), fp1, sp1);
                read_q(s + 1, 0, fq0, sq0);
            } else {
                multiply(Count<kI1>(), kI0, 0, fp1, fq0);
                weave<kReadP0, (kI1 ? kI1 : 1) * kEach, kAll1>();
                read_q(s + 1, 0, fq0, sq0);
                multiply(Count<kI1>(), kI0, 2, fp1, fq1);
                weave<kReadQ, (kI1 ? kI1 : 1) * kEach, 0>();
            }
            wait_and_meet<kAll0 + kAll1>();
        }
        if constexpr (kE4m3) {
            constexpr int kLast = kI1 ? kI1 : kI0, kLastAt = kI1 ? kI0 : 0;
            unrolled<kLag>([&](auto cn) {
                constexpr int m = 4 * kLast + decltype(cn)::value - kLag;
                add_late(Count<kLastAt + m / 2 % kLast>(), Count<m / (2 * kLast) * 2 + m % 2>());
            });
        }
        wait_and_meet<0>();  // the operands' LDS is free, and no load outlives the block
    };
    if constexpr (kProduct == kGradWeight) {
        sweep(Count<kGroups>());
    } else {
        const int groups = (t.rows + 63) / 64;
        if constexpr (kGroups >= 4) {
            if (groups >= 4)
                sweep(Count<4>());
            else if (groups == 3)
                sweep(Count<3>());
            else if (groups == 2)
                sweep(Count<2>());
        }
        if (groups == 1)
            sweep(Count<1>());
    }

    // The accumulators leave through LDS, 16 rows by 32 columns of a wave at a time
    // and with no barrier: a lane holds 4 columns of 16 rows, and memory wants
    // 16 bytes per lane of few rows.  (From the registers, 8 bytes per lane and a
    // residual load before each store, 1021 x 8 rows of 2048 x 7168 with bias and
    // residual took 425 us of which 113 were this.)
    f32x4 *out = reinterpret_cast<f32x4 *>(lds + wave * Lds::kOutWave);
    const int lr = lane >> 2, v = lane & 3;  // of 8 columns, when read back
    const auto through = [&](const Acc &lo, const Acc &hi, float(&z)[8]) {
        const int row = lane & 15, quad = lane >> 4;
        out[row * 8 + (quad ^ (row & 7))] = to_f32(lo);
        out[row * 8 + ((quad + 4) ^ (row & 7))] = to_f32(hi);
        // lanes read what others wrote: a wave's LDS accesses keep their order,
        // and here the compiler has to keep it too (it moved the writes of
        // lanes with nothing to store under their condition)
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        const f32x4 x = out[lr * 8 + ((v * 2) ^ (lr & 7))];
        const f32x4 y = out[lr * 8 + ((v * 2 + 1) ^ (lr & 7))];
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            z[i] = x[i];
            z[4 + i] = y[i];
        }
    };
    const int col[2] = {w.col0 + wn * 32 + v * 8, w.col0 + 128 + wn * 32 + v * 8};
    float bias[2][8] = {};
    if (kProduct == kForward && a.bias) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int c = gated ? col[0] + h * a.out_cols : col[h];
            if ((gated ? col[0] : col[h]) < a.out_cols) {
                const f32x4 *b = reinterpret_cast<const f32x4 *>(
                    a.bias + (size_t)t.expert * a.weight_rows + c);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    bias[h][i] = b[i / 4][i % 4];
            }
        }
    }
    // int8: the channels' scales, by columns as the biases
    float channel[2][8] = {};
    if constexpr (kInt8) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int c = gated ? col[0] + h * a.out_cols : col[h];
            if ((gated ? col[0] : col[h]) < a.out_cols) {
                const float *sw = a.weight_scales + (size_t)t.expert * a.weight_rows + c;
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    channel[h][i] = sw[i];
            }
        }
    }
    constexpr int kBatch = kMI < 4 ? kMI : 4;  // row blocks whose residuals are in flight
#pragma unroll
    for (int i0 = 0; i0 < kMI; i0 += kBatch) {
        bf16x8 res[kBatch][2] = {};  // an unset vector as an argument would be undefined
        if (kProduct == kForward && a.residual) {
#pragma unroll
            for (int i = 0; i < kBatch; ++i)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int r = ((i0 + i) * kTileWavesM + wm) * 16 + lr;
                    if (r < t.rows && col[h] < a.out_cols && !(gated && h))
                        res[i][h] = *reinterpret_cast<const bf16x8 *>(
                            a.residual + (size_t)(t.row0 + r) * a.out_cols + col[h]);
                }
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int block_row = ((i0 + i) * kTileWavesM + wm) * 16;
            if (block_row >= t.rows)
                break;
            const int r = block_row + lr;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float z[8], up[8] = {};
                through(acc[i0 + i][h * 2], acc[i0 + i][h * 2 + 1], z);
                if (gated) {
                    if (h)
                        break;
                    through(acc[i0 + i][2], acc[i0 + i][3], up);
                }
                if (r >= t.rows || col[h] >= a.out_cols)
                    continue;
                if constexpr (kInt8) {
                    const float sx = a.scales[t.row0 + r];
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        z[k] *= sx * channel[h][k];
                        up[k] *= sx * channel[1][k];
                    }
                }
                if constexpr (kProduct == kForward) {
                    finish_forward8(a, t.row0 + r, col[h], z, up, bias[h], bias[1],
                                    res[i][h]);
                } else {
                    const size_t row =
                        kProduct == kGradInput
                            ? (size_t)(t.row0 + r)
                            : (size_t)t.expert * a.out_rows + t.row_tile * kBM + r;
                    const size_t to = row * a.out_cols + col[h];
                    if (kProduct == kGradWeight && a.out_fp32) {
                        f32x4 *o = reinterpret_cast<f32x4 *>(a.out + to * 4);
                        o[0] = f32x4{z[0], z[1], z[2], z[3]};
                        o[1] = f32x4{z[4], z[5], z[6], z[7]};
                    } else {
                        bf16x8 o;
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            o[k] = (__bf16)z[k];
                        *reinterpret_cast<bf16x8 *>(a.out + to * 2) = o;
                    }
                }
            }
        }
    }
}
#endif

template <int kType, int kGroups>
__global__ __launch_bounds__(kTileWaves *kWave) void k_product_tile(const ProductArgs a)
{
#ifdef __HIP_DEVICE_COMPILE__
    __shared__ __align__(1024) uint8_t lds[TileLds<kType == kTypeE4m3, kGroups>::kBytes];
    product_tile<kForward, kType, kGroups>(a, blockIdx.x, lds);
#endif
}

// ---------------------------------------------------------------------------
// Few rows per expert: the weights stream past them
// ---------------------------------------------------------------------------
//
// With at most kMI * 16 rows per tile the weights are the traffic, each element
// used once.  A block owns 16 output columns (gated: 16 gate and 16 up rows) of
// one row tile; its four waves take the contraction's 128-byte steps in turn, so
// a block reads 512 contiguous bytes of each weight row per round, and add up
// through LDS at the end.  A load takes whole 128-byte lines of 8 rows, past the
// caches, and a wave turns them through 2 KiB of LDS of its own into fragments
// of 16 rows.  (Loaded as fragments, 64 bytes of 16 rows, one token's eight
// experts of 7168 x 4096 took 89 us, 5.3 TB/s; as lines 83, and past the caches
// 72, 6.6 TB/s; with the loads' depth chosen below 68 to 70.)  Rows that are not whole
// lines (kWhole false) go through the caches, as half of each line is another step's: past
// them 64 int8 experts of 2 x 2048 x 4112 with 12 rows each took 150 us, so 130; 8 rows, bf16
// and 4104 columns 235 and 202.

constexpr int kStreamWaves = 4;

template <int kType, int kMI, bool kGated, bool kWhole>
__global__ __launch_bounds__(kStreamWaves *kWave) void k_product_stream(const ProductArgs a)
{
    constexpr int kQ = kGated ? 2 : 1;
    constexpr bool kE4m3 = kType == kTypeE4m3, kInt8 = kType == kTypeInt8;
    typedef typename AccumulatorOf<kType>::type Acc;
    __shared__ __align__(16) Acc part[kStreamWaves][kMI * kQ][kWave];
    __shared__ TileIndex index;
    __shared__ __align__(16) uint8_t turn[kStreamWaves][2][kQ][16 * kStepBytes];
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x / kWave);
    Tile t;
    build_index<kStreamWaves * kWave>(a, kMI * 16, index);
    if (!find_tile(a, index, tile_number(blockIdx.x), kMI * 16, t))
        return;
    const int col0 = t.col_tile * 16;
    const int at = (lane >> 4) * 16;  // this lane's bytes of each half step
    const uint8_t *qp[kQ][2], *pp[kMI];
    const float *sx[kMI], *sw[kQ];
    const int bytes = a.contract * element_bytes(kType), blocks = a.contract / 128;
#pragma unroll
    for (int q = 0; q < kQ; ++q) {
        int c;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            c = col0 + h * 8 + (lane >> 3);
            c = (c < a.out_cols ? c : a.out_cols - 1) + q * a.out_cols;
            qp[q][h] = a.q + ((size_t)t.expert * a.weight_rows + c) * a.q_bytes + (lane & 7) * 16;
        }
        if constexpr (kE4m3) {
            c = col0 + (lane >> 4) * 4;
            c = (c < a.out_cols ? c : a.out_cols - 1) + q * a.out_cols;
            sw[q] = a.weight_scales +
                    ((size_t)t.expert * ((a.weight_rows + 127) / 128) + c / 128) * blocks;
        }
    }
#pragma unroll
    for (int i = 0; i < kMI; ++i) {
        int r = i * 16 + (lane & 15);
        r = t.row0 + (r < t.rows ? r : t.rows - 1);
        pp[i] = a.p + (size_t)r * a.p_bytes + at;
        if constexpr (kE4m3)
            sx[i] = a.scales + (size_t)r * blocks;
    }
    Acc acc[kMI][kQ];
#pragma unroll
    for (int i = 0; i < kMI; ++i)
#pragma unroll
        for (int q = 0; q < kQ; ++q)
            acc[i][q] = Acc{0, 0, 0, 0};

    auto one = [&](const i32x4 (&w)[kQ][2], const i32x4 (&x)[kMI][2], int s) {
#pragma unroll
        for (int i = 0; i < kMI; ++i) {
#pragma unroll
            for (int q = 0; q < kQ; ++q) {
                if constexpr (kE4m3) {
                    const f32x4 d = mfma_e4m3(join(w[q][0], w[q][1]), join(x[i][0], x[i][1]),
                                              f32x4{0, 0, 0, 0});
                    const float f = sx[i][s] * sw[q][s];
#pragma unroll
                    for (int v = 0; v < 4; ++v)
                        acc[i][q][v] = __builtin_fmaf(d[v], f, acc[i][q][v]);
                } else {
                    multiply_add(w[q][0], x[i][0], acc[i][q]);
                    multiply_add(w[q][1], x[i][1], acc[i][q]);
                }
            }
        }
    };
    // lines of 8 + 8 rows to fragments of 16, in one of two turns' LDS; lanes read
    // what others wrote, in the order in which the wave's LDS accesses run
    const auto turned = [&](i32x4 (&w)[kQ][2], int buf) {
        typedef StraightTile<16, 1, false> Turn;
#pragma unroll
        for (int q = 0; q < kQ; ++q)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int r = h * 8 + (lane >> 3);
                *reinterpret_cast<i32x4 *>(turn[wave][buf][q] + r * kStepBytes +
                                           ((lane & 7) ^ (r & 7)) * 16) = w[q][h];
            }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int q = 0; q < kQ; ++q)
#pragma unroll
            for (int h = 0; h < 2; ++h)
                w[q][h] = Turn::frag(turn[wave][buf][q], 0, h, lane);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
    };
    const int full = bytes / kStepBytes;
    // steps in flight per wave: e4m3 with four held too many registers (128 x 8 rows
    // of 4096 x 4096 over 128 experts 377 us, with two 341), bf16 with two too few
    // bytes (one token 75 us, with four 69)
    constexpr int kBatch = kE4m3 ? 2 : 4;
    int s = wave;
    for (; s + (kBatch - 1) * kStreamWaves < full; s += kBatch * kStreamWaves) {
        i32x4 w[kBatch][kQ][2], x[kBatch][kMI][2];
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            const size_t o = (size_t)(s + b * kStreamWaves) * kStepBytes;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
#pragma unroll
                for (int q = 0; q < kQ; ++q) {
                    const i32x4 *from = reinterpret_cast<const i32x4 *>(qp[q][h] + o);
                    w[b][q][h] = kWhole ? __builtin_nontemporal_load(from) : *from;
                }
#pragma unroll
                for (int i = 0; i < kMI; ++i)
                    x[b][i][h] = *reinterpret_cast<const i32x4 *>(pp[i] + o + h * 64);
            }
        }
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            turned(w[b], b & 1);
            one(w[b], x[b], s + b * kStreamWaves);
        }
    }
    for (; s * kStepBytes < bytes; s += kStreamWaves) {
        i32x4 w[kQ][2], x[kMI][2];
        const size_t o = (size_t)s * kStepBytes;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            // past the row: zeros
            const bool win = s * kStepBytes + (lane & 7) * 16 < bytes;
            const bool in = s * kStepBytes + at + h * 64 < bytes;
#pragma unroll
            for (int q = 0; q < kQ; ++q)
                w[q][h] = win ? *reinterpret_cast<const i32x4 *>(qp[q][h] + o)
                              : i32x4{0, 0, 0, 0};
#pragma unroll
            for (int i = 0; i < kMI; ++i)
                x[i][h] = in ? *reinterpret_cast<const i32x4 *>(pp[i] + o + h * 64)
                             : i32x4{0, 0, 0, 0};
        }
        turned(w, 0);
        one(w, x, s);
    }
#pragma unroll
    for (int i = 0; i < kMI; ++i)
#pragma unroll
        for (int q = 0; q < kQ; ++q)
            part[wave][i * kQ + q][lane] = acc[i][q];
    __syncthreads();
    // wave i finishes row block i, adding the waves' parts in order
    for (int i = wave; i < kMI; i += kStreamWaves) {
        Acc sum[kQ];
        f32x4 z[2] = {f32x4{0, 0, 0, 0}, f32x4{0, 0, 0, 0}};
#pragma unroll
        for (int q = 0; q < kQ; ++q) {
            sum[q] = Acc{0, 0, 0, 0};
#pragma unroll
            for (int w = 0; w < kStreamWaves; ++w)
                sum[q] += part[w][i * kQ + q][lane];
            z[q] = to_f32(sum[q]);
        }
        const int r = i * 16 + (lane & 15), c = col0 + (lane >> 4) * 4;
        if (r < t.rows && c < a.out_cols) {
            if constexpr (kInt8) {
                const float sx = a.scales[t.row0 + r];
                const float *sw = a.weight_scales + (size_t)t.expert * a.weight_rows + c;
#pragma unroll
                for (int q = 0; q < kQ; ++q)
#pragma unroll
                    for (int v = 0; v < 4; ++v)
                        z[q][v] *= sx * sw[q * a.out_cols + v];
            }
            finish_forward(a, t.expert, t.row0 + r, c, z[0], z[1]);
        }
    }
}

// ---------------------------------------------------------------------------
// Gradient of the activation, and of the bias
// ---------------------------------------------------------------------------

struct ActGradArgs {
    int32_t rows, experts, cols, act;  // cols: of grad_out (gated: half of preact's)
    const int32_t *expert_off;
    const uint16_t *grad_out, *preact;
    uint16_t *dz;
};

constexpr int kActRows = 4;

// dz = grad_out * act'(preact), 8 columns per lane; gated: both halves.  dz is
// rounded to bf16 because the two products that follow take bf16 operands.
// Bytes are the bound: 32768 rows of 4096, gated, 671 MB in 122 us, 5.5 TB/s.
__global__ __launch_bounds__(kActRows *kWave) void k_act_grad(const ActGradArgs a)
{
    const int r0 = clamp_row(a.expert_off, 0, a.rows);
    const int r1 = clamp_row(a.expert_off, a.experts, a.rows);
    const bool gated = act_gated(a.act);
    const int zcols = gated ? 2 * a.cols : a.cols;
    for (int64_t row = (int64_t)r0 + (int64_t)blockIdx.x * kActRows + threadIdx.y; row < r1;
         row += (int64_t)gridDim.x * kActRows) {
        const uint16_t *dy = a.grad_out + (size_t)row * a.cols;
        const uint16_t *z = a.preact + (size_t)row * zcols;
        uint16_t *dz = a.dz + (size_t)row * zcols;
        for (int c = threadIdx.x * 8; c < a.cols; c += kWave * 8) {
            const bf16x8 g = *reinterpret_cast<const bf16x8 *>(dy + c);
            const bf16x8 z0 = *reinterpret_cast<const bf16x8 *>(z + c);
            bf16x8 o;
            if (gated) {
                const bf16x8 z1 = *reinterpret_cast<const bf16x8 *>(z + a.cols + c);
                bf16x8 u;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float d = (float)g[i], x = (float)z0[i];
                    o[i] = (__bf16)(d * (float)z1[i] * act_one_grad(a.act, x));
                    u[i] = (__bf16)(d * act_one(a.act, x));
                }
                *reinterpret_cast<bf16x8 *>(dz + a.cols + c) = u;
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    o[i] = (__bf16)((float)g[i] * act_one_grad(a.act, (float)z0[i]));
            }
            *reinterpret_cast<bf16x8 *>(dz + c) = o;
        }
    }
}

struct BiasGradArgs {
    int32_t rows, experts, cols, act;  // cols: out_features
    const int32_t *expert_off;
    const uint16_t *grad_out, *preact;  // preact unused without an activation
    float *grad_bias;                   // [experts, cols]
};

constexpr int kBiasSlices = kTileWaves, kBiasLds = kBiasSlices * (kWave * 8 + 8) * 4;

// Column sums of an expert's dz in fp32, from its factors rather than the rounded
// dz: a block takes 512 columns, its eight waves every eighth row; the waves'
// sums are added in order, so the result does not vary.
__device__ inline void bias_grad(const BiasGradArgs &a, int e, int col_block, uint8_t *lds)
{
    float(*part)[kWave * 8 + 8] = reinterpret_cast<float(*)[kWave * 8 + 8]>(lds);
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x / kWave);
    const int c = col_block * kWave * 8 + lane * 8;
    const int r0 = clamp_row(a.expert_off, e, a.rows), r1 = clamp_row(a.expert_off, e + 1, a.rows);
    const bool gated = act_gated(a.act);
    const int gcols = gated ? a.cols / 2 : a.cols;
    const bool up = gated && c >= gcols;  // out_features is a multiple of 16: never both in 8
    const int gc = up ? c - gcols : c;
    float s[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    // kRows rows' loads before the first is used; kFactors: 0 grad_out alone, 1 with z,
    // 2 with the gate's z and the up row
    const auto add_rows = [&](auto rows, auto factors, int r) {
        constexpr int kRows = decltype(rows)::value, kFactors = decltype(factors)::value;
        bf16x8 v[kRows][kFactors + 1];
#pragma unroll
        for (int b = 0; b < kRows; ++b) {
            const size_t row = (size_t)(r + b * kBiasSlices);
            v[b][0] = *reinterpret_cast<const bf16x8 *>(a.grad_out + row * gcols + gc);
            if constexpr (kFactors >= 1) {
                const uint16_t *z = a.preact + row * a.cols + gc;
                v[b][1] = *reinterpret_cast<const bf16x8 *>(z);
                if constexpr (kFactors >= 2)
                    v[b][2] = *reinterpret_cast<const bf16x8 *>(z + gcols);
            }
        }
#pragma unroll
        for (int b = 0; b < kRows; ++b)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float d = (float)v[b][0][i];
                if constexpr (kFactors == 0) {
                    s[i] += d;
                } else {
                    const float x = (float)v[b][1][i];
                    if constexpr (kFactors == 1)
                        s[i] += d * (up ? act_one(a.act, x) : act_one_grad(a.act, x));
                    else
                        s[i] += d * act_one_grad(a.act, x) * (float)v[b][2][i];
                }
            }
    };
    // (One row at a time, every step of a busy expert waits for memory: the biases
    // alone, 3808 rows of 4096 with SwiGLU, 792 us, so 410 to 450, most of it act'.)
    const auto add_all = [&](auto factors) {
        constexpr int kRows = 4;
        int r = r0 + wave;
        for (; r + (kRows - 1) * kBiasSlices < r1; r += kRows * kBiasSlices)
            add_rows(Count<kRows>(), factors, r);
        for (; r < r1; r += kBiasSlices)
            add_rows(Count<1>(), factors, r);
    };
    if (c < a.cols) {
        if (a.act == kActNone)
            add_all(Count<0>());
        else if (gated && !up)
            add_all(Count<2>());
        else
            add_all(Count<1>());
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        part[wave][lane * 8 + i] = s[i];
    __syncthreads();
    const int col = threadIdx.x;
    if (col_block * kWave * 8 + col >= a.cols)
        return;
    float sum = 0.0f;
#pragma unroll
    for (int w = 0; w < kBiasSlices; ++w)
        sum += part[w][col];
    a.grad_bias[(size_t)e * a.cols + col_block * kWave * 8 + col] = sum;
}

// The gradients that follow from dz in one launch: first the biases' column blocks,
// which take longest where one expert is busy (at the end 32768 rows of 4096 x 4096
// over 64 experts, skewed, took 325 us more with biases, so 100), then the blocks
// of the weights' tiles, then the rows', any of them none.  Each XCD's run of a part starts afresh, so
// a part holds a multiple of 8 blocks.  (One after the other, 122 rows of 256 x 520 over 8
// experts took 36 us, of which each launch was 6 to 10; together 15.  32768 rows
// of 4096 x 4096 over 64 experts, skewed: 2.3 to 2.4 ms, 0.92 to 0.95 PFLOP/s.)
struct GradArgs {
    ProductArgs weight, input;
    BiasGradArgs bias;
    int32_t bias_blocks, weight_blocks, bias_cols;  // bias_cols: column blocks of an expert
};

template <int kInputGroups>
__global__ __launch_bounds__(kTileWaves *kWave) void k_product_grads(const GradArgs a)
{
#ifdef __HIP_DEVICE_COMPILE__
    constexpr int kBytes = TileLds<false, 4>::kBytes;
    static_assert(kBytes >= kBiasLds, "the smaller parts fit");
    __shared__ __align__(1024) uint8_t lds[kBytes];
    int block = blockIdx.x;
    if (block < a.bias_blocks) {
        const int e = block / a.bias_cols;
        if (e < a.bias.experts)
            bias_grad(a.bias, e, block - e * a.bias_cols, lds);
        return;
    }
    block -= a.bias_blocks;
    if (block < a.weight_blocks)
        product_tile<kGradWeight, kTypeBf16, 4>(a.weight, block, lds);
    else
        product_tile<kGradInput, kTypeBf16, kInputGroups>(a.input, block - a.weight_blocks, lds);
#endif
}

}  // namespace epdc_layer
