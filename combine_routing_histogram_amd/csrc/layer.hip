// layer.hip -- host side of the C ABI declared in include/epdc_layer.h: argument
// checks, the choice of kernel form, and the launches.  Nothing here waits for
// the device or allocates.
#include "epdc_layer.h"
#include "layer_product.hpp"
#include "layer_gate.hpp"
#include "layer_rows.hpp"
#include "layer_few.hpp"

#include <hip/hip_runtime.h>

#include <cstdarg>
#include <cstdio>
#include <initializer_list>
#include <string>

using namespace epdc_layer;

namespace {

thread_local std::string g_last_error;

epdc_status fail(epdc_status s, const char *fmt, ...)
{
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    g_last_error = buf;
    return s;
}

epdc_status ok()
{
    g_last_error.clear();
    return EPDC_SUCCESS;
}

bool aligned(const void *p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

// An array of a call, NULL if it has none or does not touch it.
struct Array {
    const char *name;
    const void *at;
    int64_t bytes;
};

bool overlap(const Array &a, const Array &b)
{
    const uintptr_t p = (uintptr_t)a.at, q = (uintptr_t)b.at;
    return p && q && p < q + (uint64_t)b.bytes && q < p + (uint64_t)a.bytes;
}

// An output that shares no byte with the others; SUCCESS sets no message.
epdc_status check_apart(const Array &out, std::initializer_list<Array> others)
{
    for (const Array &o : others)
        if (overlap(out, o))
            return fail(EPDC_ERR_INVALID_ARGS, "%s may not overlap %s", out.name, o.name);
    return EPDC_SUCCESS;
}

template <typename F>
epdc_status launch(const char *name, F &&f)
{
    f();
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess)
        return fail(EPDC_ERR_GPU_OP, "%s launch failed: %s", name, hipGetErrorString(err));
    return EPDC_SUCCESS;
}

// ---- gate -------------------------------------------------------------------

constexpr int kMaxFeatures = 1 << 20;
constexpr int64_t kMaxExpertBytes = (int64_t)0x7fff0000;
// int8: sums of products, of up to 2^14 each, stay below 2^31
constexpr int kMaxInt8Features = (1 << 17) - 16;
constexpr int64_t kMaxThreads = (int64_t)0xffffffff;  // of a launch, in all its blocks

int gate_blocks(int64_t tokens, int experts, int limit)
{
    const int64_t per = kGateThreads / gate_lanes(tokens, experts);
    const int64_t b = (tokens + per - 1) / per;
    return (int)(b < 1 ? 1 : (b < limit ? b : limit));
}

epdc_status check_gate(const epdc_gate_args *g)
{
    if (!g)
        return fail(EPDC_ERR_INVALID_ARGS, "args is NULL");
    if (g->num_tokens < 0)
        return fail(EPDC_ERR_INVALID_ARGS, "num_tokens must be >= 0");
    if (g->num_experts < 1 || g->num_experts > kMaxExperts)
        return fail(EPDC_ERR_INVALID_ARGS, "num_experts must be in [1, %d]", kMaxExperts);
    if (g->topk < 1 || g->topk > kMaxTopk || g->topk > g->num_experts)
        return fail(EPDC_ERR_INVALID_ARGS, "topk must be in [1, %d] and at most num_experts",
                    kMaxTopk);
    if (g->score != EPDC_GATE_SOFTMAX && g->score != EPDC_GATE_SIGMOID)
        return fail(EPDC_ERR_INVALID_ARGS, "unknown score %d", g->score);
    if (g->logits_dtype != EPDC_DT_FP32 && g->logits_dtype != EPDC_DT_BF16)
        return fail(EPDC_ERR_INVALID_ARGS, "logits must be fp32 or bf16");
    if (!(g->scale > 0.0f) || g->scale > 3.4e38f)
        return fail(EPDC_ERR_INVALID_ARGS, "scale must be positive and finite");
    if (g->num_tokens > 0 && !g->logits)
        return fail(EPDC_ERR_INVALID_ARGS, "logits is required");
    if (!aligned(g->logits, 16) || !aligned(g->bias, 4))
        return fail(EPDC_ERR_INVALID_ARGS, "logits must be 16-byte aligned, bias 4-byte aligned");
    return EPDC_SUCCESS;
}

GateArgs gate_args(const epdc_gate_args *g)
{
    GateArgs a = {};
    a.tokens = g->num_tokens;
    a.experts = g->num_experts;
    a.topk = g->topk;
    a.score = g->score;
    a.renorm = g->renormalize != 0;
    a.bf16 = g->logits_dtype == EPDC_DT_BF16;
    a.scale = g->scale;
    a.logits = g->logits;
    a.bias = g->bias;
    a.mask = g->mask;
    return a;
}

// f(lanes, slots) with the lanes of a token and the logits of a lane
template <typename F>
void gate_form(int64_t tokens, int experts, F &&f)
{
    const int step = experts <= 64 ? 0 : experts <= 128 ? 1 : experts <= 256 ? 2 : 3;
    if (gate_lanes(tokens, experts) == 64) {
        switch (step) {
        case 0: f(Count<64>(), Count<1>()); break;
        case 1: f(Count<64>(), Count<2>()); break;
        case 2: f(Count<64>(), Count<4>()); break;
        default: f(Count<64>(), Count<8>()); break;
        }
    } else {
        switch (step) {
        case 0: f(Count<16>(), Count<4>()); break;
        case 1: f(Count<16>(), Count<8>()); break;
        case 2: f(Count<16>(), Count<16>()); break;
        default: f(Count<16>(), Count<32>()); break;
        }
    }
}

template <bool kBalance>
void launch_gate(int grid, size_t lds, hipStream_t st, const GateArgs &a)
{
    gate_form(a.tokens, a.experts, [&](auto lanes, auto slots) {
        k_gate<decltype(lanes)::value, decltype(slots)::value, kBalance>
            <<<grid, kGateThreads, lds, st>>>(a);
    });
}

void launch_gate_backward(int grid, hipStream_t st, const GateArgs &a)
{
    gate_form(a.tokens, a.experts, [&](auto lanes, auto slots) {
        k_gate_backward<decltype(lanes)::value, decltype(slots)::value>
            <<<grid, kGateThreads, 0, st>>>(a);
    });
}

// ---- products -----------------------------------------------------------------

bool product_type(int32_t dtype, int *type)
{
    switch (dtype) {
    case EPDC_DT_BF16: *type = kTypeBf16; return true;
    case EPDC_DT_E4M3: *type = kTypeE4m3; return true;
    case EPDC_DT_INT8: *type = kTypeInt8; return true;
    default: return false;
    }
}

// What a contraction is a multiple of: 16 bytes; e4m3 a block of scales.
int unit_features(int type) { return type == kTypeE4m3 ? 128 : type == kTypeInt8 ? 16 : 8; }

// Scales of `rows` rows (one per row or per 128 columns) and of a weight.
int64_t row_scales(int type, int64_t rows, int64_t features)
{
    return type == kTypeE4m3 ? rows * (features / 128) : type == kTypeInt8 ? rows : 0;
}
int64_t weight_scales(int type, int64_t experts, int64_t out, int64_t in)
{
    return type == kTypeE4m3 ? experts * ((out + 127) / 128) * (in / 128)
                             : type == kTypeInt8 ? experts * out : 0;
}

epdc_status check_product(const epdc_product_args *p)
{
    if (!p)
        return fail(EPDC_ERR_INVALID_ARGS, "args is NULL");
    if (p->rows < 0 || p->rows > (1 << 30))
        return fail(EPDC_ERR_INVALID_ARGS, "rows must be in [0, 2^30]");
    if (p->num_experts < 1 || p->num_experts > kMaxExperts)
        return fail(EPDC_ERR_INVALID_ARGS, "num_experts must be in [1, %d]", kMaxExperts);
    if (p->expected_rows < 0)
        return fail(EPDC_ERR_INVALID_ARGS, "expected_rows must be >= 0");
    if (p->activation < EPDC_ACT_NONE || p->activation > EPDC_ACT_GEGLU)
        return fail(EPDC_ERR_INVALID_ARGS, "unknown activation %d", p->activation);
    int type;
    if (!product_type(p->dtype, &type))
        return fail(EPDC_ERR_INVALID_ARGS, "operands must be bf16 or e4m3 or int8");
    const int unit_in = unit_features(type), unit_out = act_gated(p->activation) ? 16 : 8;
    const int most_in = type == kTypeInt8 ? kMaxInt8Features : kMaxFeatures;
    if (p->in_features < unit_in || p->in_features > most_in || p->in_features % unit_in)
        return fail(EPDC_ERR_INVALID_ARGS, "in_features must be a multiple of %d, at most %d",
                    unit_in, most_in);
    if (p->out_features < unit_out || p->out_features > kMaxFeatures ||
        p->out_features % unit_out)
        return fail(EPDC_ERR_INVALID_ARGS, "out_features must be a multiple of %d, at most 2^20",
                    unit_out);
    if ((int64_t)p->in_features * p->out_features * element_bytes(type) > kMaxExpertBytes)
        return fail(EPDC_ERR_INVALID_ARGS, "one expert's weight must be smaller than 2 GiB");
    if (!p->expert_off)
        return fail(EPDC_ERR_INVALID_ARGS, "expert_off is required");
    if (!aligned(p->expert_off, 4) || !aligned(p->bias, 16) || !aligned(p->scales, 4) ||
        !aligned(p->weight_scales, 4) || !aligned(p->input, 16) || !aligned(p->weight, 16))
        return fail(EPDC_ERR_INVALID_ARGS, "input, weight and bias must be 16-byte aligned, the "
                                           "other arrays 4-byte aligned");
    return EPDC_SUCCESS;
}

// The arrays that a product's arguments name.
struct Operands {
    Array input, scales, weight, weight_scales, bias, offsets;
};

Operands operands(const epdc_product_args &p)
{
    const int64_t rows = p.rows, experts = p.num_experts, in = p.in_features, of = p.out_features;
    int type = kTypeBf16;
    product_type(p.dtype, &type);
    const int64_t elem = element_bytes(type);
    return {{"input", p.input, rows * in * elem},
            {"scales", p.scales, row_scales(type, rows, in) * 4},
            {"weight", p.weight, experts * of * in * elem},
            {"weight_scales", p.weight_scales, weight_scales(type, experts, of, in) * 4},
            {"bias", p.bias, experts * of * 4},
            {"expert_off", p.expert_off, (experts + 1) * 4}};
}

int64_t mean_rows(const epdc_product_args &p)
{
    const int rows = p.expected_rows > 0 && p.expected_rows < p.rows ? p.expected_rows : p.rows;
    return rows / p.num_experts;
}

// Row tiles that `experts` experts with at most `rows` rows between them can
// make; their counts are known to the device only.
int64_t row_tile_bound(int64_t rows, int experts, int bm)
{
    const int64_t with_rows = rows < experts ? rows : experts;
    return (rows + with_rows * (bm - 1)) / bm;
}

// Blocks for `tiles` tiles: whole rounds of one run per XCD (tile_number).
epdc_status grid_of(int64_t tiles, int threads, int *grid)
{
    const int64_t round = kXcds * kRun, g = (tiles + round - 1) / round * round;
    if (g > kMaxThreads / threads)
        return fail(EPDC_ERR_INVALID_ARGS, "more tiles than a launch can hold");
    *grid = (int)g;
    return EPDC_SUCCESS;
}

// Column tiles of a product, and the blocks of its grid.
template <int kProduct, int kGroups>
epdc_status plan_tiles(ProductArgs &a, int *grid)
{
    const int cols_per_tile =
        kProduct == kForward && act_gated(a.act) ? kTileCols / 2 : kTileCols;
    a.col_tiles = (a.out_cols + cols_per_tile - 1) / cols_per_tile;
    int64_t tiles;
    if (kProduct == kGradWeight) {
        a.row_tiles = (a.out_rows + kGroups * 64 - 1) / (kGroups * 64);
        tiles = (int64_t)a.experts * a.row_tiles * a.col_tiles;
    } else {
        tiles = row_tile_bound(a.rows, a.experts, kGroups * 64) * a.col_tiles;
    }
    return grid_of(tiles, kTileWaves * kWave, grid);
}

template <int kType, int kGroups>
epdc_status launch_tile(hipStream_t st, ProductArgs &a)
{
    int grid;
    const epdc_status s = plan_tiles<kForward, kGroups>(a, &grid);
    if (s != EPDC_SUCCESS)
        return s;
    return launch("k_product_tile", [&] {
        k_product_tile<kType, kGroups><<<grid, kTileWaves * kWave, 0, st>>>(a);
    });
}

// f(whether rows of weight are whole lines); e4m3's are but where w is not at one's start.
template <int kType, typename F>
void line_form(const void *w, int64_t row_bytes, F &&f)
{
    if constexpr (kType == kTypeE4m3) {
        f(Count<1>());
    } else {
        if (((uintptr_t)w | (uintptr_t)row_bytes) % kStepBytes == 0)
            f(Count<1>());
        else
            f(Count<0>());
    }
}

template <int kType, int kMI>
epdc_status launch_stream(hipStream_t st, ProductArgs &a)
{
    a.col_tiles = (a.out_cols + 15) / 16;
    int grid;
    const epdc_status s = grid_of(row_tile_bound(a.rows, a.experts, kMI * 16) * a.col_tiles,
                                  kStreamWaves * kWave, &grid);
    if (s != EPDC_SUCCESS)
        return s;
    return launch("k_product_stream", [&] {
        line_form<kType>(a.q, a.q_bytes, [&](auto whole) {
            constexpr bool kWhole = decltype(whole)::value;
            if (act_gated(a.act))
                k_product_stream<kType, kMI, true, kWhole>
                    <<<grid, kStreamWaves * kWave, 0, st>>>(a);
            else
                k_product_stream<kType, kMI, false, kWhole>
                    <<<grid, kStreamWaves * kWave, 0, st>>>(a);
        });
    });
}

template <int kType>
epdc_status launch_forward(hipStream_t st, ProductArgs &a, int64_t mean)
{
    constexpr bool kE4m3 = kType == kTypeE4m3, kInt8 = kType == kTypeInt8;
    // By mean rows per expert, all that is known here of the experts' counts.  The
    // streamed form reads the weights fastest but once per 16 (32) rows of an
    // expert, the tiles once per 64 (256) at 85% of that rate.  Measured over 64
    // experts of 4096 x 4096, streamed (16), streamed (32), 64-row tiles: bf16 mean
    // 8: 327, 346, 393 us; 12: 355, 337, 394; 24: -, 366, 405; 32: -, 578, 409.
    // e4m3: 12: 195, 239, 238; 16: 261, 253, 236 (with 32 rows its registers
    // leave too few waves).  64- against 256-row tiles, bf16: 40 rows 399, 410; 64:
    // 429, 441; 80: 462, 449; 128: 520, 475.  e4m3: 40: 242, 243; 64: 250, 249; 80:
    // 280, 254; 128: 328, 270.  int8, all four: 12: 194, 197, 221, 236; 16: 256, 204, 225,
    // 241; 20: -, 218, 227, 241; 24: 356, 246, 230, 245; 96: 64- and 256-row tiles 261,
    // 264; 128: 287, 273; 160: 334, 289.
    if (mean <= (kType == kTypeBf16 ? 10 : 12))
        return launch_stream<kType, 1>(st, a);
    if constexpr (!kE4m3) {
        if (mean <= (kInt8 ? 20 : 24))
            return launch_stream<kType, 2>(st, a);
    }
    if (mean <= (kInt8 ? 96 : 64))
        return launch_tile<kType, 1>(st, a);
    return launch_tile<kType, 4>(st, a);
}

void launch_combine_grad(int grid, hipStream_t st, const CombineGradArgs &a)
{
    switch (a.topk) {
    case 1: k_combine_grad<1><<<grid, kCombineGradThreads, 0, st>>>(a); break;
    case 2: k_combine_grad<2><<<grid, kCombineGradThreads, 0, st>>>(a); break;
    case 4: k_combine_grad<4><<<grid, kCombineGradThreads, 0, st>>>(a); break;
    case 6: k_combine_grad<6><<<grid, kCombineGradThreads, 0, st>>>(a); break;
    case 8: k_combine_grad<8><<<grid, kCombineGradThreads, 0, st>>>(a); break;
    default: k_combine_grad<0><<<grid, kCombineGradThreads, 0, st>>>(a); break;
    }
}

// ---- rows -----------------------------------------------------------------------

// Blocks for `rows` rows, kTeams of them to a block at a time.
int row_blocks(int64_t rows, int threads, int teams)
{
    const int64_t most = kMaxThreads / threads < (1 << 20) ? kMaxThreads / threads : 1 << 20;
    const int64_t b = (rows + teams - 1) / teams;
    return (int)(b < most ? b : most);
}

template <int kWaves>
int team_blocks(int64_t rows)
{
    constexpr int kThreads = team_threads(kWaves);
    return row_blocks(rows, kThreads, kThreads / (kWaves * kWave));
}

// f(waves of a team, vectors of a lane) for rows of `vecs` vectors.  Eight waves of two
// where four of four would do: 4096 x 7168 into bf16 and e4m3 47 us for 52, the gradient
// of 8192 x 7168 94 for 122, one row 2.7 for 3.1.
template <typename F>
void row_form(int vecs, F &&f)
{
    if (vecs <= 64)
        f(Count<1>(), Count<1>());
    else if (vecs <= 256)
        f(Count<4>(), Count<1>());
    else if (vecs <= 512)
        f(Count<4>(), Count<2>());
    else if (vecs <= 1024)
        f(Count<8>(), Count<2>());
    else if (vecs <= 2048)
        f(Count<16>(), Count<2>());
    else
        f(Count<16>(), Count<4>());
}

epdc_status check_norm(const epdc_norm_args *n)
{
    if (!n)
        return fail(EPDC_ERR_INVALID_ARGS, "args is NULL");
    if (n->rows < 0 || n->rows > (1 << 30))
        return fail(EPDC_ERR_INVALID_ARGS, "rows must be in [0, 2^30]");
    if (n->features < 8 || n->features > kMaxNormFeatures || n->features % 8)
        return fail(EPDC_ERR_INVALID_ARGS, "features must be a multiple of 8, at most %d",
                    kMaxNormFeatures);
    if (n->weight_dtype != EPDC_DT_BF16 && n->weight_dtype != EPDC_DT_FP32)
        return fail(EPDC_ERR_INVALID_ARGS, "weight must be bf16 or fp32");
    if (!(n->eps >= 0.0f) || n->eps > 3.4e38f)
        return fail(EPDC_ERR_INVALID_ARGS, "eps must be finite and not negative");
    if (!aligned(n->input, 16) || !aligned(n->residual, 16) || !aligned(n->weight, 16))
        return fail(EPDC_ERR_INVALID_ARGS, "input, residual and weight must be 16-byte aligned");
    if (n->rows > 0 && (!n->input || !n->weight))
        return fail(EPDC_ERR_INVALID_ARGS, "input and weight are required");
    return EPDC_SUCCESS;
}

NormArgs norm_args(const epdc_norm_args &n)
{
    NormArgs a = {};
    a.rows = n.rows;
    a.vecs = n.features / 8;
    a.weight_bf16 = n.weight_dtype == EPDC_DT_BF16;
    a.features = (float)n.features;
    a.eps = n.eps;
    a.input = static_cast<const uint8_t *>(n.input);
    a.residual = static_cast<const uint8_t *>(n.residual);
    a.weight = static_cast<const uint8_t *>(n.weight);
    return a;
}

template <int kCodes>
void launch_norm(hipStream_t st, const NormArgs &a)
{
    row_form(a.vecs, [&](auto waves, auto vecs) {
        constexpr int kWaves = decltype(waves)::value;
        k_rms_norm<kWaves, decltype(vecs)::value, kCodes>
            <<<team_blocks<kWaves>(a.rows), team_threads(kWaves), 0, st>>>(a);
    });
}

// Blocks that share the rows of a gradient: each of their teams leaves a row of fp32
// sums, so no more of them than the chip holds at once.  (8192 x 7168, eight waves: 256
// blocks 94 and 4.9 us, 512 96 and 5.1.)
constexpr int norm_grad_blocks(int waves) { return waves < 8 ? 512 : 256; }
constexpr int norm_grad_teams(int waves)
{
    return norm_grad_blocks(waves) * (team_threads(waves) / (waves * kWave));
}

int64_t norm_scratch(int features)
{
    int teams = 0;
    row_form(features / 8, [&](auto waves, auto) {
        teams = norm_grad_teams(decltype(waves)::value);
    });
    return (int64_t)teams * features * (int64_t)sizeof(float);
}

// Columns of a scale of a format of codes; 0 for none of them.
int code_unit(int32_t dtype)
{
    return dtype == EPDC_DT_E4M3 ? kCodeBlock : dtype == EPDC_DT_INT8 ? 16 : 0;
}

template <int kWaves, int kV>
void launch_int8(hipStream_t st, const QuantArgs &a)
{
    k_quantize_int8<kWaves, kV><<<team_blocks<kWaves>(a.rows), team_threads(kWaves), 0, st>>>(a);
}

// ---- a layer for few tokens -----------------------------------------------------------

epdc_status check_few(const epdc_few_args *args, int *of_type)
{
    if (!args)
        return fail(EPDC_ERR_INVALID_ARGS, "args is NULL");
    const epdc_few_args &p = *args;
    if (p.num_tokens < 0 || p.num_tokens > kFewTokens)
        return fail(EPDC_ERR_INVALID_ARGS, "num_tokens must be in [0, %d]", kFewTokens);
    if (p.topk < 1 || p.topk > kMaxTopk)
        return fail(EPDC_ERR_INVALID_ARGS, "topk must be in [1, %d]", kMaxTopk);
    if (p.num_experts < 1 || p.num_experts > kMaxExperts || p.first_expert < 0 ||
        p.first_expert > kMaxExperts)
        return fail(EPDC_ERR_INVALID_ARGS,
                    "num_experts must be in [1, %d] and first_expert in [0, %d]", kMaxExperts,
                    kMaxExperts);
    if (p.activation < EPDC_ACT_NONE || p.activation > EPDC_ACT_GEGLU)
        return fail(EPDC_ERR_INVALID_ARGS, "unknown activation %d", p.activation);
    int type;
    if (!product_type(p.dtype, &type))
        return fail(EPDC_ERR_INVALID_ARGS, "weights must be bf16, e4m3 or int8");
    const int unit = unit_features(type);
    if (p.hidden < unit || p.hidden > kMaxFeatures || p.hidden % unit || p.inner < unit ||
        p.inner > kMaxFeatures || p.inner % unit)
        return fail(EPDC_ERR_INVALID_ARGS, "hidden and inner must be multiples of %d, at most %d",
                    unit, kMaxFeatures);
    const bool gated = act_gated(p.activation);
    const int64_t H = p.hidden, I = p.inner, up = gated ? 2 * I : I;
    if (up * H * element_bytes(type) > kMaxExpertBytes ||
        (int64_t)p.num_tokens * p.topk * I * 2 > kMaxExpertBytes)
        return fail(EPDC_ERR_INVALID_ARGS,
                    "one expert's weight, and the rows of h, must be smaller than 2 GiB");
    *of_type = type;
    return EPDC_SUCCESS;
}

template <int kType, int kRows>
epdc_status launch_few(hipStream_t st, const FewArgs &a)
{
    const int64_t tiles =
        row_tile_bound(a.tokens * a.topk, a.experts, kRows) * ((a.inner + 15) / 16);
    const int up = (int)(tiles < kFewUpBlocks ? tiles : kFewUpBlocks);
    const int down = (a.hidden + 15) / 16 * a.splits;
    epdc_status s = launch("k_few_up", [&] {
        line_form<kType>(a.w1, (int64_t)a.hidden * element_bytes(kType), [&](auto whole) {
            constexpr bool kWhole = decltype(whole)::value;
            if (act_gated(a.act))
                k_few_up<kType, kRows, true, kWhole><<<up, kFewUpWaves * kWave, 0, st>>>(a);
            else
                k_few_up<kType, kRows, false, kWhole><<<up, kFewUpWaves * kWave, 0, st>>>(a);
        });
    });
    if (s == EPDC_SUCCESS)
        s = launch("k_few_down", [&] {
            line_form<kType>(a.w2, (int64_t)a.inner * element_bytes(kType), [&](auto whole) {
                k_few_down<kType, kRows, decltype(whole)::value>
                    <<<down, kFewDownWaves * kWave, 0, st>>>(a);
            });
        });
    return s;
}

// Blocks that share a column tile of the down product: as many as take the least time, in
// rounds of 512 blocks (two to a CU), each as long as a wave's steps and four more, which the
// routing and joining the blocks' sums come to; but no wave fewer than four steps (40 tiles,
// 20 e4m3 experts of 1280 columns: 11.9 us with 6 blocks a tile, 15.8 with 8).  With one block
// a tile and with these, us: 64 tiles, 8 bf16 of 2048 23.4, 11.3; the 40 tiles 34.4, 11.9; 128
// tiles, 32 int8 of 1024 28.6, 21.7; 129 tiles, 32 int8 of 1040 40.4, 33.0; 257 tiles, 82
// int8 of 2064 199, 148.
int few_splits(int type, int64_t pairs, int experts, int hidden, int inner)
{
    const int tiles = (hidden + 15) / 16, step = kStepBytes / element_bytes(type);
    const int64_t active = pairs < experts ? pairs : experts;
    const int64_t steps = active * ((inner + step - 1) / step);
    int best = 1;
    double least = 0.0;
    for (int n = 1; n <= kFewMostSplits && (n == 1 || n * 4 * kFewDownWaves <= steps); ++n) {
        const int64_t rounds = ((int64_t)tiles * n + 511) / 512;
        const double time = (double)rounds * ((double)steps / (n * kFewDownWaves) + 4.0);
        if (n == 1 || time < least) {
            best = n;
            least = time;
        }
    }
    return best;
}

// Scratch: h, then the tickets and the sums of the down product's blocks.
struct FewScratch {
    int splits;
    int64_t h, ticket, partial;   // bytes of each, multiples of 256
    int64_t bytes() const { return h + ticket + partial; }
};

FewScratch few_scratch(const epdc_few_args &p, int type)
{
    const auto whole = [](int64_t n) { return (n + 255) / 256 * 256; };
    const int64_t pairs = (int64_t)p.num_tokens * p.topk, tiles = (p.hidden + 15) / 16;
    FewScratch s;
    s.splits = few_splits(type, pairs, p.num_experts, p.hidden, p.inner);
    s.h = whole(pairs * p.inner * 2);
    s.ticket = s.splits > 1 ? whole(tiles * 4) : 0;
    s.partial = s.splits > 1 ? whole(tiles * s.splits * p.num_tokens * 16 * 4) : 0;
    return s;
}

template <int kType>
epdc_status launch_few_rows(hipStream_t st, const FewArgs &a)
{
    // By the mean rows of an expert: an expert of more rows than a unit's is read once per
    // unit.  64 tokens, experts of 4096 x 1024, us of both launches with units of 4, 16, 32
    // rows, int8: 1: 100, 107, 138; 2: 139, 144, 175; 4: 194, 167, 202; 10: 354, 196, 220;
    // 16 (32 experts): 265, 139, 136; 32 (16 experts): 239, 124, 118.  bf16, 16 and 32: 1:
    // 168, 176; 10: 314, 320; 16: 220, 179; 32: 183, 142.  (Even routing; one expert of far
    // more rows than the mean is read once per unit of its own.)
    const int mean = a.tokens * a.topk / a.experts;
    if constexpr (kType != kTypeBf16) {
        if (a.tokens <= kFewLineRows || mean <= 2)
            return launch_few<kType, kFewLineRows>(st, a);
    }
    if (a.tokens <= 16 || mean <= 12)
        return launch_few<kType, 16>(st, a);
    return launch_few<kType, 32>(st, a);
}

}  // namespace

extern "C" {

epdc_status epdc_gate_scratch_bytes(int32_t max_tokens, int32_t num_experts, size_t *bytes)
{
    if (max_tokens < 0 || num_experts < 1 || num_experts > kMaxExperts || !bytes)
        return fail(EPDC_ERR_INVALID_ARGS, "max_tokens >= 0, num_experts in [1, %d] and bytes "
                                           "are required", kMaxExperts);
    // the most blocks a call of up to max_tokens tokens takes: a wave per token
    // needs more of them than 16 lanes
    const int64_t wave = gate_wave_tokens(num_experts);
    const int a = gate_blocks(max_tokens < wave ? max_tokens : wave, num_experts, kGateMaxBlocks);
    const int b = gate_blocks(max_tokens, num_experts, kGateMaxBlocks);
    *bytes = 256 + sizeof(float) * (size_t)((a > b ? a : b) + kGateMaxFan) *
                       (size_t)gate_partial_words(num_experts);
    return ok();
}

epdc_status epdc_gate(const epdc_gate_args *args, void *stream, float *weights, int32_t *indices,
                      int32_t *counts, float *losses, void *scratch)
{
    epdc_status s = check_gate(args);
    if (s != EPDC_SUCCESS)
        return s;
    if (args->num_tokens > 0 && (!weights || !indices))
        return fail(EPDC_ERR_INVALID_ARGS, "weights and indices are required");
    const bool balance = counts != nullptr;
    if ((losses != nullptr) != balance || (scratch != nullptr) != balance)
        return fail(EPDC_ERR_INVALID_ARGS,
                    "counts, losses and scratch must all be given or all NULL");
    if (!aligned(weights, 4) || !aligned(indices, 4) || !aligned(counts, 4) ||
        !aligned(losses, 4) || !aligned(scratch, 256))
        return fail(EPDC_ERR_INVALID_ARGS,
                    "scratch must be 256-byte aligned, the other outputs 4-byte aligned");
    if (args->num_tokens == 0 && !balance)
        return ok();
    GateArgs a = gate_args(args);
    a.weights = weights;
    a.indices = indices;
    a.counts = counts;
    a.losses = losses;
    hipStream_t st = static_cast<hipStream_t>(stream);
    if (balance) {
        a.ticket = static_cast<uint32_t *>(scratch);
        a.partial = reinterpret_cast<float *>(static_cast<uint8_t *>(scratch) + 256);
        const int grid = gate_blocks(a.tokens, a.experts, kGateMaxBlocks);
        const size_t lds = sizeof(float) * ((size_t)a.experts + 1 +
                                            kGateThreads / 64 * (size_t)a.experts +
                                            kGateThreads / gate_lanes(a.tokens, a.experts));
        s = launch("k_gate", [&] { launch_gate<true>(grid, lds, st, a); });
    } else {
        s = launch("k_gate",
                   [&] { launch_gate<false>(gate_blocks(a.tokens, a.experts, 1 << 20), 0, st, a); });
    }
    return s == EPDC_SUCCESS ? ok() : s;
}

epdc_status epdc_gate_backward(const epdc_gate_args *args, void *stream, const int32_t *indices,
                               const float *grad_weights, const int32_t *counts,
                               const float *grad_losses, void *grad_logits)
{
    epdc_status s = check_gate(args);
    if (s != EPDC_SUCCESS)
        return s;
    if ((counts != nullptr) != (grad_losses != nullptr))
        return fail(EPDC_ERR_INVALID_ARGS, "counts and grad_losses must both be given or both NULL");
    if (args->num_tokens > 0 && (!grad_logits || (grad_weights && !indices)))
        return fail(EPDC_ERR_INVALID_ARGS,
                    "grad_logits is required, and indices with grad_weights");
    if (!aligned(grad_logits, 16) || !aligned(indices, 4) || !aligned(grad_weights, 4) ||
        !aligned(counts, 4) || !aligned(grad_losses, 4))
        return fail(EPDC_ERR_INVALID_ARGS,
                    "grad_logits must be 16-byte aligned, the other arrays 4-byte aligned");
    if (args->num_tokens == 0)
        return ok();
    GateArgs a = gate_args(args);
    a.in_indices = indices;
    a.grad_weights = grad_weights;
    a.in_counts = counts;
    a.grad_losses = grad_losses;
    a.grad_logits = grad_logits;
    s = launch("k_gate_backward", [&] {
        launch_gate_backward(gate_blocks(a.tokens, a.experts, 1 << 20),
                             static_cast<hipStream_t>(stream), a);
    });
    return s == EPDC_SUCCESS ? ok() : s;
}

epdc_status epdc_expert_product(const epdc_product_args *args, void *stream, const void *residual,
                                void *out, void *preact)
{
    epdc_status s = check_product(args);
    if (s != EPDC_SUCCESS)
        return s;
    int type = kTypeBf16;
    product_type(args->dtype, &type);
    const bool scaled = type != kTypeBf16;
    if (scaled != (args->scales != nullptr) || scaled != (args->weight_scales != nullptr))
        return fail(EPDC_ERR_INVALID_ARGS,
                    "scales and weight_scales belong to e4m3 and int8 operands, both of them");
    if (args->rows > 0 && (!args->input || !args->weight || !out))
        return fail(EPDC_ERR_INVALID_ARGS, "input, weight and out are required");
    if (!aligned(residual, 16) || !aligned(out, 16) || !aligned(preact, 16))
        return fail(EPDC_ERR_INVALID_ARGS, "residual, out and preact must be 16-byte aligned");
    if (args->rows == 0)
        return ok();
    const int cols =
        act_gated(args->activation) ? args->out_features / 2 : args->out_features;
    const Operands in = operands(*args);
    const Array to = {"out", out, (int64_t)args->rows * cols * 2},
                z = {"preact", preact, (int64_t)args->rows * args->out_features * 2},
                res = {"residual", residual, to.bytes};
    // out may be the residual: what is added to an element is read before it is written
    s = check_apart(to, {in.input, in.scales, in.weight, in.weight_scales, in.bias, in.offsets, z,
                         residual == out ? Array{} : res});
    if (s == EPDC_SUCCESS)
        s = check_apart(z, {in.input, in.scales, in.weight, in.weight_scales, in.bias, in.offsets,
                            res});
    if (s != EPDC_SUCCESS)
        return s;
    ProductArgs a = {};
    a.rows = args->rows;
    a.experts = args->num_experts;
    a.contract = args->in_features;
    a.p_bytes = a.q_bytes = args->in_features * element_bytes(type);
    a.weight_rows = args->out_features;
    a.act = args->activation;
    a.out_cols = cols;
    a.p = static_cast<const uint8_t *>(args->input);
    a.q = static_cast<const uint8_t *>(args->weight);
    a.scales = args->scales;
    a.weight_scales = args->weight_scales;
    a.bias = args->bias;
    a.residual = static_cast<const uint16_t *>(residual);
    a.expert_off = args->expert_off;
    a.out = static_cast<uint8_t *>(out);
    a.preact = static_cast<uint16_t *>(preact);
    hipStream_t st = static_cast<hipStream_t>(stream);
    const int64_t mean = mean_rows(*args);
    s = type == kTypeE4m3   ? launch_forward<kTypeE4m3>(st, a, mean)
        : type == kTypeInt8 ? launch_forward<kTypeInt8>(st, a, mean)
                            : launch_forward<kTypeBf16>(st, a, mean);
    return s == EPDC_SUCCESS ? ok() : s;
}

epdc_status epdc_expert_backward(const epdc_product_args *args, void *stream,
                                 const void *grad_out, const void *preact, void *dz,
                                 void *grad_input, void *grad_weight, int32_t grad_weight_dtype,
                                 float *grad_bias)
{
    epdc_status s = check_product(args);
    if (s != EPDC_SUCCESS)
        return s;
    if (args->dtype != EPDC_DT_BF16)
        return fail(EPDC_ERR_INVALID_ARGS, "the gradients take bf16 operands");
    if (grad_weight_dtype != EPDC_DT_BF16 && grad_weight_dtype != EPDC_DT_FP32)
        return fail(EPDC_ERR_INVALID_ARGS, "grad_weight must be bf16 or fp32");
    const bool act = args->activation != EPDC_ACT_NONE;
    if (args->rows > 0) {
        if (!grad_out || (grad_input && !args->weight) || (grad_weight && !args->input))
            return fail(EPDC_ERR_INVALID_ARGS, "grad_out is required, weight for grad_input and "
                                               "input for grad_weight");
        if (act && (!preact || (!dz && (grad_input || grad_weight))))
            return fail(EPDC_ERR_INVALID_ARGS, "an activation's gradient needs preact and dz");
    }
    if (!aligned(grad_out, 16) || !aligned(preact, 16) || !aligned(dz, 16) ||
        !aligned(grad_input, 16) || !aligned(grad_weight, 16) || !aligned(grad_bias, 4))
        return fail(EPDC_ERR_INVALID_ARGS,
                    "payload arrays must be 16-byte aligned, grad_bias 4-byte aligned");
    hipStream_t st = static_cast<hipStream_t>(stream);
    const int in = args->in_features, of = args->out_features;
    const bool with_dz = act && args->rows > 0 && (grad_input || grad_weight);
    {
        const Operands r = operands(*args);
        const bool gated = act_gated(args->activation), rows = args->rows > 0;
        const int64_t z_bytes = (int64_t)args->rows * of * 2;
        // what the products and the biases read behind the activation's gradient
        const Array dy = {"grad_out", rows ? grad_out : nullptr, gated ? z_bytes / 2 : z_bytes},
                    z = {"preact", act && rows ? preact : nullptr, z_bytes},
                    d = {"dz", with_dz ? dz : nullptr, z_bytes},
                    x = grad_weight && rows ? r.input : Array{},
                    w = grad_input && rows ? r.weight : Array{},
                    dy_read = with_dz && !grad_bias ? Array{} : dy,
                    z_read = grad_bias ? z : Array{};
        const Array gx = {"grad_input", rows ? grad_input : nullptr, r.input.bytes},
                    gw = {"grad_weight", grad_weight,
                          r.weight.bytes * (grad_weight_dtype == EPDC_DT_FP32 ? 2 : 1)},
                    gb = {"grad_bias", grad_bias, r.bias.bytes};
        // dz may take the place of one of its factors, element by element, unless
        // the biases' gradient reads that again
        const bool on_z = dz == preact && !grad_bias,
                   on_dy = dz == grad_out && !gated && !grad_bias;
        s = check_apart(d, {x, w, on_z ? Array{} : z, on_dy ? Array{} : dy, r.offsets});
        if (s == EPDC_SUCCESS)
            s = check_apart(gx, {x, w, d, dy_read, z_read, gw, gb, r.offsets});
        if (s == EPDC_SUCCESS)
            s = check_apart(gw, {x, w, d, dy_read, z_read, gb, r.offsets});
        if (s == EPDC_SUCCESS)
            s = check_apart(gb, {x, w, d, dy_read, z_read, r.offsets});
        if (s != EPDC_SUCCESS)
            return s;
    }
    ProductArgs a = {};
    a.rows = args->rows;
    a.experts = args->num_experts;
    a.weight_rows = of;
    a.p = static_cast<const uint8_t *>(with_dz ? dz : grad_out);
    a.p_bytes = of * 2;
    a.q_bytes = in * 2;
    a.out_cols = in;
    a.expert_off = args->expert_off;
    GradArgs g = {};
    g.weight = g.input = a;
    // few rows per expert: 64-row tiles for the rows' gradient, as in the forward
    const bool few = mean_rows(*args) <= 64;
    int64_t blocks = 0;
    if (grad_weight) {
        g.weight.out_rows = of;
        g.weight.out_fp32 = grad_weight_dtype == EPDC_DT_FP32;
        g.weight.q = static_cast<const uint8_t *>(args->input);
        g.weight.out = static_cast<uint8_t *>(grad_weight);
        s = plan_tiles<kGradWeight, 4>(g.weight, &g.weight_blocks);
        if (s != EPDC_SUCCESS)
            return s;
        blocks += g.weight_blocks;
    }
    if (grad_input && args->rows > 0) {
        g.input.contract = of;
        g.input.q = static_cast<const uint8_t *>(args->weight);
        g.input.out = static_cast<uint8_t *>(grad_input);
        int input_blocks;
        s = few ? plan_tiles<kGradInput, 1>(g.input, &input_blocks)
                : plan_tiles<kGradInput, 4>(g.input, &input_blocks);
        if (s != EPDC_SUCCESS)
            return s;
        blocks += input_blocks;
    }
    if (grad_bias) {
        g.bias.rows = args->rows;
        g.bias.experts = args->num_experts;
        g.bias.cols = of;
        g.bias.expert_off = args->expert_off;
        g.bias.act = args->activation;
        g.bias.grad_out = static_cast<const uint16_t *>(grad_out);
        g.bias.preact = static_cast<const uint16_t *>(preact);
        g.bias.grad_bias = grad_bias;
        g.bias_cols = (of + kWave * 8 - 1) / (kWave * 8);
        g.bias_blocks = (args->num_experts * g.bias_cols + kXcds - 1) / kXcds * kXcds;
        blocks += g.bias_blocks;
    }
    if (blocks > kMaxThreads / (kTileWaves * kWave))
        return fail(EPDC_ERR_INVALID_ARGS, "more tiles than a launch can hold");
    if (with_dz) {
        ActGradArgs d = {};
        d.rows = args->rows;
        d.experts = args->num_experts;
        d.act = args->activation;
        d.cols = act_gated(d.act) ? of / 2 : of;
        d.expert_off = args->expert_off;
        d.grad_out = static_cast<const uint16_t *>(grad_out);
        d.preact = static_cast<const uint16_t *>(preact);
        d.dz = static_cast<uint16_t *>(dz);
        const int rounds = (args->rows + kActRows - 1) / kActRows;
        s = launch("k_act_grad", [&] {
            k_act_grad<<<rounds < 16384 ? rounds : 16384, dim3(kWave, kActRows), 0, st>>>(d);
        });
        if (s != EPDC_SUCCESS)
            return s;
    }
    if (blocks > 0) {
        s = launch("k_product_grads", [&] {
            if (few)
                k_product_grads<1><<<(int)blocks, kTileWaves * kWave, 0, st>>>(g);
            else
                k_product_grads<4><<<(int)blocks, kTileWaves * kWave, 0, st>>>(g);
        });
        if (s != EPDC_SUCCESS)
            return s;
    }
    return ok();
}

epdc_status epdc_combine_backward(void *stream, int32_t num_tokens, int32_t topk, int32_t hidden,
                                  const int32_t *slot_of, const void *grad_output,
                                  const void *input, const float *weights, void *grad_input,
                                  float *grad_weights)
{
    if (num_tokens < 0 || topk < 1 || topk > kMaxTopk ||
        (int64_t)num_tokens * topk > (int64_t)(1 << 30))
        return fail(EPDC_ERR_INVALID_ARGS,
                    "num_tokens >= 0, topk in [1, %d] and num_tokens*topk <= 2^30 are required",
                    kMaxTopk);
    if (hidden < 8 || hidden % 8 != 0 || hidden > (1 << 24))
        return fail(EPDC_ERR_INVALID_ARGS, "hidden must be a positive multiple of 8, at most 2^24");
    if (num_tokens > 0 && (!slot_of || !grad_output || (grad_weights && !input)))
        return fail(EPDC_ERR_INVALID_ARGS, "slot_of and grad_output are required, and input with "
                                           "grad_weights");
    if (!aligned(slot_of, 4) || !aligned(grad_output, 16) || !aligned(input, 16) ||
        !aligned(weights, 4) || !aligned(grad_input, 16) || !aligned(grad_weights, 4))
        return fail(EPDC_ERR_INVALID_ARGS,
                    "rows must be 16-byte aligned, the other arrays 4-byte aligned");
    if (num_tokens == 0 || (!grad_input && !grad_weights))
        return ok();
    const int64_t pairs = (int64_t)num_tokens * topk;
    const Array slots = {"slot_of", slot_of, pairs * 4},
                dy = {"grad_output", grad_output, (int64_t)num_tokens * hidden * 2},
                x = {"input", grad_weights ? input : nullptr, pairs * hidden * 2},
                w = {"weights", weights, pairs * topk * 4},
                gx = {"grad_input", grad_input, x.bytes},
                gw = {"grad_weights", grad_weights, pairs * 4};
    // a row's gradient may take its place: the thread that writes an element has read it
    epdc_status apart = check_apart(gx, {slots, dy, grad_input == input ? Array{} : x, w, gw});
    if (apart == EPDC_SUCCESS)
        apart = check_apart(gw, {slots, dy, x, w});
    if (apart != EPDC_SUCCESS)
        return apart;
    CombineGradArgs a = {};
    a.tokens = num_tokens;
    a.topk = topk;
    a.row_vecs = hidden / 8;
    a.slot_of = slot_of;
    a.grad_output = static_cast<const uint8_t *>(grad_output);
    a.input = static_cast<const uint8_t *>(input);
    a.weights = weights;
    a.grad_input = static_cast<uint8_t *>(grad_input);
    a.grad_weights = grad_weights;
    hipStream_t st = static_cast<hipStream_t>(stream);
    // one launch, unless there are more tokens than it holds blocks
    constexpr int kBlocks = (int)(kMaxThreads / kCombineGradThreads);
    for (int64_t first = 0; first < num_tokens; first += kBlocks) {
        a.first = (int)first;
        const int grid = (int)(num_tokens - first < kBlocks ? num_tokens - first : kBlocks);
        const epdc_status s = launch("k_combine_grad", [&] { launch_combine_grad(grid, st, a); });
        if (s != EPDC_SUCCESS)
            return s;
    }
    return ok();
}

epdc_status epdc_rms_norm(const epdc_norm_args *args, void *stream, void *out, void *sum,
                          void *codes, float *scales, int32_t codes_dtype)
{
    epdc_status s = check_norm(args);
    if (s != EPDC_SUCCESS)
        return s;
    const int unit = code_unit(codes_dtype);
    if (codes_dtype != EPDC_DT_BF16 && !unit)
        return fail(EPDC_ERR_INVALID_ARGS, "codes must be e4m3 or int8, or bf16 for none");
    if (unit && args->features % unit)
        return fail(EPDC_ERR_INVALID_ARGS, "features must be a multiple of %d for these codes",
                    unit);
    if (!unit && (codes || scales))
        return fail(EPDC_ERR_INVALID_ARGS, "codes and scales belong to e4m3 and int8");
    if (!aligned(out, 16) || !aligned(sum, 16) || !aligned(codes, 16) || !aligned(scales, 4))
        return fail(EPDC_ERR_INVALID_ARGS,
                    "out, sum and codes must be 16-byte aligned, scales 4-byte aligned");
    if (args->rows == 0)
        return ok();
    if (unit && (!codes || !scales))
        return fail(EPDC_ERR_INVALID_ARGS, "codes and scales are required");
    if (!out && !unit)
        return fail(EPDC_ERR_INVALID_ARGS, "out or codes are required");
    const int64_t n = (int64_t)args->rows * args->features;
    const Array x = {"input", args->input, n * 2}, r = {"residual", args->residual, n * 2},
                w = {"weight", args->weight,
                     (int64_t)args->features * (args->weight_dtype == EPDC_DT_BF16 ? 2 : 4)};
    const Array o = {"out", out, n * 2}, t = {"sum", sum, n * 2}, c = {"codes", codes, n},
                f = {"scales", scales,
                     4 * (codes_dtype == EPDC_DT_E4M3 ? n / kCodeBlock : (int64_t)args->rows)};
    // a row is read whole before any of it is written: sum may take the place of what it adds
    s = check_apart(t, {sum == args->input ? Array{} : x, sum == args->residual ? Array{} : r, w,
                        o, c, f});
    if (s == EPDC_SUCCESS)
        s = check_apart(o, {x, r, w, c, f});
    if (s == EPDC_SUCCESS)
        s = check_apart(c, {x, r, w, f});
    if (s == EPDC_SUCCESS)
        s = check_apart(f, {x, r, w});
    if (s != EPDC_SUCCESS)
        return s;
    NormArgs a = norm_args(*args);
    a.out = static_cast<uint8_t *>(out);
    a.sum = static_cast<uint8_t *>(sum);
    a.codes = static_cast<uint8_t *>(codes);
    a.scales = scales;
    hipStream_t st = static_cast<hipStream_t>(stream);
    s = launch("k_rms_norm", [&] {
        if (codes_dtype == EPDC_DT_E4M3)
            launch_norm<kCodesE4m3>(st, a);
        else if (codes_dtype == EPDC_DT_INT8)
            launch_norm<kCodesInt8>(st, a);
        else
            launch_norm<kCodesNone>(st, a);
    });
    return s == EPDC_SUCCESS ? ok() : s;
}

epdc_status epdc_rms_norm_scratch_bytes(int32_t features, size_t *bytes)
{
    if (features < 8 || features > kMaxNormFeatures || features % 8 || !bytes)
        return fail(EPDC_ERR_INVALID_ARGS,
                    "features, a multiple of 8 and at most %d, and bytes are required",
                    kMaxNormFeatures);
    *bytes = (size_t)norm_scratch(features);
    return ok();
}

epdc_status epdc_rms_norm_backward(const epdc_norm_args *args, void *stream, const void *grad_out,
                                   const void *grad_sum, void *grad_input, float *grad_weight,
                                   void *scratch)
{
    epdc_status s = check_norm(args);
    if (s != EPDC_SUCCESS)
        return s;
    if (args->residual)
        return fail(EPDC_ERR_INVALID_ARGS, "the gradient takes the sum as input, and no residual");
    if ((grad_weight != nullptr) != (scratch != nullptr))
        return fail(EPDC_ERR_INVALID_ARGS, "grad_weight and scratch must both be given or both NULL");
    if (args->rows > 0 && (!grad_out || !grad_input))
        return fail(EPDC_ERR_INVALID_ARGS, "grad_out and grad_input are required");
    if (!aligned(grad_out, 16) || !aligned(grad_sum, 16) || !aligned(grad_input, 16) ||
        !aligned(grad_weight, 16) || !aligned(scratch, 16))
        return fail(EPDC_ERR_INVALID_ARGS, "every array must be 16-byte aligned");
    const int64_t n = (int64_t)args->rows * args->features;
    const bool rows = args->rows > 0;
    const Array x = {"input", rows ? args->input : nullptr, n * 2},
                w = {"weight", rows ? args->weight : nullptr,
                     (int64_t)args->features * (args->weight_dtype == EPDC_DT_BF16 ? 2 : 4)},
                dy = {"grad_out", rows ? grad_out : nullptr, n * 2},
                ds = {"grad_sum", rows ? grad_sum : nullptr, n * 2};
    const Array dx = {"grad_input", rows ? grad_input : nullptr, n * 2},
                dw = {"grad_weight", grad_weight, (int64_t)args->features * 4},
                part = {"scratch", scratch, norm_scratch(args->features)};
    // a row's gradient may take the place of what flows in: the thread that writes an
    // element has read it
    s = check_apart(dx, {x, w, grad_input == grad_out ? Array{} : dy,
                         grad_input == grad_sum ? Array{} : ds, dw, part});
    if (s == EPDC_SUCCESS)
        s = check_apart(dw, {x, w, dy, ds, part});
    if (s == EPDC_SUCCESS)
        s = check_apart(part, {x, w, dy, ds});
    if (s != EPDC_SUCCESS)
        return s;
    hipStream_t st = static_cast<hipStream_t>(stream);
    NormArgs a = norm_args(*args);
    a.grad_out = static_cast<const uint8_t *>(grad_out);
    a.grad_sum = static_cast<const uint8_t *>(grad_sum);
    a.grad_input = static_cast<uint8_t *>(grad_input);
    a.partial = static_cast<float *>(scratch);
    int teams = 0;
    if (rows) {
        s = launch("k_rms_norm_grad", [&] {
            row_form(a.vecs, [&](auto waves, auto vecs) {
                constexpr int kWaves = decltype(waves)::value, kThreads = team_threads(kWaves);
                constexpr int kTeams = kThreads / (kWaves * kWave);
                const int most = norm_grad_blocks(kWaves), need = (a.rows + kTeams - 1) / kTeams;
                const int grid = need < most ? need : most;
                teams = grid * kTeams;
                k_rms_norm_grad<kWaves, decltype(vecs)::value><<<grid, kThreads, 0, st>>>(a);
            });
        });
        if (s != EPDC_SUCCESS)
            return s;
    }
    if (grad_weight) {
        NormWeightGradArgs g = {};
        g.teams = teams;
        g.quads = args->features / 4;
        g.partial = a.partial;
        g.grad_weight = grad_weight;
        const int grid = (g.quads + kWeightGradQuads - 1) / kWeightGradQuads;
        s = launch("k_norm_weight_grad", [&] {
            k_norm_weight_grad<<<grid, kWeightGradQuads * kWeightGradLanes, 0, st>>>(g);
        });
        if (s != EPDC_SUCCESS)
            return s;
    }
    return ok();
}

epdc_status epdc_quantize_rows(void *stream, int32_t rows, int32_t features, int32_t codes_dtype,
                               const void *input, const int32_t *expert_off, int32_t num_experts,
                               void *codes, float *scales)
{
    const int unit = code_unit(codes_dtype);
    if (!unit)
        return fail(EPDC_ERR_INVALID_ARGS, "codes must be e4m3 or int8");
    if (rows < 0 || rows > (1 << 30))
        return fail(EPDC_ERR_INVALID_ARGS, "rows must be in [0, 2^30]");
    if (features < unit || features > kMaxQuantFeatures || features % unit)
        return fail(EPDC_ERR_INVALID_ARGS, "features must be a multiple of %d, at most %d", unit,
                    kMaxQuantFeatures);
    if (expert_off && (num_experts < 1 || num_experts > kMaxExperts))
        return fail(EPDC_ERR_INVALID_ARGS, "num_experts must be in [1, %d]", kMaxExperts);
    if (rows > 0 && (!input || !codes || !scales))
        return fail(EPDC_ERR_INVALID_ARGS, "input, codes and scales are required");
    if (!aligned(input, 16) || !aligned(codes, 16) || !aligned(scales, 4) ||
        !aligned(expert_off, 4))
        return fail(EPDC_ERR_INVALID_ARGS,
                    "input and codes must be 16-byte aligned, the other arrays 4-byte aligned");
    if (rows == 0)
        return ok();
    const int64_t n = (int64_t)rows * features;
    const Array x = {"input", input, n * 2},
                off = {"expert_off", expert_off, ((int64_t)num_experts + 1) * 4},
                c = {"codes", codes, n},
                f = {"scales", scales,
                     4 * (codes_dtype == EPDC_DT_E4M3 ? n / kCodeBlock : (int64_t)rows)};
    epdc_status s = check_apart(c, {x, off, f});
    if (s == EPDC_SUCCESS)
        s = check_apart(f, {x, off});
    if (s != EPDC_SUCCESS)
        return s;
    QuantArgs a = {};
    a.rows = rows;
    a.experts = num_experts;
    a.vecs = features / 16;
    a.expert_off = expert_off;
    a.input = static_cast<const uint8_t *>(input);
    a.codes = static_cast<uint8_t *>(codes);
    a.scales = scales;
    hipStream_t st = static_cast<hipStream_t>(stream);
    if (codes_dtype == EPDC_DT_E4M3) {
        const int64_t blocks = ((int64_t)rows * a.vecs + kQuantThreads - 1) / kQuantThreads;
        s = launch("k_quantize_e4m3", [&] {
            k_quantize_e4m3<<<row_blocks(blocks, kQuantThreads, 1), kQuantThreads, 0, st>>>(a);
        });
    } else {
        s = launch("k_quantize_int8", [&] {
            if (a.vecs <= 64)
                launch_int8<1, 1>(st, a);
            else if (a.vecs <= 256)
                launch_int8<4, 1>(st, a);
            else if (a.vecs <= 512)
                launch_int8<4, 2>(st, a);
            else if (a.vecs <= 2048)
                launch_int8<16, 2>(st, a);
            else
                launch_int8<16, 8>(st, a);
        });
    }
    return s == EPDC_SUCCESS ? ok() : s;
}

epdc_status epdc_few_tokens_scratch_bytes(const epdc_few_args *args, size_t *bytes)
{
    int type;
    const epdc_status s = check_few(args, &type);
    if (s != EPDC_SUCCESS)
        return s;
    if (!bytes)
        return fail(EPDC_ERR_INVALID_ARGS, "bytes is required");
    *bytes = (size_t)few_scratch(*args, type).bytes();
    return ok();
}

epdc_status epdc_few_tokens(const epdc_few_args *args, void *stream, void *scratch, void *out)
{
    int type;
    epdc_status s = check_few(args, &type);
    if (s != EPDC_SUCCESS)
        return s;
    const epdc_few_args &p = *args;
    const bool gated = act_gated(p.activation);
    const int64_t T = p.num_tokens, pairs = T * p.topk, E = p.num_experts, H = p.hidden,
                  I = p.inner, up = gated ? 2 * I : I, elem = element_bytes(type);
    const bool scaled = type != kTypeBf16;
    if (scaled != (p.w1_scales != nullptr) || scaled != (p.w2_scales != nullptr))
        return fail(EPDC_ERR_INVALID_ARGS,
                    "w1_scales and w2_scales belong to e4m3 and int8 weights, both of them");
    if (T > 0 && (!p.input || !p.indices || !p.w1 || !p.w2 || !scratch || !out))
        return fail(EPDC_ERR_INVALID_ARGS, "input, indices, w1, w2, scratch and out are required");
    if (!aligned(p.input, 16) || !aligned(p.w1, 16) || !aligned(p.w2, 16) ||
        !aligned(scratch, 256) || !aligned(out, 16) || !aligned(p.weights, 4) || !aligned(p.indices, 4) ||
        !aligned(p.w1_scales, 4) || !aligned(p.w2_scales, 4) || !aligned(p.bias1, 4) ||
        !aligned(p.bias2, 4))
        return fail(EPDC_ERR_INVALID_ARGS, "input, w1, w2 and out must be 16-byte aligned, scratch "
                                           "256-byte aligned, the other arrays 4-byte aligned");
    if (T == 0)
        return ok();
    const FewScratch parts = few_scratch(p, type);
    const Array x = {"input", p.input, T * H * 2}, rw = {"weights", p.weights, pairs * 4},
                ids = {"indices", p.indices, pairs * 4}, w1 = {"w1", p.w1, E * up * H * elem},
                w2 = {"w2", p.w2, E * H * I * elem},
                s1 = {"w1_scales", p.w1_scales, weight_scales(type, E, up, H) * 4},
                s2 = {"w2_scales", p.w2_scales, weight_scales(type, E, H, I) * 4},
                b1 = {"bias1", p.bias1, E * up * 4}, b2 = {"bias2", p.bias2, E * H * 4};
    const Array mid = {"scratch", scratch, parts.bytes()}, to = {"out", out, T * H * 2};
    s = check_apart(mid, {x, rw, ids, w1, w2, s1, s2, b1, b2, to});
    // the input is not read any more when out is written
    if (s == EPDC_SUCCESS)
        s = check_apart(to, {out == p.input ? Array{} : x, rw, ids, w1, w2, s1, s2, b1, b2});
    if (s != EPDC_SUCCESS)
        return s;
    FewArgs a = {};
    a.tokens = p.num_tokens;
    a.topk = p.topk;
    a.experts = p.num_experts;
    a.first_expert = p.first_expert;
    a.hidden = p.hidden;
    a.inner = p.inner;
    a.act = p.activation;
    a.per_token = few_per_token(p.topk);
    a.x = static_cast<const uint8_t *>(p.input);
    a.weights = p.weights;
    a.indices = p.indices;
    a.w1 = static_cast<const uint8_t *>(p.w1);
    a.w2 = static_cast<const uint8_t *>(p.w2);
    a.s1 = p.w1_scales;
    a.s2 = p.w2_scales;
    a.b1 = p.bias1;
    a.b2 = p.bias2;
    a.h = static_cast<uint8_t *>(scratch);
    a.out = static_cast<uint8_t *>(out);
    a.splits = parts.splits;
    a.ticket = reinterpret_cast<uint32_t *>(a.h + parts.h);
    a.partial = reinterpret_cast<float *>(a.h + parts.h + parts.ticket);
    hipStream_t st = static_cast<hipStream_t>(stream);
    s = type == kTypeE4m3   ? launch_few_rows<kTypeE4m3>(st, a)
        : type == kTypeInt8 ? launch_few_rows<kTypeInt8>(st, a)
                            : launch_few_rows<kTypeBf16>(st, a);
    return s == EPDC_SUCCESS ? ok() : s;
}

const char *epdc_layer_last_error(void) { return g_last_error.c_str(); }

}  // extern "C"
