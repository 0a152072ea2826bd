// layer.hip -- host side of the C ABI declared in include/epdc_layer.h: argument
// checks, the choice of kernel form, and the launches.  Nothing here waits for
// the device or allocates.
#include "epdc_layer.h"
#include "layer_product.hpp"
#include "layer_gate.hpp"

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
    if (p->dtype != EPDC_DT_BF16 && p->dtype != EPDC_DT_E4M3)
        return fail(EPDC_ERR_INVALID_ARGS, "operands must be bf16 or e4m3");
    const bool e4m3 = p->dtype == EPDC_DT_E4M3;
    const int unit_in = e4m3 ? 128 : 8, unit_out = act_gated(p->activation) ? 16 : 8;
    if (p->in_features < unit_in || p->in_features > kMaxFeatures || p->in_features % unit_in)
        return fail(EPDC_ERR_INVALID_ARGS, "in_features must be a multiple of %d, at most 2^20",
                    unit_in);
    if (p->out_features < unit_out || p->out_features > kMaxFeatures ||
        p->out_features % unit_out)
        return fail(EPDC_ERR_INVALID_ARGS, "out_features must be a multiple of %d, at most 2^20",
                    unit_out);
    if ((int64_t)p->in_features * p->out_features * (e4m3 ? 1 : 2) > kMaxExpertBytes)
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
    const int64_t elem = p.dtype == EPDC_DT_E4M3 ? 1 : 2, blocks = in / 128;
    return {{"input", p.input, rows * in * elem},
            {"scales", p.scales, rows * blocks * 4},
            {"weight", p.weight, experts * of * in * elem},
            {"weight_scales", p.weight_scales, experts * ((of + 127) / 128) * blocks * 4},
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

template <bool kE4m3, int kGroups>
epdc_status launch_tile(hipStream_t st, ProductArgs &a)
{
    int grid;
    const epdc_status s = plan_tiles<kForward, kGroups>(a, &grid);
    if (s != EPDC_SUCCESS)
        return s;
    return launch("k_product_tile", [&] {
        k_product_tile<kE4m3, kGroups><<<grid, kTileWaves * kWave, 0, st>>>(a);
    });
}

template <bool kE4m3, int kMI>
epdc_status launch_stream(hipStream_t st, ProductArgs &a)
{
    a.col_tiles = (a.out_cols + 15) / 16;
    int grid;
    const epdc_status s = grid_of(row_tile_bound(a.rows, a.experts, kMI * 16) * a.col_tiles,
                                  kStreamWaves * kWave, &grid);
    if (s != EPDC_SUCCESS)
        return s;
    return launch("k_product_stream", [&] {
        if (act_gated(a.act))
            k_product_stream<kE4m3, kMI, true><<<grid, kStreamWaves * kWave, 0, st>>>(a);
        else
            k_product_stream<kE4m3, kMI, false><<<grid, kStreamWaves * kWave, 0, st>>>(a);
    });
}

template <bool kE4m3>
epdc_status launch_forward(hipStream_t st, ProductArgs &a, int64_t mean)
{
    // By mean rows per expert, all that is known here of the experts' counts.  The
    // streamed form reads the weights fastest but once per 16 (32) rows of an
    // expert, the tiles once per 64 (256) at 85% of that rate.  Measured over 64
    // experts of 4096 x 4096, streamed (16), streamed (32), 64-row tiles: bf16 mean
    // 8: 327, 346, 393 us; 12: 355, 337, 394; 24: -, 366, 405; 32: -, 578, 409.
    // e4m3: 12: 195, 239, 238; 16: 261, 253, 236 (with 32 rows its registers
    // leave too few waves).  64- against 256-row tiles, bf16: 40 rows 399, 410; 64:
    // 429, 441; 80: 462, 449; 128: 520, 475.  e4m3: 40: 242, 243; 64: 250, 249; 80:
    // 280, 254; 128: 328, 270.
    if (mean <= (kE4m3 ? 12 : 10))
        return launch_stream<kE4m3, 1>(st, a);
    if constexpr (!kE4m3) {
        if (mean <= 24)
            return launch_stream<kE4m3, 2>(st, a);
    }
    if (mean <= 64)
        return launch_tile<kE4m3, 1>(st, a);
    return launch_tile<kE4m3, 4>(st, a);
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
    const bool e4m3 = args->dtype == EPDC_DT_E4M3;
    if (e4m3 != (args->scales != nullptr) || e4m3 != (args->weight_scales != nullptr))
        return fail(EPDC_ERR_INVALID_ARGS,
                    "scales and weight_scales belong to e4m3 operands, both of them");
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
    a.p_bytes = a.q_bytes = args->in_features * (e4m3 ? 1 : 2);
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
    s = e4m3 ? launch_forward<true>(st, a, mean) : launch_forward<false>(st, a, mean);
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

const char *epdc_layer_last_error(void) { return g_last_error.c_str(); }

}  // extern "C"
