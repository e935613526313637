// Launch declarations of the operators around the path: the router's choice
// of experts and the products over rows (grouped by expert or over all
// tokens of a rank).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "common.h"
#include "w4_tiles.h"

namespace moe_ep {

// Columns under one fp8 scale: a row's scale per 128 columns, a weight
// matrix's per 128 x 128 block.
constexpr int kScaleBlock = 128;

struct RouteArgs {
    const uint8_t* logits;
    int64_t logits_stride;   // bytes between rows
    bool bf16;
    const float* bias;       // nullable
    int64_t T;
    int E, K, score, n_group, topk_group;
    bool renormalize;
    float scale;
    int32_t* ids;
    float* weights;
};

hipError_t launch_route_topk(const RouteArgs& a, hipStream_t stream);

// out[g][r] = act(x[g][r] . w[g]^T + bias[g]) (+ residual[r]) for every group
// g and row r below counts[g] (rows, without counts). All strides in bytes
// except those of the fp32 scale and bias arrays (elements).
struct MatmulArgs {
    const uint8_t* x;
    int64_t x_stride, x_row;
    const uint8_t* w;
    int64_t w_stride, w_row;
    const float* xs;             // fp8: row scales [rows, xs_pitch]
    int64_t xs_stride, xs_pitch;
    const float* ws;             // fp8: block scales [blocks of rows, slabs]
    int64_t ws_stride;
    const float* bias;           // nullable, [rows of w]
    int64_t bias_stride;
    const uint8_t* res;          // nullable, type of out
    int64_t res_row;
    uint8_t* out;
    int64_t out_stride, out_row;
    float* os;                   // e4m3 out: row scales [rows, os_pitch]
    int64_t os_stride, os_pitch;
    const int32_t* counts;       // nullable: every group has `rows` rows
    int32_t groups;
    int32_t rows;                // capacity of a group
    int32_t N;                   // output columns
    int32_t row_bytes;           // bytes of a row of x and of w that count
    int32_t act, out_dtype;
    bool fp8;
};

hipError_t launch_matmul(const MatmulArgs& a, hipStream_t stream);

// The same with 4-bit weights: m.w holds E2M1 codes (m.w_stride, m.w_row bytes),
// s one scale per `group` columns (E4M3 for 16, E8M0 for 32). m.row_bytes is
// that of x.
struct W4Args {
    MatmulArgs m;
    FewCut cut;                  // over all tokens, few of them
    const uint8_t* s;
    int64_t s_stride, s_row;     // bytes
    int group;
    const float* whole;          // nullable: [groups][1, or gate and up]
};

hipError_t launch_matmul_w4(const W4Args& a, hipStream_t stream);

// A router's training terms over S sequences of tokens (start: nullable, one
// sequence of all).
struct BalanceArgs {
    const uint8_t* logits;
    int64_t logits_stride;       // bytes between rows
    bool bf16;
    const int32_t* ids;
    int64_t T;
    int E, K, score;
    const int32_t* start;
    int S;
    int64_t tile;                // tokens of a block
    int32_t* counts;
    float* mean;
    int32_t* tokens;
    float* loss;
    int32_t* slot_count;         // [slots][E]; nullptr: a block per sequence, no slots
    float* slot_score;           // [slots][E]
    int32_t* slot_tokens;        // [slots]
    double* part;                // [S][ceil(E / 64)][2]: picks, picks times mean scores
    int32_t* ticket;             // [S], cleared by the call itself
};

hipError_t launch_balance(const BalanceArgs& a, hipStream_t stream);

struct RouteGradArgs {
    const uint8_t* logits;
    int64_t logits_stride;
    bool bf16;
    const int32_t* ids;
    int64_t T;
    int E, K, score;
    bool renormalize;
    float scale;
    const float* grad_weights;   // nullable
    const float* grad_loss;      // nullable, with the four below
    const int32_t* start;
    int S;
    const int32_t* counts;
    const int32_t* tokens;
    uint8_t* grad;
    int64_t grad_stride;
    bool grad_bf16;
    int64_t tile;
};

hipError_t launch_route_backward(const RouteGradArgs& a, hipStream_t stream);

}  // namespace moe_ep
