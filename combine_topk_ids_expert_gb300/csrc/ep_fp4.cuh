// ep_fp4.cuh - declarations of the router (route.cu), the 4-bit floating point
// quantisation (fp4_quant.cu) and products (expert_fp4.cu), and the layer for a few
// tokens (moe_layer.cu).
#pragma once

#include "ep_next.cuh"

namespace ep {

// ---- router (route.cu) -----------------------------------------------------------
struct RouteArgs {
    const void* logits;        // [T][E] bf16 or fp32
    const float* select;       // [T][E], or null: the logits
    int64_t T;
    int E, K;
    bool bf16, sigmoid, normalize;
    float scale;               // scores are this times the probabilities
    int32_t* ids;              // [T][K]: written (route), read (backward)
    float* scores;             // [T][K], route only
    const float* grad_scores;  // [T][K], backward only
    void* grad_logits;         // [T][E] of the logits' type, backward only
};
cudaError_t launch_route(const RouteArgs& a, const LaunchOpts& o);
cudaError_t launch_route_backward(const RouteArgs& a, const LaunchOpts& o);

// ---- 4-bit floating point (fp4_quant.cu) -----------------------------------------
struct Fp4Args {
    const void* x;             // [rows][cols] bf16; dequantisation: codes and scales are read
    int64_t rows, cols;        // cols % 128 == 0
    int64_t rows_per_scale;    // rows that share a tensor scale
    int format;
    uint8_t* codes;            // [rows][cols / 2]
    uint8_t* scales;           // tiles of 128 rows x 4 blocks
    const float* tensor_scale; // [ceil(rows / rows_per_scale)] or null
    void* out;                 // dequantisation: [rows][cols]
    bool out_f32;
};
cudaError_t launch_quantize_fp4(const Fp4Args& a, const LaunchOpts& o);
cudaError_t launch_dequantize_fp4(const Fp4Args& a, const LaunchOpts& o);

// Every token's row quantised and written to its receive rows, with their scores and sources.
struct PermuteFp4Args {
    const void* x;             // [T][D] bf16
    const float* scores;       // [T][K]
    const int32_t* pos;        // [T][K]
    int64_t T, D;              // D % 128 == 0
    int K;
    int format;
    const float* tensor_scale; // one number or null
    uint8_t* codes;            // [rows][D / 2]
    uint8_t* scales;           // tiles of 128 rows
    float* recv_scores;
    int32_t* recv_src;
};
cudaError_t launch_permute_fp4(const PermuteFp4Args& a, int num_sms, const LaunchOpts& o);

}  // namespace ep
