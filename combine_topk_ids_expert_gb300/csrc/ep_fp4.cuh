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
    int kept;                  // one kernel: tokens of a tile whose codes wait in shared memory
};
cudaError_t launch_permute_fp4(const PermuteFp4Args& a, int num_sms, const LaunchOpts& o);
// Layout and rows in one cooperative kernel; cudaErrorNotSupported where a tile's tables do not fit
// or the tiles cannot all be resident. l has at most dispatch_fp4_tiles_per_sm() tiles per SM.
// pdl_ok and small_pairs as for launch_dispatch_onepass.
int dispatch_fp4_tiles_per_sm();
cudaError_t launch_dispatch_fp4(const LayoutArgs& l, const PermuteFp4Args& a, const LaunchOpts& o,
                                bool pdl_ok, int64_t small_pairs);

// The experts' products in 4 bits (expert_fp4.cu).
struct ExpertFp4Args {
    const int32_t* cnt;            // [E]
    const int32_t* expert_offset;  // [E]
    const uint8_t* x_codes;        // [rows][din / 2]
    const uint8_t* x_scales;
    const float* x_scale;          // one number or null
    const uint8_t* w_codes;        // [E][dout or 2 dout][din / 2]
    const uint8_t* w_scales;
    const float* w_scale;          // [E] or null
    void* y;                       // [rows][dout] bf16, or codes [rows][dout / 2] with y_scales
    uint8_t* y_scales;             // glu only: quantise h (the format of x and W)
    const float* h_scale;          // its matrix's scale: one number or null
    int64_t rows, din, dout;       // din % 128 == 0, dout % 128 == 0
    int format, E, act;
    bool glu;                      // W has dout gate rows, then dout up rows; y = act(g) * u
    int kind;                      // 1 single SMs, 2 pairs (where W's rows are a multiple of 256),
                                   // 0: by the number of tiles
    int light_rows;                // as GemmArgs
    int64_t row_tiles;             // row tiles of 256 that the call is likely to have
    int64_t mean_rows;             // rows of an expert, on average over all
    uint32_t* err;
};
cudaError_t launch_expert_fp4(const ExpertFp4Args& a, int num_sms, const LaunchOpts& o);

// A whole layer for a few tokens (moe_layer.cu).
constexpr int kLayerMaxTokens = 64, kLayerMaxPairs = 512;
struct MoeLayerArgs {
    const void* x;                 // [T][D] bf16
    const float* scores;           // [T][K]
    const int32_t* ids;            // [T][K]
    int T, K, E;                   // T <= kLayerMaxTokens, T * K <= kLayerMaxPairs
    int64_t D, dff;                // multiples of 128
    int format;                    // kFp4Mx, kFp4Nv, or any other: bf16 weights
    const void* w_gate_up;         // [E][2 dff][D] bf16, or codes
    const void* w_down;            // [E][D][dff]
    const uint8_t* gate_up_scales; // 4 bits
    const uint8_t* down_scales;
    const float* gate_up_scale;    // [E] or null
    const float* down_scale;
    int act;
    float* h;                      // workspace: [T K][dff]
    uint32_t* h_most;              // [T K][dff / 32]
    float* y;                      // [T K][D]
    uint32_t* done;                // [D / 32]
    void* out;                     // [T][D]
    bool out_f32;
    uint32_t* err;
};
cudaError_t launch_moe_layer(const MoeLayerArgs& a, int num_sms, const LaunchOpts& o);

}  // namespace ep
