// expert_ffn.cu - the experts' gated feed-forward block on the receive rows,
//     h = act(x Wg^T) * (x Wu^T),   y = h Wd^T,
// and the data gradients of its products. The block's kernels are instances of
// the grouped tcgen05 tile kernel (expert_tile.cuh); y = h Wd^T is
// expert_gemm.cu's and the weight gradients are expert_wgrad.cu's.
//
// Forward: one kernel computes both projections, the activation and the product.
// Backward of a row, with dy the gradient of y and g, u the kept pre-activations:
//     dh = dy Wd,   dg = dh u act'(g),   du = dh act(g),   dx = dg Wg + du Wu.
// dh is the accumulator of one kernel and dg, du what it writes; dx is one
// product with contraction over the 2F gate and up columns.
// dg and du are rounded to bf16 (the type of the saved pre-activations, and what
// the tensor cores take) before the products that follow; dh never is.
#include "expert_tile.cuh"

namespace ep {
namespace {

template <int BN, bool PAIR, int MODE>
cudaError_t launch_mode(const GemmArgs& a, const void* x, int64_t rows, const void* w, int grid,
                        const LaunchOpts& o)
{
    int used = 0;
    return launch_cfg<CfgOf<BN, 64, PAIR, MODE>>(a, x, rows, w, grid, o, &used);
}

// Widest accumulator whose tiles occupy half of the SMs: 256 columns on an SM pair (two
// SMs to a tile), else 128, else 64 (`least`: the narrowest that the mode has). A pair's
// last rows of an expert are M = 128 tiles of 64 rows to an SM, so pairs win even where
// experts are small: 3.80 against 4.21 ms (gated projections, 65536 rows over 256
// experts, 7168 -> 2 x 2048), while narrow tiles win where few tiles are: 10.1 against
// 12.7 us (75 rows to each of 16 experts, 1024 -> 512). kind 1 or 2 asks for single SMs
// or pairs.
int accumulator_columns(const GemmArgs& a, int per_column, int sms, int least)
{
    const int64_t cols = a.dout * per_column;   // accumulator columns
    if (a.kind == 1) return cols % 256 == 0 ? 256 : cols % 128 == 0 ? 128 : 64;
    if (cols % 256 == 0 && (a.kind == 2 || 4 * a.row_tiles * (cols / 256) >= sms)) return 512;
    if (cols % 128 == 0 && (least == 128 || a.kind == 2 || 2 * a.row_tiles * (cols / 128) >= sms))
        return 128;
    return 64;
}

template <int MODE>
cudaError_t launch_dgrad_mode(const GemmArgs& a, const void* grad, int64_t rows, const void* w,
                              int grid, const LaunchOpts& o)
{
    int n = accumulator_columns(a, 1, grid, 64);
    if (n == 512) {
        const cudaError_t e = launch_mode<kPairBN, true, MODE>(a, grad, rows, w, grid, o);
        if (e != cudaErrorNotSupported) return e;
        n = 256;
    }
    if (n == 256) return launch_mode<256, false, MODE>(a, grad, rows, w, grid, o);
    if (n == 128) return launch_mode<128, false, MODE>(a, grad, rows, w, grid, o);
    return launch_mode<64, false, MODE>(a, grad, rows, w, grid, o);
}

}  // namespace

cudaError_t launch_expert_glu(const GemmArgs& a, const void* x, int64_t rows, const void* w,
                              int grid, const LaunchOpts& o)
{
    if (a.din % 64 != 0 || a.dout % 128 != 0) return cudaErrorInvalidValue;
    const int n = accumulator_columns(a, 2, grid, 128);
    if (n == 512) {
        const cudaError_t e = launch_mode<kPairBN, true, kGlu>(a, x, rows, w, grid, o);
        if (e != cudaErrorNotSupported) return e;
    }
    if (n == 128) return launch_mode<128, false, kGlu>(a, x, rows, w, grid, o);
    return launch_mode<256, false, kGlu>(a, x, rows, w, grid, o);
}

cudaError_t launch_expert_dgrad(const GemmArgs& a, bool glu, const void* grad, int64_t rows,
                                const void* w, int grid, const LaunchOpts& o)
{
    if (a.din % 64 != 0 || a.dout % 64 != 0) return cudaErrorInvalidValue;
    return glu ? launch_dgrad_mode<kDgradGlu>(a, grad, rows, w, grid, o)
               : launch_dgrad_mode<kDgrad>(a, grad, rows, w, grid, o);
}

}  // namespace ep
