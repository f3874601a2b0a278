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

// Column blocks of 256 on an SM pair (kind 2), else 256, 128 or 64 on one SM.
template <int MODE>
cudaError_t launch_dgrad_mode(const GemmArgs& a, const void* grad, int64_t rows, const void* w,
                              int grid, const LaunchOpts& o)
{
    if (a.kind >= 2 && a.dout % kPairBN == 0) {
        const cudaError_t e = launch_mode<kPairBN, true, MODE>(a, grad, rows, w, grid, o);
        if (e != cudaErrorNotSupported) return e;
    }
    if (a.dout % 256 == 0) return launch_mode<256, false, MODE>(a, grad, rows, w, grid, o);
    if (a.dout % 128 == 0) return launch_mode<128, false, MODE>(a, grad, rows, w, grid, o);
    return launch_mode<64, false, MODE>(a, grad, rows, w, grid, o);
}

}  // namespace

cudaError_t launch_expert_glu(const GemmArgs& a, const void* x, int64_t rows, const void* w,
                              int grid, const LaunchOpts& o)
{
    if (a.din % 64 != 0 || a.dout % 128 != 0) return cudaErrorInvalidValue;
    if (a.kind >= 2) {
        const cudaError_t e = launch_mode<kPairBN, true, kGlu>(a, x, rows, w, grid, o);
        if (e != cudaErrorNotSupported) return e;
    }
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
