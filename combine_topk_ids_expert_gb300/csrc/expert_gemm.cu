// expert_gemm.cu - the expert consumer between dispatch and combine: a
// grouped GEMM  y[p] = x[p] * W_e^T  over the receive rows of every expert,
// driven by the per-expert counts and offsets the layout left on the device
// ("ep: graph-safe worst-token HT dispatch+combine", "Internode" item 2: the
// counts stay on the device so graph-mode consumers never touch the host;
// "Tests": layout -> dispatch -> expert -> combine). No host round trip: the
// tile list is derived on the device from the counts.
//
// sm_103a tensor cores, written directly:
//   - one CTA per SM, persistent over output tiles of 128 rows x BN columns
//     of one expert (tile order: the column blocks of one row block first,
//     so the row block is reused from L2);
//   - light experts (at most light_rows rows: their weights are read from
//     HBM for one or two row tiles, so their tiles wait on memory) and heavy
//     ones (weights reused from L2 by many row tiles, so their tiles wait on
//     the tensor cores) form two tile sequences, each in expert order, that
//     are interleaved in proportion to their lengths: at every point of the
//     schedule both kinds run side by side, instead of a tensor-bound phase
//     followed by a memory-bound one when the routing is skewed;
//   - warp 0 (one thread) streams BK-wide K slices of the row block and of
//     the expert's weights into a shared-memory ring with TMA tensor copies
//     (128-byte swizzle for BK = 64, 64-byte for BK = 32), completion on
//     mbarriers;
//   - warp 1 owns two BN-column fp32 accumulators in tensor memory (TMEM)
//     and one thread issues tcgen05.mma (M=128, N=BN, K=16, bf16 inputs, fp32
//     accumulate) from shared-memory descriptors, committing each stage back
//     to the ring and each finished tile to the epilogue; tiles alternate
//     between the accumulators so the epilogue overlaps the next tile;
//   - warps 2-5 read the accumulator with tcgen05.ld (each warp its 32-lane
//     quarter), round to bf16 and store the rows that belong to the expert.
//
// A single-CTA 128 x 256 MMA reads 12 KB of operands from shared memory per
// K=16 step; with the ring's copies writing as much again, this kernel's MMAs
// ran at 1.46 PFLOP/s even with the copies switched off, against 2.42 PFLOP/s
// for a bare stream of the same MMAs from fixed operands.
//
// Two-SM variant (PAIR, the default where dout % 256 == 0): a cluster of two
// CTAs computes 256 x 256 tiles with tcgen05.mma.cta_group::2 (M = 256):
//   - CTA r holds rows [128r, 128r + 128) of the tile and the W rows
//     [128r, 128r + 128) of the column block, so each SM reads 8 KB per K=16
//     step and takes 32 KB per 64-wide slice into shared memory instead of 48;
//   - both CTAs' TMA copies complete on the leader's (rank 0) full barrier;
//     the leader's one MMA thread issues for both SMs, and its commits arrive
//     on both CTAs' barriers (stage release, accumulator ready);
//   - each CTA's epilogue drains its own TMEM (its 128 rows x 256 columns) and
//     tells the leader, which reuses an accumulator only after both have;
//   - an expert's last rows, when at most 128 remain, run as one M = 128 tile
//     across the pair (64 rows per CTA, loaded with a 64-row box). Its
//     accumulator holds the CTA's 64 rows twice in 128 columns: lanes 0-63
//     with output columns [0, 128), lanes 64-127 with [128, 256), so every
//     epilogue warp drains 32 rows x 128 columns.
// Tiles cover 256 rows of one expert, so an expert's last tile is padded to
// 256 rows when more than 128 remain (to 128 otherwise).
//
// Every wait is bounded; on a timeout the CTA reports EP_DEVERR_TIMEOUT,
// waits (bounded) for its copies and MMAs in flight, frees its TMEM and
// returns.
//
// The kernel itself is in expert_tile.cuh, which the gated feed-forward block's
// kernels share.
#include "expert_tile.cuh"

namespace ep {
namespace {

template <int BK>
cudaError_t launch_bk(const GemmArgs& a, const void* x, int64_t rows, const void* w, int grid,
                      const LaunchOpts& o, int* kernel_used, int* grid_used)
{
    if (a.kind >= 2 && a.dout % kPairBN == 0) {
        *kernel_used = 2;
        const cudaError_t e = launch_cfg<CfgOf<kPairBN, BK, true>>(a, x, rows, w, grid, o, grid_used);
        if (e != cudaErrorNotSupported) return e;
    }
    *kernel_used = 1;
    if (a.dout % 256 == 0)
        return launch_cfg<CfgOf<256, BK, false>>(a, x, rows, w, grid, o, grid_used);
    return launch_cfg<CfgOf<128, BK, false>>(a, x, rows, w, grid, o, grid_used);
}

}  // namespace

cudaError_t launch_expert_gemm(const GemmArgs& a, const void* x, int64_t rows, const void* w,
                               int grid, const LaunchOpts& o, int* kernel_used, int* grid_used)
{
    if (a.din % 64 != 0 || a.dout % 128 != 0) return cudaErrorInvalidValue;
    if (a.bk == 32) return launch_bk<32>(a, x, rows, w, grid, o, kernel_used, grid_used);
    return launch_bk<64>(a, x, rows, w, grid, o, kernel_used, grid_used);
}

}  // namespace ep
