// fp4_umma.cuh - the block-scaled 4-bit forms of tcgen05: descriptors, the copy of scales to
// tensor memory, the MMA, and tensor maps over codes.
//
// kind::mxf4 (blocks of 32, ue8m0) and kind::mxf4nvf4 with scale_vec::4X (blocks of 16,
// ue4m3) multiply K = 64 elements an instruction, packed two to a byte in shared memory, and
// take the scales from tensor memory: a row's scales for one instruction are bytes of one
// 32-bit word at lane row % 32, column row / 32, the same in all four groups of 32 lanes.
#pragma once

#include "fp4.cuh"
#include "umma.cuh"

namespace ep {
namespace {

constexpr int kFp4K = 64;                    // elements of one instruction
constexpr int kFp4StageK = 256;              // elements of a ring stage: 128 bytes of codes
constexpr uint32_t kScaleTile = 512;         // bytes of a tile of scales (128 rows x 4 blocks)

template <int FMT>
struct Fp4Mma {
    static constexpr int kTiles = kFp4StageK / (4 * Fp4<FMT>::kBlock);   // scale tiles of a stage: 2 or 4
    // Instruction descriptor: A and B e2m1 (bits 7-9 and 10-11 = 1), N >> 3 at bits 17-22,
    // scale type at bit 23 (1: ue8m0), M >> 4 at bits 24-28; which bytes of the scales' word
    // an instruction takes at bits 29-30 (A) and 4-5 (B): with blocks of 32 the first or
    // (2) the second two, with blocks of 16 all four.
    static __host__ __device__ constexpr uint32_t idesc(int m, int n)
    {
        return (1u << 7) | (1u << 10) | ((uint32_t)(n >> 3) << 17) |
               ((FMT == kFp4Mx ? 1u : 0u) << 23) | ((uint32_t)(m >> 4) << 24);
    }
    // Step j (of 64 elements) of a stage.
    static __device__ __forceinline__ uint32_t idesc_step(uint32_t idesc, int j)
    {
        return FMT == kFp4Mx && (j & 1) ? idesc | (2u << 29) | (2u << 4) : idesc;
    }
    static __host__ __device__ constexpr int tile_of_step(int j) { return FMT == kFp4Mx ? j >> 1 : j; }
};

// Descriptors in two halves, of which only the lower one moves (by bytes / 16; shared memory
// ends below the 14 bits of its address): what the issuing thread computes for an instruction is
// one addition. Computed whole each time they took longer than the products.
//   codes: lines of 128 bytes, 128-byte swizzle, 1024 bytes from one group of 8 to the next;
//   scales: a tile's 32 lines of 16 bytes, no swizzle, 128 bytes from one group of 8 to the next.
constexpr uint32_t kCodeDescHi = (1024 >> 4) | (1u << 14) | (2u << 29);
constexpr uint32_t kScaleDescHi = (128 >> 4) | (1u << 14);
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr) { return (saddr >> 4) | (1u << 16); }
__device__ __forceinline__ uint64_t desc_of(uint32_t lo, uint32_t hi)
{
    return (uint64_t)lo | ((uint64_t)hi << 32);
}

// A tile of scales to 4 columns of tensor memory, in all four groups of lanes. In order with
// the MMAs of the same thread.
template <bool PAIR>
__device__ __forceinline__ void tmem_copy_scales(uint32_t taddr, uint64_t desc)
{
    if (PAIR)
        asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc)
                     : "memory");
    else
        asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc)
                     : "memory");
}

template <int FMT, bool PAIR>
__device__ __forceinline__ void umma_fp4(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                         uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                         uint32_t accumulate)
{
#define EP_UMMA_FP4(GROUP, KIND)                                                                 \
    asm volatile("{\n\t.reg .pred p;\n\t"                                                        \
                 "setp.ne.b32 p, %6, 0;\n\t"                                                     \
                 "tcgen05.mma.cta_group::" GROUP ".kind::" KIND " [%0], %1, %2, %3, [%4], [%5], p;\n\t}" \
                 ::"r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sfa), "r"(sfb),         \
                 "r"(accumulate)                                                                 \
                 : "memory")
    if (FMT == kFp4Mx) {
        if (PAIR) EP_UMMA_FP4("2", "mxf4.block_scale.scale_vec::2X");
        else EP_UMMA_FP4("1", "mxf4.block_scale.scale_vec::2X");
    } else {
        if (PAIR) EP_UMMA_FP4("2", "mxf4nvf4.block_scale.scale_vec::4X");
        else EP_UMMA_FP4("1", "mxf4nvf4.block_scale.scale_vec::4X");
    }
#undef EP_UMMA_FP4
}

// Tensor map over codes [rows][cols / 2] in boxes of 128 bytes x box_rows, 128-byte swizzle.
// Columns behind the last are read as zeros.
inline bool make_code_map(CUtensorMap* m, const void* base, uint64_t cols, uint64_t rows,
                          uint32_t box_rows)
{
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[2] = {cols / 2, rows};
    const cuuint64_t strides[1] = {cols / 2};
    const cuuint32_t box[2] = {kFp4StageK / 2, box_rows};
    const cuuint32_t estr[2] = {1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Arrive on an mbarrier of any CTA of the cluster, after this thread's accesses to its own CTA's
// shared memory (and what is ordered before them: tcgen05 loads behind their fence). A release at
// cluster scope would also wait for every global access of the thread: half a microsecond to
// one, at each arrival.
__device__ __forceinline__ void mbar_arrive_cluster_own(uint32_t bar)
{
    asm volatile("fence.release.sync_restrict::shared::cta.cluster;" ::: "memory");
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// Tensor map over tiles of scales, one after the other, in boxes of box_tiles.
inline bool make_scale_map(CUtensorMap* m, const void* base, uint64_t tiles, uint32_t box_tiles)
{
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[2] = {kScaleTile / 4, tiles};
    const cuuint64_t strides[1] = {kScaleTile};
    const cuuint32_t box[2] = {kScaleTile / 4, box_tiles};
    const cuuint32_t estr[2] = {1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT32, 2, const_cast<void*>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

__device__ __forceinline__ void sts32(uint32_t addr, uint32_t v)
{
    asm volatile("st.shared.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

__device__ __forceinline__ void sts64(uint32_t addr, uint2 v)
{
    asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(addr), "r"(v.x), "r"(v.y) : "memory");
}

}  // namespace
}  // namespace ep
