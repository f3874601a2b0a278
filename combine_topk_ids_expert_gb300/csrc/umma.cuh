// umma.cuh - what the tcgen05 kernels share: shared-memory descriptors, TMA
// tensor copies, the tcgen05 allocation / MMA / commit / load forms for one CTA
// and for a pair, cluster and abort-aware waits, and the host side's tensor maps
// and cluster grids.
#pragma once

#include <cuda.h>

#include <mutex>

#include "ep_device.cuh"
#include "ep_next.cuh"

namespace ep {
namespace {

constexpr int kBM = 128;            // rows per tile = TMEM lanes = UMMA M
constexpr int kUmmaK = 16;          // K per tcgen05.mma for 16-bit inputs
constexpr int kPairBN = 256;
constexpr uint16_t kBothCtas = 0x3;
constexpr int kSmemLimit = 232448;  // dynamic shared memory per CTA on sm_103

// Shared-memory matrix descriptor for a K-major tile written by TMA with the
// 128- or 64-byte swizzle: start address >> 4 (bits 0-13), leading offset 16 B
// (unused for these layouts), stride between 8-row groups >> 4 (bits 32-45),
// descriptor version 1 (bits 46-47), swizzle mode (bits 61-63).
template <class C>
__device__ __forceinline__ uint64_t smem_desc(uint32_t saddr)
{
    return (uint64_t)((saddr >> 4) & 0x3FFFu) | ((uint64_t)1 << 16) |
           ((uint64_t)(C::kSbo >> 4) << 32) | ((uint64_t)1 << 46) | (C::kSwizzleMode << 61);
}

// The same for lines of 128 bytes whatever the element type (128-byte swizzle).
__device__ __forceinline__ uint64_t smem_desc_k128(uint32_t saddr)
{
    return (uint64_t)((saddr >> 4) & 0x3FFFu) | ((uint64_t)1 << 16) |
           ((uint64_t)(1024 >> 4) << 32) | ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}

// Descriptor of an MN-major tile (the M or N axis contiguous in memory, K across
// lines) written by TMA in boxes of 64 elements x BK lines with the 128-byte
// swizzle: a line is 64 elements of one k; leading offset = bytes from one box to
// the next 64 elements of M or N, stride offset = bytes between groups of 8 lines.
constexpr uint32_t kMnLineBytes = 128;
constexpr uint32_t kMnBoxBytes = 64 * kMnLineBytes;   // 64 elements x 64 lines
__device__ __forceinline__ uint64_t smem_desc_mn(uint32_t saddr)
{
    return (uint64_t)((saddr >> 4) & 0x3FFFu) | ((uint64_t)(kMnBoxBytes >> 4) << 16) |
           ((uint64_t)(8 * kMnLineBytes >> 4) << 32) | ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}

__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap* tm, int c0, int c1,
                                            uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(tm)), "r"(c0), "r"(c1), "r"(bar)
        : "memory");
}

// Pair form: the data lands in this CTA's shared memory, the completion on an
// mbarrier that may be the peer's (bar: a shared::cluster address).
__device__ __forceinline__ void tma_load_2d_pair(uint32_t dst, const CUtensorMap* tm, int c0,
                                                 int c1, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes.cta_group::2 "
        "[%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(tm)), "r"(c0), "r"(c1), "r"(bar)
        : "memory");
}

// shared::cluster address of the same offset in CTA rank of this cluster.
__device__ __forceinline__ uint32_t map_to_rank(uint32_t local, int rank)
{
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(local), "r"(rank));
    return r;
}

// Arrive on an mbarrier given by its shared::cluster address (any CTA of the cluster).
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t bar)
{
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar)
                 : "memory");
}

__device__ __forceinline__ void mbar_arrive(uint32_t bar)
{
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ void tc_fence_before()
{
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}

__device__ __forceinline__ void tc_fence_after()
{
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}

// tcgen05 allocation, MMA and commit; a kernel uses one CTA group throughout
// (PAIR: cta_group::2, issued for both CTAs of the pair).
template <bool PAIR>
__device__ __forceinline__ void tmem_alloc(uint32_t dst_smem, uint32_t ncols)
{
    if (PAIR)
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         dst_smem),
                     "r"(ncols)
                     : "memory");
    else
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         dst_smem),
                     "r"(ncols)
                     : "memory");
}

template <bool PAIR>
__device__ __forceinline__ void tmem_relinquish()
{
    if (PAIR) asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    else asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}

template <bool PAIR>
__device__ __forceinline__ void tmem_dealloc(uint32_t taddr, uint32_t ncols)
{
    if (PAIR)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr),
                     "r"(ncols)
                     : "memory");
    else
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(taddr),
                     "r"(ncols)
                     : "memory");
}

template <bool PAIR>
__device__ __forceinline__ void umma_bf16(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                          uint32_t idesc, uint32_t accumulate)
{
    if (PAIR)
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
            "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
            "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
            : "memory");
}

// Arrives on bar once the MMAs issued so far finish; PAIR: on bar in both CTAs.
template <bool PAIR>
__device__ __forceinline__ void umma_commit(uint32_t bar)
{
    if (PAIR)
        asm volatile(
            "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 "
            "[%0], %1;" ::"r"(bar),
            "h"(kBothCtas)
            : "memory");
    else
        asm volatile(
            "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
            : "memory");
}

// Arrives on this CTA's bar only.
template <bool PAIR>
__device__ __forceinline__ void umma_commit_local(uint32_t bar)
{
    if (PAIR)
        asm volatile(
            "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
            : "memory");
    else
        asm volatile(
            "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
            : "memory");
}

__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&v)[32])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]),
          "=r"(v[7]), "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]),
          "=r"(v[14]), "=r"(v[15]), "=r"(v[16]), "=r"(v[17]), "=r"(v[18]), "=r"(v[19]),
          "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]), "=r"(v[25]),
          "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
        : "r"(taddr));
}

__device__ __forceinline__ void tmem_wait_ld()
{
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void cluster_sync()
{
    asm volatile(
        "barrier.cluster.arrive.release.aligned;\n\t"
        "barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__device__ __forceinline__ int cluster_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return (int)r;
}

__device__ __forceinline__ int cluster_index()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%clusterid.x;" : "=r"(r));
    return (int)r;
}

__device__ __forceinline__ int cluster_count()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%nclusterid.x;" : "=r"(r));
    return (int)r;
}

// CLUSTER: with what the other CTAs of the cluster wrote before they arrived.
template <bool CLUSTER>
__device__ __forceinline__ bool mbar_try_wait_scope(uint32_t bar, uint32_t parity)
{
    if (!CLUSTER) return mbar_try_wait(bar, parity);
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(bar), "r"(parity)
        : "memory");
    return done != 0u;
}

// Bounded wait that also gives up when another role has aborted.
template <bool CLUSTER = false>
__device__ __forceinline__ bool wait_or_abort(uint32_t bar, uint32_t parity, volatile int* abort)
{
    if (mbar_try_wait_scope<CLUSTER>(bar, parity)) return true;
    const uint64_t deadline = globaltimer_ns() + kWaitLimitNs;
    while (true) {
        for (int i = 0; i < 64; ++i)
            if (mbar_try_wait_scope<CLUSTER>(bar, parity)) return true;
        if (*abort) return false;
        if (globaltimer_ns() > deadline) {
            *abort = 1;
            return false;
        }
    }
}

__device__ __forceinline__ uint32_t pack_bf16x2_rn(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// The gate's activation and its slope, in fp32. silu: g s, s + g s (1 - s) with
// s = 1 / (1 + e^-g). gelu (tanh form): (1 + tanh w) / 2 = 1 / (1 + e^-2w), so it is
// g p with p = 1 / (1 + e^-v), v = 2 sqrt(2 / pi) (g + 0.044715 g^3), and the slope
// is p + g v' p (1 - p). __expf is off by 2 + 1.2 |v| ulp of fp32 (108 where |v| = 88, less
// than a six-hundredth of an ulp of the bf16 in which results leave), __fdividef by 2; it
// gives 0 for 1 + e^-v above 2^126, so a p below fp32's least normal number is 0.
constexpr float kGeluC = 1.5957691216057308f;   // 2 sqrt(2 / pi)
__device__ __forceinline__ float sigmoid_of(float v) { return __fdividef(1.0f, 1.0f + __expf(-v)); }

__device__ __forceinline__ float act_value(float g, int act)
{
    const float v = act == 0 ? g : kGeluC * (g + 0.044715f * g * g * g);
    return g * sigmoid_of(v);
}

__device__ __forceinline__ void act_value_slope(float g, int act, float* value, float* slope)
{
    const float v = act == 0 ? g : kGeluC * (g + 0.044715f * g * g * g);
    const float dv = act == 0 ? 1.0f : kGeluC * (1.0f + 3.0f * 0.044715f * g * g);
    const float p = sigmoid_of(v);
    *value = g * p;
    const float t = p * (1.0f - p);
    *slope = t > 0.0f ? p + g * dv * t : p;   // far out g v' overflows where t is zero
}

// 32 rows x 32 bf16 columns of a warp, one row per lane, from and to memory by way of
// the warp's 2 KB of shared memory: a lane's own row would be 16 bytes of 32 different
// lines per instruction, this way an instruction covers 64 bytes of 8 rows. `base`: the
// first row's first column; rows [0, rows) exist. The row's 16-byte units are XORed with
// the row so that neither side has bank conflicts.
constexpr int kStageWarpBytes = 2048;

__device__ __forceinline__ uint32_t stage_at(uint32_t stage, int row, int unit)
{
    return stage + (uint32_t)(row * 64 + ((unit ^ ((row >> 1) & 3)) << 4));
}

__device__ __forceinline__ void sts128(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d)
{
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d)
                 : "memory");
}

__device__ __forceinline__ int4 lds_int4(uint32_t addr)
{
    int4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

__device__ __forceinline__ void warp_store_bf16x32(uint32_t stage, int lane, const float (&v)[32],
                                                   uint16_t* base, int64_t stride, int rows)
{
    __syncwarp();   // the warp is done with what the stage held
#pragma unroll
    for (int g = 0; g < 4; ++g)
        sts128(stage_at(stage, lane, g), pack_bf16x2_rn(v[8 * g + 0], v[8 * g + 1]),
               pack_bf16x2_rn(v[8 * g + 2], v[8 * g + 3]), pack_bf16x2_rn(v[8 * g + 4], v[8 * g + 5]),
               pack_bf16x2_rn(v[8 * g + 6], v[8 * g + 7]));
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int row = 8 * i + (lane >> 2), unit = lane & 3;
        const int4 w = lds_int4(stage_at(stage, row, unit));
        if (row < rows) *reinterpret_cast<int4*>(base + row * stride + 8 * unit) = w;
    }
}

// The loads of warp_load_bf16x32, which its second half takes to the lanes' rows.
__device__ __forceinline__ void warp_fetch_bf16x32(int4 (&w)[4], int lane, const uint16_t* base,
                                                   int64_t stride, int rows)
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int row = 8 * i + (lane >> 2);
        w[i] = row < rows ? ld_cg_v4(base + row * stride + 8 * (lane & 3)) : make_int4(0, 0, 0, 0);
    }
}

__device__ __forceinline__ void warp_spread_bf16x32(uint32_t stage, int lane, const int4 (&w)[4],
                                                    float (&v)[32])
{
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 4; ++i)
        sts128(stage_at(stage, 8 * i + (lane >> 2), lane & 3), (uint32_t)w[i].x, (uint32_t)w[i].y,
               (uint32_t)w[i].z, (uint32_t)w[i].w);
    __syncwarp();
#pragma unroll
    for (int g = 0; g < 4; ++g) {
        const int4 p = lds_int4(stage_at(stage, lane, g));
        const uint32_t q[4] = {(uint32_t)p.x, (uint32_t)p.y, (uint32_t)p.z, (uint32_t)p.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[8 * g + 2 * i] = __uint_as_float(q[i] << 16);
            v[8 * g + 2 * i + 1] = __uint_as_float(q[i] & 0xFFFF0000u);
        }
    }
}

__device__ __forceinline__ void as_floats(const uint32_t (&q)[32], float (&v)[32])
{
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(q[i]);
}

// Whether every lane's wait succeeded: a warp that gives up does so as a whole (what
// follows its waits are warp-wide instructions).
__device__ __forceinline__ bool warp_all(bool ok) { return __all_sync(0xffffffffu, ok) != 0; }

// Index e with pre[e] <= i < pre[e+1] of a non-decreasing prefix (i < pre[E]).
__device__ __forceinline__ int expert_of(const int* pre, int E, int i)
{
    int lo = 0, hi = E;   // invariant: pre[lo] <= i < pre[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (pre[mid] <= i) lo = mid;
        else hi = mid;
    }
    return lo;
}

// One lane of a converged warp. The values that it then issues with are the same in
// every lane, so the compiler keeps them in uniform registers, which the tcgen05
// instructions take; a role of a single lane has to move them there each time.
__device__ __forceinline__ bool elect_one()
{
    uint32_t p;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(p));
    return p != 0u;
}

// Shared-memory writes of this thread, before the async proxy (an MMA) reads them.
__device__ __forceinline__ void fence_proxy_async()
{
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                   const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                   const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn()
{
    static EncodeTiledFn fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000,
                                             cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(p);
    });
    return fn;
}

// 2-D bf16 tensor map over [rows][inner] with a box of [box_rows][bk] and the
// swizzle the UMMA descriptors expect (one swizzle span per box row).
bool make_map(CUtensorMap* m, const void* base, uint64_t inner, uint64_t rows, uint32_t box_rows,
              int bk)
{
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[2] = {inner, rows};
    const cuuint64_t strides[1] = {inner * 2};
    const cuuint32_t box[2] = {(cuuint32_t)bk, box_rows};
    const cuuint32_t estr[2] = {1, 1};
    const CUtensorMapSwizzle sw = bk == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B;
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box,
              estr, CU_TENSOR_MAP_INTERLEAVE_NONE, sw, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

void set_attrs(cudaLaunchConfig_t* cfg, cudaLaunchAttribute* attr, bool pair, bool pdl)
{
    int n = 0;
    if (pair) {
        attr[n].id = cudaLaunchAttributeClusterDimension;
        attr[n].val.clusterDim.x = 2;
        attr[n].val.clusterDim.y = 1;
        attr[n].val.clusterDim.z = 1;
        ++n;
    }
    if (pdl) {
        attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[n].val.programmaticStreamSerializationAllowed = 1;
        ++n;
    }
    cfg->attrs = attr;
    cfg->numAttrs = n;
}

// CTAs of the persistent cluster grid of `kernel` (its dynamic shared memory
// attribute already set): twice the clusters that fit at once (one CTA per SM),
// within the SM budget; 0 if no cluster fits. Cached per kernel and device.
template <typename Kernel>
int cluster_grid(Kernel kernel, int threads, size_t smem, int num_sms)
{
    // Kernels of one type share this function: an entry says whose it is. (A caller with
    // more kernels and devices than entries asks each time.)
    struct Entry {
        const void* kernel;
        int dev, fit;
    };
    static std::mutex mu;
    static Entry entries[64];
    static int used = 0;
    int dev = 0, fit = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    const void* k = reinterpret_cast<const void*>(kernel);
    std::lock_guard<std::mutex> lock(mu);
    for (int i = 0; i < used && fit == 0; ++i)
        if (entries[i].kernel == k && entries[i].dev == dev) fit = entries[i].fit;
    if (fit == 0) {
        int sms = 0;
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
        cudaLaunchConfig_t cfg = {};
        cudaLaunchAttribute attr[2];
        cfg.gridDim = dim3((unsigned)(sms & ~1));
        cfg.blockDim = dim3((unsigned)threads);
        cfg.dynamicSmemBytes = smem;
        set_attrs(&cfg, attr, true, false);
        int n = 0;
        if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess || n < 1) {
            cudaGetLastError();
            return 0;
        }
        fit = 2 * n;
        if (used < 64) entries[used++] = {k, dev, fit};
    }
    const int budget = num_sms & ~1;
    return fit < budget ? fit : budget;
}

}  // namespace
}  // namespace ep
