// expert_wgrad.cu - the weight gradients of the experts' products:
//     grad_w[e][o][i] = sum over expert e's rows p of grad[p][o] * x[p][i]
// for y = x W_e^T, driven by the device counts and offsets like expert_gemm.cu.
//
// The contraction runs over the receive rows, so both operands are MN-major: TMA
// boxes of 64 rows x 64 columns land as 64 lines of 128 bytes (128-byte swizzle)
// and the instruction descriptor marks A and B as transposed; nothing is copied
// or transposed in memory. An expert's rows start anywhere and its last K slice
// holds the next expert's rows (or rows never written) behind its own: the MMAs
// of that slice stop at the last started step of 16 rows, and warp 6 zeroes the
// lines of that step which are not the expert's, in both operands (a stale NaN
// times zero would still be a NaN), before the slice is handed to the MMA thread.
//
// Tiles: 256 x 256 of one expert's grad_w on an SM pair (cta_group::2, each CTA
// holds 128 columns of grad and 128 of x), or 128 x BN on one SM. Persistent CTAs
// take (expert, row block, column block) units, column blocks fastest. An expert
// without rows gets zeros (or keeps what it has when accumulating).
//
// Roles as in expert_tile.cuh: warp 0 copies, warp 1 issues the MMAs, warps 2-5
// drain the accumulators, warp 6 repairs last slices. Every wait is bounded.
#include "umma.cuh"

namespace ep {
namespace {

constexpr int kWgradThreads = 224;
constexpr int kWgradBK = 64;        // receive rows per ring stage

template <int BN_, bool PAIR_>
struct WCfg {
    static constexpr int BN = BN_;
    static constexpr bool PAIR = PAIR_;
    static constexpr int kTileM = PAIR ? 2 * kBM : kBM;
    static constexpr int kColsB = PAIR ? BN / 2 : BN;            // x columns this CTA holds
    static constexpr int kBoxesA = kBM / 64, kBoxesB = kColsB / 64;
    static constexpr uint32_t kBytesA = kBoxesA * kMnBoxBytes;
    static constexpr uint32_t kStageBytes = (kBoxesA + kBoxesB) * kMnBoxBytes;
    // Behind the ring: barriers and flags, every expert's rows and first row, and the
    // epilogue warps' staging.
    static constexpr int kBarBytes = 512;
    static constexpr int kTail = kBarBytes + 2 * 4 * kMaxExperts + 4 * kStageWarpBytes;
    static constexpr int kFit = (kSmemLimit - 1024 - kTail) / (int)kStageBytes;
    static constexpr int STAGES = kFit > 8 ? 8 : kFit;
    static constexpr size_t kSmem = 1024 + (size_t)STAGES * kStageBytes + kTail;
    // kind::f16, fp32 accumulate, A and B bf16 and both MN-major (bits 15, 16).
    static constexpr uint32_t kIdesc = (1u << 4) | (1u << 7) | (1u << 10) | (1u << 15) |
                                       (1u << 16) | ((uint32_t)(BN >> 3) << 17) |
                                       ((uint32_t)(kTileM >> 4) << 24);
    static constexpr uint32_t kTmemCols = 2 * BN < 32 ? 32 : 2 * BN;
    static constexpr uint32_t kReleaseCount = PAIR ? 8u : 4u;
    static_assert(8 * (4 * STAGES + 5) + 16 <= kBarBytes, "barriers fit");
    static_assert(!PAIR || BN == kPairBN, "pairs use 256-column tiles");
};

struct WUnit {
    int e, mb, nb;
    int rows, k_iters;   // the expert's rows and their K slices
};

__device__ __forceinline__ WUnit wgrad_unit(const int* cnt, int nmb, int nnb, int64_t u)
{
    WUnit w;
    const int per = nmb * nnb;
    w.e = (int)(u / per);
    const int v = (int)(u - (int64_t)w.e * per);
    w.mb = v / nnb;
    w.nb = v - w.mb * nnb;
    w.rows = cnt[w.e];
    w.k_iters = (w.rows + kWgradBK - 1) / kWgradBK;
    return w;
}

// Rows of the last K slice that need repair: the slice's own rows if they end
// inside a step of 16, else 0.
__device__ __forceinline__ int ragged_rows(int rows)
{
    const int last = rows & (kWgradBK - 1);
    return (last & (kUmmaK - 1)) ? last : 0;
}

// A ragged slice takes longer to get ready than the ring looks ahead, so it is copied
// kEarly slices before its turn: it is at position ragged_at of the ring's order and
// still the last to be multiplied (see the roles). 1366 and 1402 TFLOP/s without, 1468 and
// 1494 with (mixtral rows, down and gate/up weights); 1637 and 1714 with nothing to repair.
constexpr int kEarly = 2;
__device__ __forceinline__ int ragged_at(const WUnit& w)
{
    return ragged_rows(w.rows) ? w.k_iters - 1 - min(kEarly, w.k_iters - 1) : w.k_iters - 1;
}

template <class C>
__global__ void __launch_bounds__(kWgradThreads, 1)
expert_wgrad_kernel(const __grid_constant__ CUtensorMap tm_a,
                    const __grid_constant__ CUtensorMap tm_b, WgradArgs a)
{
    constexpr int STAGES = C::STAGES, BN = C::BN;
    constexpr bool PAIR = C::PAIR;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_u32 = smem_u32(smem_raw);
    uint8_t* smem = smem_raw + ((1024u - (raw_u32 & 1023u)) & 1023u);
    const uint32_t tiles_u32 = smem_u32(smem);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + STAGES * C::kStageBytes);
    const uint32_t full0 = smem_u32(bars);               // STAGES (pairs: the leader's count)
    const uint32_t empty0 = full0 + 8u * STAGES;         // STAGES
    const uint32_t landed0 = empty0 + 8u * STAGES;       // STAGES: a ragged slice, this CTA's copies
    const uint32_t fixed0 = landed0 + 8u * STAGES;       // STAGES: a ragged slice, repaired in both CTAs
    const uint32_t accum_full0 = fixed0 + 8u * STAGES;    // 2
    const uint32_t accum_empty0 = accum_full0 + 16u;     // 2
    const uint32_t drain = accum_empty0 + 16u;
    uint32_t* s_tmem = reinterpret_cast<uint32_t*>(bars + 4 * STAGES + 5);
    volatile int* s_abort = reinterpret_cast<volatile int*>(s_tmem + 1);
    int* s_cnt = reinterpret_cast<int*>(smem + STAGES * C::kStageBytes + C::kBarBytes);
    int* s_off = s_cnt + kMaxExperts;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int r = PAIR ? cluster_rank() : 0;
    const bool leader = r == 0;
    const int first = PAIR ? cluster_index() : (int)blockIdx.x;
    const int step = PAIR ? cluster_count() : (int)gridDim.x;
    const int nmb = (int)(a.dout / C::kTileM), nnb = (int)(a.din / BN);
    const int64_t total = (int64_t)a.E * nmb * nnb;
    const uint32_t lead_full0 = PAIR ? map_to_rank(full0, 0) : full0;
    const uint32_t lead_fixed0 = PAIR ? map_to_rank(fixed0, 0) : fixed0;
    const uint32_t lead_accum_empty0 = PAIR ? map_to_rank(accum_empty0, 0) : accum_empty0;

    if (threadIdx.x == 0) {
        for (int s = 0; s < 3 * STAGES; ++s) mbar_init(full0 + 8u * s, 1u);
        for (int s = 0; s < STAGES; ++s) mbar_init(fixed0 + 8u * s, PAIR ? 2u : 1u);
        for (int b = 0; b < 2; ++b) {
            mbar_init(accum_full0 + 8u * b, 1u);
            mbar_init(accum_empty0 + 8u * b, C::kReleaseCount);
        }
        mbar_init(drain, 1u);
        *s_abort = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc<PAIR>(smem_u32(s_tmem), C::kTmemCols);
        tmem_relinquish<PAIR>();
    }
    griddep_wait();   // counts, offsets and both operands come from earlier kernels
    for (int e = threadIdx.x; e < a.E; e += kWgradThreads) {
        s_cnt[e] = __ldcg(a.cnt + e);
        s_off[e] = __ldcg(a.expert_offset + e);
    }
    tc_fence_before();
    __syncthreads();
    if (PAIR) cluster_sync();   // the peer's barriers exist before any copy or arrival reaches them
    tc_fence_after();
    const uint32_t tmem = *s_tmem;

    if (warp == 0) {
        // ---- TMA producer (each CTA fills its own ring) --------------------
        int g = 0;
        bool ok = true;
        for (int64_t u = first; u < total && ok && !*s_abort; u += step) {
            const WUnit w = wgrad_unit(s_cnt, nmb, nnb, u);
            if (w.k_iters == 0) continue;
            const int row0 = s_off[w.e];
            const int m0 = w.mb * C::kTileM + r * kBM;
            const int n0 = w.nb * BN + r * C::kColsB;
            const bool ragged = ragged_rows(w.rows) != 0;
            const int last_at = ragged_at(w);
            for (int i = 0; i < w.k_iters; ++i, ++g) {
                const int k = i < last_at ? i : i == last_at ? w.k_iters - 1 : i - 1;   // slice
                const int s = g % STAGES;
                const uint32_t ph = (uint32_t)((g / STAGES) & 1);
                ok = warp_all(wait_or_abort(empty0 + 8u * s, ph ^ 1u, s_abort));
                if (!ok) break;
                const uint32_t sa = tiles_u32 + (uint32_t)s * C::kStageBytes;
                const uint32_t sb = sa + C::kBytesA;
                const int kr = row0 + k * kWgradBK;
                // A ragged slice completes on this CTA's own barrier, for warp 6;
                // every other one on the (leader's) full barrier.
                const bool fix = ragged && k == w.k_iters - 1;
                if (elect_one()) {
                    if (fix || !PAIR) {
                        const uint32_t bar = (fix ? landed0 : full0) + 8u * s;
                        mbar_expect_tx(bar, C::kStageBytes);
#pragma unroll
                        for (int j = 0; j < C::kBoxesA; ++j)
                            tma_load_2d(sa + j * kMnBoxBytes, &tm_a, m0 + 64 * j, kr, bar);
#pragma unroll
                        for (int j = 0; j < C::kBoxesB; ++j)
                            tma_load_2d(sb + j * kMnBoxBytes, &tm_b, n0 + 64 * j, kr, bar);
                    } else {
                        if (leader) mbar_expect_tx(full0 + 8u * s, 2u * C::kStageBytes);
                        const uint32_t bar = lead_full0 + 8u * s;
#pragma unroll
                        for (int j = 0; j < C::kBoxesA; ++j)
                            tma_load_2d_pair(sa + j * kMnBoxBytes, &tm_a, m0 + 64 * j, kr, bar);
#pragma unroll
                        for (int j = 0; j < C::kBoxesB; ++j)
                            tma_load_2d_pair(sb + j * kMnBoxBytes, &tm_b, n0 + 64 * j, kr, bar);
                    }
                }
                __syncwarp();
            }
        }
        // The copies this warp issued land before shared memory goes away: the
        // MMAs (or, after an abort, the wait limit) release their stages.
        const uint64_t deadline = globaltimer_ns() + kWaitLimitNs;
        for (int i = (g > STAGES ? g - STAGES : 0); i < g; ++i)
            mbar_wait_until(empty0 + 8u * (uint32_t)(i % STAGES), (uint32_t)((i / STAGES) & 1),
                            deadline);
    } else if (warp == 1 && leader) {
        // ---- MMA issuer (pairs: the leader's, for both SMs) ----------------
        int g = 0, tl = 0;
        bool issued = false, ok = true;
        uint32_t fixed_parity = 0u;   // per stage: the phase its next ragged slice completes
        for (int64_t u = first; u < total && ok && !*s_abort; u += step) {
            const WUnit w = wgrad_unit(s_cnt, nmb, nnb, u);
            if (w.k_iters == 0) continue;
            const int acc = tl & 1, use = tl >> 1;
            ++tl;
            ok = warp_all(wait_or_abort<PAIR>(accum_empty0 + 8u * acc, (uint32_t)((use & 1) ^ 1), s_abort));
            if (!ok) break;
            tc_fence_after();
            const uint32_t d_tmem = tmem + (uint32_t)(acc * BN);
            const bool ragged = ragged_rows(w.rows) != 0;
            const int last_at = ragged_at(w);
            for (int k = 0; k < w.k_iters; ++k) {
                const int at = g + (k < last_at ? k : k < w.k_iters - 1 ? k + 1 : last_at);
                const int s = at % STAGES;
                ok = warp_all(wait_or_abort(full0 + 8u * s, (uint32_t)((at / STAGES) & 1), s_abort));
                if (ok && ragged && k == w.k_iters - 1) {
                    ok = warp_all(wait_or_abort<PAIR>(fixed0 + 8u * s, (fixed_parity >> s) & 1u, s_abort));
                    fixed_parity ^= 1u << s;
                }
                if (!ok) break;
                tc_fence_after();
                const uint32_t sa = tiles_u32 + (uint32_t)s * C::kStageBytes;
                const int left = w.rows - k * kWgradBK;
                const int steps = left >= kWgradBK ? kWgradBK / kUmmaK
                                                   : (left + kUmmaK - 1) / kUmmaK;
                if (elect_one()) {
#pragma unroll
                    for (int j = 0; j < kWgradBK / kUmmaK; ++j)
                        if (j < steps)
                            umma_bf16<PAIR>(d_tmem, smem_desc_mn(sa + j * (kUmmaK * kMnLineBytes)),
                                            smem_desc_mn(sa + C::kBytesA + j * (kUmmaK * kMnLineBytes)),
                                            C::kIdesc, (k | j) != 0 ? 1u : 0u);
                    umma_commit<PAIR>(empty0 + 8u * s);
                    if (k == w.k_iters - 1) umma_commit<PAIR>(accum_full0 + 8u * acc);
                }
                __syncwarp();
                issued = true;
            }
            g += w.k_iters;
        }
        if (issued) {
            if (elect_one()) umma_commit_local<PAIR>(drain);
            __syncwarp();
            mbar_wait(drain, 0u);
        }
    } else if (warp >= 2 && warp < 6) {
        // ---- epilogue: TMEM -> grad_w ---------------------------------------
        const int quarter = warp & 3;
        const int m0 = r * kBM + quarter * 32;   // this warp's rows of the tile
        const uint32_t stage = smem_u32(s_off + kMaxExperts) + (uint32_t)(quarter * kStageWarpBytes);
        const uint32_t t_lane = tmem + ((uint32_t)(quarter * 32) << 16);
        int tl = 0;
        for (int64_t u = first; u < total && !*s_abort; u += step) {
            const WUnit w = wgrad_unit(s_cnt, nmb, nnb, u);
            const bool empty = w.k_iters == 0;
            if (empty && a.accumulate) continue;
            const int acc = tl & 1, use = tl >> 1;
            if (!empty) {
                if (!warp_all(wait_or_abort(accum_full0 + 8u * acc, (uint32_t)(use & 1), s_abort)))
                    break;
                tc_fence_after();
                ++tl;
            }
            const int64_t at = ((int64_t)w.e * a.dout + w.mb * C::kTileM + m0) * a.din + w.nb * BN;
#pragma unroll 1
            for (int c = 0; c < BN; c += 32) {
                float v[32];
                if (empty) {
#pragma unroll
                    for (int i = 0; i < 32; ++i) v[i] = 0.0f;
                } else {
                    uint32_t q[32];
                    tmem_ld32(t_lane + (uint32_t)(acc * BN + c), q);
                    tmem_wait_ld();
                    as_floats(q, v);
                }
                if (a.f32) {
                    float4* dst = reinterpret_cast<float4*>(static_cast<float*>(a.grad_w) + at +
                                                            lane * a.din + c);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        float4 o = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
                        if (a.accumulate) {
                            const float4 p = __ldcg(dst + i);
                            o.x += p.x; o.y += p.y; o.z += p.z; o.w += p.w;
                        }
                        dst[i] = o;
                    }
                } else {
                    uint16_t* dst = static_cast<uint16_t*>(a.grad_w) + at + c;
                    if (a.accumulate) {
                        int4 old[4];
                        float p[32];
                        warp_fetch_bf16x32(old, lane, dst, a.din, 32);
                        warp_spread_bf16x32(stage, lane, old, p);
#pragma unroll
                        for (int i = 0; i < 32; ++i) v[i] += p[i];
                    }
                    warp_store_bf16x32(stage, lane, v, dst, a.din, 32);
                }
            }
            if (!empty) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if (PAIR) mbar_arrive_cluster(lead_accum_empty0 + 8u * acc);
                    else mbar_arrive(accum_empty0 + 8u * acc);
                }
            }
        }
    } else if (warp == 6) {
        // ---- repair of ragged last slices -------------------------------------
        int g = 0;
        uint32_t parity = 0u;   // per stage: the phase its next ragged slice completes
        for (int64_t u = first; u < total && !*s_abort; u += step) {
            const WUnit w = wgrad_unit(s_cnt, nmb, nnb, u);
            const int valid = ragged_rows(w.rows);
            const int s = (g + ragged_at(w)) % STAGES;
            g += w.k_iters;
            if (valid == 0) continue;
            const uint32_t par = (parity >> s) & 1u;
            parity ^= 1u << s;
            if (!warp_all(wait_or_abort(landed0 + 8u * s, par, s_abort))) break;
            // Lines [valid, end of the step) of every box of both operands.
            const int lines = ((valid + kUmmaK - 1) & ~(kUmmaK - 1)) - valid;
            uint8_t* stage = smem + (size_t)s * C::kStageBytes;
            for (int i = lane; i < (C::kBoxesA + C::kBoxesB) * lines * 8; i += 32) {
                const int line = i >> 3, box = line / lines;
                *reinterpret_cast<int4*>(stage + box * kMnBoxBytes +
                                         (valid + line - box * lines) * kMnLineBytes +
                                         (i & 7) * 16) = make_int4(0, 0, 0, 0);
            }
            fence_proxy_async();   // the MMAs read shared memory through the async proxy
            __syncwarp();
            if (lane == 0) {
                if (leader) mbar_arrive(full0 + 8u * s);   // its phase passes without copies
                if (PAIR) mbar_arrive_cluster(lead_fixed0 + 8u * s);
                else mbar_arrive(fixed0 + 8u * s);
            }
        }
    }

    __syncwarp();
    if (threadIdx.x == 0 && *s_abort) atomicOr(a.err, kErrTimeout);
    tc_fence_before();
    __syncthreads();
    if (PAIR) cluster_sync();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc<PAIR>(tmem, C::kTmemCols);
    }
    griddep_launch_dependents();
}

template <class C>
cudaError_t launch_wcfg(const WgradArgs& a, const void* grad, const void* x, int64_t rows,
                        int num_sms, const LaunchOpts& o)
{
    cudaError_t e = cudaFuncSetAttribute(expert_wgrad_kernel<C>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::kSmem);
    if (e != cudaSuccess) return e;
    int grid = num_sms;
    if (C::PAIR) {
        grid = cluster_grid(expert_wgrad_kernel<C>, kWgradThreads, C::kSmem, num_sms);
        if (grid < 2) return cudaErrorNotSupported;
    }
    CUtensorMap ta, tb;
    if (!make_map(&ta, grad, (uint64_t)a.dout, (uint64_t)rows, kWgradBK, 64) ||
        !make_map(&tb, x, (uint64_t)a.din, (uint64_t)rows, kWgradBK, 64))
        return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(kWgradThreads);
    cfg.dynamicSmemBytes = C::kSmem;
    cfg.stream = o.stream;
    set_attrs(&cfg, attr, C::PAIR, o.pdl);
    e = cudaLaunchKernelEx(&cfg, expert_wgrad_kernel<C>, ta, tb, a);
    if (e == cudaSuccess && o.launches) ++*o.launches;
    return e;
}

}  // namespace

cudaError_t launch_expert_wgrad(const WgradArgs& a, const void* grad, const void* x, int64_t rows,
                                int grid, const LaunchOpts& o)
{
    if (a.din % 64 != 0 || a.dout % 128 != 0) return cudaErrorInvalidValue;
    if (a.dout % 256 == 0 && a.din % kPairBN == 0) {
        const cudaError_t e = launch_wcfg<WCfg<kPairBN, true>>(a, grad, x, rows, grid, o);
        if (e != cudaErrorNotSupported) return e;
    }
    if (a.din % 256 == 0) return launch_wcfg<WCfg<256, false>>(a, grad, x, rows, grid, o);
    if (a.din % 128 == 0) return launch_wcfg<WCfg<128, false>>(a, grad, x, rows, grid, o);
    return launch_wcfg<WCfg<64, false>>(a, grad, x, rows, grid, o);
}

}  // namespace ep
