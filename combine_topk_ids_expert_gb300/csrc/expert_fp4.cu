// expert_fp4.cu - the experts' products in microscaled 4-bit floating point,
//     y[p] = x[p] W_e^T,   or   h[p] = act(x[p] Wg^T) * (x[p] Wu^T)
// over each expert's receive rows, with x and W as codes and block scales (fp4.cuh) on the
// block-scaled tcgen05 instructions; h leaves as bf16 or quantised again, so that a block is
// two kernels and nothing in between is wider than 4 bits.
//
// The tile list, its schedule and the roles are the grouped GEMM's (expert_tile.cuh). What
// differs: a ring stage is 256 elements of K (128 bytes of codes, one swizzle span) with the
// scales of its rows; four more warps bring the scales, each every fourth stage. A tile of
// receive rows starts anywhere in the 128-row tiles that scales lie in, so its scales are
// copied row by row, 4 bytes for 4 blocks, to where the tile's own rows want them; W's come
// as whole tiles by TMA (gated tiles of one SM: half lines, by the warps). The issuing thread moves a
// stage's scales to tensor memory and multiplies; both run in order.
//
// Tensor memory: the accumulator of 256 columns (an SM pair, tiles of 256 rows x 256 columns)
// does not fit twice beside the scales, so the two accumulators overlap: each tile's epilogue
// drains the shared columns first and lets the next tile begin. Tiles of one SM are 128 x 128
// with two whole accumulators.
//
// Products are exact and summed in fp32; tensor scales enter in the epilogue.
//
// Measured (nv, the block with its dispatch; 8192 rows over 8 experts, 4096 -> 2 x 2048 -> 4096):
// 186 us as it was first; 160 with W's scales by TMA onto the pair's own barrier (copied row by
// row, or completed on a barrier of their own, they came late); 156 with descriptors moved by
// additions; 145 with the dispatch in one kernel; 118 with arrivals that order shared memory
// only (a release at cluster scope, 0.5 to 1 us each, was in the chain of every stage and of
// every change of tiles). A stage's MMAs take 512 cycles; the first stages of a tile, which are
// there already, take about 610. Tried without gain: the next tile found a tile ahead, codes
// prefetched to L2, scales moved to tensor memory in one stage of a tile only (to time it).
#include "ep_fp4.cuh"
#include "expert_tile.cuh"
#include "fp4_umma.cuh"

namespace ep {
namespace {

constexpr int kScaleWarps = 4, kDrainWarps = 8;
constexpr int kFp4Threads = 32 * (2 + kDrainWarps + kScaleWarps);
constexpr uint32_t kTmemAll = 512;

enum Fp4Out { kOutPlain = 0, kOutGluBf16 = 1, kOutGluFp4 = 2 };

template <int FMT_, bool PAIR_, int OUT_, int STAGES_>
struct Fp4Cfg {
    static constexpr int FMT = FMT_, OUT = OUT_, STAGES = STAGES_;
    static constexpr bool PAIR = PAIR_, GLU = OUT_ != kOutPlain;
    static constexpr bool kHalves = GLU && !PAIR;     // W's scales in half lines, by a warp
    static constexpr int BN = PAIR ? 256 : 128;
    static constexpr int kOutBN = GLU ? BN / 2 : BN;
    static constexpr int kTileRows = PAIR ? 256 : 128;
    static constexpr int kTiles = Fp4Mma<FMT>::kTiles;
    static constexpr uint32_t kBytesA = kBM * 128, kBytesB = 128 * 128;   // 128 rows of W in each CTA
    static constexpr uint32_t kScalesA = kTiles * kScaleTile;
    static constexpr uint32_t kScalesB = kTiles * (BN / 128) * kScaleTile;
    static constexpr uint32_t kStageBytes = kBytesA + kBytesB + kScalesA + kScalesB;
    static constexpr uint32_t kColsA = 4 * kTiles, kColsB = 4 * kTiles * (BN / 128);
    // Columns of scales, two stages' worth where they fit.
    static constexpr int kScaleBufs = PAIR && FMT == kFp4Nv ? 1 : 2;
    static constexpr uint32_t kScaleCols = kScaleBufs * (kColsA + kColsB);
    static constexpr uint32_t kScaleCol0 = kTmemAll - kScaleCols;
    static constexpr uint32_t kAcc1 = PAIR ? kScaleCol0 - BN : BN;        // second accumulator
    static constexpr uint32_t kIdesc = Fp4Mma<FMT>::idesc(kTileRows, BN);
    // Arrivals that let an accumulator be written again.
    static constexpr uint32_t kReleaseCount = kDrainWarps * (PAIR ? 2u : 1u);
    static constexpr uint32_t kFullCount = PAIR ? 3u : 2u;   // the copies, each CTA's scales
    static constexpr size_t kTail = kDrainWarps * kStageWarpBytes + 8 * (2 * STAGES + 6) + 16 +
                                    8 * (kMaxExperts + 1) + 4 * kMaxExperts;
    static constexpr size_t kSmem = 1024 + (size_t)STAGES * kStageBytes + kTail;
    static_assert(kSmem <= (size_t)kSmemLimit, "ring does not fit in shared memory");
    static_assert(kAcc1 + BN <= kScaleCol0, "accumulators and scales overlap");
    // A warp that serves every n-th stage waits for a slot's last release by parity: it must not
    // get there while the release before that one is out, which its own last stage rules out as
    // long as that is at most a ring's length ago.
    static_assert(kScaleWarps <= STAGES, "a warp's stages within the ring");
};

struct Fp4GemmArgs {
    const int32_t* cnt;
    const int32_t* expert_offset;
    const uint8_t* x_scales;
    const uint8_t* w_scales;
    const float* x_scale;          // one number or null
    const float* w_scale;          // [E] or null
    const float* h_scale;          // one number or null (quantised h)
    void* y;                       // bf16 rows, or codes
    uint8_t* y_scales;             // scales of quantised h
    int64_t din, dout, rows;       // rows: receive rows
    int E, act, light_rows;
    uint32_t* err;
};

// The scales of a stage that pass a warp's registers, fetched ahead of the stage's turn: those of
// the tile's 128 receive rows at row0, 4 bytes at a time, and, in the gated tiles of one SM, those
// of 64 gate rows and 64 up rows, half a line each. (W's others are copied as they lie.)
template <class C>
struct StageScales {
    uint32_t x[4][C::kTiles];
    uint2 w[C::kHalves ? 2 : 1][C::kTiles];

    __device__ __forceinline__ void fetch(const Fp4GemmArgs& a, int e, int nb, int64_t row0, int stage,
                                          int lane)
    {
        const int64_t tiles = a.din / (4 * Fp4<C::FMT>::kBlock), kt0 = (int64_t)stage * C::kTiles;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            // Rows behind the last receive row do not exist: the last one's scales instead.
            const int64_t row = min(row0 + 32 * q + lane, a.rows - 1);
            const uint8_t* src = a.x_scales + fp4_scale_at(row, kt0, tiles);
#pragma unroll
            for (int j = 0; j < C::kTiles; ++j)
                x[q][j] = kt0 + j < tiles ? __ldcg(reinterpret_cast<const uint32_t*>(src + j * 512)) : 0u;
        }
        if (C::kHalves) {
#pragma unroll
            for (int b = 0; b < (C::kHalves ? 2 : 1); ++b) {
                const int64_t row = ((int64_t)e * 2 + b) * a.dout + nb * C::kOutBN;
                const uint8_t* src = a.w_scales + fp4_scale_at(row, kt0, tiles) + lane * 16;
#pragma unroll
                for (int j = 0; j < C::kTiles; ++j)
                    w[b][j] = kt0 + j < tiles ? __ldcg(reinterpret_cast<const uint2*>(src + j * 512))
                                              : make_uint2(0u, 0u);
            }
        }
    }

    __device__ __forceinline__ void store(uint32_t s_a, uint32_t s_b, int lane) const
    {
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int j = 0; j < C::kTiles; ++j) sts32(s_a + j * kScaleTile + lane * 16 + q * 4, x[q][j]);
        if (C::kHalves) {
#pragma unroll
            for (int b = 0; b < (C::kHalves ? 2 : 1); ++b)
#pragma unroll
                for (int j = 0; j < C::kTiles; ++j)
                    sts64(s_b + j * kScaleTile + lane * 16 + b * 8, w[b][j]);
        }
    }
};

// 32 fp32 elements of a row as codes and scales in a matrix of `cols` columns.
template <int FMT>
__device__ __forceinline__ void store_fp4x32(const float (&v)[32], float g, uint8_t* codes,
                                             uint8_t* scales, int64_t row, int64_t col, int64_t cols)
{
    const int64_t tiles = cols / (4 * Fp4<FMT>::kBlock);
    float lo[16], hi[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        lo[i] = v[i];
        hi[i] = v[16 + i];
    }
    const float m0 = amax16(lo), m1 = amax16(hi);
    uint2 c0, c1;
    if (FMT == kFp4Mx) {
        const uint32_t c = fp4_scale_code<FMT>(
            __uint_as_float(max(__float_as_uint(m0), __float_as_uint(m1))), 1.0f);
        c0 = fp4_codes16<FMT, false>(lo, c, 1.0f);
        c1 = fp4_codes16<FMT, false>(hi, c, 1.0f);
        const int64_t block = col / 32;
        scales[fp4_scale_at(row, block >> 2, tiles) + (block & 3)] = (uint8_t)c;
    } else {
        const uint32_t s0 = fp4_scale_code<FMT>(m0, g), s1 = fp4_scale_code<FMT>(m1, g);
        c0 = fp4_codes16<FMT, true>(lo, s0, g);
        c1 = fp4_codes16<FMT, true>(hi, s1, g);
        const int64_t block = col / 16;
        *reinterpret_cast<uint16_t*>(scales + fp4_scale_at(row, block >> 2, tiles) + (block & 3)) =
            (uint16_t)(s0 | (s1 << 8));
    }
    *reinterpret_cast<uint4*>(codes + row * (cols / 2) + col / 2) = make_uint4(c0.x, c0.y, c1.x, c1.y);
}

template <class C>
__global__ void __launch_bounds__(kFp4Threads, 1)
expert_fp4_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b,
                  const __grid_constant__ CUtensorMap tm_s, const Fp4GemmArgs a)
{
    constexpr int STAGES = C::STAGES, BN = C::BN;
    constexpr bool PAIR = C::PAIR;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_u32 = smem_u32(smem_raw);
    uint8_t* smem = smem_raw + ((1024u - (raw_u32 & 1023u)) & 1023u);
    const uint32_t ring = smem_u32(smem);                  // codes, then the stages' scales
    const uint32_t ring_scales = ring + STAGES * (C::kBytesA + C::kBytesB);
    uint8_t* tail = smem + STAGES * C::kStageBytes;
    uint64_t* bars = reinterpret_cast<uint64_t*>(tail + kDrainWarps * kStageWarpBytes);
    const uint32_t full0 = smem_u32(bars);                 // STAGES (pairs: the leader's count)
    const uint32_t empty0 = full0 + 8u * STAGES;           // STAGES
    const uint32_t accum_full0 = empty0 + 8u * STAGES;     // 2
    const uint32_t accum_free0 = accum_full0 + 16u;        // 2 (pairs: the leader's count)
    const uint32_t drain = accum_free0 + 16u;
    uint32_t* s_tmem = reinterpret_cast<uint32_t*>(bars + 2 * STAGES + 5);
    volatile int* s_abort = reinterpret_cast<volatile int*>(s_tmem + 1);
    int* s_heavy = const_cast<int*>(reinterpret_cast<volatile int*>(s_abort + 1));
    int* s_light = s_heavy + (kMaxExperts + 1);
    int* s_cnt = s_light + (kMaxExperts + 1);
    const int E = a.E;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int r = PAIR ? cluster_rank() : 0;
    const bool leader = r == 0;
    const int first = PAIR ? cluster_index() : (int)blockIdx.x;
    const int step = PAIR ? cluster_count() : (int)gridDim.x;
    const int k_iters = (int)((a.din + kFp4StageK - 1) / kFp4StageK);
    const int nbk = (int)(a.dout / C::kOutBN);
    const uint32_t lead_full0 = PAIR ? map_to_rank(full0, 0) : full0;
    const uint32_t lead_free0 = PAIR ? map_to_rank(accum_free0, 0) : accum_free0;

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(full0 + 8u * s, C::kFullCount);
            mbar_init(empty0 + 8u * s, 1u);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(accum_full0 + 8u * b, 1u);
            mbar_init(accum_free0 + 8u * b, C::kReleaseCount);
        }
        mbar_init(drain, 1u);
        *s_abort = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc<PAIR>(smem_u32(s_tmem), kTmemAll);
        tmem_relinquish<PAIR>();
    }
    griddep_wait();   // counts, offsets and the receive rows come from earlier kernels
    if (warp == 0) row_tile_prefixes(a.cnt, E, a.light_rows, C::kTileRows, s_heavy, s_light, s_cnt);
    tc_fence_before();
    __syncthreads();
    if (PAIR) cluster_sync();
    tc_fence_after();
    const uint32_t tmem = *s_tmem;
    Schedule q;
    q.heavy = s_heavy;
    q.light = s_light;
    q.cnt = s_cnt;
    q.tile_rows = C::kTileRows;
    q.halves = false;
    q.uh = s_heavy[E] * nbk;
    q.total = q.uh + s_light[E] * nbk;
    const int total = q.total;

    if (warp == 0) {
        // ---- codes, and W's scales --------------------------------------------
        const int tiles = (int)(a.din / (4 * Fp4<C::FMT>::kBlock));
        int g = 0;
        bool ok = true;
        for (int u = first; u < total && ok && !*s_abort; u += step) {
            const TileRef p = tile_of(q, E, nbk, u);
            const int row0 = __ldcg(a.expert_offset + p.e) + p.mt * C::kTileRows + r * kBM;
            // The first of this CTA's rows of W; with the gated projections of one SM, 64 gate
            // rows and 64 up rows (a pair: gate rows in the leader, up rows in the other).
            const int w0 = C::GLU ? p.e * 2 * (int)a.dout + p.nb * C::kOutBN + r * (int)a.dout
                                  : p.e * (int)a.dout + p.nb * BN + r * 128;
            // The first of the 128-row groups of W whose scales the tile takes, and the next one's
            // distance.
            const int g0 = (C::GLU ? p.e * 2 * (int)a.dout + p.nb * C::kOutBN
                                   : p.e * (int)a.dout + p.nb * BN) >> 7;
            const int g_step = C::GLU ? (int)a.dout >> 7 : 1;
            for (int k = 0; k < k_iters; ++k, ++g) {
                const int s = g % STAGES;
                ok = warp_all(wait_or_abort(empty0 + 8u * s, (uint32_t)(((g / STAGES) & 1) ^ 1), s_abort));
                if (!ok) break;
                const uint32_t sa = ring + (uint32_t)s * (C::kBytesA + C::kBytesB);
                const uint32_t sb = sa + C::kBytesA;
                const uint32_t ss = ring_scales + (uint32_t)s * (C::kScalesA + C::kScalesB) + C::kScalesA;
                const int kc = k * (kFp4StageK / 2);
                // The last stage may be half a stage: what is copied behind the last column is not
                // multiplied.
                constexpr uint32_t kBytes = C::kBytesA + C::kBytesB + (C::kHalves ? 0u : C::kScalesB);
                if (elect_one()) {
                    const uint32_t fb = PAIR ? lead_full0 + 8u * s : full0 + 8u * s;
                    // Both CTAs of a pair copy onto the leader's barrier, which expects both.
                    if (leader) mbar_expect_tx(full0 + 8u * s, (PAIR ? 2u : 1u) * kBytes);
                    auto load = [&](uint32_t dst, const CUtensorMap* tm, int c0, int c1) {
                        if (PAIR) tma_load_2d_pair(dst, tm, c0, c1, fb);
                        else tma_load_2d(dst, tm, c0, c1, fb);
                    };
                    load(sa, &tm_a, kc, row0);
                    load(sb, &tm_b, kc, w0);
                    if (C::kHalves) {
                        load(sb + C::kBytesB / 2, &tm_b, kc, w0 + (int)a.dout);
                    } else {
#pragma unroll
                        for (int b = 0; b < BN / 128; ++b)
                            load(ss + b * C::kTiles * kScaleTile, &tm_s, 0,
                                 (g0 + b * g_step) * tiles + k * C::kTiles);
                    }
                }
                __syncwarp();
            }
        }
        // The copies this warp issued land before shared memory goes away.
        const uint64_t deadline = globaltimer_ns() + kWaitLimitNs;
        for (int i = (g > STAGES ? g - STAGES : 0); i < g; ++i)
            mbar_wait_until(empty0 + 8u * (i % STAGES), (uint32_t)((i / STAGES) & 1), deadline);
    } else if (warp == 1 && leader) {
        // ---- scales to tensor memory, products --------------------------------
        constexpr uint32_t kCodeStep = (C::kBytesA + C::kBytesB) >> 4;     // a stage's, in descriptors
        constexpr uint32_t kScaleStep = (C::kScalesA + C::kScalesB) >> 4;
        const uint32_t code0 = desc_lo(ring), scale0 = desc_lo(ring_scales);
        uint32_t code = code0, scale = scale0;         // the slot's
        uint32_t ts = 0u, phase = 0u;                  // scale columns, the slot's parity
        int s = 0, tl = 0;
        bool issued = false, ok = true;
        for (int u = first; u < total && ok && !*s_abort; u += step, ++tl) {
            const int acc = tl & 1;
            // A pair: the tile before has drained the columns that both accumulators have.
            // One SM: the last tile of this accumulator has been drained.
            if (PAIR) ok = tl == 0 || wait_or_abort<PAIR>(accum_free0, (uint32_t)((tl - 1) & 1), s_abort);
            else ok = wait_or_abort<PAIR>(accum_free0 + 8u * acc, (uint32_t)(((tl >> 1) & 1) ^ 1), s_abort);
            ok = warp_all(ok);
            if (!ok) break;
            tc_fence_after();
            const uint32_t d_tmem = tmem + (acc ? C::kAcc1 : 0u);
            int left = (int)a.din / kFp4K;             // steps of the contraction
            for (uint32_t some = 0u; left > 0; left -= kFp4StageK / kFp4K, some = 1u) {
                ok = warp_all(wait_or_abort<PAIR>(full0 + 8u * s, phase, s_abort));
                if (!ok) break;
                tc_fence_after();
                if (elect_one()) {
                    const uint32_t ta = tmem + C::kScaleCol0 + ts, tb = ta + C::kColsA;
#pragma unroll
                    for (int j = 0; j < C::kTiles; ++j)
                        tmem_copy_scales<PAIR>(ta + 4u * j,
                                               desc_of(scale + j * (kScaleTile >> 4), kScaleDescHi));
#pragma unroll
                    for (int j = 0; j < C::kTiles * (BN / 128); ++j)
                        tmem_copy_scales<PAIR>(
                            tb + 4u * j,
                            desc_of(scale + (C::kScalesA >> 4) +
                                        (j % (BN / 128) * C::kTiles + j / (BN / 128)) * (kScaleTile >> 4),
                                    kScaleDescHi));
#pragma unroll
                    for (int j = 0; j < kFp4StageK / kFp4K; ++j) {
                        if (j >= left) break;
                        const int t = Fp4Mma<C::FMT>::tile_of_step(j);
                        umma_fp4<C::FMT, PAIR>(d_tmem, desc_of(code + j * (kFp4K / 2 >> 4), kCodeDescHi),
                                               desc_of(code + ((C::kBytesA + j * (kFp4K / 2)) >> 4), kCodeDescHi),
                                               Fp4Mma<C::FMT>::idesc_step(C::kIdesc, j), ta + 4u * t,
                                               tb + 4u * t * (BN / 128), j == 0 ? some : 1u);
                    }
                    umma_commit<PAIR>(empty0 + 8u * s);
                    if (left <= kFp4StageK / kFp4K) umma_commit<PAIR>(accum_full0 + 8u * acc);
                }
                __syncwarp();
                issued = true;
                if (C::kScaleBufs == 2) ts ^= C::kColsA + C::kColsB;
                code += kCodeStep;
                scale += kScaleStep;
                if (++s == STAGES) {
                    s = 0;
                    phase ^= 1u;
                    code = code0;
                    scale = scale0;
                }
            }
        }
        if (issued) {
            if (elect_one()) umma_commit_local<PAIR>(drain);
            __syncwarp();
            mbar_wait(drain, 0u);
        }
    } else if (warp >= 2 && warp < 2 + kDrainWarps) {
        // ---- epilogue ---------------------------------------------------------
        const int quarter = warp & 3;                  // TMEM lanes this warp may read
        const int half = (warp - 2) >> 2;              // which of the blocks of 32 columns in turn
        const uint32_t t_lane = tmem + ((uint32_t)(quarter * 32) << 16);
        const uint32_t stage = ring + STAGES * C::kStageBytes + (uint32_t)((warp - 2) * kStageWarpBytes);
        const float gx = a.x_scale ? __ldcg(a.x_scale) : 1.0f;
        const float gh = C::OUT == kOutGluFp4 && a.h_scale ? __ldcg(a.h_scale) : 1.0f;
        constexpr int kBlocks = C::kOutBN / 32;        // of output columns
        constexpr int kRounds = kBlocks / 2;
        int tl = 0;
        for (int u = first; u < total && !*s_abort; u += step, ++tl) {
            const int acc = tl & 1;
            const uint32_t t_acc = t_lane + (acc ? C::kAcc1 : 0u);
            const TileRef p = tile_of(q, E, nbk, u);
            const int m_in = p.mt * C::kTileRows + r * kBM + 32 * quarter;
            const int rows = q.cnt[p.e] - m_in;        // of this warp's 32
            const int64_t row0 = (int64_t)__ldcg(a.expert_offset + p.e) + m_in;
            const float gw = gx * (a.w_scale ? __ldcg(a.w_scale + p.e) : 1.0f);
            if (!warp_all(wait_or_abort(accum_full0 + 8u * acc, (uint32_t)((tl >> 1) & 1), s_abort))) break;
            tc_fence_after();
            const int64_t col0 = (int64_t)p.nb * C::kOutBN;
#pragma unroll 1
            for (int i = 0; i < kRounds; ++i) {
                // The first accumulator shares its last columns with the second's first ones:
                // one is drained from the end, the other from the beginning.
                const int c = 32 * (2 * (acc ? i : kRounds - 1 - i) + half);
                uint32_t q32[32];
                float v[32];
                tmem_ld32(t_acc + (uint32_t)c, q32);
                if (C::GLU) {
                    uint32_t qu[32];
                    tmem_ld32(t_acc + (uint32_t)(c + C::kOutBN), qu);
                    tmem_wait_ld();
                    // Both accumulators have no column of what is left to drain (see below).
                    if (PAIR && i == 0) {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive_cluster_own(lead_free0);
                    }
#pragma unroll
                    for (int n = 0; n < 32; ++n)
                        v[n] = __uint_as_float(qu[n]) * gw *
                               act_value(__uint_as_float(q32[n]) * gw, a.act);
                } else {
                    tmem_wait_ld();
                    if (PAIR && i == 0) {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive_cluster_own(lead_free0);
                    }
#pragma unroll
                    for (int n = 0; n < 32; ++n) v[n] = __uint_as_float(q32[n]) * gw;
                }
                if (C::OUT == kOutGluFp4) {
                    if (lane < rows)
                        store_fp4x32<C::FMT>(v, gh, static_cast<uint8_t*>(a.y), a.y_scales,
                                             row0 + lane, col0 + c, a.dout);
                } else {
                    warp_store_bf16x32(stage, lane, v,
                                       static_cast<uint16_t*>(a.y) + row0 * a.dout + col0 + c, a.dout,
                                       rows);
                }
            }
            if (!PAIR) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(accum_free0 + 8u * acc);
            }
        }
    } else if (warp >= 2 + kDrainWarps) {
        // ---- scales to shared memory: every kScaleWarps-th stage, the warp's next one on its way
        StageScales<C> next;
        int pu = first, pk = warp - 2 - kDrainWarps;   // unit and stage that are fetched for
        TileRef pp = {};
        int64_t prow0 = 0;
        auto enter = [&] {
            while (pu < total && pk >= k_iters) {
                pk -= k_iters;
                pu += step;
            }
            if (pu >= total) return;
            pp = tile_of(q, E, nbk, pu);
            prow0 = (int64_t)__ldcg(a.expert_offset + pp.e) + pp.mt * C::kTileRows + r * kBM;
        };
        enter();
        if (pu < total) next.fetch(a, pp.e, pp.nb, prow0, pk, lane);
        const int stages = first < total ? ((total - 1 - first) / step + 1) * k_iters : 0;
        for (int g = warp - 2 - kDrainWarps; g < stages && !*s_abort; g += kScaleWarps) {
            const int s = g % STAGES;
            if (!warp_all(wait_or_abort(empty0 + 8u * s, (uint32_t)(((g / STAGES) & 1) ^ 1), s_abort))) break;
            const uint32_t ss = ring_scales + (uint32_t)s * (C::kScalesA + C::kScalesB);
            next.store(ss, ss + C::kScalesA, lane);
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) {
                if (PAIR) mbar_arrive_cluster_own(lead_full0 + 8u * s);
                else mbar_arrive(full0 + 8u * s);
            }
            // Not before: the fence and the arrival would wait for these loads.
            pk += kScaleWarps;
            if (pk >= k_iters) enter();
            if (pu < total) next.fetch(a, pp.e, pp.nb, prow0, pk, lane);
        }
    }

    __syncwarp();
    if (threadIdx.x == 0 && *s_abort) atomicOr(a.err, kErrTimeout);
    tc_fence_before();
    __syncthreads();
    if (PAIR) cluster_sync();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc<PAIR>(tmem, kTmemAll);
    }
    griddep_launch_dependents();
}

template <int FMT, bool PAIR, int OUT>
cudaError_t launch_form(const ExpertFp4Args& f, int num_sms, const LaunchOpts& o)
{
    using C = Fp4Cfg<FMT, PAIR, OUT, 5>;
    auto kernel = expert_fp4_kernel<C>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::kSmem);
    if (e != cudaSuccess) return e;
    int grid = num_sms;
    if (PAIR) {
        grid = cluster_grid(kernel, kFp4Threads, C::kSmem, num_sms);
        if (grid < 2) return cudaErrorNotSupported;
    }
    CUtensorMap ta, tb, ts;
    const uint64_t wrows = (uint64_t)f.E * (uint64_t)(C::GLU ? 2 * f.dout : f.dout);
    if (!make_code_map(&ta, f.x_codes, (uint64_t)f.din, (uint64_t)f.rows, kBM) ||
        !make_code_map(&tb, f.w_codes, (uint64_t)f.din, wrows, C::kHalves ? 64 : 128) ||
        !make_scale_map(&ts, f.w_scales, wrows / 128 * (uint64_t)(f.din / (4 * Fp4<FMT>::kBlock)),
                        C::kTiles))
        return cudaErrorInvalidValue;
    Fp4GemmArgs a = {};
    a.cnt = f.cnt;
    a.expert_offset = f.expert_offset;
    a.x_scales = f.x_scales;
    a.w_scales = f.w_scales;
    a.x_scale = f.x_scale;
    a.w_scale = f.w_scale;
    a.h_scale = f.h_scale;
    a.y = f.y;
    a.y_scales = f.y_scales;
    a.din = f.din;
    a.dout = f.dout;
    a.rows = f.rows;
    a.E = f.E;
    a.act = f.act;
    a.light_rows = f.light_rows;
    a.err = f.err;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(kFp4Threads);
    cfg.dynamicSmemBytes = C::kSmem;
    cfg.stream = o.stream;
    set_attrs(&cfg, attr, PAIR, o.pdl);
    e = cudaLaunchKernelEx(&cfg, kernel, ta, tb, ts, a);
    if (e == cudaSuccess && o.launches) ++*o.launches;
    return e;
}

template <int FMT, int OUT>
cudaError_t launch_out(const ExpertFp4Args& f, int num_sms, const LaunchOpts& o)
{
    // Pairs (256 x 256) where every pair of SMs has a tile and an expert's rows fill more than a
    // tile of single SMs (128 x 128) on average. The whole block in nv, single SMs against pairs, us
    // by rows of an expert:
    //                                          8           32           64           128          256
    //     256 experts, 7168 wide, dff 2048   976 / 1049  1006 / 1080  1042 / 1114  1347 / 1171
    //     256 experts, 2048 wide, dff 512    125 / 145    134 / 152    141 / 158    189 / 177
    //     64 experts, 4096 wide, dff 2048                 173 / 182    175 / 186    226 / 199    333 / 259
    //     8 experts, 4096 wide, dff 2048      45 / 47      43 / 47      44 / 49      53 / 52      67 / 63
    //     16 experts, 1024 wide, dff 512      19 / 23      20 / 24      20 / 25      26 / 27      30 / 33
    // (the last one has a tile for every pair from 512 rows on). Skewed (Zipf), the first one takes
    // 1184 / 1173 with 64 rows on average and 1396 / 1300 with 112, uniform with 112 1103 / 1133.
    // Calls with less than a row of an expert are 7% slower to 9% faster on single SMs, by the width.
    constexpr int64_t kPairRows = 96;
    const int64_t cols = f.glu ? 2 * f.dout : f.dout;
    if (f.kind != 1 && cols % 256 == 0 &&
        (f.kind == 2 || (f.mean_rows >= kPairRows && 2 * f.row_tiles * (cols / 256) >= num_sms))) {
        const cudaError_t e = launch_form<FMT, true, OUT>(f, num_sms, o);
        if (e != cudaErrorNotSupported) return e;
    }
    return launch_form<FMT, false, OUT>(f, num_sms, o);
}

template <int FMT>
cudaError_t launch_format(const ExpertFp4Args& f, int num_sms, const LaunchOpts& o)
{
    if (!f.glu) return launch_out<FMT, kOutPlain>(f, num_sms, o);
    return f.y_scales ? launch_out<FMT, kOutGluFp4>(f, num_sms, o)
                      : launch_out<FMT, kOutGluBf16>(f, num_sms, o);
}

}  // namespace

cudaError_t launch_expert_fp4(const ExpertFp4Args& f, int num_sms, const LaunchOpts& o)
{
    return f.format == kFp4Mx ? launch_format<kFp4Mx>(f, num_sms, o)
                              : launch_format<kFp4Nv>(f, num_sms, o);
}

}  // namespace ep
