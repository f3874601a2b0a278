// expert_tile.cuh - the persistent tcgen05 kernel whose output tiles are rows of
// one expert x columns: y = x * W_e^T (expert_gemm.cu), the gated projections and
// the data gradients (expert_ffn.cu) are instances of it. The tile list comes from
// the device counts; see expert_gemm.cu for the roles, tiles and schedule.
//
// MODE says what the columns are and what the epilogue does:
//   kPlain      B tile = BN rows of W_e [dout][din] (K-major), y = acc in bf16;
//   kGlu        B tile = blocks of 64 gate rows and 64 up rows in turn, so that the
//               accumulator of one tile holds g and u of the same BN / 2 columns
//               (64 columns apart, in the same lanes for full and M = 128 pair
//               tiles alike): h = act(g) * u leaves the registers, and g, u only
//               when the caller keeps them;
//   kDgrad      contraction over the forward's output columns: B tile = 64 lines of
//               W_e [k][n] with n contiguous (MN-major boxes, no transposed copy);
//   kDgradGlu   the same, and the epilogue turns grad h into grad g and grad u with
//               the saved pre-activations, so grad h never reaches memory.
#pragma once

#include "umma.cuh"

namespace ep {
namespace {

constexpr int kGemmThreads = 192;   // warp 0 TMA, warp 1 MMA + TMEM, warps 2-5 epilogue

enum TileMode { kPlain = 0, kGlu = 1, kDgrad = 2, kDgradGlu = 3 };

// Bytes after the ring: the epilogue warps' staging, barriers, TMEM address, abort
// flag, the two per-expert tile prefixes (heavy, light) and the per-expert row counts
// (all sized for the largest expert count).
template <int STAGES>
constexpr int tail_bytes()
{
    return 4 * kStageWarpBytes + 8 * (2 * STAGES + 5) + 8 + 8 * (kMaxExperts + 1) + 4 * kMaxExperts;
}

template <int BN_, int BK_, int STAGES_, bool PAIR_, int MODE_ = kPlain>
struct Cfg {
    static constexpr int BN = BN_, BK = BK_, STAGES = STAGES_;
    static constexpr bool PAIR = PAIR_;
    static constexpr int MODE = MODE_;
    static constexpr bool kBMn = MODE == kDgrad || MODE == kDgradGlu;   // B is MN-major
    static constexpr int kOutBN = MODE == kGlu ? BN / 2 : BN;           // output columns of a tile
    static constexpr int kTileRows = PAIR ? 2 * kBM : kBM;          // rows of one work unit
    static constexpr int kRowsB = PAIR ? BN / 2 : BN;               // W rows this CTA holds
    static constexpr uint32_t kBytesA = kBM * BK * 2;
    static constexpr uint32_t kBytesB = kRowsB * BK * 2;
    static constexpr uint32_t kStageBytes = kBytesA + kBytesB;      // per CTA
    // Instruction descriptor, kind::f16: fp32 accumulate (bits 4-5 = 1), A and
    // B bf16 (bits 7-9 = 1, 10-12 = 1), A K-major (bit 15 = 0), B K-major or
    // MN-major (bit 16), N >> 3 at bits 17-22, M >> 4 at bits 24-28 (M = 256
    // across a pair).
    static constexpr uint32_t kIdesc = (1u << 4) | (1u << 7) | (1u << 10) |
                                       ((kBMn ? 1u : 0u) << 16) |
                                       ((uint32_t)(BN >> 3) << 17) |
                                       ((uint32_t)(kTileRows >> 4) << 24);
    // Pairs: an expert's last rows, when at most 128 are left, run as M = 128
    // across the pair (64 rows per CTA; same N).
    static constexpr uint32_t kIdescHalf = (kIdesc & ~(0x1Fu << 24)) |
                                           ((uint32_t)((kTileRows / 2) >> 4) << 24);
    static constexpr uint32_t kBytesAHalf = kBytesA / 2;
    static constexpr uint32_t kTmemCols = 2 * BN;                   // two accumulators per CTA
    // Epilogue warps that release an accumulator (both CTAs for a pair).
    static constexpr uint32_t kReleaseCount = PAIR ? 8u : 4u;
    // One K slice of a row is one swizzle span: 128 bytes (BK = 64) or 64 (BK = 32).
    static constexpr uint32_t kSpan = BK * 2;
    static constexpr uint64_t kSwizzleMode = (BK == 64) ? 2 : 4;   // descriptor: 128B = 2, 64B = 4
    static constexpr uint32_t kSbo = 8 * kSpan;                     // bytes between 8-row groups
    static constexpr size_t kSmem = 1024 + (size_t)STAGES * kStageBytes + tail_bytes<STAGES>();
    static_assert(BK == 64 || BK == 32, "K slice is one 128- or 64-byte swizzle span");
    static_assert(!PAIR || BN == kPairBN, "pairs use 256-column tiles");
    static_assert(MODE == kPlain || (BK == 64 && kRowsB % 64 == 0), "B in boxes of 64 x 64");
    static_assert(MODE != kGlu || kRowsB % 128 == 0, "a CTA holds gate and up blocks in pairs");
    static_assert(kSmem <= (size_t)kSmemLimit, "ring does not fit in shared memory");
};

struct TileRef {
    int e;       // expert
    int mt;      // row tile (of kTileRows rows) within the expert
    int nb;      // column block
    bool half;   // pairs: the expert's last rows, at most kTileRows / 2 of them (M = 128)
};

// The schedule: uh heavy units then, interleaved with them in proportion,
// total - uh light ones. Within a class, unit v = (row tile of the class's
// prefix, column block), column blocks fastest.
struct Schedule {
    const int* heavy;   // [E + 1] prefix of the heavy experts' row tiles (light: 0)
    const int* light;   // [E + 1] prefix of the light experts' row tiles (heavy: 0)
    const int* cnt;     // [E] rows of each expert
    int uh, total;      // heavy units, all units
    int tile_rows;      // rows of a full row tile
    bool halves;        // pairs: last row tiles of at most tile_rows / 2 rows run as M = 128
};

// Unit u is the h-th heavy unit when floor((u + 1) uh / total) steps past
// h = floor(u uh / total), else the (u - h)-th light one: the heavy units
// before u are exactly floor(u uh / total), so every unit of both classes
// appears once.
__device__ __forceinline__ TileRef tile_of(const Schedule& q, int E, int nbk, int u)
{
    const int h = (int)(((int64_t)u * q.uh) / q.total);
    const bool heavy = (int)(((int64_t)(u + 1) * q.uh) / q.total) > h;
    const int* pre = heavy ? q.heavy : q.light;
    const int v = heavy ? h : u - h;
    TileRef p;
    const int mt = v / nbk;
    p.nb = v % nbk;
    p.e = expert_of(pre, E, mt);
    p.mt = mt - pre[p.e];
    p.half = q.halves && q.cnt[p.e] - p.mt * q.tile_rows <= q.tile_rows / 2;
    return p;
}

// This CTA's part of the B tile for K slice kc of expert e, column block nb.
template <class C>
__device__ __forceinline__ void load_b(uint32_t sb, const CUtensorMap* tm, const GemmArgs& a,
                                       int e, int nb, int r, int kc, uint32_t bar)
{
    auto load = [&](uint32_t dst, int c0, int c1) {
        if (C::PAIR) tma_load_2d_pair(dst, tm, c0, c1, bar);
        else tma_load_2d(dst, tm, c0, c1, bar);
    };
    if (C::MODE == kPlain) {
        load(sb, kc, e * (int)a.dout + nb * C::BN + r * C::kRowsB);
    } else if (C::MODE == kGlu) {
        // dout gate rows, then dout up rows, of each expert.
        const int row0 = e * 2 * (int)a.dout + nb * C::kOutBN + r * (C::kRowsB / 2);
#pragma unroll
        for (int j = 0; j < C::kRowsB / 64; ++j)
            load(sb + (uint32_t)j * (64 * C::kSpan), kc,
                 row0 + (j >> 1) * 64 + ((j & 1) ? (int)a.dout : 0));
    } else {
        const int n0 = nb * C::BN + r * C::kRowsB;
#pragma unroll
        for (int j = 0; j < C::kRowsB / 64; ++j)
            load(sb + (uint32_t)j * kMnBoxBytes, n0 + 64 * j, e * (int)a.din + kc);
    }
}

// B's descriptor for K step j (of 16) of a stage.
template <class C>
__device__ __forceinline__ uint64_t desc_b(uint32_t sb, int j)
{
    return C::kBMn ? smem_desc_mn(sb + (uint32_t)j * (kUmmaK * kMnLineBytes))
                   : smem_desc<C>(sb + (uint32_t)j * (kUmmaK * 2));
}

// tm_a: box of [128 rows][BK] over the receive rows; tm_a_half: [64 rows][BK]
// (pairs' M = 128 tiles); tm_b: box of [kRowsB rows][BK] over the weights
// (half a column block per CTA for pairs), or 64 x 64 boxes (load_b).
template <class C>
__global__ void __launch_bounds__(kGemmThreads, 1)
expert_gemm_kernel(const __grid_constant__ CUtensorMap tm_a,
                   const __grid_constant__ CUtensorMap tm_a_half,
                   const __grid_constant__ CUtensorMap tm_b, GemmArgs a)
{
    constexpr int STAGES = C::STAGES, BN = C::BN, BK = C::BK;
    constexpr bool PAIR = C::PAIR;
    extern __shared__ uint8_t smem_raw[];
    // Swizzled tiles want 1024-byte alignment; the offset is the same in both
    // CTAs of a pair (the MMA reads the peer's tiles, and copies and arrivals
    // reach the peer, at the same CTA-relative offsets).
    const uint32_t raw_u32 = smem_u32(smem_raw);
    uint8_t* smem = smem_raw + ((1024u - (raw_u32 & 1023u)) & 1023u);
    const uint32_t tiles_u32 = smem_u32(smem);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + STAGES * C::kStageBytes + 4 * kStageWarpBytes);
    const uint32_t full0 = smem_u32(bars);                 // STAGES (pairs: the leader's count)
    const uint32_t empty0 = full0 + 8u * STAGES;           // STAGES
    const uint32_t accum_full0 = empty0 + 8u * STAGES;     // 2: one per accumulator
    const uint32_t accum_empty0 = accum_full0 + 16u;       // 2 (pairs: the leader's count)
    const uint32_t drain = accum_empty0 + 16u;
    uint32_t* s_tmem = reinterpret_cast<uint32_t*>(bars + 2 * STAGES + 5);
    volatile int* s_abort = reinterpret_cast<volatile int*>(s_tmem + 1);
    int* s_heavy = const_cast<int*>(reinterpret_cast<volatile int*>(s_abort + 1));   // [E + 1]
    int* s_light = s_heavy + (kMaxExperts + 1);                                        // [E + 1]
    int* s_cnt = s_light + (kMaxExperts + 1);                                          // [E]
    const int E = a.E;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int r = PAIR ? cluster_rank() : 0;
    const bool leader = r == 0;
    const int first = PAIR ? cluster_index() : (int)blockIdx.x;
    const int step = PAIR ? cluster_count() : (int)gridDim.x;
    const int k_iters = (int)(a.din / BK);
    const int nbk = (int)(a.dout / C::kOutBN);
    // The barriers the MMA thread waits on live in the leader (rank 0).
    const uint32_t lead_full0 = PAIR ? map_to_rank(full0, 0) : full0;
    const uint32_t lead_accum_empty0 = PAIR ? map_to_rank(accum_empty0, 0) : accum_empty0;

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(full0 + 8u * s, 1u);
            mbar_init(empty0 + 8u * s, 1u);
        }
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

    griddep_wait();   // counts, offsets and the receive rows come from earlier kernels

    // Prefixes over experts of their row tiles (kTileRows rows each), one per
    // class: experts with at most light_rows rows are light.
    if (warp == 0) {
        int carry_h = 0, carry_l = 0;
        if (lane == 0) s_heavy[0] = s_light[0] = 0;
        for (int base = 0; base < E; base += 32) {
            const int e = base + lane;
            const int c = (e < E) ? __ldcg(a.cnt + e) : 0;
            if (e < E) s_cnt[e] = c;
            const int m = (c + C::kTileRows - 1) / C::kTileRows;
            const bool is_light = c <= a.light_rows;
            int mh = is_light ? 0 : m, ml = is_light ? m : 0;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int nh = __shfl_up_sync(0xffffffffu, mh, d);
                const int nl = __shfl_up_sync(0xffffffffu, ml, d);
                if (lane >= d) {
                    mh += nh;
                    ml += nl;
                }
            }
            if (e < E) {
                s_heavy[e + 1] = carry_h + mh;
                s_light[e + 1] = carry_l + ml;
            }
            carry_h += __shfl_sync(0xffffffffu, mh, 31);
            carry_l += __shfl_sync(0xffffffffu, ml, 31);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (PAIR) cluster_sync();   // the peer's barriers exist before any copy or arrival reaches them
    tc_fence_after();
    const uint32_t tmem = *s_tmem;
    Schedule q;
    q.heavy = s_heavy;
    q.light = s_light;
    q.cnt = s_cnt;
    q.tile_rows = C::kTileRows;
    q.halves = PAIR;
    q.uh = s_heavy[E] * nbk;
    q.total = q.uh + s_light[E] * nbk;
    const int total = q.total;

    // The copying and the issuing warp wait as a whole and elect a lane to issue: what
    // a lane issues with is then uniform (see elect_one).
    if (warp == 0) {
        // ---- TMA producer (each CTA fills its own ring) --------------------
        int g = 0;   // k-slices issued
        bool ok = true;
        for (int u = first; u < total && ok && !*s_abort; u += step) {
            const TileRef p = tile_of(q, E, nbk, u);
            const int row0 = __ldcg(a.expert_offset + p.e) + p.mt * C::kTileRows +
                             r * (p.half ? kBM / 2 : kBM);
            for (int k = 0; k < k_iters; ++k, ++g) {
                const int s = g % STAGES;
                const uint32_t ph = (uint32_t)((g / STAGES) & 1);
                ok = warp_all(wait_or_abort(empty0 + 8u * s, ph ^ 1u, s_abort));
                if (!ok) break;
                const uint32_t sa = tiles_u32 + (uint32_t)s * C::kStageBytes;
                const uint32_t sb = sa + C::kBytesA;
                const int kc = k * BK;
                if (elect_one()) {
                    if (!PAIR) {
                        const uint32_t fb = full0 + 8u * s;
                        mbar_expect_tx(fb, C::kStageBytes);
                        tma_load_2d(sa, &tm_a, kc, row0, fb);
                        load_b<C>(sb, &tm_b, a, p.e, p.nb, r, kc, fb);
                    } else {
                        // Both CTAs' copies complete on the leader's barrier, which
                        // expects the bytes of both (an M = 128 tile: 64 rows of x per CTA).
                        if (leader)
                            mbar_expect_tx(full0 + 8u * s,
                                           2u * (p.half ? C::kBytesAHalf + C::kBytesB : C::kStageBytes));
                        const uint32_t fb = lead_full0 + 8u * s;
                        tma_load_2d_pair(sa, p.half ? &tm_a_half : &tm_a, kc, row0, fb);
                        load_b<C>(sb, &tm_b, a, p.e, p.nb, r, kc, fb);
                    }
                }
                __syncwarp();
            }
        }
        // The copies this warp issued land before shared memory goes away
        // (a pair's copies are tracked by the leader's barrier: wait for the
        // MMAs to release the stages instead).
        const uint64_t deadline = globaltimer_ns() + kWaitLimitNs;
        for (int i = (g > STAGES ? g - STAGES : 0); i < g; ++i) {
            const uint32_t s = (uint32_t)(i % STAGES), par = (uint32_t)((i / STAGES) & 1);
            if (PAIR) mbar_wait_until(empty0 + 8u * s, par, deadline);
            else mbar_wait_until(full0 + 8u * s, par, deadline);
        }
    } else if (warp == 1 && leader) {
        // ---- MMA issuer (pairs: the leader's, for both SMs) ----------------
        int g = 0, tl = 0;
        bool issued = false, ok = true;
        for (int u = first; u < total && ok && !*s_abort; u += step, ++tl) {
            const int acc = tl & 1, use = tl >> 1;      // accumulator and its use count
            ok = warp_all(wait_or_abort(accum_empty0 + 8u * acc, (uint32_t)((use & 1) ^ 1), s_abort));
            if (!ok) break;
            tc_fence_after();
            const uint32_t d_tmem = tmem + (uint32_t)(acc * BN);
            const uint32_t idesc = tile_of(q, E, nbk, u).half ? C::kIdescHalf : C::kIdesc;
            for (int k = 0; k < k_iters; ++k, ++g) {
                const int s = g % STAGES;
                ok = warp_all(wait_or_abort(full0 + 8u * s, (uint32_t)((g / STAGES) & 1), s_abort));
                if (!ok) break;
                tc_fence_after();
                const uint32_t sa = tiles_u32 + (uint32_t)s * C::kStageBytes;
                if (elect_one()) {
#pragma unroll
                    for (int j = 0; j < BK / kUmmaK; ++j)
                        umma_bf16<PAIR>(d_tmem, smem_desc<C>(sa + j * kUmmaK * 2),
                                        desc_b<C>(sa + C::kBytesA, j), idesc,
                                        (k | j) != 0 ? 1u : 0u);
                    umma_commit<PAIR>(empty0 + 8u * s);   // frees the stage (in both CTAs of a pair)
                    if (k == k_iters - 1)
                        umma_commit<PAIR>(accum_full0 + 8u * acc);   // the accumulator is complete
                }
                __syncwarp();
                issued = true;
            }
        }
        if (issued) {   // every MMA this warp issued has finished before TMEM is freed
            if (elect_one()) umma_commit_local<PAIR>(drain);
            __syncwarp();
            mbar_wait(drain, 0u);
        }
    } else if (warp >= 2) {
        // ---- epilogue: TMEM -> bf16 -> global ------------------------------
        const int quarter = warp & 3;                  // TMEM lanes this warp may read
        const uint32_t t_lane = tmem + ((uint32_t)(quarter * 32) << 16);
        const uint32_t stage = tiles_u32 + STAGES * C::kStageBytes + (uint32_t)(quarter * kStageWarpBytes);
        uint16_t* y = static_cast<uint16_t*>(a.y);
        int tl = 0;
        for (int u = first; u < total && !*s_abort; u += step, ++tl) {
            const int acc = tl & 1, use = tl >> 1;
            const uint32_t t_acc = t_lane + (uint32_t)(acc * BN);
            const TileRef p = tile_of(q, E, nbk, u);
            // The rows this warp drains and the output columns they cover. A full
            // tile: lane quarter w holds this CTA's tile rows 32w..32w+31, every
            // column. A pair's M = 128 tile: the CTA's 64 rows appear twice, lanes
            // 0-63 with output columns [0, BN/2) and lanes 64-127 with
            // [BN/2, BN), both in accumulator columns [0, BN/2).
            const int sub0 = 32 * (p.half ? quarter & 1 : quarter);
            const int col0 = p.half ? (BN / 2) * (quarter >> 1) : 0;
            const int ncols = p.half ? BN / 2 : BN;
            const int part = p.half ? kBM / 2 : kBM;       // rows of this CTA's part
            const int m_in = p.mt * C::kTileRows + r * part;
            const int rows = min(part, q.cnt[p.e] - m_in) - sub0;   // of this warp's 32
            const int64_t row0 = (int64_t)__ldcg(a.expert_offset + p.e) + m_in + sub0;
            int4 next_g[4], next_u[4];
            if (C::MODE == kDgradGlu) {
                const uint16_t* gate_up =
                    static_cast<const uint16_t*>(a.aux) + row0 * 2 * a.dout + p.nb * BN + col0;
                warp_fetch_bf16x32(next_g, lane, gate_up, 2 * a.dout, rows);
                warp_fetch_bf16x32(next_u, lane, gate_up + a.dout, 2 * a.dout, rows);
            }
            if (!warp_all(wait_or_abort(accum_full0 + 8u * acc, (uint32_t)(use & 1), s_abort))) break;
            tc_fence_after();
            if (C::MODE == kPlain || C::MODE == kDgrad) {
                uint16_t* at = y + row0 * a.dout + p.nb * BN + col0;
#pragma unroll 1
                for (int c = 0; c < ncols; c += 32) {
                    uint32_t q32[32];
                    float v[32];
                    tmem_ld32(t_acc + (uint32_t)c, q32);
                    tmem_wait_ld();
                    as_floats(q32, v);
                    warp_store_bf16x32(stage, lane, v, at + c, a.dout, rows);
                }
            } else if (C::MODE == kGlu) {
                // Accumulator columns [128 b, 128 b + 64) are g and the next 64 u of
                // the tile's output columns [64 b, 64 b + 64).
                uint16_t* gate_up = static_cast<uint16_t*>(a.aux);
                const int64_t col = p.nb * C::kOutBN + col0 / 2;
#pragma unroll 1
                for (int c = 0; c < ncols / 2; c += 32) {
                    uint32_t qg[32], qu[32];
                    float g[32], u[32];
                    const uint32_t at = (uint32_t)((c >> 6) * 128 + (c & 63));
                    tmem_ld32(t_acc + at, qg);
                    tmem_ld32(t_acc + at + 64u, qu);
                    tmem_wait_ld();
                    as_floats(qg, g);
                    as_floats(qu, u);
                    if (gate_up) {
                        uint16_t* to = gate_up + row0 * 2 * a.dout + col + c;
                        warp_store_bf16x32(stage, lane, g, to, 2 * a.dout, rows);
                        warp_store_bf16x32(stage, lane, u, to + a.dout, 2 * a.dout, rows);
                    }
#pragma unroll
                    for (int i = 0; i < 32; ++i) u[i] *= act_value(g[i], a.act);
                    warp_store_bf16x32(stage, lane, u, y + row0 * a.dout + col + c, a.dout, rows);
                }
            } else {
                // The pre-activations of the next 32 columns are on their way meanwhile.
                const int64_t at = row0 * 2 * a.dout + p.nb * BN + col0;
                const uint16_t* gate_up = static_cast<const uint16_t*>(a.aux) + at;
#pragma unroll 1
                for (int c = 0; c < ncols; c += 32) {
                    uint32_t q32[32];
                    float gh[32], g[32], u[32];
                    tmem_ld32(t_acc + (uint32_t)c, q32);
                    warp_spread_bf16x32(stage, lane, next_g, g);
                    warp_spread_bf16x32(stage, lane, next_u, u);
                    if (c + 32 < ncols) {
                        warp_fetch_bf16x32(next_g, lane, gate_up + c + 32, 2 * a.dout, rows);
                        warp_fetch_bf16x32(next_u, lane, gate_up + a.dout + c + 32, 2 * a.dout, rows);
                    }
                    tmem_wait_ld();
                    as_floats(q32, gh);
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        float value, slope;
                        act_value_slope(g[i], a.act, &value, &slope);
                        g[i] = gh[i] * u[i] * slope;
                        u[i] = gh[i] * value;
                    }
                    warp_store_bf16x32(stage, lane, g, y + at + c, 2 * a.dout, rows);
                    warp_store_bf16x32(stage, lane, u, y + at + a.dout + c, 2 * a.dout, rows);
                }
            }
            // This warp's reads of the accumulator are done: one arrival per
            // warp on the leader's barrier.
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if (PAIR) mbar_arrive_cluster(lead_accum_empty0 + 8u * acc);
                else mbar_arrive(accum_empty0 + 8u * acc);
            }
        }
    }

    __syncwarp();
    if (threadIdx.x == 0 && *s_abort) atomicOr(a.err, kErrTimeout);
    tc_fence_before();
    __syncthreads();
    // Pairs: the leader's MMAs (which read the peer's shared memory and write
    // its TMEM) and its arrivals on the peer are done before either CTA frees
    // TMEM or exits.
    if (PAIR) cluster_sync();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc<PAIR>(tmem, C::kTmemCols);
    }
    griddep_launch_dependents();
}

// Ring depths: as many stages as fit next to the tail (at most 12); a stage
// holds 128 rows and the CTA's rows_b rows of W.
template <int ROWS_B, int BK>
constexpr int stages_for()
{
    const int fit = (kSmemLimit - 1024 - tail_bytes<12>()) / (int)((kBM + ROWS_B) * BK * 2);
    return fit > 12 ? 12 : fit;
}

template <int BN, int BK, bool PAIR, int MODE = kPlain>
using CfgOf = Cfg<BN, BK, stages_for<(PAIR ? BN / 2 : BN), BK>(), PAIR, MODE>;

template <class C>
cudaError_t launch_cfg(const GemmArgs& a, const void* x, int64_t rows, const void* w, int num_sms,
                       const LaunchOpts& o, int* grid_used)
{
    cudaError_t e = cudaFuncSetAttribute(expert_gemm_kernel<C>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::kSmem);
    if (e != cudaSuccess) return e;
    int grid = num_sms;
    if (C::PAIR) {
        grid = cluster_grid(expert_gemm_kernel<C>, kGemmThreads, C::kSmem, num_sms);
        if (grid < 2) return cudaErrorNotSupported;
    }
    CUtensorMap ta, ta_half, tb;
    // The weights as the tensor map sees them: lines of K (their columns n for
    // the data gradients), one after the other over all experts.
    const uint64_t wrows = (uint64_t)a.E * (uint64_t)(C::kBMn ? a.din : C::MODE == kGlu ? 2 * a.dout : a.dout);
    const uint64_t wline = (uint64_t)(C::kBMn ? a.dout : a.din);
    if (!make_map(&ta, x, (uint64_t)a.din, (uint64_t)rows, kBM, C::BK) ||
        !make_map(&ta_half, x, (uint64_t)a.din, (uint64_t)rows, kBM / 2, C::BK) ||
        !make_map(&tb, w, wline, wrows, C::MODE == kPlain ? C::kRowsB : 64, C::BK))
        return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(kGemmThreads);
    cfg.dynamicSmemBytes = C::kSmem;
    cfg.stream = o.stream;
    set_attrs(&cfg, attr, C::PAIR, o.pdl);
    e = cudaLaunchKernelEx(&cfg, expert_gemm_kernel<C>, ta, ta_half, tb, a);
    if (e == cudaSuccess && o.launches) ++*o.launches;
    *grid_used = grid;
    return e;
}

}  // namespace
}  // namespace ep
