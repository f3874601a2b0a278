// moe_layer.cu - a whole mixture-of-experts layer for a few tokens in two kernels:
//     h[t,k] = act(Wg_e x_t) * (Wu_e x_t),           e = ids[t][k]
//     out[t] = sum_k scores[t][k] * (Wd_e h[t,k])
// with bf16 or 4-bit weights (fp4.cuh). No dispatch, no receive rows, no combine: each CTA
// works the routing out by itself from the ids (at most kMaxPairs of them).
//
// With a few rows per expert the layer is the reading of the experts' weights, so the weights
// are the M side of the tensor cores' tiles (128 rows, streamed by TMA through a ring as deep
// as shared memory) and an expert's token rows, 16 at a time, the N side. Nothing touches the
// weights on their way: 4-bit codes go to the block-scaled instructions as they lie, which
// leaves the CUDA cores with the activations alone.
//
// With bf16 weights x enters as it is, and h, fp32, as the sum of three bf16 rows: its first 8 bits,
// the next 8 and the last, cut and not rounded, so that the three are h and none of them overflows.
// With 4-bit weights a row enters as eight rows of e2m1 digits that share a power of two s for each
// block of the weights' size:
//     x = s (d0 + d1 / 8 + d2 / 64 + ... + d7 / 8^7) + rest,   -4 <= d <= 3,   |rest| <= s / 2^22,
// s = 2^floor(log2 amax): x / s is rounded to an integer of 2^-21, whose octal digits, each 4 less,
// are all values of e2m1. A bf16 element down to 2^-14 of its block's largest is exact, every other
// one and h within 2^-22 of the largest, about what fp32 sums with the largest would leave, so
// that elements beside a dominant one keep their bits. (Four digits of x and five of h left 2^-11
// and 2^-14: beside an element 3 x 2^12 times their size the others were lost.) The digits are
// columns of one product, joined in the epilogue. Taken from an integer all at once they cost what
// four cost rounded one after the other; their rows in the ring leave it 5 stages of 7. Against the
// shorter digits: 1 token 47.4 for 46.3 us (nv, 8 of 256, 7168 wide), 16 tokens 417 for 410 (mx),
// 64 tokens over 8 experts 141 for 123 (4096 wide).
// nv scales (ue4m3) reach over 18 binades only: they count from the row's largest block, and
// blocks 2^17 below it are within 2^-39 of the row's largest. mx's scales are s / 8, and the
// sums 8 times that, so that s times a digit of 2 stays finite.
//
// Work: a unit is a chunk of up to 16 rows of an expert x a tile of 128 weight rows (64 gate
// and 64 up rows of the same columns in the first kernel). A cluster of 1, 2 or 4 CTAs shares
// a unit along K, so that few units still fill the SMs; their partial sums meet in shared
// memory, each CTA adding up a share of the rows in the order of the CTAs. In the second kernel
// every pair's result goes to a workspace in fp32, and the CTA that completes a tile's last unit
// adds the experts' results in the order of k. All sums have a fixed order.
//
// Sums, h, scores and the pairs' results are fp32; the layer's result is rounded once.
//
// Measured (D 7168, dff 2048, 8 of 256 experts; rate of the weights): 1 token 115 us in bf16 (6.1
// TB/s), 44 us mx (4.3), 48 us nv (4.1); 16 tokens 1277 us (7.0), 427 us mx (5.5) and 486 us nv (5.2);
// 64 tokens 2786 us (7.1), 986 us (5.3) and 1140 us (4.9). Bound by HBM from a few tokens on;
// 64 tokens over 8 experts, 4096 wide, by the work on the rows (141 us mx, 113 us in bf16). One
// token: about 5 us to the first product of each kernel (launch, routing, the first rows behind
// their latency), 2 us from one kernel to the other, and a quarter of a wave. Steps, with the
// shorter digits of before, for 16 tokens mx: 1275 us as it was first (joins by one CTA, each load
// waited for), 725 with joins in batches, 516 with a cluster's units next to one another, 447 with
// one copy of the digits' code, 430 with descriptors moved by additions, 410 with the weights first
// to leave L2. For one token nv: 74, 69, 66, 64; 62 with loads after the arrivals, 50 with the
// weights first to leave L2.
// Tried: warps that share a stage's rows (each waits for every slot), the row loop unrolled
// over four rows (its code comes from memory in every call), the scales of the weights fetched
// before the arrival of the stage at hand.
#include "ep_fp4.cuh"
#include "fp4_umma.cuh"

namespace ep {
namespace {

constexpr int kChunkRows = 16;                  // token rows of a unit
constexpr int kDigits = 8;                      // of x and of h (4-bit weights)
constexpr int kAccCols = kChunkRows * kDigits;  // columns set aside for an accumulator
constexpr int kEpiWarps = 4, kScaleWarps = 4;
constexpr int kEpiWarp0 = 2, kScaleWarp0 = 6, kRowWarp0 = 10;
constexpr uint32_t kLayerTmem = 512;            // a CTA has its SM for itself (shared memory)
constexpr int kMaxSplit = 4;
// Of a CTA's weights in the second kernel, fetched to L2 by the first: 1 token of bf16 (2 x 4096 x
// 2048 x 2 experts) 30.0 us without, 28.8 with 96 KB, 28.4 with 192, 28.1 with 512; 1 token nv
// (8 x 7168) 46.3, 46.3, 47.6 and 50.2, where more of them is in memory's way. Those two sizes are
// all that was measured: the least amount that helped one and did not hurt the other.
constexpr int kNextBytes = 96 * 1024;
constexpr int kFmtBf16 = 2;                     // beside kFp4Mx, kFp4Nv

template <int FMT_, bool DOWN_>
struct LayerCfg {
    static constexpr int FMT = FMT_;
    static constexpr bool DOWN = DOWN_, FP4 = FMT_ != kFmtBf16;
    static constexpr int kStageK = FP4 ? kFp4StageK : 64;       // 128 bytes of a row
    // Rows of the N side that a token row becomes: digits, or h's three bf16 terms.
    static constexpr int kTerms = FP4 ? kDigits : DOWN ? 3 : 1;
    static constexpr int kCols = kChunkRows * kTerms;
    static constexpr int kTiles = FP4 ? Fp4Mma<FP4 ? FMT_ : kFp4Mx>::kTiles : 0;
    static constexpr uint32_t kBytesA = kBM * 128, kBytesB = kCols * 128;
    static constexpr uint32_t kScales = kTiles * kScaleTile;    // of A and of B, each
    static constexpr uint32_t kStageBytes = kBytesA + kBytesB + 2 * kScales;
    static constexpr uint32_t kExchange = 2 * kChunkRows * 128 * 4;
    static constexpr uint32_t kTables = 4 * kMaxExperts + (8 + 2 + 2 + 4 + 1) * kLayerMaxPairs;
    static constexpr uint32_t kFixed = 1024 + kExchange + kTables + 512;
    static constexpr int kFit = (int)((kSmemLimit - kFixed) / kStageBytes);
    static constexpr int STAGES = kFit > 12 ? 12 : kFit;
    static constexpr size_t kSmem = kFixed + (size_t)STAGES * kStageBytes;
    static constexpr uint32_t kScaleCol0 = 2 * kAccCols;               // after two accumulators
    static constexpr int kRowWarps = FP4 ? 5 : 6;                      // at most STAGES (below)
    static constexpr int kThreads = 32 * (kRowWarp0 + kRowWarps);
    // Arrivals that fill a stage: the copy of A, the warp that brings its scales, that of the rows.
    static constexpr uint32_t kFullCount = FP4 ? 3u : 2u;
    // A warp that serves every n-th stage waits for a slot's last release by parity: it must not
    // get there while the release before that one is out, which its own last stage rules out as
    // long as that is at most a ring's length ago.
    static_assert(kRowWarps <= STAGES && kScaleWarps <= STAGES, "a warp's stages within the ring");
    static_assert(kScaleCol0 + 2 * 2 * 16 <= kLayerTmem && kCols <= kAccCols && kCols <= 128,
                  "accumulators and scales");
};

struct LayerKernelArgs {
    const int32_t* ids;
    const float* scores;
    const void* rows;              // x [T][din] bf16, or h [pairs][din] fp32
    const uint8_t* w_scales;
    const float* w_scale;          // [E] or null
    float* h;                      // first kernel: [pairs][dff]
    uint32_t* h_most;              // [pairs][dff / 32]: the largest |h| (bits) of 32 columns (nv)
    float* y;                      // second kernel: [pairs][D]
    uint32_t* done;                // [D / 32] CTAs that have added their part of a unit to these columns
    int counters;                  // D / 32
    void* out;                     // [T][D]
    int T, K, E;
    int din, wrows;                // contraction; W's rows of an expert
    int tiles;                     // tiles of an expert
    int act;
    bool out_f32;
    uint32_t* err;
    // First kernel: the second one's tiles, stages and clusters, and the stages of each of its CTAs
    // that are fetched to L2 (0: none).
    int next_tiles, next_stages, next_split, next_clusters, next_fetched;
    const uint8_t* next_scales;
};

struct Chunk {
    uint16_t e, start, rows, pad;
};

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&v)[16])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]),
          "=r"(v[7]), "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]),
          "=r"(v[14]), "=r"(v[15])
        : "r"(taddr));
}

// Weights are read once in a call: first to leave L2, so that x, h, the pairs' results and the
// kernels' own code stay (each of which some warp waits for at the start of a kernel).
__device__ __forceinline__ uint64_t evict_first()
{
    uint64_t p;
    asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
    return p;
}

__device__ __forceinline__ void tma_load_2d_once(uint32_t dst, const CUtensorMap* tm, int c0, int c1,
                                                 uint32_t bar, uint64_t policy)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint "
        "[%0], [%1, {%2, %3}], [%4], %5;" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(tm)), "r"(c0), "r"(c1), "r"(bar), "l"(policy)
        : "memory");
}

__device__ __forceinline__ void tma_prefetch_2d(const CUtensorMap* tm, int c0, int c1)
{
    asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];" ::"l"(
                     reinterpret_cast<uint64_t>(tm)),
                 "r"(c0), "r"(c1)
                 : "memory");
}

__device__ __forceinline__ void st_cluster_f32(uint32_t addr, float v)
{
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}

__device__ __forceinline__ int cluster_size()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return (int)r;
}

__device__ __forceinline__ void store_out(const LayerKernelArgs& a, int64_t at, float v)
{
    if (a.out_f32) static_cast<float*>(a.out)[at] = v;
    else static_cast<uint16_t*>(a.out)[at] = (uint16_t)pack_bf16x2_rn(v, 0.0f);
}

__device__ __forceinline__ float ld_cg_f32(const float* p)
{
    float v;
    asm volatile("ld.global.cg.f32 %0, [%1];" : "=f"(v) : "l"(p));
    return v;
}

// out[t][col] of every token: the pairs' results in the order of k, as in combine. A lane has
// a column; the results of 32 pairs are on their way at a time (loaded whether or not a pair has
// an expert: a branch at each would have each waited for, 1000 cycles a pair), their scores in
// the lanes and the tokens' last pairs in a mask. What this takes, the CTA's next unit waits for.
__device__ __forceinline__ void join_experts(const LayerKernelArgs& a, int lane, int col0,
                                             const float* s_score, const uint8_t* s_ok)
{
    const int pairs = a.T * a.K;
    const float* y = a.y + col0 + lane;
    float r = 0.0f;
    int64_t at = col0 + lane;
    for (int i0 = 0; i0 < pairs; i0 += 32) {
        float v[32];
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] = ld_cg_f32(y + (int64_t)min(i0 + j, pairs - 1) * a.wrows);
        const int i = i0 + lane;
        const float score = i < pairs ? s_score[i] : 0.0f;
        const unsigned ok = __ballot_sync(~0u, i < pairs && s_ok[i]);
        const unsigned ends = __ballot_sync(~0u, i < pairs && (i + 1) % a.K == 0);
#pragma unroll
        for (int j = 0; j < 32; ++j) {
            const float s = __shfl_sync(~0u, score, j);
            if (ok >> j & 1u) r = fmaf(s, v[j], r);
            if (ends >> j & 1u) {
                store_out(a, at, r);
                r = 0.0f;
                at += a.wrows;
            }
        }
    }
}

// 2^e for -126 <= e <= 127.
__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// Exponent of s of a block (or row) whose largest magnitude has these bits: -126 .. 127, 128 if
// it is infinite or NaN.
__device__ __forceinline__ int digit_exponent(uint32_t most) { return max((int)(most >> 23), 1) - 127; }

// The ue4m3 code of 2^k, -9 <= k <= 8.
__device__ __forceinline__ uint32_t ue4m3_pow2(int k)
{
    return k >= -6 ? (uint32_t)(k + 7) << 3 : 1u << (k + 9);
}

// 8 elements of a row: 16 bytes of bf16, or 32 of fp32 (h).
template <bool F32>
struct Eight {
    int4 q[F32 ? 2 : 1];

    __device__ __forceinline__ void load(const void* rows, int64_t at, bool in)
    {
        const uint8_t* p = static_cast<const uint8_t*>(rows) + at * (F32 ? 4 : 2);
#pragma unroll
        for (int i = 0; i < (F32 ? 2 : 1); ++i) q[i] = in ? ld_cg_v4(p + 16 * i) : make_int4(0, 0, 0, 0);
    }

    __device__ __forceinline__ void floats(float (&v)[8]) const
    {
#pragma unroll
        for (int i = 0; i < (F32 ? 2 : 1); ++i) {
            const uint32_t w[4] = {(uint32_t)q[i].x, (uint32_t)q[i].y, (uint32_t)q[i].z, (uint32_t)q[i].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (F32) {
                    v[4 * i + j] = __uint_as_float(w[j]);
                } else {
                    v[2 * j] = __uint_as_float(w[j] << 16);
                    v[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
                }
            }
        }
    }
};

__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t select)
{
    uint32_t r;
    asm("prmt.b32 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(select));
    return r;
}

// An element's digits as e2m1, one to a byte: those of 8^0 .. 8^3 in lo, of 8^4 .. 8^7 in hi, of
// the integer n nearest to v f0 f1, |n| <= 2^22.
__device__ __forceinline__ void digits_of(float v, float f0, float f1, uint32_t& lo, uint32_t& hi)
{
    // 1.5 * 2^23 and n add up to the float whose bits are those of 1.5 * 2^23 and n. With 4 in
    // each of eight octal places added, n's balanced digits -4 .. 3 stand there as 0 .. 7.
    constexpr uint32_t kFours = 044444444u;
    uint32_t u = __float_as_uint(__fmaf_rn(v * f0, f1, 12582912.0f)) - __float_as_uint(12582912.0f) + kFours;
    // Octal digits to nibbles, then each to its code: bytes 0 .. 7 of a table.
    u = (u & 0x00000FFFu) | ((u << 4) & 0x0FFF0000u);
    u = (u & 0x003F003Fu) | ((u << 2) & 0x3F003F00u);
    u = (u & 0x07070707u) | ((u << 1) & 0x70707070u);
    constexpr uint32_t kBelowZero = 0x0A0C0D0Eu, kFromZero = 0x05040200u;   // -4 -3 -2 -1, 0 1 2 3
    lo = prmt(kBelowZero, kFromZero, u);
    hi = prmt(kBelowZero, kFromZero, u >> 16);
}

// 256 elements of a row, 8 in each lane, into the kDigits digit rows from n0 (a multiple of 8) on
// of a stage's B tile and the words of their scales. One copy of the code, called (the operands of
// h's fp32 in q1 too).
template <int FMT, bool H>
__device__ __noinline__ void store_digits(uint32_t sb, uint32_t sscale, int n0, int lane, int row_exp,
                                          int x0, int y0, int z0, int w0, int x1, int y1, int z1, int w1)
{
    static_assert(kDigits == 8, "a B tile's rows of 128 bytes repeat their swizzle every eight");
    Eight<H> raw;
    raw.q[0] = make_int4(x0, y0, z0, w0);
    if (H) raw.q[H ? 1 : 0] = make_int4(x1, y1, z1, w1);
    float v[8];
    raw.floats(v);
    uint32_t most = 0u;
#pragma unroll
    for (int i = 0; i < 8; ++i) most = max(most, __float_as_uint(v[i]) & 0x7FFFFFFFu);
    most = max(most, __shfl_xor_sync(~0u, most, 1));
    if (FMT == kFp4Mx) most = max(most, __shfl_xor_sync(~0u, most, 2));
    int e = digit_exponent(most);
    uint32_t code;
    if (FMT == kFp4Mx) {
        e = max(e, -124);
        code = (uint32_t)(e - 3 + 127);
    } else {
        const int k = max(e - row_exp + 8, -9);
        code = ue4m3_pow2(min(k, 8));
        e = row_exp - 8 + k;
    }
    // An infinity or a NaN: so is the row's result, whatever the digits.
    if (most >= 0x7F800000u) code = FMT == kFp4Mx ? kNanMx : kNanNv;
    // 2^(21 - e) in two factors: -107 .. 164.
    const int to = 21 - e;
    const float f0 = pow2(to >> 1), f1 = pow2(to - (to >> 1));
    // Bytes of two elements' digits, turned into words of eight elements' digits of one place.
    uint32_t p[2][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t lo0, hi0, lo1, hi1;
        digits_of(v[2 * i], f0, f1, lo0, hi0);
        digits_of(v[2 * i + 1], f0, f1, lo1, hi1);
        p[0][i] = lo0 | lo1 << 4;
        p[1][i] = hi0 | hi1 << 4;
    }
    const uint32_t to_row = sb + (uint32_t)(n0 * 128 + (lane & 3) * 4);
    const int unit = lane >> 2;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint32_t a = prmt(p[h][0], p[h][1], 0x5140u), b = prmt(p[h][2], p[h][3], 0x5140u);
        const uint32_t c = prmt(p[h][0], p[h][1], 0x7362u), d = prmt(p[h][2], p[h][3], 0x7362u);
        const uint32_t place[4] = {prmt(a, b, 0x5410u), prmt(a, b, 0x7632u), prmt(c, d, 0x5410u),
                                   prmt(c, d, 0x7632u)};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int n = 7 - (4 * h + j);      // the highest place in the first row
            sts32(to_row + (uint32_t)(n * 128 + ((unit ^ n) << 4)), place[j]);
        }
    }
    // The word of four blocks' scales, the same for each of the digits: a lane to a digit.
    constexpr int kLanes = FMT == kFp4Mx ? 4 : 2;      // of a block
    uint32_t word = code << (8 * (lane / kLanes & 3));
    word |= __shfl_xor_sync(~0u, word, kLanes);
    word |= __shfl_xor_sync(~0u, word, 2 * kLanes);
    const int n = n0 + lane % (4 * kLanes);
    if (lane % (4 * kLanes) < kDigits)
        sts32(sscale + (uint32_t)(lane / (4 * kLanes) * kScaleTile + (n & 31) * 16 + (n >> 5) * 4), word);
}

// The first 8 bits of two numbers, as bf16, and what is left of them (nothing of an infinity or a
// NaN, which these bits hold).
__device__ __forceinline__ uint32_t cut_bf16x2(float& a, float& b)
{
    const uint32_t h = prmt(__float_as_uint(a), __float_as_uint(b), 0x7632u);
    auto left = [](float v, uint32_t cut) {
        return (cut & 0x7F800000u) == 0x7F800000u ? 0.0f : v - __uint_as_float(cut);
    };
    a = left(a, h << 16);
    b = left(b, h & 0xFFFF0000u);
    return h;
}

// The weights that this CTA's successor in the second kernel reads first, to L2, while this kernel
// ends and that one works its routing out: HBM would have nothing to do.
template <class C>
__device__ __forceinline__ void fetch_next(const CUtensorMap& tm, const LayerKernelArgs& a,
                                           const Chunk* s_chunk, int chunks, int lane)
{
    const int cluster = (int)blockIdx.x / a.next_split, rank = (int)blockIdx.x % a.next_split;
    if (cluster >= a.next_clusters) return;
    const int64_t units = (int64_t)chunks * a.next_tiles;
    const int u_first = (int)(units * cluster / a.next_clusters);
    const int u_last = (int)(units * (cluster + 1) / a.next_clusters);
    const int k_first = rank * a.next_stages / a.next_split, k_last = (rank + 1) * a.next_stages / a.next_split;
    int left = a.next_fetched;
    for (int u = u_first; u < u_last; ++u) {
        const int tile = u / chunks;
        const int w0 = (s_chunk[u - tile * chunks].e * a.next_tiles + tile) * 128;
        for (int k = k_first; k < k_last; ++k) {
            if (--left < 0) return;
            if (elect_one()) {
                const int kc = k * (C::FP4 ? kFp4StageK / 2 : C::kStageK);
                tma_prefetch_2d(&tm, kc, w0);
                tma_prefetch_2d(&tm, kc, w0 + 64);
            }
            __syncwarp();
            if constexpr (C::FP4) {
                const int64_t tiles = a.wrows / 2 / (4 * Fp4<C::FMT>::kBlock), kt = (int64_t)k * C::kTiles;
                if (lane < 4 * C::kTiles && kt + lane / 4 < tiles)
                    asm volatile("prefetch.global.L2 [%0];" ::"l"(a.next_scales + fp4_scale_at(w0, kt, tiles) +
                                                                  lane * 128));
            }
        }
    }
}

template <class C>
__global__ void __launch_bounds__(C::kThreads, 1)
moe_layer_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_next,
                 const LayerKernelArgs a)
{
    constexpr int STAGES = C::STAGES, FMT = C::FMT, kRowWarps = C::kRowWarps;
    constexpr bool DOWN = C::DOWN;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_u32 = smem_u32(smem_raw);
    uint8_t* smem = smem_raw + ((1024u - (raw_u32 & 1023u)) & 1023u);
    const uint32_t ring = smem_u32(smem);
    const uint32_t ring_b = ring + STAGES * C::kBytesA;
    const uint32_t ring_s = ring_b + STAGES * C::kBytesB;
    float* s_x = reinterpret_cast<float*>(smem + STAGES * C::kStageBytes);     // [2][16][128]
    int* s_cnt = reinterpret_cast<int*>(s_x + 2 * kChunkRows * 128);           // [E]: rows, then first row
    Chunk* s_chunk = reinterpret_cast<Chunk*>(s_cnt + kMaxExperts);            // [pairs]
    uint16_t* s_list = reinterpret_cast<uint16_t*>(s_chunk + kLayerMaxPairs);  // pairs by expert
    int16_t* s_exp = reinterpret_cast<int16_t*>(s_list + kLayerMaxPairs);      // nv: exponents of the rows
    float* s_score = reinterpret_cast<float*>(s_exp + kLayerMaxPairs);         // the pairs' scores,
    uint8_t* s_ok = reinterpret_cast<uint8_t*>(s_score + kLayerMaxPairs);      // and whether they have an expert
    uint64_t* bars = reinterpret_cast<uint64_t*>(s_ok + kLayerMaxPairs);
    const uint32_t full0 = smem_u32(bars), empty0 = full0 + 8u * STAGES;
    const uint32_t accum_full0 = empty0 + 8u * STAGES, accum_free0 = accum_full0 + 16u;
    const uint32_t x_full0 = accum_free0 + 16u, x_free0 = x_full0 + 16u;
    const uint32_t drain = x_free0 + 16u;
    uint32_t* s_tmem = reinterpret_cast<uint32_t*>(bars + 2 * STAGES + 9);
    volatile int* s_abort = reinterpret_cast<volatile int*>(s_tmem + 1);
    int* s_chunks = const_cast<int*>(reinterpret_cast<volatile int*>(s_abort + 1));

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int split = cluster_size(), rank = cluster_rank();
    const int pairs = a.T * a.K;
    const int all_stages = (a.din + C::kStageK - 1) / C::kStageK;
    const int k_first = rank * all_stages / split, k_last = (rank + 1) * all_stages / split;

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(full0 + 8u * s, C::kFullCount);
            mbar_init(empty0 + 8u * s, 1u);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(accum_full0 + 8u * b, 1u);
            mbar_init(accum_free0 + 8u * b, kEpiWarps);
            mbar_init(x_full0 + 8u * b, kEpiWarps * split);
            mbar_init(x_free0 + 8u * b, kEpiWarps * split);
        }
        mbar_init(drain, 1u);
        *s_abort = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc<false>(smem_u32(s_tmem), kLayerTmem);
        tmem_relinquish<false>();
    }
    // The second kernel may start while the first one ends: by then the kernels before the
    // first one are complete, and with them the ids, the scores and the weights. What the first
    // one writes (h, its maxima, the counters) is waited for where it is used.
    if (!DOWN) {
        griddep_wait();
        griddep_launch_dependents();
    }

    if (warp >= kRowWarp0) {
        // The code that takes a row apart, and x, from memory, while the other warps work the
        // routing out: what follows them there waits for a row first, and a call's weights have
        // swept both out of L2. (These bytes of the ring's first slots are written again.)
        const int w = warp - kRowWarp0;
        if constexpr (C::FP4) {
            store_digits<FMT, DOWN>(ring_b + (uint32_t)w * C::kBytesB,
                                    ring_s + (uint32_t)w * (2 * C::kScales) + C::kScales, 0, lane, 0, 0,
                                    0, 0, 0, 0, 0, 0, 0);
        }
        if constexpr (FMT == kFp4Nv && !DOWN) {
            // The rows' largest magnitudes over this CTA's part of K.
            const int c0 = k_first * C::kStageK, c1 = min(k_last * C::kStageK, a.din);
            for (int t = w; t < a.T; t += kRowWarps) {
                uint32_t m = 0u;
                for (int i0 = c0; i0 < c1; i0 += 16 * 256) {   // sixteen loads on their way
                    int4 v[16];
#pragma unroll
                    for (int n = 0; n < 16; ++n) {
                        const int i = i0 + n * 256 + lane * 8;
                        v[n] = make_int4(0, 0, 0, 0);
                        if (i < c1)
                            v[n] = ld_cg_v4(static_cast<const uint16_t*>(a.rows) + (int64_t)t * a.din + i);
                    }
#pragma unroll
                    for (int n = 0; n < 16; ++n) m = max(m, __float_as_uint(amax8(v[n])));
                }
                m = __reduce_max_sync(~0u, m);
                if (lane == 0) s_exp[t] = (int16_t)digit_exponent(m);
            }
        } else if (!DOWN) {
            const int64_t bytes = (int64_t)a.T * a.din * 2;
            for (int64_t i = ((int64_t)blockIdx.x * kRowWarps * 32 + w * 32 + lane) * 128; i < bytes;
                 i += (int64_t)gridDim.x * kRowWarps * 32 * 128)
                asm volatile("prefetch.global.L2 [%0];" ::"l"(static_cast<const uint8_t*>(a.rows) + i));
        }
    } else if (pairs <= 32) {
        // ---- routing: the pairs by expert, in chunks; few of them in one warp ---------
        if (warp == 0) {
            const int raw = lane < pairs ? __ldcg(a.ids + lane) : -1;
            const int e = valid_id(raw, a.E);
            const float score = DOWN && lane < pairs ? __ldcg(a.scores + lane) : 0.0f;
            if (!DOWN && e != raw && blockIdx.x == 0) atomicOr(a.err, kErrBadId);
            const unsigned same = __match_any_sync(~0u, e);
            // An expert's first pair counts its rows and chunks.
            const bool leads = e >= 0 && lane == __ffs(same) - 1;
            const int count = leads ? __popc(same) : 0;
            const int packed = count | ((count + kChunkRows - 1) / kChunkRows) << 16;
            int v = packed;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int n = __shfl_up_sync(~0u, v, d);
                if (lane >= d) v += n;
            }
            const int row = (v - packed) & 0xFFFF, chunk = (v - packed) >> 16;
            for (int n = 0; n * kChunkRows < count; ++n)
                s_chunk[chunk + n] = {(uint16_t)e, (uint16_t)(row + n * kChunkRows),
                                      (uint16_t)min(count - n * kChunkRows, kChunkRows), 0};
            const int first_row = __shfl_sync(~0u, row, __ffs(same) - 1);
            if (e >= 0) s_list[first_row + __popc(same & lanemask_lt(lane))] = (uint16_t)lane;
            if (lane < pairs) {
                s_ok[lane] = e >= 0;
                if (DOWN) s_score[lane] = score;
            }
            if (lane == 31) *s_chunks = v >> 16;
        }
    } else {
        // ---- routing: the pairs by expert, in chunks --------------------------------
        constexpr int kWarps = kRowWarp0;
        auto barrier = [] { asm volatile("bar.sync 1, %0;" ::"n"(32 * kWarps) : "memory"); };
        // Pairs [32 i, 32 i + 32) are warp i's, from kWarps on once more the first ones'. The rank
        // of a pair among its expert's follows the order of the pairs, so that every CTA has the
        // same rows in the same chunks: warp after warp.
        constexpr int kRounds = (kLayerMaxPairs + 32 * kWarps - 1) / (32 * kWarps);
        int mine[kRounds], my_rank[kRounds];
#pragma unroll
        for (int n = 0; n < kRounds; ++n) {
            const int i = n * 32 * kWarps + (int)threadIdx.x;
            mine[n] = -1;
            if (i < pairs) {
                const int raw = __ldcg(a.ids + i);
                mine[n] = valid_id(raw, a.E);
                if (!DOWN && mine[n] != raw && blockIdx.x == 0) atomicOr(a.err, kErrBadId);
                s_ok[i] = mine[n] >= 0;
                if (DOWN) s_score[i] = __ldcg(a.scores + i);
            }
        }
        for (int e = threadIdx.x; e < a.E; e += 32 * kWarps) s_cnt[e] = 0;
        barrier();
#pragma unroll
        for (int n = 0; n < kRounds; ++n) {
            for (int w = 0; w < kWarps && 32 * (n * kWarps + w) < pairs; ++w) {
                if (warp == w) {
                    const unsigned same = __match_any_sync(~0u, mine[n]);
                    if (mine[n] >= 0) my_rank[n] = s_cnt[mine[n]] + __popc(same & lanemask_lt(lane));
                    __syncwarp();
                    if (mine[n] >= 0 && lane == __ffs(same) - 1) s_cnt[mine[n]] += __popc(same);
                }
                barrier();
            }
        }
        if (warp == 0) {
            int rows0 = 0, chunks0 = 0;
            for (int base = 0; base < a.E; base += 32) {
                const int e = base + lane;
                const int c = e < a.E ? s_cnt[e] : 0;
                const int packed = c | ((c + kChunkRows - 1) / kChunkRows) << 16;
                int v = packed;
#pragma unroll
                for (int d = 1; d < 32; d <<= 1) {
                    const int n = __shfl_up_sync(~0u, v, d);
                    if (lane >= d) v += n;
                }
                const int row = rows0 + ((v - packed) & 0xFFFF);
                int chunk = chunks0 + ((v - packed) >> 16);
                if (e < a.E) s_cnt[e] = row;
                for (int at = 0; at < c; at += kChunkRows, ++chunk)
                    s_chunk[chunk] = {(uint16_t)e, (uint16_t)(row + at), (uint16_t)min(c - at, kChunkRows), 0};
                const int all = __shfl_sync(~0u, v, 31);
                rows0 += all & 0xFFFF;
                chunks0 += all >> 16;
            }
            if (lane == 0) *s_chunks = chunks0;
        }
        barrier();
#pragma unroll
        for (int n = 0; n < kRounds; ++n)
            if (mine[n] >= 0)
                s_list[s_cnt[mine[n]] + my_rank[n]] = (uint16_t)(n * 32 * kWarps + (int)threadIdx.x);
    }
    tc_fence_before();
    __syncthreads();
    if (split > 1) cluster_sync();   // the peers' barriers exist before anything reaches them
    tc_fence_after();
    const uint32_t tmem = *s_tmem;

    // This cluster's units, one after the other in the list of the tiles' chunks: a tile's chunks
    // are then a few clusters' work, and joining its experts' results no cluster's habit.
    const int chunks = *s_chunks, units = chunks * a.tiles;
    const int u_first = (int)((int64_t)units * cluster_index() / cluster_count());
    const int u_last = (int)((int64_t)units * (cluster_index() + 1) / cluster_count());
    const int64_t thread0 = (int64_t)blockIdx.x * C::kThreads + threadIdx.x;
    const int64_t threads = (int64_t)gridDim.x * C::kThreads;
    if (!DOWN) {
        for (int64_t i = thread0; i < a.counters; i += threads) a.done[i] = 0u;
    } else if (chunks == 0) {   // no token has an expert
        griddep_wait();
        for (int64_t i = thread0; i < (int64_t)a.T * a.wrows; i += threads) store_out(a, i, 0.0f);
    }
    if (warp == 0) {
        // ---- weights ------------------------------------------------------------
        // The first rows are asked for first: behind a ring's worth of weights on every SM they
        // would come after it. (In the second kernel the weights are there long before the rows.)
        if (!DOWN) asm volatile("bar.sync 3, %0;" ::"n"(32 * (1 + kRowWarps)) : "memory");
        const uint64_t policy = evict_first();
        int g = 0;
        bool ok = true;
        for (int u = u_first; u < u_last && ok && !*s_abort; ++u) {
            const int tile = u / chunks;
            const int w0 = s_chunk[u - tile * chunks].e * a.wrows + tile * (DOWN ? 128 : 64);
            const int w1 = w0 + (DOWN ? 64 : a.wrows / 2);
            for (int k = k_first; k < k_last; ++k, ++g) {
                const int s = g % STAGES;
                ok = warp_all(wait_or_abort(empty0 + 8u * s, (uint32_t)(((g / STAGES) & 1) ^ 1), s_abort));
                if (!ok) break;
                if (elect_one()) {
                    const uint32_t fb = full0 + 8u * s, sa = ring + (uint32_t)s * C::kBytesA;
                    const int kc = k * (C::FP4 ? kFp4StageK / 2 : C::kStageK);
                    mbar_expect_tx(fb, C::kBytesA);
                    tma_load_2d_once(sa, &tm_w, kc, w0, fb, policy);
                    tma_load_2d_once(sa + C::kBytesA / 2, &tm_w, kc, w1, fb, policy);
                }
                __syncwarp();
            }
        }
        if constexpr (!DOWN)
            if (ok) fetch_next<C>(tm_next, a, s_chunk, chunks, lane);
        // The copies this warp issued land before shared memory goes away.
        const uint64_t deadline = globaltimer_ns() + kWaitLimitNs;
        for (int i = (g > STAGES ? g - STAGES : 0); i < g; ++i)
            mbar_wait_until(empty0 + 8u * (i % STAGES), (uint32_t)((i / STAGES) & 1), deadline);
    } else if (warp == 1) {
        // ---- products -------------------------------------------------------------
        const uint32_t a0 = desc_lo(ring), b0 = desc_lo(ring_b), scale0 = desc_lo(ring_s);
        uint32_t da = a0, db = b0, ds = scale0, ts = 0u, phase = 0u;   // the slot's
        int s = 0, tl = 0;
        bool issued = false, ok = true;
        for (int u = u_first; u < u_last && ok && !*s_abort && k_last > k_first; ++u, ++tl) {
            const int acc = tl & 1;
            ok = warp_all(wait_or_abort(accum_free0 + 8u * acc, (uint32_t)(((tl >> 1) & 1) ^ 1), s_abort));
            if (!ok) break;
            tc_fence_after();
            const uint32_t d_tmem = tmem + (uint32_t)(acc * kAccCols);
            const int rows = s_chunk[u % chunks].rows;
            const int n = (rows * C::kTerms + 15) / 16 * 16;
            const uint32_t idesc = C::FP4 ? Fp4Mma<C::FP4 ? FMT : kFp4Mx>::idesc(kBM, n)
                                          : (1u << 4) | (1u << 7) | (1u << 10) |
                                                ((uint32_t)(n >> 3) << 17) | ((uint32_t)(kBM >> 4) << 24);
            for (int k = k_first; k < k_last; ++k) {
                ok = warp_all(wait_or_abort(full0 + 8u * s, phase, s_abort));
                if (!ok) break;
                tc_fence_after();
                if (elect_one()) {
                    if constexpr (C::FP4) {
                        const uint32_t ta = tmem + C::kScaleCol0 + ts, tb = ta + 16u;
#pragma unroll
                        for (int j = 0; j < C::kTiles; ++j) {
                            tmem_copy_scales<false>(ta + 4u * j,
                                                    desc_of(ds + j * (kScaleTile >> 4), kScaleDescHi));
                            tmem_copy_scales<false>(
                                tb + 4u * j, desc_of(ds + ((C::kScales + j * kScaleTile) >> 4), kScaleDescHi));
                        }
#pragma unroll
                        for (int j = 0; j < kFp4StageK / kFp4K; ++j) {
                            const int t = Fp4Mma<FMT>::tile_of_step(j);
                            umma_fp4<FMT, false>(d_tmem, desc_of(da + j * (kFp4K / 2 >> 4), kCodeDescHi),
                                                 desc_of(db + j * (kFp4K / 2 >> 4), kCodeDescHi),
                                                 Fp4Mma<FMT>::idesc_step(idesc, j), ta + 4u * t,
                                                 tb + 4u * t, k > k_first || j > 0 ? 1u : 0u);
                        }
                    } else {
#pragma unroll
                        for (int j = 0; j < C::kStageK / kUmmaK; ++j)
                            umma_bf16<false>(d_tmem, desc_of(da + j * (kUmmaK * 2 >> 4), kCodeDescHi),
                                             desc_of(db + j * (kUmmaK * 2 >> 4), kCodeDescHi), idesc,
                                             k > k_first || j > 0 ? 1u : 0u);
                    }
                    umma_commit<false>(empty0 + 8u * s);
                    if (k == k_last - 1) umma_commit<false>(accum_full0 + 8u * acc);
                }
                __syncwarp();
                issued = true;
                ts ^= 32u;
                da += C::kBytesA >> 4;
                db += C::kBytesB >> 4;
                ds += (2 * C::kScales) >> 4;
                if (++s == STAGES) {
                    s = 0;
                    phase ^= 1u;
                    da = a0;
                    db = b0;
                    ds = scale0;
                }
            }
        }
        if (issued) {
            if (elect_one()) umma_commit_local<false>(drain);
            __syncwarp();
            mbar_wait(drain, 0u);
        }
    } else if (warp < kEpiWarp0 + kEpiWarps) {
        // ---- epilogue ---------------------------------------------------------------
        const int quarter = warp & 3;                  // TMEM lanes this warp may read
        const int thread = quarter * 32 + lane;        // the tile's row of this lane
        const uint32_t t_lane = tmem + ((uint32_t)(quarter * 32) << 16);
        const uint32_t x_u32 = smem_u32(s_x);
        const int per = kChunkRows / split;            // rows that a CTA adds up, at most
        if (DOWN) griddep_wait();                      // the counters, and the workspace
        int tl = 0;
        for (int u = u_first; u < u_last && !*s_abort; ++u, ++tl) {
            const int acc = tl & 1, tile = u / chunks;
            const Chunk c = s_chunk[u - tile * chunks];
            const uint32_t x0 = x_u32 + (uint32_t)(acc * kChunkRows * 128 * 4);
            float v[kChunkRows];
            if (k_last > k_first) {
                if (!warp_all(wait_or_abort(accum_full0 + 8u * acc, (uint32_t)((tl >> 1) & 1), s_abort))) break;
                tc_fence_after();
                const uint32_t t_acc = t_lane + (uint32_t)(acc * kAccCols);
                constexpr int kRowsLoad = 16 / C::kTerms;       // rows within 16 columns
#pragma unroll
                for (int b = 0; b * kRowsLoad < kChunkRows; ++b) {
                    if (b * kRowsLoad >= c.rows) break;
                    uint32_t q[16];
                    tmem_ld16(t_acc + (uint32_t)(b * kRowsLoad * C::kTerms), q);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < kRowsLoad && b * kRowsLoad + i < kChunkRows; ++i) {
                        // The least term first.
                        float r = __uint_as_float(q[C::kTerms * i + C::kTerms - 1]);
#pragma unroll
                        for (int n = C::kTerms - 2; n >= 0; --n)
                            r = __uint_as_float(q[C::kTerms * i + n]) + (C::FP4 ? 0.125f * r : r);
                        v[b * kRowsLoad + i] = FMT == kFp4Mx ? 8.0f * r : r;
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(accum_free0 + 8u * acc);
            } else {
#pragma unroll
                for (int i = 0; i < kChunkRows; ++i) v[i] = 0.0f;
            }
            // To the CTA that adds the row up, once its readers are done with the buffer.
            if (!warp_all(wait_or_abort<true>(x_free0 + 8u * acc, (uint32_t)(((tl >> 1) & 1) ^ 1), s_abort))) break;
#pragma unroll
            for (int i = 0; i < kChunkRows; ++i) {
                if (i >= c.rows) break;
                float r = v[i];
                if (FMT == kFp4Nv) {
                    const int pair = s_list[c.start + i];
                    const int e = s_exp[DOWN ? pair : pair / a.K] - 8;   // -134 .. 120
                    r = r * pow2(e >> 1) * pow2(e - (e >> 1));
                }
                const uint32_t to = x0 + (uint32_t)((rank * per + i / split) * 128 + thread) * 4u;
                st_cluster_f32(map_to_rank(to, i % split), r);
            }
            __syncwarp();
            if (split == 1) {
                if (lane == 0) mbar_arrive(x_full0 + 8u * acc);
            } else if (lane < split) {
                mbar_arrive_cluster(map_to_rank(x_full0 + 8u * acc, lane));
            }
            if (!warp_all(wait_or_abort<true>(x_full0 + 8u * acc, (uint32_t)((tl >> 1) & 1), s_abort))) break;
            const float gw = a.w_scale ? __ldcg(a.w_scale + c.e) : 1.0f;
            const float* x = s_x + acc * kChunkRows * 128;
            for (int j = DOWN ? 0 : quarter >> 1; ; j += DOWN ? 1 : 2) {
                const int i = j * split + rank;
                if (i >= c.rows) break;
                const int pair = s_list[c.start + i];
                if (DOWN) {
                    float r = 0.0f;
                    for (int src = 0; src < split; ++src) r += x[(src * per + j) * 128 + thread];
                    a.y[(int64_t)pair * a.wrows + tile * 128 + thread] = r * gw;
                } else {
                    const int col = thread & 63;
                    float gate = 0.0f, up = 0.0f;
                    for (int src = 0; src < split; ++src) {
                        gate += x[(src * per + j) * 128 + col];
                        up += x[(src * per + j) * 128 + 64 + col];
                    }
                    gate *= gw;
                    up *= gw;
                    const float h = up * act_value(gate, a.act);
                    a.h[(int64_t)pair * (a.wrows / 2) + tile * 64 + col] = h;
                    if (FMT == kFp4Nv) {
                        const uint32_t m = __reduce_max_sync(~0u, __float_as_uint(h) & 0x7FFFFFFFu);
                        if (lane == 0)
                            a.h_most[(int64_t)pair * (a.wrows / 64) + tile * 2 + (quarter & 1)] = m;
                    }
                }
            }
            __syncwarp();
            if (split == 1) {
                if (lane == 0) mbar_arrive(x_free0 + 8u * acc);
            } else if (lane < split) {
                mbar_arrive_cluster_own(map_to_rank(x_free0 + 8u * acc, lane));
            }
            if (DOWN) {
                // This warp's 32 columns of the unit are in memory; the last of a tile's units
                // joins the experts' results there.
                __threadfence();
                __syncwarp();
                uint32_t old = 0u;
                if (lane == 0)
                    asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], 1;"
                                 : "=r"(old) : "l"(a.done + tile * 4 + quarter) : "memory");
                old = __shfl_sync(~0u, old, 0);
                if (old + 1u == (uint32_t)(chunks * split)) {
                    __threadfence();
                    join_experts(a, lane, tile * 128 + quarter * 32, s_score, s_ok);
                }
            }
        }
    } else if (warp < kScaleWarp0 + kScaleWarps) {
        // ---- scales of the weights: every kScaleWarps-th stage, by way of registers, the
        // warp's next stage on its way -----------------------------------------------------
        if constexpr (C::FP4) {
            const int64_t tiles = a.din / (4 * Fp4<FMT>::kBlock);
            const int n_k = k_last - k_first;
            const int stages = (u_last - u_first) * n_k;
            uint2 next[2][C::kTiles];
            auto fetch = [&](int g) {
                const int i = g / n_k, u = u_first + i, tile = u / chunks;
                const int64_t w0 = (int64_t)s_chunk[u - tile * chunks].e * a.wrows + tile * (DOWN ? 128 : 64);
                const int64_t kt = (int64_t)(k_first + g - i * n_k) * C::kTiles;
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    const int64_t row = w0 + b * (DOWN ? 64 : a.wrows / 2);
                    const uint8_t* src = a.w_scales + fp4_scale_at(row, kt, tiles) + lane * 16;
#pragma unroll
                    for (int j = 0; j < C::kTiles; ++j)
                        next[b][j] = kt + j < tiles ? __ldcg(reinterpret_cast<const uint2*>(src + j * 512))
                                                    : make_uint2(0u, 0u);
                }
            };
            int g = warp - kScaleWarp0;
            if (g < stages) fetch(g);
            for (; g < stages && !*s_abort; g += kScaleWarps) {
                const int s = g % STAGES;
                if (!warp_all(wait_or_abort(empty0 + 8u * s, (uint32_t)(((g / STAGES) & 1) ^ 1), s_abort))) break;
                const uint32_t dst = ring_s + (uint32_t)s * (2 * C::kScales) + (uint32_t)lane * 16u;
#pragma unroll
                for (int b = 0; b < 2; ++b)
#pragma unroll
                    for (int j = 0; j < C::kTiles; ++j) sts64(dst + j * kScaleTile + b * 8, next[b][j]);
                fence_proxy_async();
                __syncwarp();
                if (lane == 0) mbar_arrive(full0 + 8u * s);
                // Not before: the fence would wait for these loads.
                if (g + kScaleWarps < stages) fetch(g + kScaleWarps);
            }
        }
    } else {
        // ---- token rows --------------------------------------------------------------
        const int w = warp - kRowWarp0;
        if (DOWN) griddep_wait();                      // h
        // Every kRowWarps-th stage is this warp's, four rows (bf16: four times four) at a time. A
        // stage's later rows are fetched before its earlier ones are taken apart; its first ones
        // only after the arrival for the stage before: the fence and the arrival wait for the loads
        // that are out, and behind a ring's worth of weights a load takes microseconds.
        constexpr int kPerLoad = C::FP4 ? 1 : 4;       // rows that the warp covers at once
        constexpr int kAhead = 4;
        const int lane_row = C::FP4 ? 0 : lane >> 3, lane_col = (C::FP4 ? lane : lane & 7) * 8;
        const int n_k = k_last - k_first;
        const int stages = (u_last - u_first) * n_k;
        auto fetch = [&](Eight<DOWN> (&into)[kAhead], int g, int r0) {
            const int i = g / n_k;
            const Chunk c = s_chunk[(u_first + i) % chunks];
            const int col = (k_first + g - i * n_k) * C::kStageK + lane_col;
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                const int r = r0 + j * kPerLoad + lane_row;
                if (r0 + j * kPerLoad >= c.rows) break;
                const bool in = r < c.rows && col < a.din;
                const int pair = s_list[c.start + (in ? r : 0)];
                into[j].load(a.rows, (int64_t)(DOWN ? pair : pair / a.K) * a.din + col, in);
            }
        };
        Eight<DOWN> cur[kAhead], later[kAhead];
        if (w < stages) fetch(cur, w, 0);
        if (!DOWN) asm volatile("bar.arrive 3, %0;" ::"n"(32 * (1 + kRowWarps)) : "memory");
        if constexpr (FMT == kFp4Nv && DOWN) {
            // The rows' largest magnitudes, from those that the first kernel left of 32 columns.
            const int words = a.din / 32;
            for (int p0 = w * 8; p0 < pairs; p0 += kRowWarps * 8) {
                uint32_t m[8] = {};
                for (int i0 = lane; i0 < words; i0 += 64) {   // sixteen loads on their way
                    uint32_t v[8][2];
#pragma unroll
                    for (int n = 0; n < 8; ++n)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const int i = i0 + 32 * h;
                            v[n][h] = 0u;
                            if (p0 + n < pairs && i < words)
                                v[n][h] = __float_as_uint(ld_cg_f32(reinterpret_cast<const float*>(a.h_most) +
                                                                    (int64_t)(p0 + n) * words + i));
                        }
#pragma unroll
                    for (int n = 0; n < 8; ++n) m[n] = max(m[n], max(v[n][0], v[n][1]));
                }
#pragma unroll
                for (int n = 0; n < 8; ++n) {
                    const uint32_t most = __reduce_max_sync(~0u, m[n]);
                    // A pair without an expert has none, and what is there is not used.
                    if (lane == 0 && p0 + n < pairs) s_exp[p0 + n] = (int16_t)digit_exponent(most & 0x7FFFFFFFu);
                }
            }
            asm volatile("bar.sync 2, %0;" ::"n"(32 * kRowWarps) : "memory");
        }
        for (int g = w; g < stages && !*s_abort; g += kRowWarps) {
            const int s = g % STAGES;
            const Chunk c = s_chunk[(u_first + g / n_k) % chunks];
            const uint32_t sb = ring_b + (uint32_t)s * C::kBytesB;
            if (!warp_all(wait_or_abort(empty0 + 8u * s, (uint32_t)(((g / STAGES) & 1) ^ 1), s_abort))) break;
#pragma unroll 1
            for (int r0 = 0; r0 < c.rows; r0 += kAhead * kPerLoad) {
                const bool more = r0 + kAhead * kPerLoad < c.rows;
                if (more) fetch(later, g, r0 + kAhead * kPerLoad);
#pragma unroll
                for (int j = 0; j < kAhead; ++j) {
                    const int r = r0 + j * kPerLoad + lane_row;
                    if (r0 + j * kPerLoad >= c.rows) break;
                    if constexpr (C::FP4) {
                        int row_exp = 0;
                        if (FMT == kFp4Nv) {
                            const int pair = s_list[c.start + r];
                            row_exp = s_exp[DOWN ? pair : pair / a.K];
                        }
                        const int4 q0 = cur[j].q[0], q1 = cur[j].q[DOWN ? 1 : 0];
                        store_digits<FMT, DOWN>(sb, ring_s + (uint32_t)s * (2 * C::kScales) + C::kScales,
                                                r * C::kTerms, lane, row_exp, q0.x, q0.y, q0.z, q0.w, q1.x,
                                                q1.y, q1.z, q1.w);
                    } else if (r < c.rows) {
                        const uint32_t unit = (uint32_t)(lane & 7);
                        auto put = [&](int n, uint32_t w0, uint32_t w1, uint32_t w2, uint32_t w3) {
                            sts128(sb + (uint32_t)(n * 128) + ((unit ^ (uint32_t)(n & 7)) << 4), w0, w1, w2, w3);
                        };
                        if constexpr (DOWN) {
                            float v[8];
                            cur[j].floats(v);
#pragma unroll
                            for (int n = 0; n < C::kTerms; ++n) {
                                uint32_t q[4];
#pragma unroll
                                for (int i = 0; i < 4; ++i) q[i] = cut_bf16x2(v[2 * i], v[2 * i + 1]);
                                put(C::kTerms * r + n, q[0], q[1], q[2], q[3]);
                            }
                        } else {
                            const int4 q = cur[j].q[0];
                            put(r, (uint32_t)q.x, (uint32_t)q.y, (uint32_t)q.z, (uint32_t)q.w);
                        }
                    }
                }
                if (more) {
#pragma unroll
                    for (int j = 0; j < kAhead; ++j) cur[j] = later[j];
                }
            }
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) mbar_arrive(full0 + 8u * s);
            if (g + kRowWarps < stages) fetch(cur, g + kRowWarps, 0);
        }
    }

    __syncwarp();
    if (threadIdx.x == 0 && *s_abort) atomicOr(a.err, kErrTimeout);
    tc_fence_before();
    __syncthreads();
    if (split > 1) cluster_sync();   // nothing is on its way to a peer that has left
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc<false>(tmem, kLayerTmem);
    }
    if (DOWN) griddep_launch_dependents();
}

// CTAs of a grid of clusters of `split` CTAs, one to an SM, within the SM budget; 0 if none
// fits. Cached per kernel, split and device.
template <typename Kernel>
int layer_grid(Kernel kernel, int threads, size_t smem, int split, int num_sms)
{
    if (split == 1) return num_sms;
    struct Entry {
        const void* kernel;
        int dev, split, fit;
    };
    static std::mutex mu;
    static Entry entries[32];
    static int used = 0;
    int dev = 0, fit = -1;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    const void* k = reinterpret_cast<const void*>(kernel);
    std::lock_guard<std::mutex> lock(mu);
    for (int i = 0; i < used && fit < 0; ++i)
        if (entries[i].kernel == k && entries[i].dev == dev && entries[i].split == split)
            fit = entries[i].fit;
    if (fit < 0) {
        int sms = 0, n = 0;
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
        cudaLaunchConfig_t cfg = {};
        cudaLaunchAttribute attr[1];
        cfg.gridDim = dim3((unsigned)(sms / split * split));
        cfg.blockDim = dim3((unsigned)threads);
        cfg.dynamicSmemBytes = smem;
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = (unsigned)split;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) {
            cudaGetLastError();
            n = 0;
        }
        fit = n * split;
        if (used < 32) entries[used++] = {k, dev, split, fit};
    }
    return fit < num_sms / split * split ? fit : num_sms / split * split;
}

// How many CTAs share a unit: what takes the fewest steps in the CTA with the most units, each
// of which costs its share of the stages and about one more. units: as many as are likely.
template <class C>
int layer_split(int64_t units, int stages, int num_sms, int* grid)
{
    int best = 0;
    int64_t least = 0;
    for (int split = 1; split <= kMaxSplit && split <= stages; split *= 2) {
        const int ctas = layer_grid(moe_layer_kernel<C>, C::kThreads, C::kSmem, split, num_sms);
        if (ctas < split) continue;
        const int64_t clusters = ctas / split;
        const int64_t cost = (units + clusters - 1) / clusters * ((stages + split - 1) / split + 1);
        if (best == 0 || cost < least) {
            best = split;
            least = cost;
            *grid = ctas;
        }
    }
    return best;
}

// A kernel's clusters, and the map of its weights.
template <class C>
struct LayerPlan {
    int split = 0, grid = 0, stages = 0;
    CUtensorMap tm;

    cudaError_t make(const void* w, int64_t wlines, int64_t din, int64_t units, int num_sms)
    {
        const cudaError_t e = cudaFuncSetAttribute(moe_layer_kernel<C>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   (int)C::kSmem);
        if (e != cudaSuccess) return e;
        stages = (int)((din + C::kStageK - 1) / C::kStageK);
        split = layer_split<C>(units, stages, num_sms, &grid);
        if (split == 0) return cudaErrorNotSupported;
        const bool ok = C::FP4 ? make_code_map(&tm, w, (uint64_t)din, (uint64_t)wlines, 64)
                               : make_map(&tm, w, (uint64_t)din, (uint64_t)wlines, 64, 64);
        return ok ? cudaSuccess : cudaErrorInvalidValue;
    }

    cudaError_t launch(const LayerKernelArgs& a, const CUtensorMap& next, const LaunchOpts& o) const
    {
        cudaLaunchConfig_t cfg = {};
        cudaLaunchAttribute attr[2];
        int n = 0;
        if (split > 1) {
            attr[n].id = cudaLaunchAttributeClusterDimension;
            attr[n].val.clusterDim.x = (unsigned)split;
            attr[n].val.clusterDim.y = attr[n].val.clusterDim.z = 1;
            ++n;
        }
        if (o.pdl) {
            attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
            attr[n].val.programmaticStreamSerializationAllowed = 1;
            ++n;
        }
        cfg.gridDim = dim3((unsigned)grid);
        cfg.blockDim = dim3(C::kThreads);
        cfg.dynamicSmemBytes = C::kSmem;
        cfg.stream = o.stream;
        cfg.attrs = attr;
        cfg.numAttrs = n;
        const cudaError_t e = cudaLaunchKernelEx(&cfg, moe_layer_kernel<C>, tm, next, a);
        if (e == cudaSuccess && o.launches) ++*o.launches;
        return e;
    }
};

template <int FMT>
cudaError_t launch_layer_format(const MoeLayerArgs& f, int num_sms, const LaunchOpts& o)
{
    LayerKernelArgs a = {};
    a.ids = f.ids;
    a.scores = f.scores;
    a.T = f.T;
    a.K = f.K;
    a.E = f.E;
    a.act = f.act;
    a.h = f.h;
    a.h_most = f.h_most;
    a.y = f.y;
    a.done = f.done;
    a.counters = (int)(f.D / 32);
    a.out = f.out;
    a.out_f32 = f.out_f32;
    a.err = f.err;
    // Units as many as are likely: every pair another expert's.
    const int64_t pairs = (int64_t)f.T * f.K, experts = pairs < f.E ? pairs : f.E;
    LayerPlan<LayerCfg<FMT, false>> up;
    LayerPlan<LayerCfg<FMT, true>> down;
    cudaError_t e = up.make(f.w_gate_up, f.E * 2 * f.dff, f.D, experts * (f.dff / 64), num_sms);
    if (e != cudaSuccess) return e;
    e = down.make(f.w_down, f.E * f.D, f.dff, experts * (f.D / 128), num_sms);
    if (e != cudaSuccess) return e;

    a.rows = static_cast<const uint16_t*>(f.x);
    a.w_scales = f.gate_up_scales;
    a.w_scale = f.gate_up_scale;
    a.din = (int)f.D;
    a.wrows = (int)(2 * f.dff);
    a.tiles = (int)(f.dff / 64);
    a.next_tiles = (int)(f.D / 128);
    a.next_stages = down.stages;
    a.next_split = down.split;
    a.next_clusters = down.grid / down.split;
    a.next_fetched = kNextBytes / (int)LayerCfg<FMT, true>::kBytesA;
    a.next_scales = f.down_scales;
    e = up.launch(a, down.tm, o);
    if (e != cudaSuccess) return e;
    a.rows = f.h;
    a.w_scales = f.down_scales;
    a.w_scale = f.down_scale;
    a.din = (int)f.dff;
    a.wrows = (int)f.D;
    a.tiles = (int)(f.D / 128);
    return down.launch(a, down.tm, o);
}

}  // namespace

cudaError_t launch_moe_layer(const MoeLayerArgs& f, int num_sms, const LaunchOpts& o)
{
    if (f.format == kFp4Mx) return launch_layer_format<kFp4Mx>(f, num_sms, o);
    if (f.format == kFp4Nv) return launch_layer_format<kFp4Nv>(f, num_sms, o);
    return launch_layer_format<kFmtBf16>(f, num_sms, o);
}

}  // namespace ep
