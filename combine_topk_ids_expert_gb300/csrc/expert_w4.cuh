// expert_w4.cuh - the products of each expert's few rows with 4-bit weights and
// group scales, for decoding (expert_w4.cu, expert_w4_4.cu, expert_w4_16.cu instantiate it):
//     y[p][o] = sum over groups G of s[e][o][G] * sum over i in G of (q[e][o][i] - z) x[p][i]
// and the gated form h = act(g) * u over gate and up rows of the same matrix.
//
// What bounds it: the weights are read once for a handful of rows, half a byte
// each, so the floor is HBM: at its rate an SM has about 725 cycles for 16 KB of
// codes, 2900 issue slots for 32768 of them. Unpacking codes into 16-bit operands on
// mma.sync (a shift, a mask and a subtraction for every two, then operands of x and
// scales at 16 x 8 outputs a step) took 3600 instructions for as many, and 328 us where
// this kernel takes 177 and 1510 (4 rows, 64 x 4096 x 7168 codes, groups of 128). So:
//   - a nibble q, zero-extended to a byte, IS an fp8 number: read as e4m3 it is
//     q * 2^-9 exactly (the subnormals and the first binade share one step). So
//     8 codes become two 32-bit operands with one shift and two masks;
//   - 128 elements of a row of x are scaled by a power of two that puts the largest
//     into [128, 256) and split into two 8-bit terms, x = hi + lo. A bf16 has 8
//     significant bits. hi is e4m3 (4 bits, down to 2^-9); what it leaves of a number of
//     the binade 2^e is 0 to 8 times 2^(e-7), which 3 bits hold: lo is e5m2, down to
//     2^-16 (with 4 rows e4m3 of 2^5 times it, down to 2^-14). So x is exact down to
//     2^-13 of the block's largest, and off by at most 2^-21 of it below, where hi has run
//     out of bits. With one element 2^12 times the others' size these lose 0.06% to that,
//     less than bf16 has lost already (with lo as plain e4m3 it was 1.8%), and fp32 sums
//     with a product of its size lose about as much;
//   - the tensor cores multiply and sum in fp32: tcgen05.mma.kind::f8f6f4 with the
//     codes as A (128 output columns on TMEM's lanes, written there by tcgen05.st
//     without passing shared memory again) and the terms of at most NR rows as B, one
//     after the other into the same accumulator (4 rows: side by side in one MMA, and
//     the drain adds them). Each scale group has its own;
//   - draining a group, a lane holds one output column: per row, its sum less the zero
//     point times the group's sum of x, times the column's scale, for the groups of a
//     block of x together, and an fma by what undoes the block's scale, two rows an
//     instruction. The group's sum is of hi + lo, what the tensor cores multiplied, so
//     that codes that equal the zero point leave nothing behind, and it is taken off
//     before the scale's rounding.
//
// Work: tiles of 128 columns (gated: 64 gate and 64 up) of all (expert, chunk of NR
// rows), laid end to end and cut into contiguous shares, one per CTA (one CTA per SM).
// Equal shares of 16-column blocks instead left tiles cut at both ends, which take as long
// as whole ones wherever draining a slice takes longer than copying it: 66 where whole tiles
// then took 57 us (16 rows, 8 x 4096 x 4096 codes, groups of 64), 203 and 197 us (4 rows, 64
// x 4096 x 7168, groups of 128). x is converted when the expert or the chunk changes and
// stays in shared memory for the tiles that follow; the copies of the codes run ahead
// over tile boundaries all the while.
//
// Measured (a graph of calls on three sets of weights, one GB300): 177 us, 5.4 TB/s or
// 81% of a copy's rate (the same 64 x 4096 x 7168 codes); 29.5 us, 4.1 TB/s (8 experts of
// these, one row each); 46.7 us (16 rows, 8 x 4096 x 4096, groups of 64, zero points),
// where converting x (about 10 us of it) and draining the scale groups are what takes long.
//
// Roles (12 warps): 0 copies codes (TMA, slices of 256 codes of 64 columns a box, 128-byte
// swizzle), 1 issues the MMAs, 2-5 move codes to TMEM, 6-9 drain, 10-11 load scales and
// zero points and lay them out for the drain (which, doing that itself, took 85 and 706 us
// where it then took 76 and 648 without: 64 tokens over 8 and 32 over 256 experts, gated
// block); 2-9 convert x together. With 16 warps (a second set that unpacks or drains) a
// thread would have 128 registers instead of 168 and the drain spills, and with shared
// memory full what spills goes to L2: 82 where it then took 67 us; reading the next
// accumulators ahead spills too, 53 where it then took 46 us. Every wait is bounded.
#pragma once

#include "umma.cuh"

namespace ep {
namespace {

constexpr int kW4Slice = 256;             // contraction elements of a slice
constexpr int kW4Block = 16;              // output columns of a block
constexpr uint32_t kW4BoxBytes = kW4Block * kW4Slice / 2;
constexpr uint32_t kW4StageBytes = 8 * kW4BoxBytes;
constexpr int kW4MaxStages = 8, kW4MinStages = 4;
constexpr int kW4ASlots = 4;              // slices of A in TMEM, 64 columns each
constexpr int kW4DCols = 256;             // TMEM columns of accumulators, then A
constexpr uint32_t kW4ABase = kW4DCols;
constexpr int kW4MaxDSlots = 8;
constexpr uint32_t kW4StateBytes = 1024;  // barriers and small state
constexpr int kW4ScaleSets = 2;           // of 8 groups of a tile, as the drain takes them
constexpr uint32_t kW4SetBytes = 8 * 128 * 8;
constexpr int kW4Bars = 2 * kW4MaxStages + 2 * kW4ASlots + 2 * kW4MaxDSlots + 2 * kW4ScaleSets + 4;

template <int NR_, int GROUP_>
struct W4Cfg {
    static constexpr int NR = NR_, GROUP = GROUP_;
    static constexpr int N = NR < 16 ? 16 : NR;              // of the MMA (M = 128 wants 16)
    static constexpr int kConvThreads = 256;   // warps 2 and up: four unpack, four drain
    static constexpr int kThreads = 64 + kConvThreads + 64;
    static constexpr int GPS = kW4Slice / GROUP;             // scale groups of a slice
    static constexpr int GB = GPS < 128 / N ? GPS : 128 / N;             // groups per accumulator slot
    static constexpr int DSLOTS = kW4DCols / (GB * N);
    static constexpr int SPB = 8 / GPS;                      // slices whose scales a lane loads at once
    // Ring slices at most. Scales are a third as many bytes as the codes with groups of 32
    // and come through L1, which gets what the ring leaves: 20.4 against 22.0 us with 6
    // and 8 (13 rows, 8 x 2048 x 4096 codes, fp32 scales); groups of 128 want the longer
    // ring, 648 against 661 us (gated block, 32 tokens over 256 experts).
    static constexpr int STAGES = GROUP == 32 ? 6 : kW4MaxStages;
    static constexpr int STEPS = GROUP / 32;                 // MMAs (K = 32) of a group
    // kind::f8f6f4: fp32 accumulate, A and B e4m3 (0), both K-major, N, M = 128; and with
    // the second term, B e5m2 (1 at bits 10-12).
    static constexpr uint32_t kIdesc = (1u << 4) | ((uint32_t)(N >> 3) << 17) | (8u << 24);
    static constexpr uint32_t kIdescLo = kIdesc | (1u << 10);
    static constexpr uint32_t kTermBytes = NR * 128;         // a term of 128 contraction elements
    static constexpr uint32_t kPanelBytes = 2 * kTermBytes;  // hi rows, then lo rows
    // With 4 rows both terms fit the MMA's columns, so both are e4m3, and the drain adds
    // 2^-5 of the second; with more, a second MMA adds it to the first one's accumulator.
    static constexpr bool kBothTerms = 2 * NR <= 8;
    static constexpr int LD = kBothTerms ? 2 * NR : NR;      // accumulator columns of a group to drain
    static constexpr int PG = GB < 32 / LD ? GB : 32 / LD;   // groups that a lane drains at once
    static constexpr int SB = PG < 128 / GROUP ? PG : 128 / GROUP;   // of these, in one block of x
    static constexpr int kSwap = 64 * (NR + 1) * 4;          // gated: up sums on their way to gate lanes
    static_assert(GPS % GB == 0 && GB % PG == 0 && NR <= 16 && DSLOTS <= kW4MaxDSlots, "slots");
};

// Shared memory: the ring, x, its group sums, the swap area, barriers, row state, tables.
struct W4Plan {
    int stages;      // ring slices
    int panel;       // contraction elements of x held at once (a multiple of 256)
    size_t smem;
};

// Accumulators D, operand A in TMEM at d + a few columns, B in shared memory.
__device__ __forceinline__ void umma_e4m3_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                             uint32_t idesc, uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&v)[32])
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31};"
        ::"r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
          "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]),
          "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]), "r"(v[19]), "r"(v[20]), "r"(v[21]),
          "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]), "r"(v[28]),
          "r"(v[29]), "r"(v[30]), "r"(v[31]), "r"(taddr)
        : "memory");
}

__device__ __forceinline__ void tmem_wait_st()
{
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// COLS (8 or 16) accumulator columns of this lane.
template <int COLS>
__device__ __forceinline__ void tmem_ld_cols(uint32_t taddr, uint32_t* v)
{
    if (COLS == 8)
        asm volatile(
            "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
            : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]),
              "=r"(v[7])
            : "r"(taddr));
    else
        asm volatile(
            "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
            "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
            : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]),
              "=r"(v[7]), "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]),
              "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
            : "r"(taddr));
}

__device__ __forceinline__ void lds128(uint32_t addr, uint32_t (&v)[4])
{
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
                 : "r"(addr));
}

__device__ __forceinline__ void ld_cg_32(const void* p, int4& a, int4& b)
{
    asm volatile("ld.global.cg.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(a.x), "=r"(a.y), "=r"(a.z), "=r"(a.w), "=r"(b.x), "=r"(b.y), "=r"(b.z),
                   "=r"(b.w)
                 : "l"(p));
}

// Two fp32 values in one register pair, and their products and fmas, one instruction
// for both.
__device__ __forceinline__ uint64_t pair_of(uint32_t lo, uint32_t hi)
{
    return ((uint64_t)hi << 32) | lo;
}

__device__ __forceinline__ uint64_t pair_of(float lo, float hi)
{
    return pair_of(__float_as_uint(lo), __float_as_uint(hi));
}

__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b)
{
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}

// The two terms (round to nearest even) of two fp32 values below 256 that are bf16 numbers
// times a power of two: by way of f16, which holds 2^-17 and above exactly (what is smaller
// has zeros as its terms, or lo's least number) and the first term's difference too.
// SCALED: lo is 2^5 times the second term in e4m3, else the second term in e5m2, the upper
// half of an f16. Adds hi + lo, the two values that the products are of, to *sum (a pair).
template <bool SCALED>
__device__ __forceinline__ void w4_terms(uint64_t v, uint32_t* hi, uint32_t* lo, uint64_t* sum)
{
    uint32_t f, b, d, c;
    uint16_t h, l;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(f)
        : "f"(__uint_as_float((uint32_t)(v >> 32))), "f"(__uint_as_float((uint32_t)v)));
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(h) : "r"(f));
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(b) : "h"(h));
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(f), "r"(b));
    // The sums hi + lo are exact: at most f's bits.
    if (SCALED) {
        asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(d), "r"(0x50005000u));   // 2^5
        asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(l) : "r"(d));
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(c) : "h"(l));
        asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(b) : "r"(c), "r"(0x28002800u), "r"(b));   // 2^-5
    } else {
        asm("cvt.rn.satfinite.e5m2x2.f16x2 %0, %1;" : "=h"(l) : "r"(d));
        c = __byte_perm((uint32_t)l, 0u, 0x1404);
        asm("add.rn.f16x2 %0, %1, %2;" : "=r"(b) : "r"(b), "r"(c));
    }
    *hi = h;
    *lo = l;
    float s0 = __uint_as_float((uint32_t)*sum), s1 = __uint_as_float((uint32_t)(*sum >> 32));
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
        "add.rn.f32.f16 %0, a, %0;\n\tadd.rn.f32.f16 %1, b, %1;\n\t}"
        : "+f"(s0), "+f"(s1) : "r"(b));
    *sum = pair_of(s0, s1);
}

// A barrier among some warps of the CTA that gives up on an abort: each warp arrives
// once, then waits. (A hardware barrier could not be left.)
struct W4Sync {
    uint32_t bar;
    volatile int* abort;
    uint32_t phase = 0u;
    __device__ __forceinline__ bool operator()(int lane)
    {
        __syncwarp();
        if (lane == 0) mbar_arrive(bar);
        const bool ok = warp_all(wait_or_abort(bar, phase, abort));
        phase ^= 1u;
        return ok;
    }
};

// A tile: up to 8 blocks (gated: 4) of one expert's columns for one chunk of its rows.
struct W4Tile {
    int e, chunk, row0, rows, col0, blocks;
};

// How the columns of an expert are cut: nb blocks, `most` to a tile, `tiles` of these.
struct W4Cut {
    int nb, most, tiles;
};

struct W4Tables {
    const int* pre;   // [E + 1] tiles of the experts before each
    const int* cnt;   // [E]
    const int* off;   // [E]
};

template <class C>
__device__ __forceinline__ W4Tile w4_tile(const W4Tables& t, int E, const W4Cut& cut, int b)
{
    W4Tile w;
    w.e = expert_of(t.pre, E, b);
    const int local = b - t.pre[w.e];
    w.chunk = local / cut.tiles;
    const int blk = (local - w.chunk * cut.tiles) * cut.most;
    w.col0 = blk * kW4Block;
    w.row0 = t.off[w.e] + w.chunk * C::NR;
    w.rows = min(C::NR, t.cnt[w.e] - w.chunk * C::NR);
    w.blocks = min(cut.most, cut.nb - blk);
    return w;
}

// A ring position: slot and the parity of its current phase.
struct W4Ring {
    int slot = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void next(int n)
    {
        if (++slot == n) {
            slot = 0;
            phase ^= 1u;
        }
    }
};

__device__ __forceinline__ float w4_scale_at(const W4Args& a, int64_t i)
{
    // Through L1 (a lane's next groups share its sectors); complete once griddep_wait
    // has returned.
    if (a.scale_f32) {
        float v;
        asm volatile("ld.global.f32 %0, [%1];" : "=f"(v) : "l"(static_cast<const float*>(a.scales) + i));
        return v;
    }
    uint16_t v;
    asm volatile("ld.global.u16 %0, [%1];" : "=h"(v) : "l"(static_cast<const uint16_t*>(a.scales) + i));
    return __uint_as_float((uint32_t)v << 16);
}

__device__ __forceinline__ float w4_zero_at(const W4Args& a, int64_t i)
{
    if (!a.zeros) return 8.0f;
    uint32_t v;
    asm volatile("ld.global.u8 %0, [%1];" : "=r"(v) : "l"(a.zeros + i));
    return (float)v;
}

// The power of two that takes a block whose largest magnitude has these bits to [128,
// 256) (as far as fp32 reaches), and what undoes it.
__device__ __forceinline__ uint32_t w4_scale_exponent(uint32_t max_bits)
{
    return min(261u - (max_bits >> 23), 253u);
}

__device__ __forceinline__ float w4_unscale(uint32_t max_bits)
{
    return __uint_as_float((254u - w4_scale_exponent(max_bits)) << 23);
}

__device__ __forceinline__ bool w4_odd(uint32_t bits) { return (bits & 0x7F800000u) == 0x7F800000u; }

// Element j (0..7) of 8 bf16 as fp32 bits.
__device__ __forceinline__ uint32_t w4_element(const int4& v, int j)
{
    const uint32_t w = (uint32_t)((j >> 1) == 0 ? v.x : (j >> 1) == 1 ? v.y : (j >> 1) == 2 ? v.z : v.w);
    return (j & 1) ? w & 0xFFFF0000u : w << 16;
}

// The largest magnitude of 8 bf16 as bf16 bits, and the 8 with infinities and NaNs
// as zeros.
__device__ __forceinline__ uint32_t w4_largest(const int4& v)
{
    constexpr uint32_t kAbs = 0x7FFF7FFFu;
    const uint32_t m = __vmaxu2(__vmaxu2((uint32_t)v.x & kAbs, (uint32_t)v.y & kAbs),
                                __vmaxu2((uint32_t)v.z & kAbs, (uint32_t)v.w & kAbs));
    return max(m & 0xFFFFu, m >> 16);
}

__device__ __forceinline__ int4 w4_finite(const int4& v)
{
    int w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (w4_odd((uint32_t)w[i])) w[i] &= 0x0000FFFF;
        if (w4_odd((uint32_t)w[i] << 16)) w[i] &= (int)0xFFFF0000;
    }
    return make_int4(w[0], w[1], w[2], w[3]);
}

// Converts the tile's rows of x, contraction elements [k0, k0 + panel): two 8-bit terms
// of each block of 128 elements, scaled, as B of the MMAs; what undoes the scale; and
// the groups' sums of both terms. An infinity or a NaN counts as zero here and
// marks its row (its terms are added to the row's results one by one). Warps 2 and
// up; ct: thread among them.
//
// A call, not inlined: two roles come here, seldom, and neither should hold its
// registers or repeat its code.
template <class C>
__device__ __noinline__ bool w4_convert(const uint16_t* x, int rows, int din, int ct, int k0,
                                        int panel, uint8_t* s_x, float* s_xsum, int* s_odd,
                                        int* s_odd_next, W4Sync sync)
{
    // A lane takes 32 elements at a time, four lanes a block of 128.
    const int per_row = panel / 32, total = rows * per_row;
    float* s_undo = s_xsum + panel / C::GROUP * C::NR;
    // 32 bytes a load where x allows: 16 of each lane's 64 fetch every sector twice.
    const bool by32 = (reinterpret_cast<uintptr_t>(x) & 31u) == 0u;
    int4 w[4], ahead[4];
    auto load = [&](int at) {
        const int row = at / per_row, k = k0 + 32 * (at - row * per_row);
        const bool in = at < total && k < din;
        const uint16_t* p = x + (int64_t)row * din + k;
        if (by32) {
#pragma unroll
            for (int i = 0; i < 4; i += 2)
                if (in) ld_cg_32(p + 8 * i, ahead[i], ahead[i + 1]);
                else ahead[i] = ahead[i + 1] = make_int4(0, 0, 0, 0);
            return;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) ahead[i] = in ? ld_cg_v4(p + 8 * i) : make_int4(0, 0, 0, 0);
    };
    load(ct);                             // on their way while the previous tile is drained
    if (!sync(ct & 31)) return false;     // it is: x and its sums are free
    if (ct < C::NR) s_odd_next[ct] = 0;   // nobody uses the other half of the row state now
#pragma unroll 1
    for (int base = ct & ~31; base < total; base += C::kConvThreads) {   // the same for a warp
        const int at = base + (ct & 31), row = at / per_row, part = at - row * per_row;
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = ahead[i];
        load(at + C::kConvThreads);       // on their way while these are converted
        uint32_t m = 0u;
#pragma unroll
        for (int i = 0; i < 4; ++i) m = max(m, w4_largest(w[i]));
        if (m >= 0x7F80u) {   // rare: an infinity or a NaN
            s_odd[row] = 1;
            m = 0u;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                w[i] = w4_finite(w[i]);
                m = max(m, w4_largest(w[i]));
            }
        }
        m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
        m = max(m, __shfl_xor_sync(0xffffffffu, m, 2)) << 16;
        const float scale = __uint_as_float(w4_scale_exponent(m) << 23);
        const uint64_t scale2 = pair_of(scale, scale);
        uint64_t sum2 = 0ull;
        uint32_t hi[8], lo[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            // Bytes in the order of the unpacked codes: even elements, then odd ones.
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                uint32_t h[2], l[2];
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const uint64_t v = mul2(pair_of(w4_element(w[i], j + 4 * u),
                                                    w4_element(w[i], j + 4 * u + 2)), scale2);
                    w4_terms<C::kBothTerms>(v, &h[u], &l[u], &sum2);
                }
                hi[2 * i + j] = h[0] | (h[1] << 16);
                lo[2 * i + j] = l[0] | (l[1] << 16);
            }
        }
        float sum = __uint_as_float((uint32_t)sum2) + __uint_as_float((uint32_t)(sum2 >> 32));
        if (C::GROUP >= 64) sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        if (C::GROUP >= 128) sum += __shfl_xor_sync(0xffffffffu, sum, 2);
        if (at < total) {
            uint8_t* dst = s_x + (uint32_t)(part >> 2) * C::kPanelBytes + row * 128;
            const int c = 2 * (part & 3);   // the first of its two 16-byte units
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                *reinterpret_cast<uint4*>(dst + (((c + i) ^ (row & 7)) << 4)) =
                    make_uint4(hi[4 * i], hi[4 * i + 1], hi[4 * i + 2], hi[4 * i + 3]);
                *reinterpret_cast<uint4*>(dst + C::kTermBytes +
                                          (((c + i) ^ ((row + C::NR) & 7)) << 4)) =
                    make_uint4(lo[4 * i], lo[4 * i + 1], lo[4 * i + 2], lo[4 * i + 3]);
            }
            if ((part & (C::GROUP / 32 - 1)) == 0) s_xsum[part / (C::GROUP / 32) * C::NR + row] = sum;
            if ((part & 3) == 0) s_undo[(part >> 2) * C::NR + row] = w4_unscale(m);
        }
    }
    fence_proxy_async();   // the MMAs read B through the async proxy
    __syncwarp();
    return true;
}

// The terms of a row's infinities and NaNs in one output column.
__device__ __forceinline__ float w4_odd_terms(const W4Args& a, int row, int64_t wrow, int groups)
{
    const uint16_t* x = static_cast<const uint16_t*>(a.x) + (int64_t)row * a.din;
    float sum = 0.0f;
#pragma unroll 1
    for (int k = 0; k < a.din; k += 8) {
        const int4 v = ld_cg_v4(x + k);
        if (w4_largest(v) < 0x7F80u) continue;
#pragma unroll 1
        for (int j = 0; j < 8; ++j) {
            const uint32_t b = w4_element(v, j);
            if (!w4_odd(b)) continue;
            const int i = k + j;
            const int code = (a.codes[(wrow * a.din + i) >> 1] >> (4 * (i & 1))) & 15;
            const int64_t at = wrow * groups + i / a.group;
            sum += ((float)code - w4_zero_at(a, at)) * w4_scale_at(a, at) * __uint_as_float(b);
        }
    }
    return sum;
}

// Starts the scales (and zero points) of `rows` weight rows on their way to L2: the
// drain reads them a few groups at a time, too little to wait for HBM each time.
__device__ __forceinline__ void w4_prefetch_bytes(const void* p, int64_t bytes)
{
    const uintptr_t lo = (reinterpret_cast<uintptr_t>(p) + 15u) & ~(uintptr_t)15u;
    const int64_t n = (bytes - (int64_t)(lo - reinterpret_cast<uintptr_t>(p))) & ~(int64_t)15;
    if (n > 0)
        asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(lo), "r"((uint32_t)n)
                     : "memory");
}

__device__ __forceinline__ void w4_prefetch_scales(const W4Args& a, int64_t row, int rows)
{
    const int64_t groups = a.din / a.group, at = row * groups, n = rows * groups;
    w4_prefetch_bytes(static_cast<const uint8_t*>(a.scales) + at * (a.scale_f32 ? 4 : 2),
                      n * (a.scale_f32 ? 4 : 2));
    if (a.zeros) w4_prefetch_bytes(a.zeros + at, n);
}

// A column of a tile.
struct W4Lane {
    int o;             // output column
    int64_t wrow;      // weight row
    bool live;         // a column of the tile
    bool warp_live;    // its warp has one
};

__device__ __forceinline__ W4Lane w4_lane(const W4Args& a, const W4Tile& t, int64_t wrows, int r)
{
    W4Lane l;
    const int rr = a.glu ? r & 63 : r;
    l.o = t.col0 + rr;
    l.live = rr < kW4Block * t.blocks && l.o < a.dout;
    l.warp_live = (rr & ~31) < kW4Block * t.blocks;
    l.wrow = (int64_t)t.e * wrows + (a.glu && r >= 64 ? a.dout : 0) + l.o;
    return l;
}

// The scales and zero points of 8 groups as loaded: nothing is done with them until
// they are used, so that the loads' latency lies in between.
// wide: the rows' groups are a multiple of 8 and the arrays aligned to 16 (zeros 8)
// bytes, so that 8 groups are one or two loads. One at a time they kept the loads of a
// lane's own line (32 lines for a warp) busy longer than HBM needed for the codes: 49
// against 30 us without them (13 rows, 8 x 2048 x 4096 codes, groups of 32, fp32).
struct W4Scales {
    uint32_t s[8];   // fp32 bits; bf16 in pairs (wide), or one in each
    uint32_t z[2];   // bytes
};

__device__ __forceinline__ void w4_load_scales(const W4Args& a, const W4Lane& l, int groups,
                                               bool wide, int first, W4Scales& v)
{
    const int64_t at = l.wrow * groups + first;
#pragma unroll
    for (int j = 0; j < 8; ++j) v.s[j] = 0u;   // a column that is not there: scale 0
    v.z[0] = v.z[1] = 0x08080808u;
    if (!l.live || first >= groups) return;
    if (wide) {
        if (a.scale_f32) {
            const float* p = static_cast<const float*>(a.scales) + at;
            asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(v.s[0]), "=r"(v.s[1]), "=r"(v.s[2]), "=r"(v.s[3]) : "l"(p));
            asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(v.s[4]), "=r"(v.s[5]), "=r"(v.s[6]), "=r"(v.s[7]) : "l"(p + 4));
        } else {
            asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(v.s[0]), "=r"(v.s[1]), "=r"(v.s[2]), "=r"(v.s[3])
                         : "l"(static_cast<const uint16_t*>(a.scales) + at));
        }
        if (a.zeros)
            asm volatile("ld.global.v2.u32 {%0, %1}, [%2];" : "=r"(v.z[0]), "=r"(v.z[1])
                         : "l"(a.zeros + at));
        return;
    }
    uint32_t z[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const bool in = first + j < groups;
        z[j] = 0u;
        if (in && a.scale_f32)
            asm volatile("ld.global.u32 %0, [%1];" : "=r"(v.s[j])
                         : "l"(static_cast<const float*>(a.scales) + at + j));
        if (in && !a.scale_f32) {
            uint16_t b;
            asm volatile("ld.global.u16 %0, [%1];" : "=h"(b)
                         : "l"(static_cast<const uint16_t*>(a.scales) + at + j));
            v.s[j] = b;
        }
        if (in && a.zeros) asm volatile("ld.global.u8 %0, [%1];" : "=r"(z[j]) : "l"(a.zeros + at + j));
    }
    if (a.zeros) {
        v.z[0] = z[0] | (z[1] << 8) | (z[2] << 16) | (z[3] << 24);
        v.z[1] = z[4] | (z[5] << 8) | (z[6] << 16) | (z[7] << 24);
    }
}

// Into the column's places [8][128] of a set: the scale times the codes' 2^9, and minus
// the zero point in the codes' units of 2^-9.
__device__ __forceinline__ void w4_keep_scales(const W4Scales& v, bool f32, bool wide, float2* mine)
{
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const uint32_t pair = v.s[j >> 1];
        const uint32_t bits = f32 ? v.s[j] : !wide ? v.s[j] << 16 : (j & 1) ? pair & 0xFFFF0000u : pair << 16;
        const float scale = __uint_as_float(bits);
        mine[j * 128] = make_float2(scale * 512.0f,
                                    -0x1p-9f * (float)((v.z[j >> 2] >> (8 * (j & 3))) & 0xFFu));
    }
}

template <class C>
__global__ void __launch_bounds__(C::kThreads, 1)
expert_w4_kernel(const __grid_constant__ CUtensorMap tm_w,
                 const __grid_constant__ CUtensorMap tm_half, const __grid_constant__ W4Args a,
                 const __grid_constant__ W4Plan plan)
{
    constexpr int NR = C::NR, N = C::N;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    // Barriers and small state first (their addresses are then one register and
    // constants), the ring, x with its sums, the tables.
    uint8_t* state = smem_raw + ((1024u - (raw & 1023u)) & 1023u);
    const uint32_t code_full0 = smem_u32(state);
    const uint32_t code_empty0 = code_full0 + 8u * kW4MaxStages;
    const uint32_t a_full0 = code_empty0 + 8u * kW4MaxStages;
    const uint32_t a_empty0 = a_full0 + 8u * kW4ASlots;
    const uint32_t d_full0 = a_empty0 + 8u * kW4ASlots;
    const uint32_t d_empty0 = d_full0 + 8u * kW4MaxDSlots;
    const uint32_t x_full = d_empty0 + 8u * kW4MaxDSlots;
    const uint32_t drain = x_full + 8u;
    const uint32_t conv = drain + 8u;      // warps 2 and up
    const uint32_t swapped = conv + 8u;    // the drain's
    const uint32_t sc_full0 = swapped + 8u;
    const uint32_t sc_empty0 = sc_full0 + 8u * kW4ScaleSets;
    uint32_t* s_tmem = reinterpret_cast<uint32_t*>(state + 8 * kW4Bars);
    volatile int* s_abort = reinterpret_cast<volatile int*>(s_tmem + 1);
    int* s_warp = reinterpret_cast<int*>(s_tmem + 2);   // [16] scan
    // [2][NR], this tile's rows and the next ones: the row has an infinity or a NaN.
    int* s_odd0 = s_warp + 16;
    static_assert(8 * kW4Bars + 8 + 4 * 16 + 8 * NR <= (int)kW4StateBytes, "state");
    uint8_t* smem = state + kW4StateBytes;
    const int stages = plan.stages, panel = plan.panel;
    uint8_t* s_x = smem + (size_t)stages * kW4StageBytes;                 // B, panel / 128 parts
    float* s_xsum = reinterpret_cast<float*>(s_x + (size_t)panel * 2 * NR);    // [panel / GROUP][NR]
    float* s_undo = s_xsum + panel / C::GROUP * NR;                       // [panel / 128][NR]
    float* s_swap = s_undo + panel / 128 * NR;
    float2* s_scale = reinterpret_cast<float2*>(s_swap + C::kSwap / 4);   // [sets][8][128]
    int* s_pre = reinterpret_cast<int*>(s_scale + kW4ScaleSets * 8 * 128);
    const int E = a.E;
    int* s_cnt = s_pre + E + 1;
    int* s_off = s_cnt + E;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    W4Cut cut;
    cut.nb = (int)((a.dout + kW4Block - 1) / kW4Block);
    cut.most = a.glu ? 4 : 8;
    cut.tiles = (cut.nb + cut.most - 1) / cut.most;
    const int slices = (int)((a.din + kW4Slice - 1) / kW4Slice);
    const int per_panel = panel / kW4Slice;
    const int64_t wrows = a.glu ? 2 * a.dout : a.dout;   // weight rows of an expert

    if (threadIdx.x == 0) {
        for (int s = 0; s < kW4MaxStages; ++s) {
            mbar_init(code_full0 + 8u * s, 1u);
            mbar_init(code_empty0 + 8u * s, 4u);
        }
        for (int s = 0; s < kW4ASlots; ++s) {
            mbar_init(a_full0 + 8u * s, 4u);
            mbar_init(a_empty0 + 8u * s, 1u);
        }
        for (int s = 0; s < kW4MaxDSlots; ++s) {
            mbar_init(d_full0 + 8u * s, 1u);
            mbar_init(d_empty0 + 8u * s, 4u);
        }
        mbar_init(x_full, C::kConvThreads / 32);
        mbar_init(drain, 1u);
        mbar_init(conv, C::kConvThreads / 32);
        mbar_init(swapped, 4u);
        for (int s = 0; s < kW4ScaleSets; ++s) {
            mbar_init(sc_full0 + 8u * s, 2u);
            mbar_init(sc_empty0 + 8u * s, 4u);
        }
        *s_abort = 0;
        fence_mbar_init();
    }
    if ((int)threadIdx.x < 2 * NR) s_odd0[threadIdx.x] = 0;
    if (warp == 1) {
        tmem_alloc<false>(smem_u32(s_tmem), 512u);
        tmem_relinquish<false>();
    }
    griddep_wait();   // counts, offsets and the rows come from earlier kernels

    // Tiles before each expert: thread t takes experts [t c, t c + c).
    {
        const int c = (E + C::kThreads - 1) / C::kThreads, e0 = (int)threadIdx.x * c;
        int own = 0;
        for (int e = e0; e < min(E, e0 + c); ++e) {
            s_cnt[e] = __ldcg(a.cnt + e);
            s_off[e] = __ldcg(a.expert_offset + e);
            own += (s_cnt[e] + NR - 1) / NR * cut.tiles;
        }
        int incl = own;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, incl, d);
            if (lane >= d) incl += v;
        }
        if (lane == 31) s_warp[warp] = incl;
        __syncthreads();
        int at = incl - own;
        for (int w = 0; w < warp; ++w) at += s_warp[w];
        for (int e = e0; e < min(E, e0 + c); ++e) {
            s_pre[e] = at;
            at += (s_cnt[e] + NR - 1) / NR * cut.tiles;
        }
        if (threadIdx.x == C::kThreads - 1) s_pre[E] = at;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *s_tmem;
    const W4Tables tab = {s_pre, s_cnt, s_off};
    const int64_t total = s_pre[E];
    const int first = (int)(total * blockIdx.x / gridDim.x);
    const int last = (int)(total * (blockIdx.x + 1) / gridDim.x);

    if (warp == 0) {
        // ---- codes: TMA into the ring (the warp waits together, one lane issues) ----
        W4Ring c;
        int issued = 0;
        bool ok = true;
        for (int b = first; b < last && ok;) {
            const W4Tile t = w4_tile<C>(tab, E, cut, b);
            ++b;
            const int row = (int)(t.e * wrows) + t.col0;
            const int row2 = a.glu ? row + (int)a.dout : row + 64;   // of the tile's second half
            const bool whole = t.blocks == cut.most;
            if (elect_one())
                for (int half = 0; half < (a.glu ? 2 : 1); ++half)
                    w4_prefetch_scales(a, (int64_t)row + half * a.dout,
                                       min(t.blocks * kW4Block, (int)a.dout - t.col0));
            for (int k = 0; k < slices; ++k) {
                ok = warp_all(wait_or_abort(code_empty0 + 8u * c.slot, c.phase ^ 1u, s_abort));
                if (!ok) break;
                const uint32_t bar = code_full0 + 8u * c.slot;
                const uint32_t dst = smem_u32(smem) + (uint32_t)c.slot * kW4StageBytes;
                const int kb = k * (kW4Slice / 2);
                if (elect_one()) {
                    if (whole) {
                        mbar_expect_tx(bar, kW4StageBytes);
                        tma_load_2d(dst, &tm_half, kb, row, bar);
                        tma_load_2d(dst + 4 * kW4BoxBytes, &tm_half, kb, row2, bar);
                    } else {
                        mbar_expect_tx(bar, (uint32_t)(a.glu ? 2 * t.blocks : t.blocks) * kW4BoxBytes);
                        for (int j = 0; j < t.blocks; ++j) {
                            tma_load_2d(dst + j * kW4BoxBytes, &tm_w, kb, row + 16 * j, bar);
                            if (a.glu)
                                tma_load_2d(dst + (4 + j) * kW4BoxBytes, &tm_w, kb, row2 + 16 * j, bar);
                        }
                    }
                }
                __syncwarp();
                ++issued;
                c.next(stages);
            }
        }
        // The copies land before shared memory goes away (also after an abort).
        const uint64_t deadline = globaltimer_ns() + kWaitLimitNs;
        for (int i = issued > stages ? issued - stages : 0; i < issued; ++i)
            mbar_wait_until(code_full0 + 8u * (uint32_t)(i % stages), (uint32_t)(i / stages) & 1u,
                            deadline);
    } else if (warp == 1) {
        // ---- MMA issuer (the warp waits together, one lane issues) --------------
        W4Ring as, ds;
        uint32_t x_phase = 0u;
        int e_have = -1, chunk_have = -1;
        bool issued = false, ok = true;
        const uint64_t x_desc = smem_desc_k128(smem_u32(s_x));
        for (int b = first; b < last && ok;) {
            const W4Tile t = w4_tile<C>(tab, E, cut, b);
            ++b;
            const bool new_rows = t.e != e_have || t.chunk != chunk_have;
            e_have = t.e;
            chunk_have = t.chunk;
            int in_panel = 0;
            for (int k = 0; k < slices; ++k, ++in_panel) {
                if (in_panel == per_panel) in_panel = 0;
                if (in_panel == 0 && (new_rows || per_panel < slices)) {
                    ok = warp_all(wait_or_abort(x_full, x_phase, s_abort));
                    x_phase ^= 1u;
                    if (!ok) break;
                }
                ok = warp_all(wait_or_abort(a_full0 + 8u * as.slot, as.phase, s_abort));
                if (!ok) break;
                const uint64_t bx = x_desc + (uint64_t)((uint32_t)in_panel * (2u * C::kPanelBytes >> 4));
                const uint32_t at = tmem + kW4ABase + (uint32_t)as.slot * 64u;
#pragma unroll
                for (int g0 = 0; g0 < C::GPS; g0 += C::GB) {
                    if (ok) ok = warp_all(wait_or_abort(d_empty0 + 8u * ds.slot, ds.phase ^ 1u, s_abort));
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t d = tmem + (uint32_t)(ds.slot * C::GB * N);
                    if (elect_one()) {
#pragma unroll
                        for (int i = 0; i < C::GB * C::STEPS; ++i) {
                            const int step = g0 * C::STEPS + i;   // of 32 elements in the slice
                            const uint64_t hi =
                                bx + (uint64_t)(((step >> 2) * C::kPanelBytes + (step & 3) * 32) >> 4);
                            const uint32_t to = d + (uint32_t)(i / C::STEPS * N);
                            // (Where the MMA's columns are more than the terms', the rest
                            // see what follows in shared memory; nobody reads them.)
                            umma_e4m3_ts(to, at + (uint32_t)step * 8u, hi, C::kIdesc,
                                         i % C::STEPS != 0 ? 1u : 0u);
                            if (!C::kBothTerms)
                                umma_e4m3_ts(to, at + (uint32_t)step * 8u,
                                             hi + (C::kTermBytes >> 4), C::kIdescLo, 1u);
                        }
                        umma_commit<false>(d_full0 + 8u * ds.slot);
                        if (g0 + C::GB == C::GPS) umma_commit<false>(a_empty0 + 8u * as.slot);
                    }
                    __syncwarp();
                    issued = true;
                    ds.next(C::DSLOTS);
                }
                if (!ok) break;
                as.next(kW4ASlots);
            }
        }
        if (issued) {   // every MMA has finished before TMEM is freed
            if (elect_one()) umma_commit_local<false>(drain);
            __syncwarp();
            mbar_wait(drain, 0u);
        }
    } else if (warp >= 10) {
        // ---- scales and zero points, 8 groups of the tile's columns at a time -----
        const int groups = (int)(a.din / C::GROUP);
        const bool wide = groups % 8 == 0 && (reinterpret_cast<uintptr_t>(a.scales) & 15u) == 0u &&
                          (reinterpret_cast<uintptr_t>(a.zeros) & 7u) == 0u;
        const int r = (int)threadIdx.x - 320;   // columns r and r + 64 of the tile
        W4Ring set;
        W4Scales next[2];
        auto load = [&](const W4Tile& t, int k) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
                w4_load_scales(a, w4_lane(a, t, wrows, r + 64 * h), groups, wide, k * C::GPS, next[h]);
        };
        bool ok = true;
        if (first < last) load(w4_tile<C>(tab, E, cut, first), 0);
#pragma unroll 1
        for (int b = first; b < last && ok;) {
            const W4Tile t = w4_tile<C>(tab, E, cut, b);
            ++b;
#pragma unroll 1
            for (int k = 0; k < slices; k += C::SPB) {
                ok = warp_all(wait_or_abort(sc_empty0 + 8u * set.slot, set.phase ^ 1u, s_abort));
                if (!ok) break;
                float2* to = s_scale + set.slot * (8 * 128) + r;
                w4_keep_scales(next[0], a.scale_f32, wide, to);
                w4_keep_scales(next[1], a.scale_f32, wide, to + 64);
                __syncwarp();
                if (lane == 0) mbar_arrive(sc_full0 + 8u * set.slot);
                set.next(kW4ScaleSets);
                // The next 8 groups' are on their way until the drain wants them; over the
                // tile's end too.
                if (k + C::SPB < slices) load(t, k + C::SPB);
                else if (b < last) load(w4_tile<C>(tab, E, cut, b), 0);
            }
        }
    } else {
        const int ct = (int)threadIdx.x - 64;
        const int quarter = warp & 3;
        const int r = quarter * 32 + lane;                // output column of the tile / TMEM lane
        const uint32_t t_lane = tmem + ((uint32_t)(quarter * 32) << 16);
        const bool drains = warp >= 6;
        W4Sync conv_sync = {conv, s_abort};
        int e_have = -1, chunk_have = -1, half = 1;   // half: of the row state
        bool ok = true, new_rows = false;
        auto begin = [&](const W4Tile& t) {
            new_rows = t.e != e_have || t.chunk != chunk_have;
            if (new_rows) half ^= 1;
            e_have = t.e;
            chunk_have = t.chunk;
        };
        // Before slice k0 of tile t: converts the panel of its rows that begins there,
        // unless it is there. Every warp gets here for the same panels.
        auto need_x = [&](const W4Tile& t, int k0) {
            if (!new_rows && per_panel >= slices) return true;
            const bool done =
                w4_convert<C>(static_cast<const uint16_t*>(a.x) + (int64_t)t.row0 * a.din, t.rows,
                              (int)a.din, ct, k0 * kW4Slice, panel, s_x, s_xsum, s_odd0 + half * NR,
                              s_odd0 + (half ^ 1) * NR, conv_sync);
            conv_sync.phase ^= 1u;
            if (done && lane == 0) mbar_arrive(x_full);
            return done;
        };
        if (!drains) {
            // ---- codes to TMEM ----------------------------------------------------
            W4Ring c, as;
#pragma unroll 1
            for (int b = first; b < last && ok;) {
                const W4Tile t = w4_tile<C>(tab, E, cut, b);
                ++b;
                const bool warp_live = w4_lane(a, t, wrows, r).warp_live;
                begin(t);
#pragma unroll 1
                for (int k0 = 0; k0 < slices && ok; k0 += per_panel) {
                    ok = need_x(t, k0);
                    if (!ok) break;
                    const int k1 = min(slices, k0 + per_panel);
#pragma unroll 1
                    for (int k = k0; k < k1; ++k, c.next(stages), as.next(kW4ASlots)) {
                        ok = warp_all(wait_or_abort(code_full0 + 8u * c.slot, c.phase, s_abort));
                        if (!ok) break;
                        const uint32_t base = smem_u32(smem) + (uint32_t)c.slot * kW4StageBytes +
                                              (uint32_t)r * 128u;
                        ok = warp_all(wait_or_abort(a_empty0 + 8u * as.slot, as.phase ^ 1u, s_abort));
                        if (!ok) break;
                        tc_fence_after();
                        if (warp_live) {
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                uint32_t w[4][4], v[32];
#pragma unroll
                                for (int i = 0; i < 4; ++i)
                                    lds128(base + (uint32_t)(((4 * h + i) ^ (r & 7)) << 4), w[i]);
#pragma unroll
                                for (int i = 0; i < 16; ++i) {
                                    const uint32_t q = w[i >> 2][i & 3];
                                    v[2 * i] = q & 0x0F0F0F0Fu;
                                    v[2 * i + 1] = (q >> 4) & 0x0F0F0F0Fu;
                                }
                                tmem_st32(t_lane + kW4ABase + (uint32_t)(as.slot * 64 + h * 32), v);
                            }
                        }
                        if (warp_live) tmem_wait_st();
                        // The slot is free once every lane has its codes: after the stores
                        // that need them, not as soon as the loads are issued (the arrival
                        // overtook them, and the next copy what they had yet to read).
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(code_empty0 + 8u * c.slot);
                        if (lane == 0) mbar_arrive(a_full0 + 8u * as.slot);
                    }
                }
            }
        } else {
            // ---- drain ---------------------------------------------------------------
            W4Sync swap_sync = {swapped, s_abort};
            W4Ring ds, set;
            bool held = false;   // a set of scales
#pragma unroll 1
            for (int b = first; b < last && ok;) {
                const W4Tile t = w4_tile<C>(tab, E, cut, b);
                ++b;
                const bool warp_live = w4_lane(a, t, wrows, r).warp_live;
                begin(t);
                uint64_t acc[NR / 2];   // rows 2n and 2n + 1
#pragma unroll
                for (int n = 0; n < NR / 2; ++n) acc[n] = 0ull;
#pragma unroll 1
                for (int k0 = 0; k0 < slices && ok; k0 += per_panel) {
                    ok = need_x(t, k0);
                    if (!ok) break;
                    const int k1 = min(slices, k0 + per_panel);
#pragma unroll 1
                    for (int k = k0; k < k1 && ok; ++k) {
                        if ((k & (C::SPB - 1)) == 0) {
                            // The set before was last used a slice ago: nothing of it is
                            // still on its way from shared memory.
                            if (held) {
                                __syncwarp();
                                if (lane == 0) mbar_arrive(sc_empty0 + 8u * set.slot);
                                set.next(kW4ScaleSets);
                            }
                            held = true;
                            ok = warp_all(wait_or_abort(sc_full0 + 8u * set.slot, set.phase, s_abort));
                            if (!ok) break;
                        }
                        const float2* sc = s_scale + set.slot * (8 * 128) + r +
                                           (k & (C::SPB - 1)) * C::GPS * 128;
                        const float* sums = s_xsum + (k - k0) * (C::GPS * NR);
                        const float* undo = s_undo + (k - k0) * (2 * NR);
#pragma unroll 1
                        for (int g0 = 0; g0 < C::GPS; g0 += C::GB) {
                            ok = warp_all(wait_or_abort(d_full0 + 8u * ds.slot, ds.phase, s_abort));
                            if (!ok) break;
                            tc_fence_after();
                            // As many groups at a time as 32 accumulator columns hold.
                            const uint32_t d = t_lane + (uint32_t)(ds.slot * C::GB * N);
#pragma unroll
                            for (int p0 = 0; p0 < C::GB; p0 += C::PG) {
                                uint32_t q[C::PG * C::LD];
                                if (warp_live) {
#pragma unroll
                                    for (int u = 0; u < C::PG; ++u)
                                        tmem_ld_cols<C::LD>(d + (uint32_t)((p0 + u) * N), q + u * C::LD);
                                    tmem_wait_ld();
                                }
                                if (p0 + C::PG == C::GB) {   // the slot is free as soon as it is read
                                    tc_fence_before();
                                    __syncwarp();
                                    if (lane == 0) mbar_arrive(d_empty0 + 8u * ds.slot);
                                }
                                if (!warp_live) continue;
#pragma unroll
                                for (int u0 = 0; u0 < C::PG; u0 += C::SB) {
                                    const int gi = g0 + p0 + u0;
                                    uint64_t sx[C::SB], nz[C::SB];
#pragma unroll
                                    for (int u = 0; u < C::SB; ++u) {
                                        const float2 v = sc[(gi + u) * 128];
                                        sx[u] = pair_of(v.x, v.x);
                                        nz[u] = pair_of(v.y, v.y);
                                    }
                                    const ulonglong2* un =
                                        reinterpret_cast<const ulonglong2*>(undo + gi * C::GROUP / 128 * NR);
#pragma unroll
                                    for (int n4 = 0; n4 < NR / 4; ++n4) {
                                        const ulonglong2 u4 = un[n4];
                                        uint64_t d0, d1;
#pragma unroll
                                        for (int u = 0; u < C::SB; ++u) {
                                            const ulonglong2 x4 = reinterpret_cast<const ulonglong2*>(
                                                sums + (gi + u) * NR)[n4];
                                            const uint32_t* v = q + (u0 + u) * C::LD + 4 * n4;
                                            uint64_t v0 = pair_of(v[0], v[1]), v1 = pair_of(v[2], v[3]);
                                            if constexpr (C::kBothTerms) {
                                                v0 = fma2(pair_of(0x1p-5f, 0x1p-5f),
                                                          pair_of(v[NR], v[NR + 1]), v0);
                                                v1 = fma2(pair_of(0x1p-5f, 0x1p-5f),
                                                          pair_of(v[NR + 2], v[NR + 3]), v1);
                                            }
                                            v0 = fma2(nz[u], x4.x, v0);
                                            v1 = fma2(nz[u], x4.y, v1);
                                            d0 = u == 0 ? mul2(sx[u], v0) : fma2(sx[u], v0, d0);
                                            d1 = u == 0 ? mul2(sx[u], v1) : fma2(sx[u], v1, d1);
                                        }
                                        acc[2 * n4] = fma2(u4.x, d0, acc[2 * n4]);
                                        acc[2 * n4 + 1] = fma2(u4.y, d1, acc[2 * n4 + 1]);
                                    }
                                }
                            }
                            ds.next(C::DSLOTS);
                        }
                    }
                }
                if (!ok) break;
                const W4Lane l = w4_lane(a, t, wrows, r);
                float out[NR];
#pragma unroll
                for (int n = 0; n < NR; ++n)
                    out[n] = __uint_as_float((uint32_t)(acc[n / 2] >> (32 * (n & 1))));
                for (int n = 0; n < t.rows; ++n)
                    if (s_odd0[half * NR + n] && l.live) {
                        const float terms = w4_odd_terms(a, t.row0 + n, l.wrow, (int)(a.din / C::GROUP));
#pragma unroll
                        for (int m = 0; m < NR; ++m)
                            if (m == n) out[m] += terms;
                    }
                if (a.glu) {
                    float* swap = s_swap + (r & 63) * (NR + 1);
                    if (r >= 64)
#pragma unroll
                        for (int n = 0; n < NR; ++n) swap[n] = out[n];
                    ok = swap_sync(lane);
                    if (!ok) break;
                    if (r < 64)
#pragma unroll
                        for (int n = 0; n < NR; ++n)
                            if (n < t.rows) out[n] = act_value(out[n], a.act) * swap[n];
                    ok = swap_sync(lane);   // the swap area is free again
                    if (!ok) break;
                }
                if (l.live && (!a.glu || r < 64)) {
                    uint16_t* y = static_cast<uint16_t*>(a.y) + (int64_t)t.row0 * a.dout + l.o;
#pragma unroll
                    for (int n = 0; n < NR; ++n)
                        if (n < t.rows) y[n * a.dout] = (uint16_t)(pack_bf16x2_rn(out[n], 0.0f) & 0xFFFFu);
                }
            }
        }
    }

    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (threadIdx.x == 0 && *s_abort) atomicOr(a.err, kErrTimeout);
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc<false>(tmem, 512u);
    }
    griddep_launch_dependents();
}

// 2-D map of the codes: [rows][din / 2] bytes, boxes of box_rows rows x 128 bytes.
inline bool make_code_map(CUtensorMap* m, const void* base, uint64_t row_bytes, uint64_t rows,
                          int box_rows)
{
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[2] = {row_bytes, rows};
    const cuuint64_t strides[1] = {row_bytes};
    const cuuint32_t box[2] = {kW4Slice / 2, (cuuint32_t)box_rows};
    const cuuint32_t estr[2] = {1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Ring slices and x panel that fit: x whole if it leaves kW4MinStages, else in parts.
template <class C>
W4Plan w4_plan(int64_t din, int E)
{
    const size_t fixed =
        1024 + kW4StateBytes + C::kSwap + kW4ScaleSets * kW4SetBytes + 4 * (3 * (size_t)E + 1);
    const size_t per_slice = (size_t)kW4Slice * 2 * C::NR + (size_t)(C::GPS + 2) * C::NR * 4;   // of x
    const int64_t slices = (din + kW4Slice - 1) / kW4Slice;
    const int64_t fit =
        (int64_t)((kSmemLimit - fixed - (size_t)kW4MinStages * kW4StageBytes) / per_slice);
    const int64_t held = slices < fit ? slices : fit;
    W4Plan p;
    p.panel = (int)(held * kW4Slice);
    const size_t left = kSmemLimit - fixed - (size_t)held * per_slice;
    p.stages = (int)(left / kW4StageBytes);
    if (p.stages > C::STAGES) p.stages = C::STAGES;
    p.smem = fixed + (size_t)held * per_slice + (size_t)p.stages * kW4StageBytes;
    return p;
}

template <class C>
cudaError_t launch_w4_cfg(const W4Args& a, const void* codes, int num_sms, const LaunchOpts& o)
{
    const W4Plan plan = w4_plan<C>(a.din, a.E);
    cudaError_t e = cudaFuncSetAttribute(expert_w4_kernel<C>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemLimit);
    if (e != cudaSuccess) return e;
    CUtensorMap tw, th;
    const uint64_t wrows = (uint64_t)a.E * (uint64_t)a.dout * (a.glu ? 2 : 1);
    if (!make_code_map(&tw, codes, (uint64_t)a.din / 2, wrows, kW4Block) ||
        !make_code_map(&th, codes, (uint64_t)a.din / 2, wrows, 64))
        return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    cfg.gridDim = dim3((unsigned)num_sms);
    cfg.blockDim = dim3(C::kThreads);
    cfg.dynamicSmemBytes = plan.smem;
    cfg.stream = o.stream;
    set_attrs(&cfg, attr, false, o.pdl);
    e = cudaLaunchKernelEx(&cfg, expert_w4_kernel<C>, tw, th, a, plan);
    if (e == cudaSuccess && o.launches) ++*o.launches;
    return e;
}

template <int NR>
cudaError_t launch_w4_rows(const W4Args& a, const void* codes, int num_sms, const LaunchOpts& o)
{
    if (a.group == 32) return launch_w4_cfg<W4Cfg<NR, 32>>(a, codes, num_sms, o);
    if (a.group == 64) return launch_w4_cfg<W4Cfg<NR, 64>>(a, codes, num_sms, o);
    return launch_w4_cfg<W4Cfg<NR, 128>>(a, codes, num_sms, o);
}

}  // namespace
}  // namespace ep
