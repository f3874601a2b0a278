// expert_w4.cuh - the products of each expert's few rows with 4-bit weights and
// group scales, for decoding (expert_w4.cu, expert_w4_wide.cu instantiate it):
//     y[p][o] = sum over groups G of s[e][o][G] * sum over i in G of (q[e][o][i] - z) x[p][i]
// and the gated form h = act(g) * u over gate and up rows of the same matrix.
//
// What bounds it: the weights are read once for a handful of rows, half a byte
// each, so the floor is HBM. On the way a code has to become a bf16 operand in
// fewer than about three instructions per lane and code, or the SMs fall behind
// HBM: two codes at a time are masked onto the bits of 128.0 in bf16 (128 + q is
// exact there) and 128 + z is subtracted in one packed instruction, also exact.
// q - z and x are exact in bf16, so a group's sum is a plain fp32 accumulation on
// mma.sync (16 output columns x 8 rows x 16; too small and too memory-bound for
// tcgen05 to matter), and the group's scale enters once, as one fp32 fma.
//
// Layout: codes stay as a user has them, [E][dout][din / 2] bytes, the even
// element in the low nibble. The order of the contraction inside one MMA is free as
// long as both operands agree: a lane takes a 32-bit word (8 consecutive codes) of
// its row, whose masks yield the pairs (0, 4), (1, 5), (2, 6), (3, 7), and picks the
// same pairs out of 16 bytes of x.
//
// Work: a unit is 64 output columns (gated: 32 gate and 32 up) of one expert for at
// most NR of its rows over the whole contraction; an expert's row chunks follow
// each other for the same columns, so that the second finds the weights in L2.
// The contraction is cut into slices of 128 and dealt to the CTA's 8 warps in turn,
// across unit boundaries. Each warp fills its own ring of slices by TMA (codes with
// the 64-byte swizzle, which makes the word loads free of bank conflicts; x as
// [32-element chunk][row]) two slices ahead, also into the next unit, and needs no
// other warp until the unit's sums are added up through shared memory, in warp
// order. Every wait is bounded.
#pragma once

#include "umma.cuh"

namespace ep {
namespace {

constexpr int kW4Warps = 8;
constexpr int kW4Threads = 32 * kW4Warps;
constexpr int kW4Cols = 64;         // weight rows (output columns) of a unit
constexpr int kW4Slice = 128;       // contraction elements of a slice
constexpr int kW4Chunks = kW4Slice / 32;
constexpr uint32_t kW4CodeBytes = kW4Cols * kW4Slice / 2;

template <int NR_, int CPG_, bool GLU_>
struct W4Cfg {
    static constexpr int NR = NR_;          // rows of x a unit takes: 8 or 16
    static constexpr int NT = NR / 8;       // MMA row tiles (its N)
    static constexpr int CPG = CPG_;        // 32-element chunks of a scale group: 1, 2, 4
    static constexpr int GROUPS = kW4Chunks / CPG;
    static constexpr bool GLU = GLU_;
    static constexpr int kOut = GLU ? kW4Cols / 2 : kW4Cols;
    static constexpr int kPerSm = NR == 8 ? 2 : 1;
    static constexpr int SLOTS = NR == 8 ? 2 : 3;
    static constexpr uint32_t kXBytes = NR * kW4Slice * 2;
    static constexpr uint32_t kSlotBytes = kW4CodeBytes + kXBytes;
    static constexpr int kRedStride = NR + 1;
    static constexpr size_t kRing = (size_t)kW4Warps * SLOTS * kSlotBytes;
    static constexpr size_t kRed = (size_t)(kW4Warps / 2) * kW4Cols * kRedStride * 4;
    static constexpr size_t kSmemFixed = 512 + kRing + kRed + 8 * kW4Warps * SLOTS + 64;
};

// mma.sync m16n8k16: a = 16 output columns x 16, b = 16 x 8 rows.
__device__ __forceinline__ void mma_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                          uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
        "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Two codes of w as bf16 q - z: bits 0-3 and 16-19 of w onto 128.0, minus zc =
// {128 + z, 128 + z}.
__device__ __forceinline__ uint32_t w4_pair(uint32_t w, uint32_t zc)
{
    const uint32_t q = (w & 0x000F000Fu) | 0x43004300u;
    uint32_t r;
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(q), "r"(zc));
    return r;
}

__device__ __forceinline__ uint32_t lds32(uint32_t addr)
{
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr));
    return v;
}

__device__ __forceinline__ void lds128(uint32_t addr, uint32_t (&v)[4])
{
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
                 : "r"(addr));
}

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* tm, int c0, int c1,
                                            int c2, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(tm)), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
        : "memory");
}

// A warp's place in the slices of its CTA's units, dealt to the warps in turn.
struct W4Cursor {
    int unit = 0, slice;
    __device__ __forceinline__ W4Cursor(int warp, int slices) : slice(warp) { wrap(slices); }
    __device__ __forceinline__ void advance(int slices)
    {
        slice += kW4Warps;
        wrap(slices);
    }
    __device__ __forceinline__ void wrap(int slices)
    {
        while (slice >= slices) {
            slice -= slices;
            ++unit;
        }
    }
};

struct W4Unit {
    int e, row0, rows, col0;   // expert, first receive row, rows (1..NR), first output column
};

// pre[e]: units of the experts before e.
template <class C>
__device__ __forceinline__ W4Unit w4_unit(const W4Args& a, const int* pre, int E, int u)
{
    W4Unit w;
    int lo = 0, hi = E;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (pre[mid] <= u) lo = mid;
        else hi = mid;
    }
    w.e = lo;
    const int cnt = __ldcg(a.cnt + lo);
    const int chunks = (cnt + C::NR - 1) / C::NR;
    const int v = u - pre[lo];
    const int chunk = v % chunks;
    w.col0 = (v / chunks) * C::kOut;
    w.row0 = __ldcg(a.expert_offset + lo) + chunk * C::NR;
    w.rows = min(C::NR, cnt - chunk * C::NR);
    return w;
}

// Scale groups of one slice for the two weight rows that a lane looks after (row
// `lane` of each half of the unit).
template <class C>
struct W4Scales {
    float s[2][C::GROUPS];
    uint32_t z[2];             // zero points, one byte per group
};

template <class C>
__device__ __forceinline__ void w4_load_scales(const W4Args& a, const W4Unit& w, int slice,
                                               int lane, W4Scales<C>& v)
{
    const int groups = (int)(a.din / (32 * C::CPG));
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        const int o = w.col0 + (C::GLU ? 0 : 32 * half) + lane;
        const bool in = o < a.dout;
        const int64_t row = C::GLU ? ((int64_t)w.e * 2 + half) * a.dout + o
                                   : (int64_t)w.e * a.dout + o;
        v.z[half] = 0x08080808u;
        if (a.zeros) v.z[half] = 0u;
#pragma unroll
        for (int j = 0; j < C::GROUPS; ++j) {
            const int g = slice * C::GROUPS + j;
            v.s[half][j] = 0.0f;
            if (in && g < groups) {
                const int64_t at = row * groups + g;
                // Through L1: neighbouring slices read the same sectors. The scales
                // are complete once griddep_wait has returned.
                if (a.scale_f32) {
                    asm volatile("ld.global.f32 %0, [%1];"
                                 : "=f"(v.s[half][j])
                                 : "l"(static_cast<const float*>(a.scales) + at));
                } else {
                    uint16_t b;
                    asm volatile("ld.global.u16 %0, [%1];"
                                 : "=h"(b)
                                 : "l"(static_cast<const uint16_t*>(a.scales) + at));
                    v.s[half][j] = __uint_as_float((uint32_t)b << 16);
                }
                if (a.zeros) {
                    uint32_t b;
                    asm volatile("ld.global.u8 %0, [%1];" : "=r"(b) : "l"(a.zeros + at));
                    v.z[half] |= b << (8 * j);
                }
            }
        }
    }
}

template <class C>
__global__ void __launch_bounds__(kW4Threads, C::kPerSm)
expert_w4_kernel(const __grid_constant__ CUtensorMap tm_w,
                 const __grid_constant__ CUtensorMap tm_x,
                 const __grid_constant__ CUtensorMap tm_x1, W4Args a)
{
    constexpr int NT = C::NT, SLOTS = C::SLOTS;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    uint8_t* smem = smem_raw + ((512u - (raw & 511u)) & 511u);
    float* s_red = reinterpret_cast<float*>(smem + C::kRing);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kRing + C::kRed);
    int* s_sum = reinterpret_cast<int*>(bars + kW4Warps * SLOTS);   // [8] warp totals
    volatile int* s_abort = s_sum + kW4Warps;
    int* s_pre = s_sum + kW4Warps + 2;                                // [E + 1]

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, q = lane & 3;
    const int E = a.E;
    const uint32_t ring = smem_u32(smem) + (uint32_t)(warp * SLOTS) * C::kSlotBytes;
    const uint32_t bar0 = smem_u32(bars) + 8u * (uint32_t)(warp * SLOTS);
    const int nblk = (int)((a.dout + C::kOut - 1) / C::kOut);
    const int slices = (int)((a.din + kW4Slice - 1) / kW4Slice);

    if (lane == 0)
        for (int s = 0; s < SLOTS; ++s) mbar_init(bar0 + 8u * s, 1u);
    if (threadIdx.x == 0) *s_abort = 0;
    fence_mbar_init();
    griddep_wait();   // counts, offsets and the rows come from earlier kernels

    // Units before each expert: thread t takes experts [t c, t c + c).
    {
        const int c = (E + kW4Threads - 1) / kW4Threads, e0 = (int)threadIdx.x * c;
        int own = 0;
        for (int e = e0; e < min(E, e0 + c); ++e)
            own += (__ldcg(a.cnt + e) + C::NR - 1) / C::NR * nblk;
        int incl = own;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int n = __shfl_up_sync(0xffffffffu, incl, d);
            if (lane >= d) incl += n;
        }
        if (lane == 31) s_sum[warp] = incl;
        __syncthreads();
        int at = incl - own;
        for (int w = 0; w < warp; ++w) at += s_sum[w];
        for (int e = e0; e < min(E, e0 + c); ++e) {
            s_pre[e] = at;
            at += (__ldcg(a.cnt + e) + C::NR - 1) / C::NR * nblk;
        }
        if (threadIdx.x == kW4Threads - 1) s_pre[E] = at;
        __syncthreads();
    }
    const int total = s_pre[E];
    const int mine = total > (int)blockIdx.x
                         ? (total - 1 - (int)blockIdx.x) / (int)gridDim.x + 1 : 0;

    // The next slice to copy and its unit.
    W4Cursor fill(warp, slices);
    int fill_unit = -1, issued = 0;
    W4Unit fu = {};
    auto issue = [&](int slot) {
        if (fill.unit >= mine) return;
        if (fill.unit != fill_unit) {
            fu = w4_unit<C>(a, s_pre, E, (int)blockIdx.x + fill.unit * (int)gridDim.x);
            fill_unit = fill.unit;
        }
        if (lane == 0) {
            const uint32_t dst = ring + (uint32_t)slot * C::kSlotBytes;
            const uint32_t bar = bar0 + 8u * (uint32_t)slot;
            const bool one = fu.rows == 1;
            mbar_expect_tx(bar, kW4CodeBytes + (one ? kW4Slice * 2u : C::kXBytes));
            const int row = (C::GLU ? 2 : 1) * fu.e * (int)a.dout + fu.col0;
            tma_load_2d(dst, &tm_w, fill.slice * (kW4Slice / 2), row, bar);
            tma_load_2d(dst + kW4CodeBytes / 2, &tm_w, fill.slice * (kW4Slice / 2),
                        row + (C::GLU ? (int)a.dout : 32), bar);
            tma_load_3d(dst + kW4CodeBytes, one ? &tm_x1 : &tm_x, 0, fu.row0,
                        fill.slice * kW4Chunks, bar);
        }
        ++issued;
        fill.advance(slices);
    };
    for (int s = 0; s < SLOTS; ++s) issue(s);

    W4Cursor at(warp, slices);   // this warp's next slice
    int n_done = 0;              // slices it has taken
    W4Cursor ahead = at;         // the slice whose scales come next
    W4Scales<C> next;
    int next_unit = -1;
    W4Unit nu = {};
    auto prefetch = [&] {
        if (ahead.unit >= mine) return;
        if (ahead.unit != next_unit) {
            nu = w4_unit<C>(a, s_pre, E, (int)blockIdx.x + ahead.unit * (int)gridDim.x);
            next_unit = ahead.unit;
        }
        w4_load_scales<C>(a, nu, ahead.slice, lane, next);
        ahead.advance(slices);
    };
    prefetch();

    for (int iu = 0; iu < mine; ++iu) {
        const W4Unit w = w4_unit<C>(a, s_pre, E, (int)blockIdx.x + iu * (int)gridDim.x);
        const uint32_t x_rows = w.rows == 1 ? 1u : (uint32_t)C::NR;   // rows of the copied box
        float total_acc[4][NT][4] = {};
        bool ok = true;
        for (; at.unit == iu; at.advance(slices), ++n_done) {
            const int slot = n_done % SLOTS;
            const W4Scales<C> cur = next;
            prefetch();
            ok = warp_all(wait_or_abort(bar0 + 8u * slot, (uint32_t)((n_done / SLOTS) & 1), s_abort));
            if (!ok) break;
            const uint32_t codes = ring + (uint32_t)slot * C::kSlotBytes;
            const uint32_t xs = codes + kW4CodeBytes;
#pragma unroll
            for (int j = 0; j < C::GROUPS; ++j) {
                float acc[4][NT][4] = {};
                uint32_t zc[4][2];
#pragma unroll
                for (int t = 0; t < 4; ++t)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const uint32_t z = __shfl_sync(0xffffffffu, cur.z[t >> 1],
                                                       16 * (t & 1) + 8 * i + g);
                        zc[t][i] = (((z >> (8 * j)) & 0xFFu) * 0x00010001u) | 0x43004300u;
                    }
#pragma unroll
                for (int cc = 0; cc < C::CPG; ++cc) {
                    const int c = j * C::CPG + cc;
                    uint32_t b[NT][4];
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        uint32_t v[4];
                        const uint32_t r = min((uint32_t)(8 * n + g), x_rows - 1u);
                        lds128(xs + ((uint32_t)c * x_rows + r) * 64u + (uint32_t)q * 16u, v);
                        b[n][0] = __byte_perm(v[0], v[2], 0x5410);   // elements 0, 4
                        b[n][1] = __byte_perm(v[0], v[2], 0x7632);   // 1, 5
                        b[n][2] = __byte_perm(v[1], v[3], 0x5410);   // 2, 6
                        b[n][3] = __byte_perm(v[1], v[3], 0x7632);   // 3, 7
                    }
#pragma unroll
                    for (int t = 0; t < 4; ++t) {
                        // 64-byte swizzle: 16-byte unit c of line row lands at c ^ (row / 2 % 4).
                        const uint32_t r0 = (uint32_t)(16 * t + g);
                        const uint32_t sw = ((uint32_t)c ^ ((r0 >> 1) & 3u)) * 16u + (uint32_t)q * 4u;
                        const uint32_t w0 = lds32(codes + r0 * 64u + sw);
                        const uint32_t w1 = lds32(codes + (r0 + 8u) * 64u + sw);
                        uint32_t a0[4] = {w4_pair(w0, zc[t][0]), w4_pair(w1, zc[t][1]),
                                          w4_pair(w0 >> 4, zc[t][0]), w4_pair(w1 >> 4, zc[t][1])};
                        uint32_t a1[4] = {w4_pair(w0 >> 8, zc[t][0]), w4_pair(w1 >> 8, zc[t][1]),
                                          w4_pair(w0 >> 12, zc[t][0]), w4_pair(w1 >> 12, zc[t][1])};
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            mma_16816(acc[t][n], a0, b[n][0], b[n][1]);
                            mma_16816(acc[t][n], a1, b[n][2], b[n][3]);
                        }
                    }
                }
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    const float s0 = __shfl_sync(0xffffffffu, cur.s[t >> 1][j], 16 * (t & 1) + g);
                    const float s1 = __shfl_sync(0xffffffffu, cur.s[t >> 1][j], 16 * (t & 1) + 8 + g);
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        total_acc[t][n][0] = fmaf(s0, acc[t][n][0], total_acc[t][n][0]);
                        total_acc[t][n][1] = fmaf(s0, acc[t][n][1], total_acc[t][n][1]);
                        total_acc[t][n][2] = fmaf(s1, acc[t][n][2], total_acc[t][n][2]);
                        total_acc[t][n][3] = fmaf(s1, acc[t][n][3], total_acc[t][n][3]);
                    }
                }
            }
            __syncwarp();   // every lane has read the slot
            issue(slot);
        }
        // The unit's sums: warps 4-7 leave theirs in shared memory, warps 0-3 add
        // their own to them, and the four parts are added in order.
        float* red = s_red + (warp % (kW4Warps / 2)) * (kW4Cols * C::kRedStride);
        auto leave = [&](bool add) {
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        float* v = red + (16 * t + g + 8 * (i >> 1)) * C::kRedStride + 8 * n +
                                   2 * q + (i & 1);
                        *v = add ? *v + total_acc[t][n][i] : total_acc[t][n][i];
                    }
        };
        if (warp >= kW4Warps / 2) leave(false);
        __syncthreads();
        if (warp < kW4Warps / 2) leave(true);
        __syncthreads();
        if (*s_abort) break;   // the same for every warp: a wait gave up before the barrier
        uint16_t* y = static_cast<uint16_t*>(a.y);
        for (int i = threadIdx.x; i < C::kOut * w.rows; i += kW4Threads) {
            const int o = i % C::kOut, n = i / C::kOut;
            auto sum = [&](int r) {
                float v = 0.0f;
#pragma unroll
                for (int k = 0; k < kW4Warps / 2; ++k)
                    v += s_red[(k * kW4Cols + r) * C::kRedStride + n];
                return v;
            };
            float v = sum(o);
            if (C::GLU) v = act_value(v, a.act) * sum(o + 32);
            if (w.col0 + o < a.dout)
                y[(int64_t)(w.row0 + n) * a.dout + w.col0 + o] =
                    (uint16_t)(pack_bf16x2_rn(v, 0.0f) & 0xFFFFu);
        }
        __syncthreads();
    }

    // After an abort, the copies in flight land before shared memory goes away.
    if (*s_abort) {
        const uint64_t deadline = globaltimer_ns() + kWaitLimitNs;
        for (int s = 0; s < SLOTS; ++s) {
            const int k = issued - 1 - ((issued - 1 - s) % SLOTS + SLOTS) % SLOTS;   // last into s
            if (k >= 0) mbar_wait_until(bar0 + 8u * s, (uint32_t)((k / SLOTS) & 1), deadline);
        }
        if (threadIdx.x == 0) atomicOr(a.err, kErrTimeout);
    }
    griddep_launch_dependents();
}

// 2-D map of the codes: [rows][din / 2] bytes, boxes of 32 rows x 64 bytes.
inline bool make_code_map(CUtensorMap* m, const void* base, uint64_t row_bytes, uint64_t rows)
{
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[2] = {row_bytes, rows};
    const cuuint64_t strides[1] = {row_bytes};
    const cuuint32_t box[2] = {kW4Slice / 2, 32};
    const cuuint32_t estr[2] = {1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_64B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// 3-D map of the rows: 32 elements, rows, 32-element chunks; boxes of 4 chunks of box_rows rows.
inline bool make_chunk_map(CUtensorMap* m, const void* base, uint64_t din, uint64_t rows,
                           uint32_t box_rows)
{
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[3] = {32, rows, din / 32};
    const cuuint64_t strides[2] = {din * 2, 64};
    const cuuint32_t box[3] = {32, box_rows, kW4Chunks};
    const cuuint32_t estr[3] = {1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box,
              estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <class C>
cudaError_t launch_w4_cfg(const W4Args& a, const void* x, int64_t rows, const void* codes,
                          int num_sms, const LaunchOpts& o)
{
    const size_t smem = C::kSmemFixed + 4 * (size_t)(a.E + 2);
    cudaError_t e = cudaFuncSetAttribute(expert_w4_kernel<C>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    CUtensorMap tw, tx, tx1;
    const uint64_t wrows = (uint64_t)a.E * (uint64_t)a.dout * (C::GLU ? 2 : 1);
    if (!make_code_map(&tw, codes, (uint64_t)a.din / 2, wrows) ||
        !make_chunk_map(&tx, x, (uint64_t)a.din, (uint64_t)rows, C::NR) ||
        !make_chunk_map(&tx1, x, (uint64_t)a.din, (uint64_t)rows, 1))
        return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    cfg.gridDim = dim3((unsigned)(num_sms * C::kPerSm));
    cfg.blockDim = dim3(kW4Threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = o.stream;
    set_attrs(&cfg, attr, false, o.pdl);
    e = cudaLaunchKernelEx(&cfg, expert_w4_kernel<C>, tw, tx, tx1, a);
    if (e == cudaSuccess && o.launches) ++*o.launches;
    return e;
}

template <int NR>
cudaError_t launch_w4_rows(const W4Args& a, bool glu, const void* x, int64_t rows,
                           const void* codes, int num_sms, const LaunchOpts& o)
{
    switch (a.group) {
        case 32:
            return glu ? launch_w4_cfg<W4Cfg<NR, 1, true>>(a, x, rows, codes, num_sms, o)
                       : launch_w4_cfg<W4Cfg<NR, 1, false>>(a, x, rows, codes, num_sms, o);
        case 64:
            return glu ? launch_w4_cfg<W4Cfg<NR, 2, true>>(a, x, rows, codes, num_sms, o)
                       : launch_w4_cfg<W4Cfg<NR, 2, false>>(a, x, rows, codes, num_sms, o);
        case 128:
            return glu ? launch_w4_cfg<W4Cfg<NR, 4, true>>(a, x, rows, codes, num_sms, o)
                       : launch_w4_cfg<W4Cfg<NR, 4, false>>(a, x, rows, codes, num_sms, o);
    }
    return cudaErrorInvalidValue;
}

}  // namespace
}  // namespace ep
