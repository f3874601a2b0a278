// fp4_quant.cu - quantisation of bf16 matrices and of tokens on their way to the receive
// rows to microscaled 4-bit floating point (fp4.cuh has the format), and back.
//
// One thread takes 16 consecutive elements: a block of nv, half a block of mx (whose halves
// meet in one shuffle). The floor is the bytes, and without a matrix's scale that is what it
// takes: 134 M elements, 344 MB, 54 us in nv and 52 in mx (6.4 and 6.6 TB/s), 54 and 62 us back to
// bf16. With a matrix's scale 78 us: issue slots, 70% of them used (every element is multiplied and
// converted twice to see whether it lies next to a border, and where the scale comes from the
// matrix's own largest element some of most warps' elements do). Steps for that case, there and
// back: 106 + 88 us; 138 together with products of two elements in one instruction, borders found
// from two conversions (before: from each quotient's last bits), the next row on its way during
// this one's work, and one resident wave of CTAs; 133.
#include <algorithm>
#include <mutex>
#include "ep_fp4.cuh"
#include "fp4.cuh"
#include "umma.cuh"

namespace ep {
namespace {

constexpr int kThreads = 256;
constexpr int kDispatchFp4PerSm = 2;   // tiles of the one-pass dispatch on an SM
constexpr size_t kDispatchFp4Smem = 100 * 1024;   // of such a tile
// Receive rows whose codes wait in shared memory for the layout. The wait is long enough for a few
// tokens: 4096 tokens (D 4096, top 2) take 20.9 us with none kept, 20.1 with 16 rows, 19.5 with 32;
// 8192 tokens (D 7168, top 8) 105, 104 and 110, with as many as fit 128: reading and writing then
// no longer overlap. (Between the two: 32 is the first size's best, 16 the second's.)
constexpr int kKeptRows = 16;

// What 16 elements become: 8 bytes of codes, and on every fourth block's first thread the
// word of four scales.
template <int FMT, bool TENSOR_SCALE>
__device__ __forceinline__ uint2 quantize16(const int4 (&raw)[2], float g, int unit, uint32_t* word,
                                            bool* writes)
{
    float m = amax16(raw[0], raw[1]);
    if (FMT == kFp4Mx) m = __uint_as_float(max(__float_as_uint(m), __shfl_xor_sync(~0u, __float_as_uint(m), 1)));
    const uint32_t c = fp4_scale_code<FMT>(m, g);
    // The word of 4 blocks from its 4 (nv) or 8 (mx) threads.
    const int block = FMT == kFp4Mx ? unit >> 1 : unit;
    uint32_t w = c << (8 * (block & 3));
    w |= __shfl_xor_sync(~0u, w, FMT == kFp4Mx ? 2 : 1);
    w |= __shfl_xor_sync(~0u, w, FMT == kFp4Mx ? 4 : 2);
    *word = w;
    *writes = (unit & (FMT == kFp4Mx ? 7 : 3)) == 0;
    float v[16];
    bf16x16(raw[0], raw[1], v);
    return fp4_codes16<FMT, TENSOR_SCALE>(v, c, g);
}

// 32 bytes of a lane: in one access where the matrix is aligned to it (two of 16 bytes touch every
// sector of a warp's kilobyte twice), with `wide` the same for the whole grid.
__device__ __forceinline__ void load32(const uint8_t* p, bool wide, int4& a, int4& b)
{
    if (wide) {
        asm volatile("ld.global.cg.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(a.x), "=r"(a.y), "=r"(a.z), "=r"(a.w), "=r"(b.x), "=r"(b.y), "=r"(b.z),
                       "=r"(b.w)
                     : "l"(p));
    } else {
        a = ld_cg_v4(p);
        b = ld_cg_v4(p + 16);
    }
}

__device__ __forceinline__ void store32(uint8_t* p, bool wide, const uint32_t (&w)[8])
{
    if (wide) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]),
                     "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                     : "memory");
    } else {
        *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
        *reinterpret_cast<uint4*>(p + 16) = make_uint4(w[4], w[5], w[6], w[7]);
    }
}

// The scale of the matrix that a warp's row is in; its rows go up, so that a division is needed
// only where they enter another matrix.
struct RowScale {
    int64_t end = 0;
    float g = 1.0f;
    __device__ __forceinline__ void enter(const Fp4Args& a, int64_t row)
    {
        if (row < end) return;
        const uint32_t m = (uint32_t)row / (uint32_t)a.rows_per_scale;
        end = (int64_t)(m + 1) * a.rows_per_scale;
        g = __ldcg(a.tensor_scale + m);
    }
};

// A warp takes 32 units of a row after the other, the next row's on their way (grid: columns x,
// rows y, all resident at once; no index of an element is divided: that cost a quarter of the
// time).
// CTAs on an SM. Quantising with a matrix's scale takes 84 us with 5 and 78 with 4; the others take
// 54 and 52 us with 5, 57 with 4, 60 and 52 with 6. Back: 54 us (nv) and 62 (mx) with 4, 57 and
// 64 with 5, 59 and 54 with 3.
template <bool TENSOR_SCALE>
constexpr int kQuantPerSm = TENSOR_SCALE ? 4 : 5;
constexpr int kBackPerSm = 4;

template <int FMT, bool TENSOR_SCALE>
__global__ void __launch_bounds__(kThreads, kQuantPerSm<TENSOR_SCALE>) quantize_kernel(Fp4Args a)
{
    griddep_wait();
    const int lane = threadIdx.x & 31, per_row = (int)(a.cols / 16);
    const int64_t tiles = a.cols / (4 * Fp4<FMT>::kBlock);
    const int unit = (int)blockIdx.x * 32 + lane;
    const bool in = unit < per_row;       // 8 units or a multiple: lanes that share a block or a
                                          // word of scales are in or out together
    const bool wide = reinterpret_cast<uintptr_t>(a.x) % 32 == 0;
    const int64_t step = (int64_t)gridDim.y * (kThreads / 32);
    int64_t row = (int64_t)blockIdx.y * (kThreads / 32) + (threadIdx.x >> 5);
    const uint8_t* x = static_cast<const uint8_t*>(a.x) + (row * per_row + unit) * 32;
    uint8_t* codes = a.codes + (row * per_row + unit) * 8;
    int4 next[2] = {};
    if (in && row < a.rows) load32(x, wide, next[0], next[1]);
    RowScale rs;
    for (; row < a.rows; row += step) {
        const int4 raw[2] = {next[0], next[1]};
        x += step * per_row * 32;
        if (in && row + step < a.rows) load32(x, wide, next[0], next[1]);
        if (TENSOR_SCALE) rs.enter(a, row);
        uint32_t word;
        bool writes;
        const uint2 q = quantize16<FMT, TENSOR_SCALE>(raw, rs.g, unit, &word, &writes);
        if (in) {
            *reinterpret_cast<uint2*>(codes) = q;
            if (writes)
                *reinterpret_cast<uint32_t*>(
                    a.scales + fp4_scale_at(row, unit / (FMT == kFp4Mx ? 8 : 4), tiles)) = word;
        }
        codes += step * per_row * 8;
    }
    griddep_launch_dependents();
}

// 16 elements back. An element in the matrix's units is exact: nv's in fp16 (six bits, 2^-10 to
// 2688), mx's in fp32. The matrix's scale rounds it once, and bf16 once more.
template <int FMT>
__device__ __forceinline__ void dequantize16(uint2 q, uint32_t c, float g, float (&v)[16])
{
    uint32_t h2[8];
    e2m1x8_to_f16x2(q.x, reinterpret_cast<uint32_t(&)[4]>(h2[0]));
    e2m1x8_to_f16x2(q.y, reinterpret_cast<uint32_t(&)[4]>(h2[4]));
    float m = g;
    if (FMT == kFp4Mx) {
        m = ue8m0_value(c);
    } else {
        uint32_t s2;      // the scale, twice
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(s2) : "h"((uint16_t)(c * 0x101u)));
#pragma unroll
        for (int j = 0; j < 8; ++j) asm("mul.rn.f16x2 %0, %0, %1;" : "+r"(h2[j]) : "r"(s2));
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) mul2(f16_lo(h2[j]), f16_hi(h2[j]), m, v[2 * j], v[2 * j + 1]);
}

template <int FMT, bool F32>
__global__ void __launch_bounds__(kThreads, kBackPerSm) dequantize_kernel(Fp4Args a)
{
    griddep_wait();
    const int lane = threadIdx.x & 31, per_row = (int)(a.cols / 16);
    const int64_t tiles = a.cols / (4 * Fp4<FMT>::kBlock);
    const int unit = (int)blockIdx.x * 32 + lane;
    if (unit < per_row) {
        const int block = FMT == kFp4Mx ? unit >> 1 : unit;
        const bool wide = reinterpret_cast<uintptr_t>(a.out) % 32 == 0;
        const int64_t step = (int64_t)gridDim.y * (kThreads / 32);
        constexpr int kRows = 2;          // at a time, the next ones on their way
        uint2 q[kRows], qn[kRows];
        uint32_t c[kRows], cn[kRows];
        auto fetch = [&](int64_t row0) {
#pragma unroll
            for (int n = 0; n < kRows; ++n) {
                const int64_t row = min(row0 + n * step, a.rows - 1);
                qn[n] = __ldcg(reinterpret_cast<const uint2*>(a.codes + (row * per_row + unit) * 8));
                cn[n] = __ldcg(a.scales + fp4_scale_at(row, block >> 2, tiles) + (block & 3));
            }
        };
        int64_t row0 = (int64_t)blockIdx.y * (kThreads / 32) + (threadIdx.x >> 5);
        if (row0 < a.rows) fetch(row0);
        RowScale rs;
        for (; row0 < a.rows; row0 += kRows * step) {
#pragma unroll
            for (int n = 0; n < kRows; ++n) {
                q[n] = qn[n];
                c[n] = cn[n];
            }
            if (row0 + kRows * step < a.rows) fetch(row0 + kRows * step);
#pragma unroll
            for (int n = 0; n < kRows; ++n) {
                const int64_t row = row0 + n * step;
                if (row >= a.rows) break;
                if (FMT == kFp4Nv && a.tensor_scale) rs.enter(a, row);
                float v[16];
                dequantize16<FMT>(q[n], c[n], rs.g, v);
                uint8_t* o = static_cast<uint8_t*>(a.out) + (row * per_row + unit) * (F32 ? 64 : 32);
                uint32_t w[8];
                if (F32) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
#pragma unroll
                        for (int j = 0; j < 8; ++j) w[j] = __float_as_uint(v[8 * h + j]);
                        store32(o + 32 * h, wide, w);
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[j]) : "f"(v[2 * j + 1]), "f"(v[2 * j]));
                    store32(o, wide, w);
                }
            }
        }
    }
    griddep_launch_dependents();
}

// A part of a token's row, 64 units of 16 elements, is a warp's: read and quantised once, written
// to each of the token's rows. raw: the part's elements, two units a lane.
constexpr int kPermuteThreads = 256;
constexpr int kPartUnits = 64;

__device__ __forceinline__ void fetch_part(const PermuteFp4Args& a, int64_t t, int part, int per_row,
                                           int lane, int4 (&raw)[2][2])
{
    const uint8_t* x = static_cast<const uint8_t*>(a.x) + t * a.D * 2;
    const bool wide = reinterpret_cast<uintptr_t>(a.x) % 32 == 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int unit = part * kPartUnits + 32 * i + lane;
        raw[i][0] = raw[i][1] = make_int4(0, 0, 0, 0);
        if (unit < per_row) load32(x + unit * 32, wide, raw[i][0], raw[i][1]);
    }
}

// row_of(k): the receive row of the token's slot k, or -1.
template <int FMT, bool TENSOR_SCALE, class RowOf>
__device__ __forceinline__ void put_part(const PermuteFp4Args& a, int part, int per_row, int lane, float g,
                                         const int4 (&raw)[2][2], RowOf row_of)
{
    const int64_t tiles = a.D / (4 * Fp4<FMT>::kBlock);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int unit = part * kPartUnits + 32 * i + lane;
        uint32_t word;
        bool writes;
        const uint2 q = quantize16<FMT, TENSOR_SCALE>(raw[i], g, unit, &word, &writes);
        const int kt = unit / (FMT == kFp4Mx ? 8 : 4);
        for (int k = 0; k < a.K; ++k) {
            const int64_t p = row_of(k);
            if (p < 0 || unit >= per_row) continue;
            *reinterpret_cast<uint2*>(a.codes + p * (a.D / 2) + unit * 8) = q;
            if (writes) *reinterpret_cast<uint32_t*>(a.scales + fp4_scale_at(p, kt, tiles)) = word;
        }
    }
}

// After a layout of its own kernels: parts in turn over the warps.
template <int FMT, bool TENSOR_SCALE>
__global__ void __launch_bounds__(kPermuteThreads) permute_fp4_kernel(PermuteFp4Args a)
{
    griddep_wait();
    const int lane = threadIdx.x & 31;
    const int per_row = (int)(a.D / 16), parts = (per_row + kPartUnits - 1) / kPartUnits;
    const float g = TENSOR_SCALE ? __ldcg(a.tensor_scale) : 1.0f;
    const int64_t items = a.T * parts;
    for (int64_t item = ((int64_t)blockIdx.x * kPermuteThreads + threadIdx.x) >> 5; item < items;
         item += (int64_t)gridDim.x * (kPermuteThreads / 32)) {
        const int64_t t = item / parts;
        const int part = (int)(item - t * parts);
        int4 raw[2][2];
        fetch_part(a, t, part, per_row, lane, raw);
        // Lane k has the row of slot k, and of slot k + 32.
        int pos[2] = {-1, -1};
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            const int k = 32 * n + lane;
            if (k < a.K) pos[n] = __ldcg(a.pos + t * a.K + k);
            if (part == 0 && pos[n] >= 0) {
                a.recv_scores[pos[n]] = __ldcg(a.scores + t * a.K + k);
                a.recv_src[pos[n]] = (int32_t)(t * a.K + k);
            }
        }
        put_part<FMT, TENSOR_SCALE>(a, part, per_row, lane, g, raw, [&](int k) {
            return __shfl_sync(~0u, k < 32 ? pos[0] : pos[1], k & 31);
        });
    }
    griddep_launch_dependents();
}

// Layout, positions and rows in one kernel, a CTA to a tile of tokens, as the one-pass dispatch
// of whole rows (its layout, with a grid barrier or, for small calls, every id counted by every
// CTA). While the CTAs wait for one another at the barrier, the first a.kept tokens of the tile
// are quantised into shared memory, from where bulk copies bring their codes to the rows once
// these are known; the tile's other x comes to L2. Shared memory: [kLayoutWarps * Ep][3 * Ep][tile
// pairs] ints, the kept tokens' codes and words of scales.
template <int FMT, bool TENSOR_SCALE, bool SMALL>
__global__ void __launch_bounds__(kLayoutThreads, kDispatchFp4PerSm)
dispatch_fp4_kernel(LayoutArgs L, PermuteFp4Args a)
{
    extern __shared__ __align__(16) int s_dyn[];
    __shared__ int s_rank[3][kMaxRanks];
    __shared__ int s_tok[kMaxRanks];
    __shared__ int s_wsum[kLayoutWarps];
    __shared__ int s_flag;
    __shared__ uint32_t s_epoch;
    __shared__ int s_next;
    int* s_base = s_dyn;
    int* s_seed = s_base + kLayoutWarps * L.Ep;
    int* s_tot = s_seed + L.Ep;
    int* s_off = s_tot + L.Ep;
    int* s_pos = s_off + L.Ep;
    uint8_t* s_codes = reinterpret_cast<uint8_t*>(s_pos + (L.tpt * L.K + 3) / 4 * 4);
    uint32_t* s_words = reinterpret_cast<uint32_t*>(s_codes + a.kept * (a.D / 2));
    const int tile = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t t0 = (int64_t)tile * L.tpt, t1 = min(L.T, t0 + L.tpt);
    const int n_my = (int)(t1 - t0), K = L.K;
    griddep_wait();
    const int per_row = (int)(a.D / 16), parts = (per_row + kPartUnits - 1) / kPartUnits;
    const int tiles = (int)(a.D / (4 * Fp4<FMT>::kBlock));
    const float g = TENSOR_SCALE ? __ldcg(a.tensor_scale) : 1.0f;
    const int kept = SMALL ? 0 : min(n_my, a.kept);
    if (threadIdx.x == 0) s_next = 0;
    const uint8_t* x0 = static_cast<const uint8_t*>(a.x) + t0 * a.D * 2;
    for (int64_t i = (int64_t)threadIdx.x * 128 + kept * a.D * 2; i < n_my * a.D * 2; i += (int64_t)kLayoutThreads * 128)
        asm volatile("prefetch.global.L2 [%0];" ::"l"(x0 + i));
    // Parts of the kept tokens, taken in turn by whichever warp has time.
    auto keep = [&] {
        __syncwarp();
        auto take = [&] {
            int i = 0;
            if (lane == 0) i = atomicAdd(&s_next, 1);
            return __shfl_sync(~0u, i, 0);
        };
        int4 next[2][2];
        int item = take();
        const int items = kept * parts;
        if (item < items) fetch_part(a, t0 + item / parts, item % parts, per_row, lane, next);
        while (item < items) {
            const int tt = item / parts, part = item - tt * parts;
            int4 raw[2][2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                raw[i][0] = next[i][0];
                raw[i][1] = next[i][1];
            }
            item = take();
            if (item < items) fetch_part(a, t0 + item / parts, item % parts, per_row, lane, next);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int unit = part * kPartUnits + 32 * i + lane;
                uint32_t word;
                bool writes;
                const uint2 q = quantize16<FMT, TENSOR_SCALE>(raw[i], g, unit, &word, &writes);
                if (unit >= per_row) continue;
                *reinterpret_cast<uint2*>(s_codes + tt * (a.D / 2) + unit * 8) = q;
                if (writes) s_words[tt * tiles + unit / (FMT == kFp4Mx ? 8 : 4)] = word;
            }
        }
        fence_proxy_async();   // the bulk copies read the codes
    };
    if constexpr (SMALL) {
        redundant_counts(L, tile, s_seed, s_tot, s_rank);
        layout_offsets(L, s_base, s_seed, s_tot, s_off, s_rank, s_wsum);
    } else {
        if (!onepass_layout(L, tile, s_base, s_seed, s_tot, s_off, s_rank, s_tok, s_wsum, &s_flag,
                            &s_epoch, s_pos, nullptr, [] {}, keep)) {
            if (threadIdx.x == 0) atomicOr(L.err, kErrTimeout);
            griddep_launch_dependents();
            return;
        }
    }
    if (tile == 0) {
        for (int e = threadIdx.x; e < L.E; e += blockDim.x) {
            L.cnt[e] = s_tot[e];
            L.expert_offset[e] = s_off[e];
        }
        if (threadIdx.x < L.R) {
            L.rows_per_rank[threadIdx.x] = s_rank[0][threadIdx.x];
            L.rank_prefix[threadIdx.x] = s_rank[1][threadIdx.x];
            L.tokens_in_rank[threadIdx.x] = s_rank[2][threadIdx.x];
        }
    }
    tile_positions(L, tile, s_base, L.pos, s_pos, s_seed, SMALL ? nullptr : s_pos);
    // Rows the layout can have; others only after its barrier words were corrupted.
    const int64_t rows = (int64_t)L.R * L.S;
    for (int j = threadIdx.x; j < n_my * K; j += kLayoutThreads) {
        const int p = s_pos[j];
        if (p < 0) continue;
        if (p >= rows) {
            atomicOr(L.err, kErrRowOob);
            s_pos[j] = -1;
            continue;
        }
        a.recv_scores[p] = __ldcg(a.scores + t0 * K + j);
        a.recv_src[p] = (int32_t)(t0 * K + j);
    }
    __syncthreads();
    for (int j = threadIdx.x; j < kept * K; j += kLayoutThreads) {
        const int p = s_pos[j];
        if (p >= 0)
            bulk_s2g(a.codes + p * (a.D / 2), smem_u32(s_codes + j / K * (a.D / 2)), (uint32_t)(a.D / 2));
    }
    bulk_commit();
    for (int j = warp; j < kept * K; j += kLayoutWarps) {
        const int p = s_pos[j];
        if (p < 0) continue;
        for (int kt = lane; kt < tiles; kt += 32)
            *reinterpret_cast<uint32_t*>(a.scales + fp4_scale_at(p, kt, tiles)) = s_words[j / K * tiles + kt];
    }
    // The next part's elements are on their way while this one is written.
    int4 next[2][2];
    const int items = n_my * parts, first = kept * parts + warp;
    if (first < items) fetch_part(a, t0 + first / parts, first % parts, per_row, lane, next);
    for (int item = first; item < items; item += kLayoutWarps) {
        const int tt = item / parts, part = item - tt * parts;
        int4 raw[2][2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            raw[i][0] = next[i][0];
            raw[i][1] = next[i][1];
        }
        const int after = item + kLayoutWarps;
        if (after < items) fetch_part(a, t0 + after / parts, after % parts, per_row, lane, next);
        put_part<FMT, TENSOR_SCALE>(a, part, per_row, lane, g, raw, [&](int k) { return s_pos[tt * K + k]; });
    }
    bulk_wait_all();
    griddep_launch_dependents();
}

// Columns of 32 units by rows, eight to a CTA; as many CTAs as are resident at once, if need be.
dim3 grid_for(const Fp4Args& a, int per_sm)
{
    int dev = 0, sms = 0;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    const int64_t x = (a.cols / 16 + 31) / 32, rows = (a.rows + kThreads / 32 - 1) / (kThreads / 32);
    int64_t most = (int64_t)sms * per_sm / x;
    if (most < 1) most = 1;
    if (most > 65535) most = 65535;
    return dim3((unsigned)x, (unsigned)(rows < most ? rows : most));
}

}  // namespace

cudaError_t launch_quantize_fp4(const Fp4Args& a, const LaunchOpts& o)
{
    const dim3 grid = grid_for(a, a.tensor_scale ? kQuantPerSm<true> : kQuantPerSm<false>);
    if (a.format == kFp4Mx) return launch_kernel(quantize_kernel<kFp4Mx, false>, grid, kThreads, 0, o, a);
    return a.tensor_scale ? launch_kernel(quantize_kernel<kFp4Nv, true>, grid, kThreads, 0, o, a)
                          : launch_kernel(quantize_kernel<kFp4Nv, false>, grid, kThreads, 0, o, a);
}

cudaError_t launch_dequantize_fp4(const Fp4Args& a, const LaunchOpts& o)
{
    const dim3 grid = grid_for(a, kBackPerSm);
    if (a.format == kFp4Mx)
        return a.out_f32 ? launch_kernel(dequantize_kernel<kFp4Mx, true>, grid, kThreads, 0, o, a)
                         : launch_kernel(dequantize_kernel<kFp4Mx, false>, grid, kThreads, 0, o, a);
    return a.out_f32 ? launch_kernel(dequantize_kernel<kFp4Nv, true>, grid, kThreads, 0, o, a)
                     : launch_kernel(dequantize_kernel<kFp4Nv, false>, grid, kThreads, 0, o, a);
}

cudaError_t launch_permute_fp4(const PermuteFp4Args& a, int num_sms, const LaunchOpts& o)
{
    const int64_t most = (int64_t)num_sms * (2048 / kPermuteThreads);
    const int64_t items = a.T * ((a.D / 16 + kPartUnits - 1) / kPartUnits);
    const int64_t need = (items + kPermuteThreads / 32 - 1) / (kPermuteThreads / 32);
    const int grid = (int)(need < most ? need : most);
    if (a.format == kFp4Mx)
        return launch_kernel(permute_fp4_kernel<kFp4Mx, false>, grid, kPermuteThreads, 0, o, a);
    return a.tensor_scale
               ? launch_kernel(permute_fp4_kernel<kFp4Nv, true>, grid, kPermuteThreads, 0, o, a)
               : launch_kernel(permute_fp4_kernel<kFp4Nv, false>, grid, kPermuteThreads, 0, o, a);
}


int dispatch_fp4_tiles_per_sm() { return kDispatchFp4PerSm; }

namespace {

// CTAs of the one-pass dispatch that the device holds at once, 0 if it cannot be asked; the latest
// answers are kept (asking takes as long as the launch).
int64_t resident_ctas(const void* kernel, size_t smem)
{
    struct Entry {
        const void* kernel;
        int dev;
        size_t smem;
        int64_t ctas;
    };
    static std::mutex mu;
    static Entry entries[16];
    static unsigned next = 0;
    int dev = 0, sms = 0, per_sm = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    std::lock_guard<std::mutex> lock(mu);
    for (const Entry& e : entries)
        if (e.kernel == kernel && e.dev == dev && e.smem == smem) return e.ctas;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)kDispatchFp4Smem) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
        cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, kLayoutThreads, smem) != cudaSuccess)
        return 0;
    entries[next++ % 16] = {kernel, dev, smem, (int64_t)per_sm * sms};
    return (int64_t)per_sm * sms;
}

}  // namespace

cudaError_t launch_dispatch_fp4(const LayoutArgs& l, const PermuteFp4Args& args, const LaunchOpts& o,
                                bool pdl_ok, int64_t small_pairs)
{
    PermuteFp4Args a = args;
    if (!l.gbar || l.ntiles <= 0) return cudaErrorNotSupported;
    const int64_t tile_pairs = l.tpt * l.K;
    if (tile_pairs > kMaxTilePairs) return cudaErrorNotSupported;
    const size_t tables = (size_t)((kLayoutWarps + 3) * (int64_t)l.Ep + (tile_pairs + 3) / 4 * 4) * 4;
    const bool small = l.T * l.K <= small_pairs;
    const size_t token = (size_t)(a.D / 2 + a.D / (a.format == kFp4Mx ? 32 : 16));
    a.kept = 0;
    if (!small && tables < kDispatchFp4Smem)
        a.kept = (int)std::min<int64_t>(std::min<int64_t>(l.tpt, kKeptRows / l.K),
                                        (int64_t)((kDispatchFp4Smem - tables) / token));
    const size_t smem = tables + a.kept * token;
    void (*kernel)(LayoutArgs, PermuteFp4Args) =
        a.format == kFp4Mx ? (small ? dispatch_fp4_kernel<kFp4Mx, false, true>
                                    : dispatch_fp4_kernel<kFp4Mx, false, false>)
        : a.tensor_scale   ? (small ? dispatch_fp4_kernel<kFp4Nv, true, true>
                                    : dispatch_fp4_kernel<kFp4Nv, true, false>)
                           : (small ? dispatch_fp4_kernel<kFp4Nv, false, true>
                                    : dispatch_fp4_kernel<kFp4Nv, false, false>);
    // Every CTA has to be resident for the grid barrier.
    if (smem > kDispatchFp4Smem || resident_ctas(reinterpret_cast<const void*>(kernel), smem) < l.ntiles)
        return cudaErrorNotSupported;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(l.ntiles);
    cfg.blockDim = dim3(kLayoutThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = o.stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeCooperative;
    attr[0].val.cooperative = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = (o.pdl && pdl_ok) ? 2 : 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, l, a);
    if (e == cudaErrorCooperativeLaunchTooLarge) {   // fewer SMs than the device reports (MPS)
        cudaGetLastError();
        return cudaErrorNotSupported;
    }
    if (e == cudaSuccess && o.launches) ++*o.launches;
    return e;
}

}  // namespace ep
