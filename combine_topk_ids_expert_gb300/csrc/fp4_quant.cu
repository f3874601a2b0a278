// fp4_quant.cu - quantisation of bf16 matrices and of tokens on their way to the receive
// rows to microscaled 4-bit floating point (fp4.cuh has the format), and back.
//
// One thread takes 16 consecutive elements: a block of nv, half a block of mx (whose halves
// meet in one shuffle). Bound by HBM, so the work per element is what matters after the
// bytes: a product with the scale's reciprocal, a rounding fix and half a conversion.
#include "ep_fp4.cuh"
#include "fp4.cuh"

namespace ep {
namespace {

constexpr int kThreads = 256;

// What 16 elements become: 8 bytes of codes, and on every fourth block's first thread the
// word of four scales.
template <int FMT, bool TENSOR_SCALE>
__device__ __forceinline__ uint2 quantize16(const float (&v)[16], float g, int unit, uint32_t* word,
                                            bool* writes)
{
    float m = amax16(v);
    if (FMT == kFp4Mx) m = __uint_as_float(max(__float_as_uint(m), __shfl_xor_sync(~0u, __float_as_uint(m), 1)));
    const uint32_t c = fp4_scale_code<FMT>(m, g);
    // The word of 4 blocks from its 4 (nv) or 8 (mx) threads.
    const int block = FMT == kFp4Mx ? unit >> 1 : unit;
    uint32_t w = c << (8 * (block & 3));
    w |= __shfl_xor_sync(~0u, w, FMT == kFp4Mx ? 2 : 1);
    w |= __shfl_xor_sync(~0u, w, FMT == kFp4Mx ? 4 : 2);
    *word = w;
    *writes = (unit & (FMT == kFp4Mx ? 7 : 3)) == 0;
    return fp4_codes16<FMT, TENSOR_SCALE>(v, c, g);
}

template <int FMT, bool TENSOR_SCALE>
__global__ void __launch_bounds__(kThreads) quantize_kernel(Fp4Args a)
{
    griddep_wait();
    const int64_t per_row = a.cols / 16, total = a.rows * per_row;
    const int64_t tiles = a.cols / (4 * Fp4<FMT>::kBlock);
    // Whole warps stay in the loop for the shuffles; per_row is a multiple of 8, so the
    // threads that share a word of scales are on one row and in or out together.
    for (int64_t i0 = (int64_t)blockIdx.x * kThreads + (threadIdx.x & ~31); i0 < total;
         i0 += (int64_t)gridDim.x * kThreads) {
        const int64_t i = i0 + (threadIdx.x & 31);
        const bool in = i < total;
        const int64_t row = in ? i / per_row : 0;
        const int unit = in ? (int)(i - row * per_row) : 0;
        float v[16] = {};
        if (in) {
            const uint8_t* p = static_cast<const uint8_t*>(a.x) + i * 32;
            bf16x16(ld_cg_v4(p), ld_cg_v4(p + 16), v);
        }
        const float g = TENSOR_SCALE && in ? __ldcg(a.tensor_scale + row / a.rows_per_scale) : 1.0f;
        uint32_t word;
        bool writes;
        const uint2 q = quantize16<FMT, TENSOR_SCALE>(v, g, unit, &word, &writes);
        if (in) {
            *reinterpret_cast<uint2*>(a.codes + i * 8) = q;
            if (writes)
                *reinterpret_cast<uint32_t*>(
                    a.scales + fp4_scale_at(row, unit / (FMT == kFp4Mx ? 8 : 4), tiles)) = word;
        }
    }
    griddep_launch_dependents();
}

template <int FMT>
__global__ void __launch_bounds__(kThreads) dequantize_kernel(Fp4Args a)
{
    griddep_wait();
    const int64_t per_row = a.cols / 16, total = a.rows * per_row;
    const int64_t tiles = a.cols / (4 * Fp4<FMT>::kBlock);
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < total;
         i += (int64_t)gridDim.x * kThreads) {
        const int64_t row = i / per_row;
        const int unit = (int)(i - row * per_row);
        const int block = FMT == kFp4Mx ? unit >> 1 : unit;
        const uint2 q = __ldcg(reinterpret_cast<const uint2*>(a.codes + i * 8));
        const float s = fp4_scale_value<FMT>(
            __ldcg(a.scales + fp4_scale_at(row, block >> 2, tiles) + (block & 3)));
        // An element's value in the matrix's units is exact in fp32; the matrix's scale
        // rounds it once, and bf16 once more.
        const float g = a.tensor_scale ? __ldcg(a.tensor_scale + row / a.rows_per_scale) : 1.0f;
        float v[16];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t h2 = e2m1x2_to_f16x2(((j < 4 ? q.x : q.y) >> (8 * (j & 3))) & 0xFFu);
            v[2 * j] = f16_lo(h2) * s * g;
            v[2 * j + 1] = f16_hi(h2) * s * g;
        }
        if (a.out_f32) {
            float4* o = reinterpret_cast<float4*>(static_cast<float*>(a.out) + i * 16);
#pragma unroll
            for (int j = 0; j < 4; ++j) o[j] = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
        } else {
            uint32_t p[8];
#pragma unroll
            for (int j = 0; j < 8; ++j)
                asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(p[j]) : "f"(v[2 * j + 1]), "f"(v[2 * j]));
            uint4* o = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + i * 16);
            o[0] = make_uint4(p[0], p[1], p[2], p[3]);
            o[1] = make_uint4(p[4], p[5], p[6], p[7]);
        }
    }
    griddep_launch_dependents();
}

// One CTA per token at a time: read and quantised once, written to each of its rows.
constexpr int kPermuteThreads = 128;

template <int FMT, bool TENSOR_SCALE>
__global__ void __launch_bounds__(kPermuteThreads) permute_fp4_kernel(PermuteFp4Args a)
{
    __shared__ int s_pos[kMaxTopk];
    __shared__ int s_n;
    griddep_wait();
    const int per_row = (int)(a.D / 16);
    const int64_t tiles = a.D / (4 * Fp4<FMT>::kBlock);
    const float g = TENSOR_SCALE ? __ldcg(a.tensor_scale) : 1.0f;
    for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
        __syncthreads();
        if (threadIdx.x < 32) {
            int n = 0;
            for (int k0 = 0; k0 < a.K; k0 += 32) {
                const int k = k0 + (int)threadIdx.x;
                const int p = k < a.K ? __ldcg(a.pos + t * a.K + k) : -1;
                if (p >= 0) {
                    a.recv_scores[p] = __ldcg(a.scores + t * a.K + k);
                    a.recv_src[p] = (int32_t)(t * a.K + k);
                }
                const unsigned some = __ballot_sync(~0u, p >= 0);
                if (p >= 0) s_pos[n + __popc(some & lanemask_lt(threadIdx.x))] = p;
                n += __popc(some);
            }
            if (threadIdx.x == 0) s_n = n;
        }
        __syncthreads();
        const int n = s_n;
        if (n == 0) continue;
        const uint8_t* x = static_cast<const uint8_t*>(a.x) + t * a.D * 2;
        for (int u0 = (int)threadIdx.x & ~31; u0 < per_row; u0 += kPermuteThreads) {
            const int unit = u0 + ((int)threadIdx.x & 31);
            const bool in = unit < per_row;
            float v[16] = {};
            if (in) bf16x16(ld_cg_v4(x + unit * 32), ld_cg_v4(x + unit * 32 + 16), v);
            uint32_t word;
            bool writes;
            const uint2 q = quantize16<FMT, TENSOR_SCALE>(v, g, unit, &word, &writes);
            if (!in) continue;
            const int kt = unit / (FMT == kFp4Mx ? 8 : 4);
            for (int j = 0; j < n; ++j) {
                const int64_t p = s_pos[j];
                *reinterpret_cast<uint2*>(a.codes + p * (a.D / 2) + unit * 8) = q;
                if (writes) *reinterpret_cast<uint32_t*>(a.scales + fp4_scale_at(p, kt, tiles)) = word;
            }
        }
    }
    griddep_launch_dependents();
}

int grid_for(int64_t work)
{
    int dev = 0, sms = 0;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    const int64_t most = (int64_t)sms * (2048 / kThreads);
    const int64_t need = (work + kThreads - 1) / kThreads;
    return (int)(need < 1 ? 1 : need < most ? need : most);
}

}  // namespace

cudaError_t launch_quantize_fp4(const Fp4Args& a, const LaunchOpts& o)
{
    const int grid = grid_for(a.rows * (a.cols / 16));
    if (a.format == kFp4Mx) return launch_kernel(quantize_kernel<kFp4Mx, false>, grid, kThreads, 0, o, a);
    return a.tensor_scale ? launch_kernel(quantize_kernel<kFp4Nv, true>, grid, kThreads, 0, o, a)
                          : launch_kernel(quantize_kernel<kFp4Nv, false>, grid, kThreads, 0, o, a);
}

cudaError_t launch_dequantize_fp4(const Fp4Args& a, const LaunchOpts& o)
{
    const int grid = grid_for(a.rows * (a.cols / 16));
    return a.format == kFp4Mx ? launch_kernel(dequantize_kernel<kFp4Mx>, grid, kThreads, 0, o, a)
                              : launch_kernel(dequantize_kernel<kFp4Nv>, grid, kThreads, 0, o, a);
}

cudaError_t launch_permute_fp4(const PermuteFp4Args& a, int num_sms, const LaunchOpts& o)
{
    const int64_t most = (int64_t)num_sms * (2048 / kPermuteThreads);
    const int grid = (int)(a.T < most ? a.T : most);
    if (a.format == kFp4Mx)
        return launch_kernel(permute_fp4_kernel<kFp4Mx, false>, grid, kPermuteThreads, 0, o, a);
    return a.tensor_scale
               ? launch_kernel(permute_fp4_kernel<kFp4Nv, true>, grid, kPermuteThreads, 0, o, a)
               : launch_kernel(permute_fp4_kernel<kFp4Nv, false>, grid, kPermuteThreads, 0, o, a);
}

}  // namespace ep
