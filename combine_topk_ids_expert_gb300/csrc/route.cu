// route.cu - the router: each token's top-k experts and their scores, and the gradient.
//
// p is the softmax of the token's logits, or their sigmoids. The K experts are those with
// the largest values of `select` (the logits, unless given), ties to the lowest index; one
// whose value is -inf or a NaN is never chosen, and a slot without an expert has id -1 and
// score 0. Scores are scale * p, or scale * p / (sum of the chosen p).
//
// One warp to a token; lane l holds the values of experts l, l + 32, ... as integers in the
// order of the floats. A round takes the warp's maximum and the lowest index that has it
// (two warp reductions) and strikes it out. Reading the logits once is the floor; the
// rounds are what bounds large calls.
//
// Normalised scores need the chosen logits alone: with m their maximum, softmax is
// e^(l - m) / sum, and sigmoid(l) e^-min(m, 0) has no common factor left that underflows.
// Sums and probabilities are in fp32.
#include "ep_fp4.cuh"
#include "ep_device.cuh"

namespace ep {
namespace {

constexpr int kRouteThreads = 128;   // 4 tokens to a CTA
constexpr float kInf = __builtin_huge_valf();

__device__ __forceinline__ float load_logit(const void* p, bool bf16, int64_t i)
{
    if (bf16)
        return __uint_as_float((uint32_t)__ldcg(static_cast<const unsigned short*>(p) + i) << 16);
    return __ldcg(static_cast<const float*>(p) + i);
}

// Integers in the order of the floats, both zeros alike; 0 for what must not be chosen.
__device__ __forceinline__ uint32_t order_of(float v)
{
    if (!(v > -kInf)) return 0u;
    const uint32_t b = __float_as_uint(v + 0.0f);
    return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(~0u, v, d);
    return v;
}

__device__ __forceinline__ float warp_max(float v)
{
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v = fmaxf(v, __shfl_xor_sync(~0u, v, d));
    return v;
}

// sigmoid(l) e^-m for m <= 0, where m = 0 if any of the logits it is used for is above 0.
__device__ __forceinline__ float sigmoid_over(float l, float m)
{
    const float e = expf(-fabsf(l));
    return l >= 0.0f ? 1.0f / (1.0f + e) : expf(l - m) / (1.0f + e);
}

// A token's softmax statistics over all experts: the maximum and the sum of e^(l - max).
template <int NV>
__device__ __forceinline__ void softmax_of_row(const float (&v)[NV], float* most, float* sum)
{
    float m = -kInf, s = 0.0f;
#pragma unroll
    for (int j = 0; j < NV; ++j) m = fmaxf(m, v[j]);
    m = warp_max(m);
#pragma unroll
    for (int j = 0; j < NV; ++j) s += m > -kInf ? expf(v[j] - m) : 0.0f;
    *most = m;
    *sum = warp_sum(s);
}

template <int NV, bool BF16>
__global__ void __launch_bounds__(kRouteThreads) route_kernel(RouteArgs a)
{
    griddep_wait();
    const int lane = threadIdx.x & 31;
    const int64_t t = ((int64_t)blockIdx.x * kRouteThreads + threadIdx.x) >> 5;
    if (t < a.T) {
        const int64_t row = t * a.E;
        uint32_t key[NV];
        float v[NV];
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int e = j * 32 + lane;
            const bool in = e < a.E;
            v[j] = -kInf;
            if (in && (!a.select || !a.normalize)) v[j] = load_logit(a.logits, BF16, row + e);
            key[j] = !in ? 0u : order_of(a.select ? __ldcg(a.select + row + e) : v[j]);
        }
        int mine[2] = {-1, -1};       // slots lane and lane + 32
        for (int k = 0; k < a.K; ++k) {
            uint32_t best = 0u;
#pragma unroll
            for (int j = 0; j < NV; ++j) best = max(best, key[j]);
            const uint32_t most = __reduce_max_sync(~0u, best);
            if (most == 0u) break;    // nothing is left
            int at = 1 << 30;
            if (best == most) {
#pragma unroll
                for (int j = NV - 1; j >= 0; --j) at = key[j] == most ? j : at;
                at = at * 32 + lane;
            }
            const int e = __reduce_min_sync(~0u, at);
            if (at == e) {
#pragma unroll
                for (int j = 0; j < NV; ++j)
                    if (j == e >> 5) key[j] = 0u;
            }
            if (lane == (k & 31)) {
                if (k < 32) mine[0] = e;
                else mine[1] = e;
            }
        }
        float l[2], p[2];
#pragma unroll
        for (int i = 0; i < 2; ++i)
            l[i] = mine[i] >= 0 ? load_logit(a.logits, BF16, row + mine[i]) : -kInf;
        float total = 1.0f;
        if (a.normalize) {
            float m = warp_max(fmaxf(l[0], l[1]));
            if (a.sigmoid) m = fminf(m, 0.0f);
#pragma unroll
            for (int i = 0; i < 2; ++i)
                p[i] = mine[i] < 0 || m == -kInf ? 0.0f
                       : a.sigmoid ? sigmoid_over(l[i], m) : expf(l[i] - m);
            total = warp_sum(p[0] + p[1]);
        } else if (a.sigmoid) {
#pragma unroll
            for (int i = 0; i < 2; ++i) p[i] = mine[i] < 0 ? 0.0f : sigmoid_over(l[i], 0.0f);
        } else {
            float m;
            softmax_of_row(v, &m, &total);
#pragma unroll
            for (int i = 0; i < 2; ++i)
                p[i] = mine[i] < 0 || m == -kInf ? 0.0f : expf(l[i] - m);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int k = i * 32 + lane;
            if (k < a.K) {
                a.ids[t * a.K + k] = mine[i];
                // A sum that is zero leaves nothing to share out; a NaN stays one.
                a.scores[t * a.K + k] = mine[i] < 0 || total == 0.0f ? 0.0f : a.scale * (p[i] / total);
            }
        }
    }
    griddep_launch_dependents();
}

// Gradient of the logits. With c_k = grad_scores_k and p, s as above:
//   sigmoid              dl_e = scale c p (1 - p)
//   softmax              dl_e = scale p_e (c_e - sum_k c_k p_k), c_e = 0 where e is not chosen
//   normalised softmax   dl_e = scale s_e (c_e - sum_k c_k s_k), over the chosen
//   normalised sigmoid   the same with a further factor 1 - p_e
// The row is put together in shared memory; an id that occurs more than once adds up in the
// order of its slots.
template <int NV, bool BF16>
__global__ void __launch_bounds__(kRouteThreads) route_backward_kernel(RouteArgs a)
{
    __shared__ float s_row[kRouteThreads / 32][NV * 32];
    griddep_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t t = ((int64_t)blockIdx.x * kRouteThreads + threadIdx.x) >> 5;
    if (t < a.T) {
        const int64_t row = t * a.E;
        int id[2];
        float l[2], c[2], w[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int k = i * 32 + lane;
            id[i] = k < a.K ? __ldcg(a.ids + t * a.K + k) : -1;
            if (id[i] < 0 || id[i] >= a.E) id[i] = -1;
            c[i] = id[i] >= 0 ? a.scale * __ldcg(a.grad_scores + t * a.K + k) : 0.0f;
            l[i] = id[i] >= 0 ? load_logit(a.logits, BF16, row + id[i]) : -kInf;
        }
        float v[NV];
        float most = 0.0f, sum = 1.0f, inner = 0.0f;
        const bool whole = !a.normalize && !a.sigmoid;
        if (whole) {
#pragma unroll
            for (int j = 0; j < NV; ++j)
                v[j] = j * 32 + lane < a.E ? load_logit(a.logits, BF16, row + j * 32 + lane) : -kInf;
            softmax_of_row(v, &most, &sum);
        } else if (a.normalize) {
            most = warp_max(fmaxf(l[0], l[1]));
            if (a.sigmoid) most = fminf(most, 0.0f);
        }
        // w: p, or s where scores are normalised.
#pragma unroll
        for (int i = 0; i < 2; ++i)
            w[i] = id[i] < 0 || most == -kInf ? 0.0f
                   : a.sigmoid ? sigmoid_over(l[i], most) : expf(l[i] - most);
        if (a.normalize) sum = warp_sum(w[0] + w[1]);
        if (sum == 0.0f) sum = 1.0f;
#pragma unroll
        for (int i = 0; i < 2; ++i) w[i] /= sum;
        if (a.normalize || whole) inner = warp_sum(c[0] * w[0] + c[1] * w[1]);
        float* r = s_row[warp];
#pragma unroll
        for (int j = 0; j < NV; ++j)
            r[j * 32 + lane] =
                whole && j * 32 + lane < a.E && most > -kInf ? -inner * (expf(v[j] - most) / sum) : 0.0f;
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if (i * 32 >= a.K) break;
            // 1 - p = sigmoid(-l).
            const float d = w[i] * (whole ? c[i] : a.normalize ? c[i] - inner : c[i]) *
                            (a.sigmoid ? sigmoid_over(-l[i], 0.0f) : 1.0f);
            const unsigned same = __match_any_sync(~0u, id[i]);
            const int earlier = id[i] >= 0 ? __popc(same & lanemask_lt(lane)) : 0;
            const int rounds = __reduce_max_sync(~0u, earlier);
            for (int n = 0; n <= rounds; ++n) {
                if (id[i] >= 0 && earlier == n) r[id[i]] += d;
                __syncwarp();
            }
        }
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int e = j * 32 + lane;
            if (e >= a.E) continue;
            if (BF16) {
                uint32_t b;
                asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(b) : "f"(0.0f), "f"(r[e]));
                static_cast<uint16_t*>(a.grad_logits)[row + e] = (uint16_t)b;
            } else {
                static_cast<float*>(a.grad_logits)[row + e] = r[e];
            }
        }
    }
    griddep_launch_dependents();
}

template <int NV>
cudaError_t launch_nv(const RouteArgs& a, bool backward, const LaunchOpts& o)
{
    const int64_t ctas = (a.T + kRouteThreads / 32 - 1) / (kRouteThreads / 32);
    const dim3 grid((unsigned)ctas);
    if (backward)
        return a.bf16 ? launch_kernel(route_backward_kernel<NV, true>, grid, kRouteThreads, 0, o, a)
                      : launch_kernel(route_backward_kernel<NV, false>, grid, kRouteThreads, 0, o, a);
    return a.bf16 ? launch_kernel(route_kernel<NV, true>, grid, kRouteThreads, 0, o, a)
                  : launch_kernel(route_kernel<NV, false>, grid, kRouteThreads, 0, o, a);
}

cudaError_t launch_any(const RouteArgs& a, bool backward, const LaunchOpts& o)
{
    if (a.E <= 32) return launch_nv<1>(a, backward, o);
    if (a.E <= 64) return launch_nv<2>(a, backward, o);
    if (a.E <= 128) return launch_nv<4>(a, backward, o);
    if (a.E <= 256) return launch_nv<8>(a, backward, o);
    if (a.E <= 512) return launch_nv<16>(a, backward, o);
    return launch_nv<32>(a, backward, o);
}

}  // namespace

cudaError_t launch_route(const RouteArgs& a, const LaunchOpts& o) { return launch_any(a, false, o); }
cudaError_t launch_route_backward(const RouteArgs& a, const LaunchOpts& o)
{
    return launch_any(a, true, o);
}

}  // namespace ep
