// route.cu - the router: each token's top-k experts and their scores, and the gradient.
//
// p is the softmax of the token's logits, or their sigmoids. The K experts are those with
// the largest values of `select` (the logits, unless given), ties to the lowest index; one
// whose value is -inf or a NaN is never chosen, and a slot without an expert has id -1 and
// score 0. Scores are scale * p, or scale * p / (sum of the chosen p).
//
// One warp to a token; lane l holds the values of NV experts from l NV on, sorted (lanes of 32 are
// searched instead). A round takes the warp's maximum of the lanes' first ones, of the lowest lane
// that has it, which moves up its list: one warp reduction, one vote. Which of its lane's experts
// a slot's value was is looked up at the end, as sorting values alone takes two instructions a
// comparison, with their places five. Reading the logits once is the floor (7.9 us for 32768 tokens
// of 256 experts with a mask); what bounds large calls is issuing instructions (82% of the slots):
// 17.0 us with 8 chosen, of these 11 for one round and 0.8 for each further one. Steps: 37 us
// unsorted, 23.5 with the places sorted along, 17.0. 512 experts (NV 16), sorted against searched:
// 25 and 16 us for one chosen, 27 and 27 for four, 31 and 45 for eight. Warps that go from token to
// token, the next one's values on their way, are slower (24.5: fewer of them fit). The gradient of
// the same tokens takes 11.7 us at a floor of 10.4 (17 with two slots to every lane, stored by single
// elements), on bf16 logits 11.0 at 5.4; that of un-normalised softmax scores, which reads and writes all
// of a row with its exponentials, 21 us for either type.
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

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(~0u, v, d);
    return v;
}

// The largest of the warp's, NaN left out.
__device__ __forceinline__ float warp_max(float v)
{
    float m;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(v));
    return m;
}

// sigmoid(l) e^-m for m <= 0, where m = 0 if any of the logits it is used for is above 0.
__device__ __forceinline__ float sigmoid_over(float l, float m)
{
    const float e = expf(-fabsf(l));
    return (l >= 0.0f ? 1.0f : expf(l - m)) / (1.0f + e);
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

// The lane's NV values of a row, experts lane NV + j: as vectors where the row allows it.
template <int NV>
__device__ __forceinline__ void load_row(const void* p, bool bf16, int64_t row, int lane, int E, float (&v)[NV])
{
    const int e0 = lane * NV;
    if (NV >= 4 && !bf16 && E % 4 == 0 && reinterpret_cast<uintptr_t>(p) % 16 == 0) {
#pragma unroll
        for (int j = 0; j < NV; j += 4) {
            int4 q = make_int4(0, 0, 0, 0);
            const bool in = e0 + j < E;
            if (in) q = ld_cg_v4(static_cast<const float*>(p) + row + e0 + j);
            const int w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
            for (int i = 0; i < 4 && j + i < NV; ++i) v[j + i] = in ? __int_as_float(w[i]) : -kInf;
        }
    } else if (NV >= 8 && bf16 && E % 8 == 0 && reinterpret_cast<uintptr_t>(p) % 16 == 0) {
#pragma unroll
        for (int j = 0; j < NV; j += 8) {
            int4 q = make_int4(0, 0, 0, 0);
            const bool in = e0 + j < E;
            if (in) q = ld_cg_v4(static_cast<const unsigned short*>(p) + row + e0 + j);
            const uint32_t w[4] = {(uint32_t)q.x, (uint32_t)q.y, (uint32_t)q.z, (uint32_t)q.w};
#pragma unroll
            for (int i = 0; i < 8 && j + i < NV; ++i)
                v[j + i] = in ? __uint_as_float(i & 1 ? w[i >> 1] & 0xFFFF0000u : w[i >> 1] << 16) : -kInf;
        }
    } else {
#pragma unroll
        for (int j = 0; j < NV; ++j) v[j] = e0 + j < E ? load_logit(p, bf16, row + e0 + j) : -kInf;
    }
}

// Sorted, the largest first: odd-even merges of neighbours, pairs of pairs, and so on.
template <int NV>
__device__ __forceinline__ void sort_down(float (&v)[NV])
{
#pragma unroll
    for (int p = 1; p < NV; p *= 2) {
#pragma unroll
        for (int k = p; k >= 1; k /= 2) {
#pragma unroll
            for (int j = k % p; j + k < NV; j += 2 * k) {
#pragma unroll
                for (int i = 0; i < k; ++i) {
                    if (i + j + k < NV && (i + j) / (2 * p) == (i + j + k) / (2 * p)) {
                        const float x = v[i + j], y = v[i + j + k];
                        v[i + j] = fmaxf(x, y);
                        v[i + j + k] = fminf(x, y);
                    }
                }
            }
        }
    }
}

// CTAs on an SM.
constexpr int route_per_sm(int nv) { return nv <= 8 ? 12 : nv == 16 ? 8 : 6; }

// WIDE: more than 32 slots, a lane then has two.
template <int NV, bool BF16, bool WIDE>
__global__ void __launch_bounds__(kRouteThreads, route_per_sm(NV)) route_kernel(RouteArgs a)
{
    griddep_wait();
    constexpr int SLOTS = WIDE ? 2 : 1;
    const int lane = threadIdx.x & 31;
    const int64_t t = ((int64_t)blockIdx.x * kRouteThreads + threadIdx.x) >> 5;
    if (t < a.T) {
        const int64_t row = t * a.E;
        const bool whole = !a.normalize && !a.sigmoid;   // a sum over all of the token's logits
        constexpr bool kSorted = NV <= 16;
        float v[NV], key[NV], sorted[kSorted ? NV : 1];
        if (a.select) {
            load_row<NV>(a.select, false, row, lane, a.E, key);
            if (whole) load_row<NV>(a.logits, BF16, row, lane, a.E, v);
        } else {
            load_row<NV>(a.logits, BF16, row, lane, a.E, key);
#pragma unroll
            for (int j = 0; j < NV; ++j) v[j] = key[j];
        }
#pragma unroll
        for (int j = 0; j < NV; ++j) key[j] = fmaxf(key[j], -kInf);   // no NaN
        if constexpr (kSorted) {
#pragma unroll
            for (int j = 0; j < NV; ++j) sorted[j] = key[j];
            sort_down(sorted);
        }
        int mine[SLOTS];              // slots lane and lane + 32: experts
        float key_of[SLOTS];          // the slots' keys,
        int from_of[SLOTS];           // and the lanes they came from
#pragma unroll
        for (int i = 0; i < SLOTS; ++i) {
            mine[i] = -1;
            key_of[i] = -kInf;
            from_of[i] = 0;
        }
        for (int k = 0; k < a.K; ++k) {
            float best = kSorted ? sorted[0] : key[0];
            int at = 0;
            if (!kSorted) {
#pragma unroll
                for (int j = 1; j < NV; ++j) {
                    at = key[j] > best ? j : at;
                    best = fmaxf(best, key[j]);
                }
            }
            const float most = warp_max(best);
            if (most == -kInf) break;    // nothing is left
            const int from = __ffs(__ballot_sync(~0u, best == most)) - 1;
            const int e = kSorted ? 0 : __shfl_sync(~0u, lane * NV + at, from);
            if (lane == from) {
#pragma unroll
                for (int j = 0; j < NV; ++j) {
                    if constexpr (kSorted) sorted[j] = j + 1 < NV ? sorted[j + 1 < NV ? j + 1 : j] : -kInf;
                    else key[j] = j == at ? -kInf : key[j];
                }
            }
#pragma unroll
            for (int i = 0; i < SLOTS; ++i) {
                if (lane == k - 32 * i) {
                    key_of[i] = most;
                    from_of[i] = from;
                    if (!kSorted) mine[i] = e;
                }
            }
        }
        if constexpr (kSorted) {
            // Where in its lane a slot's key was (sorting keys with their places takes five
            // instructions a comparison, keys alone two): of several equal ones, which come out
            // one after the other, as many are skipped as slots before this one had.
            uint64_t again = 0u;
#pragma unroll
            for (int i = 0; i < SLOTS; ++i) {
                float before = __shfl_up_sync(~0u, key_of[i], 1);
                int lane_before = __shfl_up_sync(~0u, from_of[i], 1);
                if (i > 0) {
                    const float end = __shfl_sync(~0u, key_of[0], 31);
                    const int lane_end = __shfl_sync(~0u, from_of[0], 31);
                    if (lane == 0) {
                        before = end;
                        lane_before = lane_end;
                    }
                }
                again |= (uint64_t)__ballot_sync(~0u, (i > 0 || lane > 0) && key_of[i] != -kInf &&
                                                          before == key_of[i] && lane_before == from_of[i])
                         << (32 * i);
            }
#pragma unroll
            for (int i = 0; i < SLOTS; ++i) {
                uint32_t equal = 0u;
#pragma unroll
                for (int j = 0; j < NV; ++j)
                    if (__shfl_sync(~0u, key[j], from_of[i]) == key_of[i]) equal |= 1u << j;
                if (again != 0u)
                    for (int n = __clzll(~(again << (63 - 32 * i - lane))); n > 0; --n) equal &= equal - 1u;
                if (key_of[i] != -kInf) mine[i] = from_of[i] * NV + __ffs(equal) - 1;
            }
        }
        float l[SLOTS], p[SLOTS];
#pragma unroll
        for (int i = 0; i < SLOTS; ++i)
            l[i] = mine[i] < 0 ? -kInf : a.select ? load_logit(a.logits, BF16, row + mine[i]) : key_of[i];
        float total = 1.0f;
        if (a.normalize) {
            float m = warp_max(fmaxf(l[0], l[SLOTS - 1]));
            if (a.sigmoid) m = fminf(m, 0.0f);
            float sum = 0.0f;
#pragma unroll
            for (int i = 0; i < SLOTS; ++i) {
                p[i] = mine[i] < 0 || m == -kInf ? 0.0f
                       : a.sigmoid ? sigmoid_over(l[i], m) : expf(l[i] - m);
                sum += p[i];
            }
            total = warp_sum(sum);
        } else if (a.sigmoid) {
#pragma unroll
            for (int i = 0; i < SLOTS; ++i) p[i] = mine[i] < 0 ? 0.0f : sigmoid_over(l[i], 0.0f);
        } else {
            float m;
            softmax_of_row(v, &m, &total);
#pragma unroll
            for (int i = 0; i < SLOTS; ++i)
                p[i] = mine[i] < 0 || m == -kInf ? 0.0f : expf(l[i] - m);
        }
#pragma unroll
        for (int i = 0; i < SLOTS; ++i) {
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
template <int NV, bool BF16, bool WIDE>
__global__ void __launch_bounds__(kRouteThreads) route_backward_kernel(RouteArgs a)
{
    constexpr int SLOTS = WIDE ? 2 : 1;
    __shared__ __align__(16) float s_row[kRouteThreads / 32][NV * 32];
    griddep_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t t = ((int64_t)blockIdx.x * kRouteThreads + threadIdx.x) >> 5;
    if (t < a.T) {
        const int64_t row = t * a.E;
        int id[SLOTS];
        float l[SLOTS], c[SLOTS], w[SLOTS];
#pragma unroll
        for (int i = 0; i < SLOTS; ++i) {
            const int k = i * 32 + lane;
            const int raw = k < a.K ? __ldcg(a.ids + t * a.K + k) : -1;
            const float grad = k < a.K ? __ldcg(a.grad_scores + t * a.K + k) : 0.0f;
            id[i] = raw >= 0 && raw < a.E ? raw : -1;
            c[i] = id[i] >= 0 ? a.scale * grad : 0.0f;
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
            most = warp_max(fmaxf(l[0], l[SLOTS - 1]));
            if (a.sigmoid) most = fminf(most, 0.0f);
        }
        // w: p, or s where scores are normalised.
#pragma unroll
        for (int i = 0; i < SLOTS; ++i)
            w[i] = id[i] < 0 || most == -kInf ? 0.0f
                   : a.sigmoid ? sigmoid_over(l[i], most) : expf(l[i] - most);
        if (a.normalize) sum = warp_sum(WIDE ? w[0] + w[SLOTS - 1] : w[0]);
        if (sum == 0.0f) sum = 1.0f;
#pragma unroll
        for (int i = 0; i < SLOTS; ++i) w[i] /= sum;
        if (a.normalize || whole) inner = warp_sum(WIDE ? c[0] * w[0] + c[SLOTS - 1] * w[SLOTS - 1] : c[0] * w[0]);
        float* r = s_row[warp];
        if (whole) {
#pragma unroll
            for (int j = 0; j < NV; ++j)
                r[j * 32 + lane] =
                    j * 32 + lane < a.E && most > -kInf ? -inner * (expf(v[j] - most) / sum) : 0.0f;
        } else {
#pragma unroll
            for (int j = 0; j < (NV + 3) / 4; ++j)
                if (NV >= 4 || lane < NV * 8)
                    *reinterpret_cast<float4*>(r + (j * 32 + lane) * 4) = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < SLOTS; ++i) {
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
        // Four elements to a lane where the rows allow it.
        if (a.E % 4 == 0 && reinterpret_cast<uintptr_t>(a.grad_logits) % 16 == 0) {
#pragma unroll
            for (int j = 0; j < (NV + 3) / 4; ++j) {
                const int e = (j * 32 + lane) * 4;
                if (e >= a.E) break;
                const float4 q = *reinterpret_cast<const float4*>(r + e);
                if (BF16) {
                    uint2 h;
                    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(h.x) : "f"(q.y), "f"(q.x));
                    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(h.y) : "f"(q.w), "f"(q.z));
                    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.grad_logits) + row + e) = h;
                } else {
                    *reinterpret_cast<float4*>(static_cast<float*>(a.grad_logits) + row + e) = q;
                }
            }
        } else {
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int e = j * 32 + lane;
                if (e >= a.E) break;
                if (BF16) {
                    uint32_t h;
                    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(h) : "f"(0.0f), "f"(r[e]));
                    static_cast<uint16_t*>(a.grad_logits)[row + e] = (uint16_t)h;
                } else {
                    static_cast<float*>(a.grad_logits)[row + e] = r[e];
                }
            }
        }
    }
    griddep_launch_dependents();
}

template <int NV, bool WIDE>
auto kernel_of(const RouteArgs& a, bool backward) -> void (*)(RouteArgs)
{
    if (backward)
        return a.bf16 ? route_backward_kernel<NV, true, WIDE> : route_backward_kernel<NV, false, WIDE>;
    return a.bf16 ? route_kernel<NV, true, WIDE> : route_kernel<NV, false, WIDE>;
}

template <int NV>
cudaError_t launch_nv(const RouteArgs& a, bool backward, const LaunchOpts& o)
{
    const int64_t ctas = (a.T + kRouteThreads / 32 - 1) / (kRouteThreads / 32);
    const dim3 grid((unsigned)ctas);
    auto kernel = kernel_of<NV, false>(a, backward);
    if constexpr (NV > 1)     // 32 experts never have more than 32 slots
        if (a.K > 32) kernel = kernel_of<NV, true>(a, backward);
    return launch_kernel(kernel, grid, kRouteThreads, 0, o, a);
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
