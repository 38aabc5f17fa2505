// route_grouped_backward.cu -- the gradient of the grouped router's weights and
// balance loss with respect to the logits.  A warp owns a token and holds its
// row as route_backward.cu does.
//
// With s the scores, S their sum, p = s / S, a_e = dL coef E c_e / (K n^2), the
// gradient at the scores is
//
//   g_e = (a_e - sum_j p_j a_j) / S
//         + scale (dw_k - sum_j w_j dw_j) / s_K at the chosen (renormalised: w =
//           s / s_K, s_K the chosen scores' sum), or scale dw_k (not)
//
// and at the logits s_e (1 - s_e) g_e for the logistic function, s_e (g_e -
// sum_j s_j g_j) for softmax, whose S is 1.
//
// 4096 x 384 fp32: 5.6 us, 16384 x 128 bf16: 8.1 us: start, latency of a round of
// tokens and end, as there.
#include "route_grouped.cuh"

namespace moe {
namespace {

constexpr int kBackWarps = 8;
constexpr int kBackThreads = kBackWarps * 32;
constexpr int kBackBlocks = 152 * 5;                 // five blocks a multiprocessor

template <int NV, int W, typename L>
__global__ void __launch_bounds__(kBackThreads)
route_grouped_backward_kernel(const L *__restrict__ logits, int T, int E, int K, int softmax, int renorm, float scale,
                              float coef, const int32_t *__restrict__ ids, const int32_t *__restrict__ counts,
                              const int32_t *__restrict__ routed, const float *__restrict__ grad_weights,
                              const float *__restrict__ grad_loss, L *__restrict__ grad)
{
    extern __shared__ float sm[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float *add = sm + (size_t)warp * 32 * NV;            // this warp's row of additions
#pragma unroll
    for (int j = 0; j < NV; ++j) add[j * 32 + lane] = 0.0f;
    __syncwarp();
    pdl_wait();
    pdl_trigger();
    const int k_lanes = 1 << (32 - __clz(K - 1));
    const float n = (float)max(*routed, 1);
    const float unit = grad_loss ? *grad_loss * coef * (float)E / ((float)K * n) / n : 0.0f;
    float a[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int e = lane * NV + j;
        a[j] = e < E && unit != 0.0f ? unit * (float)counts[e] : 0.0f;
    }
    const int stride = gridDim.x * kBackWarps;
    int t = blockIdx.x * kBackWarps + warp, next_id = -1;
    float ahead[NV], next_dw = 0.0f;
    auto fetch = [&](int u) {
        if (u >= T) return;
        load_row<NV, W>(logits + (size_t)u * E, E, lane, ahead);
        if (lane < K) {
            next_id = ids[(size_t)u * K + lane];
            if (grad_weights) next_dw = grad_weights[(size_t)u * K + lane];
        }
    };
    constexpr bool kAhead = NV <= 8;
    if constexpr (kAhead) fetch(t);
    for (; t < T; t += stride) {
        if constexpr (!kAhead) fetch(t);
        float x[NV];
#pragma unroll
        for (int j = 0; j < NV; ++j) x[j] = ahead[j];
        int id = next_id;
        float dw = next_dw * scale;
        if constexpr (kAhead) fetch(t + stride);
        if ((unsigned)id >= (unsigned)E) id = -1;
        float chosen = -INFINITY;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const float v = __shfl_sync(kFullMask, x[j], id / NV & 31);
            if (id >= 0 && id % NV == j) chosen = v;
        }
        if (__ballot_sync(kFullMask, id >= 0) == 0) {    // masked, or nothing open
#pragma unroll
            for (int j = 0; j < NV; ++j) x[j] = -INFINITY;
        }
        // s, and what a logit's gradient multiplies: s (1 - s), or s
        float s[NV], slope[NV], total = 0.0f, dot = 0.0f, w = 0.0f;
        if (softmax) {
            float m = warp_max(lane_max<NV>(x));
            if (!(m > -INFINITY)) m = 0.0f;
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                s[j] = weight_of(x[j], m);
                total += s[j];
            }
            total = warp_sum(total);
            const float inv = total == 0.0f ? 0.0f : __fdividef(1.0f, total);
            if (id >= 0) w = weight_of(chosen, m) * inv;
            total = 1.0f;
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                s[j] *= inv;
                slope[j] = s[j];
                dot += s[j] * a[j];
            }
            dot = warp_sum(dot);
        } else {
            float rest;
            if (id >= 0) w = logistic(chosen, rest);
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                s[j] = logistic(x[j], rest);
                slope[j] = s[j] * rest;
                total += s[j];
                dot += s[j] * a[j];
            }
            total = warp_sum(total);
            total = total == 0.0f ? 0.0f : __fdividef(1.0f, total);
            dot = warp_sum(dot) * total;
        }
        if (id < 0) dw = 0.0f;
        float v = dw;                                    // the weights' gradient at the scores
        if (renorm) {
            const float all = lanes_sum(w, k_lanes);
            const float inv = all == 0.0f ? 0.0f : __fdividef(1.0f, all);
            const float inner = __shfl_sync(kFullMask, lanes_sum(w * inv * dw, k_lanes), 0);
            v = id >= 0 ? (dw - inner) * (all == 0.0f ? 1.0f : inv) : 0.0f;
        }
        if (softmax && !renorm) {
            // sum_j s_j g_j: the loss's part sums to 0, and the renormalised weights' too
            const float inner = lanes_sum(w * v, k_lanes);
            dot += __shfl_sync(kFullMask, inner, 0);
        }
        // one id listed twice: its first lane adds them all, in k order
        const unsigned same = __match_any_sync(kFullMask, id);
        if (__any_sync(kFullMask, id >= 0 && (same & (same - 1)))) {
            float sum = 0.0f;
            for (int k = 0; k < K; ++k) {
                const float other = __shfl_sync(kFullMask, v, k);
                if (same >> k & 1) sum += other;
            }
            v = sum;
            if (lane != __ffs(same) - 1) id = -1;
        }
        if (id >= 0) add[id] = v;
        __syncwarp();
        float y[NV];
#pragma unroll
        for (int j = 0; j < NV; ++j)
            y[j] = slope[j] == 0.0f ? 0.0f : slope[j] * ((a[j] - dot) * total + add[lane * NV + j]);
        L *to = grad + (size_t)t * E + lane * NV;
#pragma unroll
        for (int j = 0; j < NV; j += W)
            if (lane * NV + j < E) store_values<W>(to + j, y + j);
        __syncwarp();
        if (id >= 0) add[id] = 0.0f;
        __syncwarp();
    }
}

template <int NV, int W, typename L>
cudaError_t run_backward(const void *logits, int T, int E, int K, int softmax, int renorm, float scale, float coef,
                         const int32_t *ids, const int32_t *counts, const int32_t *routed, const float *grad_weights,
                         const float *grad_loss, void *grad, cudaStream_t s)
{
    const int need = ceil_div(T, kBackWarps);
    return launch_pdl(route_grouped_backward_kernel<NV, W, L>, dim3(need < kBackBlocks ? need : kBackBlocks),
                      dim3(kBackThreads), (size_t)kBackThreads * NV * 4, s, static_cast<const L *>(logits),
                      T, E, K, softmax, renorm, scale, coef, ids, counts, routed, grad_weights, grad_loss,
                      static_cast<L *>(grad));
}

}  // namespace

cudaError_t launch_route_grouped_backward(const void *logits, int bf16, int T, int E, int K, int softmax, int renorm,
                                          float scale, float coef, const int32_t *ids, const int32_t *counts,
                                          const int32_t *routed, const float *grad_weights, const float *grad_loss,
                                          void *grad, cudaStream_t stream)
{
#define CALL(NV, W, L)                                                                                     \
    run_backward<NV, W, L>(logits, T, E, K, softmax, renorm, scale, coef, ids, counts, routed, grad_weights, \
                           grad_loss, grad, stream)
    MOE_GROUPED_CASES(CALL, grad);
#undef CALL
}

}  // namespace moe
