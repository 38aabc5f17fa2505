// route_backward.cu -- the gradient of the router's weights and balance loss
// with respect to the logits.  A warp owns a token and holds its row as the
// forward kernel does (route_common.cuh).
#include "route_common.cuh"

namespace moe {
namespace {

constexpr int kBackWarps = 8;
constexpr int kBackThreads = kBackWarps * 32;
constexpr int kBackBlocks = 152 * 5;                 // five blocks a multiprocessor

// grad_te = p_te (a_e - sum_j p_tj a_j) with a_e = dL coef E c_e / (K n^2),
// plus the weights' part at (renormalised) or around (not) the chosen ids.
// The row is read once and its softmax computed again.  4096 x 384 fp32: 5.0
// us on the device (2.5 TB/s), 16384 x 128 bf16: 7.2 us.  526 and 282
// instructions a token take 51 and 70 % of the issue slots of active cycles, 24
// and 40 % of the kernel's: start, latency of a round and end are the rest.
template <int NV, int W, typename L>
__global__ void __launch_bounds__(kBackThreads)
route_backward_kernel(const L *__restrict__ logits, int T, int E, int K, int renorm, float coef,
                      const int32_t *__restrict__ ids, const int32_t *__restrict__ counts,
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
    auto fetch = [&](int u) {                            // as in route_kernel
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
        float dw = next_dw;
        if constexpr (kAhead) fetch(t + stride);
        if ((unsigned)id >= (unsigned)E) id = -1;
        float chosen = -INFINITY;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const float v = __shfl_sync(kFullMask, x[j], id / NV & 31);
            if (id >= 0 && id % NV == j) chosen = v;
        }
        const bool masked = __ballot_sync(kFullMask, id >= 0) == 0;
        if (masked) {
#pragma unroll
            for (int j = 0; j < NV; ++j) x[j] = -INFINITY;
        }
        float m = warp_max(lane_max<NV>(x));
        if (!(m > -INFINITY)) m = 0.0f;
        float s = 0.0f, dot = 0.0f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            x[j] = weight_of(x[j], m);
            s += x[j];
            dot += x[j] * a[j];
        }
        s = warp_sum(s);
        const float inv = s == 0.0f ? 0.0f : __fdividef(1.0f, s);
        dot = warp_sum(dot) * inv;
        float w = id >= 0 ? weight_of(chosen, m) * inv : 0.0f;
        if (id < 0) dw = 0.0f;
        if (renorm) {
            const float total = lanes_sum(w, k_lanes);
            if (total != 0.0f) w = __fdividef(w, total);
        }
        float inner = lanes_sum(w * dw, k_lanes);
        inner = __shfl_sync(kFullMask, inner, 0);
        float v = renorm ? w * (dw - inner) : w * dw;
        if (!renorm) dot += inner;
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
        for (int j = 0; j < NV; ++j) y[j] = x[j] * inv * (a[j] - dot) + add[lane * NV + j];
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
cudaError_t run_backward(const void *logits, int T, int E, int K, int renorm, float coef,
                         const int32_t *ids, const int32_t *counts, const int32_t *routed,
                         const float *grad_weights, const float *grad_loss, void *grad,
                         cudaStream_t s)
{
    const int need = ceil_div(T, kBackWarps);
    return launch_pdl(route_backward_kernel<NV, W, L>, dim3(need < kBackBlocks ? need : kBackBlocks),
                      dim3(kBackThreads), (size_t)kBackThreads * NV * 4, s, static_cast<const L *>(logits),
                      T, E, K, renorm, coef, ids, counts, routed, grad_weights, grad_loss,
                      static_cast<L *>(grad));
}

}  // namespace

cudaError_t launch_route_backward(const void *logits, int bf16, int T, int E, int K, int renorm,
                                  float coef, const int32_t *ids, const int32_t *counts,
                                  const int32_t *routed, const float *grad_weights,
                                  const float *grad_loss, void *grad, cudaStream_t stream)
{
#define CALL(NV, W, L)                                                                          \
    run_backward<NV, W, L>(logits, T, E, K, renorm, coef, ids, counts, routed, grad_weights,    \
                             grad_loss, grad, stream)
    MOE_ROUTE_CASES(CALL, grad);
#undef CALL
}

}  // namespace moe
