// route.cu -- from router logits to top-k ids, weights, per-expert counts and
// the balance loss in one pass, and the gradient of the weights and the loss
// with respect to the logits.
//
// With p_t = softmax of row t over its open experts (logit > -inf, token not
// masked), c_e the entries that chose expert e and n the routed tokens:
//
//   loss = coef * E * sum_e (c_e / (K n)) * (sum_t p_te / n)
//
// One warp owns a token: lane l holds logits l, l + 32, ... in registers, so
// the row is read once; its maximum, sum and the K picks are warp reductions.
// Sums of p over tokens stay in registers (fp32) while a warp walks its
// tokens, then are added warp by warp and block by block in a fixed order,
// so a call's results do not depend on timing.
#include "common.cuh"
#include "internal.h"
#include "moe_layout.h"

namespace moe {
namespace {

constexpr int kRouteThreads = 256;
constexpr int kRouteWarps = kRouteThreads / 32;
constexpr int kRouteMaxBlocks = 304;      // two a multiprocessor

__device__ __forceinline__ float load_logit(const float *p) { return __ldg(p); }
__device__ __forceinline__ float load_logit(const __nv_bfloat16 *p) { return __bfloat162float(*p); }
__device__ __forceinline__ void store_logit(float *p, float v) { *p = v; }
__device__ __forceinline__ void store_logit(__nv_bfloat16 *p, float v) { *p = __float2bfloat16_rn(v); }

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFullMask, v, o);
    return v;
}

__device__ __forceinline__ float warp_max(float v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kFullMask, v, o));
    return v;
}

// An unsigned key in the order of the floats (-0 and +0 alike); 0 for -inf
// and NaN, which are never chosen.
__device__ __forceinline__ uint32_t order_key(float x)
{
    if (!(x > -INFINITY)) return 0u;
    const uint32_t u = __float_as_uint(x + 0.0f);
    return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}

// A token's logits in registers (-inf past E and in a masked row), with the
// maximum over its open experts (0 when there is none).
template <int NV, typename L>
__device__ __forceinline__ float load_row(const L *row, int E, bool masked, int lane, float (&x)[NV])
{
    float m = -INFINITY;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int e = j * 32 + lane;
        x[j] = e < E && !masked ? load_logit(row + e) : -INFINITY;
        m = fmaxf(m, x[j]);
    }
    m = warp_max(m);
    return m == -INFINITY ? 0.0f : m;
}

// x becomes exp(x - m), exactly 0 at -inf; returns the row's sum.  A NaN or
// +inf logit makes the sum NaN, and with it every probability of the row.
template <int NV>
__device__ __forceinline__ float exp_row(float (&x)[NV], float m)
{
    float s = 0.0f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        x[j] = x[j] == -INFINITY ? 0.0f : expf(x[j] - m);
        s += x[j];
    }
    return warp_sum(s);
}

template <int NV, typename L>
__global__ void __launch_bounds__(kRouteThreads)
route_kernel(const L *__restrict__ logits, int T, int E, int K, int renorm,
             const uint8_t *__restrict__ mask, int32_t *__restrict__ ids,
             float *__restrict__ weights, float *__restrict__ part_p, int32_t *__restrict__ part_c,
             int32_t *__restrict__ part_n)
{
    extern __shared__ float sm[];
    float *sum_p = sm;                                   // [E]
    int32_t *cnt = reinterpret_cast<int32_t *>(sm + E);  // [E], then the routed tokens
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int e = threadIdx.x; e <= E; e += kRouteThreads) {
        if (e < E) sum_p[e] = 0.0f;
        cnt[e] = 0;
    }
    pdl_wait();
    pdl_trigger();
    __syncthreads();

    float acc[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) acc[j] = 0.0f;

    for (int t = blockIdx.x * kRouteWarps + warp; t < T; t += gridDim.x * kRouteWarps) {
        float x[NV];
        uint32_t key[NV];
        const bool masked = mask && !mask[t];
        const float m = load_row<NV>(logits + (size_t)t * E, E, masked, lane, x);
#pragma unroll
        for (int j = 0; j < NV; ++j) key[j] = order_key(x[j]);
        const float s = exp_row<NV>(x, m);
        const float inv = s == 0.0f ? 0.0f : 1.0f / s;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            x[j] *= inv;
            acc[j] += x[j];
        }
        int my_id = -1;
        float my_w = 0.0f, total = 0.0f;
        for (int k = 0; k < K; ++k) {
            uint32_t best = 0;
            int bj = 0;
            float bp = 0.0f;
#pragma unroll
            for (int j = 0; j < NV; ++j)
                if (key[j] > best) {
                    best = key[j];
                    bj = j;
                    bp = x[j];
                }
            const uint32_t top = __reduce_max_sync(kFullMask, best);
            if (top == 0) break;                         // no open expert is left
            const int e = __reduce_min_sync(kFullMask, best == top ? bj * 32 + lane : INT32_MAX);
            const float p = __shfl_sync(kFullMask, bp, e & 31);
#pragma unroll
            for (int j = 0; j < NV; ++j)
                if (j * 32 + lane == e) key[j] = 0;
            if (lane == k) {
                my_id = e;
                my_w = p;
            }
            total += p;
        }
        if (renorm && total != 0.0f) my_w /= total;
        if (lane < K) {
            ids[(size_t)t * K + lane] = my_id;
            weights[(size_t)t * K + lane] = my_w;
            if (my_id >= 0) atomicAdd(&cnt[my_id], 1);
            if (lane == 0 && my_id >= 0) atomicAdd(&cnt[E], 1);
        }
    }
    for (int w = 0; w < kRouteWarps; ++w) {              // warp by warp: a fixed order
        if (warp == w) {
#pragma unroll
            for (int j = 0; j < NV; ++j)
                if (j * 32 + lane < E) sum_p[j * 32 + lane] += acc[j];
        }
        __syncthreads();
    }
    for (int e = threadIdx.x; e < E; e += kRouteThreads) {
        part_p[(size_t)blockIdx.x * E + e] = sum_p[e];
        part_c[(size_t)blockIdx.x * E + e] = cnt[e];
    }
    if (threadIdx.x == 0) part_n[blockIdx.x] = cnt[E];
}

// The blocks' parts in block order: counts, routed tokens and the loss.
__global__ void __launch_bounds__(1024)
route_finish_kernel(const float *__restrict__ part_p, const int32_t *__restrict__ part_c,
                    const int32_t *__restrict__ part_n, int blocks, int E, int K, float coef,
                    int32_t *__restrict__ counts, int32_t *__restrict__ routed,
                    float *__restrict__ loss)
{
    __shared__ float red[32];
    pdl_wait();
    pdl_trigger();
    const int e = threadIdx.x, lane = e & 31, warp = e >> 5;
    int n = 0;
    for (int b = 0; b < blocks; ++b) n += part_n[b];
    float v = 0.0f;
    if (e < E) {
        float p = 0.0f;
        int c = 0;
        for (int b = 0; b < blocks; ++b) {
            p += part_p[(size_t)b * E + e];
            c += part_c[(size_t)b * E + e];
        }
        counts[e] = c;
        const float fn = (float)max(n, 1);
        v = ((float)c / ((float)K * fn)) * (p / fn);
    }
    v = warp_sum(v);
    if (lane == 0) red[warp] = v;
    __syncthreads();
    if (warp == 0) {
        v = warp_sum(red[lane]);
        if (lane == 0) {
            *loss = coef * (float)E * v;
            *routed = n;
        }
    }
}

// grad_te = p_te (a_e - sum_j p_tj a_j) with a_e = dL coef E c_e / (K n^2),
// plus the weights' part at (renormalised) or around (not) the chosen ids.
template <int NV, typename L>
__global__ void __launch_bounds__(kRouteThreads)
route_backward_kernel(const L *__restrict__ logits, int T, int E, int K, int renorm, float coef,
                      const int32_t *__restrict__ ids, const int32_t *__restrict__ counts,
                      const int32_t *__restrict__ routed, const float *__restrict__ grad_weights,
                      const float *__restrict__ grad_loss, L *__restrict__ grad)
{
    extern __shared__ float sm[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float *add = sm + (size_t)warp * E;                  // this warp's row of additions
    for (int e = lane; e < E; e += 32) add[e] = 0.0f;
    __syncwarp();
    pdl_wait();
    pdl_trigger();
    const float n = (float)max(*routed, 1);
    const float unit = grad_loss ? *grad_loss * coef * (float)E / ((float)K * n) / n : 0.0f;
    float a[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int e = j * 32 + lane;
        a[j] = e < E && unit != 0.0f ? unit * (float)counts[e] : 0.0f;
    }
    for (int t = blockIdx.x * kRouteWarps + warp; t < T; t += gridDim.x * kRouteWarps) {
        const L *row = logits + (size_t)t * E;
        int id = lane < K ? ids[(size_t)t * K + lane] : -1;
        if ((unsigned)id >= (unsigned)E) id = -1;
        const bool masked = __ballot_sync(kFullMask, id >= 0) == 0;
        float x[NV];
        const float m = load_row<NV>(row, E, masked, lane, x);
        const float s = exp_row<NV>(x, m);
        const float inv = s == 0.0f ? 0.0f : 1.0f / s;
        float dot = 0.0f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            x[j] *= inv;
            dot += x[j] * a[j];
        }
        dot = warp_sum(dot);
        float w = 0.0f, dw = 0.0f;
        if (id >= 0) {
            const float l = load_logit(row + id);
            w = l == -INFINITY ? 0.0f : expf(l - m) * inv;
            if (grad_weights) dw = grad_weights[(size_t)t * K + lane];
        }
        if (renorm) {
            const float total = warp_sum(w);
            if (total != 0.0f) w /= total;
        }
        const float inner = warp_sum(w * dw);
        float v = renorm ? w * (dw - inner) : w * dw;
        if (!renorm) dot += inner;
        // one id listed twice: its first lane adds them all, in k order
        const unsigned same = __match_any_sync(kFullMask, id);
        if (__any_sync(kFullMask, id >= 0 && (same & (same - 1)))) {
            float sum = 0.0f;
            for (int k = 0; k < K; ++k) {
                const float o = __shfl_sync(kFullMask, v, k);
                if (same >> k & 1) sum += o;
            }
            v = sum;
            if (lane != __ffs(same) - 1) id = -1;
        }
        if (id >= 0) add[id] = v;
        __syncwarp();
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int e = j * 32 + lane;
            if (e < E) store_logit(grad + (size_t)t * E + e, x[j] * (a[j] - dot) + add[e]);
        }
        __syncwarp();
        if (id >= 0) add[id] = 0.0f;
        __syncwarp();
    }
}

int route_blocks(int T)
{
    const int need = ceil_div(T, kRouteWarps);
    return need < 1 ? 1 : need < kRouteMaxBlocks ? need : kRouteMaxBlocks;
}

template <int NV, typename L>
cudaError_t run_forward(const void *logits, int T, int E, int K, int renorm, float coef,
                        const uint8_t *mask, int32_t *ids, float *weights, int32_t *counts,
                        int32_t *routed, float *loss, void *workspace, cudaStream_t s)
{
    const int blocks = route_blocks(T);
    float *part_p = static_cast<float *>(workspace);
    int32_t *part_c = reinterpret_cast<int32_t *>(part_p + (size_t)blocks * E);
    int32_t *part_n = part_c + (size_t)blocks * E;
    cudaError_t e = launch_pdl(route_kernel<NV, L>, dim3(blocks), dim3(kRouteThreads),
                               (2 * (size_t)E + 1) * 4, s, static_cast<const L *>(logits), T, E,
                               K, renorm, mask, ids, weights, part_p, part_c, part_n);
    if (e != cudaSuccess) return e;
    return launch_pdl(route_finish_kernel, dim3(1), dim3(1024), 0, s, part_p, part_c, part_n,
                      blocks, E, K, coef, counts, routed, loss);
}

template <int NV, typename L>
cudaError_t run_backward(const void *logits, int T, int E, int K, int renorm, float coef,
                         const int32_t *ids, const int32_t *counts, const int32_t *routed,
                         const float *grad_weights, const float *grad_loss, void *grad,
                         cudaStream_t s)
{
    return launch_pdl(route_backward_kernel<NV, L>, dim3(route_blocks(T)), dim3(kRouteThreads),
                      (size_t)kRouteWarps * E * 4, s, static_cast<const L *>(logits), T, E, K,
                      renorm, coef, ids, counts, routed, grad_weights, grad_loss,
                      static_cast<L *>(grad));
}

}  // namespace

size_t route_workspace_bytes(int T, int E)
{
    const size_t blocks = route_blocks(T);
    return (blocks * ((size_t)E * 8 + 4) + 255) / 256 * 256;
}

// Values a lane holds: the smallest of these that covers E.
#define MOE_ROUTE_CASES(CALL)                                                   \
    if (bf16) {                                                                 \
        if (E <= 64) return CALL(2, __nv_bfloat16);                             \
        if (E <= 128) return CALL(4, __nv_bfloat16);                            \
        if (E <= 256) return CALL(8, __nv_bfloat16);                            \
        if (E <= 512) return CALL(16, __nv_bfloat16);                           \
        return CALL(32, __nv_bfloat16);                                         \
    }                                                                           \
    if (E <= 64) return CALL(2, float);                                         \
    if (E <= 128) return CALL(4, float);                                        \
    if (E <= 256) return CALL(8, float);                                        \
    if (E <= 512) return CALL(16, float);                                       \
    return CALL(32, float);

cudaError_t launch_route(const void *logits, int bf16, int T, int E, int K, int renorm, float coef,
                         const uint8_t *mask, int32_t *ids, float *weights, int32_t *counts,
                         int32_t *routed, float *loss, void *workspace, cudaStream_t stream)
{
#define CALL(NV, L)                                                                           \
    run_forward<NV, L>(logits, T, E, K, renorm, coef, mask, ids, weights, counts, routed, loss, \
                       workspace, stream)
    MOE_ROUTE_CASES(CALL)
#undef CALL
}

cudaError_t launch_route_backward(const void *logits, int bf16, int T, int E, int K, int renorm,
                                  float coef, const int32_t *ids, const int32_t *counts,
                                  const int32_t *routed, const float *grad_weights,
                                  const float *grad_loss, void *grad, cudaStream_t stream)
{
#define CALL(NV, L)                                                                         \
    run_backward<NV, L>(logits, T, E, K, renorm, coef, ids, counts, routed, grad_weights,   \
                        grad_loss, grad, stream)
    MOE_ROUTE_CASES(CALL)
#undef CALL
}

}  // namespace moe
