// route.cu -- from router logits to top-k ids, weights, per-expert counts and
// the balance loss in one pass.
//
// With p_t = softmax of row t over its open experts (logit not -inf, token not
// masked), c_e the entries that chose expert e and n the routed tokens:
//
//   loss = coef * E * sum_e (c_e / (K n)) * (sum_t p_te / n)
//
// One warp owns a token: lane l holds the NV logits from l * NV, so the row is
// read once, in 16-byte loads where its alignment allows, and a lower lane
// always has lower expert numbers: among equal logits the lowest lane, and in
// it the lowest place, is the lowest expert.  The maximum and each pick are
// one warp-wide maximum over the lanes' next largest: a lane keeps its logits
// sorted as well and steps on by predicated moves when its own is picked; which
// expert a pick was is looked up for all K at once, after the last.  Sums of p
// over tokens stay in registers (fp32) while a warp walks its tokens, are added
// warp by warp in a block, block by block in a cluster (distributed shared
// memory) and cluster by cluster at the end, always in that order, so a call's
// results do not depend on timing.
//
// Bound by latency, of two dependent launches first: 16384 x 128 fp32 takes 14.1
// us, of which the loop 4.8, the sums 1.5, the finishing kernel 2 and the two
// launches the rest; one token of 256 experts: 3.5 us.  In the loop the issue
// slots weigh most (338 instructions a token at E = 128, K = 8, half of them the
// picks; 61 % of the slots of active cycles, a third of the kernel's), the bytes
// least.  Sixteen warps a block, two blocks a multiprocessor (three: 17.7 against
// 16.6 us then).
#include "route_common.cuh"
#include "tensor.cuh"

namespace moe {
namespace {

constexpr int kRouteWarps = 16;
constexpr int kRouteThreads = kRouteWarps * 32;
constexpr int kRouteCluster = 8;                    // blocks that add their sums up together
constexpr int kRouteClusters = 38;                  // at most: two blocks a multiprocessor
constexpr int kSingleCluster = 8;                   // blocks of the form that needs one launch

// The call's last sums, thread e for expert e: p and c are expert e's totals.
__device__ __forceinline__ float loss_term(float p, int c, int n, int K)
{
    const float fn = (float)max(n, 1);
    return ((float)c / ((float)K * fn)) * (p / fn);
}

struct RouteOut {
    int32_t *counts, *routed;
    float *loss;
    float coef;
};

// KT > 0: K is KT, and the picks are unrolled.
// SINGLE: the grid is one cluster, which writes the results; otherwise every
// cluster writes its totals to part[cluster]: E probability sums, E counts and
// the routed tokens.
template <int NV, int W, int KT, bool SINGLE, typename L>
__global__ void __launch_bounds__(kRouteThreads, NV > 16 ? 1 : 2)
route_kernel(const L *__restrict__ logits, int T, int E, int any_k, int renorm,
             const uint8_t *__restrict__ mask, int32_t *__restrict__ ids,
             float *__restrict__ weights, uint32_t *__restrict__ part, RouteOut o)
{
    const int K = KT > 0 ? KT : any_k;
    extern __shared__ float sm[];
    float *const sums = sm;                              // [kRouteWarps][E]
    int32_t *const cnt = reinterpret_cast<int32_t *>(sm + (size_t)kRouteWarps * E);     // [E] and the routed tokens
    uint32_t *const inbox = reinterpret_cast<uint32_t *>(cnt + E + 1);  // [blocks][2 share + 1], see below
    __shared__ float warp_terms[kRouteWarps];
    __shared__ float terms[kSingleCluster];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
    for (int e = threadIdx.x; e <= E; e += kRouteThreads) cnt[e] = 0;
    pdl_wait();
    pdl_trigger();
    __syncthreads();

    const int k_lanes = 1 << (32 - __clz(K - 1));        // K, rounded up to a power of two
    int routed = 0;                                      // tokens with a first pick (lane 0)
    bool bad = false;                                    // a token's probabilities are NaN
    float acc[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) acc[j] = 0.0f;

    // The next token's row is on its way while one is worked on, where a lane
    // has the registers for it.
    constexpr bool kAhead = NV <= 8;
    const int stride = gridDim.x * kRouteWarps;
    int t = blockIdx.x * kRouteWarps + warp;
    float ahead[NV];
    uint8_t open = 1;
    auto fetch = [&](int u) {
        if (u >= T) return;
        load_row<NV, W>(logits + (size_t)u * E, E, lane, ahead);
        if (mask) open = mask[u];
    };
    if constexpr (kAhead) fetch(t);
    for (; t < T; t += stride) {
        if constexpr (!kAhead) fetch(t);
        float x[NV];
#pragma unroll
        for (int j = 0; j < NV; ++j) x[j] = ahead[j];
        const bool masked = !open;
        if constexpr (kAhead) fetch(t + stride);
        if (masked) {
#pragma unroll
            for (int j = 0; j < NV; ++j) x[j] = -INFINITY;
        }
        float m = warp_max(lane_max<NV>(x));
        if (!(m > -INFINITY)) m = 0.0f;
        float p[NV], s = 0.0f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            p[j] = weight_of(x[j], m);
            s += p[j];
        }
        s = warp_sum(s);
        bad |= s != s;
        const float inv = s == 0.0f ? 0.0f : __fdividef(1.0f, s);
#pragma unroll
        for (int j = 0; j < NV; ++j) acc[j] += p[j] * inv;

        // Pick number `lane`: its logit, and the lane that holds it.  Past the
        // last open number the picks are -inf, and not taken below.
        float mine = -INFINITY;
        int from = 0;
        float next[NV];
#pragma unroll
        for (int j = 0; j < NV; ++j) next[j] = x[j] > -INFINITY ? x[j] + 0.0f : -INFINITY;  // no NaN, one zero
        if constexpr (NV <= 16) sort_values<NV>(next);
        float best = NV <= 16 ? next[0] : lane_max<NV>(next);
        auto pick = [&](int k) {
            const float top = warp_max(best);
            const int owner = __ffs(__ballot_sync(kFullMask, best == top)) - 1;
            if (lane == k) {
                mine = top;
                from = owner;
            }
            if constexpr (NV <= 16) {
#pragma unroll
                for (int j = 0; j + 1 < NV; ++j) next[j] = lane == owner ? next[j + 1] : next[j];
                next[NV - 1] = lane == owner ? -INFINITY : next[NV - 1];
                best = next[0];
            } else if (lane == owner) {
                int at = 0;
#pragma unroll
                for (int j = NV - 1; j >= 0; --j)
                    if (next[j] == top) at = j;
#pragma unroll
                for (int j = 0; j < NV; ++j)
                    if (j == at) next[j] = -INFINITY;
                best = lane_max<NV>(next);
            }
        };
        if constexpr (KT > 0) {
#pragma unroll
            for (int k = 0; k < KT; ++k) pick(k);
        } else {
            for (int k = 0; k < K; ++k) pick(k);
        }
        // Its place among the owner's logits: equal ones were picked in order.
        const unsigned alike = __match_any_sync(kFullMask, __float_as_int(mine)) & __match_any_sync(kFullMask, from);
        int before = __popc(alike & ((1u << lane) - 1)), place = 0;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const bool same = __shfl_sync(kFullMask, x[j], from) == mine;
            if (same && before == 0) place = j;
            before -= same;
        }
        const bool taken = lane < K && mine > -INFINITY;
        float w = taken ? weight_of(mine, m) * inv : 0.0f;
        if (renorm) {
            const float total = lanes_sum(w, k_lanes);
            if (total != 0.0f) w = __fdividef(w, total);
        }
        const int id = taken ? from * NV + place : -1;
        if (lane < K) {
            ids[(size_t)t * K + lane] = id;
            weights[(size_t)t * K + lane] = w;
        }
        if (taken) atomicAdd(&cnt[id], 1);
        routed += taken;
    }
#pragma unroll
    for (int j = 0; j < NV; ++j)
        if (lane * NV + j < E) sums[warp * E + lane * NV + j] = acc[j];
    // NaN logits are behind every number: where a token's numbers were fewer than
    // K, its NaN ones take the picks that are left, lowest index first, with NaN
    // for weights.  Rare, so after the loop, whose registers are all in use.
    if (bad)
        for (t = blockIdx.x * kRouteWarps + warp; t < T; t += stride) {
            if (mask && !mask[t]) continue;
            int32_t *const id = ids + (size_t)t * K;
            float *const w = weights + (size_t)t * K;
            __syncwarp();
            const int numbers = __popc(__ballot_sync(kFullMask, lane < K && id[lane] >= 0));
            int picks = numbers;
            for (int e0 = 0; e0 < E && picks < K; e0 += 32) {
                const float x = e0 + lane < E ? to_float(logits[(size_t)t * E + e0 + lane]) : 0.0f;
                const unsigned nans = __ballot_sync(kFullMask, x != x);
                const int k = picks + __popc(nans & ((1u << lane) - 1));
                if (x != x && k < K) {
                    id[k] = e0 + lane;
                    w[k] = x;
                    atomicAdd(&cnt[e0 + lane], 1);
                }
                picks += __popc(nans);
            }
            if (lane < K && lane >= picks) w[lane] = 0.0f;      // no expert, so no weight
            routed += numbers == 0 && picks > 0;
        }
    if (lane == 0) atomicAdd(&cnt[E], routed);
    // Expert e is added up by block e % blocks of the cluster: every block puts
    // its sums, its counts and its routed tokens in that block's inbox.
    const int rank = (int)cluster_rank(), blocks = SINGLE ? (int)gridDim.x : kRouteCluster;
    const int share = ceil_div(E, blocks), box = 2 * share + 1;
    asm volatile("barrier.cluster.wait.aligned;" ::: "memory");      // the others have started
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += kRouteThreads) {
        float v = sums[e];
#pragma unroll
        for (int w = 1; w < kRouteWarps; ++w) v += sums[w * E + e];
        const uint32_t to = cluster_addr(smem_addr(inbox + rank * box + e / blocks), e % blocks);
        st_cluster_u32(to, __float_as_uint(v));
        st_cluster_u32(to + 4 * share, (uint32_t)cnt[e]);
    }
    if (threadIdx.x < blocks) st_cluster_u32(cluster_addr(smem_addr(inbox + rank * box + 2 * share), threadIdx.x), (uint32_t)cnt[E]);
    cluster_sync_all();
    int n = 0;
    for (int b = 0; b < blocks; ++b) n += (int)inbox[b * box + 2 * share];
    float term = 0.0f;
    for (int i = threadIdx.x; i < share; i += kRouteThreads) {
        const int e = i * blocks + rank;
        if (e >= E) break;
        float v = 0.0f;
        int c = 0;
        for (int b = 0; b < blocks; ++b) {
            v += __uint_as_float(inbox[b * box + i]);
            c += (int)inbox[b * box + share + i];
        }
        if constexpr (SINGLE) {
            o.counts[e] = c;
            term += loss_term(v, c, n, K);
        } else {
            uint32_t *q = part + (size_t)(blockIdx.x / kRouteCluster) * (2 * E + 1);
            q[e] = __float_as_uint(v);
            q[E + e] = (uint32_t)c;
        }
    }
    if constexpr (SINGLE) {
        term = warp_sum(term);
        if (lane == 0) warp_terms[warp] = term;
        __syncthreads();
        if (threadIdx.x == 0) {
            float v = 0.0f;
            for (int w = 0; w < kRouteWarps; ++w) v += warp_terms[w];
            st_cluster_u32(cluster_addr(smem_addr(&terms[rank]), 0), __float_as_uint(v));
        }
        cluster_sync_all();
        if (rank == 0 && threadIdx.x == 0) {
            float v = 0.0f;
            for (int b = 0; b < blocks; ++b) v += terms[b];
            *o.loss = o.coef * (float)E * v;
            *o.routed = n;
        }
    } else if (rank == 0 && threadIdx.x == 0) {
        part[(size_t)(blockIdx.x / kRouteCluster) * (2 * E + 1) + 2 * E] = (uint32_t)n;
    }
}

// The clusters' totals in order: counts, routed tokens and the loss.  `lanes`
// threads (E rounded up to a warp) take each a share of the clusters, whose
// sums are then added in order.
__global__ void __launch_bounds__(1024)
route_finish_kernel(const uint32_t *__restrict__ part, int clusters, int E, int K, int lanes, RouteOut o)
{
    __shared__ float share_p[1024];
    __shared__ int32_t share_c[1024];
    __shared__ float red[32];
    const int groups = blockDim.x / lanes, g = threadIdx.x / lanes, e = threadIdx.x - g * lanes;
    const int each = ceil_div(clusters, groups), lane = threadIdx.x & 31;
    pdl_wait();
    pdl_trigger();
    const size_t row = 2 * (size_t)E + 1;
    static_assert(kRouteClusters <= 64);
    int n = lane < clusters ? (int)part[lane * row + 2 * E] : 0;
    if (lane + 32 < clusters) n += (int)part[(lane + 32) * row + 2 * E];
    float p = 0.0f;
    int c = 0;
    if (e < E) {
        const int last = min(clusters, (g + 1) * each);
        for (int b0 = g * each; b0 < last; b0 += 8) {
            uint32_t vp[8], vc[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                vp[j] = b0 + j < last ? part[(b0 + j) * row + e] : 0u;
                vc[j] = b0 + j < last ? part[(b0 + j) * row + E + e] : 0u;
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                p += __uint_as_float(vp[j]);
                c += (int)vc[j];
            }
        }
    }
    share_p[threadIdx.x] = p;
    share_c[threadIdx.x] = c;
    __syncthreads();
    n = __reduce_add_sync(kFullMask, n);
    float v = 0.0f;
    if (threadIdx.x < E) {
        for (int i = 1; i < groups; ++i) {
            p += share_p[i * lanes + e];
            c += share_c[i * lanes + e];
        }
        o.counts[e] = c;
        v = loss_term(p, c, n, K);
    }
    v = warp_sum(v);
    if (lane == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    if (threadIdx.x < 32) {
        v = warp_sum(threadIdx.x < blockDim.x / 32 ? red[threadIdx.x] : 0.0f);
        if (threadIdx.x == 0) {
            *o.loss = o.coef * (float)E * v;
            *o.routed = n;
        }
    }
}

// Blocks of one cluster that writes the results itself, or 0 where two
// launches over all multiprocessors are quicker: by tokens a warp, fewer the
// wider the rows (one and two launches, a call among others: E = 128, 512
// tokens 6.7 and 7.9 us; E = 256, 256 tokens 6.1 and 8.7, 512 tokens 8.9 and
// 7.7; E = 1000, 256 tokens 23.3 and 20.4).
int single_blocks(int T, int E)
{
    const int need = ceil_div(T, kRouteWarps);
    for (int b = 1; b <= kSingleCluster; b *= 2)
        if (need <= b) return b;
    const int tokens = E <= 128 ? 4 : E <= 512 ? 2 : 1;
    return need <= tokens * kSingleCluster ? kSingleCluster : 0;
}

int route_clusters(int T)
{
    const int need = ceil_div(ceil_div(T, kRouteWarps), kRouteCluster);
    return need < kRouteClusters ? need : kRouteClusters;
}

template <int NV, int W, typename L>
cudaError_t run_forward(const void *logits, int T, int E, int K, int renorm, float coef,
                        const uint8_t *mask, int32_t *ids, float *weights, int32_t *counts,
                        int32_t *routed, float *loss, void *workspace, cudaStream_t s)
{
    // sums, counts, and an inbox of at most E + kSingleCluster experts' pairs
    const size_t smem = ((size_t)(kRouteWarps + 1) * E + 1 + 2 * (E + kSingleCluster) + kSingleCluster) * 4;
    const RouteOut o{counts, routed, loss, coef};
    const int single = single_blocks(T, E);
    // K = 8, the models' usual, has its own form with the picks unrolled (8192
    // tokens, unrolled and not: E = 64 9.8 and 10.9 us, 128 10.1 and 11.1, 256 13.5
    // and 14.4, 384 16.4 and 17.5, 512 25.6 and 27.8, 1000 68.1 and 69.8; bf16 gains
    // as much); rows read value by value not
    constexpr int KT = W > 1 ? 8 : 0;
    auto *const kernel = K == KT ? single ? route_kernel<NV, W, KT, true, L> : route_kernel<NV, W, KT, false, L>
                                : single ? route_kernel<NV, W, 0, true, L> : route_kernel<NV, W, 0, false, L>;
    if (smem > 40 << 10) {
        const cudaError_t e = allow_dynamic_smem(reinterpret_cast<const void *>(kernel), smem);
        if (e != cudaSuccess) return e;
    }
    const int blocks = single ? single : route_clusters(T) * kRouteCluster;
    uint32_t *part = static_cast<uint32_t *>(workspace);
    cudaError_t e = launch_pdl_clusters(kernel, dim3(blocks), dim3(kRouteThreads), smem, s,
                                        single ? single : kRouteCluster, static_cast<const L *>(logits),
                                        T, E, K, renorm, mask, ids, weights, part, o);
    if (e != cudaSuccess || single) return e;
    const int lanes = ceil_div(E, 32) * 32;
    return launch_pdl(route_finish_kernel, dim3(1), dim3(1024 / lanes * lanes), 0, s, part,
                      blocks / kRouteCluster, E, K, lanes, o);
}

}  // namespace

size_t route_workspace_bytes(int T, int E)
{
    const size_t clusters = single_blocks(T, E) ? 1 : route_clusters(T);
    return (clusters * (2 * (size_t)E + 1) * 4 + 255) / 256 * 256;
}

cudaError_t launch_route(const void *logits, int bf16, int T, int E, int K, int renorm, float coef,
                         const uint8_t *mask, int32_t *ids, float *weights, int32_t *counts,
                         int32_t *routed, float *loss, void *workspace, cudaStream_t stream)
{
#define CALL(NV, W, L)                                                                       \
    run_forward<NV, W, L>(logits, T, E, K, renorm, coef, mask, ids, weights, counts, routed, \
                            loss, workspace, stream)
    MOE_ROUTE_CASES(CALL, logits);
#undef CALL
}

}  // namespace moe
