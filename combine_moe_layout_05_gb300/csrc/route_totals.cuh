// route_totals.cuh -- the second half of the router's kernels: the sums of
// probabilities and the counts that each warp and block has gathered are added
// up in a cluster of blocks (distributed shared memory), cluster by cluster in
// a finishing kernel where there are more, always in that order, and give the
// counts, the routed tokens and the balance loss.
#pragma once

#include "route_common.cuh"
#include "tensor.cuh"

namespace moe {
namespace {

constexpr int kRouteCluster = 8;                    // blocks that add their sums up together
constexpr int kMostClusters = 96;                   // that the finishing kernel adds up
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

// Shared memory: sums, counts, and an inbox of at most E + kSingleCluster
// experts' pairs.
template <int WARPS>
size_t route_smem(int E)
{
    return ((size_t)(WARPS + 1) * E + 1 + 2 * (E + kSingleCluster) + kSingleCluster) * 4;
}

// For a whole block: sums [WARPS][pitch] each warp's, cnt [E] and the routed tokens
// the block's.  SINGLE: the grid is one cluster, which writes the results;
// otherwise every cluster writes its totals to part[cluster]: E probability
// sums, E counts and the routed tokens.  Ends the cluster barrier that the
// kernel began (arrive) when it started.
template <int WARPS, bool SINGLE>
__device__ __forceinline__ void route_totals(const float *sums, int pitch, const int32_t *cnt, uint32_t *inbox, int E, int K,
                                             uint32_t *part, const RouteOut &o)
{
    constexpr int THREADS = WARPS * 32;
    __shared__ float warp_terms[WARPS];
    __shared__ float terms[kSingleCluster];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    // Expert e is added up by block e % blocks of the cluster: every block puts
    // its sums, its counts and its routed tokens in that block's inbox.
    const int rank = (int)cluster_rank(), blocks = SINGLE ? (int)gridDim.x : kRouteCluster;
    const int share = ceil_div(E, blocks), box = 2 * share + 1;
    asm volatile("barrier.cluster.wait.aligned;" ::: "memory");      // the others have started
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += THREADS) {
        float v = sums[e];
#pragma unroll
        for (int w = 1; w < WARPS; ++w) v += sums[w * pitch + e];
        const uint32_t to = cluster_addr(smem_addr(inbox + rank * box + e / blocks), e % blocks);
        st_cluster_u32(to, __float_as_uint(v));
        st_cluster_u32(to + 4 * share, (uint32_t)cnt[e]);
    }
    if (threadIdx.x < blocks) st_cluster_u32(cluster_addr(smem_addr(inbox + rank * box + 2 * share), threadIdx.x), (uint32_t)cnt[E]);
    cluster_sync_all();
    int n = 0;
    for (int b = 0; b < blocks; ++b) n += (int)inbox[b * box + 2 * share];
    float term = 0.0f;
    for (int i = threadIdx.x; i < share; i += THREADS) {
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
            for (int w = 0; w < WARPS; ++w) v += warp_terms[w];
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
    static_assert(kMostClusters <= 96);
    int n = lane < clusters ? (int)part[lane * row + 2 * E] : 0;
    if (lane + 32 < clusters) n += (int)part[(lane + 32) * row + 2 * E];
    if (lane + 64 < clusters) n += (int)part[(lane + 64) * row + 2 * E];
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

cudaError_t launch_route_finish(const uint32_t *part, int clusters, int E, int K, const RouteOut &o, cudaStream_t s)
{
    const int lanes = ceil_div(E, 32) * 32;
    return launch_pdl(route_finish_kernel, dim3(1), dim3(1024 / lanes * lanes), 0, s, part, clusters, E, K, lanes, o);
}

// Blocks of one cluster that writes the results itself, or 0 where two
// launches over all multiprocessors are quicker: by tokens a warp, fewer the
// wider the rows (moe_route, 16 warps a block, one and two launches, a call among
// others: E = 128, 512 tokens 6.7 and 7.9 us; E = 256, 256 tokens 6.1 and 8.7, 512
// tokens 8.9 and 7.7; E = 1000, 256 tokens 23.3 and 20.4).  moe_route_grouped has 8
// warps and takes longer for a token, so its border is earlier than this rule's
// (one and two launches, bias and groups: E = 128, 64 tokens 5.1 and 6.8 us, 128
// 7.0 and 6.8, 256 10.5 and 6.8; E = 256, 64 tokens 6.0 and 7.5, 128 8.2 and 7.6;
// E = 512, 64 tokens 8.1 and 9.7, 128 11.9 and 10.0; E = 1000, 64 tokens 16.3 and
// 18.2, where the rule ends): between 65 tokens and the rule's end it costs up to
// 3.7 us.
template <int WARPS>
int single_blocks(int T, int E)
{
    const int need = ceil_div(T, WARPS);
    for (int b = 1; b <= kSingleCluster; b *= 2)
        if (need <= b) return b;
    const int tokens = E <= 128 ? 4 : E <= 512 ? 2 : 1;
    return need <= tokens * kSingleCluster ? kSingleCluster : 0;
}

// PER_SM: blocks a multiprocessor.
template <int WARPS, int PER_SM>
int route_clusters(int T)
{
    constexpr int most = 152 * PER_SM / kRouteCluster;
    static_assert(most <= kMostClusters);
    const int need = ceil_div(ceil_div(T, WARPS), kRouteCluster);
    return need < most ? need : most;
}

template <int WARPS, int PER_SM>
size_t totals_workspace_bytes(int T, int E)
{
    const size_t clusters = single_blocks<WARPS>(T, E) ? 1 : route_clusters<WARPS, PER_SM>(T);
    return (clusters * (2 * (size_t)E + 1) * 4 + 255) / 256 * 256;
}

}  // namespace
}  // namespace moe
