// route_grouped.cu -- from router logits to top-k ids, weights, counts and the
// balance loss, with softmax or sigmoid scores, a bias that takes part in the
// choice alone, and groups of experts of which the best few stay.
//
// A warp owns a token and holds its row as route.cu does; the picks, the sums
// and their order are that kernel's too.  What differs is that the choice goes
// by computed values, c = s + bias, where route.cu's goes by the logits
// themselves: fp32 scores are off by a few units in the last place, and two
// experts nearer than that could come out in the wrong order (of 16384 tokens
// with 256 experts some 20 have such a pair).  So every choice is checked
// against a bound on its error, and a token that fails is chosen again
// (choose_exactly): values in 64 bits, of those experts alone that fp32 cannot
// tell apart.  Without a bias the picks go by logits, and only the groups'
// values need the check.
#include "route_grouped.cuh"
#include "route_totals.cuh"

#include <cfloat>

namespace moe {
namespace {

constexpr int kGroupedWarps = 8;
constexpr int kGroupedThreads = kGroupedWarps * 32;
constexpr int kGroupedPerSm = 3;                     // blocks a multiprocessor
constexpr float kUnit = 5.9604645e-8f;               // 2^-24

struct Rules {
    const float *bias;                               // [E] or null
    int softmax, groups, top_groups, group_top, renorm;
    float scale;
};

// A value to choose by: NaN is behind every number.
__device__ __forceinline__ float rankable(float c) { return c >= -FLT_MAX ? c : -FLT_MAX; }
__device__ __forceinline__ double rankable(double c) { return c >= -(double)FLT_MAX ? c : -(double)FLT_MAX; }

template <typename T>
__device__ __forceinline__ T warp_max_of(T v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const T w = __shfl_xor_sync(kFullMask, v, o);
        v = w > v ? w : v;
    }
    return v;
}

// The two largest of a warp's pairs a >= b (each lane's), over `lanes` lanes.
template <typename T>
__device__ __forceinline__ void top_two(T &a, T &b, int lanes)
{
    for (int o = lanes >> 1; o > 0; o >>= 1) {
        const T a2 = __shfl_xor_sync(kFullMask, a, o), b2 = __shfl_xor_sync(kFullMask, b, o);
        const T low = a2 < a ? a2 : a, second = b2 > b ? b2 : b;
        a = a2 > a ? a2 : a;
        b = low > second ? low : second;
    }
}

template <typename T>
__device__ __forceinline__ void insert(T v, T &a, T &b)
{
    if (v > a) {
        b = a;
        a = v;
    } else if (v > b) {
        b = v;
    }
}

// A group's value from its largest two (-inf: no open expert).
template <typename T>
__device__ __forceinline__ T group_value(T a, T b, int group_top)
{
    return group_top == 2 && b > -INFINITY ? a + b : a;
}

// Which groups stay, bit g for group g: lane g has value g (-inf past the last).
template <typename T>
__device__ __forceinline__ unsigned best_groups(T value, int groups, int lane, int top)
{
    int before = 0;
    for (int g = 0; g < groups; ++g) {
        const T v = __shfl_sync(kFullMask, value, g);
        before += v > value || (v == value && g < lane);
    }
    return __ballot_sync(kFullMask, lane < groups && before < top);
}

// What a row's scores are made with: softmax's maximum and the reciprocal of its sum.
struct Row {
    float m, inv;
};

__device__ __forceinline__ float score_of(float x, const Rules &r, const Row &row)
{
    float rest;
    return r.softmax ? weight_of(x, row.m) * row.inv : logistic(x, rest);
}

// A bound on the error of a score plus bias c: (|z| + 8) 2^-24 of the score for
// the logistic function, (|z| + 64) 2^-24 for softmax (z the distance to the
// maximum; the sum's share is below 7 + 4 + its 37 additions, the quotient's 5),
// and the addition's rounding.
__device__ __forceinline__ float error_of(float x, float s, float c, const Rules &r, const Row &row)
{
    const float z = r.softmax ? row.m - x : fabsf(x);
    return kUnit * ((s > 0.0f ? s * (z + (r.softmax ? 64.0f : 8.0f)) : 0.0f) + fabsf(c));
}

// The token's choice again, for a warp, where fp32 leaves it open.  value: lane
// g's group value.  room_g, room: differences of group values and of keys that
// fp32 cannot tell from 0.  scratch: E words of shared memory of the warp's own.
// Writes ids[0 .. K).
template <typename L>
__device__ __noinline__ void choose_exactly(const L *logits, int E, int K, const Rules r, const Row row, float value,
                                            float room_g, float room, float *scratch, int32_t *ids)
{
    const int lane = threadIdx.x & 31, size = E / r.groups;
    const bool limited = r.top_groups < r.groups;
    double sum = 1.0;
    if (r.softmax) {
        sum = 0.0;
        for (int e = lane; e < E; e += 32) {
            const float x = to_float(logits[e]);
            if (x > -INFINITY) sum += exp((double)x - (double)row.m);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kFullMask, sum, o);
    }
    // -inf for an expert that is not open
    auto nearly = [&](int e) {
        const float x = to_float(logits[e]);
        return x == -INFINITY ? x : rankable(score_of(x, r, row) + (r.bias ? r.bias[e] : 0.0f));
    };
    auto exactly = [&](int e) {
        const double x = to_float(logits[e]), b = r.bias ? r.bias[e] : 0.0f;
        return rankable((r.softmax ? exp(x - (double)row.m) / sum : 1.0 / (1.0 + exp(-x))) + b);
    };
    // what the picks go by: without a bias the logits
    auto key = [&](int e) {
        const float x = to_float(logits[e]);
        return r.bias || x == -INFINITY ? nearly(e) : rankable(x);
    };
    auto exact_key = [&](int e) { return r.bias ? exactly(e) : rankable((double)to_float(logits[e])); };
    unsigned kept = kFullMask;
    if (limited) {
        // Groups near the border are valued exactly; the others keep their side of it.
        kept = best_groups(value, r.groups, lane, r.top_groups);
        const bool mine = lane < r.groups && value > -INFINITY;
        const float least = -warp_max_of(mine && (kept >> lane & 1) ? -value : -INFINITY);
        const float most = warp_max_of(mine && !(kept >> lane & 1) ? value : -INFINITY);
        const unsigned open = __ballot_sync(kFullMask, mine && value >= least - room_g && value <= most + room_g);
        double exact = kept >> lane & 1 ? DBL_MAX : -DBL_MAX;
        for (unsigned left = open; left; left &= left - 1) {
            const int g = __ffs(left) - 1;
            float a = -INFINITY, b = -INFINITY;
            for (int i = lane; i < size; i += 32) insert(nearly(g * size + i), a, b);
            top_two(a, b, 32);
            const float from = (b > -INFINITY ? b : a) - room;
            double u = -INFINITY, v = -INFINITY;
            for (int i = lane; i < size; i += 32)
                if (nearly(g * size + i) >= fmaxf(from, -FLT_MAX)) insert(exactly(g * size + i), u, v);
            top_two(u, v, 32);
            const double w = group_value(u, v, r.group_top);
            if (lane == g) exact = w;
        }
        if (!(lane < r.groups && value > -INFINITY)) exact = -INFINITY;
        kept = best_groups(exact, r.groups, lane, r.top_groups);
    }
    auto stays = [&](int e) { return !limited || (kept >> (e / size) & 1); };
    // The Kth largest fp32 key: what is below it by more than the errors is out.
    for (int e = lane; e < E; e += 32) scratch[e] = stays(e) ? key(e) : -INFINITY;
    float least = -FLT_MAX;
    for (int k = 0; k < K; ++k) {
        float top = -INFINITY;
        int at = -1;
        for (int e = lane; e < E; e += 32)
            if (scratch[e] > top) {
                top = scratch[e];
                at = e;
            }
        const float all = warp_max_of(top);
        least = all;
        if (!(all > -INFINITY)) break;
        if (lane == __ffs(__ballot_sync(kFullMask, top == all)) - 1) scratch[at] = -INFINITY;
    }
    const float from = fmaxf(r.bias ? least - room : least, -FLT_MAX);
    __syncwarp();
    uint16_t *const list = reinterpret_cast<uint16_t *>(scratch);
    int n = 0;
    for (int e0 = 0; e0 < E; e0 += 32) {
        const int e = e0 + lane;
        const bool in = e < E && stays(e) && key(e) >= from;
        const unsigned all = __ballot_sync(kFullMask, in);
        if (in) list[n + __popc(all & ((1u << lane) - 1))] = (uint16_t)e;
        n += __popc(all);
    }
    __syncwarp();
    // Each candidate's place is the number of better ones (their list is in order of experts).
    for (int a0 = 0; a0 < n; a0 += 32) {
        const int i = a0 + lane, e = i < n ? list[i] : 0;
        const double v = i < n ? exact_key(e) : 0.0;
        int before = 0;
        for (int b0 = 0; b0 < n; b0 += 32) {
            const double w = b0 == a0 ? v : b0 + lane < n ? exact_key(list[b0 + lane]) : 0.0;
            for (int j = 0; j < min(32, n - b0); ++j) {
                const double o = __shfl_sync(kFullMask, w, j);
                before += o > v || (o == v && b0 + j < i);
            }
        }
        if (i < n && before < K) ids[before] = e;
    }
    if (lane >= n && lane < K) ids[lane] = -1;
    __syncwarp();
}

// KT > 0: K is KT, and the picks are unrolled.  single: the grid is one cluster.
template <int NV, int W, int KT, typename L>
__global__ void __launch_bounds__(kGroupedThreads, NV > 16 ? 1 : kGroupedPerSm)
route_grouped_kernel(const L *__restrict__ logits, int T, int E, int any_k, const Rules r,
                     const uint8_t *__restrict__ mask, int32_t *ids, float *__restrict__ weights,
                     uint32_t *__restrict__ part, RouteOut o, bool single)
{
    const int K = KT > 0 ? KT : any_k;
    extern __shared__ float sm[];
    float *const sums = sm;                              // [kGroupedWarps][E]; until then a warp's scratch
    int32_t *const cnt = reinterpret_cast<int32_t *>(sm + (size_t)kGroupedWarps * E);     // [E] and the routed tokens
    uint32_t *const inbox = reinterpret_cast<uint32_t *>(cnt + E + 1);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
    for (int e = threadIdx.x; e <= E; e += kGroupedThreads) cnt[e] = 0;
    pdl_wait();
    pdl_trigger();
    __syncthreads();

    const int k_lanes = 1 << (32 - __clz(K - 1));        // K, rounded up to a power of two
    const int size = E / r.groups;                       // experts a group
    const bool limited = r.top_groups < r.groups;
    // a group is a power of two of lanes, all of their values in it
    const int group_lanes = size % NV == 0 && ((size / NV) & (size / NV - 1)) == 0 ? size / NV : 0;
    int routed = 0;                                      // tokens with a first pick (lane 0)
    float acc[NV], b[NV], largest = 0.0f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        acc[j] = 0.0f;
        b[j] = r.bias && lane * NV + j < E ? r.bias[lane * NV + j] : 0.0f;
        largest = fmaxf(largest, fabsf(b[j]));
    }
    largest = warp_max(largest);

    constexpr bool kAhead = NV <= 8;
    const int stride = gridDim.x * kGroupedWarps;
    int t = blockIdx.x * kGroupedWarps + warp;
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
        Row row{0.0f, 0.0f};
        float s[NV], total = 0.0f;
        if (r.softmax) {
            row.m = warp_max(lane_max<NV>(x));
            if (!(row.m > -INFINITY)) row.m = 0.0f;
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                s[j] = weight_of(x[j], row.m);
                total += s[j];
            }
            total = warp_sum(total);
            row.inv = total == 0.0f ? 0.0f : __fdividef(1.0f, total);
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                s[j] *= row.inv;
                acc[j] += s[j];
            }
        } else {
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                float rest;
                s[j] = logistic(x[j], rest);
                total += s[j];
            }
            total = warp_sum(total);
            const float inv = total == 0.0f ? 0.0f : __fdividef(1.0f, total);
#pragma unroll
            for (int j = 0; j < NV; ++j) acc[j] += s[j] * inv;
        }
        // The scores' errors at most, for differences of keys and of group values:
        // a score is at most `top`, and |z| times it at most a third of a unit.
        const float top_score = r.softmax ? row.inv : 1.0f;
        const float room = 4.0f * kUnit * ((r.softmax ? 65.0f : 9.0f) * top_score + top_score + largest), room_g = 3.0f * room;

        // key: what the picks go by; -inf where an expert is not open or its group is out
        float key[NV], value = -INFINITY;
        bool unsure = false;
#pragma unroll
        for (int j = 0; j < NV; ++j) key[j] = x[j] == -INFINITY ? x[j] : rankable(s[j] + b[j]);
        if (limited) {
            if (group_lanes > 0) {
                float a = key[0], c = -INFINITY;
#pragma unroll
                for (int j = 1; j < NV; ++j) {
                    c = fmaxf(c, fminf(a, key[j]));
                    a = fmaxf(a, key[j]);
                }
                top_two(a, c, group_lanes);
                value = __shfl_sync(kFullMask, group_value(a, c, r.group_top), lane * group_lanes & 31);
            } else {
                float *const mine = sums + warp * E;
#pragma unroll
                for (int j = 0; j < NV; ++j)
                    if (lane * NV + j < E) mine[lane * NV + j] = key[j];
                __syncwarp();
                for (int g = 0; g < r.groups; ++g) {
                    float a = -INFINITY, c = -INFINITY;
                    for (int i = lane; i < size; i += 32) insert(mine[g * size + i], a, c);
                    top_two(a, c, 32);
                    if (lane == g) value = group_value(a, c, r.group_top);
                }
                __syncwarp();
            }
            if (lane >= r.groups) value = -INFINITY;
            else if (value > -INFINITY) value = fmaxf(value, -FLT_MAX);
            const unsigned kept = best_groups(value, r.groups, lane, r.top_groups);
            const bool stays = kept >> lane & 1;
            const float least = -warp_max(stays && value > -INFINITY ? -value : -INFINITY);
            const float most = warp_max(stays ? -INFINITY : value);
            unsure = most > -INFINITY && least - most <= room_g;
#pragma unroll
            for (int j = 0; j < NV; ++j)
                if (!(kept >> ((unsigned)(lane * NV + j) / (unsigned)size & 31) & 1)) key[j] = -INFINITY;
        }
        if (!r.bias) {
#pragma unroll
            for (int j = 0; j < NV; ++j) key[j] = key[j] > -INFINITY ? rankable(x[j] + 0.0f) : key[j];
        }

        // Pick number `lane`: its key, and the lane that holds it (route.cu).
        float mine = -INFINITY;
        int from = 0;
        float next[NV];
#pragma unroll
        for (int j = 0; j < NV; ++j) next[j] = key[j];
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
        // Its place among the owner's keys (equal ones were picked in order), and its logit.
        const unsigned alike = __match_any_sync(kFullMask, __float_as_int(mine)) & __match_any_sync(kFullMask, from);
        int before = __popc(alike & ((1u << lane) - 1)), place = 0;
        float chosen = -INFINITY;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const bool same = __shfl_sync(kFullMask, key[j], from) == mine;
            const float xj = __shfl_sync(kFullMask, x[j], from);
            if (same && before == 0) {
                place = j;
                chosen = xj;
            }
            before -= same;
        }
        bool taken = lane < K && mine > -INFINITY;
        int id = taken ? from * NV + place : -1;
        if (r.bias) {
            // The last pick against the best that was left, and each against the next.
            const float left = warp_max(best), error = error_of(chosen, score_of(chosen, r, row), mine, r, row);
            const float next_key = __shfl_down_sync(kFullMask, mine, 1), next_x = __shfl_down_sync(kFullMask, chosen, 1);
            const float both = error + __shfl_down_sync(kFullMask, error, 1);
            const int next_id = __shfl_down_sync(kFullMask, id, 1);
            bool near = taken && lane == K - 1 && left > -INFINITY && mine - left <= room;
            if (taken && lane < K - 1 && next_key > -INFINITY && mine - next_key <= 2.0f * both)
                near = next_x != chosen || r.bias[next_id] != r.bias[id];       // the same expert twice is in order
            unsure |= __any_sync(kFullMask, near);
        }
        if (unsure) {
            choose_exactly<L>(logits + (size_t)t * E, E, K, r, row, value, room_g, room, sums + warp * E, ids + (size_t)t * K);
            id = lane < K ? ids[(size_t)t * K + lane] : -1;
            taken = id >= 0;
            chosen = taken ? to_float(logits[(size_t)t * E + id]) : -INFINITY;
            __syncwarp();
        }
        float w = taken ? score_of(chosen, r, row) : 0.0f;
        if (r.renorm) {
            const float all = lanes_sum(w, k_lanes);
            if (all != 0.0f) w = __fdividef(w, all);
        }
        if (lane < K) {
            ids[(size_t)t * K + lane] = id;
            weights[(size_t)t * K + lane] = w * r.scale;
        }
        if (taken) atomicAdd(&cnt[id], 1);
        routed += taken;
    }
    __syncwarp();
#pragma unroll
    for (int j = 0; j < NV; ++j)
        if (lane * NV + j < E) sums[warp * E + lane * NV + j] = acc[j];
    if (lane == 0) atomicAdd(&cnt[E], routed);
    if (single) route_totals<kGroupedWarps, true>(sums, cnt, inbox, E, K, part, o);
    else route_totals<kGroupedWarps, false>(sums, cnt, inbox, E, K, part, o);
}

template <int NV, int W, typename L>
cudaError_t run_grouped(const void *logits, int T, int E, int K, const Rules &r, float coef, const uint8_t *mask,
                        int32_t *ids, float *weights, int32_t *counts, int32_t *routed, float *loss, void *workspace,
                        cudaStream_t s)
{
    const size_t smem = route_smem<kGroupedWarps>(E);
    const RouteOut o{counts, routed, loss, coef};
    const int single = single_blocks<kGroupedWarps>(T, E);
    constexpr int KT = W > 1 ? 8 : 0;                    // as in route.cu
    auto *const kernel = K == KT ? route_grouped_kernel<NV, W, KT, L> : route_grouped_kernel<NV, W, 0, L>;
    if (smem > 40 << 10) {
        const cudaError_t e = allow_dynamic_smem(reinterpret_cast<const void *>(kernel), smem);
        if (e != cudaSuccess) return e;
    }
    const int blocks = single ? single : route_clusters<kGroupedWarps, kGroupedPerSm>(T) * kRouteCluster;
    uint32_t *part = static_cast<uint32_t *>(workspace);
    cudaError_t e = launch_pdl_clusters(kernel, dim3(blocks), dim3(kGroupedThreads), smem, s,
                                        single ? single : kRouteCluster, static_cast<const L *>(logits),
                                        T, E, K, r, mask, ids, weights, part, o, single > 0);
    if (e != cudaSuccess || single) return e;
    return launch_route_finish(part, blocks / kRouteCluster, E, K, o, s);
}

}  // namespace

size_t route_grouped_workspace_bytes(int T, int E)
{
    return totals_workspace_bytes<kGroupedWarps, kGroupedPerSm>(T, E);
}

cudaError_t launch_route_grouped(const void *logits, int bf16, int T, int E, int K, int softmax, const float *bias,
                                 int groups, int top_groups, int group_top, int renorm, float scale, float coef,
                                 const uint8_t *mask, int32_t *ids, float *weights, int32_t *counts, int32_t *routed,
                                 float *loss, void *workspace, cudaStream_t stream)
{
    const Rules r{bias, softmax, groups, top_groups, group_top, renorm, scale};
#define CALL(NV, W, L)                                                                    \
    run_grouped<NV, W, L>(logits, T, E, K, r, coef, mask, ids, weights, counts, routed, loss, workspace, stream)
    MOE_GROUPED_CASES(CALL, logits);
#undef CALL
}

}  // namespace moe
