// expert_matmul.cu -- packed bf16 rows times their experts' weights, with bias,
// activation and residual in the same pass (expert_matmul_common.cuh).
#include "expert_matmul_common.cuh"

namespace moe {
namespace {

template <bool G> using Wide = Shape<kForward, G, 2, 256, 6, 2>;
template <bool G> using Mid = Shape<kForward, G, 2, 128, 8, 2>;
template <bool G> using Narrow = Shape<kForward, G, 1, 32, 10, 1>;
template <bool G> using Split = Shape<kForward, G, 1, 32, 9, 1, true>;

template <bool G>
cudaError_t launch(const void *x, const void *w, const int32_t *offsets, int rows, int H, int N, int E, const Store &st,
                   uint32_t *dev_error, cudaStream_t stream, long long wait_limit, int stall)
{
    const int channels = G ? N / 2 : N;
    int sms = 0;
    cudaError_t e = device_sm_count(&sms);
    if (e != cudaSuccess) return e;
    CUtensorMap map_w;
    if (G) {                                           // 16 gate channels, then their 16 up channels
        const uint64_t dims[4] = {(uint64_t)H, (uint64_t)channels, 2, (uint64_t)E};
        const uint64_t strides[3] = {(uint64_t)H, (uint64_t)channels * H, (uint64_t)N * H};
        const uint32_t box[4] = {kStep, 16, 2, 1};
        if (!tensor_map(&map_w, w, 4, dims, strides, box)) return cudaErrorInvalidValue;
    } else if (!rows_map(&map_w, w, (uint64_t)E * N, H, kChannels)) {
        return cudaErrorInvalidValue;
    }
    const Sizes z{rows, N, channels, H, E};
    auto go = [&](auto shape, int parts) {
        using S = decltype(shape);
        RowMaps map_x;
        if (!row_maps<S>(&map_x, x, rows, H)) return cudaErrorInvalidValue;
        const int64_t tiles = most_tiles<S>(rows, E) * ceil_div(channels, S::OUT * S::CG);
        return run<S>(map_w, map_x, offsets, z, st, tiles, sms, parts, dev_error, 1, wait_limit, stall, stream);
    };
    // Few tiles: share the contraction, as far as every tile's cluster runs at
    // once and the contraction is long enough for the cluster's exchange (16 or 32
    // rows of one expert, shared out and not: 7168 -> 2048 15.8 and 19.5 us, 4096 ->
    // 4096 11.9 and 12.3, 2048 -> 2048 9.6 and 7.8).
    const int64_t tiles = most_tiles<Split<G>>(rows, E) * ceil_div(channels, Split<G>::OUT);
    const int steps = ceil_div(H, kStep);
    if (tiles * 2 <= sms && steps >= 64) {
        int clusters[3];
        e = split_clusters<expert_matmul_kernel<Split<G>>>(Split<G>::THREADS, Split<G>::bytes(MOE_MAX_EXPERTS), clusters);
        if (e != cudaSuccess) return e;
        int parts = 1;
        for (int p = 2; p <= 8 && steps >= 8 * p; p *= 2)
            if (tiles <= clusters[p / 4]) parts = p;
        if (parts > 1) return go(Split<G>{}, parts);
    }
    // By rows an expert, on average.  Narrow and Mid: 7.8 and 10.9 us at 16 rows of one
    // expert (2048 -> 2048), 138 and 140 at 8 rows of 32 (7168 -> 2048), but 83.8 and
    // 80.7 at 16 rows of 64 (2048 -> 2048), and from 32 rows on Narrow reads weights
    // twice (93.8 and 83.8 at 48).  The average does not see rows that are a few
    // experts': 8 of 256 with 512 rows each (2048 -> 2048) 74.6 and 29.4.  Mid and
    // Wide, even loads: the border is between 128 and 160 rows (64 experts, 2048 ->
    // 2048: 87.9 and 90.8 at 96, 90.4 and 93.4 at 128, 105 and 96 at 160, 381 and 338 at
    // 1024; 32, 7168 -> 2048: 150 and 157 at 96, 153 and 161 at 128, 184 and 165 at 160;
    // 64, 512 -> 4096: 51.3 and 51.7 at 96, 54.7 and 54.5 at 128).  Rows in proportion
    // to 1 / rank, nearer to what routing gives: 95.1 and 91.8 at 96, 159 and 163 (172
    // and 161 at 128), 55.7 and 53.7; 48 experts, 2056 -> 1008, 46.6 and 43.7.
    if (rows <= 16 * E) return go(Narrow<G>{}, 1);
    return rows >= 96 * E ? go(Wide<G>{}, 1) : go(Mid<G>{}, 1);
}

}  // namespace

cudaError_t launch_expert_matmul(const void *x, const void *w, const float *bias, const int32_t *offsets, int rows,
                                 int H, int N, int E, int activation, const void *residual, void *pre, void *out,
                                 uint32_t *dev_error, cudaStream_t stream, int64_t wait_cycles, int stall)
{
    const long long limit = wait_cycles > 0 ? wait_cycles : kWaitLimitCycles;
    const Store st{bias, static_cast<const __nv_bfloat16 *>(residual), static_cast<__nv_bfloat16 *>(pre), out,
                   activation, 0, 0};
    return activation == MOE_ACT_SWIGLU
               ? launch<true>(x, w, offsets, rows, H, N, E, st, dev_error, stream, limit, stall)
               : launch<false>(x, w, offsets, rows, H, N, E, st, dev_error, stream, limit, stall);
}

}  // namespace moe

// Test hook, deliberately absent from the public header: the product with a
// chosen bound on every wait (in clock cycles; 0: the default) and, in the
// CTAs of the first tiles, one barrier that waits for an arrival that never
// comes: stall 0 a step landed, 1 its slot free again, 2 landed in both CTAs of
// a pair, 3 sums ready, 4 sums stored, 5 the other CTAs' sums (where the
// contraction is split); anything else none.  A test uses it to see a bounded
// wait expire: the kernel sets MOE_DEV_ERR_TIMEOUT and finishes, and the
// context stays usable.  Arguments are checked by the caller (tests only).
extern "C" __attribute__((visibility("default"))) int32_t
moe_testing_expert_matmul(const void *x, const void *weights, const int32_t *expert_offsets, int32_t rows, int32_t H,
                          int32_t N, int32_t E, int32_t activation, void *out, uint32_t *dev_error, int64_t wait_cycles,
                          int32_t stall, cudaStream_t stream)
{
    const cudaError_t e = moe::launch_expert_matmul(x, weights, nullptr, expert_offsets, rows, H, N, E, activation, nullptr,
                                                    nullptr, out, dev_error, stream, wait_cycles, stall);
    return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}
