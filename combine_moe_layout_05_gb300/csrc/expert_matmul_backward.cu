// expert_matmul_backward.cu -- the gradients of the experts' product with
// respect to the rows and to the weights (expert_matmul_common.cuh).
#include "expert_matmul_common.cuh"

namespace moe {
namespace {

using RowsWide = Shape<kRows, false, 2, 256, 6, 2>;
using RowsMid = Shape<kRows, false, 2, 128, 8, 2>;
using RowsNarrow = Shape<kRows, false, 1, 32, 10, 1>;
using Weights = Shape<kWeights, false, 2, 256, 5, 2>;

}  // namespace

cudaError_t launch_expert_matmul_rows(const void *grad_pre, const void *w, const int32_t *offsets, int rows, int H,
                                      int N, int E, void *grad_x, uint32_t *dev_error, cudaStream_t stream,
                                      int64_t wait_cycles, int stall)
{
    const long long limit = wait_cycles > 0 ? wait_cycles : kWaitLimitCycles;
    int sms = 0;
    const cudaError_t e = device_sm_count(&sms);
    if (e != cudaSuccess) return e;
    CUtensorMap map_w;                                 // [E, N, H]: past an expert's N are zeros, not the next one's
    const uint64_t dims[3] = {(uint64_t)H, (uint64_t)N, (uint64_t)E}, strides[2] = {(uint64_t)H, (uint64_t)N * H};
    const uint32_t box[3] = {64, kStep, 1};
    if (!tensor_map(&map_w, w, 3, dims, strides, box)) return cudaErrorInvalidValue;
    const Sizes z{rows, N, H, N, E};
    const Store st{nullptr, nullptr, nullptr, grad_x, MOE_ACT_NONE, 0, 0};
    auto go = [&](auto shape) {
        using S = decltype(shape);
        RowMaps map_g;
        if (!row_maps<S>(&map_g, grad_pre, rows, N)) return cudaErrorInvalidValue;
        const int64_t tiles = most_tiles<S>(rows, E) * ceil_div(H, S::OUT * S::CG);
        return run<S>(map_w, map_g, offsets, z, st, tiles, sms, 1, dev_error, 1, limit, stall, stream);
    };
    // As for the product itself (64 experts, 2048 -> 2048, Mid and Wide: 85.4 and 85.0 us
    // at 64 rows an expert, 88.4 and 87.2 at 96, 103 and 92.5 at 160, 392 and 339 at 1024).
    if (rows <= 16 * E) return go(RowsNarrow{});
    return rows >= 96 * E ? go(RowsWide{}) : go(RowsMid{});
}

cudaError_t launch_expert_matmul_weights(const void *grad_pre, const void *x, const int32_t *offsets, int rows, int H,
                                         int N, int E, void *grad_w, int f32, int accumulate, uint32_t *dev_error,
                                         int clear, cudaStream_t stream, int64_t wait_cycles, int stall)
{
    const long long limit = wait_cycles > 0 ? wait_cycles : kWaitLimitCycles;
    int sms = 0;
    const cudaError_t e = device_sm_count(&sms);
    if (e != cudaSuccess) return e;
    CUtensorMap map_g;
    RowMaps map_x;
    if (!rows_map(&map_g, grad_pre, rows, N, kStep) || !rows_map(&map_x.box[0], x, rows, H, kStep))
        return cudaErrorInvalidValue;
    const uint64_t dims[3] = {(uint64_t)H, (uint64_t)N, (uint64_t)E}, strides[2] = {(uint64_t)H, (uint64_t)N * H};
    const uint32_t box[3] = {f32 ? 32u : 64u, 32, 1};
    if (!tensor_map(&map_x.box[1], grad_w, 3, dims, strides, box, f32 != 0)) return cudaErrorInvalidValue;
    for (int m = 2; m < kBoxes; ++m) map_x.box[m] = map_x.box[0];
    const Sizes z{rows, N, H, 0, E};
    const Store st{nullptr, nullptr, nullptr, grad_w, MOE_ACT_NONE, f32, accumulate};
    const int64_t tiles = (int64_t)E * ceil_div(H, Weights::NT) * ceil_div(N, Weights::OUT * Weights::CG);
    return run<Weights>(map_g, map_x, offsets, z, st, tiles, sms, 1, dev_error, clear, limit, stall, stream);
}

}  // namespace moe

// Test hook, deliberately absent from the public header: one gradient (weights
// != 0: the weights' in bf16, else the rows') with a bound on every wait and a
// barrier held back, as moe_testing_expert_matmul has them.
extern "C" __attribute__((visibility("default"))) int32_t
moe_testing_expert_matmul_backward(const void *grad_pre, const void *other, const int32_t *expert_offsets, int32_t rows,
                                   int32_t H, int32_t N, int32_t E, int32_t weights, void *out, uint32_t *dev_error,
                                   int64_t wait_cycles, int32_t stall, cudaStream_t stream)
{
    const cudaError_t e =
        weights ? moe::launch_expert_matmul_weights(grad_pre, other, expert_offsets, rows, H, N, E, out, 0, 0, dev_error, 1,
                                                    stream, wait_cycles, stall)
                : moe::launch_expert_matmul_rows(grad_pre, other, expert_offsets, rows, H, N, E, out, dev_error, stream,
                                                 wait_cycles, stall);
    return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}
