// expert_matmul_int8.cu -- packed int8 rows times their experts' int8
// weights, with a scale for each row and each output channel.
//
//   out[r, n] = bf16((sum_h x[r, h] * w[e, n, h]) * x_scale[r] * w_scale[e, n])
//   for the rows r of expert e, [offsets[e], offsets[e+1])
//
// A block owns 64 channels of one expert and walks that expert's rows 64 at a
// time; the sums are int32 and exact.
#include "common.cuh"
#include "internal.h"
#include "moe_layout.h"

namespace moe {
namespace {

constexpr int kTile = 64;        // rows and channels of a tile
constexpr int kStepWords = 16;   // 64 bytes of the contraction a step
constexpr int kPad = 1;

__global__ void __launch_bounds__(256)
expert_matmul_int8_kernel(const uint8_t *__restrict__ x, const float *__restrict__ xs,
                          const uint8_t *__restrict__ w, const float *__restrict__ ws,
                          const int32_t *__restrict__ offsets, int rows, int H, int N,
                          __nv_bfloat16 *__restrict__ out)
{
    __shared__ uint32_t sx[kTile][kStepWords + kPad], sw[kTile][kStepWords + kPad];
    pdl_wait();
    pdl_trigger();
    const int e = blockIdx.y, n0 = blockIdx.x * kTile;
    const int lo = max(0, min(rows, offsets[e])), hi = max(lo, min(rows, offsets[e + 1]));
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const int lr = threadIdx.x >> 2, lc = (threadIdx.x & 3) * 16;    // 16 bytes of a tile row each
    for (int r0 = lo; r0 < hi; r0 += kTile) {
        int acc[4][4] = {};
        for (int h0 = 0; h0 < H; h0 += kStepWords * 4) {
            uint4 vx = make_uint4(0, 0, 0, 0), vw = vx;
            if (h0 + lc < H) {
                if (r0 + lr < hi) vx = *reinterpret_cast<const uint4 *>(x + (size_t)(r0 + lr) * H + h0 + lc);
                if (n0 + lr < N)
                    vw = *reinterpret_cast<const uint4 *>(w + ((size_t)e * N + n0 + lr) * H + h0 + lc);
            }
            __syncthreads();
            const int c = lc / 4;
            sx[lr][c] = vx.x, sx[lr][c + 1] = vx.y, sx[lr][c + 2] = vx.z, sx[lr][c + 3] = vx.w;
            sw[lr][c] = vw.x, sw[lr][c + 1] = vw.y, sw[lr][c + 2] = vw.z, sw[lr][c + 3] = vw.w;
            __syncthreads();
#pragma unroll
            for (int c2 = 0; c2 < kStepWords; ++c2) {
                int a[4], b[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    a[i] = (int)sx[ty * 4 + i][c2];
                    b[i] = (int)sw[tx + 16 * i][c2];
                }
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) acc[i][j] = __dp4a(a[i], b[j], acc[i][j]);
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = r0 + ty * 4 + i;
            if (r >= hi) continue;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int n = n0 + tx + 16 * j;
                if (n < N)
                    out[(size_t)r * N + n] = __float2bfloat16_rn((float)acc[i][j] * xs[r] * ws[(size_t)e * N + n]);
            }
        }
    }
}

}  // namespace

cudaError_t launch_expert_matmul_int8(const void *x, const float *x_scales, const void *w,
                                      const float *w_scales, const int32_t *offsets, int rows,
                                      int H, int N, int E, void *out, cudaStream_t stream)
{
    return launch_pdl(expert_matmul_int8_kernel, dim3(ceil_div(N, kTile), E), dim3(256), 0, stream,
                      static_cast<const uint8_t *>(x), x_scales, static_cast<const uint8_t *>(w),
                      w_scales, offsets, rows, H, N, static_cast<__nv_bfloat16 *>(out));
}

}  // namespace moe
