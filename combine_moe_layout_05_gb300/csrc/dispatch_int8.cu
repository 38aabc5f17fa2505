// dispatch_int8.cu -- quantise each token row to int8 with one scale and pack
// it into the token's K slots.
//
//   scale = max |x| * (1/127),  code = rint(x / scale)      (fp32, IEEE division)
//
// A block owns a token: it reads the row for its maximum, reads it again (out
// of L1 or L2) to quantise, and writes 16 codes a thread to every slot.
#include "common.cuh"
#include "internal.h"
#include "moe_layout.h"
#include "rowops.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;

// max |x| over 8 bf16 values as raw magnitude bits: for IEEE numbers the
// order of the magnitudes is the order of their bits, and NaN ranks highest,
// so one NaN or infinity in a row is seen.
__device__ __forceinline__ uint32_t amax_bits(const uint4 &v)
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) m = max(m, max(w[i] << 16 & 0x7fff0000u, w[i] & 0x7fff0000u));
    return m;
}

__device__ __forceinline__ uint32_t code_of(float x, float scale)
{
    const int q = __float2int_rn(__fdiv_rn(x, scale));
    return (uint32_t)max(-127, min(127, q)) & 0xffu;
}

__device__ __forceinline__ uint2 codes8(const uint4 &v, float scale)
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t q[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) q[i] = code_of(bf16_lo(w[i]), scale) | code_of(bf16_hi(w[i]), scale) << 8;
    return make_uint2(q[0] | q[1] << 16, q[2] | q[3] << 16);
}

__global__ void __launch_bounds__(kThreads)
dispatch_int8_kernel(const uint4 *__restrict__ tokens, int K, int H,
                     const int32_t *__restrict__ dst_row, int rows, uint8_t *__restrict__ packed,
                     float *__restrict__ scales)
{
    __shared__ uint32_t red[kThreads / 32];
    pdl_wait();
    pdl_trigger();
    const int t = blockIdx.x, units = H >> 4;
    const uint4 *row = tokens + (size_t)t * (H >> 3);
    uint32_t m = 0;
    for (int u = threadIdx.x; u < units; u += kThreads)
        m = max(m, max(amax_bits(row[2 * u]), amax_bits(row[2 * u + 1])));
    m = __reduce_max_sync(kFullMask, m);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) m = max(m, red[w]);
    const bool bad = m >= 0x7f800000u;           // infinity or NaN somewhere in the row
    const float scale = bad ? __int_as_float(0x7fc00000) : __uint_as_float(m) * (1.0f / 127.0f);
    const int32_t *slots = dst_row + (size_t)t * K;
    for (int u = threadIdx.x; u < units; u += kThreads) {
        uint4 q = make_uint4(0, 0, 0, 0);
        if (m != 0 && !bad) {
            const uint2 a = codes8(row[2 * u], scale), b = codes8(row[2 * u + 1], scale);
            q = make_uint4(a.x, a.y, b.x, b.y);
        }
        store_to_slots<0>(slots, K, rows, packed, (size_t)H, (size_t)u * 16, q);
    }
    if (threadIdx.x < K) {
        const int r = slots[threadIdx.x];
        if ((unsigned)r < (unsigned)rows) scales[r] = scale;
    }
}

}  // namespace

cudaError_t launch_dispatch_int8(const void *tokens, int T, int H, int K, const int32_t *dst_row,
                                 void *packed, float *scales, cudaStream_t stream)
{
    return launch_pdl(dispatch_int8_kernel, dim3(T), dim3(kThreads), 0, stream,
                      static_cast<const uint4 *>(tokens), K, H, dst_row, T * K,
                      static_cast<uint8_t *>(packed), scales);
}

}  // namespace moe
