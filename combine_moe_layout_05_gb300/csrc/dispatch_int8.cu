// dispatch_int8.cu -- quantise each token row to int8 with one scale and pack
// it into the token's K slots.
//
//   scale = max |x| * (1/127),  code = rint(x / scale)      (fp32, IEEE division)
//
// HBM-bound: a row is read once and its codes written K times.  A block owns a
// token and a thread P pieces of 16 values, which stay in registers between
// the row's maximum and the quantising; a longer row than the largest block
// holds is read a second time, out of L1 or L2.  16384 x 4096, K = 8: 99 us,
// 6.77 TB/s; 128 x 7168: 3.4 us, one round of loads, a barrier and the stores.
#include "common.cuh"
#include "internal.h"
#include "moe_layout.h"
#include "rowops.cuh"

namespace moe {
namespace {

constexpr int kMaxThreads = 512;

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

// P pieces of 16 values a thread; P == 0: any number, read twice.  KT: slots a
// token, or 0 where that is not known here.
template <int P, int KT>
__global__ void __launch_bounds__(kMaxThreads)
dispatch_int8_kernel(const uint4 *__restrict__ tokens, int K, int H,
                     const int32_t *__restrict__ dst_row, int rows, uint8_t *__restrict__ packed,
                     float *__restrict__ scales)
{
    __shared__ uint32_t red[kMaxThreads / 32];
    pdl_wait();
    pdl_trigger();
    const int t = blockIdx.x, units = H >> 4, threads = blockDim.x;
    const uint4 *row = tokens + (size_t)t * (H >> 3);
    const int32_t *slots = dst_row + (size_t)t * K;
    const int k_count = KT > 0 ? KT : K;
    int slot = -1;
    if (threadIdx.x < k_count) slot = slots[threadIdx.x];
    constexpr int R = P > 0 ? P : 1;
    uint4 a[R], b[R];
    uint32_t m = 0;
    if constexpr (P > 0) {
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const int u = threadIdx.x + i * threads;
            a[i] = b[i] = make_uint4(0, 0, 0, 0);
            if (u < units) {
                a[i] = ld_stream_v4(row + 2 * u);
                b[i] = ld_stream_v4(row + 2 * u + 1);
            }
        }
#pragma unroll
        for (int i = 0; i < P; ++i) m = max(m, max(amax_bits(a[i]), amax_bits(b[i])));
    } else {
        for (int u = threadIdx.x; u < units; u += threads)
            m = max(m, max(amax_bits(row[2 * u]), amax_bits(row[2 * u + 1])));
    }
    m = __reduce_max_sync(kFullMask, m);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = m;
    __syncthreads();
    for (int w = 0; w < threads / 32; ++w) m = max(m, red[w]);
    const bool bad = m >= 0x7f800000u;           // infinity or NaN somewhere in the row
    const float scale = bad ? __int_as_float(0x7fc00000) : __uint_as_float(m) * (1.0f / 127.0f);
    if ((unsigned)slot < (unsigned)rows) scales[slot] = scale;
    auto write = [&](int u, const uint4 &va, const uint4 &vb) {
        uint4 q = make_uint4(0, 0, 0, 0);
        if (m != 0 && !bad) {
            const uint2 x = codes8(va, scale), y = codes8(vb, scale);
            q = make_uint4(x.x, x.y, y.x, y.y);
        }
        store_to_slots<KT>(slots, k_count, rows, packed, (size_t)H, (size_t)u * 16, q);
    };
    if constexpr (P > 0) {
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const int u = threadIdx.x + i * threads;
            if (u < units) write(u, a[i], b[i]);
        }
    } else {
        for (int u = threadIdx.x; u < units; u += threads) write(u, row[2 * u], row[2 * u + 1]);
    }
}

template <int P>
cudaError_t run(const void *tokens, int T, int H, int K, const int32_t *dst_row, void *packed, float *scales,
                int threads, cudaStream_t s)
{
    auto go = [&](auto *kernel) {
        return launch_pdl(kernel, dim3(T), dim3(threads), 0, s, static_cast<const uint4 *>(tokens), K, H, dst_row,
                          T * K, static_cast<uint8_t *>(packed), scales);
    };
    if (K == 8) return go(dispatch_int8_kernel<P, 8>);
    if (K == 1) return go(dispatch_int8_kernel<P, 1>);
    return go(dispatch_int8_kernel<P, 0>);
}

}  // namespace

cudaError_t launch_dispatch_int8(const void *tokens, int T, int H, int K, const int32_t *dst_row,
                                 void *packed, float *scales, cudaStream_t stream)
{
    const int units = H / 16;
    const int P = ceil_div(units, kMaxThreads);
    const int threads = P <= 2 ? ceil_div(ceil_div(units, P), 32) * 32 : kMaxThreads;
    if (P == 1) return run<1>(tokens, T, H, K, dst_row, packed, scales, threads, stream);
    if (P == 2) return run<2>(tokens, T, H, K, dst_row, packed, scales, threads, stream);
    return run<0>(tokens, T, H, K, dst_row, packed, scales, threads, stream);
}

}  // namespace moe
