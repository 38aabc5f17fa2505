// activation_backward.cu -- the gradient at the experts' values before the
// activation, and the sum over each expert's rows that is its bias gradient.
//
//   grad_pre[r, n] = grad_out[r, n] a'(pre[r, n]);  gated, with g and u the two
//   halves of a row: grad_out u a'(g) and grad_out a(g)
//   grad_bias[e, n] = sum over the rows r of expert e of grad_pre[r, n]  (unrounded)
//
// Bound by HBM: each value is read once and written once, 16 bytes a load, four
// rows of loads in flight a thread.  The bias sum is taken in the same pass: a
// block has a chunk of one expert's rows by a strip of columns and adds its rows
// up in fp32 (a thread's rows, then the threads of a column, always in that
// order); a second kernel adds an expert's chunks up in order.  So a call's
// results do not depend on timing, and the largest expert's rows are as many
// chunks as they need.
//
// 131072 rows of 4096, gated, 128 experts: 420 us without the bias (6.4 TB/s), 432
// with it.  4662 rows of 1032: 7.0 and 12.9 us,
// starts and two rounds of loads; the second kernel and its launch are 6.
// Two, three or four blocks a multiprocessor, with two or four rows in flight,
// differ by 5 %.
#include "activation.cuh"
#include "expert_tiles.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kBlocks = 152 * 4;
constexpr int kInFlight = 4;                         // rows

__device__ __forceinline__ void unpack8(const uint4 &v, float *x)
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = bf16_lo(w[i]);
        x[2 * i + 1] = bf16_hi(w[i]);
    }
}

__device__ __forceinline__ uint4 pack8(const float *x)
{
    return {pack_bf16x2_rn(x[0], x[1]), pack_bf16x2_rn(x[2], x[3]), pack_bf16x2_rn(x[4], x[5]), pack_bf16x2_rn(x[6], x[7])};
}

__device__ __forceinline__ uint4 load8(const __nv_bfloat16 *p) { return *reinterpret_cast<const uint4 *>(p); }

// pre and grad_pre may be one tensor, and grad_out and grad_pre where not
// gated: a thread reads its values before it writes them.
// first_chunk: for the finishing kernel, [E + 1]; partial: [most][N].
template <bool GATED, bool BIAS>
__global__ void __launch_bounds__(kThreads)
activation_backward_kernel(const __nv_bfloat16 *pre, const __nv_bfloat16 *grad_out, const int32_t *__restrict__ offsets,
                           int rows, int N, int E, int activation, __nv_bfloat16 *grad_pre,
                           int32_t *__restrict__ first_chunk, float *__restrict__ partial, int most, int columns, int chunk_rows)
{
    constexpr int HALVES = GATED ? 2 : 1;
    extern __shared__ int32_t sm[];                  // BIAS: first rows, first chunks of the experts
    __shared__ float red[BIAS ? HALVES * 8 : 1][kThreads];
    __shared__ int warp_tiles[kThreads / 32];
    int32_t *const first_row = sm, *const first_tile = sm + E + 1;
    pdl_wait();
    pdl_trigger();
    int chunks, begin = 0, end = 0;
    if constexpr (BIAS) {
        fill_table<kThreads>(offsets, rows, E, chunk_rows, first_row, first_tile, warp_tiles);
        chunks = min(first_tile[E], most);           // more only where offsets decrease
        if (blockIdx.x == 0)
            for (int e = threadIdx.x; e <= E; e += kThreads) first_chunk[e] = min(first_tile[e], most);
    } else {
        begin = max(0, min(rows, offsets[0]));
        end = max(begin, min(rows, offsets[E]));
        chunks = (int)((unsigned)(end - begin + chunk_rows - 1) / (unsigned)chunk_rows);
    }
    const int C = N / HALVES, strips = ceil_div(C, columns * 8);
    const int lanes = kThreads / columns;            // of rows; the threads past them have none
    const int ty = threadIdx.x / columns, tx = threadIdx.x - ty * columns;
    const int64_t items = (int64_t)chunks * strips;
    for (int64_t i = blockIdx.x; i < items; i += gridDim.x) {
        const int chunk = (int)(i / strips), c = ((int)(i - (int64_t)chunk * strips) * columns + tx) * 8;
        int row, last;
        if constexpr (BIAS) {
            int e = 0;                               // first_tile[e] <= chunk < first_tile[e + 1]
            for (int step = 512; step > 0; step >>= 1)
                if (e + step < E && first_tile[e + step] <= chunk) e += step;
            row = first_row[e] + (chunk - first_tile[e]) * chunk_rows;
            last = min(row + chunk_rows, first_row[e + 1]);
        } else {
            row = begin + chunk * chunk_rows;
            last = min(row + chunk_rows, end);
        }
        float sum[HALVES * 8];
#pragma unroll
        for (int j = 0; j < HALVES * 8; ++j) sum[j] = 0.0f;
        if (c < C && ty < lanes)
            for (int r0 = row + ty; r0 < last; r0 += lanes * kInFlight) {
                uint4 z[kInFlight][HALVES], dy[kInFlight];
#pragma unroll
                for (int k = 0; k < kInFlight; ++k) {
                    const int r = r0 + k * lanes;
                    if (r >= last) continue;
                    dy[k] = load8(grad_out + (size_t)r * C + c);
                    if (activation != MOE_ACT_NONE)
#pragma unroll
                        for (int h = 0; h < HALVES; ++h) z[k][h] = load8(pre + (size_t)r * N + h * C + c);
                }
#pragma unroll
                for (int k = 0; k < kInFlight; ++k) {
                    const int r = r0 + k * lanes;
                    if (r >= last) continue;
                    float g[8], y[HALVES * 8];
                    unpack8(dy[k], g);
                    if constexpr (GATED) {
                        float a[8], u[8];
                        unpack8(z[k][0], a);
                        unpack8(z[k][1], u);
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            const float s = sigmoid_approx(a[j]);
                            y[j] = g[j] * u[j] * silu_slope(a[j], s);
                            y[8 + j] = g[j] * a[j] * s;
                        }
                    } else if (activation == MOE_ACT_NONE) {
#pragma unroll
                        for (int j = 0; j < 8; ++j) y[j] = g[j];
                    } else {
                        float a[8];
                        unpack8(z[k][0], a);
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            y[j] = g[j] * (activation == MOE_ACT_SILU ? silu_slope(a[j], sigmoid_approx(a[j])) : gelu_slope(a[j]));
                    }
                    if constexpr (BIAS)
#pragma unroll
                        for (int j = 0; j < HALVES * 8; ++j) sum[j] += y[j];
                    if (grad_pre)
#pragma unroll
                        for (int h = 0; h < HALVES; ++h) st_v4(grad_pre + (size_t)r * N + h * C + c, pack8(y + 8 * h));
                }
            }
        if constexpr (BIAS) {
#pragma unroll
            for (int j = 0; j < HALVES * 8; ++j) red[j][threadIdx.x] = sum[j];
            __syncthreads();
            // HALVES * 8 * columns sums, thread by thread over the row lanes
            for (int k = threadIdx.x; k < HALVES * 8 * columns; k += kThreads) {
                const int j = k / columns, x = k - j * columns;
                float v = 0.0f;
                for (int y = 0; y < lanes; ++y) v += red[j][y * columns + x];
                const int at = c - tx * 8 + x * 8 + (j & 7);
                if (at < C) partial[(size_t)chunk * N + (j >> 3) * C + at] = v;
            }
            __syncthreads();
        }
    }
}

// Expert blockIdx.y's chunks: every kFinishLanes-th one by one thread, then the
// threads of a column in order.
constexpr int kFinishColumns = 64, kFinishLanes = 4;

__global__ void __launch_bounds__(kFinishColumns * kFinishLanes)
bias_finish_kernel(const int32_t *__restrict__ first_chunk, const float *__restrict__ partial, int N,
                   float *__restrict__ grad_bias)
{
    __shared__ float sums[kFinishLanes][kFinishColumns];
    pdl_wait();
    pdl_trigger();
    const int x = threadIdx.x % kFinishColumns, lane = threadIdx.x / kFinishColumns;
    const int n = blockIdx.x * kFinishColumns + x, e = blockIdx.y, last = first_chunk[e + 1];
    float v = 0.0f;
    if (n < N)
        for (int c0 = first_chunk[e] + lane; c0 < last; c0 += 8 * kFinishLanes) {
            float p[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int c = c0 + j * kFinishLanes;
                p[j] = c < last ? partial[(size_t)c * N + n] : 0.0f;
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) v += p[j];
        }
    sums[lane][x] = v;
    __syncthreads();
    if (lane == 0 && n < N) {
        for (int i = 1; i < kFinishLanes; ++i) v += sums[i][x];
        grad_bias[(size_t)e * N + n] = v;
    }
}

size_t table_bytes(int E) { return ((size_t)(E + 1) * 4 + 255) / 256 * 256; }

// Threads along a row, eight columns each: strips of at most 64, of equal width.
int columns_of(int C)
{
    const int vectors = ceil_div(C, 8), strips = ceil_div(vectors, 64);
    return ceil_div(vectors, strips);
}

// Rows a chunk: as many as still give every block one (4662 rows of 1032 columns,
// 48 experts, with the bias: 19.9 us with 128 rows, 12.9 with 32).
int rows_a_chunk(int rows, int N)
{
    int chunk = 128;
    while (chunk > 32 && (int64_t)(rows / chunk) * ceil_div(N, columns_of(N) * 8) < kBlocks) chunk /= 2;
    return chunk;
}

int64_t most_chunks(int rows, int E, int chunk) { return (int64_t)(rows < E ? rows : E) + rows / chunk; }

}  // namespace

size_t activation_backward_workspace_bytes(int rows, int N, int E)
{
    return table_bytes(E) + ((size_t)most_chunks(rows, E, rows_a_chunk(rows, N)) * N * 4 + 255) / 256 * 256;
}

cudaError_t launch_activation_backward(const void *pre, const void *grad_out, const int32_t *offsets, int rows, int N,
                                       int E, int activation, void *grad_pre, float *grad_bias, void *workspace,
                                       cudaStream_t stream)
{
    const bool gated = activation == MOE_ACT_SWIGLU;
    const int C = gated ? N / 2 : N;
    const int columns = columns_of(C), chunk = rows_a_chunk(rows, N), most = (int)most_chunks(rows, E, chunk);
    const int64_t items = (int64_t)most * ceil_div(C, columns * 8);
    const dim3 grid((unsigned)(items < 1 ? 1 : items < kBlocks ? items : kBlocks));
    int32_t *const first = static_cast<int32_t *>(workspace);
    float *const partial = grad_bias ? reinterpret_cast<float *>(static_cast<char *>(workspace) + table_bytes(E)) : nullptr;
    auto *const kernel = gated ? grad_bias ? activation_backward_kernel<true, true> : activation_backward_kernel<true, false>
                               : grad_bias ? activation_backward_kernel<false, true> : activation_backward_kernel<false, false>;
    const cudaError_t e = launch_pdl(kernel, grid, dim3(kThreads), grad_bias ? 2 * (size_t)(E + 1) * 4 : 0, stream,
                                     static_cast<const __nv_bfloat16 *>(pre), static_cast<const __nv_bfloat16 *>(grad_out),
                                     offsets, rows, N, E, activation, static_cast<__nv_bfloat16 *>(grad_pre), first, partial,
                                     most, columns, chunk);
    if (e != cudaSuccess || !grad_bias) return e;
    return launch_pdl(bias_finish_kernel, dim3(ceil_div(N, kFinishColumns), E), dim3(kFinishColumns * kFinishLanes), 0, stream,
                      first, partial, N, grad_bias);
}

}  // namespace moe
