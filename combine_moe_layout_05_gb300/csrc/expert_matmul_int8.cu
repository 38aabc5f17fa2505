// expert_matmul_int8.cu -- packed int8 rows times their experts' int8
// weights, with a scale for each row and each output channel.
//
//   out[r, n] = bf16((sum_h x[r, h] * w[e, n, h]) * x_scale[r] * w_scale[e, n])
//   for the rows r of expert e, [offsets[e], offsets[e+1])
//
// sm_103a has no 8-bit integer matrix instruction of the tcgen05 kind, and an
// int8 value is exactly a fp16 value: the codes travel as bytes through HBM,
// L2 and the copies into shared memory, and are widened on the way to the
// fp16 tensor cores.  A product is below 2^14 and the fp32 accumulator exact
// up to 2^24, so the sum is the integer's while partial sums stay below that.
//
// A tile is 128 channels a CTA (256 a pair of CTAs) by up to NT rows of one
// expert.  Channels are the instruction's M, so that a tile with few rows
// still feeds it 128 lanes; the row count is its N and is what the expert has
// left, rounded up.  Warps of a CTA:
//
//   one copies 128-byte-wide tiles of weights and rows into a ring;
//   one issues the matrix instructions (the pair's first CTA's);
//   4 GA widen the weights into TMEM (operand A), one channel a thread;
//   WB GB widen the rows into shared memory (operand B), one row a thread;
//   four scale the sums and store them, one channel a thread.
//
// A pair shares each other's widened rows: every CTA widens half of the tile's
// rows, which is what keeps shared memory from being the bound (a 128-wide
// step of a full tile moves 16 KB in, 32 KB through the widening warps and
// 32 KB into the tensor core, in 1024 cycles of the instruction).
#include "common.cuh"
#include "internal.h"
#include "moe_layout.h"
#include "tensor.cuh"

#include <mutex>

namespace moe {
namespace {

constexpr int kStep = 128;                 // bytes of the contraction a ring slot holds
constexpr int kHalf = 64;                  // of them in a slot of widened operands
constexpr int kChannels = 128;             // channels a CTA
constexpr int kTmemColumns = 512;

// CG: CTAs a tile.  NT: rows a tile at most.  N8: ring slots of int8 tiles.
// NC: slots of widened operands.  ND: accumulators.  GA, GB: groups of warps
// that widen the weights and the rows; a group takes every GA-th (GB-th) step,
// since one step's latency (barrier, loads, stores and their wait) is several
// times its issue slots.
template <int CG_, int NT_, int N8_, int NC_, int ND_, int GA_, int GB_>
struct Shape {
    static constexpr int CG = CG_, NT = NT_, N8 = N8_, NC = NC_, ND = ND_, GA = GA_, GB = GB_;
    static constexpr int BR = NT / CG;                 // rows a CTA widens at most
    static constexpr int BOX = CG == 2 ? 32 : 16;      // rows a copy
    static constexpr int QUANTUM = CG == 2 ? 32 : 16;  // rows of a tile are a multiple of
    static constexpr int A8 = kChannels * kStep, B8 = BR * kStep, B16 = BR * kHalf * 2;
    static constexpr int SLOT8 = A8 + B8;
    static constexpr int ACOL = kHalf / 2;             // TMEM columns of a widened slot
    static_assert(ND * NT + NC * ACOL <= kTmemColumns);
    // warps: 0 copies, 1 issues, then those that widen and those that store;
    // the TMEM lanes a warp reaches are those of its number modulo 4
    static constexpr int WB = BR / 32;                 // warps of a group that widens rows
    static constexpr int A0 = 4, E0 = A0 + 4 * GA, B0 = WB * GB <= 2 ? 2 : E0 + 4;
    static constexpr int WARPS = B0 == 2 ? E0 + 4 : B0 + WB * GB;
    static constexpr int THREADS = WARPS * 32;
    static constexpr int BARS = 2 * N8 + 2 * NC + 2 * ND + 1;
    // ring, widened rows, 16 x 32 outputs and the row scales of each storing
    // warp, barriers, flags, expert table
    static constexpr int OFF16 = N8 * SLOT8;
    static constexpr int OFFTURN = OFF16 + NC * B16;
    static constexpr int OFFS = OFFTURN + 4 * 1024;
    static constexpr int OFFBAR = OFFS + 4 * NT * 4;
    static constexpr int OFFTAB = OFFBAR + (BARS * 8 + 15) / 16 * 16 + 32;
    static constexpr int bytes(int E) { return OFFTAB + 2 * (E + 1) * 4 + 1024; }
};
using Wide = Shape<2, 256, 3, 6, 1, 2, 2>;
using Narrow = Shape<1, 32, 8, 12, 2, 4, 2>;

// One tile: the rows [row, row + valid) of expert e, `n` of them after
// rounding up, and the channels from `channel`.
struct Tile {
    int e, row, valid, n, channel;
};

// Experts' first rows and first tiles, in shared memory.
struct Table {
    const int *first_row;      // [E + 1]
    const int *first_tile;     // [E + 1]
};

template <typename S>
__device__ __forceinline__ Tile tile_of(const Table &t, int E, int channel_tiles, int i)
{
    const int tt = i / channel_tiles;
    int lo = 0, hi = E;                                // first_tile[lo] <= tt < first_tile[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (t.first_tile[mid] <= tt) lo = mid;
        else hi = mid;
    }
    const int base = t.first_tile[lo], tiles = t.first_tile[lo + 1] - base;
    const int rows = t.first_row[lo + 1] - t.first_row[lo];
    // an expert's rows are split evenly; a share is at most NT, so no tile is empty
    const int share = ceil_div(ceil_div(rows, tiles), S::QUANTUM) * S::QUANTUM;
    Tile r;
    r.e = lo;
    r.row = t.first_row[lo] + (tt - base) * share;
    r.valid = min(share, rows - (tt - base) * share);
    r.n = ceil_div(r.valid, S::QUANTUM) * S::QUANTUM;
    r.channel = (i - tt * channel_tiles) * kChannels * S::CG;
    return r;
}

// Four int8 codes to four fp16: with its sign bit flipped a code is b + 128,
// which below 0x64 is the fp16 1024 + (b + 128); 1152 off is exact.
__device__ __forceinline__ void widen4(uint32_t w, uint32_t &lo, uint32_t &hi)
{
    const uint32_t u = w ^ 0x80808080u;
    const uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
    const __half2 c = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));
    const __half2 x = __hsub2(*reinterpret_cast<const __half2 *>(&a), c);
    const __half2 y = __hsub2(*reinterpret_cast<const __half2 *>(&b), c);
    lo = *reinterpret_cast<const uint32_t *>(&x);
    hi = *reinterpret_cast<const uint32_t *>(&y);
}

__device__ __forceinline__ uint4 lds128(uint32_t addr)
{
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
    return v;
}

__device__ __forceinline__ void sts128(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d)
{
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" :: "r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

template <typename S>
__global__ void __launch_bounds__(S::THREADS, 1)
expert_matmul_int8_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_x,
                          const float *__restrict__ x_scales, const float *__restrict__ w_scales,
                          const int32_t *__restrict__ offsets, int rows, int H, int N, int E,
                          __nv_bfloat16 *__restrict__ out, uint32_t *__restrict__ dev_error)
{
    extern __shared__ uint8_t raw[];
    const uint32_t base = (smem_addr(raw) + 1023) & ~1023u;
    uint8_t *const generic = raw + (base - smem_addr(raw));
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t rank = S::CG == 2 ? cluster_rank() : 0;

    const uint32_t bar0 = base + S::OFFBAR;
    auto full8 = [&](int i) { return bar0 + 8 * i; };
    auto empty8 = [&](int i) { return bar0 + 8 * (S::N8 + i); };
    auto full16 = [&](int i) { return bar0 + 8 * (2 * S::N8 + i); };
    auto empty16 = [&](int i) { return bar0 + 8 * (2 * S::N8 + S::NC + i); };
    auto full_d = [&](int i) { return bar0 + 8 * (2 * S::N8 + 2 * S::NC + i); };
    auto empty_d = [&](int i) { return bar0 + 8 * (2 * S::N8 + 2 * S::NC + S::ND + i); };
    const uint32_t drained = bar0 + 8 * (S::BARS - 1);
    uint32_t *const flags = reinterpret_cast<uint32_t *>(generic + S::OFFBAR + (S::BARS * 8 + 15) / 16 * 16);
    volatile int *const abort = reinterpret_cast<volatile int *>(flags + 1);
    int *const first_row = reinterpret_cast<int *>(generic + S::OFFTAB);
    int *const first_tile = first_row + E + 1;

    if (tid == 0) {
        prefetch_map(&map_w);
        prefetch_map(&map_x);
        uint64_t *b = reinterpret_cast<uint64_t *>(generic + S::OFFBAR);
        for (int i = 0; i < S::N8; ++i) mbar_init(b + i, 1), mbar_init(b + S::N8 + i, 4 + S::WB);
        b += 2 * S::N8;
        for (int i = 0; i < S::NC; ++i) mbar_init(b + i, (4 + S::WB) * S::CG), mbar_init(b + S::NC + i, 1);
        b += 2 * S::NC;
        for (int i = 0; i < S::ND; ++i) mbar_init(b + i, 1), mbar_init(b + S::ND + i, 4 * S::CG);
        mbar_init(b + 2 * S::ND, 1);
        *abort = 0;
        fence_barrier_init();
    }
    if (warp == 1) tmem_alloc<S::CG>(smem_addr(flags), kTmemColumns);
    pdl_wait();
    pdl_trigger();

    // Tiles an expert, then their running sum: thread t has experts 2t, 2t + 1.
    {
        static_assert(2 * S::THREADS > MOE_MAX_EXPERTS);
        __shared__ int warp_tiles[S::WARPS];
        int tiles[2], before = 0;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int e = 2 * tid + j;
            tiles[j] = 0;
            if (e <= E) {
                const int lo = max(0, min(rows, offsets[e]));
                first_row[e] = lo;
                if (e < E) tiles[j] = ceil_div(max(0, min(rows, offsets[e + 1]) - lo), S::NT);
            }
        }
        int sum = tiles[0] + tiles[1];
        const int mine = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(kFullMask, sum, o);
            if (lane >= o) sum += v;
        }
        if (lane == 31) warp_tiles[warp] = sum;
        tc_fence_before();
        __syncthreads();
        for (int w = 0; w < warp; ++w) before += warp_tiles[w];
        before += sum - mine;
        if (2 * tid <= E) first_tile[2 * tid] = before;
        if (2 * tid + 1 <= E) first_tile[2 * tid + 1] = before + tiles[0];
    }
    if (dev_error && blockIdx.x == 0 && tid == 0) *dev_error = 0;
    __syncthreads();
    if constexpr (S::CG == 2) cluster_sync_all();
    tc_fence_after();
    const uint32_t tmem = flags[0];

    const Table table{first_row, first_tile};
    const int channel_tiles = ceil_div(N, kChannels * S::CG);
    const int items = first_tile[E] * channel_tiles;
    const int steps = ceil_div(H, kStep), halves = 2 * steps;
    uint64_t *const bars = reinterpret_cast<uint64_t *>(generic + S::OFFBAR);
    const int group = blockIdx.x / S::CG, groups = gridDim.x / S::CG;

    if (warp == 0) {
        int issued = 0;
        bool ok = true;
        for (int i = group; i < items && ok; i += groups) {
            const Tile t = tile_of<S>(table, E, channel_tiles, i);
            const int half = t.n / S::CG, boxes = ceil_div(half, S::BOX);
            const int wr = t.e * N + t.channel + (int)rank * kChannels, xr = t.row + (int)rank * half;
            const uint32_t bytes = S::A8 + boxes * S::BOX * kStep;
            for (int k = 0; k < steps; ++k, ++issued) {
                const int s = issued % S::N8;
                ok = __all_sync(kFullMask, mbar_wait_bounded(empty8(s), (issued / S::N8 & 1) ^ 1, abort));
                if (!ok) break;
                const uint32_t slot = base + s * S::SLOT8;
                if (elect_one()) {
                    mbar_arrive_expect(bars + s, bytes);
                    tile_load_2d(slot, &map_w, k * kStep, wr, full8(s));
                    for (int b = 0; b < boxes; ++b)
                        tile_load_2d(slot + S::A8 + b * S::BOX * kStep, &map_x, k * kStep, xr + b * S::BOX, full8(s));
                }
                __syncwarp();
            }
        }
        if (!ok)                                       // the copies in flight land first
            for (int j = max(0, issued - S::N8); j < issued; ++j)
                mbar_drain_bounded(full8(j % S::N8), j / S::N8 & 1);
    } else if (warp == 1) {
        if (rank == 0) {
            int c = 0, d = 0;
            bool ok = true;
            for (int i = group; i < items && ok; i += groups, ++d) {
                const Tile t = tile_of<S>(table, E, channel_tiles, i);
                const uint32_t idesc = instruction_desc_f16(kChannels * S::CG, t.n);
                const uint32_t acc = tmem + d % S::ND * S::NT;
                ok = __all_sync(kFullMask, mbar_wait_bounded(empty_d(d % S::ND), (d / S::ND & 1) ^ 1, abort));
                if (!ok) break;
                tc_fence_after();
                for (int k = 0; k < halves; ++k, ++c) {
                    const int s = c % S::NC;
                    ok = __all_sync(kFullMask, mbar_wait_bounded(full16(s), c / S::NC & 1, abort));
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t a = tmem + S::ND * S::NT + s * S::ACOL;
                    const uint64_t b = operand_desc(base + S::OFF16 + s * S::B16);
                    const int subs = min(4, (H - k * kHalf) >> 4);
                    if (elect_one()) {
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            if (j < subs) mma_f16_ts<S::CG>(acc, a + 8 * j, b + 2 * j, idesc, (k | j) != 0);
                        mma_commit<S::CG>(empty16(s));
                        if (k == halves - 1) mma_commit<S::CG>(full_d(d % S::ND));
                    }
                    __syncwarp();
                }
            }
            if (!ok) {                                 // what was issued finishes first
                if (elect_one()) mma_commit<S::CG>(drained);
                __syncwarp();
                mbar_drain_bounded(drained, 0);
            }
        }
    } else if (warp >= S::E0 && warp < S::E0 + 4) {
        const int quarter = warp & 3;
        float *const row_scale = reinterpret_cast<float *>(generic + S::OFFS) + quarter * S::NT;
        __nv_bfloat16 *const turned = reinterpret_cast<__nv_bfloat16 *>(generic + S::OFFTURN) + quarter * 512;
        const bool vector_out = N % 8 == 0;
        int d = 0;
        bool ok = true;
        for (int i = group; i < items && ok; i += groups, ++d) {
            const Tile t = tile_of<S>(table, E, channel_tiles, i);
            const int ch = t.channel + (int)rank * kChannels + quarter * 32 + lane;
            __syncwarp();                              // the last tile's scales have been read
            float xs[S::NT / 32];
#pragma unroll
            for (int j = 0; j < S::NT / 32; ++j)
                xs[j] = j * 32 + lane < t.valid ? x_scales[t.row + j * 32 + lane] : 0.0f;
            const float ws = ch < N ? w_scales[(size_t)t.e * N + ch] : 0.0f;
#pragma unroll
            for (int j = 0; j < S::NT / 32; ++j) row_scale[j * 32 + lane] = xs[j];
            __syncwarp();
            ok = __all_sync(kFullMask, mbar_wait_bounded(full_d(d % S::ND), d / S::ND & 1, abort));
            if (!ok) break;
            tc_fence_after();
            const uint32_t acc = tmem + d % S::ND * S::NT + ((uint32_t)quarter << 21);
            const int ch0 = ch - lane;
            const bool vectors = vector_out && ch0 + 32 <= N;
            for (int c0 = 0; c0 < t.n; c0 += 16) {
                uint32_t v[16];
                tmem_load_x16(acc + c0, v);
                tmem_wait_ld();
                if (c0 + 16 >= t.n) {                  // all read: the accumulator is free
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive_pair(S::CG == 2 ? cluster_addr(empty_d(d % S::ND), 0) : empty_d(d % S::ND));
                }
                __nv_bfloat16 y[16];
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    y[j] = __float2bfloat16_rn(__uint_as_float(v[j]) * row_scale[c0 + j] * ws);
                if (vectors) {
                    // 16 rows of 32 channels turned in shared memory, then 16 bytes a lane
#pragma unroll
                    for (int j = 0; j < 16; ++j) turned[j * 32 + lane] = y[j];
                    __syncwarp();
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const int r = c0 + j * 8 + (lane >> 2);
                        const uint4 q = reinterpret_cast<const uint4 *>(turned)[j * 32 + lane];
                        if (r < t.valid) st_v4(out + (size_t)(t.row + r) * N + ch0 + (lane & 3) * 8, q);
                    }
                    __syncwarp();
                } else if (ch < N) {
                    __nv_bfloat16 *o = out + (size_t)(t.row + c0) * N + ch;
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        if (c0 + j < t.valid) o[(size_t)j * N] = y[j];
                }
            }
        }
    } else if (warp >= S::A0 && warp < S::E0) {
        // weights: group `g` has every GA-th step, and in it a thread one channel
        const int g = (warp - S::A0) >> 2, r = (warp & 3) * 32 + lane;
        int n = 0;
        bool ok = true;
        for (int i = group; i < items && ok; i += groups)
            for (int k = 0; k < steps && ok; ++k, ++n) {
                if (n % S::GA != g) continue;
                const int s = n % S::N8;
                ok = __all_sync(kFullMask, mbar_wait_bounded(full8(s), n / S::N8 & 1, abort));
                const uint32_t src = base + s * S::SLOT8 + r * kStep;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int m = 2 * n + h, c = m % S::NC;
                    if (!ok) break;
                    uint32_t v[32];
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const uint4 x = lds128(src + (((4 * h + q) ^ (r & 7)) << 4));
                        widen4(x.x, v[8 * q], v[8 * q + 1]);
                        widen4(x.y, v[8 * q + 2], v[8 * q + 3]);
                        widen4(x.z, v[8 * q + 4], v[8 * q + 5]);
                        widen4(x.w, v[8 * q + 6], v[8 * q + 7]);
                    }
                    ok = __all_sync(kFullMask, mbar_wait_bounded(empty16(c), (m / S::NC & 1) ^ 1, abort));
                    if (!ok) break;
                    tc_fence_after();
                    tmem_store_x32(tmem + S::ND * S::NT + c * S::ACOL + ((uint32_t)(warp & 3) << 21), v);
                    if (h == 1 && lane == 0) mbar_arrive(bars + S::N8 + s);
                    tmem_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_pair(S::CG == 2 ? cluster_addr(full16(c), 0) : full16(c));
                }
            }
        for (int j = max(0, 2 * n - S::NC); j < 2 * n && ok; ++j)     // the last slots' arrivals are in
            ok = __all_sync(kFullMask, mbar_wait_bounded(empty16(j % S::NC), j / S::NC & 1, abort));
    } else if (warp >= S::B0 && warp < S::B0 + S::WB * S::GB) {
        // rows: group `g` has every GB-th step, and in it a thread one row
        const int g = (warp - S::B0) / S::WB, r = (warp - S::B0) % S::WB * 32 + lane;
        int n = 0;
        bool ok = true;
        for (int i = group; i < items && ok; i += groups) {
            const bool live = r < tile_of<S>(table, E, channel_tiles, i).n / S::CG;
            for (int k = 0; k < steps && ok; ++k, ++n) {
                if (n % S::GB != g) continue;
                const int s = n % S::N8;
                ok = __all_sync(kFullMask, mbar_wait_bounded(full8(s), n / S::N8 & 1, abort));
                const uint32_t src = base + s * S::SLOT8 + S::A8 + r * kStep;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int m = 2 * n + h, c = m % S::NC;
                    if (!ok) break;
                    uint32_t v[32];
                    if (live) {
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            const uint4 x = lds128(src + (((4 * h + q) ^ (r & 7)) << 4));
                            widen4(x.x, v[8 * q], v[8 * q + 1]);
                            widen4(x.y, v[8 * q + 2], v[8 * q + 3]);
                            widen4(x.z, v[8 * q + 4], v[8 * q + 5]);
                            widen4(x.w, v[8 * q + 6], v[8 * q + 7]);
                        }
                    }
                    ok = __all_sync(kFullMask, mbar_wait_bounded(empty16(c), (m / S::NC & 1) ^ 1, abort));
                    if (!ok) break;
                    if (live) {
                        const uint32_t dst = base + S::OFF16 + c * S::B16 + r * 128;
#pragma unroll
                        for (int q = 0; q < 8; ++q)
                            sts128(dst + ((q ^ (r & 7)) << 4), v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
                        fence_async_shared();
                    }
                    __syncwarp();
                    if (lane == 0) {
                        if (h == 1) mbar_arrive(bars + S::N8 + s);
                        mbar_arrive_pair(S::CG == 2 ? cluster_addr(full16(c), 0) : full16(c));
                    }
                }
            }
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if constexpr (S::CG == 2) cluster_sync_all();      // the peer is done with this CTA's memory
    tc_fence_after();
    if (tid == 0 && *abort && dev_error) atomicOr(dev_error, MOE_DEV_ERR_TIMEOUT);
    if (warp == 1) tmem_free<S::CG>(tmem, kTmemColumns);
}

using EncodeFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                              const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                              CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encode_fn()
{
    static std::once_flag once;
    static EncodeFn fn = nullptr;
    std::call_once(once, [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeFn>(p);
    });
    return fn;
}

// [rows, H] bytes, in boxes of kStep bytes by `box` rows, 128-byte swizzle.
bool byte_map(CUtensorMap *map, const void *p, uint64_t rows, uint64_t H, uint32_t box)
{
    const EncodeFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[2] = {H, rows}, strides[1] = {H};
    const cuuint32_t boxes[2] = {kStep, box}, ones[2] = {1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(p), dims, strides, boxes, ones,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename S>
cudaError_t run(const void *x, const float *x_scales, const void *w, const float *w_scales,
                const int32_t *offsets, int rows, int H, int N, int E, void *out, uint32_t *dev_error,
                cudaStream_t stream)
{
    CUtensorMap map_w, map_x;
    if (!byte_map(&map_w, w, (uint64_t)E * N, H, kChannels) || !byte_map(&map_x, x, rows, H, S::BOX))
        return cudaErrorInvalidValue;
    const size_t smem = S::bytes(E);
    cudaError_t e = allow_dynamic_smem(reinterpret_cast<const void *>(&expert_matmul_int8_kernel<S>), smem);
    if (e != cudaSuccess) return e;
    int sms = 0;
    e = device_sm_count(&sms);
    if (e != cudaSuccess) return e;
    // tiles there can be at most: every expert's last one may be short
    const int64_t most = ((int64_t)(rows < E ? rows : E) + rows / S::NT) * ceil_div(N, kChannels * S::CG);
    const int64_t groups = most < sms / S::CG ? most : sms / S::CG;
    return launch_pdl_clusters(expert_matmul_int8_kernel<S>, dim3((unsigned)groups * S::CG), dim3(S::THREADS), smem,
                               stream, S::CG, map_w, map_x, x_scales, w_scales, offsets, rows, H, N, E,
                               static_cast<__nv_bfloat16 *>(out), dev_error);
}

}  // namespace

cudaError_t launch_expert_matmul_int8(const void *x, const float *x_scales, const void *w,
                                      const float *w_scales, const int32_t *offsets, int rows,
                                      int H, int N, int E, void *out, uint32_t *dev_error,
                                      cudaStream_t stream)
{
    if (rows <= (int64_t)Narrow::NT * E)
        return run<Narrow>(x, x_scales, w, w_scales, offsets, rows, H, N, E, out, dev_error, stream);
    return run<Wide>(x, x_scales, w, w_scales, offsets, rows, H, N, E, out, dev_error, stream);
}

}  // namespace moe
