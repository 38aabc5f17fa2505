// expert_tiles.cuh -- how the grouped matrix products cut packed rows into
// tiles: each expert's rows split evenly into tiles of at most S::NT rows, each
// tile by kChannels * S::CG output channels; and what their launches share.
#pragma once

#include <mutex>

#include "common.cuh"
#include "internal.h"
#include "moe_layout.h"
#include "tensor.cuh"

namespace moe {
namespace {

constexpr int kChannels = 128;             // channels a CTA

// One tile: the rows [row, row + valid) of expert e and the channels from
// `channel`.  CTA r of a pair has the rows from r * share; the share is
// split into parts (a sum with an accumulator of its own), and n[p] counts the
// pair's rows in part p: part 0 is the first n[0] / CG of each share.
struct Tile {
    int e, row, valid, n[2], channel;
};

// Experts' first rows and first tiles, in shared memory.
struct Table {
    const int *first_row;      // [E + 1]
    const int *first_tile;     // [E + 1]
};

// Fills the table, for a whole block of THREADS threads: tiles of NT rows an expert, then
// their running sum; thread t has PER experts in a row.  warp_tiles: a word a
// warp.  Ends with the block synchronised; tcgen05 work of before is ordered.
template <int THREADS>
__device__ __forceinline__ void fill_table(const int32_t *offsets, int rows, int E, int NT, int *first_row,
                                           int *first_tile, int *warp_tiles)
{
    constexpr int PER = MOE_MAX_EXPERTS / THREADS + 1;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int tiles[PER], before = 0, sum = 0;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        const int e = PER * tid + j;
        tiles[j] = 0;
        if (e <= E) {
            const int lo = max(0, min(rows, offsets[e]));
            first_row[e] = lo;
            if (e < E) tiles[j] = (int)((unsigned)(max(0, min(rows, offsets[e + 1]) - lo) + NT - 1) / (unsigned)NT);
        }
        sum += tiles[j];
    }
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
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        if (PER * tid + j <= E) first_tile[PER * tid + j] = before;
        before += tiles[j];
    }
    __syncthreads();
}

// Tile i, for a whole warp; at: its expert or one before it, and its expert
// afterwards.  A warp goes through its tiles in order, so the search goes on
// from the last one's expert, 32 experts a step.
template <typename S>
__device__ __forceinline__ Tile tile_of(const Table &t, int E, int channel_tiles, int i, int &at)
{
    const int tt = (int)((unsigned)i / (unsigned)channel_tiles);
    for (unsigned passed = kFullMask; passed == kFullMask; at += __popc(passed)) {
        const int e = at + 1 + (int)(threadIdx.x & 31);
        passed = __ballot_sync(kFullMask, e < E && t.first_tile[e] <= tt);
    }
    const int lo = at;                                 // first_tile[lo] <= tt < first_tile[lo + 1]
    const int base = t.first_tile[lo], tiles = t.first_tile[lo + 1] - base;
    const int rows = t.first_row[lo + 1] - t.first_row[lo];
    // an expert's rows are split evenly; a share is at most NT, so no tile is empty
    const int share = ceil_div((int)((unsigned)(rows + tiles - 1) / (unsigned)tiles), S::QUANTUM) * S::QUANTUM;
    Tile r;
    r.e = uniform(lo);
    r.row = uniform(t.first_row[lo] + (tt - base) * share);
    r.valid = uniform(min(share, rows - (tt - base) * share));
    const int n = ceil_div(r.valid, S::QUANTUM) * S::QUANTUM;
    r.n[0] = S::PARTS == 1 ? n : ceil_div(n, 2 * S::QUANTUM) * S::QUANTUM;
    r.n[1] = n - r.n[0];
    r.channel = (i - tt * channel_tiles) * kChannels * S::CG;
    return r;
}

// Tiles of rows there can be at most: every expert's last one may be short.
template <typename S>
int64_t most_tiles(int rows, int E)
{
    return (int64_t)(rows < E ? rows : E) + rows / S::NT;
}

// Clusters of 2, 4 and 8 CTAs of KERNEL that the current device runs at a time,
// looked up once for each device.
template <auto *KERNEL>
cudaError_t split_clusters(int threads, size_t smem, int (&clusters)[3])
{
    constexpr int kMaxDevices = 64;
    static std::mutex mu;
    static int known[kMaxDevices][3];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    const std::lock_guard<std::mutex> lock(mu);
    for (int i = 0; i < 3; ++i) {
        int &n = known[dev][i];
        if (n == 0) {
            e = allow_dynamic_smem(reinterpret_cast<const void *>(KERNEL), smem);
            if (e != cudaSuccess) return e;
            cudaLaunchConfig_t cfg = {};
            cfg.gridDim = dim3(2 << i);
            cfg.blockDim = dim3(threads);
            cfg.dynamicSmemBytes = smem;
            cudaLaunchAttribute attr;
            attr.id = cudaLaunchAttributeClusterDimension;
            attr.val.clusterDim.x = 2u << i;
            attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
            cfg.attrs = &attr;
            cfg.numAttrs = 1;
            e = cudaOccupancyMaxActiveClusters(&n, KERNEL, &cfg);
            if (e != cudaSuccess) return e;
        }
        clusters[i] = n;
    }
    return cudaSuccess;
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

// A tensor map of boxes of 128-byte lines, swizzled, zeros outside.  Unlike a launch
// the driver's call does not make the device's context the calling thread's, and
// fails in a thread that has none yet (autograd's, whose first work is a gradient
// here): cudaSetDevice does, and the call is made again.
bool encode_tiled(CUtensorMap *map, CUtensorMapDataType type, int rank, const void *p, const cuuint64_t *dims,
                  const cuuint64_t *strides, const cuuint32_t *box)
{
    static const cuuint32_t ones[4] = {1, 1, 1, 1};
    const EncodeFn fn = encode_fn();
    if (!fn) return false;
    auto encode = [&] {
        return fn(map, type, rank, const_cast<void *>(p), dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
    };
    if (encode()) return true;
    int dev = 0;
    return cudaGetDevice(&dev) == cudaSuccess && cudaSetDevice(dev) == cudaSuccess && encode();
}

}  // namespace
}  // namespace moe
