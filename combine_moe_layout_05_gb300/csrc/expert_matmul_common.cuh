// expert_matmul_common.cuh -- the grouped bf16 products of the experts on the
// fifth-generation tensor cores: one kernel for the forward product and its
// two gradients.
//
//   kForward  out[r, c]     = act(sum_h x[r, h] w[e, c, h] + bias[e, c]) + residual[r, c]
//   kRows     grad_x[r, h]  = sum_n grad_pre[r, n] w[e, n, h]
//   kWeights  grad_w[e, n, h] = sum over e's rows r of grad_pre[r, n] x[r, h]
//
// In each the instruction's M are 128 "channels" a CTA (256 a pair): output
// channels, the hidden size, or (kWeights) the weights' rows; an expert with one
// row still feeds 128 lanes.  Its N are a tile's "rows": packed rows, or (kWeights)
// the hidden size, as many as are left, rounded up.  Operands lie in shared
// memory as the copy engine's 128-byte swizzle leaves them, in the order that
// global memory has: along the contraction (K-major) for x and the forward
// weights, across it (MN-major) for the weights in kRows and for both operands in
// kWeights.
//
// Warps of a CTA: one copies 64-wide steps of both operands into a ring; one
// issues the matrix instructions (the pair's first CTA's); in a pair one tells
// the first CTA that a step has landed, and in kWeights clears the rows of the
// next expert in an expert's last step; 4 SETS add the bias, activate, add the
// residual, turn the sums in shared memory and store them, while the other
// accumulator is summed.  In kWeights a lane of the sums is a row of the output,
// which goes to memory as whole lines.
//
// What bounds it: the tensor cores where an expert has some 350 rows (16384 rows,
// 16 experts, 4096 -> 4096 gated: their pipe is busy 96.7 % of active cycles forward,
// 95 % in the rows' gradient), the weights' bytes below that.  256 rows by 256
// channels a pair read 128 operations a byte from L2, which feeds that rate; the
// ring is what is left of shared memory.  131072 skewed rows over 128 experts,
// 4096 -> 4096 gated: 2.47 ms in a burst (1.78 PFLOP/s), 2.9 under the power cap
// (1.5); 1024 rows over 256 experts, 7168 -> 4096 gated: 2.0 ms, 7.4 TB/s of
// weights.  Gradients of the first: rows 2.49 ms, weights 2.69 (a ring of 5); of
// the second: 2.1 and 2.5 ms.
//
// Tiles of several experts at a time, so that memory-bound and compute-bound ones
// overlap, lost 9 % and more: weights no longer stay in L2 from tile to tile.
#pragma once

#include "activation.cuh"
#include "expert_tiles.cuh"

namespace moe {
namespace {

enum Pass { kForward, kRows, kWeights };

constexpr int kStep = 64;                  // of the contraction a ring slot holds: a swizzled line of bf16
constexpr int kMaxShared = 227 * 1024;

// CG: CTAs a tile.  NT: rows a tile at most.  STAGES: slots of the ring.
// GATED: the channels come in pairs (gate and up), 16 of each in 32 lanes.
// SPLIT: a cluster's CTAs each sum a share of the contraction.
template <Pass PASS_, bool GATED_, int CG_, int NT_, int STAGES_, int SETS_, bool SPLIT_ = false>
struct Shape {
    static constexpr Pass PASS = PASS_;
    static constexpr bool GATED = GATED_, SPLIT = SPLIT_;
    static constexpr int CG = CG_, NT = NT_, STAGES = STAGES_, PARTS = 1;
    static constexpr int BR = NT / CG;                 // rows a CTA copies at most
    static constexpr int QUANTUM = 16 * CG;            // rows of a tile are a multiple of
    static constexpr bool A_MN = PASS != kForward, B_MN = PASS == kWeights;
    static_assert(!SPLIT || (CG == 1 && PASS == kForward));
    static_assert(!B_MN || (CG == 2 && BR == 128));
    static_assert(!GATED || PASS == kForward);
    static constexpr int A = kChannels * kStep * 2, B = BR * kStep * 2, SLOT = A + B;
    static constexpr int OUT = GATED ? kChannels / 2 : kChannels;      // output channels a CTA
    static constexpr int SETS = SETS_;                 // sets of four warps that store, by turns of 16 rows
    static constexpr int E0 = 4, WARPS = E0 + 4 * SETS, THREADS = WARPS * 32;
    static constexpr int BARS = 3 * STAGES + 4 + 1 + SPLIT;
    static constexpr int TMEM = 2 * NT;                // two accumulators
    static_assert((TMEM & (TMEM - 1)) == 0 && TMEM >= 32 && TMEM <= 512);
    // ring, 16 x 32 outputs (kWeights: 32 lines) of each storing warp, the other
    // CTAs' sums (SPLIT: NT x 128 fp32), barriers, flags, expert table
    static constexpr int TURN = PASS == kWeights ? 4096 : 1024;
    static constexpr int OFFTURN = STAGES * SLOT;
    static constexpr int OFFBOX = OFFTURN + 4 * SETS * TURN;
    static constexpr int OFFBAR = OFFBOX + SPLIT * NT * kChannels * 4;
    static constexpr int OFFTAB = OFFBAR + (BARS * 8 + 15) / 16 * 16 + 32;
    static constexpr int bytes(int E) { return OFFTAB + 2 * (E + 1) * 4; }
    static_assert(bytes(MOE_MAX_EXPERTS) <= kMaxShared);
    static_assert(WARPS * 4 <= 4 * SETS * TURN);
    static_assert(OFFTURN % 1024 == 0);
};

// Copies of rows come in these heights; a tile takes the one that covers its share.
constexpr int kBoxes = 4, kLeastBox = 16;
struct RowMaps {
    CUtensorMap box[kBoxes];    // 16, 32, 64, 128 rows; kWeights: 64 x 64, and the output's
};

// What is stored, and where.
struct Store {
    const float *bias;              // [E, N] or null
    const __nv_bfloat16 *residual;  // [rows, channels] or null; may be out
    __nv_bfloat16 *pre;             // [rows, N] or null
    void *out;
    int activation;                 // MOE_ACT_*
    int f32, accumulate;            // kWeights: out is fp32; is added to
};

// The sizes of a product.  N: the weights' rows an expert.  channels: the length
// of an output row.  depth: the contraction's length (kWeights: each expert's rows).
struct Sizes {
    int rows, N, channels, depth, E;
};

// One tile: columns [row, row + valid) of the instruction's N, padded to n, of
// which CTA r of a pair has those from r * share; the contraction from `first`
// on in `steps` steps, with `tail` left in the last one.
struct Job {
    int e, row, valid, n, share, channel, first, steps, tail;
};

template <typename S>
__device__ __forceinline__ Job job_of(const Table &t, const Sizes &z, int channel_tiles, int row_tiles, int i, int &at)
{
    Job j;
    if constexpr (S::PASS == kWeights) {
        // tiles of the same rows of the weights follow each other: they are written
        // about together, and memory likes its rows whole
        const int q = (int)((unsigned)i / (unsigned)row_tiles);
        j.e = (int)((unsigned)q / (unsigned)channel_tiles);
        j.row = (i - q * row_tiles) * S::NT;
        j.valid = min(S::NT, z.channels - j.row);
        j.share = ceil_div(j.valid, 128) * 64;
        j.n = 2 * j.share;
        j.channel = (q - j.e * channel_tiles) * S::OUT * S::CG;
        j.first = uniform(t.first_row[j.e]);
        const int count = max(0, uniform(t.first_row[j.e + 1]) - j.first);
        j.steps = (int)((unsigned)(count + kStep - 1) / kStep);
        j.tail = count - (j.steps - 1) * kStep;
    } else {
        const Tile r = tile_of<S>(t, z.E, channel_tiles, i, at);
        j.e = r.e;
        j.row = r.row;
        j.valid = r.valid;
        j.n = r.n[0];
        j.share = j.n / S::CG;
        j.channel = r.channel / (kChannels / S::OUT);
        j.first = 0;
        j.steps = ceil_div(z.depth, kStep);
        j.tail = z.depth - (j.steps - 1) * kStep;
    }
    return j;
}

// The barrier that a test holds back in the first tile's CTAs: the first of a
// kind (0 to 5: a step landed, its slot free, landed in both CTAs, sums ready,
// sums stored, the other CTAs' sums), or none.
template <typename S>
__device__ __forceinline__ int stalled_barrier(int kind)
{
    if (kind < 0 || kind >= 5 + S::SPLIT) return -1;
    if (kind < 3) return kind * S::STAGES;
    return 3 * S::STAGES + (kind == 3 ? 0 : kind == 4 ? 2 : 5);
}

// 16 rows of 32 lanes in shared memory: 64 bytes a row, its 16-byte pieces permuted.
__device__ __forceinline__ uint32_t piece_at(uint32_t turned, int r, int piece)
{
    return turned + r * 64 + ((piece ^ (r >> 1 & 3)) << 4);
}

// Of 16 rows the first `left`, or all, LANES lanes wide, to channels from ch0 on (below
// `channels`) of `to`, which points at the first row.  TWO: the upper half of
// the lanes belongs `channels` further on.  A lane reads and writes the same
// elements in load_rows and store_rows, so that both may be one tensor.
template <int LANES, bool TWO>
__device__ __forceinline__ void store_rows(uint32_t turned, __nv_bfloat16 *to, int ld, int left, int ch0, int channels,
                                           bool vectors)
{
    const int lane = threadIdx.x & 31;
    constexpr int SPAN = TWO ? LANES / 2 : LANES;      // channels of one run of columns
    if (vectors) {
        constexpr int PIECES = LANES / 8, PER = 32 / PIECES;
#pragma unroll
        for (int j = 0; j < 16 / PER; ++j) {
            const int r = PER * j + lane / PIECES, p = lane % PIECES, c = ch0 + 8 * p % SPAN;
            if (r < left && c < channels)
                st_v4(to + (size_t)r * ld + c + (TWO && 8 * p >= SPAN ? channels : 0), lds128(piece_at(turned, r, p)));
        }
    } else {
        const int c = ch0 + lane % SPAN;
        if (lane < LANES && c < channels) {
            __nv_bfloat16 *o = to + c + (TWO && lane >= SPAN ? channels : 0);
            for (int r = 0; r < min(16, left); ++r, o += ld) {
                uint16_t v;
                asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(piece_at(turned, r, lane >> 3) + (lane & 7) * 2));
                *reinterpret_cast<uint16_t *>(o) = v;
            }
        }
    }
}

template <int LANES>
__device__ __forceinline__ void load_rows(uint32_t turned, const __nv_bfloat16 *from, int ld, int left, int ch0,
                                          int channels, bool vectors)
{
    const int lane = threadIdx.x & 31;
    if (vectors) {
        constexpr int PIECES = LANES / 8, PER = 32 / PIECES;
#pragma unroll
        for (int j = 0; j < 16 / PER; ++j) {
            const int r = PER * j + lane / PIECES, p = lane % PIECES, c = ch0 + 8 * p;
            uint4 v = {0, 0, 0, 0};
            if (r < left && c < channels) v = *reinterpret_cast<const uint4 *>(from + (size_t)r * ld + c);
            sts128(piece_at(turned, r, p), v.x, v.y, v.z, v.w);
        }
    } else if (lane < LANES) {
        const int c = ch0 + lane;
        for (int r = 0; r < 16; ++r) {
            const uint16_t v = r < left && c < channels ? reinterpret_cast<const uint16_t *>(from)[(size_t)r * ld + c] : 0;
            asm volatile("st.shared.u16 [%0], %1;" :: "r"(piece_at(turned, r, lane >> 3) + (lane & 7) * 2), "h"(v) : "memory");
        }
    }
}

template <typename S>
__global__ void __launch_bounds__(S::THREADS, 1)
expert_matmul_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ RowMaps map_b,
                     const int32_t *__restrict__ offsets, const Sizes z, const Store st,
                     uint32_t *__restrict__ dev_error, int clear, long long wait_limit, int stall)
{
    extern __shared__ __align__(1024) uint8_t generic[];   // the swizzle is of addresses; no other shared arrays
    const uint32_t base = smem_addr(generic);
    const int tid = threadIdx.x, lane = tid & 31, warp = uniform(tid >> 5);
    const uint32_t rank = S::CG == 2 ? uniform(cluster_rank()) : 0;

    uint64_t *const bars = reinterpret_cast<uint64_t *>(generic + S::OFFBAR);
    const uint32_t bar0 = base + S::OFFBAR;
    auto full = [&](int i) { return bar0 + 8 * i; };
    auto empty = [&](int i) { return bar0 + 8 * (S::STAGES + i); };
    auto ready = [&](int i) { return bar0 + 8 * ((S::CG == 2 ? 2 * S::STAGES : 0) + i); };    // alone: landed is ready
    auto full_d = [&](int i) { return bar0 + 8 * (3 * S::STAGES + i); };
    auto empty_d = [&](int i) { return bar0 + 8 * (3 * S::STAGES + 2 + i); };
    const uint32_t drained = bar0 + 8 * (3 * S::STAGES + 4), box_full = drained + 8;
    // SPLIT: which share of the contraction is this CTA's, of how many
    const int parts = S::SPLIT ? cluster_size() : 1, part = S::SPLIT ? (int)uniform(cluster_rank()) : 0;
    uint32_t *const flags = reinterpret_cast<uint32_t *>(generic + S::OFFBAR + (S::BARS * 8 + 15) / 16 * 16);
    WaitState *const waits = reinterpret_cast<WaitState *>(flags + 2);
    const int group = blockIdx.x / (S::CG * parts), groups = gridDim.x / (S::CG * parts);
    int *const first_row = reinterpret_cast<int *>(generic + S::OFFTAB);
    int *const first_tile = first_row + z.E + 1;

    if (tid == 0) {
        prefetch_map(&map_a);
        for (int m = 0; m < (S::B_MN ? 1 : kBoxes) && kLeastBox << m <= S::BR; ++m) prefetch_map(&map_b.box[m]);
        // a stalled barrier expects one arrival more than it gets
        const int held = group == 0 ? stalled_barrier<S>(stall) : -1;
        int at = 0;
        auto init = [&](int barriers, uint32_t arrivals) {
            for (int i = 0; i < barriers; ++i, ++at) mbar_init(bars + at, arrivals + (at == held));
        };
        init(S::STAGES, 1);
        init(S::STAGES, 1);
        init(S::STAGES, S::CG);
        init(2, 1);
        init(2, 4 * S::SETS * S::CG);
        init(1, 1);
        if (S::SPLIT) init(1, 4 * parts);
        waits->limit = wait_limit;
        waits->abort = 0;
        fence_barrier_init();
    }
    if (warp == 1) tmem_alloc<S::CG>(smem_addr(flags), S::TMEM);
    pdl_wait();
    pdl_trigger();
    fill_table<S::THREADS>(offsets, z.rows, z.E, S::NT, first_row, first_tile,
                                  reinterpret_cast<int *>(generic + S::OFFTURN));     // not in use yet
    if (dev_error && clear && blockIdx.x == 0 && tid == 0) *dev_error = 0;
    if constexpr (S::CG == 2 || S::SPLIT) cluster_sync_all();
    tc_fence_after();
    const uint32_t tmem = uniform(flags[0]);

    const Table table{first_row, first_tile};
    const int channel_tiles = ceil_div(S::PASS == kWeights ? z.N : z.channels, S::OUT * S::CG);
    const int row_tiles = ceil_div(z.channels, S::NT);
    const int items = (S::PASS == kWeights ? z.E * row_tiles : uniform(first_tile[z.E])) * channel_tiles;
    auto job = [&](int i, int &at) {
        Job j = job_of<S>(table, z, channel_tiles, row_tiles, i, at);
        if constexpr (S::SPLIT) {
            const int all = j.steps, begin = all * part / parts, end = all * (part + 1) / parts;
            j.first = begin * kStep;
            j.steps = end - begin;
            if (end < all) j.tail = kStep;
        }
        return j;
    };

    if (warp == 0) {
        int issued = 0, at = 0;
        bool ok = true;
        for (int i = group; i < items && ok; i += groups) {
            const Job t = job(i, at);
            int m = 0;
            if constexpr (!S::B_MN)
                while (kLeastBox << m < t.share) ++m;
            const uint32_t bytes = S::A + (S::B_MN ? t.share : kLeastBox << m) * kStep * 2;
            const int ch = t.channel + (int)rank * S::OUT, row = t.row + (int)rank * t.share;
            for (int k = 0; k < t.steps; ++k, ++issued) {
                const int s = issued % S::STAGES, d = t.first + k * kStep;
                ok = __all_sync(kFullMask, mbar_wait_bounded(empty(s), (issued / S::STAGES & 1) ^ 1, waits));
                if (!ok) break;
                const uint32_t a = base + s * S::SLOT, b = a + S::A;
                if (elect_one()) {
                    mbar_arrive_expect(bars + s, bytes);
                    if constexpr (S::GATED) {
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            tile_load_4d(a + q * 32 * kStep * 2, &map_a, d, ch + 16 * q, 0, t.e, full(s));
                    } else if constexpr (S::PASS == kForward) {
                        tile_load_2d(a, &map_a, d, t.e * z.N + ch, full(s));
                    } else {
#pragma unroll
                        for (int q = 0; q < 2; ++q)
                            if constexpr (S::PASS == kRows)
                                tile_load_3d(a + q * 64 * kStep * 2, &map_a, ch + 64 * q, d, t.e, full(s));
                            else
                                tile_load_2d(a + q * 64 * kStep * 2, &map_a, ch + 64 * q, d, full(s));
                    }
                    if constexpr (S::B_MN) {
                        for (int q = 0; q < t.share; q += 64)
                            tile_load_2d(b + q * kStep * 2, &map_b.box[0], row + q, d, full(s));
                    } else {
                        tile_load_2d(b, &map_b.box[m], d, row, full(s));
                    }
                }
                __syncwarp();
            }
        }
        // The copies in flight land first: if another warp gave up, nobody else waits for them.
        for (int j = max(0, issued - S::STAGES); j < issued; ++j)
            mbar_drain_bounded(full(j % S::STAGES), j / S::STAGES & 1, waits);
        for (int j = max(0, issued - S::STAGES); j < issued && ok; ++j)   // the last slots' arrivals are in
            ok = __all_sync(kFullMask, mbar_wait_bounded(empty(j % S::STAGES), j / S::STAGES & 1, waits));
        // What was issued finishes first, whoever gave up: it uses the TMEM and the memory of both CTAs.
        mbar_drain_bounded(drained, 0, waits);
    } else if (warp == 1) {
        if (rank == 0) {
            int s = 0, phase = 0, u = 0, at = 0;       // slot; accumulators used so far
            const uint64_t a_first = S::A_MN ? operand_desc_mn(base, 64 * kStep * 2) : operand_desc(base);
            const uint64_t b_first = S::B_MN ? operand_desc_mn(base + S::A, 64 * kStep * 2) : operand_desc(base + S::A);
            constexpr int A_STEP = S::A_MN ? 16 * 128 / 16 : 2, B_STEP = S::B_MN ? 16 * 128 / 16 : 2;
            bool ok = true;
            for (int i = group; i < items && ok; i += groups) {
                const Job t = job(i, at);
                if (t.steps <= 0) continue;
                const uint32_t idesc = instruction_desc_bf16(kChannels * S::CG, t.n, S::A_MN, S::B_MN);
                const uint32_t acc = tmem + (u & 1) * S::NT;
                const int last = (t.tail + 15) >> 4;
                ok = __all_sync(kFullMask, mbar_wait_bounded(empty_d(u & 1), (u >> 1 & 1) ^ 1, waits));
                tc_fence_after();
                for (int k = 0; k < t.steps && ok; ++k) {
                    ok = __all_sync(kFullMask, mbar_wait_bounded(ready(s), phase, waits));
                    if (!ok) break;
                    tc_fence_after();
                    const uint64_t a = a_first + s * (S::SLOT / 16), b = b_first + s * (S::SLOT / 16);
                    if (elect_one()) {
                        if (k < t.steps - 1) {
#pragma unroll
                            for (int q = 0; q < kStep / 16; ++q)
                                mma_f16_ss<S::CG>(acc, a + q * A_STEP, b + q * B_STEP, idesc, k > 0 || q > 0);
                            mma_commit<S::CG>(empty(s));
                        } else {
                            for (int q = 0; q < last; ++q)
                                mma_f16_ss<S::CG>(acc, a + q * A_STEP, b + q * B_STEP, idesc, k > 0 || q > 0);
                            mma_commit<S::CG>(empty(s));
                            mma_commit<S::CG>(full_d(u & 1));
                        }
                    }
                    __syncwarp();
                    if (++s == S::STAGES) s = 0, phase ^= 1;
                }
                ++u;
            }
            // all that was issued, given up or not: the copying warps of both CTAs wait for it
            if (elect_one()) mma_commit<S::CG>(drained);
            __syncwarp();
            // The storing warps' last arrivals come from the other CTA too and must
            // find this one's barriers here: it leaves after they are in.
            for (int v = max(0, u - 2); v < u && ok; ++v)
                ok = __all_sync(kFullMask, mbar_wait_bounded(empty_d(v & 1), v >> 1 & 1, waits));
        }
    } else if (warp == 2) {
        if constexpr (S::CG == 2) {
            int n = 0, at = 0;
            bool ok = true;
            for (int i = group; i < items && ok; i += groups) {
                const Job t = job(i, at);
                for (int k = 0; k < t.steps; ++k, ++n) {
                    const int s = n % S::STAGES;
                    ok = __all_sync(kFullMask, mbar_wait_bounded(full(s), n / S::STAGES & 1, waits));
                    if (!ok) break;
                    if constexpr (S::B_MN) {
                        // The last instruction's rows past the expert's are the next
                        // one's: both operands are cleared there, for either may hold a NaN.
                        const int dirty = ((t.tail + 15) & ~15) - t.tail;
                        if (k == t.steps - 1 && dirty > 0) {
                            const uint32_t line = base + s * S::SLOT + t.tail * 128;
                            for (int block = 0; block < 2 + t.share / 64; ++block)     // B's blocks follow A's
                                for (int p = lane; p < dirty * 8; p += 32)
                                    sts128(line + block * 64 * kStep * 2 + p * 16, 0, 0, 0, 0);
                            fence_async_shared();
                            __syncwarp();
                        }
                    }
                    if (lane == 0) mbar_arrive_pair(cluster_addr(ready(s), 0));
                    __syncwarp();
                }
            }
        }
    } else if (warp >= S::E0) {
        const int quarter = warp & 3, set = (warp - S::E0) >> 2;
        const uint32_t turned = base + S::OFFTURN + (warp - S::E0) * S::TURN;
        constexpr int LANES = S::OUT / 4;              // output channels a warp
        __nv_bfloat16 *const out = static_cast<__nv_bfloat16 *>(st.out);
        const bool vectors = z.channels % 8 == 0;
        int u = 0, at = 0;
        bool ok = true;
        for (int i = group; i < items && ok; i += groups) {
            const Job t = job(i, at);
            const int ch0 = t.channel + (int)rank * S::OUT + quarter * LANES;
            const size_t row0 = (size_t)t.row;
            float bias[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            if constexpr (S::PASS == kForward && !S::SPLIT)
                if (st.bias) {
#pragma unroll
                    for (int q = 0; q < 4; ++q) {      // lane / 4's channel of eight; gated: up's follow gate's
                        const int c = ch0 + 8 * q % LANES + (lane >> 2);
                        if (c < z.channels) bias[q] = st.bias[(size_t)t.e * z.N + c + (8 * q < LANES ? 0 : z.channels)];
                    }
                }
            if constexpr (S::PASS == kWeights) {
                // A lane is a row of the output: 64 columns of 32 rows at a time go to
                // shared memory and from there, as whole lines, to the output (plain
                // stores of 64 bytes a row left the load/store unit 88 % busy and memory
                // at 4.9 TB/s).
                const bool none = t.steps <= 0;        // an expert without rows
                if (none && st.accumulate) continue;
                const int d = u & 1;
                const uint32_t acc = tmem + d * S::NT + ((uint32_t)quarter << 21);
                if (!none) {
                    ok = __all_sync(kFullMask, mbar_wait_bounded(full_d(d), u >> 1 & 1, waits));
                    ++u;
                    if (!ok) break;
                    tc_fence_after();
                }
                auto release = [&] {                   // all read: the accumulator is free
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0 && !none) mbar_arrive_pair(cluster_addr(empty_d(d), 0));
                };
                if (64 * set >= t.n) release();
                for (int c0 = 64 * set; c0 < t.n; c0 += 64 * S::SETS) {
                    uint32_t v[4][16];
                    if (!none) {
#pragma unroll
                        for (int q = 0; q < 4; ++q) tmem_load_x16(acc + c0 + 16 * q, v[q]);
                        tmem_wait_ld();
                    } else {
#pragma unroll
                        for (int q = 0; q < 64; ++q) v[q >> 4][q & 15] = 0;
                    }
                    if (c0 + 64 * S::SETS >= t.n) release();
                    const bool inside = c0 < t.valid && ch0 < z.N;
                    const uint32_t row = turned + lane * 128;
                    auto send = [&](int c) {
                        fence_async_shared();
                        __syncwarp();
                        if (lane == 0) {
                            if (inside && t.row + c < z.channels) {
                                if (st.accumulate) tile_add_3d(&map_b.box[1], t.row + c, ch0, t.e, turned);
                                else tile_store_3d(&map_b.box[1], t.row + c, ch0, t.e, turned);
                            }
                            bulk_commit();
                        }
                    };
                    auto settle = [&] {                // the last lines have been read from shared memory
                        if (lane == 0) bulk_wait_read<0>();
                        __syncwarp();
                    };
                    if (st.f32) {
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            settle();
#pragma unroll
                            for (int q = 0; q < 8; ++q) {
                                const uint32_t *w = v[2 * h + (q >> 2)] + 4 * (q & 3);
                                sts128(row + ((q ^ (lane & 7)) << 4), w[0], w[1], w[2], w[3]);
                            }
                            send(c0 + 32 * h);
                        }
                    } else {
                        settle();
#pragma unroll
                        for (int q = 0; q < 8; ++q) {
                            const uint32_t *w = v[q >> 1] + 8 * (q & 1);
                            uint32_t y[4];
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                y[j] = pack_bf16x2_rn(__uint_as_float(w[2 * j]), __uint_as_float(w[2 * j + 1]));
                            sts128(row + ((q ^ (lane & 7)) << 4), y[0], y[1], y[2], y[3]);
                        }
                        send(c0);
                    }
                }
                continue;
            }
            // Reads of 16 rows a warp leave memory waiting (65536 rows of 512 inputs, 4096 outputs
            // and a residual: 540 to 620 us), so a tile's residual is asked for at once (455 to 515).
            if constexpr (S::PASS == kForward && !S::SPLIT)
                if (st.residual && ch0 < z.channels)
                    for (int r = 32 * set + lane; r < t.valid; r += 32 * S::SETS)
                        prefetch_l2(st.residual + (row0 + r) * z.channels + ch0);
            const int d = u & 1;
            ok = __all_sync(kFullMask, mbar_wait_bounded(full_d(d), u >> 1 & 1, waits));
            ++u;
            if (!ok) break;
            tc_fence_after();
            const uint32_t acc = tmem + d * S::NT + ((uint32_t)quarter << 21);
            auto release = [&] {                       // all read: the accumulator is free
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_pair(S::CG == 2 ? cluster_addr(empty_d(d), 0) : empty_d(d));
            };
            if constexpr (S::SPLIT) {
                // Row c is added up by CTA c % parts: its sums go to that CTA's
                // box, [part][row / parts][128 channels].  A cluster has one tile
                // at most, so a box is written once.
                const int each = t.n / parts;
                for (int c0 = 0; c0 < t.n; c0 += 16) {
                    uint32_t v[16];
                    tmem_load_16x16(acc + c0, v);
                    tmem_load_16x16(acc + c0 + (16u << 16), v + 8);
                    tmem_wait_ld();
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        const int c = c0 + 8 * (j >> 2 & 1) + 2 * (lane & 3) + (j & 1);
                        const int ch = quarter * 32 + 16 * (j >> 3) + 8 * (j >> 1 & 1) + (lane >> 2);
                        st_cluster_u32(cluster_addr(base + S::OFFBOX + ((part * each + c / parts) * kChannels + ch) * 4,
                                                    c % parts), v[j]);
                    }
                }
                release();
                __syncwarp();
                if (lane < parts) mbar_arrive_release(cluster_addr(box_full, lane));
                __syncwarp();
                ok = __all_sync(kFullMask, mbar_wait_bounded(box_full, 0, waits));
                if (!ok) break;
                const int c = ch0 + lane % LANES, at_n = c + (lane < LANES ? 0 : z.channels);   // its row of the weights
                const float b = st.bias && c < z.channels ? st.bias[(size_t)t.e * z.N + at_n] : 0.0f;
                const float *box = reinterpret_cast<const float *>(generic + S::OFFBOX) + quarter * 32 + lane;
                for (int n = 0; n < each; ++n) {
                    const int r = n * parts + part;
                    float y = 0.0f;
                    for (int q = 0; q < parts; ++q) y += box[(q * each + n) * kChannels];
                    y += b;
                    const bool inside = r < t.valid && c < z.channels;
                    if (st.pre && inside) st.pre[(row0 + r) * z.N + at_n] = __float2bfloat16_rn(y);
                    if constexpr (S::GATED) y = silu(y) * __shfl_down_sync(kFullMask, y, 16);
                    else if (st.activation == MOE_ACT_SILU) y = silu(y);
                    else if (st.activation == MOE_ACT_GELU) y = gelu(y);
                    if (inside && lane < LANES) {
                        if (st.residual) y += __bfloat162float(st.residual[(row0 + r) * z.channels + c]);
                        out[(row0 + r) * z.channels + c] = __float2bfloat16_rn(y);
                    }
                }
                continue;
            }
            uint32_t next[16];
            if (16 * set >= t.n) release();
            else {
                tmem_load_16x16(acc + 16 * set, next);
                tmem_load_16x16(acc + 16 * set + (16u << 16), next + 8);
            }
            for (int c0 = 16 * set; c0 < t.n; c0 += 16 * S::SETS) {
                const int left = t.valid - c0;         // rows of these 16 (none: below 1)
                const size_t row = row0 + c0;
                uint32_t res[8];
                if constexpr (S::PASS == kForward)
                    if (st.residual) {
                        load_rows<LANES>(turned, st.residual + row * z.channels, z.channels, left, ch0, z.channels, vectors);
                        __syncwarp();
                        const int j = lane & 7, q = lane >> 3;
                        uint32_t w[4];
                        load_turned_x4(S::GATED ? piece_at(turned, 8 * (q >> 1) + j, q & 1) : piece_at(turned, j, q), w);
#pragma unroll
                        for (int k = 0; k < 4; ++k) res[k] = w[k];
                        if constexpr (!S::GATED) {
                            load_turned_x4(piece_at(turned, 8 + j, q), w);
#pragma unroll
                            for (int k = 0; k < 4; ++k) res[4 + k] = w[k];
                        }
                        __syncwarp();
                    }
                // v[8 hi + 4 b + 2 lo + j]: lane 16 hi + 8 lo + lane / 4, row 8 b + 2 (lane % 4) + j
                float v[16];
                tmem_wait_ld();
#pragma unroll
                for (int j = 0; j < 16; ++j) v[j] = __uint_as_float(next[j]);
                if (c0 + 16 * S::SETS < t.n) {
                    tmem_load_16x16(acc + c0 + 16 * S::SETS, next);
                    tmem_load_16x16(acc + c0 + 16 * S::SETS + (16u << 16), next + 8);
                } else {
                    release();
                }
                auto turn = [&](const float (&y)[16], int channels) {      // 8 rows of 4 times 8 channels, twice
                    const int j = lane & 7, q = lane >> 3;
                    if (channels == 32) {
#pragma unroll
                        for (int b = 0; b < 2; ++b)
                            store_turned_x4(piece_at(turned, 8 * b + j, q),
                                            pack_bf16x2_rn(y[4 * b], y[4 * b + 1]), pack_bf16x2_rn(y[4 * b + 2], y[4 * b + 3]),
                                            pack_bf16x2_rn(y[4 * b + 8], y[4 * b + 9]),
                                            pack_bf16x2_rn(y[4 * b + 10], y[4 * b + 11]));
                    } else {
                        store_turned_x4(piece_at(turned, 8 * (q >> 1) + j, q & 1),
                                        pack_bf16x2_rn(y[0], y[1]), pack_bf16x2_rn(y[2], y[3]),
                                        pack_bf16x2_rn(y[4], y[5]), pack_bf16x2_rn(y[6], y[7]));
                    }
                    __syncwarp();
                };
                if constexpr (S::PASS == kForward) {
                    if (st.bias) {
#pragma unroll
                        for (int j = 0; j < 16; ++j) v[j] += bias[2 * (j >> 3) + (j >> 1 & 1)];
                    }
                    if (st.pre) {
                        turn(v, 32);
                        store_rows<32, S::GATED>(turned, st.pre + row * z.N, z.N, left, ch0, z.channels,
                                                 vectors && z.N % 8 == 0);
                        __syncwarp();
                    }
                    if constexpr (S::GATED) {
#pragma unroll
                        for (int j = 0; j < 8; ++j) v[j] = silu(v[j]) * v[8 + j];
                    } else if (st.activation == MOE_ACT_SILU) {
#pragma unroll
                        for (int j = 0; j < 16; ++j) v[j] = silu(v[j]);
                    } else if (st.activation == MOE_ACT_GELU) {
#pragma unroll
                        for (int j = 0; j < 16; ++j) v[j] = gelu(v[j]);
                    }
                    if (st.residual) {                 // words of two rows: [b][channels of eight]
#pragma unroll
                        for (int b = 0; b < 2; ++b)
#pragma unroll
                            for (int q = 0; q < LANES / 8; ++q) {
                                float *y = v + 8 * (q >> 1) + 4 * b + 2 * (q & 1);
                                const uint32_t w = res[b * (LANES / 8) + q];
                                y[0] += bf16_lo(w);
                                y[1] += bf16_hi(w);
                            }
                    }
                }
                turn(v, LANES);
                store_rows<LANES, false>(turned, out + row * z.channels, z.channels, left, ch0, z.channels, vectors);
                __syncwarp();
            }
        }
        if constexpr (S::PASS == kWeights)
            if (lane == 0) bulk_wait_all();            // given up or not, before the block leaves
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if constexpr (S::CG == 2 || S::SPLIT) cluster_sync_all();      // the peer is done with this CTA's memory
    tc_fence_after();
    if (tid == 0 && waits->abort && dev_error) atomicOr(dev_error, MOE_DEV_ERR_TIMEOUT);
    if (warp == 1) tmem_free<S::CG>(tmem, S::TMEM);
}

// A tensor of bf16 or fp32, innermost dimension first; strides of the others in
// elements (multiples of 8); boxes of 128-byte lines, swizzled, zeros outside.
bool tensor_map(CUtensorMap *map, const void *p, int rank, const uint64_t *dims, const uint64_t *strides,
                const uint32_t *box, bool f32 = false)
{
    cuuint64_t d[4], s[3];
    cuuint32_t b[4];
    for (int i = 0; i < rank; ++i) {
        d[i] = dims[i];
        b[i] = box[i];
        if (i > 0) s[i - 1] = strides[i - 1] * (f32 ? 4 : 2);
    }
    return encode_tiled(map, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, p, d, s, b);
}

// [rows, width] in boxes of 64 by `box` rows.
bool rows_map(CUtensorMap *map, const void *p, uint64_t rows, uint64_t width, uint32_t box)
{
    const uint64_t dims[2] = {width, rows}, strides[1] = {width};
    const uint32_t boxes[2] = {kStep, box};
    return tensor_map(map, p, 2, dims, strides, boxes);
}

template <typename S>
bool row_maps(RowMaps *maps, const void *p, uint64_t rows, uint64_t width)
{
    for (int m = 0; m < kBoxes; ++m)                   // higher boxes than a CTA's rows are not used
        if (kLeastBox << m > S::BR) maps->box[m] = maps->box[0];
        else if (!rows_map(&maps->box[m], p, rows, width, kLeastBox << m)) return false;
    return true;
}

template <typename S>
cudaError_t run(const CUtensorMap &map_a, const RowMaps &map_b, const int32_t *offsets, const Sizes &z, const Store &st,
                int64_t tiles, int sms, int parts, uint32_t *dev_error, int clear, long long wait_limit, int stall,
                cudaStream_t stream)
{
    const size_t smem = S::bytes(z.E);
    const cudaError_t e = allow_dynamic_smem(reinterpret_cast<const void *>(&expert_matmul_kernel<S>), smem);
    if (e != cudaSuccess) return e;
    const int64_t groups = tiles < sms / (S::CG * parts) ? tiles : sms / (S::CG * parts);
    return launch_pdl_clusters(expert_matmul_kernel<S>, dim3((unsigned)groups * S::CG * parts), dim3(S::THREADS), smem,
                               stream, S::CG * parts, map_a, map_b, offsets, z, st, dev_error, clear, wait_limit, stall);
}

}  // namespace
}  // namespace moe
