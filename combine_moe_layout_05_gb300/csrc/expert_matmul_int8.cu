// expert_matmul_int8.cu -- packed int8 rows times their experts' int8
// weights, with a scale for each row and each output channel.
//
//   out[r, n] = bf16((sum_h x[r, h] * w[e, n, h]) * x_scale[r] * w_scale[e, n])
//   for the rows r of expert e, [offsets[e], offsets[e+1])
//
// sm_103a has no 8-bit integer matrix instruction of the tcgen05 kind, and an
// int8 value is exactly a fp16 value: the codes travel as bytes through HBM,
// L2 and the copies into shared memory, and are widened on the way to the
// fp16 tensor cores.  A product is at most 2^14 and the fp32 accumulator exact
// up to 2^24, so the sum is the integer's while partial sums stay below that;
// past it the accumulator rounds or truncates to 24 bits at each instruction.
//
// A tile is 128 channels a CTA (256 a pair of CTAs) by up to NT rows of one
// expert.  Channels are the instruction's M, so that a tile with few rows
// still feeds it 128 lanes; the row count is its N and is what the expert has
// left, rounded up.  Warps of a CTA:
//
//   one copies 128-byte-wide tiles of weights and rows into a ring;
//   one issues the matrix instructions (the pair's first CTA's);
//   4 GA widen the weights into TMEM (operand A), one channel a thread;
//   WB GB widen the rows into shared memory (operand B), 16 bytes a thread;
//   4 SETS scale the sums, turn them in shared memory and store them.
//
// A pair shares each other's widened rows: every CTA widens half of the tile's
// rows, which keeps shared memory within its 128 bytes a cycle (a 128-byte step
// of 256 rows moves 32 KB in, 32 KB to the widening warps, 32 KB of widened
// rows back and 32 KB to the tensor core, in the instruction's 1024 cycles).
//
// Measured: 131072 rows, 4096 -> 2048, 128 experts 1.23 ms (1.79 PFLOP/s, 96 %
// of a library bf16 product's rate) in a burst and 1.38 under the power cap;
// 1024 rows over 256 experts, 7168 -> 2048, 0.54 ms (7.0 TB/s of weights:
// HBM-bound); 32768 skewed rows over 384 experts, 7168 -> 2048, 1.12 ms in a
// burst, 1.20 under the cap (547 tiles of 60 rows on average, 600 to 700 cycles
// a step; HBM takes 706 for the first tile of an expert, L2 feeds the others).
#include "expert_tiles.cuh"

#include <mutex>
#include <type_traits>

namespace moe {
namespace {

constexpr int kStep = 128;                 // bytes of the contraction a ring slot holds
constexpr int kTmemColumns = 512;
constexpr int kMaxShared = 227 * 1024;

// CG: CTAs a tile.  NT: rows a tile at most.  PARTS: parts a tile's rows are
// summed in, each with its accumulator.  KS: the contraction's share of a slot
// of widened operands.  N8, NC: slots of int8 tiles and of widened operands.
// GA, GB: groups of warps that widen the weights and the rows; a group takes
// every GA-th (GB-th) step, since one step's latency (barrier, loads, stores
// and their wait) is several times its issue slots.
// SPLIT: a cluster's CTAs each sum a share of the contraction.
template <int CG_, int NT_, int PARTS_, int KS_, int N8_, int NC_, int GA_, int GB_, bool SPLIT_ = false>
struct Shape {
    static constexpr bool SPLIT = SPLIT_;
    static_assert(!SPLIT || (CG_ == 1 && PARTS_ == 1 && KS_ == kStep));
    static constexpr int CG = CG_, NT = NT_, PARTS = PARTS_, KS = KS_, N8 = N8_, NC = NC_, GA = GA_, GB = GB_;
    static constexpr int BR = NT / CG;                 // rows a CTA widens at most
    static constexpr int QUANTUM = 16 * CG;            // rows of a part are a multiple of
    static constexpr int PER = kStep / KS;             // widened slots a step
    static constexpr int BURST = 3;                    // slots a part runs ahead at a tile's ends
    static constexpr int A8 = kChannels * kStep, B8 = BR * kStep, B16 = BR * KS * 2;
    static constexpr int SLOT8 = A8 + B8;
    static constexpr int UNIT = NT / PARTS;            // TMEM columns of an accumulator
    static constexpr int ACOL0 = 2 * UNIT, ACOL = KS / 2;   // and of the widened weights
    static_assert(ACOL0 + NC * ACOL <= kTmemColumns && BURST <= NC);
    // A barrier's parity tells a use from the one before, not from the one
    // before that, so a group that waits for a use has to know that the one
    // before is over.  Widened slots are consumed in order, and a group has
    // waited for the last but one round of its own.  Byte slots may land out
    // of order: there a slot belongs to the same group in every round, which
    // has then worked on its last use itself.
    static_assert(GA * PER <= NC && GB * PER <= NC && N8 % GA == 0 && N8 % GB == 0);
    // warps: 0 copies, 1 issues, then those that widen and those that store;
    // the TMEM lanes a warp reaches are those of its number modulo 4
    static constexpr int WB = 4;                       // warps of a group that widens rows
    static_assert(BR * (KS / 64) <= 8 * WB * 4);
    // Sets of four warps that store, two where a tile has more than 32 rows: a
    // short contraction waits for them (64 experts of 128 rows, 512 -> 4096, in
    // the 128-row form: 63.8 us with one set, 56.7 with two, and 53.7 since they
    // multiply in pairs and keep the scales of their own rows only).
    static constexpr int SETS = CG;
    static constexpr int A0 = 4, E0 = A0 + 4 * GA, B0 = E0 + 4 * SETS, WARPS = B0 + WB * GB;
    static constexpr int THREADS = WARPS * 32;
    static constexpr int BARS = 2 * N8 + 2 * NC + 4 + 1 + SPLIT;
    // ring, widened rows, 16 x 32 outputs and the row scales of each storing
    // warp, barriers, flags, expert table
    static constexpr int OFF16 = N8 * SLOT8;
    static constexpr int OFFTURN = OFF16 + NC * B16;
    static constexpr int OFFBOX = OFFTURN + 4 * SETS * 1024;  // SPLIT: the other CTAs' sums, NT x 128 fp32
    static constexpr int OFFS = OFFBOX + SPLIT * NT * kChannels * 4;
    static constexpr int SCALES = PARTS == 1 ? NT / SETS : NT;    // rows a storing warp needs the scales of
    static constexpr int OFFBAR = OFFS + 4 * SETS * SCALES * 4;
    static constexpr int OFFTAB = OFFBAR + (BARS * 8 + 15) / 16 * 16 + 32;
    static constexpr int bytes(int E) { return OFFTAB + 2 * (E + 1) * 4; }
    static_assert(bytes(MOE_MAX_EXPERTS) <= kMaxShared);
};
// Shared memory and TMEM are what the numbers divide: a deep byte ring where
// HBM feeds it (Narrow: 8 slots, 144 KB), two accumulators in all, and as many
// widened slots as are left.  Cycles a step, weights in L2: Narrow 552 (16
// rows) and 584 (32), Mid 613 (64) and 704 (128), Wide 1233 (256; 1024 are the
// instruction's).
using Wide = Shape<2, 256, 2, 64, 4, 4, 2, 2>;
using Mid = Shape<2, 128, 1, 128, 6, 4, 2, 2>;
using Narrow = Shape<1, 32, 1, 128, 8, 6, 4, 2>;
using Split = Shape<1, 32, 1, 128, 4, 6, 4, 2, true>;

// Copies of rows come in these heights; a tile takes the one that covers its
// share, so that a step is one copy of weights and one of rows.
constexpr int kBoxes = 4, kLeastBox = 16;
struct RowMaps {
    CUtensorMap box[kBoxes];    // 16, 32, 64, 128 rows
};

// Two products at once.
__device__ __forceinline__ float2 mul2(float2 a, float2 b)
{
    float2 r;
    asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmul.rn.f32x2 x, x, y;\n\t"
        "mov.b64 {%0, %1}, x;\n\t}" : "=f"(r.x), "=f"(r.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
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

__device__ __forceinline__ void widen16(const uint4 &x, uint32_t *v)
{
    widen4(x.x, v[0], v[1]);
    widen4(x.y, v[2], v[3]);
    widen4(x.z, v[4], v[5]);
    widen4(x.w, v[6], v[7]);
}

// The instructions of one slot of widened operands: B's 64-wide blocks follow
// each other, 128 bytes a row.
template <typename S, int COUNT>
__device__ __forceinline__ void mma_slot(uint32_t acc, uint32_t a, uint64_t b, uint32_t idesc, bool accumulate)
{
#pragma unroll
    for (int q = 0; q < COUNT; ++q)
        mma_f16_ts<S::CG>(acc, a + 8 * q, b + (q >> 2) * (S::BR * 128 / 16) + (q & 3) * 2, idesc, accumulate || q > 0);
}

template <typename S>
__device__ __forceinline__ void mma_slot_n(uint32_t acc, uint32_t a, uint64_t b, uint32_t idesc, bool accumulate, int count)
{
    for (int q = 0; q < count; ++q)
        mma_f16_ts<S::CG>(acc, a + 8 * q, b + (q >> 2) * (S::BR * 128 / 16) + (q & 3) * 2, idesc, accumulate || q > 0);
}

// The barrier that a test holds back in the first tile's CTAs: the first of a
// kind (0 to 6), or none.
template <typename S>
__device__ __forceinline__ int stalled_barrier(int kind)
{
    if (kind < 0 || kind >= 6 + S::SPLIT) return -1;
    if (kind < 4) return (kind > 0 ? S::N8 : 0) + (kind > 1 ? S::N8 : 0) + (kind > 2 ? S::NC : 0);
    return 2 * S::N8 + 2 * S::NC + (kind == 4 ? 0 : kind == 5 ? 2 : 5);
}

template <typename S>
__global__ void __launch_bounds__(S::THREADS, 1)
expert_matmul_int8_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ RowMaps map_x,
                          const float *__restrict__ x_scales, const float *__restrict__ w_scales,
                          const int32_t *__restrict__ offsets, int rows, int H, int N, int E,
                          __nv_bfloat16 *__restrict__ out, uint32_t *__restrict__ dev_error,
                          long long wait_limit, int stall)
{
    extern __shared__ __align__(1024) uint8_t generic[];   // the swizzle is of addresses; no other shared arrays
    const uint32_t base = smem_addr(generic);
    const int tid = threadIdx.x, lane = tid & 31, warp = uniform(tid >> 5);
    const uint32_t rank = S::CG == 2 ? uniform(cluster_rank()) : 0;

    const uint32_t bar0 = base + S::OFFBAR;
    auto full8 = [&](int i) { return bar0 + 8 * i; };
    auto empty8 = [&](int i) { return bar0 + 8 * (S::N8 + i); };
    auto full16 = [&](int i) { return bar0 + 8 * (2 * S::N8 + i); };
    auto empty16 = [&](int i) { return bar0 + 8 * (2 * S::N8 + S::NC + i); };
    auto full_d = [&](int i) { return bar0 + 8 * (2 * S::N8 + 2 * S::NC + i); };
    auto empty_d = [&](int i) { return bar0 + 8 * (2 * S::N8 + 2 * S::NC + 2 + i); };
    const uint32_t drained = bar0 + 8 * (2 * S::N8 + 2 * S::NC + 4), box_full = drained + 8;
    // SPLIT: which share of the contraction is this CTA's, of how many
    const int parts = S::SPLIT ? cluster_size() : 1, part = S::SPLIT ? (int)uniform(cluster_rank()) : 0;
    uint32_t *const flags = reinterpret_cast<uint32_t *>(generic + S::OFFBAR + (S::BARS * 8 + 15) / 16 * 16);
    WaitState *const waits = reinterpret_cast<WaitState *>(flags + 2);
    const int group = blockIdx.x / (S::CG * parts), groups = gridDim.x / (S::CG * parts);
    int *const first_row = reinterpret_cast<int *>(generic + S::OFFTAB);
    int *const first_tile = first_row + E + 1;

    if (tid == 0) {
        prefetch_map(&map_w);
        for (int m = 0; kLeastBox << m <= S::BR; ++m) prefetch_map(&map_x.box[m]);
        // a stalled barrier expects one arrival more than it gets
        const int held = group == 0 ? stalled_barrier<S>(stall) : -1;
        int at = 0;
        auto init = [&](int barriers, uint32_t arrivals) {
            for (int i = 0; i < barriers; ++i, ++at)
                mbar_init(reinterpret_cast<uint64_t *>(generic + S::OFFBAR) + at, arrivals + (at == held));
        };
        init(S::N8, 1);
        init(S::N8, 4 + S::WB);
        init(S::NC, (4 + S::WB) * S::CG);
        init(S::NC, 1);
        init(2, 1);
        init(2, 4 * S::SETS * S::CG);
        init(1, 1);
        if (S::SPLIT) init(1, 4 * parts);
        waits->limit = wait_limit;
        waits->abort = 0;
        fence_barrier_init();
    }
    if (warp == 1) tmem_alloc<S::CG>(smem_addr(flags), kTmemColumns);
    pdl_wait();
    pdl_trigger();

    static_assert(S::WARPS * 4 <= 4 * S::SETS * 1024);
    fill_table<S::THREADS>(offsets, rows, E, S::NT, first_row, first_tile,
                                  reinterpret_cast<int *>(generic + S::OFFTURN));     // not in use yet
    if (dev_error && blockIdx.x == 0 && tid == 0) *dev_error = 0;
    if constexpr (S::CG == 2 || S::SPLIT) cluster_sync_all();
    tc_fence_after();
    const uint32_t tmem = uniform(flags[0]);

    const Table table{first_row, first_tile};
    const int channel_tiles = ceil_div(N, kChannels * S::CG);
    const int items = uniform(first_tile[E]) * channel_tiles;
    const int all_steps = ceil_div(H, kStep), step0 = all_steps * part / parts;
    const int steps = all_steps * (part + 1) / parts - step0;
    const int slots = S::SPLIT ? steps : ceil_div(H, S::KS), h0 = step0 * kStep;
    uint64_t *const bars = reinterpret_cast<uint64_t *>(generic + S::OFFBAR);

    if (warp == 0) {
        int issued = 0, at = 0;
        bool ok = true;
        for (int i = group; i < items && ok; i += groups) {
            const Tile t = tile_of<S>(table, E, channel_tiles, i, at);
            const int share = (t.n[0] + t.n[1]) / S::CG;
            int m = 0;
            while (kLeastBox << m < share) ++m;
            const int wr = t.e * N + t.channel + (int)rank * kChannels, xr = t.row + (int)rank * share;
            const uint32_t bytes = S::A8 + (kLeastBox << m) * kStep;
            for (int k = 0; k < steps; ++k, ++issued) {
                const int s = issued % S::N8;
                ok = __all_sync(kFullMask, mbar_wait_bounded(empty8(s), (issued / S::N8 & 1) ^ 1, waits));
                if (!ok) break;
                const uint32_t slot = base + s * S::SLOT8;
                if (elect_one()) {
                    mbar_arrive_expect(bars + s, bytes);
                    tile_load_2d(slot, &map_w, h0 + k * kStep, wr, full8(s));
                    tile_load_2d(slot + S::A8, &map_x.box[m], h0 + k * kStep, xr, full8(s));
                }
                __syncwarp();
            }
        }
        // The copies in flight land first: if another warp gave up, nobody else waits for them.
        for (int j = max(0, issued - S::N8); j < issued; ++j)
            mbar_drain_bounded(full8(j % S::N8), j / S::N8 & 1, waits);
    } else if (warp == 1) {
        if (rank == 0) {
            int c = 0, cphase = 0;                     // slot of widened operands
            int u = 0, at = 0;                         // accumulators used so far
            const uint64_t b_first = operand_desc(base + S::OFF16);
            constexpr int kFull = S::KS / 16;          // instructions a slot
            const int last = min(kFull, (H - h0 - (slots - 1) * S::KS) >> 4);        // and in the last one
            bool ok = true;
            auto wait_free = [&](int v) {
                ok = __all_sync(kFullMask, mbar_wait_bounded(empty_d(v & 1), (v >> 1 & 1) ^ 1, waits));
                tc_fence_after();
            };
            auto wait_slot = [&](int s, int phase) {
                ok = __all_sync(kFullMask, mbar_wait_bounded(full16(s), phase, waits));
                tc_fence_after();
            };
            for (int i = group; i < items && ok; i += groups) {
                const Tile t = tile_of<S>(table, E, channel_tiles, i, at);
                const uint32_t idesc0 = instruction_desc_f16(kChannels * S::CG, t.n[0]);
                const uint32_t idesc1 = instruction_desc_f16(kChannels * S::CG, t.n[1]);
                const uint32_t b_part = t.n[0] / S::CG * (128 / 16);       // part 1's rows follow part 0's
                const uint32_t acc0 = tmem + (u & 1) * S::UNIT, acc1 = tmem + (u + 1 & 1) * S::UNIT;
                // slots by turns between the parts, but the first and the last
                // few one part after the other: one accumulator is drained
                // while the other is summed
                if constexpr (S::PARTS == 2) {
                    const bool two = t.n[1] > 0;
                    int k = 0;
                    bool ready = false;                // the next slot has been seen full
                    while (k < slots && ok) {
                        const int left = slots - k;
                        int s = c, ph = cphase;
                        if (k > 0 && left > S::BURST) {
                            if (!ready) wait_slot(s, ph);
                            if (!ok) break;
                            const uint32_t a = tmem + S::ACOL0 + s * S::ACOL;
                            const uint64_t b0 = b_first + s * (S::B16 / 16), b1 = b0 + b_part;
                            const uint32_t empty = empty16(s);
                            if (elect_one()) mma_slot<S, kFull>(acc0, a, b0, idesc0, true);
                            __syncwarp();
                            // the next slot is asked for while instructions wait in the queue
                            if (++s == S::NC) s = 0, ph ^= 1;
                            ready = __all_sync(kFullMask, mbar_test_cluster(full16(s), ph));
                            if (elect_one()) {
                                if (two) mma_slot<S, kFull>(acc1, a, b1, idesc1, true);
                                mma_commit<S::CG>(empty);
                            }
                            __syncwarp();
                            if (ready) tc_fence_after();
                            ++k;
                        } else {
                            const int count = min(S::BURST, left);
                            if (k == 0) wait_free(u);
                            for (int j = 0; j < count && ok; ++j) {
                                if (!ready) wait_slot(s, ph);
                                ready = false;
                                if (!ok) break;
                                if (elect_one()) {
                                    mma_slot_n<S>(acc0, tmem + S::ACOL0 + s * S::ACOL, b_first + s * (S::B16 / 16), idesc0,
                                                  k + j > 0, k + j == slots - 1 ? last : kFull);
                                    if (k + j == slots - 1) mma_commit<S::CG>(full_d(u & 1));
                                }
                                __syncwarp();
                                if (++s == S::NC) s = 0, ph ^= 1;
                            }
                            if (k == 0 && ok) wait_free(u + 1);
                            if (!ok) break;
                            s = c, ph = cphase;
                            for (int j = 0; j < count; ++j) {
                                if (elect_one()) {
                                    if (two)
                                        mma_slot_n<S>(acc1, tmem + S::ACOL0 + s * S::ACOL, b_first + s * (S::B16 / 16) + b_part,
                                                      idesc1, k + j > 0, k + j == slots - 1 ? last : kFull);
                                    mma_commit<S::CG>(empty16(s));
                                    if (k + j == slots - 1) mma_commit<S::CG>(full_d(u + 1 & 1));
                                }
                                __syncwarp();
                                if (++s == S::NC) s = 0, ph ^= 1;
                            }
                            k += count;
                        }
                        c = s, cphase = ph;
                    }
                } else {
                    wait_free(u);
                    for (int k = 0; k < slots && ok; ++k) {
                        wait_slot(c, cphase);
                        if (!ok) break;
                        const uint32_t a = tmem + S::ACOL0 + c * S::ACOL;
                        const uint64_t b = b_first + c * (S::B16 / 16);
                        if (elect_one()) {
                            if (k < slots - 1) {
                                mma_slot<S, kFull>(acc0, a, b, idesc0, k > 0);
                                mma_commit<S::CG>(empty16(c));
                            } else {
                                mma_slot_n<S>(acc0, a, b, idesc0, k > 0, last);
                                mma_commit<S::CG>(empty16(c));
                                mma_commit<S::CG>(full_d(u & 1));
                            }
                        }
                        __syncwarp();
                        if (++c == S::NC) c = 0, cphase ^= 1;
                    }
                }
                u += S::PARTS;
            }
            // all that was issued, given up or not: the widening warps of both CTAs wait for it
            if (elect_one()) mma_commit<S::CG>(drained);
            __syncwarp();
            // The storing warps' last arrivals come from the other CTA too and must
            // find this one's barriers here: it leaves after they are in.
            for (int v = max(0, u - 2); v < u && ok; ++v)
                ok = __all_sync(kFullMask, mbar_wait_bounded(empty_d(v & 1), v >> 1 & 1, waits));
        }
    } else if (warp >= S::E0 && warp < S::B0) {
        // set by set, 16 rows at a time
        const int quarter = warp & 3, set = (warp - S::E0) >> 2;
        float *const row_scale = reinterpret_cast<float *>(generic + S::OFFS) + (warp - S::E0) * S::SCALES;
        const uint32_t turned = base + S::OFFTURN + (warp - S::E0) * 1024;
        int u = 0, at = 0;
        bool ok = true;
        // the next tile and its scales are on their way while one is stored
        Tile next_tile;
        float next_xs[S::SCALES / 32], next_ws[4];
        auto fetch = [&](int i) {
            if (i >= items) return;
            next_tile = tile_of<S>(table, E, channel_tiles, i, at);
#pragma unroll
            for (int j = 0; j < S::SCALES / 32; ++j) {
                // all rows, or every SETS-th 16 of them where the sets take them by turns
                const int k = j * 32 + lane;
                const int r = S::PARTS == 1 ? (k >> 4) * 16 * S::SETS + 16 * set + (k & 15) : k;
                next_xs[j] = r < next_tile.valid ? x_scales[next_tile.row + r] : 0.0f;
            }
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int ch = next_tile.channel + (int)rank * kChannels + quarter * 32 + 8 * q + (lane >> 2);
                next_ws[q] = ch < N ? w_scales[(size_t)next_tile.e * N + ch] : 0.0f;
            }
        };
        fetch(group);
        for (int i = group; i < items && ok; i += groups) {
            const Tile t = next_tile;
            const int ch0 = t.channel + (int)rank * kChannels + quarter * 32;
            const float ws[4] = {next_ws[0], next_ws[1], next_ws[2], next_ws[3]};
            __syncwarp();                              // the last tile's scales have been read
#pragma unroll
            for (int j = 0; j < S::SCALES / 32; ++j) row_scale[j * 32 + lane] = next_xs[j];
            __syncwarp();
            fetch(i + groups);
            const bool vectors = N % 8 == 0;
            for (int p = 0; p < S::PARTS && ok; ++p, ++u) {
                const int d = u & 1, n = t.n[p], mine = n / S::CG;
                ok = __all_sync(kFullMask, mbar_wait_bounded(full_d(d), u >> 1 & 1, waits));
                if (!ok) break;
                tc_fence_after();
                const uint32_t acc = tmem + d * S::UNIT + ((uint32_t)quarter << 21);
                if constexpr (S::SPLIT) {
                    // Row c is added up by CTA c % parts: its sums go to that
                    // CTA's box, [part][row / parts][128 channels].  A cluster
                    // has one tile at most, so a box is written once.
                    const int each = n / parts;
                    for (int c0 = 0; c0 < n; c0 += 16) {
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
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bars + 2 * S::N8 + 2 * S::NC + 2 + d);
                    if (lane < parts) mbar_arrive_release(cluster_addr(box_full, lane));
                    __syncwarp();
                    ok = __all_sync(kFullMask, mbar_wait_bounded(box_full, 0, waits));
                    if (!ok) break;
                    const int ch = ch0 + lane;
                    const float scale = ch < N ? w_scales[(size_t)t.e * N + ch] : 0.0f;
                    const float *box = reinterpret_cast<const float *>(generic + S::OFFBOX) + quarter * 32 + lane;
                    for (int i = 0; i < each; ++i) {
                        const int c = i * parts + part;
                        float sum = 0.0f;
                        for (int q = 0; q < parts; ++q) sum += box[(q * each + i) * kChannels];
                        if (c < t.valid && ch < N)
                            out[(size_t)(t.row + c) * N + ch] = __float2bfloat16_rn(sum * row_scale[c] * scale);
                    }
                    continue;
                }
                auto release = [&] {                   // all read: the accumulator is free
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_pair(S::CG == 2 ? cluster_addr(empty_d(d), 0) : empty_d(d));
                };
                uint32_t next[16];
                if (16 * set >= n) release();
                if (16 * set < n) {
                    tmem_load_16x16(acc + 16 * set, next);
                    tmem_load_16x16(acc + 16 * set + (16u << 16), next + 8);
                }
                for (int c0 = 16 * set; c0 < n; c0 += 16 * S::SETS) {
                    uint32_t v[16];
                    tmem_wait_ld();
#pragma unroll
                    for (int j = 0; j < 16; ++j) v[j] = next[j];
                    if (c0 + 16 * S::SETS < n) {
                        tmem_load_16x16(acc + c0 + 16 * S::SETS, next);
                        tmem_load_16x16(acc + c0 + 16 * S::SETS + (16u << 16), next + 8);
                    } else {
                        release();
                    }
                    // the tile's row of column c0: the second CTA's share follows the first's
                    const int second = S::CG == 2 && c0 >= mine;
                    const int r0 = c0 + (p ? t.n[0] / S::CG : 0) + (second ? (t.n[0] + t.n[1]) / 2 - mine : 0);
                    const float *rs = row_scale + (S::PARTS == 1 ? r0 / S::SETS & ~15 : r0) + 2 * (lane & 3);
#pragma unroll
                    for (int b = 0; b < 2; ++b) {      // 8 rows, of 4 times 8 channels
                        const float2 r = *reinterpret_cast<const float2 *>(rs + 8 * b);
                        uint32_t y[4];
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            const uint32_t *w = v + 8 * (q >> 1) + 4 * b + 2 * (q & 1);
                            const float2 z = mul2(mul2({__uint_as_float(w[0]), __uint_as_float(w[1])}, r), {ws[q], ws[q]});
                            y[q] = pack_bf16x2_rn(z.x, z.y);
                        }
                        const int j = lane & 7;        // a row of 64 bytes, its 16-byte pieces permuted
                        store_turned_x4(turned + (8 * b + j) * 64 + (((lane >> 3) ^ (j >> 1 & 3)) << 4),
                                        y[0], y[1], y[2], y[3]);
                    }
                    __syncwarp();
                    if (vectors) {
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            const int r = 8 * j + (lane >> 2);
                            const uint4 q = lds128(turned + r * 64 + (((lane & 3) ^ (r >> 1 & 3)) << 4));
                            if (r0 + r < t.valid && ch0 + (lane & 3) * 8 < N)
                                st_v4(out + (size_t)(t.row + r0 + r) * N + ch0 + (lane & 3) * 8, q);
                        }
                    } else if (ch0 + lane < N) {
                        const __nv_bfloat16 *y = reinterpret_cast<const __nv_bfloat16 *>(generic + (turned - base));
                        __nv_bfloat16 *o = out + (size_t)(t.row + r0) * N + ch0 + lane;
                        const int rows_left = min(16, t.valid - r0);
                        if (rows_left == 16) {
                            const int turn = lane >> 3, in = lane & 7;
#pragma unroll
                            for (int half = 0; half < 16; half += 8) {
                                __nv_bfloat16 q[8];
#pragma unroll
                                for (int r = 0; r < 8; ++r) q[r] = y[(half + r) * 32 + ((turn ^ (r >> 1 & 3)) << 3) + in];
#pragma unroll
                                for (int r = 0; r < 8; ++r, o += N) *o = q[r];
                            }
                        } else {
#pragma unroll 4
                            for (int r = 0; r < rows_left; ++r, o += N)
                                *o = y[r * 32 + (((lane >> 3) ^ (r >> 1 & 3)) << 3) + (lane & 7)];
                        }
                    }
                    __syncwarp();
                }
            }
        }
    } else if (warp >= S::A0 && warp < S::E0) {
        // weights: group `g` has every GA-th step, and in it a thread one channel
        const int g = (warp - S::A0) >> 2, r = (warp & 3) * 32 + lane;
        // a row's 16-byte pieces are permuted by the row's low bits: piece q is
        // at piece q ^ (r & 7), a flip of address bits
        const uint32_t row = base + r * kStep + ((r & 7) << 4);
        int n0 = 0, m0 = 0;                            // steps, and widened slots, of the tiles before
        bool ok = true;
        for (int i = group; i < items && ok; i += groups, n0 += steps, m0 += slots)
            for (int k = (g + S::GA - n0 % S::GA) % S::GA; k < steps && ok; k += S::GA) {
                const int n = n0 + k, s = n % S::N8;
                ok = __all_sync(kFullMask, mbar_wait_bounded(full8(s), n / S::N8 & 1, waits));
                const uint32_t src = row + s * S::SLOT8;
#pragma unroll 1
                for (int h = 0; h < S::PER; ++h) {
                    if (!ok || k * S::PER + h >= slots) break;
                    const int m = m0 + k * S::PER + h, c = m % S::NC;
                    const uint32_t half = src ^ (h << 6);
                    const uint32_t dst = tmem + S::ACOL0 + c * S::ACOL + ((uint32_t)(warp & 3) << 21);
                    uint32_t v[32];
#pragma unroll
                    for (int w = 0; w < S::KS / 64; ++w) {
#pragma unroll
                        for (int q = 0; q < 4; ++q) widen16(lds128(half ^ (4 * w + q) << 4), v + 8 * q);
                        if (w == 0) {
                            ok = __all_sync(kFullMask, mbar_wait_bounded(empty16(c), (m / S::NC & 1) ^ 1, waits));
                            if (!ok) break;
                            tc_fence_after();
                        }
                        tmem_store_x32(dst + 32 * w, v);
                    }
                    if (!ok) break;
                    tmem_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_pair(S::CG == 2 ? cluster_addr(full16(c), 0) : full16(c));
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(bars + S::N8 + s);
            }
        for (int j = max(0, m0 - S::NC); j < m0 && ok; ++j)           // the last slots' arrivals are in
            ok = __all_sync(kFullMask, mbar_wait_bounded(empty16(j % S::NC), j / S::NC & 1, waits));
        // What was issued finishes first, whoever gave up: it uses the TMEM and the memory of both CTAs.
        mbar_drain_bounded(drained, 0, waits);
    } else if (warp >= S::B0 && warp < S::B0 + S::WB * S::GB) {
        // rows: group `g` has every GB-th step; a warp takes 8 rows by 64 bytes at
        // a time, a thread 16 bytes, so that few rows are spread over all warps
        const int g = (warp - S::B0) / S::WB, w = (warp - S::B0) % S::WB;
        int n0 = 0, m0 = 0, at = 0;
        bool ok = true;
        for (int i = group; i < items && ok; i += groups, n0 += steps, m0 += slots) {
            const Tile t = tile_of<S>(table, E, channel_tiles, i, at);
            const int blocks = (t.n[0] + t.n[1]) / (8 * S::CG);
            for (int k = (g + S::GB - n0 % S::GB) % S::GB; k < steps && ok; k += S::GB) {
                const int n = n0 + k, s = n % S::N8;
                ok = __all_sync(kFullMask, mbar_wait_bounded(full8(s), n / S::N8 & 1, waits));
                const uint32_t src = base + s * S::SLOT8 + S::A8;
#pragma unroll 1
                for (int h = 0; h < S::PER; ++h) {
                    if (!ok || k * S::PER + h >= slots) break;
                    const int m = m0 + k * S::PER + h, c = m % S::NC;
                    // pieces a warp, rounded up: the rows past the tile's are in the
                    // slot's memory (with two halves there are none: blocks is even),
                    // and no instruction reads them
                    auto widen = [&](auto pieces) {
                        constexpr int U = decltype(pieces)::value;
                        uint32_t v[U][8];
#pragma unroll
                        for (int j = 0; j < U; ++j) {
                            const int at = w + S::WB * j, half = S::KS > 64 && at >= blocks, block = at - half * blocks;
                            const int r = 8 * block + (lane & 7), q = 4 * (h + half) + (lane >> 3);
                            widen16(lds128(src + r * kStep + ((q ^ (r & 7)) << 4)), v[j]);
                        }
                        ok = __all_sync(kFullMask, mbar_wait_bounded(empty16(c), (m / S::NC & 1) ^ 1, waits));
                        if (!ok) return;
#pragma unroll
                        for (int j = 0; j < U; ++j) {
                            const int at = w + S::WB * j, half = S::KS > 64 && at >= blocks, block = at - half * blocks;
                            const int r = 8 * block + (lane & 7), q = 2 * (lane >> 3);
                            const uint32_t row = base + S::OFF16 + c * S::B16 + half * S::BR * 128 + r * 128;
                            sts128(row + ((q ^ (r & 7)) << 4), v[j][0], v[j][1], v[j][2], v[j][3]);
                            sts128(row + (((q + 1) ^ (r & 7)) << 4), v[j][4], v[j][5], v[j][6], v[j][7]);
                        }
                    };
                    constexpr int kMost = S::BR / 8 * (S::KS / 64) / S::WB;
                    const int pieces = ceil_div(blocks * (S::KS / 64), S::WB);
                    if (pieces == 1) widen(std::integral_constant<int, 1>());
                    else if (kMost <= 2 || pieces == 2) widen(std::integral_constant<int, 2>());
                    else if (pieces == 3) widen(std::integral_constant<int, kMost <= 2 ? 2 : 3>());
                    else widen(std::integral_constant<int, kMost <= 2 ? 2 : 4>());
                    if (!ok) break;
                    fence_async_shared();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_pair(S::CG == 2 ? cluster_addr(full16(c), 0) : full16(c));
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(bars + S::N8 + s);
            }
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if constexpr (S::CG == 2 || S::SPLIT) cluster_sync_all();      // the peer is done with this CTA's memory
    tc_fence_after();
    if (tid == 0 && waits->abort && dev_error) atomicOr(dev_error, MOE_DEV_ERR_TIMEOUT);
    if (warp == 1) tmem_free<S::CG>(tmem, kTmemColumns);
}

// [rows, H] bytes, in boxes of kStep bytes by `box` rows, 128-byte swizzle.
bool byte_map(CUtensorMap *map, const void *p, uint64_t rows, uint64_t H, uint32_t box)
{
    const cuuint64_t dims[2] = {H, rows}, strides[1] = {H};
    const cuuint32_t boxes[2] = {kStep, box};
    return encode_tiled(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, p, dims, strides, boxes);
}

template <typename S>
cudaError_t run(const void *x, const float *x_scales, const void *w, const float *w_scales,
                const int32_t *offsets, int rows, int H, int N, int E, int sms, int parts, void *out,
                uint32_t *dev_error, long long wait_limit, int stall, cudaStream_t stream)
{
    CUtensorMap map_w;
    RowMaps map_x;
    if (!byte_map(&map_w, w, (uint64_t)E * N, H, kChannels)) return cudaErrorInvalidValue;
    for (int m = 0; m < kBoxes; ++m)                   // higher boxes than a CTA's rows are not used
        if (kLeastBox << m > S::BR) map_x.box[m] = map_x.box[0];
        else if (!byte_map(&map_x.box[m], x, rows, H, kLeastBox << m)) return cudaErrorInvalidValue;
    const size_t smem = S::bytes(E);
    cudaError_t e = allow_dynamic_smem(reinterpret_cast<const void *>(&expert_matmul_int8_kernel<S>), smem);
    if (e != cudaSuccess) return e;
    const int64_t tiles = most_tiles<S>(rows, E) * ceil_div(N, kChannels * S::CG);
    const int64_t groups = tiles < sms / (S::CG * parts) ? tiles : sms / (S::CG * parts);
    return launch_pdl_clusters(expert_matmul_int8_kernel<S>, dim3((unsigned)groups * S::CG * parts), dim3(S::THREADS),
                               smem, stream, S::CG * parts, map_w, map_x, x_scales, w_scales, offsets, rows, H, N, E,
                               static_cast<__nv_bfloat16 *>(out), dev_error, wait_limit, stall);
}

}  // namespace

cudaError_t launch_expert_matmul_int8(const void *x, const float *x_scales, const void *w,
                                      const float *w_scales, const int32_t *offsets, int rows,
                                      int H, int N, int E, void *out, uint32_t *dev_error,
                                      cudaStream_t stream, int64_t wait_cycles, int stall)
{
    const long long wait_limit = wait_cycles > 0 ? wait_cycles : kWaitLimitCycles;
    int sms = 0;
    cudaError_t e = device_sm_count(&sms);
    if (e != cudaSuccess) return e;
    auto go = [&](auto shape, int parts) {
        return run<decltype(shape)>(x, x_scales, w, w_scales, offsets, rows, H, N, E, sms, parts, out, dev_error,
                                    wait_limit, stall, stream);
    };
    // Few tiles: share the contraction, as far as every tile's cluster runs at
    // once and the steps saved outweigh the cluster's barriers (30 tiles of 4272:
    // 12.2 -> 9.3 us; 4 tiles of 992, 8 steps: 6.4 -> 7.2 us).
    const int64_t tiles = most_tiles<Split>(rows, E) * ceil_div(N, kChannels);
    const int steps = ceil_div(H, kStep);
    if (tiles * 2 <= sms && steps >= 16) {
        int clusters[3];
        e = split_clusters<expert_matmul_int8_kernel<Split>>(Split::THREADS, Split::bytes(MOE_MAX_EXPERTS), clusters);
        if (e != cudaSuccess) return e;
        int parts = 1;
        for (int p = 2; p <= 8 && steps >= 4 * p; p *= 2)
            if (tiles <= clusters[p / 4]) parts = p;
        if (parts > 1) return go(Split{}, parts);
    }
    // By rows an expert, on average; up to 16 measured with even counts only.
    // Narrow and Mid: 56.3 and 58.1 us at 8 (15 experts, 6208 -> 3586), 93 and 53
    // us at 64 (64, 1024 -> 4096).  Mid and Wide: 68 and 77 us at 128 (64, 2048 ->
    // 2048), 248 and 232 us at 384 (32, 7168 -> 2048), 667 and 638 us at 1024 (64,
    // 4096 -> 2048).  A short contraction leaves Wide waiting for its stores, which
    // Mid's alternate accumulators hide: 300 and 321 us (64 experts of 1024 rows,
    // 512 -> 4096), equal at 2560.
    if (rows <= 16 * E) return go(Narrow{}, 1);
    return rows >= 384 * E && steps >= 20 ? go(Wide{}, 1) : go(Mid{}, 1);
}

}  // namespace moe

// Test hook, deliberately absent from the public header: the product with a
// chosen bound on every wait (in clock cycles; 0: the default) and, in the
// CTAs of the first tiles, one barrier that waits for an arrival that never
// comes: stall 0 a tile's bytes in shared memory, 1 their slot free again, 2
// widened operands, 3 their slot free again, 4 sums ready, 5 sums stored, 6 the
// other CTAs' sums (where the contraction is split); anything else none.  A
// test uses it to see a bounded wait expire: the kernel sets
// MOE_DEV_ERR_TIMEOUT and finishes, and the context stays usable.  Arguments
// are checked by the caller (tests only).
extern "C" __attribute__((visibility("default"))) int32_t
moe_testing_expert_matmul_int8(const void *x, const float *x_scales, const void *weights,
                               const float *w_scales, const int32_t *expert_offsets, int32_t rows,
                               int32_t H, int32_t N, int32_t E, void *out, uint32_t *dev_error,
                               int64_t wait_cycles, int32_t stall, cudaStream_t stream)
{
    const cudaError_t e = moe::launch_expert_matmul_int8(x, x_scales, weights, w_scales, expert_offsets, rows, H, N, E,
                                                         out, dev_error, stream, wait_cycles, stall);
    return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}
