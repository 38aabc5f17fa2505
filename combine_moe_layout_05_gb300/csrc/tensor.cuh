// tensor.cuh -- the fifth-generation tensor core path as hand-written PTX:
// tiled copies into shared memory, tensor memory (TMEM) allocation and
// access, matrix instructions and the barriers between them, for one CTA or
// a pair of CTAs that work on one tile.
//
// Waits are bounded as in bulk.cuh: a wait that outlives its limit returns
// false, so a missing arrival becomes an error status instead of a hang.
#pragma once

#include <cuda.h>

#include "bulk.cuh"

namespace moe {

// About 2 s; the longest tile takes well under 1 ms.  Counted in clock cycles:
// a read of the nanosecond timer takes long enough to delay every wait.
constexpr long long kWaitLimitCycles = 4000000000ll;

// A block's, in its shared memory: how long a wait may take, and whether one
// took longer.
struct WaitState {
    long long limit;
    volatile int abort;
};

__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

__device__ __forceinline__ int cluster_size()
{
    uint32_t n;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(n));
    return (int)n;
}

// Every thread of the cluster; orders shared memory of both CTAs.
__device__ __forceinline__ void cluster_sync_all()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Address of this CTA's shared variable in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t cluster_addr(uint32_t addr, uint32_t rank)
{
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}

__device__ __forceinline__ void st_cluster_u32(uint32_t cluster_at, uint32_t v)
{
    asm volatile("st.shared::cluster.u32 [%0], %1;" :: "r"(cluster_at), "r"(v) : "memory");
}

// One arrival on a barrier of the cluster, after this warp's earlier writes to
// the cluster's shared memory (synchronise the warp first).
__device__ __forceinline__ void mbar_arrive_release(uint32_t cluster_bar)
{
    asm volatile("fence.acq_rel.cluster;\n\tmbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];"
                 :: "r"(cluster_bar) : "memory");
}

// One arrival on a barrier of the pair.  What it announces is read by the
// tensor cores alone, each from its own CTA's memory, and was handed to them
// by fence.proxy.async or tcgen05.wait before: no cluster-wide release of
// ordinary writes is asked for (it costs a memory barrier, 0.4 us, each time).
// A CTA may leave only when every arrival on its barriers has been waited for:
// one that finds its target gone is a fault.
__device__ __forceinline__ void mbar_arrive_pair(uint32_t cluster_bar)
{
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" :: "r"(cluster_bar) : "memory");
}

// Lane 0's value, which the compiler then knows to be the warp's: branches on
// it do not diverge, and operands made from it stay in uniform registers.
template <typename T>
__device__ __forceinline__ T uniform(T v)
{
    return __shfl_sync(kFullMask, v, 0);
}

// True in one lane of a converged warp.  Instructions of the copy engine and
// the tensor core are issued behind it, in code the whole warp runs: behind a
// test of the lane number the compiler loops over the lanes to make their
// operands uniform, 150 cycles an instruction.
__device__ __forceinline__ bool elect_one()
{
    uint32_t one;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(one));
    return one != 0;
}

// Whether the phase with the given parity is over; asks once.
__device__ __forceinline__ bool mbar_test_cluster(uint32_t bar, uint32_t parity)
{
    uint32_t done;
    asm volatile("{\n\t.reg .pred p;\n\t"
                 "mbarrier.test_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
                 "selp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(done) : "r"(bar), "r"(parity) : "memory");
    return done != 0;
}

// The same, asleep for a while until it is.
__device__ __forceinline__ bool mbar_sleep_cluster(uint32_t bar, uint32_t parity)
{
    uint32_t done;
    asm volatile("{\n\t.reg .pred p;\n\t"
                 "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
                 "selp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(done) : "r"(bar), "r"(parity) : "memory");
    return done != 0;
}

// Waits for the phase of `bar` with the given parity; false, and w->abort set,
// when the limit passed or another thread of the block gave up.  Once, not
// inline: the kernel's warps run different loops, which together have to stay
// in the instruction cache.
static __device__ __noinline__ bool mbar_wait_long(uint32_t bar, uint32_t parity, WaitState *w)
{
    const long long start = clock64(), limit = w->limit;
    while (!mbar_sleep_cluster(bar, parity))
        if (w->abort || clock64() - start > limit) {
            w->abort = 1;
            return false;
        }
    return true;
}

__device__ __forceinline__ bool mbar_wait_bounded(uint32_t bar, uint32_t parity, WaitState *w)
{
    return mbar_sleep_cluster(bar, parity) || mbar_wait_long(bar, parity, w);
}

// The same for a copy or matrix instructions in flight, which have to land
// before the block leaves, whether it gave up or not.
__device__ __forceinline__ void mbar_drain_bounded(uint32_t bar, uint32_t parity, const WaitState *w)
{
    const long long start = clock64(), limit = w->limit;
    while (!mbar_sleep_cluster(bar, parity))
        if (clock64() - start > limit) return;
}

// Tile of a two-dimensional tensor at (column c, row r) to shared memory;
// the bytes are counted on `bar`.
__device__ __forceinline__ void tile_load_2d(uint32_t dst, const CUtensorMap *map, int c, int r, uint32_t bar)
{
    asm volatile("cp.async.bulk.tensor.2d.shared::cta.global.tile.mbarrier::complete_tx::bytes "
                 "[%0], [%1, {%2, %3}], [%4];"
                 :: "r"(dst), "l"(map), "r"(c), "r"(r), "r"(bar) : "memory");
}

__device__ __forceinline__ void tile_load_3d(uint32_t dst, const CUtensorMap *map, int c, int r, int z, uint32_t bar)
{
    asm volatile("cp.async.bulk.tensor.3d.shared::cta.global.tile.mbarrier::complete_tx::bytes "
                 "[%0], [%1, {%2, %3, %4}], [%5];"
                 :: "r"(dst), "l"(map), "r"(c), "r"(r), "r"(z), "r"(bar) : "memory");
}

__device__ __forceinline__ void tile_load_4d(uint32_t dst, const CUtensorMap *map, int c, int r, int y, int z, uint32_t bar)
{
    asm volatile("cp.async.bulk.tensor.4d.shared::cta.global.tile.mbarrier::complete_tx::bytes "
                 "[%0], [%1, {%2, %3, %4, %5}], [%6];"
                 :: "r"(dst), "l"(map), "r"(c), "r"(r), "r"(y), "r"(z), "r"(bar) : "memory");
}

// A tile from shared memory to a three-dimensional tensor, or added to what is
// there; what lies outside the tensor is left out.  In the thread's bulk group.
__device__ __forceinline__ void tile_store_3d(const CUtensorMap *map, int c, int r, int z, uint32_t src)
{
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];"
                 :: "l"(map), "r"(c), "r"(r), "r"(z), "r"(src) : "memory");
}

__device__ __forceinline__ void tile_add_3d(const CUtensorMap *map, int c, int r, int z, uint32_t src)
{
    asm volatile("cp.reduce.async.bulk.tensor.3d.global.shared::cta.add.tile.bulk_group [%0, {%1, %2, %3}], [%4];"
                 :: "l"(map), "r"(c), "r"(r), "r"(z), "r"(src) : "memory");
}

__device__ __forceinline__ void prefetch_l2(const void *p) { asm volatile("prefetch.global.L2 [%0];" :: "l"(p)); }

__device__ __forceinline__ void prefetch_map(const CUtensorMap *map)
{
    asm volatile("prefetch.tensormap [%0];" :: "l"(map) : "memory");
}

// TMEM columns, allocated and freed by one whole warp (of each CTA of a pair).
template <int CG>
__device__ __forceinline__ void tmem_alloc(uint32_t dst_smem, uint32_t columns)
{
    if constexpr (CG == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" :: "r"(dst_smem), "r"(columns) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    } else {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" :: "r"(dst_smem), "r"(columns) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
    }
}

template <int CG>
__device__ __forceinline__ void tmem_free(uint32_t base, uint32_t columns)
{
    if constexpr (CG == 1)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" :: "r"(base), "r"(columns));
    else
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" :: "r"(base), "r"(columns));
}

__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// D (TMEM, fp32) += A (TMEM, fp16) x B (shared memory, fp16, K-major) for 16
// of the contraction.  Issued by one thread (of the pair's first CTA).
template <int CG>
__device__ __forceinline__ void mma_f16_ts(uint32_t d, uint32_t a, uint64_t b_desc, uint32_t idesc, bool accumulate)
{
    if constexpr (CG == 1)
        asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                     "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
                     :: "r"(d), "r"(a), "l"(b_desc), "r"(idesc), "r"((uint32_t)accumulate) : "memory");
    else
        asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                     "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
                     :: "r"(d), "r"(a), "l"(b_desc), "r"(idesc), "r"((uint32_t)accumulate) : "memory");
}

// The same with A in shared memory too; both operands bf16 or both fp16.
template <int CG>
__device__ __forceinline__ void mma_f16_ss(uint32_t d, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, bool accumulate)
{
    if constexpr (CG == 1)
        asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                     "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}"
                     :: "r"(d), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"((uint32_t)accumulate) : "memory");
    else
        asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                     "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}"
                     :: "r"(d), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"((uint32_t)accumulate) : "memory");
}

// One arrival on `bar` (of both CTAs of a pair) once the matrix instructions
// issued so far have completed.
template <int CG>
__device__ __forceinline__ void mma_commit(uint32_t bar)
{
    if constexpr (CG == 1)
        asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" :: "r"(bar) : "memory");
    else
        asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
                     :: "r"(bar), "h"((uint16_t)3) : "memory");
}

// Shared-memory operand, K-major, 128-byte swizzle: rows of 128 bytes, groups
// of 8 rows 1024 bytes apart.
__device__ __forceinline__ uint64_t operand_desc(uint32_t addr)
{
    return (uint64_t)((addr & 0x3ffff) >> 4) | (uint64_t)1 << 16 | (uint64_t)(1024 >> 4) << 32 |
           (uint64_t)1 << 46 | (uint64_t)2 << 61;
}

// Shared-memory operand whose rows lie along the contraction (MN-major): lines
// of 128 bytes (64 rows' values of one step), 8 lines a group, groups 1024
// bytes apart; the next 64 rows are `block` bytes on.
__device__ __forceinline__ uint64_t operand_desc_mn(uint32_t addr, uint32_t block)
{
    return (uint64_t)((addr & 0x3ffff) >> 4) | (uint64_t)(block >> 4) << 16 | (uint64_t)(1024 >> 4) << 32 |
           (uint64_t)1 << 46 | (uint64_t)2 << 61;
}

// kind::f16, A and B bf16, each K-major or not, D fp32.
__device__ __forceinline__ uint32_t instruction_desc_bf16(int M, int N, bool a_mn, bool b_mn)
{
    return 1u << 4 | 1u << 7 | 1u << 10 | (uint32_t)a_mn << 15 | (uint32_t)b_mn << 16 | (uint32_t)(N >> 3) << 17 |
           (uint32_t)(M >> 4) << 24;
}

// kind::f16, A and B fp16 and K-major, D fp32.
__device__ __forceinline__ uint32_t instruction_desc_f16(int M, int N)
{
    return 1u << 4 | (uint32_t)(N >> 3) << 17 | (uint32_t)(M >> 4) << 24;
}

// 32 columns of a warp's 32 TMEM lanes, one lane a thread.
__device__ __forceinline__ void tmem_store_x32(uint32_t addr, const uint32_t (&v)[32])
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
                 "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
                 "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};"
                 :: "r"(addr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]),
                    "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]),
                    "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]),
                    "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]), "r"(v[24]),
                    "r"(v[25]), "r"(v[26]), "r"(v[27]), "r"(v[28]), "r"(v[29]), "r"(v[30]),
                    "r"(v[31])
                 : "memory");
}

// 16 columns of 16 TMEM lanes, spread over the warp as the matrix
// instructions' 8 x 8 blocks: thread t has columns 2(t%4), 2(t%4) + 1 (and 8
// more) of lanes t/4 (words 0, 1; 4, 5) and t/4 + 8 (words 2, 3; 6, 7).
__device__ __forceinline__ void tmem_load_16x16(uint32_t addr, uint32_t *v)
{
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]),
                   "=r"(v[6]), "=r"(v[7])
                 : "r"(addr) : "memory");
}

// 16 columns of a warp's 32 TMEM lanes, one lane a thread.
__device__ __forceinline__ void tmem_load_x16(uint32_t addr, uint32_t (&v)[16])
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
                   "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
                 : "r"(addr) : "memory");
}

// Four 8 x 8 blocks of 16-bit words, turned: block q's word (i, j), held by
// thread 4i + j/2, goes to word i of the row that thread 8q + j points at.
__device__ __forceinline__ void store_turned_x4(uint32_t row, uint32_t a, uint32_t b, uint32_t c, uint32_t d)
{
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};"
                 :: "r"(row), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

// And back: thread 4i + j/2 gets word (i, j) from the rows that word (i, j) was
// stored to.
__device__ __forceinline__ void load_turned_x4(uint32_t row, uint32_t (&v)[4])
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]) : "r"(row) : "memory");
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

}  // namespace moe
