// sfm_pair.cuh -- building blocks for kernels whose CTAs work in pairs: matrix
// products over the shared memory of both (tcgen05 cta_group::2), copies that
// report to a barrier of the pair's first CTA, arrivals at the other CTA's
// barriers, and waits that see what it wrote.
//
// A product of M = 128 rows in a pair takes 64 rows of A and half of the rows
// (columns of the product) of B from each CTA, at the same offsets in both.
// CTA c's tensor memory then holds its 64 rows: lanes 0-63 columns [0, N / 2),
// lanes 64-127 columns [N / 2, N), N / 2 columns wide.
//
// Products are issued by the lane that elect.sync names, inside a branch on a
// warp's number that is uniform to the compiler (__shfl_sync), with all
// descriptors computed from uniform values: a 128 x 128 x 16 product of the
// pair then takes 32 clocks and a 128 x 256 x 16 one 64 (the tensor cores'
// rate).  Issued by lane 0 of a branch on threadIdx each of them took 180.
#pragma once

#include <cuda.h>

#include "sfm_tc.cuh"

namespace sfm {
namespace tc {

__device__ __forceinline__ bool elect_one()
{
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}\n" : "=r"(p));
    return p != 0;
}

__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

// Address of a shared variable in another CTA of the cluster.
__device__ __forceinline__ uint32_t in_cta(uint32_t addr, uint32_t rank)
{
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}

__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}


// Arrive at a barrier of either CTA.  This thread's writes to its own CTA's memory (made visible to the tensor cores by a
// proxy fence) and its tensor memory accesses come before it; what it wrote into the other CTA's does after
// arrive_remote_release() alone, which waits for those writes and took 1500 clocks per softmax warp and tile.
__device__ __forceinline__ void arrive_remote(uint32_t cluster_bar)
{
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_bar) : "memory");
}

__device__ __forceinline__ void arrive_remote_release(uint32_t cluster_bar)
{
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_bar) : "memory");
}

__device__ __forceinline__ void store_remote(uint32_t cluster_addr, uint32_t v)
{
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(cluster_addr), "r"(v) : "memory");
}

__device__ __forceinline__ void or_remote(uint32_t cluster_addr, uint32_t v)
{
    asm volatile("red.relaxed.cluster.shared::cluster.or.b32 [%0], %1;" ::"r"(cluster_addr), "r"(v) : "memory");
}

__device__ __forceinline__ void fence_cluster() { asm volatile("fence.acq_rel.cluster;" ::: "memory"); }

__device__ __forceinline__ void expect_tx(uint32_t bar, uint32_t bytes)
{
    asm volatile("mbarrier.arrive.expect_tx.release.cta.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}

__device__ __forceinline__ bool pair_try_wait(uint32_t bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}\n"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}

// Wait for a phase that threads of either CTA complete; bounded like mbar_wait.
__device__ __forceinline__ bool pair_wait(uint32_t bar, uint32_t parity, volatile int *abort)
{
    if (pair_try_wait(bar, parity)) return true;
    const uint64_t t0 = globaltimer_ns();
    while (!pair_try_wait(bar, parity)) {
        if (*abort) return false;
        if (globaltimer_ns() - t0 > kTimeoutNs) {
            *abort = 1;
            return false;
        }
    }
    return true;
}

// The same for a whole warp: one verdict for all lanes.
__device__ __forceinline__ bool pair_wait_warp(uint32_t bar, uint32_t parity, volatile int *abort)
{
    const bool ok = pair_wait(bar, parity, abort);
    return __all_sync(0xffffffffu, ok);
}

__device__ __forceinline__ void pair_alloc(uint32_t dst_smem, uint32_t ncols)
{
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst_smem), "r"(ncols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void pair_dealloc(uint32_t taddr, uint32_t ncols)
{
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}

// A shared-memory matrix descriptor (sdesc_sw128) as two words: operands a few bytes on differ in the first one only, by the
// bytes / 16, so that a product needs one addition per operand.
struct Desc {
    uint32_t lo, hi;
};

__device__ __forceinline__ Desc desc_sw128(uint32_t addr, uint32_t lbo, uint32_t sbo)
{
    const uint64_t d = sdesc_sw128(addr, lbo, sbo);
    return {static_cast<uint32_t>(d), static_cast<uint32_t>(d >> 32)};
}

__device__ __forceinline__ uint64_t desc_at(const Desc &d, uint32_t bytes)
{
    return static_cast<uint64_t>(d.hi) << 32 | (d.lo + (bytes >> 4));
}

__device__ __forceinline__ void pair_mma(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}\n"
        ::"r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Arrive at this barrier of both CTAs once every product issued so far is done.
__device__ __forceinline__ void pair_commit(uint32_t bar)
{
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
                 "h"((uint16_t)3)
                 : "memory");
}

// Copy a box into this CTA's memory, counted at a barrier of the pair (a shared::cluster address).
__device__ __forceinline__ void pair_load(uint32_t dst, const CUtensorMap *map, int x, int y, int z, uint32_t cluster_bar)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
        ::"r"(dst), "l"(map), "r"(x), "r"(y), "r"(z), "r"(cluster_bar)
        : "memory");
}

// The same from rows in groups of eight (four dimensions: values, rows of a group, blocks, groups).
__device__ __forceinline__ void pair_load_octets(uint32_t dst, const CUtensorMap *map, int block, int octet, uint32_t cluster_bar)
{
    asm volatile(
        "cp.async.bulk.tensor.4d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %2, %3, %4}], [%5];"
        ::"r"(dst), "l"(map), "r"(0), "r"(block), "r"(octet), "r"(cluster_bar)
        : "memory");
}

__device__ __forceinline__ void prefetch_map(const CUtensorMap *map)
{
    asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}

}  // namespace tc
}  // namespace sfm
