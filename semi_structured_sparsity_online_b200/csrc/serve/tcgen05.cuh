// PTX wrappers of the 5th-generation tensor cores for the serving kernels:
// tensor memory, shared-memory descriptors, MMAs, commits, TMA boxes.
#pragma once

#include <cudaTypedefs.h>

#include "../device.cuh"

namespace ss24 {
namespace tc {

// Waits for the barrier's phase with the given parity; false if that takes
// longer than limit_ns. The timer is looked at late: reading it takes longer
// than most waits here last.
__device__ __forceinline__ bool wait(uint64_t *bar, uint32_t parity, uint64_t limit_ns)
{
    uint64_t t0 = 0;
    for (int n = 0;; ++n) {
        if (mbar_try_wait(bar, parity))
            return true;
        if (n >= 64 && n % 64 == 0) {
            const uint64_t t = global_timer_ns();
            if (t0 == 0)
                t0 = t;
            else if (t - t0 > limit_ns)
                return false;
        }
    }
}

// The same by a whole warp, with one answer for all lanes: one that gave up by
// itself would leave the others in the next vote or shuffle.
__device__ __forceinline__ bool wait_warp(uint64_t *bar, uint32_t parity, uint64_t limit_ns)
{
    return __all_sync(kFull, wait(bar, parity, limit_ns));
}

// The warp's number, and a value that is the same in all its lanes, in a form
// the compiler takes as uniform.
__device__ __forceinline__ int uniform(int v) { return __shfl_sync(kFull, v, 0); }

// Shared-memory matrix descriptor of a 128-byte swizzled operand: its high word
// is the same for all (groups of 8 rows 1024 bytes apart, version 1, the
// swizzle), its low word holds the address and the leading byte offset in
// 16-byte units, so that a step along the operand is an addition to it.
__device__ __forceinline__ uint64_t desc(uint32_t low)
{
    constexpr uint32_t kHigh = 64u | 1u << 14 | 2u << 29;
    return static_cast<uint64_t>(kHigh) << 32 | low;
}
// K-major operand: rows of 128 bytes.
__device__ __forceinline__ uint32_t desc_low_kmajor(uint32_t addr) { return (addr >> 4) + (1u << 16); }
__device__ __forceinline__ uint64_t desc_kmajor(uint32_t addr) { return desc(desc_low_kmajor(addr)); }
// MN-major operand (the MMA's m or n contiguous): rows of k with 128 bytes of
// n each, the next 128 bytes of n n_stride bytes on.
__device__ __forceinline__ uint32_t desc_low_mnmajor(uint32_t addr, uint32_t n_stride)
{
    return (addr >> 4) + (n_stride >> 4 << 16);
}

__device__ __forceinline__ void alloc(uint32_t *dst_smem, uint32_t cols)
{
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(dst_smem)),
                 "r"(cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::);
}
__device__ __forceinline__ void dealloc(uint32_t taddr, uint32_t cols)
{
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(cols) : "memory");
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
// Generic-proxy writes to shared memory become visible to the tensor cores.
__device__ __forceinline__ void fence_proxy() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void commit(uint64_t *bar, bool lead)
{
    asm volatile("{\n .reg .pred q;\n setp.ne.b32 q, %1, 0;\n"
                 " @q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(smem_u32(bar)),
                 "r"(static_cast<uint32_t>(lead))
                 : "memory");
}
__device__ __forceinline__ void wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// MMAs and commits are issued by the lane with `lead` set, but by code that the
// whole warp runs: descriptors then stay in uniform registers. In a branch of
// one lane each operand moves there first, which measured 76 cycles an MMA of 64.

// D[tmem] (+)= A[smem] B[smem], INT8 x INT8 -> INT32
__device__ __forceinline__ void mma_i8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate,
                                         bool lead)
{
    asm volatile("{\n .reg .pred p, q;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 q, %5, 0;\n"
                 " @q tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
                 "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(static_cast<uint32_t>(lead))
                 : "memory");
}

// D[tmem] (+)= A[smem] B[smem], fp16 x fp16 -> binary32
__device__ __forceinline__ void mma_f16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate,
                                         bool lead)
{
    asm volatile("{\n .reg .pred p, q;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 q, %5, 0;\n"
                 " @q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
                 "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(static_cast<uint32_t>(lead))
                 : "memory");
}
// the same with A in tensor memory (two values of k per 32-bit column)
__device__ __forceinline__ void mma_f16_ta(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate,
                                         bool lead)
{
    asm volatile("{\n .reg .pred p, q;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 q, %5, 0;\n"
                 " @q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
                 "r"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(static_cast<uint32_t>(lead))
                 : "memory");
}

// 32 consecutive columns of this thread's lane (not waited for).
__device__ __forceinline__ void ld32(uint32_t taddr, uint32_t (&v)[32])
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
                 "%14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
                   "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]),
                   "=r"(v[15]), "=r"(v[16]), "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]),
                   "=r"(v[22]), "=r"(v[23]), "=r"(v[24]), "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]),
                   "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
                 : "r"(taddr));
}
__device__ __forceinline__ void ld16(uint32_t taddr, uint32_t (&v)[16])
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
                 "%14, %15}, [%16];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
                   "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]),
                   "=r"(v[15])
                 : "r"(taddr));
}

__device__ __forceinline__ void st32(uint32_t taddr, const uint32_t (&v)[32])
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, "
                 "%13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};"
                 ::"r"(taddr),
                 "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]),
                 "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(v[16]),
                 "r"(v[17]), "r"(v[18]), "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]), "r"(v[24]),
                 "r"(v[25]), "r"(v[26]), "r"(v[27]), "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31])
                 : "memory");
}

// ---- pairs of CTAs (cta_group::2): the even rank of a cluster of two issues
// the MMAs for both; shared-memory offsets and tensor-memory addresses are the
// same in both ----

__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync()
{
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The shared-memory address of CTA `rank` of the cluster at this CTA's `addr`.
__device__ __forceinline__ uint32_t cluster_addr(uint32_t addr, uint32_t rank)
{
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
// Arrival on a barrier of the cluster (an address from cluster_addr). What it
// hands over went through a proxy or tcgen05 fence of its own before: a release
// at cluster scope, which also waits for the thread's global loads, measured
// 1000 cycles an arrival in the attention kernel.
__device__ __forceinline__ void arrive_cluster(uint32_t addr)
{
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(addr) : "memory");
}
__device__ __forceinline__ void alloc_pair(uint32_t *dst_smem, uint32_t cols)
{
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(dst_smem)),
                 "r"(cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::);
}
__device__ __forceinline__ void dealloc_pair(uint32_t taddr, uint32_t cols)
{
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(cols) : "memory");
}
// Arrives on the barrier at `bar`'s offset in both CTAs once the MMAs issued
// before it have finished.
__device__ __forceinline__ void commit_pair(uint64_t *bar, bool lead)
{
    asm volatile("{\n .reg .pred q;\n setp.ne.b32 q, %2, 0;\n"
                 " @q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n}\n" ::"r"(
                     smem_u32(bar)),
                 "h"(static_cast<uint16_t>(3)), "r"(static_cast<uint32_t>(lead))
                 : "memory");
}
__device__ __forceinline__ void mma_i8_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate,
                                         bool lead)
{
    asm volatile("{\n .reg .pred p, q;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 q, %5, 0;\n"
                 " @q tcgen05.mma.cta_group::2.kind::i8 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
                 "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(static_cast<uint32_t>(lead))
                 : "memory");
}
__device__ __forceinline__ void mma_f16_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate,
                                         bool lead)
{
    asm volatile("{\n .reg .pred p, q;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 q, %5, 0;\n"
                 " @q tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
                 "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(static_cast<uint32_t>(lead))
                 : "memory");
}
__device__ __forceinline__ void mma_f16_ta_pair(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate,
                                         bool lead)
{
    asm volatile("{\n .reg .pred p, q;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 q, %5, 0;\n"
                 " @q tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
                 "r"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(static_cast<uint32_t>(lead))
                 : "memory");
}
// A box into this CTA's shared memory, completing on a barrier of the pair (an
// address from cluster_addr).
__device__ __forceinline__ void tma_box_pair(uint32_t dst_smem, const CUtensorMap *map, int32_t c_inner, int32_t c_outer,
                                             uint32_t bar)
{
    asm volatile("cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
                 " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst_smem),
                 "l"(reinterpret_cast<uint64_t>(map)), "r"(c_inner), "r"(c_outer), "r"(bar)
                 : "memory");
}

// 2-D tiled TMA load of one box, completing on `bar`. c_inner times the
// element size is a multiple of 16 bytes.
__device__ __forceinline__ void tma_box(uint32_t dst_smem, const CUtensorMap *map, int32_t c_inner, int32_t c_outer,
                                        uint64_t *bar)
{
    asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
                 " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst_smem),
                 "l"(reinterpret_cast<uint64_t>(map)), "r"(c_inner), "r"(c_outer), "r"(smem_u32(bar))
                 : "memory");
}

} // namespace tc
} // namespace ss24
