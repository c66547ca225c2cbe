// tc.cuh -- the fifth-generation tensor cores, from PTX: tensor-map copies,
// tensor memory, matrix instructions of a pair of blocks, and waits with a limit.
#pragma once

#include <cuda.h> // CUtensorMap
#include <cuda_runtime.h>
#include <stdint.h>

#include "rra_device.cuh"

namespace rra {

// ---------------------------------------------------------------- barriers

// A wait gives up after this long, or when another of its block has: `stop` is a
// word in shared memory, `stalled` one that the host reads.
constexpr uint64_t kWaitLimitNs = 4000000000ull;

// One test of a phase; what either block of the pair did before it is visible.
__device__ __forceinline__ bool try_wait_cluster(uint64_t *bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile("{\n\t.reg .pred p;\n\t"
                 "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
                 "selp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(ok)
                 : "r"(smem_u32(bar)), "r"(parity)
                 : "memory");
    return ok != 0;
}

__device__ __forceinline__ bool wait_limited(uint64_t *bar, uint32_t parity, volatile uint32_t *stop,
                                             unsigned *stalled)
{
    if (try_wait_cluster(bar, parity))
        return true;
    const uint64_t t0 = global_ns();
    for (uint32_t i = 1;; ++i) {
        if (try_wait_cluster(bar, parity))
            return true;
        if (i % 64 == 0) {
            if (*stop)
                return false;
            if (global_ns() - t0 > kWaitLimitNs) {
                *stop = 1;
                *reinterpret_cast<volatile unsigned *>(stalled) = 1;
                return false;
            }
        }
    }
}

// Barrier `id` of `threads` threads of the block.
__device__ __forceinline__ void named_barrier(int id, int threads)
{
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
// The same; true where all of them say so.
__device__ __forceinline__ bool named_all(int id, int threads, bool yes)
{
    uint32_t r;
    asm volatile("{\n\t.reg .pred p, q;\n\t"
                 "setp.ne.u32 p, %3, 0;\n\t"
                 "barrier.cta.red.and.pred q, %1, %2, p;\n\t"
                 "selp.u32 %0, 1, 0, q;\n\t}"
                 : "=r"(r)
                 : "r"(id), "r"(threads), "r"((uint32_t)yes)
                 : "memory");
    return r != 0;
}

// The address of this block's shared memory `p` in block `rank` of its cluster.
__device__ __forceinline__ uint32_t cluster_address(const void *p, uint32_t rank)
{
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
    return a;
}

__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

__device__ __forceinline__ void cluster_barrier()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n\t"
                 "barrier.cluster.wait.acquire.aligned;" ::
                     : "memory");
}

// One arrival on a barrier of a block of the cluster.
__device__ __forceinline__ void arrive_at(uint32_t bar)
{
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar)
                 : "memory");
}

// ---------------------------------------------------------------- tensor maps

__device__ __forceinline__ void prefetch_map(const CUtensorMap *m)
{
    asm volatile("prefetch.tensormap [%0];" ::"l"(m) : "memory");
}

// A box of plane z of the tensor from (x, y) on to shared memory; its bytes count on
// `bar`, a cluster address (of either block of the pair).
__device__ __forceinline__ void load_box(void *to, const CUtensorMap *m, int x, int y, int z,
                                         uint32_t bar)
{
    asm volatile("cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile."
                 "mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_u32(to)),
                 "l"(m), "r"(x), "r"(y), "r"(z), "r"(bar)
                 : "memory");
}

// ---------------------------------------------------------------- tensor memory

constexpr uint32_t kTmemColumns = 512;

__device__ __forceinline__ void tmem_alloc(uint32_t *to)
{
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(to)),
                 "r"(kTmemColumns)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
}

__device__ __forceinline__ void tmem_free(uint32_t at)
{
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(at),
                 "r"(kTmemColumns));
}

// 32 columns of this warp's 32 lanes, a lane each.
__device__ __forceinline__ void tmem_load(uint32_t at, uint32_t (&r)[32])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
          "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
          "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(at));
}

// 16 columns.
__device__ __forceinline__ void tmem_load(uint32_t at, uint32_t (&r)[16])
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 "
                 "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
                   "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]),
                   "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
                 : "r"(at));
}

__device__ __forceinline__ void tmem_store(uint32_t at, const uint32_t (&r)[32])
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
        "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(at),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
        "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
        "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]),
        "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]),
        "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}

__device__ __forceinline__ void tmem_stored()
{
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void tmem_loaded()
{
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void tc_fence_before()
{
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_after()
{
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}

// ---------------------------------------------------------------- matrix instructions

// Operands lie in shared memory as tensor maps with 128-byte swizzle leave them.
// Along k: rows of 64 elements of k (128 bytes), groups of 8 rows 1024 bytes apart;
// 16 elements of k are 32 bytes.  Along the rows (m or n): for each k a line of 64
// rows (128 bytes), groups of 8 k 1024 bytes apart, the next 64 rows `block` bytes on;
// 16 elements of k are 2048 bytes.
__device__ __forceinline__ uint64_t operand_along_k(const void *p)
{
    return (uint64_t)((smem_u32(p) >> 4) & 0x3fff) | (uint64_t)1 << 16 | (uint64_t)(1024 >> 4) << 32 |
           (uint64_t)1 << 46 | (uint64_t)2 << 61;
}
__device__ __forceinline__ uint64_t operand_along_rows(const void *p, uint32_t block)
{
    return (uint64_t)((smem_u32(p) >> 4) & 0x3fff) | (uint64_t)(block >> 4) << 16 |
           (uint64_t)(1024 >> 4) << 32 | (uint64_t)1 << 46 | (uint64_t)2 << 61;
}
// The same operand 16 elements of k further, in units of the descriptor's address.
constexpr uint64_t kStepAlongK = 32 >> 4, kStepAlongRows = 2048 >> 4;

// Shape and types of one instruction: fp32 sums of bf16 or fp16 products.
__host__ __device__ constexpr uint32_t mma_kind(bool bf16, bool a_rows, bool b_rows, int m, int n)
{
    return 1u << 4 | (bf16 ? 1u : 0u) << 7 | (bf16 ? 1u : 0u) << 10 | (a_rows ? 1u : 0u) << 15 |
           (b_rows ? 1u : 0u) << 16 | (uint32_t)(n >> 3) << 17 | (uint32_t)(m >> 4) << 24;
}

// sums[at] (+)= a b, over both blocks of the pair; one thread of the first block.
__device__ __forceinline__ void mma_pair(uint32_t at, uint64_t a, uint64_t b, uint32_t kind, bool add)
{
    asm volatile("{\n\t.reg .pred p;\n\t"
                 "setp.ne.u32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(at),
                 "l"(a), "l"(b), "r"(kind), "r"((uint32_t)add)
                 : "memory");
}

// An arrival at `bar` of both blocks when the instructions so far are done.
__device__ __forceinline__ void mma_commit_pair(uint64_t *bar)
{
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster."
                 "multicast::cluster.b64 [%0], %1;" ::"r"(smem_u32(bar)),
                 "h"((uint16_t)3)
                 : "memory");
}

} // namespace rra
