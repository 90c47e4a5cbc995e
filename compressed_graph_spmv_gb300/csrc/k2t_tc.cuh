// k2t_tc.cuh -- tensor-core (tcgen05) and mbarrier instructions of sm_103a
// that the attention kernels use, and the shared-memory layouts they read.
#pragma once

#include <cstdint>

namespace k2t {
namespace tc {

__device__ __forceinline__ uint32_t saddr(const void *p) { return (uint32_t)__cvta_generic_to_shared(p); }

// ---- mbarriers --------------------------------------------------------------
__device__ __forceinline__ void bar_init(uint64_t *b, uint32_t count)
{
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(saddr(b)), "r"(count) : "memory");
}
__device__ __forceinline__ void bar_arrive(uint64_t *b)
{
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(saddr(b)) : "memory");
}
__device__ __forceinline__ bool bar_test(uint64_t *b, uint32_t parity)
{
    uint32_t ok;
    asm volatile("{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(ok) : "r"(saddr(b)), "r"(parity) : "memory");
    return ok;
}
__device__ __forceinline__ bool bar_peek(uint64_t *b, uint32_t parity)   // without waiting
{
    uint32_t ok;
    asm volatile("{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(ok) : "r"(saddr(b)), "r"(parity) : "memory");
    return ok;
}
// Bounded wait: gives up after about a second (2^31 cycles), or when another
// warp of the block has; false tells the caller to leave its loop.
__device__ __forceinline__ bool bar_wait(uint64_t *b, uint32_t parity, volatile uint32_t *gave_up)
{
    if (bar_test(b, parity)) return true;
    const long long start = clock64();
    while (!bar_test(b, parity)) {
        if (*gave_up) return false;
        if (clock64() - start > (1ll << 31)) {
            *gave_up = 1;
            return false;
        }
    }
    return true;
}
// The same bound for a warp that polls several barriers.
struct Patience {
    volatile uint32_t *gave_up;
    long long start;
    __device__ explicit Patience(volatile uint32_t *g)
    {
        gave_up = g;
        start = clock64();
    }
    __device__ void restart() { start = clock64(); }
    __device__ bool more()
    {
        __nanosleep(20);      // polling takes issue slots from the warps that share the scheduler
        if (clock64() - start > (1ll << 31)) *gave_up = 1;
        return !*gave_up;
    }
};
// Counts on the barrier once this thread's earlier cp.async copies have landed (part of the barrier's count).
__device__ __forceinline__ void cp_arrive(uint64_t *b)
{
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(saddr(b)) : "memory");
}
// Writes of this thread to shared memory, made visible to the tensor cores' reads.
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// ---- tensor memory ------------------------------------------------------------
__device__ __forceinline__ void alloc(uint32_t *at, uint32_t columns)
{
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(saddr(at)), "r"(columns) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void dealloc(uint32_t at, uint32_t columns)
{
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(at), "r"(columns) : "memory");
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// 32 columns of this warp's 32 lanes (lane = thread), as bits.
__device__ __forceinline__ void ld32(uint32_t (&r)[32], uint32_t at)
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(at) : "memory");
}
__device__ __forceinline__ void st32(uint32_t at, const uint32_t (&r)[32])
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
        "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(at),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
        "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
        "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31]) : "memory");
}
__device__ __forceinline__ void st16(uint32_t at, const uint32_t (&r)[16])
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(at),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]) : "memory");
}

__device__ __forceinline__ void ld16(uint32_t (&r)[16], uint32_t at)
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
                 : "r"(at) : "memory");
}
__device__ __forceinline__ void st8(uint32_t at, const uint32_t (&r)[8])
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(at), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}

__device__ __forceinline__ void ld8(uint32_t (&r)[8], uint32_t at)
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(at) : "memory");
}
__device__ __forceinline__ void st4(uint32_t at, const uint32_t (&r)[4])
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3])
                 : "memory");
}

__device__ __forceinline__ void load(uint32_t (&r)[32], uint32_t at) { ld32(r, at); }
__device__ __forceinline__ void load(uint32_t (&r)[16], uint32_t at) { ld16(r, at); }
__device__ __forceinline__ void store(uint32_t at, const uint32_t (&r)[32]) { st32(at, r); }
__device__ __forceinline__ void store(uint32_t at, const uint32_t (&r)[16]) { st16(at, r); }
__device__ __forceinline__ void store(uint32_t at, const uint32_t (&r)[8]) { st8(at, r); }

// ---- matrix products ------------------------------------------------------------
// Operand tiles in shared memory: panels of 64 16-bit values (128 bytes) a
// row, 1024-byte groups of 8 rows, the 16-byte chunks of a row xored with the
// row's number in its group (128-byte swizzle).  The same bytes are
//  - a K-major operand: rows are M or N, the 64 values lie along K;
//  - an MN-major operand: rows are K, the 64 values lie along M or N, panels
//    `panel` bytes apart continue M or N.
__device__ __forceinline__ uint64_t desc(uint32_t addr, uint32_t panel)
{
    return (uint64_t)((addr & 0x3ffff) >> 4) | ((uint64_t)(panel >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
           (1ull << 46) | (2ull << 61);
}
// Byte offset of 16-byte chunk c (of the whole row) of row r in such a tile.
__device__ __forceinline__ uint32_t chunk(uint32_t r, uint32_t c, uint32_t panel)
{
    return (c >> 3) * panel + r * 128 + (((c & 7) ^ (r & 7)) << 4);
}
// kind::f16 with fp32 accumulators, M = 128, N = n.
__device__ __forceinline__ uint32_t idesc(bool bf16, uint32_t n, bool a_mn, bool b_mn)
{
    return (1u << 4) | ((bf16 ? 1u : 0u) << 7) | ((bf16 ? 1u : 0u) << 10) | ((a_mn ? 1u : 0u) << 15) |
           ((b_mn ? 1u : 0u) << 16) | ((n >> 3) << 17) | ((128u >> 4) << 24);
}
// The products are issued by one lane of a warp whose lanes all run the issuing
// code: descriptors and addresses then stay in uniform registers, where the
// instruction wants them.  `off` (bytes, a multiple of 16) moves an operand's start.
__device__ __forceinline__ bool elect()
{
    uint32_t one;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(one));
    return one;
}
__device__ __forceinline__ void mma_ss(bool lead, uint32_t d, uint64_t a, uint32_t a_off, uint64_t b, uint32_t b_off, uint32_t id, bool add)
{
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %4, 0;\n\tsetp.ne.u32 q, %5, 0;\n\t"
                 "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
                 "l"(a + (a_off >> 4)), "l"(b + (b_off >> 4)), "r"(id), "r"((uint32_t)add), "r"((uint32_t)lead) : "memory");
}
__device__ __forceinline__ void mma_ts(bool lead, uint32_t d, uint32_t a, uint64_t b, uint32_t b_off, uint32_t id, bool add)
{
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %4, 0;\n\tsetp.ne.u32 q, %5, 0;\n\t"
                 "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
                 "r"(a), "l"(b + (b_off >> 4)), "r"(id), "r"((uint32_t)add), "r"((uint32_t)lead) : "memory");
}
// After a wait ran out: lets the products in flight end (at most 2^28 cycles) before tensor memory is freed.
__device__ __forceinline__ void commit(bool lead, uint64_t *b);
__device__ __forceinline__ void drain(bool lead, uint64_t *b, uint32_t parity)
{
    commit(lead, b);
    const long long start = clock64();
    while (!bar_peek(b, parity) && clock64() - start < (1ll << 28)) {}
}
// The leading lane's arrival on the barrier, when every product that it has issued so far is done.
__device__ __forceinline__ void commit(bool lead, uint64_t *b)
{
    if (lead) asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(saddr(b)) : "memory");
}

// A box of a tensor from shared memory (128-byte swizzle): what lies past the tensor's sides is left out.
__device__ __forceinline__ void store_box(const void *map, uint32_t from, int32_t x, int32_t y, int32_t z)
{
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(map), "r"(from), "r"(x),
                 "r"(y), "r"(z) : "memory");
}
__device__ __forceinline__ void stores_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
__device__ __forceinline__ void stores_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }   // sources free
__device__ __forceinline__ void stores_done() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

// Programmatic launches: the next kernel's blocks may be set up; the kernel before has ended and its writes are seen.
__device__ __forceinline__ void grid_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

}  // namespace tc
}  // namespace k2t
